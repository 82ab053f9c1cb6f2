"""What a decoder layer on low-precision weights needs beside its linear layers, as a user calls it, beside its plain form.

Five operators; the first two serve training too:

  rotate       the norm of every query and key head behind the QKV projection with the position rotation
               in the same pass (RMS norm over the head, one weight for all query and one for all key heads)
  rotate_grad  its backward pass: the gradient of the projection's output and of the two weights
  adapted      a linear layer of a few tokens on 4-bit weights with a low-rank adapter for each request
  moe          a mixture-of-experts layer of a few tokens on 4-bit weights: router, the chosen experts'
               gated products, and their sum
  logits       penalties for repeated words, biases and a grammar's mask on the logits of the next words

`own` selects the implementation of run(): False is elementary torch arithmetic in 32 bits (angles and
the router's products in 64), rounded once at the end; True is the library's kernels.  Sizes are those
of this repository's workloads (hidden 4096, 32 heads, 31 x 512 = 15,872 tokens, QKV 4096 -> 12288, a
512 -> 384 small linear) or generic.
"""
import math

import torch

own = False

NVFP4, NVFP4_2D, MXFP4 = "nvfp4", "nvfp4_2d", "mxfp4"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token's queries and keys: latency alone
        {"name": "rotate_one_token", "op": "rotate", "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128,
         "base": 500000.0, "interleaved": False, "far": True, "dtype": "bf16"},
        # the layer's training step: 31 sequences of 512 tokens behind the QKV projection
        {"name": "rotate_layer", "op": "rotate", "tokens": 15872, "heads": 32, "kv_heads": 32, "dim": 128, "rotary": 128,
         "base": 10000.0, "interleaved": False, "far": False, "dtype": "bf16"},
        # an odd batch of a model held in fp32, neighbouring pairs turned, a part of each head not turned
        {"name": "rotate_grad_odd", "op": "rotate_grad", "tokens": 509, "heads": 6, "kv_heads": 2, "dim": 72, "rotary": 36,
         "base": 10000.0, "interleaved": True, "far": True, "dtype": "fp32"},
        # the training step's backward pass
        {"name": "rotate_grad_layer", "op": "rotate_grad", "tokens": 15872, "heads": 32, "kv_heads": 32, "dim": 128, "rotary": 128,
         "base": 10000.0, "interleaved": False, "far": False, "dtype": "bf16"},
        # one request through a small linear layer with an adapter of rank 8: latency
        {"name": "adapted_small", "op": "adapted", "tokens": 1, "rows": 384, "cols": 512, "rank": 8, "adapters": 3, "fmt": NVFP4},
        # eight requests with adapters of their own through the QKV projection
        {"name": "adapted_qkv", "op": "adapted", "tokens": 8, "rows": 12288, "cols": 4096, "rank": 16, "adapters": 32, "fmt": NVFP4_2D},
        # five requests, wide adapters, through the MLP down projection
        {"name": "adapted_down", "op": "adapted", "tokens": 5, "rows": 4096, "cols": 16384, "rank": 64, "adapters": 8, "fmt": MXFP4},
        # one token through a small layer of eight experts: latency
        {"name": "moe_small", "op": "moe", "tokens": 1, "hidden": 512, "inter": 384, "experts": 8, "top": 2, "fmt": NVFP4},
        # five tokens, sizes that no tile divides
        {"name": "moe_odd", "op": "moe", "tokens": 5, "hidden": 2080, "inter": 992, "experts": 21, "top": 3, "fmt": MXFP4},
        # eight requests decoded together through a layer of 64 experts
        {"name": "moe_batch", "op": "moe", "tokens": 8, "hidden": 4096, "inter": 1536, "experts": 64, "top": 8, "fmt": NVFP4},
        # the next word of one request
        {"name": "logits_one", "op": "logits", "rows": 1, "vocab": 32000, "history": 700, "dtype": "fp32"},
        # the next words of 64 requests with long contexts over an odd vocabulary
        {"name": "logits_batch", "op": "logits", "rows": 64, "vocab": 131073, "history": 8192, "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotate", "rotate_grad", "adapted", "moe", "logits"))
    if op in ("rotate", "rotate_grad"):
        dim = rng.choice((64, 80, 96, 128, 128, 192, 256, 2 * _log(rng, 8, 128)))
        rotary = dim if rng.random() < 0.6 else max(2, dim // 4 * 2)
        kv = _log(rng, 1, 32)
        heads = kv * rng.choice((1, 2, 4, 7, 8))
        tokens = _log(rng, 1, max(2, min(20000, 15872 * 8192 // ((heads + kv) * dim))))
        return {"op": op, "tokens": tokens, "heads": heads, "kv_heads": kv, "dim": dim, "rotary": rotary,
                "base": rng.choice((10000.0, 500000.0)), "interleaved": rng.random() < 0.3, "far": rng.random() < 0.5,
                "dtype": rng.choice(("bf16", "bf16", "fp32")) if tokens < 8000 else "bf16"}
    if op == "adapted":
        cols = 32 * _log(rng, 4, 512)
        rows = _log(rng, 64, 16384 * 4096 // max(cols, 4096))
        return {"op": op, "tokens": _log(rng, 1, 24), "rows": rows, "cols": cols, "rank": rng.choice((8, 16, 16, 32, 40, 64)),
                "adapters": _log(rng, 1, 32), "fmt": rng.choice((NVFP4, NVFP4_2D, MXFP4))}
    if op == "moe":
        experts = _log(rng, 4, 64)
        hidden, inter = 32 * _log(rng, 4, 128), 32 * _log(rng, 2, 48)
        top = rng.randint(1, min(8, experts))
        return {"op": op, "tokens": _log(rng, 1, max(2, 64 // top)), "hidden": hidden, "inter": inter, "experts": experts, "top": top,
                "fmt": rng.choice((NVFP4, NVFP4_2D, MXFP4))}
    vocab = _log(rng, 500, 200000)
    rows = _log(rng, 1, max(2, min(256, 64 * 131073 // vocab)))
    return {"op": op, "rows": rows, "vocab": vocab, "history": _log(rng, 1, 8192), "dtype": rng.choice(("fp32", "fp32", "bf16"))}


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def work(case):
    op = case["op"]
    if op in ("rotate", "rotate_grad"):
        n, e = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"], 2 if case["dtype"] == "bf16" else 4
        if op == "rotate":  # queries and keys in and out, the two weights and the positions in
            return {"bytes": 2 * n * e + 2 * case["dim"] * e + 8 * case["tokens"], "flops": 7 * n}
        # gradients and inputs in, input gradients out; the weights in, their gradients out in fp32
        return {"bytes": 3 * n * e + 2 * case["dim"] * (e + 4) + 8 * case["tokens"], "flops": 14 * n}
    if op == "adapted":
        m, n, k, r = case["tokens"], case["rows"], case["cols"], case["rank"]
        used = case["adapters"] * (1.0 - (1.0 - 0.9 / case["adapters"]) ** m)  # adapters that some request has
        weights = n * k // 2 + n * (k // (32 if case["fmt"] == MXFP4 else 16))
        return {"bytes": int(weights + used * 2 * r * (n + k)) + 2 * m * (k + n), "flops": 2 * m * (n * k + r * (n + k))}
    if op == "moe":
        m, d, f, e, top = (case[n] for n in ("tokens", "hidden", "inter", "experts", "top"))
        used = e * (1.0 - (1.0 - top / e) ** m)  # experts that some token has chosen
        values = 3 * d * f
        return {"bytes": int(used * (values // 2 + values // (32 if case["fmt"] == MXFP4 else 16))) + 2 * e * d + 4 * m * d + 12 * m * top,
                "flops": 2 * m * (top * values + e * d)}
    t, v, e = case["rows"], case["vocab"], 2 if case["dtype"] == "bf16" else 4
    return {"bytes": 2 * t * v * e + t * (-(-v // 32) * 4 + 4 * case["history"]), "flops": 6 * t * v}


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _quantize(w, fmt):
    """fp32 [N, K] -> packed E2M1 codes [N, K/2], u8 block scales [N, K/block], fp32 tensor scale or None."""
    n, k = w.shape
    blk = 32 if fmt == MXFP4 else 16
    b = w.view(n, k // blk, blk)
    top = b.abs().amax(-1)
    if fmt == MXFP4:
        e = torch.ceil(torch.log2((top / 6.0).clamp_min(1e-30))).clamp(-127, 127)
        sf, step, ts = (e + 127).to(torch.uint8), torch.exp2(e), None
    else:
        if fmt == NVFP4_2D:  # one scale for 16 x 16 values
            pad = -n % 16
            t = torch.nn.functional.pad(top, (0, 0, 0, pad)).view((n + pad) // 16, 16, k // 16).amax(1, keepdim=True)
            top = t.expand(-1, 16, -1).reshape(n + pad, k // 16)[:n]
        ts = (w.abs().amax() / 2688.0).reshape(1)
        s8 = (top / (6.0 * ts)).to(torch.float8_e4m3fn)
        sf, step = s8.view(torch.uint8), s8.float() * ts
    mag = (b / step.unsqueeze(-1).clamp_min(1e-30)).abs_()
    code = torch.bucketize(mag, torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device="cuda"), out_int32=True).to(torch.uint8)
    code = (code | ((b < 0).to(torch.uint8) << 3)).view(n, k // 2, 2)
    return (code[..., 0] | (code[..., 1] << 4)).contiguous(), sf, ts


def _to_gemm_layout(sf, fmt):
    """[N, blocks] scales -> the tensor-core layout the GEMM and the quantizer use: 128-row groups of
    512-byte atoms, row 32 j + i of a group keeping 4 consecutive blocks at bytes 16 i + 4 j."""
    n, nb = sf.shape
    per = 8 if fmt == MXFP4 else 16
    groups, atoms = -(-n // 128), -(-nb // per) * (per // 4)
    full = torch.zeros((groups * 128, atoms * 4), dtype=torch.uint8, device="cuda")
    full[:n, :nb] = sf
    return full.view(groups, 4, 32, atoms, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _from_gemm_layout(sf, n, nb):
    groups = -(-n // 128)
    return sf.view(groups, -1, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(groups * 128, -1)[:n, :nb]


def _weights(g, n, k, std, fmt):
    codes, sf, ts = _quantize(std * _randn(g, n, k), fmt)
    return {"rows": n, "cols": k, "codes": codes, "scales": _to_gemm_layout(sf, fmt), "tensor_scale": ts}


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op in ("rotate", "rotate_grad"):
        t, hq, hk, d, dt = case["tokens"], case["heads"], case["kv_heads"], case["dim"], _dtype(case)
        # what the QKV projection leaves: heads of different size, a few outlying columns; values behind the keys
        qkv = _randn(g, t, hq + 2 * hk, d) * (0.2 + 3.0 * _rand(g, 1, hq + 2 * hk, 1)) * (0.5 + _rand(g, t, 1, 1))
        qkv[:, :, 3:: max(4, d // 2)] *= 8.0
        # sequences of 512 from their first token, or each token anywhere in a long context
        positions = torch.randint(0, 1 << 20, (t,), generator=g, device="cuda") if case["far"] else torch.arange(t, device="cuda") % 512
        s = {"op": op, "qkv": qkv.view(t, -1).to(dt), "heads": hq, "kv_heads": hk, "dim": d, "rotary": case["rotary"], "base": case["base"],
             "interleaved": case["interleaved"], "positions": positions, "q_weight": (1.0 + 0.2 * _randn(g, d)).to(dt),
             "k_weight": (1.0 + 0.2 * _randn(g, d)).to(dt)}
        if op == "rotate_grad":
            s["dy"] = (1e-3 * _randn(g, t, (hq + hk) * d)).to(dt)
        return s
    if op == "adapted":
        m, n, k, r, count, fmt = (case[v] for v in ("tokens", "rows", "cols", "rank", "adapters", "fmt"))
        index = torch.randint(0, count, (m,), generator=g, device="cuda")
        index[_rand(g, m) < 0.1] = -1  # a request without an adapter
        return {"op": op, "fmt": fmt, "w": _weights(g, n, k, 0.02, fmt), "x": _randn(g, m, k).bfloat16(),
                "a": (_randn(g, count, r, k) / math.sqrt(k)).bfloat16(), "b": (0.3 * _randn(g, count, n, r)).bfloat16(),
                "scale": 0.5 + _rand(g, count), "index": index}
    if op == "moe":
        m, d, f, e, fmt = (case[v] for v in ("tokens", "hidden", "inter", "experts", "fmt"))
        return {"op": op, "fmt": fmt, "experts": e, "top": case["top"], "x": _randn(g, m, d).bfloat16(),
                "router": (_randn(g, e, d) / math.sqrt(d)).bfloat16(), "up": _weights(g, e * 2 * f, d, 0.02, fmt),
                "down": _weights(g, e * d, f, 0.02, fmt)}
    t, v, n = case["rows"], case["vocab"], case["history"]
    logits = (4.0 * _randn(g, t, v)).to(_dtype(case))
    # words as texts repeat them: few often, many once; contexts of different length, part prompt and part answer
    history = (v * _rand(g, t, n) ** 4).long().clamp_max(v - 1)
    lengths = (_rand(g, t) * (n + 1)).long().clamp_max(n)
    lengths[0] = n
    prompt = (_rand(g, t) * (lengths + 1)).long().minimum(lengths)
    # half of the requests are free, the others may take a sixteenth of the words
    words = torch.randint(-(1 << 31), 1 << 31, (4, t, -(-v // 32)), generator=g, device="cuda")
    allowed = words[0] & words[1] & words[2] & words[3]
    allowed[0::2] = -1
    each = 8  # biased words of a request
    return {"op": op, "logits": logits, "history": history, "lengths": lengths, "prompt": prompt, "repetition": 1.0 + 0.3 * _rand(g, t),
            "frequency": 0.5 * _rand(g, t), "presence": 0.5 * _rand(g, t), "bias_offsets": each * torch.arange(t + 1, device="cuda"),
            "bias_words": torch.rand(t, v, generator=g, device="cuda").topk(each, 1).indices.reshape(-1), "bias_values": 5.0 * _randn(g, t * each),
            "allowed": allowed.int()}


# ------------------------------------------------------------------------------------------ one pass
_lib = None


def _lpq():
    global _lib
    if _lib is None:
        from precision_transformer_gemms_gb300 import lpq
        _lib = lpq
    return _lib


def run(state):
    return (_run_own if own else _run_plain)(state)


def _copy(lpq, w, fmt):
    fmt = {NVFP4: lpq.NVFP4, NVFP4_2D: lpq.NVFP4_2D, MXFP4: lpq.MXFP4}[fmt]
    return lpq.Copy.of_parts(fmt, w["rows"], w["cols"], w["codes"], w["scales"], w["tensor_scale"])


def _run_own(s):
    lpq, op = _lpq(), s["op"]
    if op == "rotate":
        return lpq.qk_norm_rope(s["qkv"], s["heads"], s["kv_heads"], s["dim"], s["positions"], s["q_weight"], s["k_weight"],
                                rotary_dim=s["rotary"], base=s["base"], interleaved=s["interleaved"], eps=EPS)
    if op == "rotate_grad":
        dx, dq, dk = lpq.qk_norm_rope_backward(s["dy"], s["qkv"], s["heads"], s["kv_heads"], s["dim"], s["positions"], s["q_weight"],
                                               s["k_weight"], rotary_dim=s["rotary"], base=s["base"], interleaved=s["interleaved"], eps=EPS)
        return {"dx": dx, "dq_weight": dq, "dk_weight": dk}
    if op == "adapted":
        adapters = lpq.Adapters(s["a"], s["b"], s["scale"])
        return lpq.matvec(s["x"], _copy(lpq, s["w"], s["fmt"]), adapters=adapters, index=s["index"])
    if op == "moe":
        ids, probs = lpq.moe_route(s["x"], s["router"], s["top"])
        y = lpq.moe(s["x"], _copy(lpq, s["up"], s["fmt"]), _copy(lpq, s["down"], s["fmt"]), s["experts"], ids, probs)
        return {"y": y, "ids": ids, "probs": probs}
    return lpq.adjust_logits(s["logits"], history=s["history"], lengths=s["lengths"], prompt=s["prompt"], repetition=s["repetition"],
                             frequency=s["frequency"], presence=s["presence"], bias=(s["bias_offsets"], s["bias_words"], s["bias_values"]),
                             allowed=s["allowed"])


def _angles(s):
    """cos and sin [t, 1, rotary / 2] of every position and pair, fp32 of angles in 64 bits."""
    r = s["rotary"]
    freqs = float(s["base"]) ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
    angle = s["positions"].double()[:, None, None] * freqs
    return angle.cos().float(), angle.sin().float()


def _turn(s, v, cos, sin):
    """The first `rotary` values of every head turned by the angles, the others as they are."""
    r = s["rotary"]
    if s["interleaved"]:
        a, b = v[..., 0:r:2], v[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = v[..., : r // 2], v[..., r // 2: r]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, v[..., r:]), -1)


def _dequantize(codes, sf, fmt):
    """fp32 values [..., K] of packed codes [..., K/2] and block scales [..., K/block]."""
    blk = 32 if fmt == MXFP4 else 16
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    w = table[torch.stack((codes & 15, codes >> 4), -1).int()].view(*codes.shape[:-1], -1, blk)
    scale = torch.exp2(sf.float() - 127.0) if fmt == MXFP4 else sf.contiguous().view(torch.float8_e4m3fn).float()
    return (w * scale[..., None]).flatten(-2)


def _plain_scales(w, fmt):
    return _from_gemm_layout(w["scales"], w["rows"], w["cols"] // (32 if fmt == MXFP4 else 16))


def _run_plain(s):
    op = s["op"]
    if op in ("rotate", "rotate_grad"):
        hq, hk, d, dt = s["heads"], s["kv_heads"], s["dim"], s["qkv"].dtype
        t = s["positions"].shape[0]
        x = s["qkv"].view(t, hq + 2 * hk, d)[:, : hq + hk].float()
        w = torch.cat((s["q_weight"].float().expand(hq, d), s["k_weight"].float().expand(hk, d)))
        rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        cos, sin = _angles(s)
        if op == "rotate":
            return _turn(s, x * rstd * w, cos, sin).to(dt).view(t, -1)
        g = _turn(s, s["dy"].view(t, hq + hk, d).float(), cos, -sin)
        xhat = x * rstd
        dw = (g * xhat).sum(0)
        g = g * w
        dx = rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))
        return {"dx": dx.to(dt).view(t, -1), "dq_weight": dw[:hq].sum(0), "dk_weight": dw[hq:].sum(0)}
    if op == "adapted":
        x, has = s["x"].float(), s["index"] >= 0
        y = x @ _dequantize(s["w"]["codes"], _plain_scales(s["w"], s["fmt"]), s["fmt"]).T
        if s["w"]["tensor_scale"] is not None:
            y = y * s["w"]["tensor_scale"]
        at = s["index"].clamp_min(0)
        inner = s["a"][at].float() @ x[:, :, None]
        outer = (s["b"][at].float() @ inner)[:, :, 0] * s["scale"][at][:, None]
        return (y + torch.where(has[:, None], outer, 0.0)).bfloat16()
    if op == "moe":
        e, top, fmt, m = s["experts"], s["top"], s["fmt"], s["x"].shape[0]
        scores = s["x"].double() @ s["router"].double().T  # (which experts are largest depends on the last bits)
        best, ids = torch.sort(scores, dim=1, descending=True, stable=True)
        ids, best = ids[:, :top].contiguous(), best[:, :top].float()
        probs = (best - best[:, :1]).exp()
        probs = probs / probs.sum(1, keepdim=True)
        up, down = s["up"], s["down"]

        def chosen(w):
            w4 = _dequantize(w["codes"].view(e, -1, w["cols"] // 2)[ids], _plain_scales(w, fmt).reshape(e, w["rows"] // e, -1)[ids], fmt)
            return w4 if w["tensor_scale"] is None else w4 * w["tensor_scale"]

        gu = (chosen(up) @ s["x"].float()[:, None, :, None])[..., 0]
        gate, lin = gu.chunk(2, -1)
        h = gate / (1.0 + (-gate).exp()) * lin
        y = (chosen(down) @ h[..., None])[..., 0]
        return {"y": (y * probs[:, :, None]).sum(1).bfloat16(), "ids": ids, "probs": probs}
    x, (t, v) = s["logits"].float(), s["logits"].shape
    at, n = torch.arange(s["history"].shape[1], device="cuda")[None], s["lengths"][:, None]
    spot = s["history"] + v * torch.arange(t, device="cuda")[:, None]
    counts = lambda mask: torch.zeros(t * v, device="cuda").scatter_add_(0, spot.reshape(-1), mask.float().reshape(-1)).view(t, v)  # noqa: E731
    said, answered = counts(at < n), counts((at >= s["prompt"][:, None]) & (at < n))
    rep = s["repetition"][:, None]
    x = torch.where(said > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * answered - s["presence"][:, None] * (answered > 0)
    row = torch.repeat_interleave(torch.arange(t, device="cuda"), s["bias_offsets"].diff(), output_size=s["bias_words"].shape[0])
    x = x.reshape(-1).scatter_add(0, row * v + s["bias_words"], s["bias_values"]).view(t, v)
    bits = (s["allowed"][:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    return torch.where(bits.view(t, -1)[:, :v] > 0, x, -math.inf).to(s["logits"].dtype)


# ------------------------------------------------------------------------------------------ in 64 bits
def _exact_weights(w, fmt, rows=slice(None)):
    """Rows of a weight matrix from its codes, scales and tensor scale, by tables of what each byte stands for."""
    codes = w["codes"][rows].long()
    low = torch.tensor([(-1 if c & 8 else 1) * E2M1[c & 7] for c in range(256)], device="cuda", dtype=torch.float64)
    high = torch.tensor([(-1 if c & 128 else 1) * E2M1[(c >> 4) & 7] for c in range(256)], device="cuda", dtype=torch.float64)
    blk = 32 if fmt == MXFP4 else 16
    sf = _from_gemm_layout(w["scales"], w["rows"], w["cols"] // blk)[rows].long()
    if fmt == MXFP4:
        values = torch.tensor([2.0 ** (c - 127) for c in range(256)], device="cuda", dtype=torch.float64)
    else:
        values = torch.tensor([(c & 7) * 2.0 ** -9 if c & 127 < 8 else (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10) for c in range(256)],
                              device="cuda", dtype=torch.float64) * w["tensor_scale"].double()
    both = torch.stack((low[codes], high[codes]), -1).view(codes.shape[0], -1, blk)
    return (both * values[sf][..., None]).flatten(1)


def exact(case, seed):
    """run()'s outputs from the definitions in 64 bits: rotations as complex products, gradients by differentiating the definition."""
    s, op = prepare(case, seed), case["op"]
    if op in ("rotate", "rotate_grad"):
        hq, hk, d, r = s["heads"], s["kv_heads"], s["dim"], s["rotary"]
        freqs = torch.tensor([float(s["base"]) ** (-2.0 * i / r) for i in range(r // 2)], device="cuda", dtype=torch.float64)
        grad = op == "rotate_grad"
        qw, kw = (s[n].double().requires_grad_(grad) for n in ("q_weight", "k_weight"))
        out, dq, dk = [], torch.zeros_like(qw), torch.zeros_like(kw)
        for rows in torch.arange(case["tokens"], device="cuda").split(2048):
            angle = s["positions"][rows].double()[:, None] * freqs
            spin = torch.polar(torch.ones_like(angle), angle)[:, None]
            x = s["qkv"][rows][:, : (hq + hk) * d].double().requires_grad_(grad)
            heads = x.view(-1, hq + hk, d)
            normed = heads * (heads.square().sum(-1, keepdim=True) / d + EPS).rsqrt()
            normed = torch.cat((normed[:, :hq] * qw, normed[:, hq:] * kw), 1)
            if s["interleaved"]:
                turned = torch.view_as_real(torch.view_as_complex(normed[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * spin).flatten(-2)
            else:
                z = torch.complex(normed[..., : r // 2], normed[..., r // 2: r]) * spin
                turned = torch.cat((z.real, z.imag), -1)
            y = torch.cat((turned, normed[..., r:]), -1).flatten(1)
            if grad:
                got = torch.autograd.grad(y, (x, qw, kw), s["dy"][rows].double())
                out.append(got[0])
                dq += got[1]
                dk += got[2]
            else:
                out.append(y)
        return {"dx": torch.cat(out), "dq_weight": dq.detach(), "dk_weight": dk.detach()} if grad else torch.cat(out)
    if op == "adapted":
        x, fmt = s["x"].double(), s["fmt"]
        y = torch.cat([torch.nn.functional.linear(x, _exact_weights(s["w"], fmt, slice(lo, lo + 4096))) for lo in range(0, case["rows"], 4096)], 1)
        for i, which in enumerate(s["index"].tolist()):
            if which >= 0:
                y[i] += s["scale"][which].double() * torch.mv(s["b"][which].double(), torch.mv(s["a"][which].double(), x[i]))
        return y
    if op == "moe":
        x, fmt, f, d = s["x"].double(), s["fmt"], case["inter"], case["hidden"]
        scores = torch.nn.functional.linear(x, s["router"].double()).cpu()
        y = torch.zeros_like(x)
        ids = [sorted(range(case["experts"]), key=lambda e: (-row[e], e))[: case["top"]] for row in scores.tolist()]
        probs = torch.stack([torch.softmax(row[chosen], 0) for row, chosen in zip(scores, ids)]).cuda()
        for which in sorted(set(sum(ids, []))):
            up = _exact_weights(s["up"], fmt, slice(which * 2 * f, (which + 1) * 2 * f))
            down = _exact_weights(s["down"], fmt, slice(which * d, (which + 1) * d))
            for i, chosen in enumerate(ids):
                if which in chosen:
                    gate, lin = torch.mv(up, x[i]).split(f)
                    y[i] += probs[i, chosen.index(which)] * torch.mv(down, torch.nn.functional.silu(gate) * lin)
        return {"y": y, "ids": torch.tensor(ids, device="cuda"), "probs": probs}
    x, v = s["logits"].double(), case["vocab"]
    starts, words, values = s["bias_offsets"].tolist(), s["bias_words"], s["bias_values"].double()
    for i, (n, p) in enumerate(zip(s["lengths"].tolist(), s["prompt"].tolist())):
        row = x[i]
        seen = torch.unique(s["history"][i, :n])
        was = row[seen]
        row[seen] = torch.where(was > 0, was / s["repetition"][i].double(), was * s["repetition"][i].double())
        back, times = torch.unique(s["history"][i, p:n], return_counts=True)
        row[back] -= s["frequency"][i].double() * times + s["presence"][i].double()
        here = slice(starts[i], starts[i + 1])
        row.index_add_(0, words[here], values[here])
        bits = s["allowed"][i].cpu().numpy().view("uint8")
        import numpy as np
        row[torch.from_numpy(np.unpackbits(bits, bitorder="little")[:v] == 0).cuda()] = -math.inf
    return x
