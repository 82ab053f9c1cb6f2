"""The operators around a transformer's linear layers, as a user calls them, beside their plain forms.

Five operators take a model from its hidden states to the next token:

  norm       layer norm of the hidden states, with the row statistics its backward pass needs and
             the output's amax (what the quantizer of the next linear layer scales with)
  norm_grad  its backward pass: input gradient and the weight's and bias's gradients, summed over rows
  loss       softmax cross entropy of a vocabulary projection h w^T per token, logits not kept
  loss_grad  its gradient with respect to the hidden states and the projection's weights
  matvec     a linear layer of a few tokens on 4-bit weights with group scales (decoding)

`own` selects the implementation of run(): False is elementary torch arithmetic in 32 bits, rounded
once at the end; True is the library's kernels.  Sizes are those of this repository's workloads
(hidden 4096, intermediate 16384, 31 x 512 = 15,872 tokens, a 512 -> 384 small linear) or generic.
"""
import math

import torch

own = False

EPS = 1e-5
IGNORE = -100
NVFP4, NVFP4_2D, MXFP4 = "nvfp4", "nvfp4_2d", "mxfp4"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the norm before a linear layer while decoding one sequence: latency alone
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16"},
        # the norm before the QKV projection of a training step, feeding the NVFP4 quantizer
        {"name": "norm_layer", "op": "norm", "rows": 15872, "cols": 4096, "dtype": "bf16"},
        # a ragged batch of an odd-sized model held in fp32
        {"name": "norm_grad_odd", "op": "norm_grad", "rows": 509, "cols": 1023, "dtype": "fp32"},
        # the training step's backward pass through the norm
        {"name": "norm_grad_layer", "op": "norm_grad", "rows": 15872, "cols": 4096, "dtype": "bf16"},
        # the loss of one short sequence over a small vocabulary: latency
        {"name": "loss_small", "op": "loss", "rows": 33, "cols": 512, "vocab": 1009, "weighted": True},
        # evaluation of half a training batch over a subword vocabulary
        {"name": "loss_batch", "op": "loss", "rows": 7936, "cols": 4096, "vocab": 32000, "weighted": False},
        # the gradient of a ragged batch over an odd vocabulary, per-token weights
        {"name": "loss_grad_ragged", "op": "loss_grad", "rows": 1001, "cols": 1024, "vocab": 50001, "weighted": True},
        # the gradient of half a training batch (mean over the tokens that have a label)
        {"name": "loss_grad_batch", "op": "loss_grad", "rows": 7936, "cols": 4096, "vocab": 32000, "weighted": False},
        # one token through a small linear layer: latency
        {"name": "matvec_small", "op": "matvec", "tokens": 1, "rows": 384, "cols": 512, "fmt": NVFP4},
        # one token through the QKV projection
        {"name": "matvec_qkv", "op": "matvec", "tokens": 1, "rows": 12288, "cols": 4096, "fmt": NVFP4_2D},
        # two sequences decoded together through the MLP down projection
        {"name": "matvec_down", "op": "matvec", "tokens": 2, "rows": 4096, "cols": 16384, "fmt": MXFP4},
        # seven sequences decoded together through an odd vocabulary projection
        {"name": "matvec_vocab", "op": "matvec", "tokens": 7, "rows": 131073, "cols": 4096, "fmt": NVFP4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "loss", "loss_grad", "matvec"))
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            cols = (cols + 15) // 16 * 16
        rows = _log(rng, 1, max(2, min(20000, 15872 * 4096 // cols)))
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(("bf16", "bf16", "fp32"))}
    if op in ("loss", "loss_grad"):
        cols = 8 * _log(rng, 8, 512)
        vocab = _log(rng, 64, 131072)
        rows = _log(rng, 1, min(16384, 7936 * 4096 * 32000 // (cols * vocab)))
        return {"op": op, "rows": rows, "cols": cols, "vocab": vocab, "weighted": rng.random() < 0.5}
    cols = 32 * _log(rng, 4, 512)
    rows = _log(rng, 64, 131072 * 4096 // max(cols, 4096))
    return {"op": op, "tokens": _log(rng, 1, 16), "rows": rows, "cols": cols,
            "fmt": rng.choice((NVFP4, NVFP4_2D, MXFP4))}


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n, e, c = case["rows"] * case["cols"], (2 if case["dtype"] == "bf16" else 4), case["cols"]
        if op == "norm":  # x in, y out; weight and bias in; mean and rstd out
            return {"bytes": 2 * n * e + 2 * c * e + 8 * case["rows"] + 4, "flops": 8 * n}
        # dy and x in, dx out; weight in; both parameter gradients out in fp32; mean and rstd in
        return {"bytes": 3 * n * e + c * e + 8 * c + 8 * case["rows"], "flops": 14 * n}
    if op in ("loss", "loss_grad"):
        t, d, v = case["rows"], case["cols"], case["vocab"]
        if op == "loss":
            return {"bytes": 2 * (t + v) * d + 16 * t, "flops": 2 * t * d * v}
        # the logits again (they are not kept), then one product for each gradient
        return {"bytes": 4 * (t + v) * d + 16 * t, "flops": 6 * t * d * v}
    m, n, k = case["tokens"], case["rows"], case["cols"]
    return {"bytes": n * k // 2 + n * (k // (32 if case["fmt"] == MXFP4 else 16)) + 2 * m * (k + n), "flops": 2 * m * n * k}


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


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


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op in ("norm", "norm_grad"):
        t, c, dt = case["rows"], case["cols"], _dtype(case)
        # the residual stream: rows of different size and offset, a few outlying columns
        x = _randn(g, t, c) * (0.5 + 2.0 * torch.rand(t, 1, generator=g, device="cuda")) + 0.3 * _randn(g, t, 1)
        x[:, :: max(1, c // 4)] *= 20.0
        s = {"op": op, "x": x.to(dt), "weight": (1.0 + 0.1 * _randn(g, c)).to(dt)}
        if op == "norm":
            s["bias"] = (0.1 * _randn(g, c)).to(dt)
            return s
        x = s["x"].double()
        mean = x.mean(1)
        s["mean"] = mean.float()
        s["rstd"] = (x.sub_(mean[:, None]).square_().mean(1) + EPS).rsqrt().float()
        s["dy"] = (1e-3 * _randn(g, t, c)).to(dt)
        return s
    if op in ("loss", "loss_grad"):
        t, d, v = case["rows"], case["cols"], case["vocab"]
        w = (0.02 * _randn(g, v, d)).bfloat16()
        labels = torch.randint(0, v, (t,), generator=g, device="cuda")
        # hidden states that lean towards their label to different degrees, as during training
        pull = 8.0 * torch.rand(t, 1, generator=g, device="cuda")
        far = w.float()[labels]
        h = (_randn(g, t, d) + pull * far / far.norm(dim=1, keepdim=True)).bfloat16()
        labels[torch.rand(t, generator=g, device="cuda") < 0.05] = IGNORE  # padding and prompts
        s = {"op": op, "h": h, "w": w, "labels": labels}
        if op == "loss_grad":
            valid = labels != IGNORE
            weight = torch.rand(t, generator=g, device="cuda") if case["weighted"] else torch.ones(t, device="cuda")
            s["dloss"] = torch.where(valid, weight / valid.sum().clamp_min(1), 0.0)
            s["lse"] = torch.cat([torch.logsumexp(r.float() @ w.float().T, 1) for r in h.split(4096)])
        return s
    m, n, k, fmt = case["tokens"], case["rows"], case["cols"], case["fmt"]
    parts = [_quantize(0.02 * _randn(g, n, k), fmt)]
    codes, sf, ts = parts.pop()
    return {"op": op, "fmt": fmt, "rows": n, "cols": k, "x": _randn(g, m, k).bfloat16(), "codes": codes,
            "scales": _to_gemm_layout(sf, fmt), "tensor_scale": ts}


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


def _run_own(s):
    lpq, op = _lpq(), s["op"]
    if op == "norm":
        amax = torch.empty(1, dtype=torch.float32, device=s["x"].device)
        y, mean, rstd = lpq.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, amax=amax)
        return {"y": y, "mean": mean, "rstd": rstd, "amax": amax}
    if op == "norm_grad":
        dx, dweight, dbias = lpq.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op == "loss":
        loss, lse = lpq.linear_cross_entropy(s["h"], s["w"], s["labels"])
        return {"loss": loss, "lse": lse}
    if op == "loss_grad":
        dh, dw = lpq.linear_cross_entropy_backward(s["h"], s["w"], s["labels"], s["lse"], s["dloss"])
        return {"dh": dh, "dw": dw}
    fmt = {NVFP4: lpq.NVFP4, NVFP4_2D: lpq.NVFP4_2D, MXFP4: lpq.MXFP4}[s["fmt"]]
    w = lpq.Copy.of_parts(fmt, s["rows"], s["cols"], s["codes"], s["scales"], s["tensor_scale"])
    return lpq.matvec(s["x"], w)


def _run_plain(s):
    op = s["op"]
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        c = x - mean
        rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
        y = (c * rstd * s["weight"].float() + s["bias"].float()).to(s["x"].dtype)
        return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0], "amax": y.abs().amax().float().reshape(1)}
    if op == "norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        wdy = dy * s["weight"].float()
        dx = rstd * (wdy - wdy.mean(1, keepdim=True) - xhat * (wdy * xhat).mean(1, keepdim=True))
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}
    if op == "loss":
        logits = s["h"].float() @ s["w"].float().T
        top = logits.amax(1, keepdim=True)
        lse = (logits - top).exp().sum(1).log() + top[:, 0]
        valid = s["labels"] >= 0
        at = logits.gather(1, s["labels"].clamp_min(0)[:, None])[:, 0]
        return {"loss": torch.where(valid, lse - at, 0.0), "lse": lse}
    if op == "loss_grad":
        h, w = s["h"].float(), s["w"].float()
        d = h @ w.T
        d.sub_(s["lse"][:, None]).exp_()
        valid = s["labels"] >= 0
        d.scatter_add_(1, s["labels"].clamp_min(0)[:, None], -valid.float()[:, None])
        d.mul_(torch.where(valid, s["dloss"], 0.0)[:, None])
        return {"dh": (d @ w).bfloat16(), "dw": (d.T @ h).bfloat16()}
    codes, n, k = s["codes"], s["rows"], s["cols"]
    blk = 32 if s["fmt"] == MXFP4 else 16
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    w = table[torch.stack((codes & 15, codes >> 4), -1).int()].view(n, k // blk, blk)
    sf = _from_gemm_layout(s["scales"], n, k // blk)
    scale = torch.exp2(sf.float() - 127.0) if s["fmt"] == MXFP4 else sf.contiguous().view(torch.float8_e4m3fn).float()
    y = s["x"].float() @ (w * scale[..., None]).view(n, k).T
    return (y if s["tensor_scale"] is None else y * s["tensor_scale"]).bfloat16()


# ------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """run()'s outputs from the definitions in 64 bits: gradients by differentiating the definition."""
    if case["op"] == "loss_grad" and 6 * case["rows"] * case["cols"] * case["vocab"] > 8e12:
        return None
    s, op = prepare(case, seed), case["op"]
    if op in ("norm", "norm_grad"):
        x = s["x"].double().requires_grad_(op == "norm_grad")
        weight = s["weight"].double().requires_grad_(op == "norm_grad")
        bias = s["bias"].double() if op == "norm" else torch.zeros_like(weight, requires_grad=True)
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(bias, (x - mean) * rstd, weight)
        if op == "norm":
            return {"y": y, "mean": mean.flatten(), "rstd": rstd.flatten(), "amax": None}
        dx, dw, db = torch.autograd.grad(y, (x, weight, bias), s["dy"].double())
        return {"dx": dx, "dweight": dw, "dbias": db}
    if op in ("loss", "loss_grad"):
        h, w = (s[n].double().requires_grad_(op == "loss_grad") for n in ("h", "w"))
        valid = s["labels"] != IGNORE
        losses, lses, dh, dw = [], [], [], torch.zeros_like(w)
        for lo in range(0, case["rows"], 2048):
            rows = slice(lo, lo + 2048)
            part = h[rows].detach().requires_grad_(op == "loss_grad")
            logp = torch.log_softmax(torch.nn.functional.linear(part, w), dim=1)
            loss = torch.nn.functional.nll_loss(logp, s["labels"][rows], reduction="none", ignore_index=IGNORE)
            if op == "loss":
                losses.append(loss)
                lses.append((part * w[0]).sum(1) - logp[:, 0])
            else:
                got = torch.autograd.grad(torch.where(valid[rows], loss * s["dloss"][rows].double(), 0.0).sum(), (part, w))
                dh.append(got[0])
                dw += got[1]
        if op == "loss":
            return {"loss": torch.cat(losses), "lse": torch.cat(lses)}
        return {"dh": torch.cat(dh), "dw": dw}
    codes, fmt = s["codes"].long(), s["fmt"]
    low = torch.tensor([(-1 if c & 8 else 1) * E2M1[c & 7] for c in range(256)], device="cuda", dtype=torch.float64)
    high = torch.tensor([(-1 if c & 128 else 1) * E2M1[(c >> 4) & 7] for c in range(256)], device="cuda", dtype=torch.float64)
    blk = 32 if fmt == MXFP4 else 16
    sf = _from_gemm_layout(s["scales"], case["rows"], case["cols"] // blk).long()
    if fmt == MXFP4:
        values = torch.tensor([2.0 ** (c - 127) for c in range(256)], device="cuda", dtype=torch.float64)
    else:
        values = torch.tensor([(c & 7) * 2.0 ** -9 if c & 127 < 8 else (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10) for c in range(256)],
                              device="cuda", dtype=torch.float64) * s["tensor_scale"].double()
    scale = values[sf].repeat_interleave(blk // 2, 1)
    x = s["x"].double()
    y = [x[:, 0::2] @ (low[c] * f).T + x[:, 1::2] @ (high[c] * f).T for c, f in zip(codes.split(16384), scale.split(16384))]
    return torch.cat(y, 1)
