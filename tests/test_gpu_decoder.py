"""The decoder's operators together, as decoding and training use them."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq, synth
from precision_transformer_gemms_gb300.head import LanguageHead
from test_gpu_moe import values

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Layer:
    """One decoder layer on 4-bit weights over a context of one token (its attention is
    the value itself), and the language head behind it."""

    def __init__(self, fmt, d=512, heads=8, kv=2, dim=64, experts=8, inter=256, vocab=1104, rank=8, adapters=3):
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")
        q = lambda n, k: lpq.quantize((r(n, k) / k ** 0.5).to(BF), fmt, lpq.ROWWISE).row
        self.d, self.heads, self.kv, self.dim, self.experts, self.vocab = d, heads, kv, dim, experts, vocab
        self.norms = [((1 + 0.1 * r(d)).to(BF), (0.1 * r(d)).to(BF)) for _ in range(2)]
        self.qkv, self.out = q((heads + 2 * kv) * dim, d), q(d, heads * dim)
        self.adapters = lpq.Adapters((r(adapters, rank, d) / d ** 0.5).to(BF), (0.3 * r(adapters, (heads + 2 * kv) * dim, rank)).to(BF),
                                     0.5 + torch.rand(adapters, generator=g, device="cuda"))
        self.qw, self.kw = (1 + 0.2 * r(dim)).to(BF), (1 + 0.2 * r(dim)).to(BF)
        self.router = (r(experts, d) / d ** 0.5).to(BF)
        self.up, self.down = q(experts * 2 * inter, d), q(experts * d, inter)
        self.head = LanguageHead((1 + 0.1 * r(d)).to(BF), (0.1 * r(d)).to(BF), (r(vocab, d) / d ** 0.5).to(BF)).freeze(fmt)

    def step(self, x, positions, index, controls):
        m, used = x.shape[0], (self.heads + self.kv) * self.dim
        h, _, _ = lpq.layer_norm(x, *self.norms[0])
        qkv = lpq.matvec(h, self.qkv, adapters=self.adapters, index=index)
        lpq.qk_norm_rope(qkv, self.heads, self.kv, self.dim, positions, self.qw, self.kw, out=qkv)
        attended = qkv[:, used:].view(m, self.kv, 1, self.dim).expand(-1, -1, self.heads // self.kv, -1).reshape(m, -1)
        x = x + lpq.matvec(attended, self.out)
        h, _, _ = lpq.layer_norm(x, *self.norms[1])
        ids, probs = lpq.moe_route(h, self.router, 2)
        x = x + lpq.moe(h, self.up, self.down, self.experts, ids, probs)
        return self.head.logits(x, controls=controls), qkv, ids

    def in_64_bits(self, x, positions, index, ids):
        """Queries and keys, and logits before the controls, from the definitions on the
        weights that the copies stand for; the experts are those that were chosen."""
        x, m, dim = x.double(), x.shape[0], self.dim
        norm = lambda v, w, b: torch.nn.functional.layer_norm(v, (self.d,), w.double(), b.double(), 1e-5)
        h = norm(x, *self.norms[0])
        qkv = h @ values(self.qkv).T
        a, b, s = (t.double() for t in (self.adapters.a, self.adapters.b, self.adapters.scale))
        for i, e in enumerate(index.tolist()):
            if e >= 0:
                qkv[i] += s[e] * (b[e] @ (a[e] @ h[i]))
        qkv = qkv.view(m, -1, dim)
        w = torch.cat((self.qw.double().expand(self.heads, dim), self.kw.double().expand(self.kv, dim)))
        qk = qkv[:, : self.heads + self.kv]
        qk = qk * (qk.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        f = torch.tensor([10000.0 ** (-2.0 * i / dim) for i in range(dim // 2)], device="cuda", dtype=torch.float64)
        turn = torch.polar(torch.ones(m, 1, dim // 2, device="cuda", dtype=torch.float64), (positions.double()[:, None] * f)[:, None])
        z = torch.complex(qk[..., : dim // 2].contiguous(), qk[..., dim // 2:].contiguous()) * turn
        attended = qkv[:, self.heads + self.kv:].repeat_interleave(self.heads // self.kv, 1).reshape(m, -1)
        x = x + attended @ values(self.out).T
        h = norm(x, *self.norms[1])
        probs = torch.softmax((h @ self.router.double().T).gather(1, ids), 1)
        up, down = values(self.up).view(self.experts, -1, self.d), values(self.down).view(self.experts, self.d, -1)
        y = torch.zeros_like(x)
        for i, row in enumerate(ids.tolist()):
            for j, e in enumerate(row):
                gate, lin = (up[e] @ h[i]).chunk(2)
                y[i] += probs[i, j] * (down[e] @ (torch.nn.functional.silu(gate) * lin))
        x = x + y
        return torch.cat((z.real, z.imag), -1).reshape(m, -1), norm(x, self.head.weight, self.head.bias) @ values(self.head.frozen).T


def request(layer, m, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(m, layer.d, generator=g, device="cuda").to(BF)
    positions = torch.randint(0, 100000, (m,), generator=g, device="cuda")
    index = torch.randint(-1, 3, (m,), generator=g, device="cuda")
    history = torch.randint(0, layer.vocab, (m, 50), generator=g, device="cuda")
    controls = dict(history=history, lengths=torch.randint(0, 51, (m,), generator=g, device="cuda"), repetition=1 + torch.rand(m, generator=g, device="cuda"),
                    frequency=torch.rand(m, generator=g, device="cuda"), presence=torch.rand(m, generator=g, device="cuda"),
                    allowed=torch.randint(-(1 << 31), 1 << 31, (m, (layer.vocab + 31) // 32), generator=g, device="cuda").int())
    return x, positions, index, controls


@pytest.mark.parametrize("fmt", [lpq.NVFP4, lpq.NVFP4_2D, lpq.MXFP4])
@pytest.mark.parametrize("m", [1, 6, 19])
def test_decoding_a_step(fmt, m):
    """Each stage's bf16 result is off by 2^-8 of its values at most; norms, turns and
    products with random weights keep the relative size of what comes in, a sum of two
    the larger one: 3 roundings up to the queries and keys, 11 up to the logits, in
    the 2-norm."""
    layer = Layer(fmt)
    x, positions, index, controls = request(layer, m)
    logits, qkv, ids = layer.step(x, positions, index, None)
    want_qk, want = layer.in_64_bits(x, positions, index, ids)
    used = want_qk.shape[1]
    assert (qkv[:, :used].double() - want_qk).norm() <= 3 * 2.0 ** -8 * want_qk.norm()
    assert (logits.double() - want).norm() <= 11 * 2.0 ** -8 * want.norm()
    assert torch.equal(layer.step(x, positions, index, controls)[0], lpq.adjust_logits(logits, **controls))


def test_a_step_captured_and_on_another_stream():
    layer = Layer(lpq.NVFP4)
    requests = [request(layer, 4, seed) for seed in range(3)]
    want = []
    for r in requests:
        want.append(layer.step(*r)[0])
        torch.cuda.synchronize()
    for _ in range(5):
        assert all(torch.equal(layer.step(*r)[0], w) for r, w in zip(requests, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = layer.step(*requests[1])[0]
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(other, want[1])
    x, positions, index, controls = (t.clone() if isinstance(t, torch.Tensor) else {k: v.clone() for k, v in t.items()} for t in requests[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits = layer.step(x, positions, index, controls)[0]
    for (a, b, c, d), w in zip(requests, want):
        x.copy_(a)
        positions.copy_(b)
        index.copy_(c)
        for k, v in d.items():
            controls[k].copy_(v)
        graph.replay()
        assert torch.equal(logits, w)


def test_training_through_the_projection():
    """QKV Fprop, head norm and rotation, their backward pass into the gradient that the
    projection's Dgrad and Wgrad read (bf16), against differentiation in 64 bits: the
    projection's and its gradient's rounding, and the results' own, 2^-8 each, the
    first entering through the norm's statistics, too."""
    t, d, heads, kv, dim = 320, 256, 4, 2, 64
    used, n = (heads + kv) * dim, (heads + 2 * kv) * dim
    x, w = synth.bf16_normal((t, d), 1.0, 0, "cuda"), synth.bf16_normal((n, d), 0.06, 1, "cuda")
    dy, dv = synth.bf16_normal((t, used), 1e-3, 2, "cuda"), synth.bf16_normal((t, n - used), 1e-3, 3, "cuda")
    qw, kw = (1 + 0.2 * torch.randn(dim, device="cuda")).to(BF), (1 + 0.2 * torch.randn(dim, device="cuda")).to(BF)
    positions = torch.arange(t, device="cuda") % 64
    both = lpq.ROWWISE | lpq.COLWISE
    qx, qweight = lpq.quantize(x, lpq.BF16, both), lpq.quantize(w, lpq.BF16, both)
    qkv = lpq.gemm(lpq.FPROP, qx.row, qweight.row)
    y = lpq.qk_norm_rope(qkv, heads, kv, dim, positions, qw, kw)
    dqkv = torch.empty_like(qkv)
    dqkv[:, used:] = dv
    _, dqw, dkw = lpq.qk_norm_rope_backward(dy, qkv, heads, kv, dim, positions, qw, kw, out=dqkv)
    qd = lpq.quantize(dqkv, lpq.BF16, both)
    dx, dw = lpq.gemm(lpq.DGRAD, qd.row, qweight.col), lpq.gemm(lpq.WGRAD, qd.col, qx.col)

    leaves = [v.double().requires_grad_() for v in (x, w, qw, kw)]
    full = leaves[0] @ leaves[1].T
    qk = full[:, :used].view(t, heads + kv, dim)
    qk = qk * (qk.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    qk = torch.cat((qk[:, :heads] * leaves[2], qk[:, heads:] * leaves[3]), 1)
    f = torch.tensor([10000.0 ** (-2.0 * i / dim) for i in range(dim // 2)], device="cuda", dtype=torch.float64)
    a = (positions.double()[:, None] * f)[:, None]
    lo, hi = qk[..., : dim // 2], qk[..., dim // 2:]
    want = torch.cat((lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()), -1).reshape(t, used)
    assert (y.double() - want).norm() <= 2 * 2.0 ** -8 * want.norm()
    grads = torch.autograd.grad((want * dy.double()).sum() + (full[:, used:] * dv.double()).sum(), leaves)
    for name, got, g in zip(("x", "w", "q_weight", "k_weight"), (dx, dw, dqw, dkw), grads):
        assert (got.double() - g).norm() <= 4 * 2.0 ** -8 * g.norm(), name
