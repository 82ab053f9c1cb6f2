"""Calls on a stream other than the current one: their memory is that stream's,
and neither stream's pending work meets the other's."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq, synth

pytestmark = pytest.mark.gpu
T, D, V = 256, 512, 1024


def pool_of(t):
    """The stream whose pool the tensor's memory comes from."""
    p = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= p < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the caching allocator's memory")


@pytest.fixture(scope="module")
def data():
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    x, w = r(T, D), (0.05 * r(V, D)).bfloat16()
    _, mean, rstd = lpq.layer_norm(x)
    labels = torch.randint(0, V, (T,), generator=g, device="cuda")
    _, lse = lpq.linear_cross_entropy(x, w, labels)
    return dict(x=x, w=w, mean=mean, rstd=rstd, labels=labels, lse=lse, dloss=torch.ones(T, device="cuda"), weight=r(D), bias=r(D),
                q=lpq.quantize(w, lpq.NVFP4, lpq.ROWWISE).row, qx=lpq.quantize(x, lpq.NVFP4, lpq.ROWWISE).row)


CALLS = {
    "layer_norm": lambda d, **k: lpq.layer_norm(d["x"], d["weight"], d["bias"], **k),
    "layer_norm_backward": lambda d, **k: lpq.layer_norm_backward(d["x"], d["x"], d["mean"], d["rstd"], d["weight"], **k),
    "no_param_grads": lambda d, **k: lpq.layer_norm_backward(d["x"], d["x"], d["mean"], d["rstd"], param_grads=False, **k)[0],
    "linear_cross_entropy": lambda d, **k: lpq.linear_cross_entropy(d["x"], d["w"], d["labels"], **k),
    "linear_cross_entropy_backward": lambda d, **k: lpq.linear_cross_entropy_backward(d["x"], d["w"], d["labels"], d["lse"], d["dloss"], **k),
    "matvec": lambda d, **k: lpq.matvec(d["x"][:3], d["q"], **k),
    "quantize": lambda d, **k: lpq.quantize(d["x"], lpq.NVFP4, lpq.ROWWISE | lpq.COLWISE, **k),
    "amax": lambda d, **k: lpq.amax(d["x"], rht=True, **k),
    "gemm": lambda d, **k: lpq.gemm(lpq.FPROP, d["qx"], d["q"], **k),
}


@pytest.mark.parametrize("name", CALLS)
def test_results_come_from_the_streams_memory(data, name):
    want = list(lpq._tensors(CALLS[name](data)))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = list(lpq._tensors(CALLS[name](data, stream=s)))
    s.synchronize()
    assert len(got) == len(want) > 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)
        assert pool_of(a) == s.cuda_stream and pool_of(b) == torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("name", CALLS)
def test_the_current_streams_work_keeps_its_memory(data, name):
    """Blocks of the results' sizes, given back while work on them is pending: a call
    on another stream leaves them alone."""
    like = list(lpq._tensors(CALLS[name](data)))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(30_000_000)  # some 15 ms ahead of what follows
    kept = []
    for t in like:
        block = torch.full_like(t, 7)
        kept.append(block.clone())
        del block
    got = list(lpq._tensors(CALLS[name](data, stream=s)))
    s.synchronize()
    for a, b in zip(got, like):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    for k in kept:
        assert torch.equal(k, torch.full_like(k, 7))


@pytest.mark.parametrize("name", CALLS)
def test_results_outlive_the_callers_use(data, name):
    """Results used and dropped on the current stream: the other stream's next call
    does not write over them before that use."""
    want = list(lpq._tensors(CALLS[name](data)))
    x = synth.bf16_normal((T, D), 3.0, 5, "cuda")
    other = dict(data, x=x, qx=lpq.quantize(x, lpq.NVFP4, lpq.ROWWISE).row)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = CALLS[name](data, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(30_000_000)
    copies = [t.clone() for t in lpq._tensors(got)]
    del got
    for _ in range(3):
        CALLS[name](other, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b)
