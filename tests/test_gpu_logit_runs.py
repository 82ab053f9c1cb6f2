"""Rows whose last run of words may begin behind their end, and words far outside the
vocabulary in contexts and biases, which count for nothing."""
import pytest
import torch

from precision_transformer_gemms_gb300 import lpq
from test_gpu_logits import BF, F32, check, make

pytestmark = pytest.mark.gpu


def foreign(words, v):
    """Every second one of `words` replaced by one that is not in the vocabulary."""
    far = [v, v + 1, v + 5000, 1 << 20, (1 << 31) - 1, -(1 << 31), 1 << 32, (1 << 32) + 3, -1, -2, -8, (1 << 63) - 1, -(1 << 63), 1 << 62]
    far = torch.tensor(far, device="cuda")
    flat = words.reshape(-1)
    flat[::2] = far[torch.arange(flat[::2].numel(), device="cuda") % len(far)]


def many(v):
    """Rows that make large runs of words."""
    return 152 * 2 * 4096 // v + 1


# residues of a run's words (FP32 1024, 4096 and 8192, bf16 2048, 4096 and 8192) just below a whole run; contexts
# from 2048 words on take the largest runs
CASES = [(dt, v, 2, 60) for dt, v in ((F32, 1022), (F32, 1023), (F32, 1024), (F32, 3070), (BF, 2042), (BF, 2045), (BF, 2047), (BF, 2048), (BF, 6143))]
CASES += [(dt, v, many(v), n) for dt, v in ((F32, 4094), (F32, 8191), (F32, 50174), (F32, 131070), (BF, 4090), (BF, 8186), (BF, 131071), (BF, 65530))
          for n in (60, 2100)]


@pytest.mark.parametrize("dt,v,t,n", CASES)
@pytest.mark.parametrize("lead", [0, 1, 3])
def test_words_outside_the_vocabulary(dt, v, t, n, lead):
    logits, c = make(t, v + lead, n, dt, seed=v + lead, biases=9)
    logits = logits[:, lead:]
    c["allowed"] = c["allowed"][:, : (v + 31) // 32]
    foreign(c["history"], v)
    foreign(c["bias"][1], v)
    out = torch.empty(t, v + lead, device="cuda", dtype=dt)[:, lead:]
    got = lpq.adjust_logits(logits, **c, out=out)
    few = list(range(min(t, 4))) + [t - 1] * (t > 4)  # rows that are compared one by one
    offsets, words, values = c["bias"]
    for i in few:
        row = {k: x[i:i + 1] for k, x in c.items() if k != "bias"}
        check(logits[i:i + 1], {**row, "bias": (offsets[i:i + 2], words, values)}, got[i:i + 1])
    # every row as if those words were not there
    for x in (c["history"], words):
        x[(x < 0) | (x >= v)] = -1
    assert torch.equal(lpq.adjust_logits(logits, **c), got)


@pytest.mark.parametrize("dt", [BF, F32])
def test_bias_offsets_of_any_size(dt):
    """Offsets are taken within the list: no bias where a row's begin beyond it or end before they begin."""
    top, v, t = (1 << 63) - 1, 700, 12
    logits, c = make(t, v, 20, dt, seed=3)
    words, values = torch.arange(100, device="cuda"), torch.linspace(1, 3, 100, device="cuda")
    offsets = [0, top, top - 5, top - 31, 40, -top - 1, 30, 1 << 32, 100, 101, -1, 3, top]
    c["bias"] = torch.tensor(offsets, device="cuda"), words, values
    got = lpq.adjust_logits(logits, **c)
    within = lambda n: min(max(n, 0), 100)
    for i in range(t):
        ends = [within(offsets[i]), max(within(offsets[i]), within(offsets[i + 1]))]
        row = {k: x[i:i + 1] for k, x in c.items() if k != "bias"}
        check(logits[i:i + 1], {**row, "bias": (torch.tensor(ends, device="cuda"), words, values)}, got[i:i + 1])
