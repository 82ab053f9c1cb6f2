"""A language model's head on liblpq: the final layer norm, the vocabulary
projection with its loss and gradients for training, and the same projection
on 4-bit weights for decoding.

Every step runs in liblpq's kernels; torch supplies memory, the per-token
weights of the mean loss and the caller's optimizer.
"""
import torch

from . import lpq


class LanguageHead:
    """Final norm (weight, bias [d]) and vocabulary weights w [v, d] (bf16).

    Training: ``loss, saved = head.loss(x, labels)`` and ``head.backward(saved)``.
    Decoding: ``head.freeze()`` once, then ``head.logits(x)`` for the few tokens
    of a step or ``head.prompt_logits(x)`` for the many of a prompt.

    With ``stream=s`` a call runs on s from its first to its last step and takes
    all its memory there (lpq.on_stream).
    """

    def __init__(self, weight, bias, w, eps=1e-5):
        assert w.dtype == torch.bfloat16 and w.dim() == 2 and weight.numel() == w.shape[1]
        self.weight, self.bias, self.w, self.eps = weight, bias, w, eps
        self.frozen = None

    def loss(self, x, labels, stream=None):
        """Mean cross entropy of the hidden states x [t, d] (bf16) over the rows
        whose label is a word (0 .. v - 1); returns (loss, saved)."""
        if stream is not None:
            return lpq.on_stream(stream, self.loss, x, labels)
        h, mean, rstd = lpq.layer_norm(x, self.weight, self.bias, eps=self.eps)
        losses, lse = lpq.linear_cross_entropy(h, self.w, labels)
        valid = (labels >= 0) & (labels < self.w.shape[0])
        dloss = valid / valid.sum().clamp_min(1)
        return (losses * dloss).sum(), (x, h, mean, rstd, labels, lse, dloss)

    def backward(self, saved, stream=None):
        """Gradients of the mean loss: {"x", "weight", "bias", "w"}."""
        if stream is not None:
            return lpq.on_stream(stream, self.backward, saved)
        x, h, mean, rstd, labels, lse, dloss = saved
        dh, dw = lpq.linear_cross_entropy_backward(h, self.w, labels, lse, dloss)
        dx, dweight, dbias = lpq.layer_norm_backward(dh, x, mean, rstd, self.weight)
        return {"x": dx, "weight": dweight, "bias": dbias, "w": dw}

    def freeze(self, fmt=lpq.NVFP4, stream=None):
        """Quantizes the vocabulary weights for decoding (NVFP4, NVFP4_2D or MXFP4)."""
        freeze = lambda: lpq.quantize(self.w.contiguous(), fmt, lpq.ROWWISE).row
        self.frozen = freeze() if stream is None else lpq.on_stream(stream, freeze)
        return self

    def logits(self, x, stream=None, controls=None):
        """FP32 logits [t, v] of a few hidden states x [t, d] on the frozen
        weights; the activations stay bf16.  `controls`: keywords of
        lpq.adjust_logits (penalties, biases, mask), applied in place."""
        if stream is not None:
            return lpq.on_stream(stream, self.logits, x, controls=controls)
        assert self.frozen is not None, "freeze() the head first"
        h, _, _ = lpq.layer_norm(x, self.weight, self.bias, eps=self.eps)
        logits = lpq.matvec(h, self.frozen, out_fp32=True)
        return logits if controls is None else lpq.adjust_logits(logits, **controls, out=logits)

    def prompt_logits(self, x, stream=None):
        """FP32 logits of many hidden states on the frozen weights through the
        block-scaled GEMM, the states in NVFP4 (MXFP4 on MXFP4 weights).  The norm's
        amax scales the NVFP4 quantizer, which then runs without an amax pass of its
        own."""
        if stream is not None:
            return lpq.on_stream(stream, self.prompt_logits, x)
        assert self.frozen is not None, "freeze() the head first"
        fmt, flags = (lpq.MXFP4, lpq.ROWWISE) if self.frozen.fmt == lpq.MXFP4 else (lpq.NVFP4, lpq.ROWWISE | lpq.GIVEN_AMAX)
        q = lpq.alloc(fmt, x.shape[0], x.shape[1], lpq.ROWWISE, device=x.device)
        h, _, _ = lpq.layer_norm(x, self.weight, self.bias, eps=self.eps, amax=q.row.amax)  # (MXFP4 has none)
        lpq.quantize(h, fmt, flags, out=q)
        return lpq.gemm(lpq.FPROP, q.row, self.frozen, out_fp32=True)
