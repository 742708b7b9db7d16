"""Sampling of the next token from its logits (moe_sample of
include/moe_model.h).  Argument marshalling only."""
from . import moe
from .attention import _on_gpu, _scope, _vector

_TYPES = {}  # torch dtype -> the library's code (filled on first use)


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, probs=None, stream=None):
    """One token a row of logits [rows, vocab] (bf16, fp16 or fp32; rows may
    be strided) from uniform numbers u float32 [rows] in [0, 1).  temperature
    float32, top_k int32, top_p float32 and min_p float32 hold one value a row;
    None leaves the step out (temperature 1).  Returns (tokens int32 [rows],
    probs float32 [rows]: the token's share of the kept mass); a row without a
    finite-or-greater logit gives token -1."""
    import torch
    if not _TYPES:
        _TYPES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    if logits.dim() != 2 or logits.shape[1] < 1:
        raise ValueError("logits must be [rows, vocab]")
    code = _TYPES.get(logits.dtype)
    if code is None:
        raise ValueError(f"logits: expected bfloat16, float16 or float32, got {logits.dtype}")
    rows, vocab = logits.shape
    if (vocab > 1 and logits.stride(1) != 1) or (rows > 1 and logits.stride(0) < vocab):
        raise ValueError("logits: rows must be contiguous and must not overlap")
    dev = _on_gpu(logits, "logits")
    f32, i32 = torch.float32, torch.int32
    ptrs = [_vector(u, "u", f32, rows, dev), _vector(temperature, "temperature", f32, rows, dev),
            _vector(top_k, "top_k", i32, rows, dev), _vector(top_p, "top_p", f32, rows, dev),
            _vector(min_p, "min_p", f32, rows, dev)]
    raw, scope = _scope(dev, stream)
    with scope:
        if tokens is None:
            tokens = torch.empty(rows, dtype=i32, device=dev)
        if probs is None:
            probs = torch.empty(rows, dtype=f32, device=dev)
        moe.check(moe.lib().moe_sample(logits.data_ptr(), code, rows, vocab, logits.stride(0) if rows > 1 else vocab, *ptrs,
                                       _vector(tokens, "tokens", i32, rows, dev), _vector(probs, "probs", f32, rows, dev),
                                       raw), "moe_sample")
    return tokens, probs
