"""Sampling of the next token from its logits (moe_sample of
include/moe_model.h).  Argument marshalling only."""
import torch

from . import moe
from .attention import _f32, _i32, _int32, _native, _on_gpu, _raw_stream, _scope, _vector

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, probs=None, stream=None):
    """One token a row of logits [rows, vocab] (bf16, fp16 or fp32; rows may
    be strided) from uniform numbers u float32 [rows] in [0, 1).  temperature
    float32, top_k int32, top_p float32 and min_p float32 hold one value a row;
    None leaves the step out (temperature 1).  Returns (tokens int32 [rows],
    probs float32 [rows]: the token's share of the kept mass, without a
    gradient); a row without a logit above -infinity gives token -1."""
    if stream is None:
        r = _native().sample(logits, u, temperature, top_k, top_p, min_p, tokens, probs)
        if r is not None:
            return r if type(r) is tuple else moe.check(r, "moe_sample")
    if logits.dim() != 2 or logits.shape[1] < 1:
        raise ValueError("logits must be [rows, vocab]")
    code = _TYPES.get(logits.dtype)
    if code is None:
        raise ValueError(f"logits: expected bfloat16, float16 or float32, got {logits.dtype}")
    rows, vocab = logits.shape
    _int32(rows=rows, vocab=vocab)
    stride, es = logits.stride()
    if rows <= 1:
        stride = vocab
    if (vocab > 1 and es != 1) or stride < vocab:
        raise ValueError("logits: rows must be contiguous and must not overlap")
    dev = _on_gpu(logits, "logits")
    scope = _scope(dev, stream)
    if scope is not None:
        with scope:
            return sample(logits, u, temperature, top_k, top_p, min_p, tokens, probs)
    if u is None:
        raise ValueError("u: one uniform number a row")
    if tokens is None:
        tokens = u.new_empty(rows, dtype=_i32)
    if probs is None:
        probs = u.new_empty(rows, dtype=_f32)
    status = moe.lib().moe_sample(
        logits.data_ptr(), code, rows, vocab, stride, _vector(u, "u", _f32, rows, dev),
        _vector(temperature, "temperature", _f32, rows, dev), _vector(top_k, "top_k", _i32, rows, dev),
        _vector(top_p, "top_p", _f32, rows, dev), _vector(min_p, "min_p", _f32, rows, dev),
        _vector(tokens, "tokens", _i32, rows, dev), _vector(probs, "probs", _f32, rows, dev), _raw_stream(dev))
    if status:
        moe.check(status, "moe_sample")
    return tokens, probs
