"""Batches and caches for the GPU tests of the sequence-side operators."""
import numpy as np


def bf16(x):
    """float64 -> the nearest bf16's value (and what torch rounds it to)."""
    import torch
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def make_batch(news, lens, page, rng, extra_pages=3, pad_rows=0, wide=0, share=0):
    """Random distinct pages for each sequence.  Returns (KvBatch, table
    [n_seqs, max_pages], number of pages).  pad_rows: rows behind the last
    sequence; wide: unused table columns, filled with entries out of range;
    share: leading pages that all sequences have in common."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    need = [max(0, -(-n // page)) for n in lens]
    n_pages = sum(need) + extra_pages + share
    order = rng.permutation(n_pages)
    width = max(max(need), 1)
    table = np.full((len(lens), width + wide), 2 ** 30, np.int32)
    at = share
    for i, n in enumerate(need):
        table[i, :min(share, n)] = order[:min(share, n)]
        own = max(0, n - share)
        table[i, share:share + own] = order[at:at + own]
        at += own
    cu = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    b = attention.KvBatch(dev(table), dev(lens), dev(cu), int(cu[-1]) + pad_rows, max(1, max(news)))
    return b, table, n_pages


def whole(batch_table, lens):
    """A batch whose new tokens are all of the sequences' tokens."""
    import torch
    from quantized_expert_ffn_gemv_gb300 import attention
    cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    return attention.KvBatch(dev(batch_table), dev(lens), dev(cu), int(cu[-1]), max(1, max(lens)))


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)
