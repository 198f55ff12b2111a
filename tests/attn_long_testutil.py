"""Tolerances of attention over the cache in parts or over selected pages.

As in attn_testutil, with A = sum_j p_j |v_j| and M = the largest scale sum_i |q_i k_i| of a row:
* scores are sums of d fp32 terms: off by at most (d + 8) 2^-23 M, which moves a weight by that much, twice;
* weights: e^x to 2^-21, then fp16 operands: 2^-11, or 2^-21 as two terms (fp32 inputs); sums over the keys in
  blocks and parts: 2^-17 of A bounds them for the lengths used here;
* the output's own half step, eps / 2 of its type.

Shared prefixes in bf16 at d = 64 and 128: a query is two e4m3 terms of the row scaled so that its largest element
is in 2^7..2^8.  An element of 2^k..2^(k+1), 8 bits, is a multiple of 2^(k-7); the first term (4 bits) leaves at
most 2^(k-4) of it, a multiple of 2^(k-7) again, which 4 bits hold where 2^(k-7) is no less than e4m3's smallest
step, 2^-9.  Below that the rest is off by half that step, 2^-10, which is 2^-17 of the row's largest element: a
score is off by at most 2^-17 scale max |q| sum |k|."""
import numpy as np
import torch

from oracle import attention as ref


def query_terms(q, k_pages, k_scale, lens, table, scale=None):
    """What two e4m3 terms of the queries may move a row's scores by, [B, D, Hq]: q [B, D, Hq, d] fp64."""
    B, D, Hq, d = q.shape
    N, Hkv = k_scale.shape
    size = np.nan_to_num(np.abs(ref.e4m3_values()[k_pages])).sum(-1).max(-1) * k_scale  # [N, Hkv]
    out = np.zeros((B, D, Hq))
    for n in range(B):
        ids = [x for x in table[n, :-(-max(int(lens[n]), 0) // 64)] if 0 <= x < N]
        if ids:
            most = np.repeat(size[ids].max(0), Hq // Hkv)
            out[n] = 2.0 ** -17 * (d ** -0.5 if scale is None else scale) * np.abs(q[n]).max(-1) * most
    return out


def bounds(out, absout, mag, d, dtype, more=0.0):
    """(tolerance of out, tolerance of lse) for fp64 results; more: what moves the scores besides."""
    score = (d + 8) * 2.0 ** -23 * mag + more
    w = (2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -21) + 2.0 ** -17
    tol = absout * (2 * score[..., None] + 2.0 ** -20 + w) + np.abs(out) * (torch.finfo(dtype).eps / 2) + 1e-38
    return tol, 2 * score + 2.0 ** -17
