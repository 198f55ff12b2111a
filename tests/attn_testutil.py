"""Shared helpers of the attention tests: caches, inputs and tolerances.

Tolerances are element-wise and follow from the arithmetic, not from results.
With A = sum_j p_j |v_j| (the attention over |v|) and M = the largest
scale sum_i |q_i k_i| of the row:

* scores: products are exact or rounded to 2^-22 (fp32 as two fp16 terms),
  sums of d terms in fp32, so a score is off by at most (d + 8) 2^-23 M, which
  moves a weight by that much relatively, twice (numerator and sum);
* weights: e^x to 2^-21, then as an operand rounded to 2^-9 (bf16, prompts),
  2^-11 (fp16, cache, bf16 outputs) or 2^-21 (fp32, or two fp16 terms);
* the output's own rounding: 2^-9 |o| for bf16, 2^-23 |o| for fp32, and sums
  over n keys in fp32: relative to A, 2^-24 per addition of a block, bounded
  by 2^-17 for the lengths used here.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import attention as ref

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g).to(dtype)


def np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def bounds(out, absout, mag, d, dtype):
    """(tolerance of out, tolerance of lse) for fp64 results."""
    score = (d + 8) * 2.0 ** -23 * mag
    if dtype == torch.bfloat16:
        w, own = 2.0 ** -9 + 2.0 ** -17, 2.0 ** -9
    else:
        w, own = 2.0 ** -21 + 2.0 ** -17, 2.0 ** -23
    tol = absout * (2 * score[..., None] + 2.0 ** -20 + w) + np.abs(out) * own + 1e-38
    return tol, 2 * score + 2.0 ** -17


def check(got, want, tol, what):
    got = np64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fin = np.isfinite(want)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    assert same[~fin].all(), f"{what}: non-finite values differ"
    err = np.abs(got[fin] - want[fin])
    tol = np.broadcast_to(tol, want.shape)[fin]
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} out of tolerance, worst ratio "
                           f"{np.nanmax(err / tol):.3g}, max error {np.nanmax(err):.3g}")


def make_cache(g, pages, heads, d, spread=1.0):
    """(uint8 k, v pages and fp32 power-of-two scales) of quantised normal values; scales differ between pages."""
    out = []
    for shape, flip in (((pages, heads, 64, d), False), ((pages, heads, d, 64), True)):
        gain = torch.exp2(torch.round(spread * torch.randn((pages, heads), generator=g)))
        x = np64(torch.randn(shape, generator=g)) * gain.numpy()[:, :, None, None]
        s = np.array([[ref.pow2_need(np.abs(x[p, h]).max()) for h in range(heads)] for p in range(pages)])
        out += [torch.from_numpy(ref.e4m3_round(x / s[:, :, None, None])), torch.from_numpy(s).float()]
    k, ks, v, vs = out
    return k, v, ks, vs


def to_device(cache):
    from gated_delta_rule_decode_gb300 import attn
    k, v, ks, vs = cache
    f8 = torch.float8_e4m3fn
    return attn.KVCache(k.cuda().view(f8), v.cuda().view(f8), ks.cuda(), vs.cuda())


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
