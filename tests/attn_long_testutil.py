"""Tolerances of attention over the cache in parts or over selected pages.

As in attn_testutil, with A = sum_j p_j |v_j| and M = the largest scale sum_i |q_i k_i| of a row:
* scores are sums of d fp32 terms: off by at most (d + 8) 2^-23 M, which moves a weight by that much, twice;
* weights: e^x to 2^-21, then fp16 operands: 2^-11, or 2^-21 as two terms (fp32 inputs); sums over the keys in
  blocks and parts: 2^-17 of A bounds them for the lengths used here;
* the output's own half step, eps / 2 of its type."""
import numpy as np
import torch


def bounds(out, absout, mag, d, dtype):
    """(tolerance of out, tolerance of lse) for fp64 results."""
    score = (d + 8) * 2.0 ** -23 * mag
    w = (2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -21) + 2.0 ** -17
    tol = absout * (2 * score[..., None] + 2.0 ** -20 + w) + np.abs(out) * (torch.finfo(dtype).eps / 2) + 1e-38
    return tol, 2 * score + 2.0 ** -17
