"""Error bounds of the weight-accumulating calls, from the arithmetic they do,
and the cases their tests share.

Notation: u = 2^-24, half a step of fp32.  A score is a sum of d_h + 2 r exact
bf16 products in fp32, each addition off by at most 2 u of the running sum of
magnitudes (tensor cores may truncate), and p = q B_h^K enters as a bf16 high
and low part: the high part leaves at most 2^-8 of an element and the low part
2^-8 of that, 2^-16.  So, with scale and key scale folded in,
  delta_hj = 2^-16 sum |p z| + 2 u (d_h + 3 r + 8) (sum |q k| + sum |p| |z|)
bounds a score's error (8 more steps: scale, log2 conversion and the like); the
probabilities exp(s - lse) move by at most expm1(delta_hj + max_j delta_hj) of
themselves; the exponential and the roundings of its argument, s log2 e and
lse log2 e, add 4 u (|s| + |lse| + 4) to the exponent.
"""
import math

import numpy as np
import torch

from compressed_cache_decode_gb300 import inputs
from oracle import lrkv_oracle as O

U = 2.0 ** -24
NAMES = ("q", "k_s", "v_s", "z_k", "z_v", "b_k", "b_v", "seq_lens")


def f64(t):
    return t.detach().cpu().double().numpy()


def score_error(q, k_s, z_k, b_k, h, scale, key_scale=None, positions=None):
    """Bound [T, L] of the error of row_scores() of q [T, d_h] computed as above;
    with positions the key is rebuilt and turned in fp32 (cos and sin rounded to
    fp32, a turned shared row possibly in two bf16 parts)."""
    q, k_s, z, B = np.abs(f64(q)), np.abs(f64(k_s)), np.abs(f64(z_k)[:, h]), f64(b_k)[h]
    dh, r = B.shape
    if positions is None:
        p = q @ np.abs(B)                             # >= |q B| element by element
        pz, qk = p @ z.T, q @ k_s.T
        err = 2.0 ** -16 * pz + 2 * U * (dh + 3 * r + 8) * (qk + pz)
    else:
        key = k_s + z @ np.abs(B).T                   # magnitudes of the rebuilt key
        qs = q.reshape(q.shape[0], -1, 2).sum(-1)     # a turned pair meets both of its elements
        pairs = qs @ key.reshape(len(key), -1, 2).sum(-1).T
        shared = qs @ k_s.reshape(len(key), -1, 2).sum(-1).T
        err = 2 * U * (dh + 2 * r + 16) * pairs + 2.0 ** -16 * shared
    err = err * scale
    return err if key_scale is None else err * np.abs(f64(key_scale))


def weight_bound(scores, lse, err):
    """Bound [L] of the error of sum over queries of exp(s - lse): scores, err
    [T, L] (-inf where a query does not look), lse [T] with the same error as
    the scores of its row."""
    look = np.isfinite(scores)
    a = np.where(look, np.exp(np.where(look, scores, 0) - lse[:, None]), 0.0)
    top = np.max(np.where(look, err, 0.0), axis=1, keepdims=True)
    # + the exponential (2 u) and the rounding of its argument in the log2 domain
    arg = (np.abs(np.where(look, scores, 0)) + np.abs(lse[:, None]) + 4) * 4 * U
    return np.sum(a * np.expm1(np.where(look, err, 0.0) + top + arg), axis=0), a


def decode_bounds(case, b, h, scale, key_scale=None, positions=None, sections=None):
    """(out, lse, weights) error bounds of one (sequence, head)."""
    L = int(case["seq_lens"][b])
    ks = None if key_scale is None else key_scale[b, h, :L]
    pos = None if positions is None else positions[b, :L]
    q = case["q"][b, h:h + 1]
    s = O.row_scores(q, case["k_s"][b, :L], case["z_k"][b, :L], case["b_k"], h, scale, ks, pos, sections)
    err = score_error(q, case["k_s"][b, :L], case["z_k"][b, :L], case["b_k"], h, scale, ks, pos)
    m = s.max()
    lse = np.array([m + math.log(np.exp(s - m).sum())])
    w, a = weight_bound(s, lse, err)
    V = np.abs(f64(case["v_s"][b, :L])) + np.abs(f64(case["z_v"][b, :L, h])) @ np.abs(f64(case["b_v"][h])).T
    # probabilities in two bf16 parts (2^-16), L + r + 64 additions and merges
    out = (w + a[0] * (2.0 ** -16 + 2 * U * (L + 128))) @ V
    return out, err.max() + (abs(lse[0]) + 4 + L) * 2 * U, w


def random_prior(shape, seed):
    return torch.rand(shape, generator=torch.Generator().manual_seed(seed)) * 2


def random_positions(B, L, axes, top, seed):
    return torch.randint(0, top, (B, L, axes), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)


def paged(case, page_size, seed):
    return inputs.paged_from_contiguous(case, page_size=page_size, seed=seed)


def cuda(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
