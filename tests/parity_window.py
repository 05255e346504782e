"""Helpers of the tests of the rotating append, the 8-bit cache and window attention.

Bounds (u = 2^-24; a rounding is off by at most half a step, relative to the value 2^-8 in bf16, 2^-11 in fp16,
2^-4 in e4m3):

  * a rotated value x0 c - x1 s: the fraction of a turn reaches float32 with 2^-25, its sine and cosine are then off
    by at most 2 pi 2^-25 + 2^-23, each product and the difference round once: together below 2^-20 (|x0| + |x1|);
    the stored type adds its own rounding;
  * attention: with weights w_j (1 + d_j) in place of w_j, out moves by at most max|d| sum_j w_j |v_j - out| /
    (1 - max|d|).  d holds the rounding of p (2^-8 where p is bf16, 2^-11 where it is fp16), the score's error in the
    exponent (the sum of 128 exact products in float32, at most 130 u of the running sum of magnitudes, and at most
    8 u of the score for the factors; a factor 2 covers the maximum it is taken against), and ex2.approx and the
    float32 sums over the rows (below 2^-18).  The output's own rounding adds 2^-8 |out|.
"""
from __future__ import annotations

import torch

import block_sparse_attention_maxpool_b200 as msa
from oracle import cache_ops as C

U = 2.0 ** -24
P_BF16, P_FP16 = 2.0 ** -8, 2.0 ** -11


def norm_of(f8):
    """norm_round of a call: see check_attention (prefill calls may or may not expand an 8-bit cache)."""
    return P_FP16 if f8 else 0.0


POISON = float("nan")


def check_attention(got, want, spread, reach, p_round, kv_round=0.0, norm_round=0.0):
    """kv_round: rounding of the K and V values themselves (2^-8 where an 8-bit cache with scales that are no powers
    of two is expanded to bf16): a score moves by kv_round times ``reach`` at most, out by kv_round sum_j w_j |v_j|,
    which is at most spread + |out|.
    norm_round: where the sum of the p is not that of the rounded p (single queries over an 8-bit cache: p in fp16, 2^-11),
    out = sum_j w_j (1 + d_j) v_j, off by at most |d| sum_j w_j |v_j| <= |d| (spread + |out|), of which p_round covers
    the first part."""
    d = p_round + 2 * (138 * U + kv_round) * reach + 2.0 ** -18
    tol = d / (1 - d).clamp_min(0.5) * spread + 2.0 ** -8 * want.abs() * (1 + 2.0 ** -7) + 1e-30
    tol = tol + (kv_round + norm_round) * (spread + want.abs())
    g = got.double().cpu()
    assert bool(g.isfinite().all()), "not finite"
    err = (g - want).abs()
    worst = (err / tol).max()
    assert bool((err <= tol).all()), f"error {err.max():.3e}, {worst:.2f} of its bound at {(err > tol).nonzero()[0].tolist()}"
    return float(worst)


def check_rotated(got, x, pos, rope_freq, interleaved, own_round):
    """got: rows as stored, x: the rows before the turn [n][...][128]."""
    want = C.rotate_rows(x, pos, rope_freq, interleaved)
    r = 2 * rope_freq.numel()
    mag = torch.zeros_like(want)
    a = torch.arange(r // 2)
    i, j = (2 * a, 2 * a + 1) if interleaved else (a, a + r // 2)
    both = x[..., i].double().abs() + x[..., j].double().abs()
    mag[..., i] = mag[..., j] = both
    err = (got.double().cpu() - want).abs()
    tol = 2.0 ** -20 * mag + own_round * (want.abs() + 2.0 ** -20 * mag) + 2.0 ** -26
    assert bool((err <= tol).all()), f"rotated value off by {(err / tol).max():.2f} of its bound"
    assert torch.equal(got[..., r:].cpu().double(), x[..., r:].to(got.dtype).double()), "dims past rot_dim are copied"


def random_pages(S, nblk, spare, gen):
    """A block table of shuffled pages and the number of pages."""
    n = S * nblk + spare
    return torch.randperm(n, generator=gen)[:S * nblk].view(S, nblk).to(torch.int32), n


def to_pool(cache, table, n_pages, fill):
    """cache [S][G][cap][...] -> pages [n_pages][G][128][...] (spare pages hold ``fill``)."""
    S, G, cap = cache.shape[:3]
    pool = torch.full((n_pages, G, 128) + cache.shape[3:], fill, dtype=cache.dtype)
    for s in range(S):
        for b in range(cap // 128):
            if 0 <= int(table[s, b]) < n_pages:
                pool[int(table[s, b])] = cache[s, :, b * 128:b * 128 + 128]
    return pool


def scale_pool(scale, table, n_pages):
    S, G, nblk = scale.shape
    pool = torch.full((n_pages, G), POISON, dtype=scale.dtype)
    for s in range(S):
        for b in range(nblk):
            pool[int(table[s, b])] = scale[s, :, b]
    return pool


def quantise(x, pow2=True):
    """x [S][G][cap][128] float32 -> (e4m3 codes as float8 tensor, scale [S][G][nblk])."""
    S, G, cap, D = x.shape
    blk = x.view(S, G, cap // 128, 128, D)
    amax = blk.abs().amax((3, 4))
    if pow2:
        scale = torch.tensor([C.needed_scale(float(a)) for a in amax.flatten()]).view(amax.shape).float()
    else:
        scale = (amax / 448).float() * 1.0000002
    q = (blk / scale[..., None, None]).clamp(-448, 448).view(S, G, cap, D).to(torch.float8_e4m3fn)
    return q, scale


def device_error(expect=0):
    err = msa.msa_get_device_error()
    assert err == expect, f"device error word {err:#x}, expected {expect:#x}"


