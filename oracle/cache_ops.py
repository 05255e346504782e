"""Plain FP64 CPU forms of the rotating append, the 8-bit cache and window attention.

TEST INFRASTRUCTURE ONLY, like the rest of the oracle: it shares no code with
the CUDA path, takes CPU tensors of any float type (converted exactly) and
computes in float64, one row at a time.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64
MIN_EXP = -100


def rotate_row(x: torch.Tensor, pos: int, inv_freq: torch.Tensor, interleaved: bool) -> torch.Tensor:
    """x [..., d] turned at position pos: pair i by pos * inv_freq[i]."""
    y = x.to(F64).clone()
    r = 2 * inv_freq.numel()
    for i in range(r // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        angle = pos * float(inv_freq[i])
        c, s = math.cos(angle), math.sin(angle)
        x0, x1 = x[..., a].to(F64), x[..., b].to(F64)
        y[..., a], y[..., b] = x0 * c - x1 * s, x1 * c + x0 * s
    return y


def rotate_rows(x: torch.Tensor, pos: torch.Tensor, inv_freq: torch.Tensor, interleaved: bool) -> torch.Tensor:
    """rotate_row of x[t] at pos[t]."""
    return torch.stack([rotate_row(x[t], int(pos[t]), inv_freq, interleaved) for t in range(x.shape[0])]) \
        if x.shape[0] else x.to(F64)


# every finite e4m3 value, ascending, with its code
def _e4m3_value(code: int) -> float:
    exp, man = (code >> 3) & 15, code & 7
    v = man * 2.0 ** -9 if exp == 0 else (1 + man / 8) * 2.0 ** (exp - 7)
    return -v if code & 128 else v


_CODES = sorted((c for c in range(256) if c & 127 != 127), key=lambda c: (_e4m3_value(c), -c))
_VALUES = torch.tensor([_e4m3_value(c) for c in _CODES], dtype=F64)
_POSITIVE = torch.tensor([_e4m3_value(c) for c in range(127)], dtype=F64)


def round_e4m3(x: torch.Tensor) -> torch.Tensor:
    """x (float64) to the nearest e4m3 value, ties to the even code, +-448 beyond; NaN stays NaN."""
    mag = x.abs().clamp_max(448.0)
    hi = torch.searchsorted(_POSITIVE, mag.nan_to_num(0.0)).clamp(1, 126)
    lo = hi - 1
    up, down = _POSITIVE[hi] - mag, mag - _POSITIVE[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    out = torch.where(take_hi, _POSITIVE[hi], _POSITIVE[lo])
    return torch.where(x.isnan(), x, torch.copysign(out, x))


def needed_scale(amax: float) -> float:
    """The smallest power of two with amax <= 448 times it, at least 2^-100."""
    e = MIN_EXP
    if amax > 0:
        e = max(e, math.frexp(amax / 448.0)[1] - 1)
        if math.ldexp(448.0, e) < amax:
            e += 1
    return math.ldexp(1.0, e)


def fp8_append(values: torch.Tensor, scale: torch.Tensor, rows: torch.Tensor, stream, pos, block: int = 128):
    """Append rows [n][G][D] (float64) to an 8-bit cache given as its e4m3
    values [S][G][cap][D] (float64) and scales [S][G][nblk].  Returns new
    (values, scale)."""
    values, scale = values.clone(), scale.to(F64).clone()
    touched: dict = {}
    for t in range(rows.shape[0]):
        touched.setdefault((int(stream[t]), int(pos[t]) // block), []).append(t)
    for (s, b), toks in touched.items():
        fresh = any(int(pos[t]) % block == 0 for t in toks)
        for g in range(rows.shape[1]):
            x = torch.stack([rows[t, g] for t in toks])
            finite = x[x.isfinite()].abs()
            need = needed_scale(float(finite.max()) if finite.numel() else 0.0)
            held = float(scale[s, g, b])
            before = held if held > 0 and not fresh else 0.0
            after = max(before, need)
            span = slice(b * block, b * block + block)
            if before > 0 and after > before:
                values[s, g, span] = round_e4m3(values[s, g, span] * (before / after))
            scale[s, g, b] = after
            for t in toks:
                values[s, g, int(pos[t])] = round_e4m3(rows[t, g] / after)
    return values, scale


def fp8_values(values: torch.Tensor, scale: torch.Tensor, block: int = 128) -> torch.Tensor:
    """The rows an 8-bit cache stands for: values [S][G][cap][D], scales [S][G][nblk]."""
    return values.to(F64) * scale.to(F64).repeat_interleave(block, dim=2)[..., None]


def visible_slots(pos: int, window: int, n_sink: int) -> list[int]:
    return [j for j in range(pos + 1) if j > pos - window or j < n_sink]


def attention_rows(q, k_cache, v_cache, q_stream, q_pos, rows_of, scale: float):
    """Attention of every query over the slots rows_of(i, g, s, p): q [n][Hq][D],
    caches [S][G][cap][D].  Returns float64 (out, spread, reach), all [n][Hq][D]
    or [n][Hq][1]: spread = sum_j w_j |v_j - out|, reach = the largest
    sum_d |scale q_d k_jd|; both bound what rounding can do to a result.  A
    query outside the caches, or with no row, gives zeros."""
    n, Hq, D = q.shape
    S, G, cap, _ = k_cache.shape
    out = torch.zeros((n, Hq, D), dtype=F64)
    spread, reach = torch.zeros_like(out), torch.zeros((n, Hq, 1), dtype=F64)
    for i in range(n):
        s, p = int(q_stream[i]), int(q_pos[i])
        if not (0 <= s < S and 0 <= p < cap):
            continue
        for g in range(G):
            rows = rows_of(i, g, s, p)
            if len(rows) == 0:
                continue
            idx = torch.as_tensor(rows, dtype=torch.long)
            k, v = k_cache[s, g].index_select(0, idx).to(F64), v_cache[s, g].index_select(0, idx).to(F64)
            h = slice(g * (Hq // G), (g + 1) * (Hq // G))
            qs = q[i, h].to(F64)
            w = torch.softmax(qs @ k.T * scale, dim=1)
            out[i, h] = w @ v
            for d in range(0, D, 32):                      # [heads][rows][32] at a time
                spread[i, h, d:d + 32] = torch.einsum("hr,hrd->hd", w, (v[None, :, d:d + 32] - out[i, h, None, d:d + 32]).abs())
            reach[i, h] = (qs.abs() @ k.abs().T).amax(1, keepdim=True) * abs(scale)
    return out, spread, reach


def window_attention(q, k_cache, v_cache, q_stream, q_pos, window: int, n_sink: int, scale: float, hidden=()):
    """attention_rows over each query's visible slots; ``hidden``: (stream,
    slot) pairs left out (unmapped pages)."""
    gone: dict = {}
    for s, j in hidden:
        gone.setdefault(s, set()).add(j)
    return attention_rows(q, k_cache, v_cache, q_stream, q_pos,
                          lambda i, g, s, p: [j for j in visible_slots(p, window, n_sink) if j not in gone.get(s, ())],
                          scale)


def selected_attention(q, k_cache, v_cache, sel, q_stream, q_pos, scale: float, block: int = 128):
    """attention_rows over the slots j <= p of each (query, group)'s selected blocks."""
    def rows_of(i, g, s, p):
        return [j for b in sel[i, g].tolist() if 0 <= b <= p // block
                for j in range(b * block, min(b * block + block, p + 1))]
    return attention_rows(q, k_cache, v_cache, q_stream, q_pos, rows_of, scale)
