"""fp64 oracle of the answering path: rotary positions and their gradient, the
paged key/value cache with its rounding to e4m3, and attention of one new
token over the pages.

TEST INFRASTRUCTURE ONLY (like the rest of ``oracle/``); it shares no code with
the CUDA path.  Plain numpy loops over the definitions; every function takes
torch tensors or numpy arrays and returns float64 numpy arrays.
"""

from __future__ import annotations

import numpy as np

from . import _f64
from .fp8 import e4m3_to_f64


def _int(x) -> np.ndarray:
    if hasattr(x, "detach"):
        x = x.detach().to("cpu").numpy()
    return np.asarray(x).astype(np.int64)


def codes(t8) -> np.ndarray:
    """The byte codes of an e4m3 tensor (float8_e4m3fn or uint8)."""
    if hasattr(t8, "detach"):
        import torch

        t8 = t8.detach().to("cpu")
        t8 = (t8 if t8.dtype == torch.uint8 else t8.view(torch.uint8)).numpy()
    return np.asarray(t8)


# ------------------------------------------------------------------ positions
def rope_angles(pos, inv_freq, sections) -> np.ndarray:
    """theta [B, N, d/2] = pos[axis(i)] inv_freq[i], pos [axes, B, N]."""
    pos, f = _int(pos), _f64(inv_freq)
    axis = np.concatenate([np.full(s, a, dtype=np.int64) for a, s in enumerate(sections)])
    return np.stack([pos[axis[i]].astype(np.float64) * f[i] for i in range(len(f))], axis=-1)


def rope(x, pos, inv_freq, sections, interleaved=False, inverse=False) -> np.ndarray:
    """x [B, H, N, d] turned pair by pair; ``inverse`` turns by -theta."""
    x = _f64(x)
    B, H, N, d = x.shape
    th = rope_angles(np.broadcast_to(_int(pos), (len(sections), B, N)), inv_freq, sections)
    th = (-th if inverse else th)[:, None]
    ia = np.arange(d // 2) * 2 if interleaved else np.arange(d // 2)
    ib = ia + 1 if interleaved else ia + d // 2
    y = np.empty_like(x)
    y[..., ia] = x[..., ia] * np.cos(th) - x[..., ib] * np.sin(th)
    y[..., ib] = x[..., ib] * np.cos(th) + x[..., ia] * np.sin(th)
    return y


# ---------------------------------------------------------------- e4m3 rows
_CODE_VALUES = e4m3_to_f64(np.arange(128))  # 0 .. 448 ascending, then NaN
_CODE_VALUES = _CODE_VALUES[:127]


def nearest_e4m3(x) -> np.ndarray:
    """Byte codes of the nearest e4m3 values (ties to the even code), at most
    +-448; NaN becomes code 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.clip(np.searchsorted(_CODE_VALUES, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _CODE_VALUES[lo], _CODE_VALUES[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def row_descale(x) -> np.ndarray:
    """Factors [...] of rows x [..., d]: the smallest power of two, at least
    2^-126, with the largest finite |x| <= 448 descale; 1 for zeros."""
    x = np.asarray(x, dtype=np.float64)
    amax = np.max(np.where(np.isfinite(x), np.abs(x), 0.0), axis=-1)
    out = np.ones_like(amax)
    for i, a in np.ndenumerate(amax):
        if a > 0:
            e = -126
            while 448.0 * 2.0 ** e < a:
                e += 1
            out[i] = 2.0 ** e
    return out


def quantise_rows(x):
    """(codes uint8 [..., d], factors [...]) of rows x."""
    x = _f64(x)
    s = row_descale(x)
    return nearest_e4m3(x / s[..., None]), s


# -------------------------------------------------------------------- cache
def cache_values(cache, descale=None) -> np.ndarray:
    """The values a cache stands for, float64 [pages, Hkv, page_size, d]."""
    if descale is None:
        return _f64(cache)
    return e4m3_to_f64(codes(cache)) * _f64(descale)[..., None]


def gather(values, table_row, positions) -> np.ndarray:
    """Rows [Hkv, len(positions), d] of one sequence; a position on a page
    outside the cache is a row of NaN."""
    P, Hkv, ps, d = values.shape
    out = np.full((Hkv, len(positions), d), np.nan)
    for i, p in enumerate(positions):
        page = int(table_row[p // ps])
        if 0 <= page < P:
            out[:, i] = values[page, :, p % ps]
    return out


def decode(q, kvals, vvals, page_table, seq_lens, scale: float, window: int = 0) -> dict:
    """O [B, Hq, d], L [B, Hq] of one token per sequence, and what bounds the
    rounding of a computation of them: A = sum_j p_j |v_j| [B, Hq, d] and
    S = max_j scale sum_i |q_i k_ji| [B, Hq].  Positions on bad pages are
    skipped."""
    q = _f64(q)
    B, Hq, d = q.shape[0], q.shape[1], q.shape[-1]
    q = q.reshape(B, Hq, d)
    table, lens = _int(page_table), _int(seq_lens)
    Hkv, ps = kvals.shape[1], kvals.shape[2]
    g = Hq // Hkv
    o, A = np.zeros((B, Hq, d)), np.zeros((B, Hq, d))
    L, S = np.full((B, Hq), -np.inf), np.zeros((B, Hq))
    n = np.zeros(B, dtype=np.int64)
    for b in range(B):
        top = min(max(int(lens[b]), 0), table.shape[1] * ps)
        lo = max(0, top - window) if window > 0 else 0
        pos = [p for p in range(lo, top) if 0 <= table[b, p // ps] < kvals.shape[0]]
        n[b] = len(pos)
        if not pos:
            continue
        k, v = gather(kvals, table[b], pos), gather(vvals, table[b], pos)
        for h in range(Hq):
            s = scale * (k[h // g] @ q[b, h])
            S[b, h] = scale * np.max(np.abs(k[h // g]) @ np.abs(q[b, h]))
            m = np.max(s)
            e = np.exp(s - m)
            L[b, h] = m + np.log(np.sum(e))
            p = e / np.sum(e)
            o[b, h] = p @ v[h // g]
            A[b, h] = p @ np.abs(v[h // g])
    return {"O": o, "L": L, "A": A, "S": S, "n": n}
