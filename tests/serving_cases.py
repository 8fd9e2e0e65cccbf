"""Shared builders of the paged-cache tests: shuffled page tables, caches with
everything that no sequence holds filled with NaN, and their oracle values."""

import numpy as np
import torch

from attention_backward_pass_attn_gb300.inputs import make_tensor
from oracle import serving


def page_table(lens, page, seed, spare=2, slack=1):
    """(table int32 [B, pages + slack], num_pages): shuffled pages; entries
    that no position needs hold numbers that name no page."""
    need = [-(-int(n) // page) for n in lens]
    total = sum(need) + spare
    order = np.random.default_rng(seed).permutation(total)
    table = np.full((len(need), max(need + [0]) + slack), 2 ** 30, dtype=np.int32)
    table[:, -1] = -7
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return torch.from_numpy(table), total


def rows_held(table, lens, page, num_pages):
    """bool [num_pages, page]: the rows that some position falls on."""
    held = np.zeros((num_pages, page), dtype=bool)
    for b, n in enumerate(lens):
        for p in range(int(n)):
            held[int(table[b, p // page]), p % page] = True
    return held


def filled_cache(lens, page, Hkv, d, seed, fp8, slack=1, std=1.0):
    """A cache whose held rows are random and whose other rows are NaN (in
    8 bits: NaN codes, with NaN and infinite factors).  Returns a dict of CPU
    tensors kc, vc, kd, vd, table and of fp64 values k64, v64."""
    table, P = page_table(lens, page, seed, slack=slack)
    held = torch.from_numpy(rows_held(table, lens, page, P))[:, None, :]
    out = {"table": table, "P": P}
    for i, n in enumerate("kv"):
        x = make_tensor((P, Hkv, page, d), seed + 31 * i, std=std)
        if fp8:
            c, s = serving.quantise_rows(x)
            c = torch.where(held[..., None], torch.from_numpy(c), torch.tensor(0x7F, dtype=torch.uint8))
            s = torch.where(held, torch.from_numpy(s).float(),
                            torch.tensor(float("nan") if i else float("inf")))
            out[n + "c"], out[n + "d"] = c.view(torch.float8_e4m3fn), s
            out[n + "64"] = serving.cache_values(c, s)
        else:
            x = torch.where(held[..., None], x, torch.tensor(float("nan"), dtype=x.dtype))
            out[n + "c"], out[n + "d"] = x, None
            out[n + "64"] = serving.cache_values(x)
    return out


def cuda(t):
    return None if t is None else t.cuda()
