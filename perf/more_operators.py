"""Attention whose scores are changed before the softmax, in training and in
answering, and the key/value cache in four bits that answers from it, as a
user calls them.

Four families, told apart by a case's ``"op"``:

  fwd / bwd    attention of a whole sequence with capped scores, a bias that
               falls with distance, a prefix that sees itself whole, a sliding
               window or packed documents; key heads shared by query heads
  decode       attention of the newest token of each sequence over its pages,
               with the same cap and bias, from bf16, e4m3 or 4-bit pages
  write/read   new keys and values into 4-bit pages, and rows of them back

Definitions used by the plain forms and by ``exact``:

  score        x_ij = scale <q_i, k_j>; with a cap, cap tanh(x_ij / cap); with
               slopes, minus slope[h] |i - j|
  mask         causal: j <= i, or j < prefix[b]; a window also hides
               j <= i - window, documents j < doc[b, i].  Not causal: nothing
  fwd          l_i = logsumexp_j, o_i = sum_j exp(x_ij - l_i) v_j; query head h
               reads key head h // (Hq / Hkv)
  bwd          P = exp(x - l), D_i = <do_i, o_i>, dX = P (do v^T - D), times
               1 - tanh^2 under a cap; dq = scale dX k, dk = scale dX^T q,
               dv = P^T do, dk and dv summed over the query heads of a key head
  cache        [pages][Hkv][page_size][d]; position p of sequence b lives in
               page table[b][p // page_size], row p % page_size
  4-bit row    32 values in a row share a factor f = amax / 7 rounded to five
               significant bits (ties to even; 1 for zeros, at least 2^-120);
               value = clamp(round(x / f), -7, 7) f, ties to even.  Byte i of a
               row: element 2i in its low four bits, 2i + 1 in the others,
               each plus 8
  e4m3 row     descale = the smallest power of two with amax <= 448 descale
               (1 for a row of zeros), value = e4m3(x / descale)
  decode       as fwd's last row over the last `window` (0: all) of a
               sequence's `len` positions; no position: o = 0, l = -inf
"""

import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16
E4M3 = torch.float8_e4m3fn
GROUP = 32  # values of a 4-bit row that share a factor


# --------------------------------------------------------------------- cases
def listed():
    return [
        # A short packed batch on a sliding-window layer of a small capped model.
        {"name": "fwd_b2_n513_h8kv2_d64_cap_w128", "op": "fwd", "B": 2, "N": 513, "Hkv": 2, "group": 4,
         "d": 64, "causal": True, "cap": 30.0, "alibi": False, "mask": "window", "window": 128},
        # A long prompt of a capped model with shared key heads, the largest work of a forward.
        {"name": "fwd_b1_n16384_h16kv4_d128_cap", "op": "fwd", "B": 1, "N": 16384, "Hkv": 4, "group": 4,
         "d": 128, "causal": True, "cap": 50.0, "alibi": False, "mask": "none", "window": 0},
        # Fine-tuning on images and text: each image and its question see themselves whole.
        {"name": "bwd_b2_n2047_h16_d64_cap_prefix", "op": "bwd", "B": 2, "N": 2047, "Hkv": 16, "group": 1,
         "d": 64, "causal": True, "cap": 50.0, "alibi": False, "mask": "prefix", "window": 0},
        # A training step of a model that knows positions by a distance bias.
        {"name": "bwd_b1_n8192_h32kv8_d128_alibi", "op": "bwd", "B": 1, "N": 8192, "Hkv": 8, "group": 4,
         "d": 128, "causal": True, "cap": 0.0, "alibi": True, "mask": "none", "window": 0},
        # One user's next token of a capped model, on a window layer: all latency.
        {"name": "decode_b1_kv4x2_len700_cap_w512", "op": "decode", "B": 1, "Hkv": 4, "group": 2, "d": 64,
         "page": 16, "len": 700, "ragged": False, "window": 512, "bits": 16, "cap": 50.0, "alibi": False},
        # A serving batch with a distance bias over an 8-bit cache.
        {"name": "decode_b16_kv8x4_4k_alibi_e4m3", "op": "decode", "B": 16, "Hkv": 8, "group": 4, "d": 128,
         "page": 64, "len": 4096, "ragged": True, "window": 0, "bits": 8, "cap": 0.0, "alibi": True},
        # One very long document in a 4-bit cache: the length is split over the GPU.
        {"name": "decode_b1_kv8x4_128k_int4", "op": "decode", "B": 1, "Hkv": 8, "group": 4, "d": 128,
         "page": 128, "len": 131072, "ragged": False, "window": 0, "bits": 4, "cap": 0.0, "alibi": False},
        # A large batch of a capped model over a 4-bit cache.
        {"name": "decode_b32_kv8x8_8k_cap_int4", "op": "decode", "B": 32, "Hkv": 8, "group": 8, "d": 128,
         "page": 64, "len": 8192, "ragged": True, "window": 0, "bits": 4, "cap": 50.0, "alibi": False},
        # A decode step's append: one token a sequence.
        {"name": "write_b64_t1_int4", "op": "write", "B": 64, "Hkv": 8, "d": 128, "page": 64, "T": 1,
         "before": 4000, "ragged": True},
        # A prompt's keys and values, padded batch.
        {"name": "write_b4_t8192_int4", "op": "write", "B": 4, "Hkv": 16, "d": 128, "page": 64, "T": 8192,
         "before": 0, "ragged": True},
        # A short prefix back out of the cache.
        {"name": "read_b2_t700_d64_int4", "op": "read", "B": 2, "Hkv": 4, "d": 64, "page": 16, "T": 700,
         "before": 100, "ragged": True},
        # A long cached prefix back in bf16, for attention of the rest of a prompt.
        {"name": "read_b4_t8192_int4", "op": "read", "B": 4, "Hkv": 16, "d": 128, "page": 64, "T": 8192,
         "before": 0, "ragged": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "decode", "decode", "decode", "write", "read"])
    d = rng.choice([64, 128])
    cap, alibi = rng.choice([(30.0, False), (50.0, False), (0.0, True), (50.0, True), (0.0, False)])
    if op in ("fwd", "bwd"):
        group = rng.choice([1, 1, 2, 3, 4, 8])
        B, Hkv = _log(rng, 1, 8), rng.choice([h for h in (1, 2, 4, 8, 16, 32) if h * group <= 32])
        causal = rng.random() < 0.8
        # N^2 heads d of the largest listed case of either op, both halves of the square counted
        most = 16 * 16384 ** 2 if op == "fwd" else 32 * 8192 ** 2
        N = _log(rng, 1, min(16384, math.isqrt(most * 128 // (B * Hkv * group * d * (1 if causal else 2)))))
        mask = rng.choice(["none", "none", "window", "documents", "prefix"]) if causal else "none"
        return {"op": op, "B": B, "N": N, "Hkv": Hkv, "group": group, "d": d, "causal": causal, "cap": cap,
                "alibi": alibi, "mask": mask,
                "window": _log(rng, 1, 4096) if mask == "window" or rng.random() < 0.3 and mask == "documents" else 0}
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if op == "decode":
        B, Hkv = _log(rng, 1, 64), rng.choice([1, 2, 3, 4, 8, 16])
        bits = rng.choice([16, 8, 4, 4])
        if bits != 4 and not cap and not alibi:
            cap = 30.0
        most = min(131072, 134000000 // (B * Hkv * d))
        return {"op": op, "B": B, "Hkv": Hkv, "group": rng.choice([1, 2, 4, 5, 8, 12, 16]), "d": d,
                "page": page, "len": _log(rng, 1, most), "ragged": rng.random() < 0.7,
                "window": rng.choice([0, 0, _log(rng, 1, 8192)]), "bits": bits, "cap": cap, "alibi": alibi}
    B, Hkv = _log(rng, 1, 64), rng.choice([1, 2, 3, 4, 8, 16])
    most = min(16384, 60000000 // (B * Hkv * d))
    return {"op": op, "B": B, "Hkv": Hkv, "d": d, "page": page, "T": _log(rng, 1, most),
            "before": rng.choice([0, _log(rng, 1, 500)]), "ragged": rng.random() < 0.7}


# -------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(shape, g, dtype=BF16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _slopes(H):
    """The usual ladder of distance slopes, 2^-8/H to 2^-8."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device=DEV)


def _queries(shape, cap, g):
    """Queries of heads of unequal sharpness: capped models have scores of tens,
    and some of them reach the cap."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    if cap:
        x = x * (1 + 9 * torch.rand((1, shape[1], 1, 1), generator=g, device=DEV) ** 2)
    return x.to(BF16)


def _lengths(B, most, ragged, seed, least=1):
    """[B] int32: all `most`, or spread over [least, most] with one sequence
    at `most` and, in a batch of eight or more, one empty slot."""
    g = torch.Generator().manual_seed(int(seed) + 17)
    n = torch.full((B,), most, dtype=torch.int32)
    if ragged:
        n = torch.randint(least, most + 1, (B,), generator=g, dtype=torch.int32)
        n[0] = most
        if B >= 8:
            n[B - 1] = 0
    return n


def _table(lens, page, seed, most=0):
    """A page table for sequences of `lens` positions, pages shuffled as a pool
    hands them out after a while.  The pool holds these sequences, or as many
    of `most` positions.  Returns (table, pages)."""
    need = [max(1, -(-int(n) // page)) for n in lens]
    total = max(sum(need), len(need) * -(-most // page)) + 3
    order = torch.randperm(total, generator=torch.Generator().manual_seed(int(seed) + 29)).to(torch.int32)
    table = torch.zeros((len(need), max(need)), dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table.to(DEV), total


def _documents(B, N, seed):
    """int32 [B, N]: the first position of each position's document, documents
    of unequal length packed one behind the other."""
    g = torch.Generator().manual_seed(int(seed) + 41)
    starts = torch.rand((B, N), generator=g) < 5.0 / max(N, 5)
    at = torch.where(starts, torch.arange(N).expand(B, N), torch.zeros((B, N), dtype=torch.long))
    return torch.cummax(at, dim=1).values.to(torch.int32).to(DEV)


def _cache(pages, Hkv, page, d, g, bits):
    """Key and value pages holding earlier tokens (some head channels larger
    than the rest, as trained keys have), with their factors or None."""
    gain = 1 + 3 * (torch.rand((Hkv, 1, d), generator=g, device=DEV) > 0.97).float()
    out = []
    for which in ("k", "v"):
        x = _randn((pages, Hkv, page, d), g)
        x = (x * gain).to(BF16) if which == "k" else x
        out.append((x, None) if bits == 16 else _quantise8(x) if bits == 8 else _quantise4(x))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def prepare(case, seed):
    g, op, d = _gen(seed), case["op"], case["d"]
    if op in ("fwd", "bwd"):
        B, N, Hkv, H = case["B"], case["N"], case["Hkv"], case["Hkv"] * case["group"]
        s = {"op": op, "causal": case["causal"], "scale": 1 / math.sqrt(d), "cap": case["cap"],
             "slopes": _slopes(H) if case["alibi"] else None, "window": case["window"],
             "doc": _documents(B, N, seed) if case["mask"] == "documents" else None, "prefix": None}
        if case["mask"] == "prefix":
            h = torch.Generator().manual_seed(int(seed) + 53)
            s["prefix"] = torch.randint(0, max(1, N // 2) + 1, (B,), generator=h, dtype=torch.int32).to(DEV)
        s["q"] = _queries((B, H, N, d), case["cap"], g)
        # keys and values as one fused projection [B][N][heads][d] leaves them
        x = _randn((B, N, 2 * Hkv, d), g)
        s["k"], s["v"] = x[:, :, :Hkv].transpose(1, 2), x[:, :, Hkv:].transpose(1, 2)
        if op == "bwd":
            f = _plain_fwd(s)
            s.update(o=f["o"], lse=f["lse"], do=_randn((B, H, N, d), g))
        return s
    B, Hkv, page = case["B"], case["Hkv"], case["page"]
    bits = case["bits"] if op == "decode" else 4
    if op == "decode":
        lens = _lengths(B, case["len"], case["ragged"], seed)
    else:
        count = _lengths(B, case["T"], case["ragged"], seed, least=min(1, case["T"] - 1))
        before = _lengths(B, case["before"], case["ragged"], seed + 1, least=0) if case["before"] else count * 0
        lens = before + count
    table, pages = _table(lens, page, seed, 0 if op == "decode" else case["before"] + case["T"])
    kc, vc, kd, vd = _cache(pages, Hkv, page, d, g, bits)
    s = {"op": op, "kc": kc, "vc": vc, "kd": kd, "vd": vd, "table": table, "d": d}
    if op == "decode":
        H = Hkv * case["group"]
        s.update(q=_queries((B, H, 1, d), case["cap"], g), lens=lens.to(DEV), window=case["window"],
                 scale=1 / math.sqrt(d), cap=case["cap"], slopes=_slopes(H) if case["alibi"] else None)
        return s
    s.update(T=case["T"], start=before.to(DEV), count=count.to(DEV))
    if op == "write":  # heads of one fused projection [B][T][heads][d]
        x = _randn((B, case["T"], 2 * Hkv, d), g)
        s["k"], s["v"] = x[:, :, :Hkv].transpose(1, 2), x[:, :, Hkv:].transpose(1, 2)
    return s


# ------------------------------------------------------------ 8 and 4 bits
def _quantise8(x):
    """bf16 [..., d] -> (float8_e4m3fn values [..., d], factors [...])."""
    x = x.float()
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp_min(-126)
    s = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))
    return (x / s.unsqueeze(-1)).to(E4M3), s


def _quantise4(x):
    """bf16 [..., d] -> (packed uint8 [..., d / 2], bf16 factors [..., d / 32])."""
    x = x.float().unflatten(-1, (-1, GROUP))
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax / 7)  # m in [0.5, 1): five bits of it are 1/32s
    f = torch.ldexp(torch.round(m * 32), e - 5).clamp_min(2.0 ** -120)
    f = torch.where(amax > 0, f, torch.ones_like(f))
    c = torch.clamp(torch.round(x / f.unsqueeze(-1)), -7, 7).flatten(-2) + 8
    c = c.to(torch.uint8)
    return c[..., 0::2] | c[..., 1::2] << 4, f.to(BF16)


def _values4(c, f):
    """fp32 [..., d] that packed codes and their factors stand for."""
    x = torch.stack([c & 15, c >> 4], -1).flatten(-2).float() - 8
    return (x.unflatten(-1, (-1, GROUP)) * f.float().unsqueeze(-1)).flatten(-2)


# --------------------------------------------------------------- plain forms
def _scores(s, q, k, h, g, b):
    """(x, dx/ds, visible): changed scores fp32 [heads, N, N] of query heads h
    (a slice) of batch element b against their key heads' k [heads / g, N, d]."""
    H, N, d = q.shape
    x = torch.matmul(q.view(H // g, g * N, d), k.transpose(1, 2)).view(H, N, N) * s["scale"]
    i, j = torch.arange(N, device=DEV)[:, None], torch.arange(N, device=DEV)[None, :]
    slope = None
    if s["cap"]:
        t = torch.tanh(x / s["cap"])
        x, slope = s["cap"] * t, 1 - t * t
    if s["slopes"] is not None:
        x = x - s["slopes"][h, None, None] * (i - j).abs()
    seen = None
    if s["causal"]:
        seen = j <= i
        if s["window"]:
            seen = seen & (j > i - s["window"])
        if s["doc"] is not None:
            seen = seen & (j >= s["doc"][b, :, None])
        if s["prefix"] is not None:
            seen = seen | (j < s["prefix"][b])
    return x, slope, seen


def _blocks(s):
    """(b, slice of query heads, slice of key heads): as many whole groups of
    heads at a time as fit 2^28 scores."""
    B, H, N, _ = s["q"].shape
    Hkv = s["k"].shape[1]
    g = H // Hkv
    n = max(1, min(Hkv, 2 ** 28 // max(1, g * N * N)))
    for b in range(B):
        for h in range(0, Hkv, n):
            yield b, slice(h * g, min(h + n, Hkv) * g), slice(h, min(h + n, Hkv)), g


def _plain_fwd(s):
    B, H, N, d = s["q"].shape
    o = torch.empty((B, H, N, d), dtype=BF16, device=DEV)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=DEV)
    for b, h, hk, g in _blocks(s):
        x, _, seen = _scores(s, s["q"][b, h].float(), s["k"][b, hk].float(), h, g, b)
        if seen is not None:
            x = x.masked_fill(~seen, float("-inf"))
        m = x.amax(-1, keepdim=True)
        x = torch.exp(x - m)
        z = x.sum(-1, keepdim=True)
        n = x.shape[0]
        o[b, h] = (torch.matmul(x.view(n // g, g * N, N), s["v"][b, hk].float()).view(n, N, d) / z).to(BF16)
        lse[b, h] = (m + torch.log(z)).squeeze(-1)
    return {"o": o, "lse": lse}


def _plain_bwd(s):
    dq = torch.empty(s["q"].shape, dtype=BF16, device=DEV)
    dk = torch.empty(s["k"].shape, dtype=BF16, device=DEV)
    dv = torch.empty(s["k"].shape, dtype=BF16, device=DEV)
    for b, h, hk, g in _blocks(s):
        q, k, v = s["q"][b, h].float(), s["k"][b, hk].float(), s["v"][b, hk].float()
        do, o = s["do"][b, h].float(), s["o"][b, h].float()
        n, N, d = q.shape
        p, slope, seen = _scores(s, q, k, h, g, b)
        p = torch.exp(p - s["lse"][b, h].unsqueeze(-1))
        if seen is not None:
            p = p.masked_fill(~seen, 0.0)
        dv[b, hk] = torch.matmul(p.view(n // g, g * N, N).transpose(1, 2), do.view(n // g, g * N, d)).to(BF16)
        dx = torch.matmul(do.view(n // g, g * N, d), v.transpose(1, 2)).view(n, N, N)
        dx = p * (dx - (do * o).sum(-1, keepdim=True))
        if slope is not None:
            dx = dx * slope
        dx = (dx * s["scale"]).view(n // g, g * N, N)
        dq[b, h] = torch.matmul(dx, k).view(n, N, d).to(BF16)
        dk[b, hk] = torch.matmul(dx.transpose(1, 2), q.view(n // g, g * N, d)).to(BF16)
    return {"dq": dq, "dk": dk, "dv": dv}


def _rows(s, pos):
    """(page, row) of positions pos [B, T]."""
    page = s["kc"].shape[2]
    at = (pos // page).clamp(0, s["table"].shape[1] - 1).long()
    return torch.gather(s["table"], 1, at).long(), (pos % page).long()


def _fetch(cache, factor, pg, row):
    """fp32 [B, Hkv, T, d] of the rows (pg, row) [B, T]."""
    if factor is None:
        x = cache[pg, :, row].float()
    elif factor.dim() == 3:
        x = cache.view(torch.uint8)[pg, :, row].view(E4M3).float() * factor[pg, :, row].unsqueeze(-1)
    else:
        x = _values4(cache[pg, :, row], factor[pg, :, row])
    return x.transpose(1, 2)


def _plain_decode(s):
    q = s["q"].float()
    B, H, _, d = q.shape
    Hkv = s["kc"].shape[1]
    most = s["table"].shape[1] * s["kc"].shape[2]
    pos = torch.arange(most, device=DEV).expand(B, most)
    pg, row = _rows(s, pos)
    lens = s["lens"].long().unsqueeze(1)
    seen = pos < lens
    if s["window"]:
        seen = seen & (pos >= lens - s["window"])
    k = _fetch(s["kc"], s["kd"], pg, row)
    x = torch.matmul(q.view(B, Hkv, H // Hkv, d), k.transpose(2, 3)) * s["scale"]
    del k
    if s["cap"]:
        x = s["cap"] * torch.tanh(x / s["cap"])
    if s["slopes"] is not None:
        x = x - s["slopes"].view(Hkv, H // Hkv, 1) * (lens - 1 - pos).abs()[:, None, None]
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    v = _fetch(s["vc"], s["vd"], pg, row) * seen[:, None, :, None]
    o = torch.matmul(p, v) / torch.where(z > 0, z, torch.ones_like(z))
    return {"o": o.view(B, H, 1, d).to(BF16), "lse": (m + torch.log(z)).view(B, H, 1)}


def _plain_write(s):
    t = torch.arange(s["T"], device=DEV).unsqueeze(0)
    count = s["count"].long().unsqueeze(1)
    # a token past its sequence's count is the last one of the count again,
    # and an empty sequence writes back what its first row holds
    src = torch.minimum(t, (count - 1).clamp_min(0))
    some = (count > 0).expand(-1, s["T"])[:, :, None, None]
    pg, row = _rows(s, s["start"].long().unsqueeze(1) + src)
    for new, cache, factor in ((s["k"], s["kc"], s["kd"]), (s["v"], s["vc"], s["vd"])):
        x = torch.gather(new.transpose(1, 2), 1, src[:, :, None, None].expand(-1, -1, new.shape[1], new.shape[3]))
        x, f = _quantise4(x)
        cache[pg, :, row] = torch.where(some, x, cache[pg, :, row])
        factor[pg, :, row] = torch.where(some, f, factor[pg, :, row])
    return _held(s)


def _plain_read(s):
    t = torch.arange(s["T"], device=DEV).unsqueeze(0)
    inside = (t < s["count"].unsqueeze(1))[:, None, :, None]
    pg, row = _rows(s, s["start"].long().unsqueeze(1) + t)
    pick = lambda c, f: torch.where(inside, _fetch(c, f, pg, row), torch.zeros((), device=DEV)).to(BF16)  # noqa: E731
    return {"k": pick(s["kc"], s["kd"]), "v": pick(s["vc"], s["vd"])}


def _held(s):
    """The cache after a write: the arrays themselves, codes as whole numbers
    in their bytes and the factors that make values of them."""
    return {"k_cache": s["kc"], "k_descale": s["kd"], "v_cache": s["vc"], "v_descale": s["vd"]}


# ----------------------------------------------------------------------- run
def run(state):
    s = state
    if own:
        import attention_backward_pass_attn_gb300 as attn

        if s["op"] in ("fwd", "bwd"):
            how = dict(causal=s["causal"], scale=s["scale"], softcap=s["cap"], slopes=s["slopes"],
                       window=s["window"], doc=s["doc"], prefix=s["prefix"])
            if s["op"] == "fwd":
                o, lse = attn.attn_fwd_score(s["q"], s["k"], s["v"], **how)
                return {"o": o, "lse": lse}
            dq, dk, dv = attn.attn_bwd_score(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], **how)
            return {"dq": dq, "dk": dk, "dv": dv}
        if s["op"] == "decode":
            o, lse = attn.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], scale=s["scale"],
                                      k_descale=s["kd"], v_descale=s["vd"], window=s["window"],
                                      softcap=s["cap"], slopes=s["slopes"])
            return {"o": o, "lse": lse}
        if s["op"] == "write":
            attn.kv_cache_write(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["start"], count=s["count"],
                                k_descale=s["kd"], v_descale=s["vd"])
            return _held(s)
        k, v = attn.kv_cache_read(s["kc"], s["vc"], s["table"], s["start"], s["T"], count=s["count"],
                                  k_descale=s["kd"], v_descale=s["vd"])
        return {"k": k, "v": v}
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "decode": _plain_decode, "write": _plain_write,
            "read": _plain_read}[s["op"]](s)


# ---------------------------------------------------------------------- work
def _pairs(case):
    """Visible (query, key) pairs of one head of a batch element; of prefixes
    and documents, at their expected lengths."""
    N, w = case["N"], case["window"]
    if not case["causal"]:
        return N * N
    w = min(w, N) if w else N
    if case["mask"] == "documents":  # about six documents
        n = max(1, N // 6)
        w = min(w, n)
        return (n * w - w * (w - 1) // 2) * (N // n)
    pairs = N * w - w * (w - 1) // 2
    if case["mask"] == "prefix":
        pairs += (N // 4) ** 2 // 2
    return pairs


def work(case):
    """Expected lengths stand in for the drawn ones: a ragged batch has one
    sequence at the longest and the others at half of it."""
    B, d, Hkv = case["B"], case["d"], case["Hkv"]
    if case["op"] in ("fwd", "bwd"):
        H, N, bwd = Hkv * case["group"], case["N"], case["op"] == "bwd"
        rows = B * N * d * 2  # bytes of one head of one tensor
        return {"bytes": rows * ((4 * H + 4 * Hkv) if bwd else (2 * H + 2 * Hkv)) + 4 * B * H * N,
                "flops": (10 if bwd else 4) * B * H * d * _pairs(case)}
    bits = case["bits"] if case["op"] == "decode" else 4
    most = case["len"] if case["op"] == "decode" else case["T"]
    others = B - 1 - (1 if B >= 8 else 0)
    tokens = most + others * most // 2 if case["ragged"] else B * most
    row = {16: 2 * d, 8: d + 4, 4: d // 2 + d // 16}[bits]
    if case["op"] == "decode":
        if case["window"]:
            tokens = sum(min(case["window"], n) for n in [most] + [most // 2] * others) if case["ragged"] \
                else B * min(case["window"], most)
        H = Hkv * case["group"]
        return {"bytes": tokens * Hkv * 2 * row + 4 * B * H * d + 4 * B * H + 4 * tokens // case["page"],
                "flops": 4 * tokens * H * d}
    full = B * case["T"] if case["op"] == "read" else tokens  # a read writes every row, zeros past the count
    return {"bytes": 2 * Hkv * (tokens * row + full * 2 * d), "flops": 2 * Hkv * tokens * d}


# --------------------------------------------------------------------- exact
def _head_64(case, s, b, h):
    """(x, dx/ds) float64 [N, N] of one query head, -inf where masked."""
    N = case["N"]
    x = s["q"][b, h].double() @ s["k"][b, h // case["group"]].double().T * s["scale"]
    der = None
    if case["cap"]:
        x = torch.tanh(x.div_(case["cap"]))
        der = 1 - x * x
        x = x.mul_(case["cap"])
    at = torch.arange(N, device=DEV, dtype=torch.float64)
    if s["slopes"] is not None:
        x -= s["slopes"][h].double() * (at[:, None] - at[None, :]).abs_()
    if case["causal"]:
        hidden = at[None, :] > at[:, None]
        if s["prefix"] is not None:
            hidden &= (at >= s["prefix"][b])[None, :]
        if s["window"]:
            hidden |= at[None, :] <= at[:, None] - s["window"]
        if s["doc"] is not None:
            hidden |= at[None, :] < s["doc"][b][:, None]
        x.masked_fill_(hidden, float("-inf"))
    return x, der


def _value_64(cache, factor, pages, h):
    """float64 [positions, d] of head h on the pages of one sequence, in order."""
    x = cache[pages, h]
    if factor is None:
        x = x.double()
    elif factor.dim() == 3:
        x = x.double() * factor[pages, h].double().unsqueeze(-1)
    else:
        y = torch.empty(x.shape[:-1] + (2 * x.shape[-1],), dtype=torch.float64, device=DEV)
        y[..., 0::2] = torch.remainder(x.double(), 16) - 8
        y[..., 1::2] = torch.floor(x.double() / 16) - 8
        x = y * torch.repeat_interleave(factor[pages, h].double(), GROUP, dim=-1)
    return x.reshape(-1, x.shape[-1])


def exact(case, seed):
    s = prepare(case, seed)
    op, B, d, Hkv = case["op"], case["B"], case["d"], case["Hkv"]
    G = case.get("group", 1)
    H = Hkv * G
    like = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=DEV)  # noqa: E731
    if op == "fwd":
        N = case["N"]
        o, lse = like(B, H, N, d), like(B, H, N)
        for b in range(B):
            for h in range(H):
                x, _ = _head_64(case, s, b, h)
                lse[b, h] = torch.logsumexp(x, -1)
                o[b, h] = x.sub_(lse[b, h, :, None]).exp_() @ s["v"][b, h // G].double()
        return {"o": o, "lse": lse}
    if op == "bwd":
        N = case["N"]
        dq, dk, dv = like(B, H, N, d), like(B, Hkv, N, d), like(B, Hkv, N, d)
        for b in range(B):
            for h in range(H):
                x, der = _head_64(case, s, b, h)
                p = x.sub_(s["lse"][b, h].double()[:, None]).exp_()
                q, k, v = s["q"][b, h].double(), s["k"][b, h // G].double(), s["v"][b, h // G].double()
                do = s["do"][b, h].double()
                dv[b, h // G] += p.T @ do
                y = do @ v.T
                y -= (do * s["o"][b, h].double()).sum(-1, keepdim=True)
                y *= p
                if der is not None:
                    y *= der
                dq[b, h] = s["scale"] * (y @ k)
                dk[b, h // G] += s["scale"] * (y.T @ q)
        return {"dq": dq, "dk": dk, "dv": dv}
    page = case["page"]
    if op == "decode":
        o = like(B, H, 1, d)
        lse = torch.full((B, H, 1), float("-inf"), dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["lens"].tolist()):
            lo = max(0, n - case["window"]) if case["window"] else 0
            if n <= lo:
                continue
            pages = s["table"][b, lo // page:-(-n // page)].long()
            cut = slice(lo - lo // page * page, n - lo // page * page)
            away = torch.arange(n - 1 - lo, -1, -1, device=DEV, dtype=torch.float64)
            for h in range(Hkv):
                k = _value_64(s["kc"], s["kd"], pages, h)[cut]
                v = _value_64(s["vc"], s["vd"], pages, h)[cut]
                heads = slice(h * G, (h + 1) * G)
                x = s["q"][b, heads, 0].double() @ k.T * s["scale"]
                if case["cap"]:
                    x = torch.tanh(x / case["cap"]) * case["cap"]
                if s["slopes"] is not None:
                    x = x - s["slopes"][heads].double()[:, None] * away
                l = torch.logsumexp(x, -1)
                o[b, heads, 0] = torch.exp(x - l[:, None]) @ v
                lse[b, heads, 0] = l
        return {"o": o, "lse": lse}
    start, count = s["start"].tolist(), s["count"].tolist()
    if op == "write":
        out = {}
        for new, cache, factor, name in ((s["k"], s["kc"], s["kd"], "k"), (s["v"], s["vc"], s["vd"], "v")):
            c, f = cache.clone(), factor.double()
            for b in range(B):
                n = torch.arange(start[b], start[b] + count[b], device=DEV)
                pg, row = s["table"][b].long()[n // page], n % page
                x = new[b, :, :count[b]].double().transpose(0, 1)
                a = x.abs().reshape(*x.shape[:-1], d // GROUP, GROUP).amax(-1)
                z = torch.where(a > 0, a, torch.ones_like(a)) / 7
                step = torch.exp2(torch.floor(torch.log2(z)) - 4)  # five bits: 16 .. 31 steps
                z = torch.clamp_min(torch.round(z / step) * step, 2.0 ** -120)
                z = torch.where(a > 0, z, torch.ones_like(z))
                f[pg, :, row] = z
                y = torch.round(x / torch.repeat_interleave(z, GROUP, dim=-1)).clamp_(-7, 7)
                c[pg, :, row] = (y[..., 0::2] + 8 + 16 * (y[..., 1::2] + 8)).to(torch.uint8)
            out[name + "_cache"], out[name + "_descale"] = c, f
        return out
    out = {}
    for cache, factor, name in ((s["kc"], s["kd"], "k"), (s["vc"], s["vd"], "v")):
        y = like(B, Hkv, case["T"], d)
        for b in range(B):
            for h in range(Hkv):
                if count[b]:
                    x = _value_64(cache, factor, s["table"][b].long(), h)
                    y[b, h, :count[b]] = x[start[b]:start[b] + count[b]]
        out[name] = y
    return out
