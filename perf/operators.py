"""The operators of a model's answering path, as a user calls them: rotary
positions on queries and keys (with their gradient, for training), the paged
key/value cache as it is written and read back, and the attention of one new
token over that cache.

Three families, told apart by a case's ``"op"``:

  decode      attention of the newest token of each sequence over its pages
  write/read  new keys and values into the pages (bf16, or e4m3 with a factor
              for every token and head), and rows of the pages back as bf16
  rope        q and k turned by their positions on one or several axes;
              ``"direction"`` says whether forward or gradient

Definitions used by the plain forms and by ``exact``:

  cache       [pages][Hkv][page_size][d]; position p of sequence b lives in
              page table[b][p // page_size], row p % page_size
  e4m3 row    descale = the smallest power of two with amax <= 448 descale
              (1 for a row of zeros), value = e4m3(x / descale), ties to even
  decode      s_j = scale <q, k_j> over the last `window` (0: all) of the
              sequence's `len` positions, o = softmax(s) v, l = logsumexp(s);
              no position: o = 0, l = -inf
  rope        pair i of head row x is (x[i], x[i + d/2]), or (x[2i], x[2i+1])
              when interleaved; it turns by angle pos[axis(i)] inv_freq[i],
              the gradient by minus that angle
"""

import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16
E4M3 = torch.float8_e4m3fn


# --------------------------------------------------------------------- cases
def listed():
    return [
        # One user's next token early in a chat: all latency.
        {"name": "decode_b1_h16_len500_d64", "op": "decode", "B": 1, "Hkv": 16, "group": 1, "d": 64,
         "page": 16, "len": 500, "ragged": False, "window": 0, "e4m3": False},
        # A serving batch of unequal chats, shared key heads.
        {"name": "decode_b16_kv8x4_4k_ragged", "op": "decode", "B": 16, "Hkv": 8, "group": 4, "d": 128,
         "page": 64, "len": 4096, "ragged": True, "window": 0, "e4m3": False},
        # One very long document: the length has to be split over the GPU.
        {"name": "decode_b1_kv8x4_128k", "op": "decode", "B": 1, "Hkv": 8, "group": 4, "d": 128,
         "page": 128, "len": 131072, "ragged": False, "window": 0, "e4m3": False},
        # A large batch over an 8-bit cache, the largest traffic.
        {"name": "decode_b32_kv8x8_8k_e4m3", "op": "decode", "B": 32, "Hkv": 8, "group": 8, "d": 128,
         "page": 64, "len": 8192, "ragged": True, "window": 0, "e4m3": True},
        # Sliding-window layers: only the last 4096 of 16384 positions count.
        {"name": "decode_b8_kv4x5_w4096_e4m3", "op": "decode", "B": 8, "Hkv": 4, "group": 5, "d": 64,
         "page": 32, "len": 16384, "ragged": True, "window": 4096, "e4m3": True},
        # A decode step's append: one token a sequence, rounded to 8 bits.
        {"name": "write_b64_t1_e4m3", "op": "write", "B": 64, "Hkv": 8, "d": 128, "page": 64, "T": 1,
         "before": 4000, "ragged": True, "e4m3": True},
        # A prompt's keys and values, padded batch, rounded to 8 bits.
        {"name": "write_b4_t8192_e4m3", "op": "write", "B": 4, "Hkv": 16, "d": 128, "page": 64, "T": 8192,
         "before": 0, "ragged": True, "e4m3": True},
        # A cached prefix back in bf16, for attention of the rest of a prompt.
        {"name": "read_b4_t8192_e4m3", "op": "read", "B": 4, "Hkv": 16, "d": 128, "page": 64, "T": 8192,
         "before": 0, "ragged": True, "e4m3": True},
        # A short prefix out of a bf16 cache.
        {"name": "read_b2_t700_d64", "op": "read", "B": 2, "Hkv": 4, "d": 64, "page": 16, "T": 700,
         "before": 100, "ragged": True, "e4m3": False},
        # A decode step's rotation, far into the text.
        {"name": "rope_b64_n1_h32kv8", "op": "rope", "direction": "fwd", "B": 64, "N": 1, "H": 32, "Hkv": 8,
         "d": 128, "axes": 1, "interleaved": False, "offset": 900000},
        # A video's tokens before attention: time, height and width.
        {"name": "rope_b1_n16384_h16_video", "op": "rope", "direction": "fwd", "B": 1, "N": 16384, "H": 16,
         "Hkv": 16, "d": 128, "axes": 3, "interleaved": False, "offset": 0},
        # The gradient of an image's rotation: height and width, neighbours paired.
        {"name": "rope_bwd_b2_n2047_h16_image", "op": "rope", "direction": "bwd", "B": 2, "N": 2047, "H": 16,
         "Hkv": 16, "d": 64, "axes": 2, "interleaved": True, "offset": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "write", "read", "rope", "rope"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if op == "decode":
        B, Hkv = _log(rng, 1, 64), rng.choice([1, 2, 3, 4, 8, 16])
        most = min(131072, 134000000 // (B * Hkv * d))
        return {"op": op, "B": B, "Hkv": Hkv, "group": rng.choice([1, 2, 4, 5, 8, 12, 16]), "d": d,
                "page": page, "len": _log(rng, 1, most), "ragged": rng.random() < 0.7,
                "window": rng.choice([0, 0, _log(rng, 1, 8192)]), "e4m3": rng.random() < 0.5}
    if op in ("write", "read"):
        B, Hkv = _log(rng, 1, 64), rng.choice([1, 2, 3, 4, 8, 16])
        most = min(16384, 60000000 // (B * Hkv * d))
        return {"op": op, "B": B, "Hkv": Hkv, "d": d, "page": page, "T": _log(rng, 1, most),
                "before": rng.choice([0, _log(rng, 1, 500)]), "ragged": rng.random() < 0.7,
                "e4m3": rng.random() < 0.7}
    B, H = _log(rng, 1, 64), rng.choice([1, 3, 8, 16, 32])
    Hkv = rng.choice([h for h in (1, 2, 3, 4, 8, 16, 32) if H % h == 0])
    return {"op": op, "direction": rng.choice(["fwd", "bwd"]), "B": B,
            "N": _log(rng, 1, min(16384, 66000000 // (B * (H + Hkv) * d))), "H": H, "Hkv": Hkv, "d": d,
            "axes": rng.choice([1, 2, 3]), "interleaved": rng.random() < 0.5,
            "offset": rng.choice([0, _log(rng, 1, 1000000)])}


# -------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(shape, g, dtype=BF16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


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
    """A page table for sequences of `lens` positions, pages in the order a
    pool hands them out after a while: shuffled.  The pool holds these
    sequences, or as many of `most` positions.  Returns (table, pages)."""
    need = [max(1, -(-int(n) // page)) for n in lens]
    total = max(sum(need), len(need) * -(-most // page)) + 3
    order = torch.randperm(total, generator=torch.Generator().manual_seed(int(seed) + 29)).to(torch.int32)
    table = torch.zeros((len(need), max(need)), dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table.to(DEV), total


def _pow2_descale(x):
    """[..., d] float32 -> the row's factor [...]: the smallest power of two
    with amax <= 448 descale, 1 for a row of zeros."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp_min(-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))


def _quantise(x):
    """bf16 [..., d] -> (float8_e4m3fn values [..., d], factors [...])."""
    x = x.float()
    s = _pow2_descale(x)
    return (x / s.unsqueeze(-1)).to(E4M3), s


def _cache(pages, Hkv, page, d, g, e4m3):
    """Key and value pages holding earlier tokens (some head channels larger
    than the rest, as trained keys have), with their factors or None."""
    gain = 1 + 3 * (torch.rand((Hkv, 1, d), generator=g, device=DEV) > 0.97).float()
    out = []
    for which in ("k", "v"):
        x = _randn((pages, Hkv, page, d), g)
        x = (x * gain).to(BF16) if which == "k" else x
        out.append(_quantise(x) if e4m3 else (x, None))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _rope_plan(case):
    """(sections, inv_freq [d/2] fp32, axis [d/2]): every axis has a ladder of
    its own frequencies 10000^(-j / pairs of that axis)."""
    half, A = case["d"] // 2, case["axes"]
    sections = {1: (half,), 2: (half // 2, half - half // 2),
                3: (half // 4, 3 * half // 8, half - half // 4 - 3 * half // 8)}[A]
    inv = torch.cat([10000.0 ** (-torch.arange(s, dtype=torch.float64) / s) for s in sections])
    axis = torch.cat([torch.full((s,), a, dtype=torch.long) for a, s in enumerate(sections)])
    return sections, inv.to(torch.float32).to(DEV), axis.to(DEV)


def _positions(case, seed):
    """int32 [axes, B, N]: running text, an image row by row, or a video frame
    by frame, each sequence from an offset of its own."""
    B, N, A = case["B"], case["N"], case["axes"]
    n = torch.arange(N)
    side = max(1, int(math.isqrt(N if A == 2 else max(1, N // 4))))
    ways = {1: [n], 2: [n // side, n % side], 3: [n // (side * side), n // side % side, n % side]}[A]
    start = torch.randint(0, 1 + case["offset"], (B, 1), generator=torch.Generator().manual_seed(int(seed) + 3))
    return torch.stack([w[None, :] + start for w in ways]).to(torch.int32).to(DEV)


def prepare(case, seed):
    g, op, d = _gen(seed), case["op"], case["d"]
    if op == "rope":
        B, N, H, Hkv = case["B"], case["N"], case["H"], case["Hkv"]
        sections, inv, axis = _rope_plan(case)
        s = {"op": op, "bwd": case["direction"] == "bwd", "interleaved": case["interleaved"],
             "sections": sections, "inv": inv, "axis": axis, "pos": _positions(case, seed)}
        if s["bwd"]:  # gradients as the attention's backward pass leaves them
            s["q"], s["k"] = _randn((B, H, N, d), g), _randn((B, Hkv, N, d), g)
        else:  # heads of one fused projection [B][N][heads][d]
            x = _randn((B, N, H + 2 * Hkv, d), g)
            s["q"], s["k"] = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2)
        return s
    B, Hkv, page, e4m3 = case["B"], case["Hkv"], case["page"], case["e4m3"]
    if op == "decode":
        lens = _lengths(B, case["len"], case["ragged"], seed)
    else:
        count = _lengths(B, case["T"], case["ragged"], seed, least=min(1, case["T"] - 1))
        before = _lengths(B, case["before"], case["ragged"], seed + 1, least=0) if case["before"] else count * 0
        lens = before + count
    table, pages = _table(lens, page, seed, 0 if op == "decode" else case["before"] + case["T"])
    kc, vc, kd, vd = _cache(pages, Hkv, page, d, g, e4m3)
    s = {"op": op, "kc": kc, "vc": vc, "kd": kd, "vd": vd, "table": table}
    if op == "decode":
        H = Hkv * case["group"]
        s.update(q=_randn((B, H, 1, d), g), lens=lens.to(DEV), window=case["window"], scale=1 / math.sqrt(d))
        return s
    s.update(T=case["T"], start=before.to(DEV), count=count.to(DEV))
    if op == "write":  # heads of one fused projection [B][T][heads][d]
        x = _randn((B, case["T"], 2 * Hkv, d), g)
        s["k"], s["v"] = x[:, :, :Hkv].transpose(1, 2), x[:, :, Hkv:].transpose(1, 2)
    return s


# --------------------------------------------------------------- plain forms
def _rows(s, pos):
    """(page, row) of positions pos [B, T]."""
    page = s["kc"].shape[2]
    at = (pos // page).clamp(0, s["table"].shape[1] - 1).long()
    return torch.gather(s["table"], 1, at).long(), (pos % page).long()


def _fetch(cache, factor, pg, row):
    """fp32 [B, Hkv, T, d] of the rows (pg, row) [B, T]."""
    x = (cache.view(torch.uint8) if factor is not None else cache)[pg, :, row]
    if factor is not None:
        x = x.view(E4M3).float() * factor[pg, :, row].unsqueeze(-1)
    return x.float().transpose(1, 2)


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
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    v = _fetch(s["vc"], s["vd"], pg, row) * seen[:, None, :, None]
    o = torch.matmul(p, v) / torch.where(z > 0, z, torch.ones_like(z))
    return {"o": o.view(B, H, 1, d).to(BF16), "lse": (m + torch.log(z)).view(B, H, 1)}


def _plain_write(s):
    T = s["T"]
    t = torch.arange(T, device=DEV).unsqueeze(0)
    count = s["count"].long().unsqueeze(1)
    # a token past its sequence's count is the last one of the count again,
    # and an empty sequence writes back what its first row holds
    src = torch.minimum(t, (count - 1).clamp_min(0))
    some = (count > 0).expand(-1, T)
    pg, row = _rows(s, s["start"].long().unsqueeze(1) + src)
    out = {}
    for new, cache, factor, name in ((s["k"], s["kc"], s["kd"], "k"), (s["v"], s["vc"], s["vd"], "v")):
        x = torch.gather(new.transpose(1, 2), 1, src[:, :, None, None].expand(-1, -1, new.shape[1], new.shape[3]))
        flat, keep = cache, some[:, :, None, None]
        if factor is not None:
            x, f = _quantise(x)
            x, flat = x.view(torch.uint8), cache.view(torch.uint8)
            factor[pg, :, row] = torch.where(some[:, :, None], f, factor[pg, :, row])
            out[name + "_descale"] = factor
        flat[pg, :, row] = torch.where(keep, x, flat[pg, :, row])
        out[name + "_cache"] = cache
    return out


def _plain_read(s):
    t = torch.arange(s["T"], device=DEV).unsqueeze(0)
    inside = (t < s["count"].unsqueeze(1))[:, None, :, None]
    pg, row = _rows(s, s["start"].long().unsqueeze(1) + t)
    pick = lambda c, f: torch.where(inside, _fetch(c, f, pg, row), torch.zeros((), device=DEV)).to(BF16)  # noqa: E731
    return {"k": pick(s["kc"], s["kd"]), "v": pick(s["vc"], s["vd"])}


def _plain_rope(s):
    # angles in 64 bits: positions near 2^20 times a frequency need more than 24
    angle = s["pos"][s["axis"]].permute(1, 2, 0).double() * s["inv"].double()
    if s["bwd"]:
        angle = -angle
    c, n = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    out = []
    for x in (s["q"], s["k"]):
        x = x.float()
        half = x.shape[-1] // 2
        a, b = (x[..., 0::2], x[..., 1::2]) if s["interleaved"] else (x[..., :half], x[..., half:])
        y = (a * c - b * n, b * c + a * n)
        out.append((torch.stack(y, -1).flatten(-2) if s["interleaved"] else torch.cat(y, -1)).to(BF16))
    return {"q": out[0], "k": out[1]}


# ----------------------------------------------------------------------- run
def run(state):
    s = state
    if own:
        import attention_backward_pass_attn_gb300 as attn

        if s["op"] == "decode":
            o, lse = attn.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], scale=s["scale"],
                                      k_descale=s["kd"], v_descale=s["vd"], window=s["window"])
            return {"o": o, "lse": lse}
        if s["op"] == "write":
            attn.kv_cache_write(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["start"], count=s["count"],
                                k_descale=s["kd"], v_descale=s["vd"])
            out = {"k_cache": s["kc"], "v_cache": s["vc"]}
            return out if s["kd"] is None else dict(out, k_descale=s["kd"], v_descale=s["vd"])
        if s["op"] == "read":
            k, v = attn.kv_cache_read(s["kc"], s["vc"], s["table"], s["start"], s["T"], count=s["count"],
                                      k_descale=s["kd"], v_descale=s["vd"])
            return {"k": k, "v": v}
        turn = attn.rope_bwd if s["bwd"] else attn.rope_fwd
        q, k = turn(s["q"], s["k"], s["pos"], s["inv"], sections=s["sections"], interleaved=s["interleaved"])
        return {"q": q, "k": k}
    return {"decode": _plain_decode, "write": _plain_write, "read": _plain_read, "rope": _plain_rope}[s["op"]](s)


# ---------------------------------------------------------------------- work
def work(case):
    """Expected lengths stand in for the drawn ones: a ragged batch has one
    sequence at the longest and the others at half of it."""
    B, d = case["B"], case["d"]
    if case["op"] == "rope":
        n = B * case["N"] * (case["H"] + case["Hkv"]) * d
        return {"bytes": 4 * n + 4 * case["axes"] * B * case["N"] + 2 * d, "flops": 3 * n}
    Hkv = case["Hkv"]
    most = case["len"] if case["op"] == "decode" else case["T"]
    others = B - 1 - (1 if B >= 8 else 0)
    tokens = most + others * most // 2 if case["ragged"] else B * most
    row = d + 4 if case["e4m3"] else 2 * d
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
def _e4m3_64(x):
    """float64 -> the nearest e4m3 values (ties to even, at most 448)."""
    a = x.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a)))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return torch.sign(x) * torch.clamp_max(torch.round(a / step) * step, 448.0)


def _value_64(cache, factor, pages, h):
    """float64 [positions, d] of head h on the pages of one sequence, in order."""
    x = cache[pages, h].double()
    if factor is not None:
        x = x * factor[pages, h].double().unsqueeze(-1)
    return x.reshape(-1, x.shape[-1])


def exact(case, seed):
    s = prepare(case, seed)
    op, B, d = case["op"], case["B"], case["d"]
    if op == "rope":
        out = {}
        turns = s["pos"].double()
        for name in ("q", "k"):
            x = s[name].double()
            y = torch.empty(x.shape, dtype=torch.float64, device=DEV)
            for i in range(d // 2):
                a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + d // 2)
                z = turns[int(s["axis"][i])] * s["inv"][i].double() * (-1 if s["bwd"] else 1)
                co, si = torch.cos(z)[:, None], torch.sin(z)[:, None]
                y[..., a] = co * x[..., a] - si * x[..., b]
                y[..., b] = si * x[..., a] + co * x[..., b]
            out[name] = y
        return out
    page = case["page"]
    Hkv = case["Hkv"]
    if op == "decode":
        H, G = Hkv * case["group"], case["group"]
        o = torch.zeros((B, H, 1, d), dtype=torch.float64, device=DEV)
        lse = torch.full((B, H, 1), float("-inf"), dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["lens"].tolist()):
            lo = max(0, n - case["window"]) if case["window"] else 0
            if n <= lo:
                continue
            pages = s["table"][b, lo // page:-(-n // page)].long()
            cut = slice(lo - lo // page * page, n - lo // page * page)
            for h in range(Hkv):
                k = _value_64(s["kc"], s["kd"], pages, h)[cut]
                v = _value_64(s["vc"], s["vd"], pages, h)[cut]
                x = s["q"][b, h * G:(h + 1) * G, 0].double() @ k.T * s["scale"]
                l = torch.logsumexp(x, -1)
                o[b, h * G:(h + 1) * G, 0] = torch.exp(x - l[:, None]) @ v
                lse[b, h * G:(h + 1) * G, 0] = l
        return {"o": o, "lse": lse}
    start, count = s["start"].tolist(), s["count"].tolist()
    if op == "write":
        out = {}
        for new, cache, factor, name in ((s["k"], s["kc"], s["kd"], "k"), (s["v"], s["vc"], s["vd"], "v")):
            c = cache.double()
            f = None if factor is None else factor.double()
            for b in range(B):
                n = torch.arange(start[b], start[b] + count[b], device=DEV)
                pg, row = s["table"][b].long()[n // page], n % page
                x = new[b, :, :count[b]].double().transpose(0, 1)
                if f is not None:
                    a = x.abs().amax(-1)
                    e = torch.ceil(torch.log2(torch.where(a > 0, a, torch.ones_like(a)) / 448))
                    z = torch.where(a > 0, torch.exp2(e), torch.ones_like(a))
                    f[pg, :, row] = z
                    x = _e4m3_64(x / z.unsqueeze(-1))
                c[pg, :, row] = x
            out[name + "_cache"] = c
            if f is not None:
                out[name + "_descale"] = f
        return out
    out = {}
    for cache, factor, name in ((s["kc"], s["kd"], "k"), (s["vc"], s["vd"], "v")):
        y = torch.zeros((B, Hkv, case["T"], d), dtype=torch.float64, device=DEV)
        for b in range(B):
            for h in range(Hkv):
                if count[b]:
                    x = _value_64(cache, factor, s["table"][b].long(), h)
                    y[b, h, :count[b]] = x[start[b]:start[b] + count[b]]
        out[name] = y
    return out
