"""Attention of one new token over 4-bit caches, and with changed scores over
caches of every type, against the fp64 oracle within bounds that count every
rounding; and the whole path, from a prompt's attention to the next token's."""

import math

import numpy as np
import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab
from attention_backward_pass_attn_gb300.inputs import make_tensor
from oracle import int4
from oracle import score as so
from serving_cases import cuda, filled_cache, page_table, rows_held

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from attention_backward_pass_attn_gb300 import build as abuild

    abuild.build()
    ab.load_library()
    assert ab.attn_last_device_error() == ab.ATTN_OK
    yield
    assert ab.attn_last_device_error() == ab.ATTN_OK


def int4_cache(lens, page, Hkv, d, seed, std=1.0):
    """As serving_cases.filled_cache, in four bits: rows that no position falls
    on hold arbitrary codes and NaN factors."""
    table, P = page_table(lens, page, seed)
    held = rows_held(table, lens, page, P)
    out = {"table": table, "P": P}
    rng = np.random.default_rng(seed)
    for n in "kv":
        b = rng.integers(0, 256, size=(P, Hkv, page, d // 2)).astype(np.uint8)
        b = np.where((b & 15) == 0, b | 1, b)       # codes from -7 on
        b = np.where((b >> 4) == 0, b | 0x10, b)
        f = np.exp2(rng.integers(-5, 1, size=(P, Hkv, page, d // 32))) \
            * rng.integers(16, 32, size=(P, Hkv, page, d // 32)) / 64 * std
        out[n + "64"] = int4.values(b, f)
        f = np.where(held[:, None, :, None], f, np.nan)
        out[n + "c"], out[n + "d"] = torch.from_numpy(b), torch.from_numpy(f).to(torch.bfloat16)
    return out


def cache_of(kind, lens, page, Hkv, d, seed, std=1.0):
    return int4_cache(lens, page, Hkv, d, seed, std) if kind == "int4" else \
        filled_cache(lens, page, Hkv, d, seed, kind == "e4m3", std=std)


def check(kind, lens, Hkv, group, d, page, window=0, cap=0.0, slopes=None, seed=0, q_std=2.0):
    c = cache_of(kind, lens, page, Hkv, d, seed + 5)
    B, H = len(lens), Hkv * group
    q = make_tensor((B, H, 1, d), seed + 3, std=q_std)
    sl = None
    if slopes is not None:
        sl = torch.tensor([slopes * 2.0 ** (-8.0 * (h + 1) / H) for h in range(H)])
    scale = 1 / math.sqrt(d)
    args = (q.cuda(), c["kc"].cuda(), c["vc"].cuda(), c["table"].cuda(),
            torch.tensor(lens, dtype=torch.int32).cuda())
    kw = dict(k_descale=cuda(c["kd"]), v_descale=cuda(c["vd"]), window=window, softcap=cap,
              slopes=cuda(sl))
    o, lse = ab.attn_decode(*args, **kw)
    ref = so.decode(q, c["k64"], c["v64"], c["table"], lens, scale, window, cap, sl)
    got_o, got_l = o.double().cpu().numpy()[:, :, 0], lse.double().cpu().numpy()[:, :, 0]
    none = np.isneginf(ref["L"])
    assert np.array_equal(np.isneginf(got_l), none) and not got_o[none].any()
    assert np.all(np.isfinite(got_o))
    off = np.abs(got_l[~none] - ref["L"][~none]) / ref["dL"][~none]
    assert off.max(initial=0.0) <= 1.0, "L: %.3f of its bound" % off.max()
    off = np.abs(got_o - ref["O"])[~none] / ref["dO"][~none]
    assert off.max(initial=0.0) <= 1.0, "O: %.3f of its bound" % off.max()
    again = ab.attn_decode(*args, **kw)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)  # bit for bit


SHAPES = [
    # Hkv, group, d, page, lens, window
    (1, 1, 64, 16, [1], 0),
    (1, 1, 128, 16, [2], 0),
    (2, 4, 128, 16, [15, 16, 17], 0),
    (1, 8, 64, 32, [0, 1, 0, 63, 64, 65, 31, 0], 0),
    (3, 5, 64, 48, [100, 7, 129], 0),
    (2, 2, 128, 64, [0, 0], 0),
    (2, 12, 128, 64, [200, 333], 0),
    (1, 40, 128, 32, [70, 300], 0),
    (16, 1, 64, 16, [500], 0),
    (2, 4, 128, 256, [1000, 1, 257], 0),
    (2, 4, 128, 16, [300, 299, 20, 5], 17),
    (1, 3, 64, 32, [500, 64, 33, 1], 1),
    (2, 8, 64, 48, [257, 256, 255, 0], 100),
    (2, 9, 128, 48, [640, 90], 2 ** 40),
]


@pytest.mark.parametrize("Hkv,group,d,page,lens,window", SHAPES)
def test_int4(Hkv, group, d, page, lens, window):
    check("int4", lens, Hkv, group, d, page, window, seed=sum(lens) + d)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("Hkv,group,d,page,lens,window", SHAPES)
def test_cap_and_slopes(Hkv, group, d, page, lens, window, kind):
    check(kind, lens, Hkv, group, d, page, window, cap=6.0, slopes=1.0, seed=sum(lens) + d, q_std=4.0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("cap,slopes,q_std", [
    (0.0, 1.0, 2.0), (0.0, -0.02, 2.0), (0.0, 300.0, 2.0), (30.0, None, 8.0), (1e-3, None, 2.0),
    (1e30, None, 2.0), (50.0, None, 0.05), (2.0, 0.0, 20.0)])
def test_changes(cap, slopes, q_std, kind):
    check(kind, [700, 33], 2, 4, 128, 64, cap=cap, slopes=slopes, q_std=q_std)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("Hkv,group,d,lens", [
    (1, 1, 64, [9000]), (1, 2, 128, [6000, 0, 2500]), (2, 4, 128, [4001, 3, 0, 130]),
    (1, 13, 128, [3001, 5])])
def test_long_sequences_are_split_and_joined(Hkv, group, d, lens, kind):
    check(kind, lens, Hkv, group, d, 32, cap=9.0, slopes=0.1, q_std=3.0)
    check("int4", lens, Hkv, group, d, 32)


@pytest.mark.parametrize("d", [64, 128])
def test_int4_is_the_bf16_cache_of_its_values(d):
    """The values a 4-bit cache stands for are bf16 numbers: attention over
    them in a bf16 cache differs by fp32 rounding alone."""
    lens, Hkv, group, page = [900, 77], 2, 4, 64
    c = int4_cache(lens, page, Hkv, d, 9)
    held = torch.from_numpy(rows_held(c["table"], lens, page, c["P"]))[:, None, :, None]
    q = make_tensor((2, Hkv * group, 1, d), 3, std=2.0).cuda()
    tail = (c["table"].cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    o, lse = ab.attn_decode(q, c["kc"].cuda(), c["vc"].cuda(), *tail, k_descale=c["kd"].cuda(),
                            v_descale=c["vd"].cuda())
    wide = [torch.where(held, torch.from_numpy(c[n + "64"]), torch.tensor(0.0).double())
            .to(torch.bfloat16).cuda() for n in "kv"]
    o2, lse2 = ab.attn_decode(q, *wide, *tail)
    assert float((lse - lse2).abs().max()) <= 2e-5
    assert float((o.float() - o2.float()).abs().max()) <= 2 ** -8 * float(o2.abs().max()) + 1e-6


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[900, 77], [9000, 1]])
@pytest.mark.parametrize("e", [-112, -30, 13, 100])
def test_int4_factors_of_any_size(e, lens, d):
    """Powers of two at K's factors and off the scale leave every bit; at V's
    they come out again.  (Around factors of 0.4: those of 2^-110 to 2^11 and
    the others take different paths.)"""
    Hkv, group, page = 2, 4, 64
    c = int4_cache(lens, page, Hkv, d, 11)
    q = make_tensor((2, Hkv * group, 1, d), 12, std=2.0).cuda()
    args = (q, c["kc"].cuda(), c["vc"].cuda(), c["table"].cuda(),
            torch.tensor(lens, dtype=torch.int32).cuda())
    kd, vd = c["kd"].cuda(), c["vd"].cuda()
    o, lse = ab.attn_decode(*args, scale=0.125, k_descale=kd, v_descale=vd)
    o1, lse1 = ab.attn_decode(*args, scale=0.125 * 2.0 ** -e, k_descale=kd * 2.0 ** e, v_descale=vd)
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    o2, lse2 = ab.attn_decode(*args, scale=0.125, k_descale=kd, v_descale=vd * 2.0 ** e)
    assert torch.equal(lse, lse2)
    # At V's 2^-112 results below 2^-126 are bf16 numbers of steps of 2^-133, off
    # by 2^-134, 2^-22 of what they are times 2^112; and terms of weights of 2^-20
    # and less end at fp32's 2^-149, 2 x 9000 of them 2^-37 each at most, 2^-22
    # too, which may change a result by a step.
    step = (o2.double() * 2.0 ** -e - o.double()).abs()
    assert bool((step <= (2 ** -7 * o.double().abs() + 2 ** -21 if e < -100 else 0)).all())
    # one row alone outside, and the same in a bf16 cache of the values
    at = (int(c["table"][0, 40 // page]), 1, 40 % page)
    kd, vd = kd.clone(), vd.clone()
    kd[at] *= 2.0 ** min(e, 12)
    vd[at] *= 2.0 ** min(e, 20)
    o, lse = ab.attn_decode(*args, scale=2.0 ** -14, k_descale=kd, v_descale=vd)
    held = torch.from_numpy(rows_held(c["table"], lens, page, c["P"]))[:, None, :, None].cuda()
    both = []
    for codes, f in ((args[1], kd), (args[2], vd)):
        n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double() - 8
        x = n * f.double().repeat_interleave(32, -1)
        both.append(torch.where(held, x, 0.0).to(torch.bfloat16))
    o2, lse2 = ab.attn_decode(q, *both, *args[3:], scale=2.0 ** -14)
    assert float((lse - lse2).abs().max()) <= 2e-5
    assert float((o.float() - o2.float()).abs().max()) <= 2 ** -8 * float(o2.abs().max()) + 1e-6


def test_special_values_in_an_int4_cache():
    """A NaN factor at a visible position shows where it counts, and only there."""
    lens, Hkv, d, page = [100], 2, 64, 16
    c = int4_cache(lens, page, Hkv, d, 4)
    q = make_tensor((1, 4, 1, d), 5).cuda()
    at = (int(c["table"][0, 50 // page]), 1, 50 % page)

    def run(name, group):
        f = {n: c[n].clone() for n in ("kd", "vd")}
        f[name][at + (group,)] = float("nan")
        return ab.attn_decode(q, c["kc"].cuda(), c["vc"].cuda(), c["table"].cuda(),
                              torch.tensor(lens, dtype=torch.int32).cuda(), k_descale=f["kd"].cuda(),
                              v_descale=f["vd"].cuda())
    o, lse = run("kd", 0)
    assert not torch.isnan(o[:, :2]).any() and torch.isnan(o[:, 2:]).all()
    assert torch.isnan(lse[:, 2:]).all() and not torch.isnan(lse[:, :2]).any()
    o, lse = run("vd", 1)
    assert not torch.isnan(lse).any() and not torch.isnan(o[:, :2]).any()
    assert not torch.isnan(o[:, 2:, :, :32]).any() and torch.isnan(o[:, 2:, :, 32:]).all()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float8_e4m3fn, "int4"])
@pytest.mark.parametrize("how", [dict(softcap=20.0), dict(slopes=True), dict(softcap=10.0, slopes=True, window=90)])
def test_a_prompt_and_its_next_tokens(kind, how):
    """A capped model answers: the prompt's keys and values go into the cache,
    attn_fwd_score runs over what the cache holds, and every further token's
    attn_decode is the last row that attn_fwd_score gives for the longer text."""
    B, Hq, Hkv, d, page, N, more = 2, 8, 2, 128, 32, 150, 4
    how = dict(how)
    if how.get("slopes"):
        how["slopes"] = torch.tensor([2.0 ** -(h + 1) for h in range(Hq)], device="cuda")
    table, P = page_table([N + more] * B, page, 6)
    table = table.cuda()
    cache = ab.alloc_kv_cache(P, Hkv, page, d, "cuda", kind)
    fac = dict(k_descale=cache[2], v_descale=cache[3])
    g = torch.Generator().manual_seed(2)
    q, k, v = ((torch.randn((B, h, N + more, d), generator=g) * s).to(torch.bfloat16).cuda()
               for h, s in ((Hq, 3.0), (Hkv, 1.0), (Hkv, 1.0)))
    at = lambda n: torch.full((B,), n, dtype=torch.int32, device="cuda")  # noqa: E731
    ab.kv_cache_write(k[:, :, :N], v[:, :, :N], cache[0], cache[1], table, at(0), **fac)
    for t in range(N, N + more):
        ab.kv_cache_write(k[:, :, t:t + 1], v[:, :, t:t + 1], cache[0], cache[1], table, at(t), **fac)
        o, lse = ab.attn_decode(q[:, :, t:t + 1].contiguous(), cache[0], cache[1], table, at(t + 1),
                                **fac, **how)
        held = ab.kv_cache_read(cache[0], cache[1], table, at(0), t + 1, **fac)
        ref, refl = ab.attn_fwd_score(q[:, :, :t + 1], *held, causal=True, **how)
        # either side's own roundings: the prompt's P meets V in bf16 (2^-8 of
        # sum p |v|), its result and the token's are rounded to bf16 (2^-8);
        # scores of some tens off by fp32 steps
        room = 2 ** -8 * (held[1].abs().amax(2).repeat_interleave(Hq // Hkv, 1) + 2 * ref[:, :, -1].abs())
        assert bool(((o[:, :, 0] - ref[:, :, -1]).abs().float() <= room.float()).all())
        assert float((lse[:, :, 0] - refl[:, :, -1]).abs().max()) <= 1e-4


def test_gradients_reach_through_the_prompt():
    """A training step of the same model: forward and backward of what the
    answering path above runs, rotated first."""
    B, Hq, Hkv, N, d = 1, 4, 2, 130, 64
    g = torch.Generator().manual_seed(8)
    x = (torch.randn((B, N, Hq + 2 * Hkv, d), generator=g)).to(torch.bfloat16).cuda()
    q, k, v = (t.transpose(1, 2) for t in x.split((Hq, Hkv, Hkv), dim=2))
    pos = torch.arange(N, dtype=torch.int32, device="cuda").view(1, 1, N)
    inv = (10000.0 ** (-torch.arange(d // 2) / (d // 2))).float().cuda()
    qr, kr = ab.rope_fwd(q, k, pos, inv)
    kw = dict(causal=True, softcap=15.0)
    o, lse = ab.attn_fwd_score(qr, kr, v, **kw)
    do = torch.randn((B, Hq, N, d), generator=g).to(torch.bfloat16).cuda()
    dq, dk, dv = ab.attn_bwd_score(qr, kr, v, o, do, lse, **kw)
    ref = so.backward(qr, kr, v, o, do, lse, scale=1 / math.sqrt(d), cap=15.0)
    for t, n in ((dq, "Q"), (dk, "K"), (dv, "V")):
        assert np.all(np.abs(t.double().cpu().numpy() - ref["d" + n]) <= ref["e" + n])
    dq, dk = ab.rope_bwd(dq, dk, pos, inv)
    assert dq.shape == q.shape and dk.shape == k.shape


@pytest.mark.parametrize("kind", ["bf16", "int4"])
def test_captured_calls_replay_on_new_lengths(kind):
    lens, Hkv, d, page = [300, 40], 2, 64, 16
    c = cache_of(kind, lens, page, Hkv, d, 12)
    q = make_tensor((2, 8, 1, d), 5).cuda()
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    dev = [cuda(c[x]) for x in ("kc", "vc", "kd", "vd", "table")]
    run = lambda: ab.attn_decode(q, dev[0], dev[1], dev[4], n, k_descale=dev[2],  # noqa: E731
                                 v_descale=dev[3], softcap=5.0)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = run()
    for now in ([300, 40], [17, 0], [1, 39]):
        n.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        want = run()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
