"""Attention of one new token over the paged cache on the GPU against the fp64
oracle.

Tolerances.  With n visible positions, A = sum_j p_j |v_j| and
S = max_j scale sum_i |q_i k_ji|:

- a score is a sum of d products of exact factors in fp32 (each step off by at
  most 2^-23 of the running size, which S bounds), then scaled and shifted in
  fp32, and 2^x is good to 2^-22 relative: |ds| <= e = ((d + 8) 2^-23 + 2^-22) S;
- L: e, plus the rounding of a sum of n terms (n 2^-24) and of the result
  (2^-22 |L| with the two logarithms' constants): e + n 2^-24 + 2^-22 (1 + |L|);
- O: weights off by 2 e + n 2^-23 together with their sum, their rounding
  before the product with v (2^-11 at most), the accumulation (n 2^-23), all
  times A; then one rounding to bf16, 2^-8 |O|.
"""

import math

import numpy as np
import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab
from attention_backward_pass_attn_gb300.inputs import make_tensor
from oracle import serving
from serving_cases import cuda, filled_cache

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


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def run(q, c, lens, **kw):
    return ab.attn_decode(q.cuda(), cuda(c["kc"]), cuda(c["vc"]), c["table"].cuda(),
                          i32(lens).cuda(), k_descale=cuda(c["kd"]), v_descale=cuda(c["vd"]), **kw)


def check(o, lse, ref, d):
    o, lse = f64(o)[:, :, 0], f64(lse)[:, :, 0]
    n = ref["n"][:, None]
    e = ((d + 8) * 2.0 ** -23 + 2.0 ** -22) * ref["S"]
    some = np.broadcast_to(n > 0, lse.shape)
    assert np.all(np.isneginf(lse[~some])) and np.all(o[~some] == 0)
    tol_l = e + n * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(np.where(some, ref["L"], 0)))
    dl = np.abs(lse[some] - ref["L"][some])
    assert np.all(dl <= tol_l[some]), "L off by %.2e" % dl.max()
    rel = (2 * e + n * 2.0 ** -22 + 2.0 ** -11)[..., None]
    do = np.abs(o - ref["O"])
    tol = np.abs(ref["O"]) * 2.0 ** -8 + rel * ref["A"] * (1 + 2.0 ** -8)
    assert np.all(do <= tol), "O off by %.2e" % do.max()


CASES = [
    # Hkv, group, d, page, lens, window
    (1, 1, 64, 16, [1], 0),
    (1, 1, 128, 16, [2], 0),
    (2, 4, 128, 16, [15, 16, 17], 0),
    (1, 8, 64, 32, [0, 1, 0, 63, 64, 65, 31, 0], 0),
    (3, 5, 64, 48, [100, 7, 129], 0),
    (2, 2, 128, 64, [0, 0], 0),
    (2, 12, 128, 64, [200, 333], 0),
    (1, 16, 64, 128, [513], 0),
    (1, 40, 128, 32, [70, 300], 0),
    (2, 33, 64, 16, [90], 0),
    (16, 1, 64, 16, [500], 0),
    (2, 4, 128, 256, [1000, 1], 0),
    (2, 4, 128, 16, [300, 299, 20, 5], 17),
    (1, 3, 64, 32, [500, 64, 33, 1], 1),
    (2, 8, 64, 48, [257, 256, 255, 0], 100),
    (1, 2, 128, 64, [700, 90], 5000),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hkv,group,d,page,lens,window", CASES)
def test_decode_against_the_oracle(Hkv, group, d, page, lens, window, fp8):
    """Every row that no visible position falls on is NaN, and page-table
    entries that no position needs name no page."""
    seed = 700 + 10 * sum(lens) + d + group
    B, Hq = len(lens), Hkv * group
    c = filled_cache(lens, page, Hkv, d, seed, fp8)
    q = make_tensor((B, Hq, 1, d), seed + 3, std=2.0)
    if window:  # what the window hides may hold anything
        for b, n in enumerate(lens):
            for p in range(0, max(0, n - window)):
                at = (int(c["table"][b, p // page]), slice(None), p % page)
                if fp8:
                    c["kc"].view(torch.uint8)[at] = 0x7F
                    c["vc"].view(torch.uint8)[at] = 0xFF
                    c["kd"][at], c["vd"][at] = float("inf"), float("nan")
                else:
                    c["kc"][at], c["vc"][at] = float("nan"), float("-inf")
    scale = 1 / math.sqrt(d)
    o, lse = run(q, c, lens, window=window)
    check(o, lse, serving.decode(q, c["k64"], c["v64"], c["table"], lens, scale, window), d)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_split_over_a_long_sequence(fp8):
    """One long sequence beside short and empty ones: the long one is split
    over many blocks and joined, the others are not."""
    lens, Hkv, group, d, page = [4001, 3, 0, 130, 1500], 2, 4, 128, 64
    c = filled_cache(lens, page, Hkv, d, 77, fp8)
    q = make_tensor((len(lens), Hkv * group, 1, d), 78, std=3.0)
    o, lse = run(q, c, lens)
    ref = serving.decode(q, c["k64"], c["v64"], c["table"], lens, 1 / math.sqrt(d))
    check(o, lse, ref, d)
    o2, lse2 = run(q, c, lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # bit for bit


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hkv,group,d,lens", [
    (1, 1, 64, [9000]), (1, 1, 128, [6000, 0, 2500]), (1, 2, 128, [5000]), (2, 2, 64, [9001, 70]),
    (1, 3, 64, [7777]), (1, 6, 128, [5003]), (1, 13, 128, [3001, 5]), (3, 4, 128, [3500])])
def test_decode_many_parts(Hkv, group, d, lens, fp8):
    """Few heads and long sequences: dozens of blocks share a head, and their
    parts are joined in two steps."""
    c = filled_cache(lens, 32, Hkv, d, 60 + group, fp8)
    q = make_tensor((len(lens), Hkv * group, 1, d), 61 + group, std=2.0)
    o, lse = run(q, c, lens)
    check(o, lse, serving.decode(q, c["k64"], c["v64"], c["table"], lens, 1 / math.sqrt(d)), d)
    for _ in range(3):
        o2, lse2 = run(q, c, lens)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_large_scores(fp8):
    """Scores of several hundred, one key far above the rest, and factors of
    very different sizes: nothing overflows."""
    lens, Hkv, group, d, page = [260, 70], 1, 4, 64, 16
    c = filled_cache(lens, page, Hkv, d, 5, fp8, std=8.0)
    q = make_tensor((2, 4, 1, d), 6, std=8.0)
    if fp8:
        c["vd"][c["vd"].isfinite()] *= 1e-3
        rows = c["table"][0, :4]
        c["vd"][rows[1]] *= 1e6
        c["v64"] = serving.cache_values(c["vc"], c["vd"])
    o, lse = run(q, c, lens, scale=1.0)
    check(o, lse, serving.decode(q, c["k64"], c["v64"], c["table"], lens, 1.0), d)


def test_decode_factors_of_any_size():
    """A huge row that the softmax leaves almost out, rows of zeros with factor
    1 among tiny ones, and a range of 2^90 between factors: the small rows'
    part of the output is as exact as if they stood alone."""
    lens, Hkv, d, page = [96, 96, 96], 1, 64, 16
    c = filled_cache(lens, page, Hkv, d, 55, True)
    q = make_tensor((3, 4, 1, d), 56)
    held = c["table"][:, :6].long()
    for b in range(3):
        c["vd"][held[b]] *= 2.0 ** -60 if b == 2 else 2.0 ** -40
    # sequence 0: position 5 has a value of 2^0 and a weight of about e^-100
    at = (held[0, 0], 0, 5)
    c["vd"][at] = 1.0
    c["kc"].view(torch.uint8)[at] = torch.from_numpy(serving.nearest_e4m3(-np.sign(f64(q)[0, 0, 0])))
    c["kd"][at] = 100 * 8 / float(np.abs(f64(q)[0, 0, 0]).sum())
    # sequence 1: every third row is zeros, factor 1; sequence 2: one row of 2^30
    for p in range(0, 96, 3):
        z = (held[1, p // page], 0, p % page)
        c["vc"].view(torch.uint8)[z] = 0
        c["vd"][z] = 1.0
    c["vd"][held[2, 3], 0, 7] = 2.0 ** 30
    c["k64"] = serving.cache_values(c["kc"], c["kd"])
    c["v64"] = serving.cache_values(c["vc"], c["vd"])
    o, lse = run(q, c, lens)
    check(o, lse, serving.decode(q, c["k64"], c["v64"], c["table"], lens, 1 / 8), d)


def test_decode_nan_and_inf_of_visible_rows_show():
    """A NaN or infinity at a visible position reaches the heads that read it,
    and no others."""
    lens, Hkv, group, d, page = [50, 50], 2, 2, 64, 16
    for fp8 in (False, True):
        c = filled_cache(lens, page, Hkv, d, 15, fp8)
        at = (int(c["table"][0, 1]), 0, 3)
        if fp8:
            c["kc"].view(torch.uint8)[at][5] = 0x7F
        else:
            c["kc"][at][5] = float("nan")
        q = make_tensor((2, 4, 1, d), 16)
        o, lse = run(q, c, lens)
        assert torch.isnan(o[0, :2]).all() and torch.isnan(lse[0, :2]).all()
        assert torch.isfinite(o[0, 2:]).all() and torch.isfinite(o[1]).all()
        c = filled_cache(lens, page, Hkv, d, 15, fp8)
        qn = q.clone()
        qn[1, 3, 0, 7] = float("nan")
        o, lse = run(qn, c, lens)
        assert torch.isnan(o[1, 3]).all() and torch.isnan(lse[1, 3]).all()
        assert torch.isfinite(o[1, :3]).all() and torch.isfinite(o[0]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_queries_of_any_magnitude(fp8, d):
    """Heads of one sequence from zero over subnormal numbers to ordinary ones,
    large and tiny elements in one head; an infinite element leaves the other
    heads bit for bit."""
    lens, Hkv, group, page = [90, 300], 2, 8, 16
    c = filled_cache(lens, page, Hkv, d, 17, fp8)
    q = make_tensor((2, Hkv * group, 1, d), 18)
    for h, e in enumerate([None, -133, -126, -100, -40, -14, -3, 0] * 2):
        q[:, h] = 0 if e is None else (q[:, h].double() * 2.0 ** e).to(q.dtype)
    q[:, 9, :, ::2] *= 2.0 ** -60
    q[:, 10, :, 1::3] *= 2.0 ** 8
    o, lse = run(q, c, lens)
    check(o, lse, serving.decode(q, c["k64"], c["v64"], c["table"], lens, d ** -0.5), d)
    bad = q.clone()
    bad[1, 5, 0, 6], bad[1, 12, 0, d - 1] = float("inf"), float("-inf")
    o2, lse2 = run(bad, c, lens)
    others = [h for h in range(16) if h not in (5, 12)]
    assert torch.equal(o2[:, others], o[:, others]) and torch.equal(lse2[:, others], lse[:, others])
    assert torch.equal(o2[0], o[0]) and not torch.isfinite(lse2[1, [5, 12]]).any()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_bad_pages_and_lengths(fp8):
    """Entries outside the cache and lengths outside the table: the positions
    are skipped, the error word says so, and good sequences are unharmed."""
    lens, Hkv, group, d, page = [100, 64, 30, 48], 2, 3, 64, 16
    c = filled_cache(lens, page, Hkv, d, 25, fp8, slack=0)
    c["table"][0, 2], c["table"][1, 3] = c["P"], -1
    c["table"][2, :] = 2 ** 31 - 1
    q = make_tensor((4, 6, 1, d), 26)
    o, lse = run(q, c, lens)
    assert ab.attn_device_error_word() == (ab.ATTN_ERR_DEVICE, 4 << 24 | 0x502)
    check(o, lse, serving.decode(q, c["k64"], c["v64"], c["table"], lens, 1 / 8), d)
    c = filled_cache(lens, page, Hkv, d, 25, fp8, slack=0)
    bad = [10 ** 9, -5, 30, 48]
    c["table"][0, 6:] = 0
    held = [112, 0, 30, 48]
    ref = serving.decode(q, np.nan_to_num(c["k64"]), np.nan_to_num(c["v64"]), c["table"], held, 1 / 8)
    for n in "kv":
        if fp8:
            u = c[n + "c"].view(torch.uint8)
            u[u == 0x7F] = 0
            c[n + "d"] = torch.nan_to_num(c[n + "d"], nan=0.0, posinf=0.0)
        else:
            c[n + "c"] = torch.nan_to_num(c[n + "c"])
    o, lse = run(q, c, bad)
    assert ab.attn_device_error_word() == (ab.ATTN_ERR_DEVICE, 4 << 24 | 0x501)
    check(o, lse, ref, d)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_many_sequences(fp8):
    """More sequences than a block has threads, most of them empty or a few
    positions long, and more head blocks than thread blocks."""
    rng = np.random.default_rng(8)
    lens = [int(n) for n in rng.choice([0, 0, 1, 5, 16, 17, 40, 100, 300], 700)]
    lens[-1] = 0
    c = filled_cache(lens, 16, 2, 64, 81, fp8)
    q = make_tensor((len(lens), 4, 1, 64), 82)
    o, lse = run(q, c, lens)
    check(o, lse, serving.decode(q, c["k64"], c["v64"], c["table"], lens, 1 / 8), 64)


@pytest.mark.parametrize("fp8", [False, True])
def test_cache_beyond_32_bits(fp8):
    """A cache of more than 2^31 values (2^32 in 8 bits), its last pages used:
    written, attended and read back."""
    Hkv, d, page, n = 2, 128, 64, 200
    P = ((1 << 32 if fp8 else 1 << 31) // (Hkv * d * page)) + 40
    kc, vc = (torch.empty((P, Hkv, page, d), device="cuda",
                          dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16) for _ in range(2))
    kd, vd = ((torch.empty((P, Hkv, page), device="cuda") for _ in range(2)) if fp8
              else (None, None))
    table = torch.tensor([[P - 1, P - 7, P - 3, P - 20], [P - 2, 0, P // 2, P - 21]],
                         dtype=torch.int32).cuda()
    x = make_tensor((2, n, 2 * Hkv, d), 90).cuda()
    k, v = x[:, :, :Hkv].transpose(1, 2), x[:, :, Hkv:].transpose(1, 2)
    zero, lens = i32([0, 0]).cuda(), i32([n, n - 9]).cuda()
    ab.kv_cache_write(k, v, kc, vc, table, zero, lens, kd, vd)
    q = make_tensor((2, 8, 1, d), 91)
    o, lse = ab.attn_decode(q.cuda(), kc, vc, table, lens, k_descale=kd, v_descale=vd)
    kr, vr = ab.kv_cache_read(kc, vc, table, zero, n, lens, kd, vd)
    # the oracle on the rounded rows, laid out as a small cache of their own
    small = torch.arange(8, dtype=torch.int32).view(2, 4)
    val = []
    for t in (k, v):
        t = t.contiguous().cpu()
        if fp8:
            code, fac = serving.quantise_rows(t)
            t = torch.from_numpy(serving.e4m3_to_f64(code) * fac[..., None])
        t = torch.nn.functional.pad(t.double(), (0, 0, 0, 4 * page - n))
        val.append(t.view(2, Hkv, 4, page, d).permute(0, 2, 1, 3, 4).reshape(8, Hkv, page, d).numpy())
    check(o, lse, serving.decode(q, val[0], val[1], small, [n, n - 9], 1 / math.sqrt(d)), d)
    for got, w in ((kr, val[0]), (vr, val[1])):
        w = w.reshape(2, 4, Hkv, page, d).transpose(0, 2, 1, 3, 4).reshape(2, Hkv, 4 * page, d)[:, :, :n]
        w[1, :, n - 9:] = 0
        assert np.array_equal(f64(got), w)


def test_decode_takes_bytes_and_given_outputs():
    """uint8 views of an e4m3 cache, and outputs of the caller's."""
    lens = [70, 33]
    c = filled_cache(lens, 16, 2, 64, 45, True)
    q = make_tensor((2, 4, 1, 64), 46)
    ref = run(q, c, lens)
    out = torch.empty(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 4, 1, device="cuda")
    c["kc"], c["vc"] = c["kc"].view(torch.uint8), c["vc"].view(torch.uint8)
    got = run(q, c, lens, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_decode_workspace_contents_do_not_matter():
    """A workspace of NaN bytes, then the same workspace after another batch."""
    d, page, Hkv, group = 128, 16, 2, 4
    c = filled_cache([2000, 40], page, Hkv, d, 35, False)
    c2 = filled_cache([17, 900], page, Hkv, d, 36, False)
    q = make_tensor((2, 8, 1, d), 37)
    ws = ab.alloc_decode_workspace(d, "cuda")
    ws.fill_(0xFF)
    o1, l1 = run(q, c, [2000, 40], workspace=ws)
    run(q, c2, [17, 900], workspace=ws)
    o2, l2 = run(q, c, [2000, 40], workspace=ws)
    assert torch.equal(o1, o2) and torch.equal(l1, l2) and torch.isfinite(o1).all()


def test_decode_refusals():
    kc, vc, _, _ = ab.alloc_kv_cache(4, 2, 16, 64, "cuda")
    q = make_tensor((3, 4, 1, 64), 1).cuda()
    table, lens = torch.zeros(3, 2, dtype=torch.int32).cuda(), i32([1, 1, 1]).cuda()
    good = dict(q=q, k_cache=kc, v_cache=vc, page_table=table, seq_lens=lens)
    kd = torch.ones(4, 2, 16, device="cuda")
    for change in (dict(q=q[:2]), dict(q=q[:, :3]), dict(q=q.float()), dict(q=q[:, :, 0]),
                   dict(q=q.expand(3, 4, 1, 64)[:, :, :, ::2]), dict(seq_lens=lens[:2]),
                   dict(seq_lens=lens.long()), dict(k_descale=kd), dict(k_descale=kd, v_descale=kd),
                   dict(v_cache=vc[:, :1]), dict(page_table=table.T), dict(k_cache=kc.cpu()),
                   dict(out=q[:2]), dict(lse=torch.zeros(3, 4, device="cuda")),
                   dict(q=torch.zeros(3, 4, 2, 64, dtype=torch.bfloat16, device="cuda")),
                   dict(workspace=torch.zeros(1 << 24, dtype=torch.uint8))):
        args = dict(good)
        args.update(change)
        with pytest.raises(ValueError):
            ab.attn_decode(**args)
    for change, status in ((dict(window=-1), ab.ATTN_ERR_INVALID_ARG),
                           (dict(scale=0.0), ab.ATTN_ERR_INVALID_ARG),
                           (dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")),
                            ab.ATTN_ERR_WORKSPACE)):
        args = dict(good)
        args.update(change)
        with pytest.raises(ab.AttnError) as e:
            ab.attn_decode(**args)
        assert e.value.status == status
    empty = torch.zeros(0, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = ab.attn_decode(empty, kc, vc, table[:0], lens[:0])
    assert o.shape == (0, 4, 1, 64) and lse.shape == (0, 4, 1)
