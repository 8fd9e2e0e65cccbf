"""The 4-bit paged cache on the GPU, bit for bit against exact arithmetic
(oracle/int4.py): codes, factors, what is read back, and what stays as it was."""

import numpy as np
import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab
from attention_backward_pass_attn_gb300.inputs import make_tensor
from oracle import int4
from serving_cases import page_table

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


def filled(P, Hkv, page, d):
    """A cache of recognisable bytes and factors."""
    kc, vc, kd, vd = ab.alloc_kv_cache(P, Hkv, page, d, "cuda", "int4")
    kc.fill_(0x3A), vc.fill_(0xC5), kd.fill_(0.25), vd.fill_(3.0)
    return kc, vc, kd, vd


def check_written(k, v, cache, table, start, count, page):
    """Every row of the cache: the written ones are the oracle's, the others
    what they were."""
    P, Hkv, _, d = cache[0].shape[0], cache[0].shape[1], page, k.shape[-1]
    want = [t.cpu().numpy().copy() if t.dtype == torch.uint8 else t.double().cpu().numpy().copy()
            for t in filled(P, Hkv, page, d)]
    for x, c, f in ((k, want[0], want[2]), (v, want[1], want[3])):
        for b in range(k.shape[0]):
            for t in range(int(count[b])):
                p = int(start[b]) + t
                at = (int(table[b, p // page]), slice(None), p % page)
                codes, f[at] = int4.quantise(x[b, :, t].double().cpu().numpy())
                c[at] = int4.pack(codes)
    for got, ref, fac in ((cache[0], want[0], want[2]), (cache[1], want[1], want[3])):
        nan = np.repeat(np.isnan(fac), 16, axis=-1)
        assert np.array_equal(got.cpu().numpy()[~nan], ref[~nan])
    for got, ref in ((cache[2], want[2]), (cache[3], want[3])):
        assert np.array_equal(got.double().cpu().numpy(), ref, equal_nan=True)


@pytest.mark.parametrize("Hkv,d,page,start,count", [
    (1, 64, 16, [0], [1]), (2, 128, 16, [0, 5], [17, 1]), (3, 64, 48, [100, 0, 7], [30, 0, 64]),
    (4, 128, 64, [0, 63, 64, 1], [65, 2, 1, 0]), (1, 128, 256, [300], [100])])
def test_rows_are_rounded_exactly(Hkv, d, page, start, count):
    lens = [s + c for s, c in zip(start, count)]
    table, P = page_table(lens, page, 3)
    T = max(count) + 2  # a padded batch
    k, v = (make_tensor((len(lens), Hkv, T, d), 11 + i, std=2.0).cuda() for i in range(2))
    cache = filled(P, Hkv, page, d)
    s, c = (torch.tensor(x, dtype=torch.int32).cuda() for x in (start, count))
    ab.kv_cache_write(k, v, cache[0], cache[1], table.cuda(), s, count=c, k_descale=cache[2],
                      v_descale=cache[3])
    check_written(k, v, cache, table, start, count, page)
    # and back: the values the codes stand for, without another rounding
    kr, vr = ab.kv_cache_read(cache[0], cache[1], table.cuda(), s, T, count=c, k_descale=cache[2],
                              v_descale=cache[3])
    for got, new in ((kr, k), (vr, v)):
        for b, n in enumerate(count):
            codes, f = int4.quantise(new[b, :, :n].double().cpu().numpy().reshape(-1, d)) if n \
                else (np.zeros((0, d)), np.zeros((0, d // 32)))
            ref = codes * np.repeat(f, 32, axis=-1)
            assert np.array_equal(got[b, :, :n].double().cpu().numpy().reshape(-1, d), ref)
            assert not got[b, :, n:].any()


@pytest.mark.parametrize("d", [64, 128])
def test_ties_and_the_whole_range(d):
    """Values on and beside every tie, powers over bf16's whole range, zeros,
    subnormals, infinities and NaN."""
    rows = []
    rng = np.random.default_rng(0)
    for e in (-133, -130, -126, -120, -60, -8, -1, 0, 1, 7, 60, 120, 125):
        top = rng.integers(128, 256, size=8)
        for t in top:
            # multiples of half a factor: ties between neighbouring codes
            r = np.concatenate([[t], rng.integers(-t, t + 1, size=d - 1)]).astype(np.float64)
            rows.append(r * 2.0 ** (e - 7))
    for f in (16, 17, 19, 22, 25, 31):  # x / f exactly at k + 1/2
        half = np.arange(-15, 16, 2) * f / 2.0
        r = np.zeros(d)
        r[:16], r[16] = half, 7 * f
        r[32:48], r[48] = -half / 64, -7 * f / 64
        rows.append(r)
    rows += [np.zeros(d), np.full(d, float(torch.finfo(torch.bfloat16).max))]
    special = rng.standard_normal((6, d))
    special[0, 3] = np.inf
    special[1, 40] = -np.inf
    special[2, 0] = np.nan
    special[3, 33], special[3, 34] = np.nan, np.inf
    special[4, :32] = np.inf
    special[5, :] = np.nan
    x = torch.from_numpy(np.concatenate([np.array(rows), special])).to(torch.bfloat16)
    T, page = x.shape[0], 64
    k, v = x[None, None].cuda(), x.flip(0)[None, None].contiguous().cuda()
    table, P = page_table([T], page, 1)
    cache = filled(P, 1, page, d)
    zero = torch.zeros(1, dtype=torch.int32).cuda()
    ab.kv_cache_write(k, v, cache[0], cache[1], table.cuda(), zero, k_descale=cache[2],
                      v_descale=cache[3])
    check_written(k, v, cache, table, [0], [T], page)
    kr, _ = ab.kv_cache_read(cache[0], cache[1], table.cuda(), zero, T, k_descale=cache[2],
                             v_descale=cache[3])
    codes, f = int4.quantise(x.double().numpy())
    ref = codes * np.repeat(f, 32, axis=-1)
    got = kr[0, 0].double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)])


def test_rows_of_a_fused_projection():
    B, T, Hkv, d, page = 2, 37, 3, 128, 32
    x = make_tensor((B, T, 2 * Hkv, d), 8).cuda()
    k, v = x[:, :, :Hkv].transpose(1, 2), x[:, :, Hkv:].transpose(1, 2)
    table, P = page_table([T, T], page, 2)
    zero = torch.zeros(B, dtype=torch.int32).cuda()
    caches = [filled(P, Hkv, page, d) for _ in range(2)]
    for c, (a, b) in zip(caches, ((k, v), (k.contiguous(), v.contiguous()))):
        ab.kv_cache_write(a, b, c[0], c[1], table.cuda(), zero, k_descale=c[2], v_descale=c[3])
    assert all(torch.equal(a, b) for a, b in zip(*caches))


def test_token_by_token_is_the_prompt_at_once():
    T, Hkv, d, page = 40, 2, 64, 16
    k, v = (make_tensor((1, Hkv, T, d), 21 + i).cuda() for i in range(2))
    table, P = page_table([T], page, 5)
    one, many = filled(P, Hkv, page, d), filled(P, Hkv, page, d)
    ab.kv_cache_write(k, v, many[0], many[1], table.cuda(), torch.zeros(1, dtype=torch.int32).cuda(),
                      k_descale=many[2], v_descale=many[3])
    for t in range(T):
        ab.kv_cache_write(k[:, :, t:t + 1], v[:, :, t:t + 1], one[0], one[1], table.cuda(),
                          torch.tensor([t], dtype=torch.int32).cuda(), k_descale=one[2],
                          v_descale=one[3])
    assert all(torch.equal(a, b) for a, b in zip(one, many))


def test_bad_pages_and_positions_are_skipped_and_recorded():
    Hkv, d, page = 1, 64, 16
    table = torch.tensor([[0, 99, -1, 1]], dtype=torch.int32).cuda()
    k, v = (make_tensor((1, Hkv, 70, d), 31 + i).cuda() for i in range(2))
    cache = filled(3, Hkv, page, d)
    s = torch.zeros(1, dtype=torch.int32).cuda()
    ab.kv_cache_write(k, v, cache[0], cache[1], table, s, k_descale=cache[2], v_descale=cache[3])
    assert ab.attn_last_device_error() == ab.ATTN_ERR_DEVICE
    want = filled(3, Hkv, page, d)
    good = torch.tensor([[0, 1]], dtype=torch.int32).cuda()
    pick = torch.cat([k[:, :, :16], k[:, :, 48:64]], 2), torch.cat([v[:, :, :16], v[:, :, 48:64]], 2)
    ab.kv_cache_write(*pick, want[0], want[1], good, s, k_descale=want[2], v_descale=want[3])
    assert all(torch.equal(a, b) for a, b in zip(cache, want))
    kr, vr = ab.kv_cache_read(cache[0], cache[1], table, s, 70, k_descale=cache[2],
                              v_descale=cache[3])
    assert ab.attn_last_device_error() == ab.ATTN_ERR_DEVICE
    assert not kr[:, :, 16:48].any() and not vr[:, :, 64:].any() and kr[:, :, 48:64].any()


def test_refusals():
    kc, vc, kd, vd = ab.alloc_kv_cache(2, 1, 16, 64, "cuda", "int4")
    k = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    s = torch.zeros(1, dtype=torch.int32, device="cuda")

    def write(**changes):
        a = dict(kc=kc, vc=vc, kd=kd, vd=vd)
        a.update(changes)
        ab.kv_cache_write(k, k, a["kc"], a["vc"], table, s, k_descale=a["kd"], v_descale=a["vd"])
    write()
    with pytest.raises(ValueError, match="torch.uint8"):
        write(kc=kc.view(torch.int8))
    with pytest.raises(ValueError, match="v_descale must have shape"):
        write(vd=vd[..., :1])
    with pytest.raises(ValueError, match="v_descale must be torch.bfloat16"):
        write(vd=vd.float())
    with pytest.raises(ValueError, match="come together"):
        write(vd=None)
    with pytest.raises(ValueError, match="k must have shape"):  # rows of 64, not of 32 values
        ab.kv_cache_write(k[..., :32], k[..., :32], kc, vc, table, s, k_descale=kd, v_descale=vd)
    with pytest.raises(ValueError, match="multiple of 32"):
        ab.alloc_kv_cache(1, 1, 16, 48, "cuda", "int4")
    with pytest.raises(ValueError, match="int4"):
        ab.alloc_kv_cache(1, 1, 16, 64, "cuda", torch.int8)


def test_pages_beyond_32_bits_of_bytes():
    """The last pages of a cache of 4.4 GB a tensor: the same bits as the same
    rows in a small one, written, read and attended to."""
    Hkv, d, page, T = 8, 128, 256, 700
    P = 2 ** 32 // (Hkv * page * d // 2) + 1000
    k, v = (make_tensor((1, Hkv, T, d), 61 + i).cuda() for i in range(2))
    q = make_tensor((1, 4 * Hkv, 1, d), 63).cuda()
    zero = torch.zeros(1, dtype=torch.int32).cuda()
    lens = torch.tensor([T], dtype=torch.int32).cuda()
    big, small = filled(P, Hkv, page, d), filled(3, Hkv, page, d)
    assert big[0].numel() > 2 ** 32
    got = []
    for c, first in ((big, P - 3), (small, 0)):
        table = (torch.arange(3, dtype=torch.int32)[None] + first).cuda()
        f = dict(k_descale=c[2], v_descale=c[3])
        ab.kv_cache_write(k, v, c[0], c[1], table, zero, **f)
        got.append((*ab.kv_cache_read(c[0], c[1], table, zero, T, **f),
                    *ab.attn_decode(q, c[0], c[1], table, lens, softcap=30.0, **f),
                    *ab.attn_decode(q, c[0], c[1], table, lens, **f)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    for a, b in zip(big, small):
        assert torch.equal(a[-3:], b)
        assert bool((a[:-3] == a[0, 0, 0, 0]).all())  # and nothing else was written
