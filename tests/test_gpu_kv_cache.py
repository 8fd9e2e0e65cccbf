"""The paged key/value cache on the GPU: what is written, where, and what
stays as it was, against the fp64 oracle.

Writing is exact: bf16 rows are copied, e4m3 rows have one correct code and
factor each (division by a power of two is exact), so codes and factors must
be equal.  Reading rounds value x factor once to bf16 (half a step, 2^-8),
after a product in fp32 (2^-24); with a power-of-two factor whose product is a
normal number it is exact, four significant bits fitting eight.
"""

import numpy as np
import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab
from attention_backward_pass_attn_gb300.inputs import make_tensor
from oracle import serving
from serving_cases import cuda, filled_cache, page_table

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


def leftover(P, Hkv, page, d, fp8, seed):
    """A cache full of an earlier owner's bytes, as CPU tensors."""
    g = torch.Generator().manual_seed(seed)
    if not fp8:
        return [make_tensor((P, Hkv, page, d), seed + i) for i in range(2)] + [None, None]
    c = [torch.randint(0, 256, (P, Hkv, page, d), generator=g, dtype=torch.uint8) for _ in range(2)]
    s = [torch.rand((P, Hkv, page), generator=g) for _ in range(2)]
    return c + s


def expect_written(cache, k, v, table, start, count, page):
    """The oracle's cache after the write: bytes (or bf16) and factors."""
    kc, vc, kd, vd = (None if t is None else t.clone() for t in cache)
    P = kc.shape[0]
    for new, c, s in ((k, kc, kd), (v, vc, vd)):
        if s is not None:
            code, fac = serving.quantise_rows(new)
        for b in range(len(start)):
            for t in range(int(count[b])):
                p = int(start[b]) + t
                if p < 0 or p // page >= table.shape[1] or not 0 <= int(table[b, p // page]) < P:
                    continue
                at = (int(table[b, p // page]), slice(None), p % page)
                if s is None:
                    c[at] = new[b, :, t]
                else:
                    c[at] = torch.from_numpy(code[b, :, t])
                    s[at] = torch.from_numpy(fac[b, :, t]).float()
    return kc, vc, kd, vd


def same(got, ref):
    for g, r, n in zip(got, ref, ("k_cache", "v_cache", "k_descale", "v_descale")):
        if r is None:
            continue
        g, r = g.cpu(), r
        if g.dtype == torch.bfloat16:
            g, r = g.view(torch.int16), r.view(torch.int16)
        elif g.dtype == torch.float8_e4m3fn:
            g = g.view(torch.uint8)
        assert torch.equal(g, r), "%s: %d differ" % (n, int((g != r).sum()))


WRITES = [
    # B, Hkv, T, d, page, start, count
    (1, 1, 1, 64, 16, [0], None),
    (1, 2, 1, 128, 16, [15], None),
    (3, 2, 5, 64, 16, [0, 14, 31], [5, 3, 0]),
    (2, 3, 40, 128, 48, [47, 0], [40, 33]),
    (4, 1, 33, 128, 32, [0, 1, 31, 32], [0, 33, 1, 32]),
    (2, 8, 130, 64, 64, [63, 200], None),
    (9, 4, 1, 128, 256, [0, 1, 2, 255, 256, 257, 511, 5, 6], [1, 1, 1, 1, 1, 1, 1, 0, 0]),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,Hkv,T,d,page,start,count", WRITES)
def test_write_everything_else_stays(B, Hkv, T, d, page, start, count, fp8):
    seed = 100 * B + T + d
    n = [T] * B if count is None else count
    table, P = page_table([s + c for s, c in zip(start, n)], page, seed)
    cache = leftover(P, Hkv, page, d, fp8, seed)
    x = make_tensor((B, T, 2 * Hkv, d), seed + 5)
    # rows of every kind: zeros, tiny, huge, one outlier, a tie of amax
    x[0, 0, 0] = 0
    x[-1, -1, -1] *= 2.0 ** -130
    x[-1, 0, 0] *= 2.0 ** 100
    x[0, -1, -1, 3] = 448.0
    for b in range(B):  # a padded batch's filling must not be looked at
        x[b, n[b]:] = float("nan")
    k, v = x[:, :, :Hkv].transpose(1, 2), x[:, :, Hkv:].transpose(1, 2)
    dev = [cuda(t) for t in cache]
    xd = x.cuda()
    ab.kv_cache_write(xd[:, :, :Hkv].transpose(1, 2), xd[:, :, Hkv:].transpose(1, 2), dev[0],
                      dev[1], table.cuda(), i32(start).cuda(),
                      None if count is None else i32(count).cuda(), dev[2], dev[3])
    same(dev, expect_written(cache, k, v, table, start, n, page))


def test_write_special_values():
    """Infinities saturate without moving the row's factor, NaN stays NaN,
    subnormal rows, and both zeros."""
    d = 64
    rows = torch.zeros(12, d)
    rows[0, :4] = torch.tensor([float("inf"), 3.0, -2.0, 0.1])
    rows[1, :3] = torch.tensor([float("-inf"), float("nan"), 1.0])
    rows[2] = float("nan")
    rows[3] = float("inf")
    rows[4, :2] = torch.tensor([2.0 ** -133, -2.0 ** -133])
    rows[5, :2] = torch.tensor([3.38e38, 1.0])
    rows[6, :3] = torch.tensor([-0.0, 0.0, 2.0 ** -126])
    rows[7] = torch.linspace(-448, 448, d)
    rows[8] = torch.linspace(0.0625, 1.96, d)
    rows[9, 0], rows[9, 1] = 450.0, 2.0 ** -9
    rows[10] = 1.75
    rows[11] = 1.765625
    x = rows.to(torch.bfloat16).view(1, 1, 12, d)
    kc, vc, kd, vd = ab.alloc_kv_cache(1, 1, 16, d, "cuda", torch.float8_e4m3fn)
    z = i32([0]).cuda()
    ab.kv_cache_write(x.cuda(), x.cuda(), kc, vc, z.view(1, 1), z, None, kd, vd)
    code, fac = serving.quantise_rows(x)
    got = serving.codes(kc)[0, 0, :12]
    assert np.array_equal(kd.cpu().numpy()[0, 0, :12], fac[0, 0].astype(np.float32))
    nan = np.isnan(f64(x)[0, 0])
    assert np.all((got[nan] & 0x7F) == 0x7F)
    assert np.array_equal(got[~nan], code[0, 0][~nan])
    assert torch.equal(kc.view(torch.uint8), vc.view(torch.uint8)) and torch.equal(kd, vd)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,Hkv,T,d,page,start,count", WRITES)
def test_read_back(B, Hkv, T, d, page, start, count, fp8):
    seed = 300 * B + T + d
    n = [T] * B if count is None else count
    lens = [s + c for s, c in zip(start, n)]
    c = filled_cache(lens, page, Hkv, d, seed, fp8)
    if fp8:  # any positive factors, not the writer's powers of two alone
        c["kd"] = c["kd"] * 1.2345
        c["k64"] = serving.cache_values(c["kc"], c["kd"])
    k, v = ab.kv_cache_read(cuda(c["kc"]), cuda(c["vc"]), c["table"].cuda(), i32(start).cuda(), T,
                            None if count is None else i32(count).cuda(), cuda(c["kd"]),
                            cuda(c["vd"]))
    for got, val, exact in ((k, c["k64"], not fp8), (v, c["v64"], True)):
        ref = np.zeros((B, Hkv, T, d))
        for b in range(B):
            ref[b, :, :n[b]] = serving.gather(val, c["table"][b].numpy(),
                                              range(start[b], start[b] + n[b]))
        assert np.all(np.isfinite(ref))
        tol = 0 if exact else np.abs(ref) * (2.0 ** -8 + 2.0 ** -23)
        assert np.all(np.abs(f64(got) - ref) <= tol)


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_pages_and_positions_are_skipped_and_reported(fp8):
    """Entries outside the cache, starts below zero and past the table: the
    kernels check each index before they follow it."""
    B, Hkv, T, d, page = 4, 2, 20, 64, 16
    table = i32([[0, 1, 2], [3, 99, 4], [-1, 5, 2 ** 30], [6, 7, 8]])
    start, count = [-3, 10, 0, 40], [20, 20, 20, 20]
    cache = leftover(9, Hkv, page, d, fp8, 3)
    x = make_tensor((B, Hkv, T, d), 4)
    dev = [cuda(t) for t in cache]
    ab.kv_cache_write(x.cuda(), x.cuda(), dev[0], dev[1], table.cuda(), i32(start).cuda(),
                      i32(count).cuda(), dev[2], dev[3])
    assert ab.attn_last_device_error() == ab.ATTN_ERR_DEVICE
    assert ab.attn_last_device_error() == ab.ATTN_OK
    same(dev, expect_written(cache, x, x, table, start, count, page))
    k, _ = ab.kv_cache_read(dev[0], dev[1], table.cuda(), i32(start).cuda(), T,
                            i32(count).cuda(), dev[2], dev[3])
    assert ab.attn_last_device_error() == ab.ATTN_ERR_DEVICE
    k = f64(k)
    for b in range(B):
        for t in range(T):
            p = start[b] + t
            if p < 0 or p >= 48 or not 0 <= int(table[b, p // page]) < 9:
                assert np.all(k[b, :, t] == 0)
            else:
                assert np.any(k[b, :, t] != 0)
    assert ab.attn_last_device_error() == ab.ATTN_OK


def test_refusals():
    kc, vc, kd, vd = ab.alloc_kv_cache(4, 2, 16, 64, "cuda", torch.float8_e4m3fn)
    x = make_tensor((3, 2, 5, 64), 1).cuda()
    table, start = torch.zeros(3, 2, dtype=torch.int32).cuda(), i32([0, 0, 0]).cuda()
    good = dict(k=x, v=x, k_cache=kc, v_cache=vc, page_table=table, start=start, k_descale=kd,
                v_descale=vd)
    bf = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    for change in (dict(k_descale=None), dict(k_descale=None, v_descale=None), dict(k_cache=bf),
                   dict(v_cache=vc[:3]), dict(k_descale=kd.double()), dict(k_descale=kd[:3]),
                   dict(page_table=table.long()), dict(page_table=table[:2]),
                   dict(page_table=table[0]), dict(start=start[:2]), dict(start=start.long()),
                   dict(count=start[:1]), dict(k=x[:2]), dict(v=x[:, :1]), dict(k=x.float()),
                   dict(k=x[:, :, :4]), dict(k_cache=kc.transpose(1, 2)), dict(start=start.cpu()),
                   dict(k=x.transpose(2, 3)), dict(k_cache=kc[0])):
        args = dict(good)
        args.update(change)
        with pytest.raises(ValueError):
            ab.kv_cache_write(**args)
    with pytest.raises(ValueError):
        ab.kv_cache_read(kc, vc, table, start, 5, None, kd, vd, out=(x, x.float()))
    with pytest.raises(ValueError):
        ab.alloc_kv_cache(4, 2, 16, 64, "cuda", torch.float16)
    odd = torch.zeros(4, 2, 24, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ab.AttnError) as e:
        ab.kv_cache_read(odd, odd, table, start, 5)
    assert e.value.status == ab.ATTN_ERR_UNSUPPORTED
    ab.kv_cache_write(x[:, :, :0], x[:, :, :0], kc, vc, table, start, None, kd, vd)  # T = 0
    assert torch.all(kc.view(torch.uint8) == 0)
