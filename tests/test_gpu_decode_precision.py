"""How many bits attn_decode's answers have.

Bounds, with A = sum_j p_j |v_j|, S = max_j scale sum_i |q_i k_ji|, and c the
number of roundings a running sum goes through: a thread's keys (16 of a run of
16 KT keys, one after another, in two products), its share's runs, the warps,
the lanes, and the parts of the joins, at most 64 of those:

- a score: e = ((d + 8) 2^-23 + 2^-22) S, products being exact;
- L: e + c 2^-24 + 2^-22 (1 + |L|);
- O: 2 e + c 2^-22 for weights, their sum and the accumulation, 2^-21 for two
  exponentials, 2^-16 for the weights as two bf16 numbers, all of A; then the
  rounding of the result, 2^-8 |O|.
"""

import math

import numpy as np
import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab
from oracle import serving
from test_gpu_decode import cuda_ready, f64, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def random_cache(lens, page, Hkv, d, seed, fp8):
    """A cache of random rows, on the GPU, all pages in random order."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    P, mp = sum(need) + 1, max(need)
    order = torch.randperm(P, generator=g).to(torch.int32)
    table = torch.full((len(lens), mp), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    c = {"table": table}
    for n in "kv":
        x = torch.randn((P, Hkv, page, d), generator=g)
        if fp8:
            c[n + "c"] = (x * 64).to(torch.float8_e4m3fn)
            c[n + "d"] = 2.0 ** -6 * (1 + 0.5 * torch.rand((P, Hkv, page), generator=g))
        else:
            c[n + "c"], c[n + "d"] = x.to(torch.bfloat16), None
    return c


def values(c, n):
    """fp64 values [pages, Hkv, page, d] of a cache that is on the CPU."""
    x = c[n + "c"].double()
    return (x if c[n + "d"] is None else x * c[n + "d"].double()[..., None]).numpy()


def answer(c, q, lens, **kw):
    cu = {k: None if v is None else v.cuda() for k, v in c.items()}
    return ab.attn_decode(q.cuda(), cu["kc"], cu["vc"], cu["table"], i32(lens).cuda(),
                          k_descale=cu["kd"], v_descale=cu["vd"], **kw)


def reference(c, q, lens, scale):
    """O, L, A, S as serving.decode gives them, whole sequences at a time."""
    B, Hq, _, d = q.shape
    k, v, q = values(c, "k"), values(c, "v"), f64(q)
    Hkv, page = k.shape[1], k.shape[2]
    out = {n: np.zeros((B, Hq, d)) for n in "OA"}
    out.update(L=np.full((B, Hq), -np.inf), S=np.zeros((B, Hq)))
    for b, n in enumerate(lens):
        if not n:
            continue
        pages = c["table"][b, :-(-n // page)].long().numpy()
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            kk, vv = (t[pages, hk].reshape(-1, d)[:n] for t in (k, v))
            s = scale * (kk @ q[b, h, 0])
            w = np.exp(s - s.max())
            out["L"][b, h] = s.max() + np.log(w.sum())
            out["S"][b, h] = scale * np.max(np.abs(kk) @ np.abs(q[b, h, 0]))
            out["O"][b, h] = w @ vv / w.sum()
            out["A"][b, h] = w @ np.abs(vv) / w.sum()
    return out


def chain(lens, Hkv, group, d, fp8):
    """c of the bounds above: 64, and two roundings for every 16 keys of the
    longest share (a warp takes a quarter of a unit's keys)."""
    unit = {(64, False): 128, (128, False): 64, (64, True): 256, (128, True): 128}[d, fp8]
    blocks = -(-group // 16)
    W = sum(-(-n // unit) for n in lens) * Hkv * blocks
    grid = (3 if -(-group // blocks) <= 8 else 2) * \
        torch.cuda.get_device_properties(0).multi_processor_count
    units = -(-W // min(W, grid))
    return 64 + 4 * units * unit // 4 // 16


def check(o, lse, ref, c, d):
    o, lse = f64(o)[:, :, 0], f64(lse)[:, :, 0]
    some = np.isfinite(ref["L"])
    assert np.all(np.isneginf(lse[~some])) and np.all(o[~some] == 0)
    e = ((d + 8) * 2.0 ** -23 + 2.0 ** -22) * ref["S"]
    dl = np.abs(lse[some] - ref["L"][some])
    assert np.all(dl <= (e + c * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(ref["L"])))[some]), dl.max()
    rel = (2 * e + c * 2.0 ** -22 + 2.0 ** -21 + 2.0 ** -16)[..., None]
    do = np.abs(o - ref["O"])
    tol = np.abs(ref["O"]) * 2.0 ** -8 + rel * ref["A"] * (1 + 2.0 ** -8)
    assert np.all(do <= tol), "O off by %.2e, %.1f of its bound" % (do.max(), np.nanmax(do / tol))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hkv,group,d,lens", [
    (1, 1, 64, [70000]),               # every block has a part of one head
    (1, 4, 128, [131]),
    (3, 2, 64, [40000, 70, 33000]),    # shares end inside head blocks of dozens of shares
    (3, 1, 128, [20011, 0, 17001, 5]),
    (2, 12, 64, [30000, 900, 31000]),  # two blocks an SM
    (1, 40, 128, [21000, 3]),          # three blocks of heads
    (5, 1, 64, [26000, 1, 25000, 24001])])
def test_shares_that_straddle_head_blocks(Hkv, group, d, lens, fp8):
    """More units of work than thread blocks, and head blocks of more than 32
    shares: a sequence's first part lies behind another's last in its block's
    share, and blocks own two parts, of which one or both join in two steps.
    e4m3 units are twice as long, and so are the sequences."""
    lens = [2 * n for n in lens] if fp8 else lens
    c = random_cache(lens, 64, Hkv, d, 7 + group, fp8)
    q = torch.randn((len(lens), Hkv * group, 1, d),
                    generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    ws = ab.alloc_decode_workspace(d, "cuda")
    ws.fill_(0xFF)
    o, lse = answer(c, q, lens, workspace=ws)
    check(o, lse, reference(c, q, lens, 1 / math.sqrt(d)), chain(lens, Hkv, group, d, fp8), d)
    for _ in range(3):
        o2, lse2 = answer(c, q, lens, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert ab.attn_last_device_error() == ab.ATTN_OK


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [2, 3, 30, 400])
def test_weights_have_sixteen_bits(n, d, fp8):
    """Values of either sign that cancel: the result is a small difference of
    nearly equal weights, which one bf16 number (2^-8) or one fp16 number
    (2^-11) to a weight would miss by far."""
    B, Hkv, group = 24, 1, 4
    lens = [n] * B
    c = random_cache(lens, 16, Hkv, d, 70 + n, fp8)
    sign = torch.ones(16)
    sign[1::2] = -1
    v = sign[:, None] * torch.ones(d)
    c["vc"] = v.expand(c["vc"].shape).to(c["vc"].dtype).contiguous()
    if fp8:
        c["vd"] = torch.ones_like(c["vd"])
    if n % 2:  # the odd one out weighs nothing
        p = n - 1
        for b in range(B):
            c["vc"].view(torch.uint8 if fp8 else torch.int16)[int(c["table"][b, p // 16]), 0, p % 16] = 0
    q = torch.randn((B, group, 1, d), generator=torch.Generator().manual_seed(n)).to(torch.bfloat16)
    scale = 2.0 ** -9 / math.sqrt(d)
    o, lse = answer(c, q, lens, scale=scale)
    ref = reference(c, q, lens, scale)
    assert np.abs(ref["O"]).max() <= 2.0 ** -6  # little is left of values of one
    check(o, lse, ref, chain(lens, Hkv, group, d, fp8), d)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [2, 12])
@pytest.mark.parametrize("far", [20, 30, 45, 90, 140])
def test_queries_of_a_wide_range(far, group, d, fp8):
    """Elements 2^far above the others, where every key is zero: the small
    elements are the whole score.  One head has them, its neighbours have not."""
    lens = [300, 17, 1000]
    c = random_cache(lens, 32, 1, d, far, fp8)
    c["kc"].view(torch.uint8 if fp8 else torch.int16)[..., 3::16] = 0
    q = torch.randn((3, group, 1, d), generator=torch.Generator().manual_seed(far)).double()
    q[:, 0] *= 2.0 ** (30 - far)
    q[:, 0, :, 3::16] *= 2.0 ** far
    q = q.to(torch.bfloat16)
    assert torch.isfinite(q).all()
    scale = 2.0 ** (far - 30) / math.sqrt(d)  # scores of ordinary size for that head
    if far > 30:  # the neighbours' scores would be beyond any softmax
        q[:, 1:] *= 2.0 ** (30 - far)
    o, lse = answer(c, q, lens, scale=scale)
    check(o, lse, reference(c, q, lens, scale), chain(lens, 1, group, d, fp8), d)
