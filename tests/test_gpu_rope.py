"""Rotary positions and their gradient on the GPU against the fp64 oracle.

Tolerance, per element: the result is rounded once to bf16 (half a step, 2^-8
of the value).  Before that, the angle: its turn is known to 2^-32, 2^-29
radians, and the remainder of a quarter turn, at most pi / 4, is converted and
scaled in fp32, two roundings and a constant's, 3 pi/4 2^-24 < 2^-22 radians
together; the sine and cosine of that are within 2^-22 (polynomials cut off
below 2^-25, and their last roundings); the two products and the sum round at
2^-24 each.  Together less than 2^-20 (|a| + |b|) for a pair (a, b).
"""

import numpy as np
import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab
from attention_backward_pass_attn_gb300.inputs import make_tensor
from oracle import serving

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


def sections_of(d, axes):
    half = d // 2
    return {1: (half,), 2: (half // 2 + 3, half // 2 - 3), 3: (half // 4, 0, half - half // 4),
            4: (5, 7, 9, half - 21)}[axes]


def freqs(d, base=10000.0):
    return torch.tensor(base ** (-np.arange(d // 2) / (d // 2)), dtype=torch.float32)


def check(y, x, pos, f, sections, il, inverse):
    xx, d = f64(x), x.shape[-1]
    ref = serving.rope(x, pos, f, sections, il, inverse)
    ia = np.arange(d // 2) * 2 if il else np.arange(d // 2)
    ib = ia + 1 if il else ia + d // 2
    mag = np.empty_like(xx)
    mag[..., ia] = mag[..., ib] = np.abs(xx[..., ia]) + np.abs(xx[..., ib])
    tol = np.abs(ref) * 2.0 ** -8 + mag * 2.0 ** -20 * (1 + 2.0 ** -8)
    assert y.is_contiguous() and y.dtype == torch.bfloat16 and y.shape == x.shape
    bad = np.abs(f64(y) - ref) > tol
    assert not bad.any(), "%d of %d values off" % (bad.sum(), bad.size)


@pytest.mark.parametrize("direction", ["fwd", "bwd"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,Hk,N,d,axes,shared", [
    (1, 1, 1, 1, 64, 1, False), (1, 2, 0, 1, 128, 1, False), (2, 3, 1, 33, 64, 2, False),
    (3, 4, 2, 129, 128, 3, False), (2, 5, 5, 70, 128, 4, True), (5, 32, 8, 1, 128, 1, False),
    (1, 1, 3, 257, 64, 3, True), (2, 16, 16, 100, 64, 2, False)])
def test_rope_full_tensors(B, H, Hk, N, d, axes, shared, interleaved, direction):
    seed = B * 1000 + N + d
    q, k = make_tensor((B, H, N, d), seed), make_tensor((B, Hk, N, d), seed + 1)
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(-3000, 3000, (axes, 1 if shared else B, N), generator=g, dtype=torch.int32)
    f, sec = freqs(d), sections_of(d, axes)
    fn = ab.rope_fwd if direction == "fwd" else ab.rope_bwd
    yq, yk = fn(q.cuda(), k.cuda() if Hk else None, pos.cuda(), f.cuda(), sec, interleaved)
    check(yq, q, pos, f, sec, interleaved, direction == "bwd")
    if Hk:
        check(yk, k, pos, f, sec, interleaved, direction == "bwd")
    else:
        assert yk is None


def test_rope_far_positions_and_odd_frequencies():
    """Positions up to 2^30 (the oracle's own angles are then good to 2^30 2^-53
    = 2^-23 radians, inside the tolerance), negative ones, and frequencies from
    2^-140 to 7 radians a position, negative and zero among them."""
    B, H, N, d = 1, 2, 64, 64
    q = make_tensor((B, H, N, d), 5)
    g = torch.Generator().manual_seed(6)
    pos = torch.randint(-2 ** 30, 2 ** 30, (1, B, N), generator=g, dtype=torch.int32)
    pos[0, 0, :6] = torch.tensor([0, 1, -1, 2 ** 30, -2 ** 30, 2 ** 20 + 1])
    f = freqs(d)
    f[:6] = torch.tensor([0.0, 1.0, -0.75, 2.0 ** -140, 2.0 ** -30, 0.999])
    y, _ = ab.rope_fwd(q.cuda(), None, pos.cuda(), f.cuda())
    check(y, q, pos, f, (32,), False, False)
    f[6:10] = torch.tensor([6.5, -3.25, 2.0 ** 5, 1.5 * 2.0 ** 20])
    near = pos % 1000
    y, _ = ab.rope_fwd(q.cuda(), None, near.cuda(), f.cuda())
    check(y, q, near, f, (32,), False, False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_adjoint_to_its_gradient(interleaved):
    """<g, rope(x)> = <rope_bwd(g), x>, and the difference of the forward along
    a direction e is <rope_bwd(g), e>: rope is linear.  Each inner product of M
    terms is off by at most 2^-8 + 2^-19 of sum |g||y| and sum |x||dx|."""
    B, H, N, d = 2, 3, 50, 128
    x, g, e = (make_tensor((B, H, N, d), 40 + i).cuda() for i in range(3))
    pos = (torch.arange(N, dtype=torch.int32) * 7).view(1, 1, N).cuda()
    f = freqs(d).cuda()
    y, _ = ab.rope_fwd(x, None, pos, f, interleaved=interleaved)
    ye, _ = ab.rope_fwd(e, None, pos, f, interleaved=interleaved)
    dx, _ = ab.rope_bwd(g, None, pos, f, interleaved=interleaved)
    y, ye, dx, x, e, g = (f64(t) for t in (y, ye, dx, x, e, g))
    for a, b in ((np.sum(g * y) - np.sum(dx * x), np.sum(np.abs(g * y)) + np.sum(np.abs(dx * x))),
                 (np.sum(g * ye) - np.sum(dx * e), np.sum(np.abs(g * ye)) + np.sum(np.abs(dx * e)))):
        assert abs(a) <= (2.0 ** -8 + 2.0 ** -19) * b


def test_rope_strided_inputs_and_in_place():
    """Heads of a fused projection, a broadcast batch, an input on a row of a
    larger tensor: the same bits as contiguous copies.  Contiguous inputs may
    be their own outputs."""
    B, H, Hk, N, d = 3, 4, 2, 37, 64
    x = make_tensor((B, N, H + 2 * Hk, d), 9).cuda()
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hk].transpose(1, 2)
    pos = torch.arange(N, dtype=torch.int32).view(1, 1, N).cuda()
    f = freqs(d).cuda()
    ref = ab.rope_fwd(q.contiguous(), k.contiguous(), pos, f)
    got = ab.rope_fwd(q, k, pos, f)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    b = q[:1].expand(B, H, N, d)
    assert torch.equal(ab.rope_fwd(b, None, pos, f)[0], ab.rope_fwd(b.contiguous(), None, pos, f)[0])
    one = x[:, 5:6, :H].transpose(1, 2)
    assert torch.equal(ab.rope_fwd(one, None, pos[:, :, 5:6].contiguous(), f)[0],
                       ref[0][:, :, 5:6])
    qc, kc = q.contiguous(), k.contiguous()
    out = ab.rope_fwd(qc, kc, pos, f, out=(qc, kc))
    assert out[0] is qc and torch.equal(qc, ref[0]) and torch.equal(kc, ref[1])


def test_rope_empty_and_refusals():
    f = freqs(64).cuda()
    q = torch.zeros(2, 3, 0, 64, dtype=torch.bfloat16, device="cuda")
    y, _ = ab.rope_fwd(q, None, torch.zeros(1, 1, 0, dtype=torch.int32, device="cuda"), f)
    assert y.shape == q.shape
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(1, 2, 4, dtype=torch.int32, device="cuda")
    bad = [dict(pos=pos[:, :, :3]), dict(pos=pos.long()), dict(pos=pos[0]), dict(inv_freq=f[:31]),
           dict(inv_freq=f.double()), dict(sections=(31,)), dict(sections=(16, 16)),
           dict(sections=(-1,)), dict(q=q.float()), dict(q=q.transpose(2, 3)),
           dict(k=q[:, :, :3]), dict(k=q[:1]), dict(out=(q.transpose(1, 2), None)),
           dict(out=(q.float(), None)), dict(inv_freq=f.cpu()), dict(pos=pos.cpu())]
    for change in bad:
        args = dict(q=q, k=None, pos=pos, inv_freq=f)
        args.update(change)
        with pytest.raises(ValueError):
            ab.rope_fwd(**args)
    odd = torch.zeros(2, 3, 4, 66, dtype=torch.bfloat16, device="cuda")[..., :64]
    with pytest.raises(ValueError, match="multiples of 8"):
        ab.rope_fwd(odd, None, pos, f)
    with pytest.raises(ab.AttnError) as e:  # starts 8 bytes into a 16-byte line
        ab.rope_fwd(torch.zeros(2 * 3 * 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(
            2, 3, 4, 64), None, pos, f)
    assert e.value.status == ab.ATTN_ERR_INVALID_ARG
    with pytest.raises(ab.AttnError) as e:
        ab.rope_fwd(torch.zeros(1, 1, 1, 96, dtype=torch.bfloat16, device="cuda"), None,
                    pos[:, :1, :1].contiguous(), torch.ones(48, device="cuda"))
    assert e.value.status == ab.ATTN_ERR_UNSUPPORTED
