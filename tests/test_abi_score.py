"""The C ABI of attention with changed scores and of the 4-bit cache validates
on the host, before anything is launched, and the binding refuses what the C
side would misread.  CPU only."""

import ctypes
import math

import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab
from attention_backward_pass_attn_gb300 import build as abuild

FAKE = 0x10000  # a 256-byte aligned non-null address; never dereferenced
OK, INVALID, UNSUPPORTED, WORKSPACE = (ab.ATTN_OK, ab.ATTN_ERR_INVALID_ARG,
                                       ab.ATTN_ERR_UNSUPPORTED, ab.ATTN_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    abuild.build()
    return ab.load_library()


def test_declared_and_exported(lib):
    import attention_backward_pass_attn_gb300 as pkg

    for n in ("attn_fwd_score", "attn_bwd_score", "attn_score_decode", "int4_cache_write",
              "int4_cache_read"):
        assert ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
    assert callable(pkg.attn_fwd_score) and callable(pkg.attn_bwd_score)
    assert callable(pkg.alloc_score_workspace)


def score_call(lib, kind):
    def call(q=FAKE, k=FAKE, v=FAKE, strides=None, o=FAKE, L=FAKE, do=FAKE, dq=FAKE, dk=FAKE,
             dv=FAKE, B=1, Hq=4, Hkv=2, N=130, d=64, causal=1, window=0, doc=None, prefix=None,
             cap=0.0, slopes=None, scale=0.125, ws=FAKE, wsb=None):
        st = None if strides is None else (ctypes.c_int64 * 9)(*strides)
        if kind == "fwd":
            return lib.attn_fwd_score(q, k, v, st, o, L, B, Hq, Hkv, N, d, causal, window, doc,
                                      prefix, cap, slopes, scale, None)
        if wsb is None:
            wsb = lib.attn_bwd_score_workspace_size(B, Hq, Hkv, N, d, causal, window)
        return lib.attn_bwd_score(q, k, v, st, o, do, L, dq, dk, dv, B, Hq, Hkv, N, d, causal,
                                  window, doc, prefix, cap, slopes, scale, ws, wsb, None)
    return call


@pytest.mark.parametrize("kind", ["fwd", "bwd"])
def test_score_validation(lib, kind):
    call = score_call(lib, kind)
    bad = [dict(B=-1), dict(Hq=-1), dict(N=-1), dict(d=-64), dict(Hkv=0), dict(Hq=3), dict(causal=2),
           dict(window=-1), dict(causal=0, window=4), dict(causal=0, doc=FAKE),
           dict(causal=0, prefix=FAKE), dict(prefix=FAKE, window=4), dict(prefix=FAKE, doc=FAKE),
           dict(doc=FAKE + 2), dict(prefix=FAKE + 1), dict(slopes=FAKE + 2), dict(cap=-1.0),
           dict(cap=math.inf), dict(cap=math.nan), dict(cap=1e-42), dict(cap=3e38),
           dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf),
           dict(scale=3e38), dict(q=None), dict(k=None), dict(v=FAKE + 8), dict(o=None),
           dict(L=None), dict(L=FAKE + 2),
           dict(strides=(0, 64, 128, 0, 64, 128, 0, 64, 4)),     # not 16 bytes
           dict(strides=(0, 64, 128, 0, 0, 128, 0, 64, 128)),    # an expanded head
           dict(strides=(0, 64, -128, 0, 64, 128, 0, 64, 128))]
    if kind == "bwd":
        bad += [dict(do=None), dict(dq=FAKE + 4), dict(dk=None), dict(dv=FAKE + 8)]
    for b in bad:
        assert call(**b) == INVALID, b
    assert call(d=96) == UNSUPPORTED
    assert call(B=1 << 12, Hq=1 << 10, Hkv=1, N=1 << 10) == UNSUPPORTED
    assert call(strides=(0, 64, 128, 0, 1 << 39, 128, 0, 64, 128)) == UNSUPPORTED
    for empty in (dict(B=0), dict(N=0)):
        assert call(q=None, k=None, v=None, o=None, L=None, do=None, dq=None, dk=None, dv=None,
                    ws=None, wsb=0, **empty) == OK
    if kind == "bwd":
        assert call(Hq=0) == INVALID                       # dK and dV of nothing
        assert call(ws=None) == WORKSPACE and call(ws=FAKE + 16) == WORKSPACE
        need = lib.attn_bwd_score_workspace_size(1, 4, 2, 130, 64, 1, 0)
        assert need >= lib.attn_bwd_workspace_size(1, 4, 130, 64) and call(wsb=need - 1) == WORKSPACE


def test_workspace_size(lib):
    """The plain backward's, and the sums of a key head whose query heads are
    dealt to several blocks: where there are few key heads, not where many."""
    size = lib.attn_bwd_score_workspace_size
    one = 2 * 4096 * 128 * 4  # dK and dV of one part
    plain = lib.attn_bwd_workspace_size(1, 8, 4096, 128)
    assert size(1, 8, 8, 4096, 128, 1, 0) == plain
    assert size(1, 8, 1, 4096, 128, 1, 0) - plain in [s * one for s in (2, 4, 8)]
    assert size(16, 8, 4, 4096, 128, 0, 0) == lib.attn_bwd_workspace_size(16, 8, 4096, 128)
    assert size(0, 8, 1, 4096, 128, 1, 0) == 0 and size(1, 8, 3, 4096, 128, 1, 0) == 0
    assert size(1, 8, 1, 4096, 128, 1, 0) % 256 == 0


def cache_call(lib, kind):
    def call(x=FAKE, kc=FAKE, vc=FAKE, kf=FAKE, vf=FAKE, table=FAKE, start=FAKE, count=None, B=2,
             Hkv=2, T=4, d=64, ps=16, P=8, mp=4, strides=None, Hq=4, window=0, cap=0.0, slopes=None,
             scale=0.125, type=2, ws=FAKE, wsb=None, out=FAKE):
        if kind == "write":
            st = None if strides is None else (ctypes.c_int64 * 6)(*strides)
            return lib.int4_cache_write(x, x, st, kc, vc, kf, vf, table, start, count, B, Hkv, T, d,
                                        ps, P, mp, None)
        if kind == "read":
            return lib.int4_cache_read(kc, vc, kf, vf, table, start, count, x, x, B, Hkv, T, d, ps,
                                       P, mp, None)
        wsb = lib.attn_decode_workspace_size(d) if wsb is None else wsb
        return lib.attn_score_decode(x, kc, vc, kf, vf, type, table, start, out, out, B, Hq, Hkv, d,
                                     ps, P, mp, window, cap, slopes, scale, ws, wsb, None)
    return call


@pytest.mark.parametrize("kind", ["write", "read", "decode"])
def test_cache_validation(lib, kind):
    call = cache_call(lib, kind)
    assert call(d=96) == UNSUPPORTED and call(ps=24) == UNSUPPORTED
    assert call(ps=1 << 16, mp=1 << 15) == UNSUPPORTED
    for bad in (dict(ps=0), dict(P=0), dict(mp=0), dict(Hkv=0), dict(B=-1), dict(kc=None),
                dict(vc=FAKE + 8), dict(kf=None), dict(vf=None), dict(vf=FAKE + 1), dict(table=None),
                dict(table=FAKE + 2), dict(x=None), dict(x=FAKE + 8), dict(start=None)):
        assert call(**bad) == INVALID, bad
    assert call(B=0, x=None, kc=None, vc=None, kf=None, vf=None, table=None, start=None) == OK
    if kind != "decode":
        assert call(T=-1) == INVALID and call(count=FAKE + 2) == INVALID
        assert call(T=0, x=None, kc=None, vc=None, kf=None, vf=None, table=None, start=None) == OK
        assert call(B=1 << 12, Hkv=1 << 10, T=1 << 10) == UNSUPPORTED


def test_decode_validation(lib):
    call = cache_call(lib, "decode")
    for bad in (dict(type=3), dict(type=-1), dict(type=0), dict(type=1, kf=None), dict(type=1, vf=FAKE + 2),
                dict(Hq=3), dict(Hq=-2), dict(window=-1), dict(cap=-1.0), dict(cap=math.inf),
                dict(cap=math.nan), dict(cap=1e-42), dict(cap=3e38), dict(slopes=FAKE + 2),
                dict(scale=0.0), dict(scale=math.nan), dict(out=None)):
        assert call(**bad) == INVALID, bad
    assert call(ws=None) == WORKSPACE and call(ws=FAKE + 16) == WORKSPACE
    assert call(wsb=lib.attn_decode_workspace_size(64) - 1) == WORKSPACE
    assert call(B=1 << 20, Hq=1 << 12) == UNSUPPORTED


def test_binding_refuses_host_tensors():
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ab.attn_fwd_score(q, q, q, True)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ab.attn_bwd_score(q, q, q, q, q, torch.zeros(1, 2, 4), True)
    with pytest.raises(TypeError):
        ab.attn_fwd_score(None, q, q, True)
