"""The answering path's C ABI validates on the host, before anything is
launched, and its binding refuses what the C side would misread.  CPU only."""

import ctypes
import os
import re

import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab
from attention_backward_pass_attn_gb300 import build as abuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # a 16-byte aligned non-null address; never dereferenced
OK, INVALID, UNSUPPORTED, WORKSPACE = (ab.ATTN_OK, ab.ATTN_ERR_INVALID_ARG,
                                       ab.ATTN_ERR_UNSUPPORTED, ab.ATTN_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    abuild.build()
    return ab.load_library()


def test_declared_and_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "attn.h")).read(),
                  flags=re.S)
    names = set(re.findall(r"\b((?:rope|kv_cache|attn_decode)[a-z0-9_]*)\s*\(", text))
    assert names == {"rope_fwd", "rope_bwd", "kv_cache_write", "kv_cache_read", "attn_decode",
                     "attn_decode_workspace_size"}
    for n in names:
        assert ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
        import attention_backward_pass_attn_gb300 as pkg

        if not n.endswith("_size"):
            assert callable(getattr(pkg, n))


@pytest.mark.parametrize("fn", ["rope_fwd", "rope_bwd"])
def test_rope_validation(lib, fn):
    def call(q=FAKE, k=FAKE, pos=FAKE, f=FAKE, sections=(32,), axes=None, il=0, strides=None,
             oq=FAKE, ok=FAKE, B=1, H=2, Hk=1, N=4, d=64, pb=1):
        sec = None if sections is None else (ctypes.c_int * 4)(*sections)
        st = None if strides is None else (ctypes.c_int64 * 6)(*strides)
        return getattr(lib, fn)(q, k, pos, f, sec, len(sections or ()) if axes is None else axes,
                                il, st, oq, ok, B, H, Hk, N, d, pb, None)
    assert call(d=96, sections=(48,)) == UNSUPPORTED
    assert call(sections=(31,)) == INVALID          # does not cover the pairs
    assert call(sections=(16, 17)) == INVALID
    assert call(sections=(40, -8)) == INVALID
    assert call(sections=None, axes=1) == INVALID
    assert call(axes=0) == INVALID and call(axes=5) == INVALID
    assert call(il=2) == INVALID
    assert call(B=-1) == INVALID and call(N=-1) == INVALID and call(H=-1) == INVALID
    assert call(B=3, pb=2) == INVALID
    assert call(q=None) == INVALID and call(k=None) == INVALID and call(pos=None) == INVALID
    assert call(f=None) == INVALID and call(oq=None) == INVALID and call(ok=None) == INVALID
    assert call(q=FAKE + 8) == INVALID and call(ok=FAKE + 2) == INVALID
    assert call(pos=FAKE + 2) == INVALID
    assert call(B=2, pb=2, strides=(4, 64, 64, 0, 0, 64)) == INVALID   # not 16 bytes
    assert call(strides=(0, -64, 64, 0, 0, 64)) == INVALID
    assert call(B=1 << 16, N=1 << 16) == UNSUPPORTED
    for empty in (dict(B=0, pb=0), dict(N=0), dict(H=0, Hk=0)):
        assert call(q=None, k=None, pos=None, f=None, oq=None, ok=None, **empty) == OK


def cache_args(kind):
    """call(**changes) of kv_cache_write, kv_cache_read or attn_decode."""
    lib = ab.load_library()

    def call(x=FAKE, kc=FAKE, vc=FAKE, kd=None, vd=None, table=FAKE, start=FAKE, count=None,
             B=2, Hkv=2, T=4, d=64, ps=16, P=8, mp=4, strides=None, Hq=4, window=0, scale=0.125,
             ws=FAKE, wsb=None, out=FAKE):
        if kind == "write":
            st = None if strides is None else (ctypes.c_int64 * 6)(*strides)
            return lib.kv_cache_write(x, x, st, kc, vc, kd, vd, table, start, count, B, Hkv, T, d,
                                      ps, P, mp, None)
        if kind == "read":
            return lib.kv_cache_read(kc, vc, kd, vd, table, start, count, x, x, B, Hkv, T, d, ps,
                                     P, mp, None)
        wsb = lib.attn_decode_workspace_size(d) if wsb is None else wsb
        return lib.attn_decode(x, kc, vc, kd, vd, table, start, out, out, B, Hq, Hkv, d, ps, P,
                               mp, window, scale, ws, wsb, None)
    return call


@pytest.mark.parametrize("kind", ["write", "read", "decode"])
def test_cache_validation(lib, kind):
    call = cache_args(kind)
    assert call(d=96) == UNSUPPORTED
    assert call(ps=8) == UNSUPPORTED and call(ps=24) == UNSUPPORTED
    assert call(ps=1 << 16, mp=1 << 15) == UNSUPPORTED       # positions beyond 31 bits
    assert call(ps=4096, mp=(1 << 19) - 1) == UNSUPPORTED    # or too near their end
    for bad in (dict(ps=0), dict(ps=-16), dict(P=0), dict(mp=0), dict(Hkv=0), dict(B=-1),
                dict(kc=None), dict(vc=FAKE + 8), dict(table=None), dict(table=FAKE + 2),
                dict(kd=FAKE), dict(vd=FAKE), dict(kd=FAKE, vd=FAKE + 2), dict(x=None),
                dict(x=FAKE + 8), dict(start=None), dict(start=FAKE + 1)):
        assert call(**bad) == INVALID, bad
    assert call(B=0, x=None, kc=None, vc=None, table=None, start=None) == OK


@pytest.mark.parametrize("kind", ["write", "read"])
def test_cache_rows_validation(lib, kind):
    call = cache_args(kind)
    assert call(T=-1) == INVALID
    assert call(T=0, x=None, kc=None, vc=None, table=None, start=None) == OK
    assert call(count=FAKE + 2) == INVALID
    assert call(B=1 << 12, Hkv=1 << 10, T=1 << 10) == UNSUPPORTED
    if kind == "write":
        assert call(strides=(64, 64, 4, 64, 64, 64)) == INVALID
        assert call(strides=(64, 64, 64, -8, 64, 64)) == INVALID


def test_decode_validation(lib):
    call = cache_args("decode")
    assert call(Hq=3) == INVALID and call(Hq=-2) == INVALID
    assert call(window=-1) == INVALID
    for s in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert call(scale=s) == INVALID
    assert call(out=None) == INVALID
    assert call(ws=None) == WORKSPACE and call(ws=FAKE + 16) == WORKSPACE
    assert call(wsb=lib.attn_decode_workspace_size(64) - 1) == WORKSPACE
    assert call(B=1 << 20, Hq=1 << 12) == UNSUPPORTED
    assert call(Hq=0, x=None, kc=None, vc=None, table=None, start=None) == OK
    assert lib.attn_decode_workspace_size(96) == 0
    assert lib.attn_decode_workspace_size(128) > lib.attn_decode_workspace_size(64) > 0
    assert lib.attn_decode_workspace_size(64) % 256 == 0


def test_binding_refuses_host_tensors():
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ab.attn_decode(q, kc, kc, i, i[0])
    with pytest.raises(ValueError, match="CUDA tensor"):
        ab.kv_cache_write(q, q, kc, kc, i, i[0])
    with pytest.raises(ValueError, match="CUDA tensor"):
        ab.kv_cache_read(kc, kc, i, i[0], 1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ab.rope_fwd(q, None, i[None], torch.ones(32))
    with pytest.raises(TypeError):
        ab.rope_fwd(None, None, i[None], torch.ones(32))
