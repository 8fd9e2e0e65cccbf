"""Calls of the answering path that its documentation allows and whose sizes or
streams are out of the ordinary."""

import ctypes
import os
import re
import subprocess
import sys
import threading

import pytest
import torch

import attention_backward_pass_attn_gb300 as attn
from attention_backward_pass_attn_gb300 import binding as ab
from attention_backward_pass_attn_gb300.inputs import make_tensor
from test_gpu_decode import cuda_ready, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def small(B=2, Hkv=2, d=64, page=16, n=70, seed=5):
    """A cache with its table and lengths, and queries, on the GPU."""
    mp = -(-n // page)
    kc, vc, _, _ = ab.alloc_kv_cache(B * mp, Hkv, page, d, "cuda")
    table = torch.arange(B * mp, dtype=torch.int32).view(B, mp).cuda()
    x = make_tensor((B, Hkv, n, d), seed).cuda()
    ab.kv_cache_write(x, x, kc, vc, table, torch.zeros(B, dtype=torch.int32, device="cuda"))
    return make_tensor((B, 2 * Hkv, 1, d), seed + 1).cuda(), kc, vc, table, i32([n] * B).cuda()


def same(a, b):
    return torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_kept_workspaces_of_two_streams_at_once():
    """Long sequences, so that every block leaves parts, on two streams of the
    pool that take turns, without a workspace of the caller's."""
    batches = [small(B=1, n=5000 + 900 * i, seed=20 + i) for i in range(2)]
    ref = [ab.attn_decode(*x) for x in batches]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for x, s, g in zip(batches, streams, got):
            with torch.cuda.stream(s):
                g.append(ab.attn_decode(*x))
    torch.cuda.synchronize()
    for g, r in zip(got, ref):
        assert all(same(x, r) for x in g)
    held = {h for _, h in ab._decode_workspaces}
    assert {s.cuda_stream for s in streams} <= held


def external_stream():
    cudart = torch.cuda.cudart()
    handle = ctypes.c_void_p()
    assert int(cudart.cudaStreamCreate(ctypes.addressof(handle))) == 0
    return handle.value, cudart


@pytest.mark.parametrize("given", [False, True])
def test_streams_of_another_owner_have_no_kept_workspace(given):
    args = small(n=3000)
    ref = ab.attn_decode(*args)
    torch.cuda.synchronize()
    for _ in range(3):
        handle, cudart = external_stream()
        if given:
            got = ab.attn_decode(*args, stream=handle)
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(handle)):
                got = ab.attn_decode(*args)
        torch.cuda.synchronize()
        assert same(got, ref)
        assert handle not in {h for _, h in ab._decode_workspaces}
        assert int(cudart.cudaStreamDestroy(handle)) == 0


def test_the_per_thread_stream_takes_a_workspace():
    args = small(n=3000)
    ref = ab.attn_decode(*args)
    ws = ab.alloc_decode_workspace(64, "cuda")
    out, lse = torch.zeros_like(ref[0]), torch.zeros_like(ref[1])
    torch.cuda.synchronize()
    with pytest.raises(ValueError, match="workspace"):
        ab.attn_decode(*args, stream=2)
    ab.attn_decode(*args, out=out, lse=lse, workspace=ws, stream=2)
    torch.cuda.synchronize()
    assert same((out, lse), ref)


def test_a_workspace_that_is_not_its_own_memory_is_refused():
    """An expanded byte has as many bytes as asked for, and memory for one."""
    args = small()
    n = ab.load_library().attn_decode_workspace_size(64)
    one = torch.zeros(1, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        ab.attn_decode(*args, workspace=one.expand(n))
    with pytest.raises(ValueError, match="contiguous"):
        ab.attn_decode(*args, workspace=torch.zeros(n, 2, dtype=torch.uint8, device="cuda")[:, 0])
    with pytest.raises(TypeError):
        ab.attn_decode(*args, workspace=n)


def test_windows_beyond_32_bits_are_not_wrapped():
    args = small()
    whole = ab.attn_decode(*args)
    for w in (70, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 40):
        assert same(ab.attn_decode(*args, window=w), whole)
    assert not same(ab.attn_decode(*args, window=5), whole)
    for w in (-1, -2 ** 31, -2 ** 32, -2 ** 32 + 5):
        with pytest.raises(ab.AttnError) as e:
            ab.attn_decode(*args, window=w)
        assert e.value.status == ab.ATTN_ERR_INVALID_ARG


def test_an_append_beyond_32_bits_is_refused():
    """One token in memory, expanded to more than an int's worth of tokens."""
    _, kc, vc, table, _ = small()
    before = kc.clone()
    x = torch.ones(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    for T in (2 ** 29, 2 ** 31, 2 ** 32 + 1):
        x4 = x.expand(2, 2, T, 64)
        with pytest.raises(ab.AttnError) as e:
            ab.kv_cache_write(x4, x4, kc, vc, table, start)
        assert e.value.status == ab.ATTN_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert torch.equal(kc, before)


def test_heads_whose_values_pass_31_bits():
    """2^24 heads of 128 values: an empty sequence's zeros, and a sequence of
    one position, whose answer is its value."""
    H, d = 1 << 24, 128
    kc, vc, _, _ = ab.alloc_kv_cache(2, 1, 16, d, "cuda")
    v = make_tensor((1, 1, 1, d), 3).cuda()
    table = i32([[0], [1]]).cuda()
    kc[1, 0, 0], vc[1, 0, 0] = v[0, 0, 0], v[0, 0, 0]
    q = torch.zeros(2, H, 1, d, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, float("nan"))
    o, lse = ab.attn_decode(q, kc, vc, table, i32([0, 1]).cuda(), out=out)
    assert bool((o[0] == 0).all()) and bool(torch.isneginf(lse[0]).all())
    assert bool((o[1] == v[0]).all()) and bool((lse[1] == 0).all())


def test_readme_prompt_and_tokens():
    """The README's prompt with shared key heads and a padded batch, and the
    prompt's last tokens once more as tokens after the rest of it: attn_fwd's
    last rows, each kernel within 1e-2 of the largest value as its own tests
    hold it, over a bf16 cache; and over the README's e4m3 one it runs."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "README.md")).read()
    code = [b for b in re.findall(r"```python\n(.*?)```", text, flags=re.S)
            if "kv_cache_write" in b]
    assert len(code) == 2
    scope = {"torch": torch, "attn": attn}
    for b in code:
        exec(b, scope)
    x = make_tensor((2, 90, 48, 128), 12).cuda()
    n = torch.tensor([90, 33], dtype=torch.int32).cuda()
    last = x[torch.arange(2), (n - 1).long().cpu()].unsqueeze(1)
    for e4m3 in (True, False):
        if not e4m3:
            scope["kc"], scope["vc"], scope["ks"], scope["vs"] = ab.alloc_kv_cache(
                4096, 8, 64, 128, "cuda")
        o, lens = scope["prompt"](x, n)
        assert o.shape == (2, 32, 90, 128) and lens is n
        o1, after = scope["token"](last, lens - 1)
        assert torch.equal(after, n) and torch.isfinite(o1).all()
    for b in range(2):
        want, got = o[b, :, int(n[b]) - 1].float(), o1[b, :, 0].float()
        assert float((want - got).abs().max()) <= 2e-2 * float(want.abs().max())


COLD = """
import torch
import attention_backward_pass_attn_gb300 as attn

B, H, Hkv, d = 2, 4, 2, 64
g = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn(B, 1, H + 2 * Hkv, d, device="cuda", generator=g).to(torch.bfloat16)
freq = torch.ones(d // 2, device="cuda")
table = torch.arange(8, dtype=torch.int32, device="cuda").view(B, 4)
lens = torch.full((B,), 20, dtype=torch.int32, device="cuda")
kc, vc, ks, vs = attn.alloc_kv_cache(8, Hkv, 16, d, "cuda", torch.float8_e4m3fn)
after = lens + 1
torch.cuda.synchronize()

def step():
    q, k, v = (t.transpose(1, 2) for t in x.split((H, Hkv, Hkv), dim=2))
    q, k = attn.rope_fwd(q, k, lens.view(1, B, 1), freq)
    attn.kv_cache_write(k, v, kc, vc, table, lens, k_descale=ks, v_descale=vs)
    o, lse = attn.attn_decode(q, kc, vc, table, after, k_descale=ks, v_descale=vs)
    kr, vr = attn.kv_cache_read(kc, vc, table, lens, 1, k_descale=ks, v_descale=vs)
    return o, lse, kr, vr, attn.rope_bwd(q, k, lens.view(1, B, 1), freq)[0]

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
for a, b in zip(got, step()):
    assert torch.equal(a, b)
assert attn.attn_last_device_error() == 0
"""


def test_a_process_may_begin_with_a_capture():
    """The first calls of a process, captured: nothing of their set-up is
    forbidden there."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", COLD], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert p.returncode == 0, p.stderr


def test_threads_on_streams_of_their_own():
    """Host threads that call at once, each on a stream of the pool, without
    workspaces of the caller's."""
    batches = [small(B=1, n=4000 + 333 * i, seed=40 + i) for i in range(4)]
    ref = [ab.attn_decode(*x) for x in batches]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [ab.attn_decode(*batches[i]) for _ in range(50)]
            torch.cuda.current_stream().synchronize()
        wrong.extend(i for g in got if not same(g, ref[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
