"""The answering path as it is used: a prompt through rope_fwd, attn_fwd and
kv_cache_write, then one token after another through rope_fwd, kv_cache_write
and attn_decode; its training twin through attn_bwd and rope_bwd; captured in a
graph; and on two streams at once.

The answer of each step is held to the fp64 oracle on the same bf16 values,
with attn_decode's tolerance, and to attn_fwd's last row within both kernels'
own (1e-2 of the largest value, as its parity tests hold it).
"""

import math

import numpy as np
import pytest
import torch

import oracle
from attention_backward_pass_attn_gb300 import binding as ab
from attention_backward_pass_attn_gb300.inputs import make_tensor
from oracle import serving
from test_gpu_decode import check

pytestmark = pytest.mark.gpu

TOL = 1e-2


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


def freqs(d):
    return torch.tensor(10000.0 ** (-np.arange(d // 2) / (d // 2)), dtype=torch.float32).cuda()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,window", [(64, 0), (128, 0), (128, 50)])
def test_prompt_then_tokens(d, window, fp8):
    B, H, N, steps, page = 2, 4, 90, 5, 16
    prompt = [N, 61]                      # the second prompt is shorter: a padded batch
    qkv = make_tensor((B, N + steps, 3, H, d), 1000 + d).cuda()
    f = freqs(d)
    mp = -(-(N + steps) // page)
    kc, vc, kd, vd = ab.alloc_kv_cache(B * mp + 1, H, page, d, "cuda",
                                       torch.float8_e4m3fn if fp8 else torch.bfloat16)
    table = (torch.randperm(B * mp, generator=torch.Generator().manual_seed(3)) + 1)
    table = table.to(torch.int32).view(B, mp).cuda()
    lens = torch.tensor(prompt, dtype=torch.int32).cuda()
    zero = torch.zeros_like(lens)

    def heads(lo, hi):
        return (qkv[:, lo:hi, i].transpose(1, 2) for i in range(3))

    # the prompt
    q, k, v = heads(0, N)
    pos = torch.arange(N, dtype=torch.int32).view(1, 1, N).cuda()
    q, k = ab.rope_fwd(q, k, pos, f)
    v = v.contiguous()
    o, _ = ab.attn_fwd(q, k, v, True, window=window)
    ab.kv_cache_write(k, v, kc, vc, table, zero, lens, kd, vd)
    kr, vr = ab.kv_cache_read(kc, vc, table, zero, N, lens, kd, vd)
    if not fp8:
        for b in range(B):
            assert torch.equal(kr[b, :, :prompt[b]], k[b, :, :prompt[b]])
            assert torch.equal(vr[b, :, :prompt[b]], v[b, :, :prompt[b]])
    assert torch.all(kr[1, :, prompt[1]:] == 0)

    # one token after another
    keys, values = k, v
    for t in range(steps):
        q1, k1, v1 = heads(N + t, N + t + 1)
        q1, k1 = ab.rope_fwd(q1, k1, lens.view(1, B, 1), f)
        ab.kv_cache_write(k1, v1, kc, vc, table, lens, None, kd, vd)
        lens = lens + 1
        o1, l1 = ab.attn_decode(q1, kc, vc, table, lens, k_descale=kd, v_descale=vd, window=window)
        ref = serving.decode(q1, serving.cache_values(kc, kd), serving.cache_values(vc, vd), table,
                             lens, 1 / math.sqrt(d), window)
        check(o1, l1, ref, d)
        if not fp8:  # sequence 0 against the whole attention: its last row
            keys = torch.cat([keys[:1], k1[:1]], 2)
            values = torch.cat([values[:1], v1[:1].contiguous()], 2)
            qq = torch.zeros_like(keys)
            qq[:, :, -1:] = q1[:1]
            of, lf = ab.attn_fwd(qq, keys, values, True, window=window)
            assert float((of[0, :, -1].float() - o1[0, :, 0].float()).abs().max()) <= \
                2 * TOL * float(of[0, :, -1].float().abs().max())
            assert float((lf[0, :, -1] - l1[0, :, 0]).abs().max()) <= 2e-2


def test_training_through_rotary_positions():
    """rope_fwd -> attn_fwd -> attn_bwd -> rope_bwd against the oracle's chain
    (1e-2 of the largest value, the attention backward's tolerance, and the
    rotation's rounding of 2^-8 of it), and against a difference of the loss."""
    B, H, N, d = 1, 2, 100, 64
    q, k, v, do = (make_tensor((B, H, N, d), 50 + i) for i in range(4))
    f, sec = freqs(d), (12, 20)
    pos = torch.stack([torch.arange(N) // 10, torch.arange(N) % 10]).to(torch.int32).view(2, 1, N)
    qr, kr = ab.rope_fwd(q.cuda(), k.cuda(), pos.cuda(), f, sec)
    o, lse = ab.attn_fwd(qr, kr, v.cuda(), True)
    dq, dk, dv = ab.attn_bwd(qr, kr, v.cuda(), o, do.cuda(), lse, True)
    dq, dk = ab.rope_bwd(dq, dk, pos.cuda(), f, sec)
    scale = 1 / math.sqrt(d)

    def turned(x):
        return serving.rope(x, pos, f, sec)
    ref = oracle.attention_forward_backward(turned(q), turned(k), f64(v), f64(do), True, scale)
    rq = serving.rope(ref["dQ"], pos, f, sec, inverse=True)
    rk = serving.rope(ref["dK"], pos, f, sec, inverse=True)
    for g, r in ((dq, rq), (dk, rk), (dv, ref["dV"])):
        assert np.max(np.abs(f64(g) - r)) <= (TOL + 2.0 ** -8) * np.max(np.abs(r))
    # the loss <dO, O> along a direction, in fp64, against the GPU's gradient
    e = make_tensor((B, H, N, d), 60)
    h = 1e-4

    def loss(s):
        oo, _ = oracle.attention_forward(turned(f64(q) + s * f64(e)), turned(k), f64(v), True, scale)
        return float(np.sum(f64(do) * oo))
    num = (loss(h) - loss(-h)) / (2 * h)
    # |<dq - rq, e>| <= its tolerance in every element
    assert abs(num - np.sum(f64(dq) * f64(e))) <= \
        (TOL + 2.0 ** -8) * np.max(np.abs(rq)) * np.sum(np.abs(f64(e))) + 1e-6 * abs(num)


def step_state(seed, fp8=True, B=3, H=8, Hkv=2, d=128, page=32, n=700):
    g = torch.Generator().manual_seed(seed)
    mp = -(-n // page)
    kc, vc, kd, vd = ab.alloc_kv_cache(B * mp, Hkv, page, d, "cuda",
                                       torch.float8_e4m3fn if fp8 else torch.bfloat16)
    table = torch.randperm(B * mp, generator=g).to(torch.int32).view(B, mp).cuda()
    x = make_tensor((B, n, 2 * Hkv, d), seed).cuda()
    lens = torch.tensor([n - 40, n - 300, 5], dtype=torch.int32).cuda()
    ab.kv_cache_write(x[:, :, :Hkv].transpose(1, 2), x[:, :, Hkv:].transpose(1, 2), kc, vc, table,
                      torch.zeros_like(lens), lens, kd, vd)
    qkv = make_tensor((B, 1, H + 2 * Hkv, d), seed + 1).cuda()
    return dict(kc=kc, vc=vc, kd=kd, vd=vd, table=table, lens=lens, qkv=qkv, H=H, Hkv=Hkv, d=d, B=B,
                f=freqs(d), ws=ab.alloc_decode_workspace(d, "cuda"),
                q=torch.empty(B, H, 1, d, dtype=torch.bfloat16, device="cuda"),
                k=torch.empty(B, Hkv, 1, d, dtype=torch.bfloat16, device="cuda"),
                o=torch.empty(B, H, 1, d, dtype=torch.bfloat16, device="cuda"),
                lse=torch.empty(B, H, 1, dtype=torch.float32, device="cuda"),
                after=torch.empty_like(lens))


def step(s, stream=None):
    H, Hkv = s["H"], s["Hkv"]
    x = s["qkv"]
    ab.rope_fwd(x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2),
                s["lens"].view(1, s["B"], 1), s["f"], out=(s["q"], s["k"]), stream=stream)
    ab.kv_cache_write(s["k"], x[:, :, H + Hkv:].transpose(1, 2), s["kc"], s["vc"], s["table"],
                      s["lens"], None, s["kd"], s["vd"], stream=stream)
    torch.add(s["lens"], 1, out=s["after"])
    ab.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["after"], k_descale=s["kd"],
                   v_descale=s["vd"], out=s["o"], lse=s["lse"], workspace=s["ws"], stream=stream)


@pytest.mark.parametrize("fp8", [False, True])
def test_step_in_a_graph_follows_the_lengths(fp8):
    """A captured step replays on the lengths, tables and tokens of that
    moment, and gives the eager step's bits.  Two graphs share one workspace."""
    s = step_state(91, fp8)
    other = step_state(92, fp8)
    other["ws"] = s["ws"]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step(s)
        step(other)
    torch.cuda.synchronize()
    graphs = []
    for x in (s, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step(x)
        graphs.append(g)
    tokens = [make_tensor(s["qkv"].shape, 200 + i).cuda() for i in range(3)]
    got = []
    for t in tokens:
        for x, g in zip((s, other), graphs):
            x["qkv"].copy_(t)
            g.replay()
            got.append((x["o"].clone(), x["lse"].clone()))
            x["lens"].add_(1)
    torch.cuda.synchronize()
    eager = [step_state(91, fp8), step_state(92, fp8)]
    for x in eager:
        step(x)
    at = 0
    for t in tokens:
        for x in eager:
            x["qkv"].copy_(t)
            step(x)
            assert torch.equal(got[at][0], x["o"]) and torch.equal(got[at][1], x["lse"])
            x["lens"].add_(1)
            at += 1


def test_steps_on_two_streams_at_once():
    states = [step_state(95), step_state(96)]
    for x in states:
        step(x)
    torch.cuda.synchronize()
    ref = [(x["o"].clone(), x["lse"].clone()) for x in states]
    for x in states:
        x["o"].zero_()
        x["lse"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for x, s in zip(states, streams):
            with torch.cuda.stream(s):
                step(x)
    torch.cuda.synchronize()
    for x, (o, l) in zip(states, ref):
        assert torch.equal(x["o"], o) and torch.equal(x["lse"], l)


def test_chained_calls_see_finished_results():
    """No host synchronisation between calls that feed each other, many times:
    the kernels start before their predecessors end, and must wait for their
    data.  The same with a synchronisation after each call."""
    def chain(sync):
        s = step_state(99)
        outs = []
        for i in range(12):
            step(s)
            if sync:
                torch.cuda.synchronize()
            s["qkv"][:, 0, :s["H"]] = s["o"][:, :, 0]
            s["lens"].add_(1)
            outs.append(s["o"].clone())
        torch.cuda.synchronize()
        return outs
    for a, b in zip(chain(False), chain(True)):
        assert torch.equal(a, b)


def test_what_a_call_allocates_belongs_to_its_stream():
    """Results and workspaces of calls on another stream than the current one
    are not handed out again on the current one while that stream still works:
    a long queue of calls there, and allocations here meanwhile."""
    s = step_state(98)
    step(s)
    torch.cuda.synchronize()
    ref = s["o"].clone()
    other = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(30):
        with torch.cuda.stream(other):
            torch.mm(busy, busy)  # the calls below wait behind it
        o, lse = ab.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["after"],
                                k_descale=s["kd"], v_descale=s["vd"], stream=other)
        ab.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["after"], k_descale=s["kd"],
                       v_descale=s["vd"], stream=other)  # dropped at once
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(12)]
    other.synchronize()
    assert torch.equal(o, ref)
    del junk, lse
    for handle in (other.cuda_stream, other):
        with torch.cuda.stream(other):
            pass
        o, _ = ab.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["after"],
                              k_descale=s["kd"], v_descale=s["vd"], stream=handle)
        other.synchronize()
        assert torch.equal(o, ref)


def test_a_stream_argument_is_used():
    s = step_state(97)
    step(s)
    torch.cuda.synchronize()
    ref = s["o"].clone()
    s["o"].zero_()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        step(s, stream=other)
    other.synchronize()
    assert torch.equal(s["o"], ref)


def test_readme_example_runs():
    """The README's answering example, a step further than it goes: two tokens
    from empty sequences."""
    import os
    import re

    import attention_backward_pass_attn_gb300 as attn

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "README.md")).read()
    code = [b for b in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "attn_decode" in b]
    assert len(code) == 1
    scope = {"torch": torch, "attn": attn}
    exec(code[0], scope)
    first = scope["o"]
    x = torch.randn(2, 1, 48, 128, device="cuda").to(torch.bfloat16)
    second, lens = scope["token"](x, scope["lens"])
    assert first.shape == second.shape == (2, 32, 1, 128)
    assert torch.isfinite(first).all() and torch.isfinite(second).all()
    assert lens.tolist() == [2, 2]
    # one position: the answer is that position's value, as e4m3 rounds it
    assert torch.equal(first[:, ::4], first[:, 1::4])
