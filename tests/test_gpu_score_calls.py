"""How attention with changed scores is called: refusals, given outputs, other
streams, captured graphs, empty problems, and tensors of more than 2^31
elements."""

import math

import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab

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


def randn(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def operands(B=1, H=4, Hk=2, N=200, d=64, seed=0):
    return (randn(B, H, N, d, seed=seed), randn(B, Hk, N, d, seed=seed + 1),
            randn(B, Hk, N, d, seed=seed + 2), randn(B, H, N, d, seed=seed + 3))


def near(a, b):
    """dQ of two runs: fp32 sums in another order, then one rounding to bf16."""
    return float((a.float() - b.float()).abs().max()) <= 2 ** -7 * float(b.abs().max())


def test_refusals():
    q, k, v, do = operands()
    B, H, N, d = q.shape

    def fwd(q=q, k=k, v=v, causal=True, **kw):
        return ab.attn_fwd_score(q, k, v, causal, **kw)
    fwd()
    with pytest.raises(ValueError, match="multiple of k's"):
        fwd(k=randn(B, 3, N, d), v=randn(B, 3, N, d))
    with pytest.raises(ValueError, match="must not be expanded"):
        fwd(k=k[:, :1].expand(-1, 2, -1, -1))
    with pytest.raises(ValueError, match="torch.bfloat16"):
        fwd(q=q.half())
    with pytest.raises(ValueError, match="v must have shape"):
        fwd(v=v[:, :, :-1])
    with pytest.raises(ValueError, match="contiguous in its head dimension"):
        fwd(q=randn(B, H, d, N).transpose(2, 3))
    with pytest.raises(ValueError, match="multiples of 8"):
        fwd(q=randn(B, H, N, d + 4)[..., :d])
    with pytest.raises(ValueError, match="slopes must have shape"):
        fwd(slopes=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="slopes must be torch.float32"):
        fwd(slopes=torch.ones(H, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError, match="doc must be torch.int32"):
        fwd(doc=torch.zeros((B, N), device="cuda", dtype=torch.int64))
    with pytest.raises(ValueError, match="prefix must have shape"):
        fwd(prefix=torch.zeros((B + 1,), device="cuda", dtype=torch.int32))
    with pytest.raises(ValueError, match="on CUDA device"):
        fwd(slopes=torch.ones(H))
    with pytest.raises(ValueError, match="out must be contiguous"):
        fwd(out=randn(B, N, H, d).transpose(1, 2))
    pre = torch.zeros((B,), device="cuda", dtype=torch.int32)
    for kw in (dict(prefix=pre, window=3), dict(causal=False, prefix=pre), dict(causal=False, window=3),
               dict(softcap=-1.0), dict(softcap=math.inf), dict(softcap=math.nan), dict(scale=0.0),
               dict(window=-1)):
        with pytest.raises(ab.AttnError) as e:
            fwd(**kw)
        assert e.value.status == ab.ATTN_ERR_INVALID_ARG
    with pytest.raises(ab.AttnError) as e:
        fwd(q=randn(B, H, N, 32), k=randn(B, 2, N, 32), v=randn(B, 2, N, 32))
    assert e.value.status == ab.ATTN_ERR_UNSUPPORTED
    o, lse = fwd()
    with pytest.raises(ValueError, match="do must be contiguous"):
        ab.attn_bwd_score(q, k, v, o, randn(B, N, H, d).transpose(1, 2), lse, True)
    with pytest.raises(ab.AttnError) as e:
        ab.attn_bwd_score(q, k, v, o, do, lse, True,
                          workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    assert e.value.status == ab.ATTN_ERR_WORKSPACE
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        ab.attn_bwd_score(q, k, v, o, do, lse, True,
                          workspace=torch.empty(1 << 24, dtype=torch.uint8, device="cuda")[::2])


def test_given_outputs_and_workspace():
    q, k, v, do = operands()
    kw = dict(causal=True, softcap=4.0)
    o, lse = ab.attn_fwd_score(q, k, v, **kw)
    out, l2 = torch.empty_like(o), torch.empty_like(lse)
    got = ab.attn_fwd_score(q, k, v, out=out, lse=l2, **kw)
    assert got[0] is out and got[1] is l2 and torch.equal(out, o) and torch.equal(l2, lse)
    want = ab.attn_bwd_score(q, k, v, o, do, lse, **kw)
    ws = ab.alloc_score_workspace(1, 4, 2, 200, 64, q.device)
    mine = [torch.full_like(t, float("nan")) for t in (q, k, v)]
    for _ in range(2):  # whatever the workspace held
        got = ab.attn_bwd_score(q, k, v, o, do, lse, dq=mine[0], dk=mine[1], dv=mine[2], workspace=ws, **kw)
        assert all(a is b for a, b in zip(got, mine))
        assert near(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
        ws.fill_(0xFF)


@pytest.mark.parametrize("shape", [(0, 4, 2, 8), (2, 4, 2, 0), (2, 0, 2, 8)])
def test_empty_problems(shape):
    B, H, Hk, N = shape
    q, k = torch.empty((B, H, N, 64), dtype=torch.bfloat16, device="cuda"), \
        torch.empty((B, Hk, N, 64), dtype=torch.bfloat16, device="cuda")
    o, lse = ab.attn_fwd_score(q, k, k, True)
    assert o.shape == q.shape and lse.shape == q.shape[:3]
    if H:
        dq, dk, dv = ab.attn_bwd_score(q, k, k, o, o, lse, True)
        assert dq.shape == q.shape and dk.shape == k.shape and dv.shape == k.shape
    else:  # dK and dV would be sums of nothing
        with pytest.raises(ab.AttnError):
            ab.attn_bwd_score(q, k, k, o, o, lse, True)


@pytest.mark.parametrize("how", ["current", "argument"])
def test_other_streams(how):
    q, k, v, do = operands(B=2, N=700, d=128)
    kw = dict(causal=True, softcap=6.0, slopes=torch.tensor([0.1, 0.2, 0.3, 0.4], device="cuda"))
    o, lse = ab.attn_fwd_score(q, k, v, **kw)
    want = ab.attn_bwd_score(q, k, v, o, do, lse, **kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):  # calls that overlap, each with a workspace of its own
        for s in streams:
            if how == "current":
                with torch.cuda.stream(s):
                    f = ab.attn_fwd_score(q, k, v, **kw)
                    got.append((f, ab.attn_bwd_score(q, k, v, f[0], do, f[1], **kw)))
            else:
                f = ab.attn_fwd_score(q, k, v, stream=s, **kw)
                got.append((f, ab.attn_bwd_score(q, k, v, f[0], do, f[1], stream=s, **kw)))
    torch.cuda.synchronize()
    for f, b in got:
        assert torch.equal(f[0], o) and torch.equal(f[1], lse)
        assert near(b[0], want[0]) and torch.equal(b[1], want[1]) and torch.equal(b[2], want[2])


def test_captured_training_step_replays_on_new_inputs():
    static = operands(B=2, N=300, d=64)
    doc = torch.zeros((2, 300), dtype=torch.int32, device="cuda")
    kw = dict(causal=True, softcap=5.0, doc=doc)

    def step(q, k, v, do):
        o, lse = ab.attn_fwd_score(q, k, v, **kw)
        return (o, lse) + ab.attn_bwd_score(q, k, v, o, do, lse, **kw)
    step(*static)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs alive at once, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, step(*static)))
        graphs[-1] = (graph, graphs[-1][1])
    for seed in (10, 20, 30):
        for t, new in zip(static, operands(B=2, N=300, d=64, seed=seed)):
            t.copy_(new)
        starts = torch.tensor([0, seed], device="cuda")  # another packing too
        doc.copy_((torch.arange(300, device="cuda")[None] >= starts[:, None]).int() * starts[:, None].int())
        want = step(*static)
        for graph, got in graphs:
            graph.replay()
            for n, (a, b) in enumerate(zip(got, want)):
                assert near(a, b) if n == 2 else torch.equal(a, b)


def test_more_than_two_to_the_31_elements():
    """The last heads' offsets need 64 bits: they equal the same heads alone."""
    Hq, Hk, N, d = 132, 11, 131035, 128
    kw = dict(causal=True, softcap=20.0, window=200)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.empty((1, Hq, N, d), dtype=torch.bfloat16, device="cuda")
    do = torch.empty_like(q)
    for h in range(Hq):
        q[0, h] = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
        do[0, h] = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
    k, v = randn(1, Hk, N, d, seed=5), randn(1, Hk, N, d, seed=6)
    assert q.numel() > 2 ** 31
    o, lse = ab.attn_fwd_score(q, k, v, **kw)
    dq, dk, dv = ab.attn_bwd_score(q, k, v, o, do, lse, **kw)
    last = slice(Hq - 12, Hq)
    q1, do1, k1, v1 = q[:, last].clone(), do[:, last].clone(), k[:, -1:].clone(), v[:, -1:].clone()
    o1, lse1 = ab.attn_fwd_score(q1, k1, v1, **kw)
    assert torch.equal(o[:, last], o1) and torch.equal(lse[:, last], lse1)
    g1 = ab.attn_bwd_score(q1, k1, v1, o1, do1, lse1, **kw)
    assert torch.equal(dk[:, -1:], g1[1]) and torch.equal(dv[:, -1:], g1[2])
    assert near(dq[:, last], g1[0])
    # and the first rows of the last head against the definition
    x = (q1[0, -1, :100].float() @ k1[0, 0, :100].float().T) / math.sqrt(d)
    x = (20 * torch.tanh(x / 20)).masked_fill(torch.ones(100, 100, device="cuda").triu(1).bool(), -math.inf)
    ref = torch.softmax(x, -1) @ v1[0, 0, :100].float()
    # weights and result rounded to bf16, 2^-8 either, of values up to |v|
    assert float((o1[0, -1, :100].float() - ref).abs().max()) <= 2 ** -7 * float(v1[0, 0, :100].abs().max())


def test_rows_behind_each_other_keep_their_own():
    """Batch elements of different content do not mix, at a length that ends
    inside a tile."""
    q, k, v, do = operands(B=3, H=6, Hk=3, N=129, d=128, seed=9)
    kw = dict(causal=False, softcap=8.0)
    o, lse = ab.attn_fwd_score(q, k, v, **kw)
    got = ab.attn_bwd_score(q, k, v, o, do, lse, **kw)
    for b in range(3):
        one = slice(b, b + 1)
        o1, l1 = ab.attn_fwd_score(q[one], k[one], v[one], **kw)
        assert torch.equal(o[one], o1) and torch.equal(lse[one], l1)
        g1 = ab.attn_bwd_score(q[one], k[one], v[one], o1, do[one].contiguous(), l1, **kw)
        assert near(got[0][one], g1[0])
        assert torch.equal(got[1][one], g1[1]) and torch.equal(got[2][one], g1[2])
