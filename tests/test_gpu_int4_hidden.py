"""What the 4-bit cache holds at rows that no position falls on has no effect on
attention over it: not on the results, and not on the time."""

import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab
from test_gpu_score import cuda_ready  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("changed", [False, True])
@pytest.mark.parametrize("hidden", [0.0, float("nan"), 2.0 ** -120, 2.0 ** 100])
@pytest.mark.parametrize("first", [0, 5])
def test_factors_of_rows_that_are_not_seen_cost_nothing(first, hidden, changed):
    """A sequence that ends inside a run of sixteen rows, or a window that begins
    in one: the factors beside are read with the run.  Calls over factors of zero, NaN or far from the
    others' range take as long as over ones: at most a quarter more, where
    walking the last blocks' keys a second time takes them twice as long."""
    Hkv, d, page, n = 8, 128, 256, 131072 - 100
    P = -(-n // page)
    kc, vc, kf, vf = ab.alloc_kv_cache(P, Hkv, page, d, "cuda", "int4")
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (kc, vc):
        t.copy_(torch.randint(17, 256, t.shape, generator=g, device="cuda", dtype=torch.int32))
    table = torch.arange(P, dtype=torch.int32, device="cuda")[None].contiguous()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = torch.randn((1, 4 * Hkv, 1, d), generator=g, device="cuda").to(torch.bfloat16)
    kw = dict(window=n - first if first else 0, softcap=50.0 if changed else 0.0)
    times, results = [], []
    for value in (1.0, hidden):
        for f in (kf, vf):
            f[P - 1, :, n % page:], f[0, :, :first] = value, value
        call = lambda: ab.attn_decode(q, kc, vc, table, lens, k_descale=kf, v_descale=vf, **kw)  # noqa: E731
        results.append(call())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(20):
                call()
        best = float("inf")
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert times[1] <= 1.25 * times[0], "%.1f and %.1f us" % tuple(50 * t for t in times)
