"""Workspaces that the binding keeps: captured graphs, batches of changing size and streams at once.

A decode cut over CTAs counts its pieces in the workspace, from zero.  So a
graph must find its counters at zero whenever it is replayed, whatever other
calls and graphs ran since, and calls that may overlap must not share counters
or partials.
"""

import pytest
import torch

from parallax_local_linear_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from parallax_local_linear_b200 import binding
    return binding


KINDS = ["decode bf16", "decode f32", "projected", "lla", "q4"]


def _cuda(x):
    return {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in x.items()}


def _call(px, kind, batch, length, seed):
    """(f, want): f(out) makes the call into `out`; want is its result with a workspace of its own."""
    if kind == "q4":
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        x = dict(q=torch.randn(batch, 4, 128, device="cuda", generator=g).bfloat16(),
                 cache=px.q4_cache(batch * -(-length // 64), 2, 128))
        n = x["cache"].shape[0] * 64
        k, v = (torch.randn(n, 2, 128, device="cuda", generator=g).bfloat16() for _ in range(2))
        px.cache_append_q4(k, v, torch.arange(n, device="cuda"), x["cache"])
        cache = x["cache"].view(batch, -1, 2, 72 * 128).transpose(1, 2).contiguous()
        ws = px.decode_q4_workspace(x["q"], cache, kv_len=length, num_ctas=97)
        f = lambda out, **kw: px.decode_q4(x["q"], x["q"], cache, kv_len=length, out=out, num_ctas=97, **kw)
        return f, f(torch.empty(x["q"].shape, device="cuda"), workspace=ws).clone()
    if kind == "projected":
        x = _cuda(W.small_decode_inputs(batch, 4, 2, 128, length, dtype="bf16", seed=seed))
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        h = torch.randn(batch, 256, device="cuda", generator=g).bfloat16()
        w = [(torch.randn(512, 256, device="cuda", generator=g) / 16).bfloat16() for _ in range(2)]
        f = lambda out: px.decode_projected(h, *w, x["k_cache"], x["v_cache"], x["scale"], out=out, num_ctas=97)
        _, q, rho = f(torch.empty(batch, 4, 128, device="cuda"))
    else:
        dtype = "f32" if kind == "decode f32" else "bf16"
        x = _cuda(W.small_decode_inputs(batch, 4, 2, 128, length, dtype=dtype, seed=seed))
        q, rho = x["q"], x["rho"]
        if kind == "lla":
            f = lambda out: px.lla_decode(q, x["k_cache"], x["v_cache"], x["scale"], 0.5, out=out, num_ctas=97)
            want = torch.empty(q.shape, device="cuda")
            f(want)
            torch.cuda.synchronize()
            return f, want
        f = lambda out: px.decode(q, rho, x["k_cache"], x["v_cache"], x["scale"], out=out, num_ctas=97)
    plan = px.DecodePlan(q, rho, x["k_cache"], x["v_cache"], x["scale"], out=torch.empty(q.shape, device="cuda"),
                         num_ctas=97)
    return f, plan.run().clone()


def _out(want):
    return torch.full_like(want, float("nan"))


def _capture(f, out):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f(out)
    return g


@pytest.mark.parametrize("kind", KINDS)
def test_a_graph_of_a_large_batch_after_smaller_calls(px, kind):
    large, large_want = _call(px, kind, 400, 200, 1)
    small, small_want = _call(px, kind, 1, 8192, 2)
    for f, w in ((large, large_want), (small, small_want), (large, large_want)):    # warm up, the largest last
        out = _out(w)
        f(out)
        assert torch.equal(out, w)
    big = _out(large_want)
    g = _capture(large, big)
    for _ in range(2):
        small(_out(small_want))
        g.replay()
        assert torch.equal(big, large_want)
        big.fill_(float("nan"))
    little = _out(small_want)
    h = _capture(small, little)
    for graphs in ((h, g), (g, h, g)):
        big.fill_(float("nan"))
        little.fill_(float("nan"))
        for one in graphs:
            one.replay()
        assert torch.equal(big, large_want) and torch.equal(little, small_want)
    assert px.last_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_a_first_or_larger_call_made_under_capture(px, kind):
    # nothing that is only recorded may count as done for calls that are made at once
    f, want = _call(px, kind, 24, 400, 3)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    out = _out(want)
    with torch.cuda.graph(g, stream=s):
        f(out)
        f(out)
    with torch.cuda.stream(s):
        eager = _out(want)
        f(eager)
    torch.cuda.synchronize()
    assert torch.equal(eager, want)
    g.replay()
    assert torch.equal(out, want) and px.last_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_streams_and_graphs_at_once(px, kind):
    calls = [_call(px, kind, 3, 4000, 4), _call(px, kind, 40, 600, 5)]
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [[_out(w) for _ in range(20)] for _, w in calls]
    torch.cuda.synchronize()
    for i in range(20):
        for s, (f, _), o in zip(streams, calls, outs):
            with torch.cuda.stream(s):
                f(o[i])
    torch.cuda.synchronize()
    for (_, w), o in zip(calls, outs):
        assert all(torch.equal(t, w) for t in o)
    last = [_out(w) for _, w in calls]
    graphs = [_capture(f, o) for (f, _), o in zip(calls, last)]
    for _ in range(10):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, w), o in zip(calls, last):
        assert torch.equal(o, w)
    assert px.last_device_error() == 0


def test_a_graph_clears_its_counters_once(px):
    # one clearing for all the calls of a capture on a stream, however many there are
    f, want = _call(px, "decode bf16", 3, 4000, 6)
    out = _out(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f(out)
        before = torch.cuda.memory_allocated()
        for _ in range(5):
            f(out)
        assert torch.cuda.memory_allocated() == before
    for _ in range(3):
        out.fill_(float("nan"))
        g.replay()
        assert torch.equal(out, want)


def test_streams_and_captures_have_workspaces_of_their_own(px):
    # what overlapping calls write must lie apart, also where a race would rarely show
    index = torch.cuda.current_device()
    for kind, counters in (("decode", 512), ("q4", 512), ("lla", 0)):
        spans = []
        def take(nbytes):
            ws, room = px._kept_workspace(kind, index, nbytes, counters)
            assert ws.numel() - room >= nbytes and room >= counters
            spans.append((ws.data_ptr(), ws.data_ptr() + ws.numel()))
            return ws
        keep = [take(1000)]
        assert keep[0].data_ptr() == take(2000).data_ptr() and spans.pop()
        for s in (torch.cuda.Stream(), torch.cuda.Stream()):
            with torch.cuda.stream(s):
                keep.append(take(1000))
        graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
        for g in graphs:
            torch.cuda.synchronize()
            with torch.cuda.graph(g):
                keep.append(take(3 << 20))
        spans.sort()
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))


def test_decode_q4_in_place(px):
    # the output in the place of the queries or the probes: each unit's rows are read before they are written
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    n = 40 * 640
    k, v = (torch.randn(n, 2, 128, device="cuda", generator=g).bfloat16() for _ in range(2))
    cache = px.q4_cache(n // 64, 2, 128)
    px.cache_append_q4(k, v, torch.arange(n, device="cuda"), cache)
    cache = cache.view(40, -1, 2, 72 * 128).transpose(1, 2).contiguous()
    q, rho = (torch.randn(40, 8, 128, device="cuda", generator=g).bfloat16() for _ in range(2))
    lens = torch.randint(0, 641, (40,), device="cuda", dtype=torch.int32)
    for ctas in (0, 1, 148):
        want = px.decode_q4(q, rho, cache, seq_lens=lens, num_ctas=ctas)
        for place in (0, 1):
            x = [q.clone(), rho.clone()]
            assert torch.equal(px.decode_q4(*x, cache, seq_lens=lens, out=x[place], num_ctas=ctas), want)


def test_threads_on_one_stream(px):
    # calls of several host threads on one stream, of sizes that make the workspace grow between them
    import threading

    calls = [_call(px, kind, b, n, 9 + b) for kind in ("decode bf16", "q4") for b, n in ((1, 4000), (40, 600), (400, 200))]
    for key in [k for k in px._workspaces if k[0] in ("decode", "q4")]:
        del px._workspaces[key]
    bad = []

    def work(f, w):
        for _ in range(30):
            out = _out(w)
            f(out)
            if not torch.equal(out, w):
                bad.append(f)

    threads = [threading.Thread(target=work, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and px.last_device_error() == 0
