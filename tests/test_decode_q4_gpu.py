"""GPU parity of the 4-bit decode.

The reference is the oracle's explicit float64 decode on the keys and values
that the cache's blocks stand for.

Tolerance, per output row, with u = 2^-24 and weights w_i, a_i = rho.k_i, abar
from the reference.  A score is an fp32 sum of d exact products and a few
more: off by at most ds_i = scale (d + 16) 2u sum |q_c| (s n + |m|)_c (2u,
since the tensor cores may truncate), and a probe value by da_i = (d + 16) 2u
sum |rho_c| (s n + |m|)_c.  A weight is then off by at most 2 max ds of
itself, plus 2^-21 for the exponential and the 22 bits in which e and e a
enter the value product (fp16's half step, 2^-11, from 128 keys on), plus
(n + 64) 2u for the sums over n keys.  With
out = sum_i w_i (1 + abar - a_i) v_i, formed from two sums of size
sum w_i (1 + |a_i - a_ref|) |v_i| each at a common offset a_ref of the
probes, the error is at most
    sum_i w_i (1 + |abar| + |a_i| + 2 A) |V_i| e  +  sum_i w_i (da_i + sum_j w_j da_j) |V_i|
with e = 4 max ds + 2^-20 (or 2^-11) + (n + 64) 4u, |V_i| = (s n + |m|) of the value and
A = max |a_i| >= |a_ref|.  The output's own rounding (half a step) is added.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import serving_oracle as S
from tests.helpers import to_f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from parallax_local_linear_b200 import binding
    return binding


def _blocks(shape, d, g, scale=1.0, poison=None):
    """Random blocks: any code, scales about scale / 4, minima around -7.5 scales."""
    lead = tuple(shape)
    b = torch.randint(0, 256, lead + (72 * d,), dtype=torch.uint8, device="cuda", generator=g)
    s = 0.28 * scale * torch.exp(0.3 * torch.randn(lead + (2 * d,), device="cuda", generator=g))
    m = -7.5 * s + 0.5 * scale * torch.randn(lead + (2 * d,), device="cuda", generator=g)
    b[..., 64 * d:] = torch.stack([s, m], -1).bfloat16().view(torch.uint8).reshape(lead + (8 * d,))
    return b


def _inputs(lens, H, Hkv, d, paged=True, seed=0, rho=0.5, qs=1.0, kv=1.0, kv_len=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, longest = len(lens), max(max(lens), 1) if kv_len is None else kv_len
    width = -(-longest // 64)
    x = dict(q=(qs * torch.randn(B, H, d, device="cuda", generator=g)).bfloat16(),
             rho=(rho * torch.randn(B, H, d, device="cuda", generator=g)).bfloat16(),
             seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), kv_len=longest, lens=lens, d=d)
    if paged:
        need = [-(-n // 64) for n in lens]
        P = sum(need) + 3
        x["cache"] = _blocks((P, Hkv), d, g, kv)
        ids = np.random.default_rng(seed).permutation(P)
        table, at = np.full((B, width + 1), -1), 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        x["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    else:
        x["cache"], x["table"] = _blocks((B, Hkv, width), d, g, kv), None
    # rows past a sequence's end: NaN parameters
    G = d // 64
    for b, n in enumerate(lens):
        if n % 64 or (not paged and n < width * 64):
            pages = [n // 64] if paged else range(n // 64, width)
            for p in pages:
                at = x["cache"][int(x["table"][b, p])] if paged else x["cache"][b, :, p]
                par = at[:, 64 * d:].view(torch.bfloat16).view(-1, 2, 64, G, 2)
                par[:, :, n % 64 if p == n // 64 else 0:] = float("nan")
    return x


def _run(px, x, scale, **kw):
    return px.decode_q4(x["q"], x["rho"], x["cache"], scale, seq_lens=x["seq_lens"], page_table=x["table"],
                        kv_len=x["kv_len"], **kw)


def _reference(x, scale):
    """(out, bound without the output's rounding), float64 [B, Hq, d]."""
    q, rho, d = to_f64(x["q"]), to_f64(x["rho"]), x["d"]
    B, H, _ = q.shape
    Hkv = x["cache"].shape[1]
    out, bound = np.zeros_like(q), np.zeros_like(q)
    mag = x["cache"].cpu().numpy().copy()
    par = np.ascontiguousarray(mag[..., 64 * d:]).view(np.uint16)
    par[..., 1::2] &= 0x7fff          # |m|
    mag[..., 64 * d:] = par.view(np.uint8)
    cache = x["cache"].cpu().numpy()
    for b, n in enumerate(x["lens"]):
        if n == 0:
            continue
        pages = -(-n // 64)
        for kvh in range(Hkv):
            pick = (lambda c: c[x["table"][b, :pages].cpu().numpy(), kvh]) if x["table"] is not None else \
                (lambda c: c[b, kvh, :pages])
            with np.errstate(invalid="ignore"):
                (k, v), (ka, va) = (tuple(t.reshape(-1, d)[:n] for t in S.q4_unblock(pick(c), d))
                                    for c in (cache, mag))
            for h in range(kvh * H // Hkv, (kvh + 1) * H // Hkv):
                out[b, h] = oracle.parallax_query(q[b, h], rho[b, h], k, v, scale)
                w = oracle.softmax_weights(scale * (k @ q[b, h]))
                a = k @ rho[b, h]
                ds = abs(scale) * (d + 16) * 2 * U * (ka @ np.abs(q[b, h])).max()
                da = (d + 16) * 2 * U * (ka @ np.abs(rho[b, h]))
                e = 4 * ds + (2.0 ** -20 if n < 128 else 2.0 ** -11) + (n + 64) * 4 * U
                coef = w * (1 + abs(w @ a) + np.abs(a) + 2 * np.abs(a).max()) * e + w * (da + w @ da)
                bound[b, h] = coef @ va
    return out, bound


def _check(px, x, scale=None, out_dtype=torch.float32, **kw):
    scale = x["d"] ** -0.5 if scale is None else scale
    ref, bound = _reference(x, scale)
    px.last_device_error()
    got = to_f64(_run(px, x, scale, out_dtype=out_dtype, **kw))
    h = torch.finfo(out_dtype).eps / 2
    assert np.isfinite(got).all()
    over = np.abs(got - ref) - (bound * (1 + h) + h * np.abs(ref))
    assert (over <= 0).all(), f"{over.max():.3e} over, at {np.unravel_index(over.argmax(), over.shape)}"
    assert px.last_device_error() == 0
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1], [2, 0, 63], [64], [65, 1, 128], [200, 129, 0, 1000]], ids=str)
@pytest.mark.parametrize("paged", [True, False])
def test_lengths(px, d, lens, paged):
    _check(px, _inputs(lens, 4, 2, d, paged, seed=len(lens) + d))


@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 1), (3, 1), (4, 1), (5, 1), (7, 1), (8, 1), (16, 8), (12, 2), (32, 4)])
def test_head_groups(px, H, Hkv):
    _check(px, _inputs([70, 300], H, Hkv, 128, seed=H))
    _check(px, _inputs([130, 3], H, Hkv, 64, seed=H, paged=False))


@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 148, 1000])
def test_grids(px, ctas):
    # any split of the work gives the definition
    x = _inputs([500, 1, 0, 64, 777, 3000], 4, 2, 128, seed=5)
    _check(px, x, num_ctas=ctas)


def test_many_sequences(px):
    rng = np.random.default_rng(1)
    _check(px, _inputs(rng.integers(0, 200, 300).tolist(), 4, 2, 64, seed=6))


def test_long_sequence(px):
    _check(px, _inputs([40000, 5], 4, 1, 128, seed=7))


def test_output_types_and_given_output(px):
    x = _inputs([100, 33], 4, 2, 128, seed=8)
    _check(px, x, out_dtype=torch.bfloat16)
    out = torch.empty(2, 4, 128, device="cuda")
    assert px.decode_q4(x["q"], x["rho"], x["cache"], seq_lens=x["seq_lens"], page_table=x["table"], out=out) is out
    assert torch.equal(out, _run(px, x, None, out_dtype=torch.float32))


@pytest.mark.parametrize("rho,qs,kv", [(0.0, 1.0, 1.0), (1.0, 1.0, 1.0), (30.0, 4.0, 1.0), (1e-6, 1e-3, 1e-4),
                                       (1.0, 1e-4, 300.0), (2e-3, 2e-3, 1e9), (1e9, 1e9, 1e-9), (1.0, 0.0, 1.0)])
def test_magnitudes(px, rho, qs, kv):
    _check(px, _inputs([300, 1, 64], 4, 2, 128, seed=9, rho=rho, qs=qs, kv=kv))


def test_scales_between_groups_and_tokens(px):
    # value groups whose scales differ by many powers of two, some of them zero (constant groups)
    x = _inputs([200, 64], 4, 2, 128, seed=10)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    par = x["cache"][..., 64 * 128:].view(torch.bfloat16).view(-1, 2, 2, 64, 2, 2)
    par *= torch.exp2(torch.randint(-12, 13, par.shape[:-1] + (1,), device="cuda", generator=g).float()).bfloat16()
    par[:, :, :, ::5, :, 0] = 0
    # (the keys' own scales stay moderate, or every row would be one key's)
    par[:, :, 0] = 0.25 * torch.nan_to_num(par[:, :, 0] / par[:, :, 0].abs().clamp(min=1e-20)) + 0 * par[:, :, 0]
    _check(px, x)


def test_peaked_rows_and_negative_scale(px):
    _check(px, _inputs([500], 4, 2, 128, seed=11), scale=1.5)
    _check(px, _inputs([500], 4, 2, 128, seed=12), scale=-0.1)
    _check(px, _inputs([500], 4, 2, 128, seed=13), scale=0.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv_len", [1, 63, 64, 200, 1000])
@pytest.mark.parametrize("H,Hkv", [(4, 2), (7, 1)])
def test_contiguous_without_lengths(px, d, kv_len, H, Hkv):
    # every sequence has kv_len tokens; kv_len need not fill its last page
    x = _inputs([kv_len] * 3, H, Hkv, d, paged=False, seed=kv_len)
    ref, bound = _reference(x, 0.1)
    got = px.decode_q4(x["q"], x["rho"], x["cache"], 0.1, kv_len=kv_len, out_dtype=torch.float32)
    assert (np.abs(to_f64(got) - ref) <= bound * (1 + U) + U * np.abs(ref)).all()
    if kv_len % 64 == 0:
        assert torch.equal(px.decode_q4(x["q"], x["rho"], x["cache"], 0.1, out_dtype=torch.float32), got)


def test_a_pool_past_32_bits(px):
    # 4.9 GB of blocks: pages, slots and rows beyond 2^32 bytes
    P, Hkv, d, n = 265_000, 2, 128, 150
    cache = torch.empty(P, Hkv, 72 * d, dtype=torch.uint8, device="cuda")
    pages = torch.tensor([[P - 1, 3, P - 7]], dtype=torch.int32, device="cuda")
    t = torch.arange(n, device="cuda")
    slots = pages[0, t // 64].long() * 64 + t % 64
    k, v = (torch.randn(n, Hkv, d, device="cuda").bfloat16() for _ in range(2))
    px.cache_append_q4(k, v, slots, cache)
    small = px.q4_cache(3, Hkv, d)
    px.cache_append_q4(k, v, t, small)
    for a, b in zip(px.cache_gather_q4(cache, slots), px.cache_gather_q4(small, t)):
        assert torch.equal(a, b)
    q, rho = (torch.randn(1, 4, d, device="cuda").bfloat16() for _ in range(2))
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = px.decode_q4(q, rho, cache, seq_lens=lens, page_table=pages)
    assert torch.equal(got, px.decode_q4(q, rho, small, seq_lens=lens,
                                         page_table=torch.arange(3, dtype=torch.int32, device="cuda")[None]))
    assert px.last_device_error() == 0


@pytest.mark.parametrize("step", [-4.0, 0.7, 1.9, 4.0])
@pytest.mark.parametrize("H", [4, 8])
def test_scores_and_values_that_rise_from_page_to_page(px, step, H):
    # every page's scores lie about `step` powers of two above (or below) the last page's, its
    # values' scales one power above: the running reference moves at every page, at some, at none
    x = _inputs([1500, 130, 90], H, 1, 128, paged=False, seed=7)
    x["q"] = x["q"].abs()
    par = x["cache"][..., 64 * 128:].view(torch.bfloat16).view(3, -1, 2, 64, 2, 2)
    p = torch.arange(par.shape[1], device="cuda").view(1, -1, 1, 1)
    mean = float(x["q"].float().sum(-1).mean())
    par[:, :, 0, :, :, 1] = (par[:, :, 0, :, :, 1] + step * np.log(2.0) * 128 ** 0.5 / mean * p).bfloat16()
    par[:, :, 1] = (par[:, :, 1].float() * torch.exp2((p % 8).float())[..., None]).bfloat16()
    _check(px, x)


def test_not_a_number_stays_in_its_rows(px):
    # NaN or infinities in one query, probe or key row reach that row's outputs and no other
    x = _inputs([100, 70], 4, 2, 128, seed=40)
    want = _run(px, x, None)
    x["q"][0, 1, 5] = float("nan")
    x["rho"][1, 2, 7] = float("inf")
    got = _run(px, x, None)
    bad = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 2] = True
    assert torch.equal(got[~bad], want[~bad]) and not torch.isfinite(got[bad].float()).any()


def test_bad_lengths_and_pages_are_reported(px):
    x = _inputs([100, 70], 4, 2, 64, seed=14)
    x["table"][0, 1] = x["cache"].shape[0]
    px.last_device_error()
    out = _run(px, x, None)
    assert px.last_device_error() == px.DEVERR_BAD_PAGE
    ok = _inputs([100, 70], 4, 2, 64, seed=14)
    assert torch.equal(out[1], _run(px, ok, None)[1])
    x["table"][0, 1] = -1
    _run(px, x, None)
    assert px.last_device_error() == px.DEVERR_BAD_PAGE
    y = _inputs([100, 70], 4, 2, 64, seed=14, paged=False)
    y["seq_lens"][0] = -3
    out = _run(px, y, None)
    assert px.last_device_error() == px.DEVERR_BAD_LENGTH and (out[0] == 0).all()
    y["seq_lens"][0] = 101
    _run(px, y, None)
    assert px.last_device_error() == px.DEVERR_BAD_LENGTH


def test_empty_cache(px):
    x = _inputs([0, 0], 4, 2, 64, seed=15)
    assert (_run(px, x, None) == 0).all()


def test_repeatable_and_workspace_is_left_clean(px):
    a = _inputs([3000, 17, 900], 4, 2, 128, seed=16)
    b = _inputs([64, 5000], 8, 1, 64, seed=17)
    first = _run(px, a, None), _run(px, b, None)
    for _ in range(5):
        assert torch.equal(_run(px, a, None), first[0]) and torch.equal(_run(px, b, None), first[1])


def test_streams_and_graphs(px):
    a, b = _inputs([3000, 17, 900], 4, 2, 128, seed=18), _inputs([2500, 1, 64], 4, 2, 128, seed=19)
    want = [_run(px, x, None) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(_run(px, x, None))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(g, want[i]) for g in got[i])
    graphs = []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _run(px, x, None)
        graphs.append((g, out))
    for _ in range(20):
        for i, (g, _) in enumerate(graphs):
            with torch.cuda.stream(streams[i]):
                g.replay()
    torch.cuda.synchronize()
    for i, (_, out) in enumerate(graphs):
        assert torch.equal(out, want[i])
    assert px.last_device_error() == 0


def test_given_workspace(px):
    # one workspace in a captured graph and in direct calls; too small or misplaced ones are refused
    x = _inputs([3000, 17, 900], 4, 2, 128, seed=30)
    want = _run(px, x, None)
    ws = px.decode_q4_workspace(x["q"], x["cache"], page_table=x["table"], kv_len=x["kv_len"])
    assert torch.equal(_run(px, x, None, workspace=ws), want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _run(px, x, None, workspace=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    assert torch.equal(_run(px, x, None, workspace=ws), want)
    for bad in (ws[:-256], ws[256:]):
        with pytest.raises(px.ParallaxError):
            _run(px, x, None, workspace=bad)
    with pytest.raises(TypeError):
        _run(px, x, None, workspace=ws.view(torch.int32))


def test_serving_step(px):
    """Lengths to output: page plan, norm with rotation, 4-bit append, 4-bit decode, over several steps."""
    torch.manual_seed(20)
    B, H, Hkv, d, P = 3, 4, 2, 128, 40
    cos, sin = (f(torch.arange(512, device="cuda")[:, None].double()
                  * 10000.0 ** (-torch.arange(0, d, 2, device="cuda") / d)).float() for f in (torch.cos, torch.sin))
    w = [(1 + 0.1 * torch.randn(d, device="cuda")).bfloat16() for _ in range(3)]
    table = torch.full((B, 6), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(P, device="cuda").int()
    cache = px.q4_cache(P, Hkv, d)
    cached = torch.zeros(B, dtype=torch.int32, device="cuda")
    head = torch.zeros(1, dtype=torch.int32, device="cuda")
    keys, values = [[] for _ in range(B)], [[] for _ in range(B)]
    for new in ([70, 3, 128], [1, 1, 1], [0, 62, 1], [1, 1, 0], [1, 1, 1]):
        rows = sum(new) + 2
        plan = px.page_plan(cached, _dev(new), table, free, num_rows=rows, num_pages=P, free_head=head)
        q, rho, k, v = (torch.randn(rows, h, d, device="cuda").bfloat16() for h in (H, H, Hkv, Hkv))
        q, rho, k = px.norm_rope(q, rho, k, cos, sin, plan.positions, q_weight=w[0], rho_weight=w[1], k_weight=w[2])
        px.cache_append_q4(k, v, plan.slot_map, cache)
        cu = plan.cu_seqlens.tolist()
        for b in range(B):
            keys[b] += list(k[cu[b]:cu[b + 1]].float().cpu().numpy())
            values[b] += list(v[cu[b]:cu[b + 1]].float().cpu().numpy())
        # every request's last new token (or any row where it has none) asks
        last = (plan.cu_seqlens[1:] - 1).clamp(min=0).long()
        out = px.decode_q4(q[last], rho[last], cache, seq_lens=plan.seq_lens, page_table=table)
        lens = plan.seq_lens.tolist()
        assert lens == [len(x) for x in keys]
        x = dict(q=q[last], rho=rho[last], cache=cache, table=table, lens=lens, d=d)
        ref, bound = _reference(x, d ** -0.5)
        assert (np.abs(to_f64(out) - ref) <= bound * 1.01 + 2.0 ** -8 * np.abs(ref)).all()
        for b in range(B):     # and the cache holds what was appended, quantised
            t = torch.arange(lens[b], device="cuda")
            slots = table[b, t // 64].long() * 64 + t % 64
            kq, vq = px.cache_gather_q4(cache, slots, out_dtype=torch.float32)
            for got, rows_ in ((kq, keys[b]), (vq, values[b])):
                want = S.q4_values(*S.q4_quantise(np.stack(rows_)))
                assert (np.abs(to_f64(got) - want) <= U * np.abs(want)).all()
        cached, head = plan.seq_lens, head + plan.pages_used
    assert px.last_device_error() == 0


def test_serving_step_with_plain_pools(px):
    """The same step over bf16 pools: append, chunked prefill of the prompts, decode of the next tokens."""
    torch.manual_seed(21)
    B, H, Hkv, d, P = 2, 4, 2, 128, 20
    table = torch.full((B, 4), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(P, device="cuda").int()
    kc, vc = (torch.full((P, Hkv, 64, d), float("nan"), device="cuda").bfloat16() for _ in range(2))
    new = [100, 65]
    plan = px.page_plan(_dev([0, 0]), _dev(new), table, free, num_rows=165, num_pages=P)
    q, rho, k, v = (torch.randn(165, h, d, device="cuda").bfloat16() for h in (H, H, Hkv, Hkv))
    px.cache_append(k, v, plan.slot_map, kc, vc)
    out = px.prefill_paged(q, rho, kc, vc, table, plan.cu_seqlens, plan.seq_lens, max_q_len=100,
                           out_dtype=torch.float32)
    last = (plan.cu_seqlens[1:] - 1).long()
    dec = px.decode(q[last], rho[last], kc, vc, seq_lens=plan.seq_lens, page_table=table, out_dtype=torch.float32)
    at = 0
    for b, n in enumerate(new):
        for h in range(H):
            ref = oracle.parallax_query(to_f64(q[at + n - 1, h]), to_f64(rho[at + n - 1, h]),
                                        to_f64(k[at:at + n, h // 2]), to_f64(v[at:at + n, h // 2]), d ** -0.5)
            for got in (out[at + n - 1, h], dec[b, h]):
                assert (np.abs(to_f64(got) - ref) <= 2e-2 * (1 + np.abs(ref))).all()
        at += n
    assert px.last_device_error() == 0


def test_training_step_through_norm_and_attention(px):
    """NormRope into ParallaxPrefill and back: gradients against differences of the float64 definition."""
    torch.manual_seed(22)
    B, H, Hkv, T, d = 1, 2, 1, 20, 128
    cos, sin = (f(torch.arange(T, device="cuda")[:, None].double()
                  * 10000.0 ** (-torch.arange(0, d, 2, device="cuda") / d)).float() for f in (torch.cos, torch.sin))
    raw = [torch.randn(B, h, T, d, device="cuda").bfloat16().requires_grad_() for h in (H, H, Hkv, Hkv)]
    w = [(s * (1 + 0.1 * torch.randn(d, device="cuda"))).bfloat16().requires_grad_() for s in (1, 0.1, 1)]
    q, rho, k = px.NormRope.apply(*raw[:3], *w, cos, sin)
    out = px.ParallaxPrefill.apply(q, rho, k, raw[3])
    dout = torch.randn_like(out)
    got = torch.autograd.grad(out, raw + w, dout)
    # the chain by the oracle, with the attention's gradients at the same rounded q, rho, k
    dq, dr, dk, dv = oracle.prefill_grads(*(to_f64(t.detach()) for t in (q, rho, k, raw[3])), to_f64(dout), d ** -0.5)
    R = S.rotation(cos.cpu().numpy(), sin.cpu().numpy(), np.arange(T), d, False)
    rows = lambda x: np.asarray(x).transpose(0, 2, 1, 3).reshape(T, -1, d)
    for x, wt, dy, gx, gw in zip(raw, w, (dq, dr, dk), got[:3], got[4:]):
        dx, dw = S.norm_rope_grad(rows(to_f64(x.detach())), rows(dy), to_f64(wt.detach()), R, 1e-6)
        # attention's own gradients keep 2e-2 of their size (its stated tolerance), which the norm's linear map carries on
        size = np.sqrt((dx ** 2).mean())
        assert np.abs(rows(to_f64(gx)) - dx).max() <= 4e-2 * (size + np.abs(dx).max())
        assert np.abs(to_f64(gw) - dw).max() <= 4e-2 * (np.sqrt((dw ** 2).mean()) + np.abs(dw).max())
    assert np.abs(to_f64(got[3]) - np.asarray(dv)).max() <= 2e-2 * (1 + np.abs(dv).max())


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")
