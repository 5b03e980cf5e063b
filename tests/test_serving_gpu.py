"""GPU parity of the page plan, the head norm with rotation and the cache rows.

References are the float64 / integer definitions of oracle.serving_oracle on
the same inputs.  Whole numbers, codes and copied rows have to be equal.

Tolerances.  A value rounded once to T is off by finfo(T).eps / 2 of itself.
Before that, norm_rope works in fp32 (u = 2^-24): the sum of d squares is off
by at most (d + 2) u of itself in any order and rsqrtf by 2 ulp, so r by less
than (d / 2 + 6) u; the products and the two terms of the rotation add fewer
than 10 u of |n_i cos| + |n_j sin|.  The bound used is (d + 16) u of that sum.
In the backward pass dn has the same bound without r, the mean of g x another
(d + 8) u of mean |g x|, and dx is off by at most (3 d + 64) u of
r (|g| + |xh| mean |g xh|), every term with its absolute values.  dw is a sum
over n rows of terms off by (d + 16) u: (n + d + 32) u of the sum of |dn xh|.
"""

import numpy as np
import pytest
import torch

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


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _within(got, ref, bound, what=""):
    got = to_f64(got)
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), f"{what}: {over.max():.3e} over at {np.unravel_index(over.argmax(), over.shape)}"


# ------------------------------------------------------------------ page plan
def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _plan_inputs(cached, width, seed=0, extra=5):
    """A table with each request's own pages and the free list, from one permutation."""
    rng = np.random.default_rng(seed)
    need = [max(0, -(-c // 64)) for c in cached]
    ids = rng.permutation(sum(need) + 4000)
    table, at = np.full((len(cached), width), -1), 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, ids[at:], len(ids)


def _check_plan(px, cached, new, width, rows, free=None, head=0, table=None, pool=None, seed=0):
    t0, f0, p0 = _plan_inputs(cached, width, seed) if table is None else (table, free, pool)
    table, free, pool = t0, f0 if free is None else free, pool or p0
    want = S.page_plan(cached, new, table, free, rows, pool, head)
    t, f = _i32(table), _i32(free)
    h = _i32([head]) if head else None
    px.last_device_error()
    got = px.page_plan(_i32(cached), _i32(new), t, f, num_rows=rows, num_pages=pool, free_head=h)
    assert np.array_equal(t.cpu(), want["table"])
    assert np.array_equal(got.seq_lens.cpu(), want["seq_lens"])
    assert np.array_equal(got.cu_seqlens.cpu(), want["cu_seqlens"])
    assert np.array_equal(got.slot_map.cpu(), want["slots"])
    assert np.array_equal(got.positions.cpu(), want["positions"])
    assert got.pages_used.item() == want["used"]
    assert px.last_device_error() == want["error"]
    return want


@pytest.mark.parametrize("cached,new,rows", [
    ([0], [1], 1), ([0], [0], 0), ([64], [1], 3), ([63], [1], 1), ([63], [2], 2), ([0, 0, 0], [0, 0, 0], 4),
    ([10, 64, 127, 128, 0], [1, 1, 1, 1, 64], 68), ([5, 0, 300], [0, 700, 1], 701)])
def test_page_plan_small(px, cached, new, rows):
    assert _check_plan(px, cached, new, 16, rows)["error"] == 0


@pytest.mark.parametrize("B,hi,seed", [(1, 5000, 0), (33, 200, 1), (512, 3, 2), (513, 90, 3), (8192, 2, 4)])
def test_page_plan_random(px, B, hi, seed):
    rng = np.random.default_rng(seed)
    cached, new = rng.integers(0, 500, B).tolist(), rng.integers(0, hi + 1, B).tolist()
    width = (500 + hi) // 64 + 2
    free = np.random.default_rng(seed + 9).permutation(60000)
    _check_plan(px, cached, new, width, sum(new) + 7, free=free, head=seed, pool=80000, seed=seed)


def test_page_plan_runs_out_of_pages(px):
    # 3 free pages: the second request does not fit, the third needs none, the fourth would fit alone
    want = _check_plan(px, [0, 0, 5, 0], [128, 100, 3, 10], 8, 260, free=[7, 8, 9], pool=60)
    # (the third one's own page is a number past this small pool)
    assert want["error"] == px.DEVERR_NO_PAGES | px.DEVERR_BAD_PAGE
    assert want["seq_lens"].tolist() == [128, 0, 8, 0] and want["used"] == 2
    assert _check_plan(px, [0], [64], 8, 64, free=[], pool=60)["error"] == px.DEVERR_NO_PAGES
    assert _check_plan(px, [3], [4], 8, 4, free=[5, 6], head=2, pool=9000)["error"] == 0
    assert _check_plan(px, [3], [90], 8, 93, free=[5, 6], head=3, pool=9000)["error"] == px.DEVERR_NO_PAGES


def test_page_plan_bad_lengths_and_pages(px):
    # negative lengths, more than the table holds, more rows than there are
    want = _check_plan(px, [-1, 5, 0, 7], [3, -2, 600, 1], 8, 604, pool=60)
    assert want["error"] & px.DEVERR_BAD_LENGTH and want["seq_lens"].tolist() == [0, 0, 0, 8]
    assert _check_plan(px, [0, 9, 4], [10, 20, 0], 8, 25)["seq_lens"].tolist() == [10, 0, 4]
    big = 2 ** 31 - 1
    assert _check_plan(px, [big, big, 0], [big, big, 1], 8, 4, table=np.full((3, 8), -1), free=[1],
                       pool=60)["error"] == px.DEVERR_BAD_LENGTH
    table = np.full((2, 4), -1)
    table[0, 0], table[1, 0] = 60, 2        # the first request's last page is outside the pool
    want = _check_plan(px, [10, 10], [100, 60], 4, 160, table=table, free=[3, -5, 9], pool=60)
    assert want["error"] == px.DEVERR_BAD_PAGE and want["table"].tolist() == [[60, 3, -1, -1], [2, -1, -1, -1]]


def test_page_plan_again_and_replayed(px):
    cached, new = [63, 200, 0], [2, 1, 130]
    table, free, pool = _plan_inputs(cached, 8)
    want = S.page_plan(cached, new, table, free, 140, pool)
    c, n, t, f = _i32(cached), _i32(new), _i32(table), _i32(free)
    call = lambda: px.page_plan(c, n, t, f, num_rows=140, num_pages=pool)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p = call()
    g.replay()
    assert np.array_equal(t.cpu(), want["table"]) and np.array_equal(p.slot_map.cpu(), want["slots"])
    # the next step's lengths in the same buffers
    cached2, new2 = [65, 201, 130], [1, 60, 0]
    want2 = S.page_plan(cached2, new2, want["table"], free[want["used"]:], 140, pool)
    c.copy_(_i32(cached2))
    n.copy_(_i32(new2))
    f.copy_(_i32(np.concatenate([free[want["used"]:], free[:want["used"]]])))
    g.replay()
    assert np.array_equal(t.cpu(), want2["table"]) and np.array_equal(p.slot_map.cpu(), want2["slots"])
    assert np.array_equal(p.positions.cpu(), want2["positions"]) and p.pages_used.item() == want2["used"]
    assert px.last_device_error() == 0


# ---------------------------------------------------------- norm and rotation
def _tables(n, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return a.cos().float().cuda(), a.sin().float().cuda()


def _as_rows(x, batched):
    """[rows, H, d] float64 of [B, H, T, d] or [N, H, d]."""
    x = to_f64(x)
    return x.transpose(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3]) if batched else x


def _row_positions(x, positions, batched):
    if not batched:
        return np.arange(x.shape[0]) if positions is None else positions.cpu().numpy()
    B, T = x.shape[0], x.shape[2]
    p = np.arange(T) if positions is None else positions.cpu().numpy()
    return np.broadcast_to(p, (B, T)).reshape(-1)


def _rope_ref(x, w, pos, cos, sin, eps, norm, interleaved, dtype):
    """Reference rows, and their bound, for rows whose position is not -1."""
    d = x.shape[-1]
    pos = np.maximum(pos, 0)
    R = None if cos is None else S.rotation(cos.cpu().numpy(), sin.cpu().numpy(), pos, d, interleaved)
    w = None if w is None else to_f64(w)
    ref = S.norm_rope(x, w, R, eps, norm)
    size = S.norm_rope(np.abs(x), None if w is None else np.abs(w), None if R is None else np.abs(R), eps, norm)
    h = _half_step(dtype)
    return ref, (d + 16) * U * size * (1 + h) + h * np.abs(ref)


ROPE = [
    # batched, B, H, Hkv, T, d, rot, interleaved, norm, dtype
    (False, 1, 1, 1, 1, 128, 128, False, True, torch.bfloat16),
    (False, 1, 16, 8, 8, 128, 128, False, True, torch.bfloat16),
    (False, 1, 6, 2, 131, 64, 64, True, True, torch.bfloat16),
    (False, 1, 5, 1, 77, 64, 32, False, True, torch.float32),
    (False, 1, 3, 3, 1001, 128, 16, True, True, torch.float32),
    (True, 2, 4, 2, 67, 128, 128, False, True, torch.bfloat16),
    (True, 1, 9, 3, 129, 128, 64, True, True, torch.bfloat16),
    (True, 3, 2, 1, 1, 64, 64, False, True, torch.float32),
    (True, 2, 16, 4, 700, 64, 16, False, True, torch.bfloat16),
    (True, 2, 2, 2, 33, 128, 128, False, False, torch.bfloat16),
    (False, 1, 4, 2, 65, 128, 0, False, True, torch.bfloat16),
]


def _rope_inputs(case, seed=0, weights=True):
    batched, B, H, Hkv, T, d, rot, inter, norm, dtype = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    shape = lambda h: (B, h, T, d) if batched else (T, h, d)
    rows = lambda h: (2 * torch.randn(shape(h), device="cuda", generator=g)).to(dtype)
    x = dict(q=rows(H), rho=rows(H), k=rows(Hkv))
    w = {n: (1 + 0.3 * torch.randn(d, device="cuda", generator=g)).to(dtype) if norm and weights else None for n in x}
    cos, sin = _tables(T + 50, rot) if rot else (None, None)
    return x, w, cos, sin


@pytest.mark.parametrize("case", ROPE, ids=str)
@pytest.mark.parametrize("own_positions", [False, True])
def test_norm_rope(px, case, own_positions):
    batched, B, H, Hkv, T, d, rot, inter, norm, dtype = case
    x, w, cos, sin = _rope_inputs(case)
    pos = None
    if own_positions:
        shape = (B, T) if batched else (T,)
        pos = torch.randint(0, T + 50, shape, device="cuda", dtype=torch.int32)
        pos.view(-1)[-1] = -1       # padding
    before = {n: torch.full_like(t, 7.0) for n, t in x.items()}
    got = px.norm_rope(x["q"], x["rho"], x["k"], cos, sin, pos, q_weight=w["q"], rho_weight=w["rho"], k_weight=w["k"],
                       eps=1e-5, norm=norm, interleaved=inter, out=tuple(before.values()))
    for name, y in zip(x, got):
        p = _row_positions(x[name], pos, batched)
        ref, bound = _rope_ref(_as_rows(x[name], batched), w[name], p, cos, sin, 1e-5, norm, inter, dtype)
        y = _as_rows(y, batched)
        live = p >= 0
        _within(torch.from_numpy(y[live]), ref[live], bound[live], name)
        assert (y[~live] == 7).all()
    assert px.last_device_error() == 0


def test_norm_rope_reads_slices_and_writes_in_place(px):
    # q, rho, k and v as one fused projection leaves them
    N, H, Hkv, d = 37, 4, 2, 128
    x = torch.randn(N, (2 * H + 2 * Hkv) * d, device="cuda").bfloat16()
    v0 = x[:, (2 * H + Hkv) * d:].clone()
    part = lambda a, n: x[:, a * d:(a + n) * d].view(N, n, d)
    q, rho, k = part(0, H), part(H, H), part(2 * H, Hkv)
    cos, sin = _tables(N, d)
    want = px.norm_rope(q.contiguous(), rho.contiguous(), k.contiguous(), cos, sin)
    got = px.norm_rope(q, rho, k, cos, sin)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    px.norm_rope(q, rho, k, cos, sin, out=(q, rho, k))
    for a, b in zip(want, (q, rho, k)):
        assert torch.equal(a, b)
    assert torch.equal(x[:, (2 * H + Hkv) * d:], v0)
    # heads of a [B, T, H, d] tensor seen as [B, H, T, d]
    y = torch.randn(2, 19, 4, 64, device="cuda").bfloat16()
    c, s = _tables(19, 64)
    assert torch.equal(px.norm_rope(y.transpose(1, 2), None, None, c, s)[0],
                       px.norm_rope(y.transpose(1, 2).contiguous(), None, None, c, s)[0])


def test_norm_rope_zero_and_huge_rows(px):
    x = torch.zeros(3, 1, 64, device="cuda")
    x[1] = 3e18
    x[2, 0, 5] = float("inf")
    y = px.norm_rope(x, None, None, None, None, eps=1e-6)[0]
    assert (y[0] == 0).all() and torch.allclose(y[1], torch.ones_like(y[1])) and not torch.isfinite(y[2]).all()


def test_norm_rope_bad_positions(px):
    x = torch.randn(4, 2, 64, device="cuda").bfloat16()
    cos, sin = _tables(10, 64)
    pos = torch.tensor([3, 10, -2, 9], dtype=torch.int32, device="cuda")
    y = torch.full_like(x, 5.0)
    px.last_device_error()
    px.norm_rope(x, None, None, cos, sin, pos, out=(y, None, None))
    assert px.last_device_error() == px.DEVERR_BAD_POSITION
    assert (y[1] == 5).all() and (y[2] == 5).all()
    dx = px.norm_rope_backward(x, None, None, x, None, None, cos, sin, pos)[0]
    assert px.last_device_error() == px.DEVERR_BAD_POSITION and (dx[1:3] == 0).all() and (dx[0] != 0).any()


@pytest.mark.parametrize("case", ROPE, ids=str)
@pytest.mark.parametrize("own_positions", [False, True])
def test_norm_rope_backward(px, case, own_positions):
    batched, B, H, Hkv, T, d, rot, inter, norm, dtype = case
    x, w, cos, sin = _rope_inputs(case, seed=3)
    dy = _rope_inputs(case, seed=4)[0]
    pos = None
    if own_positions:
        pos = torch.randint(0, T + 50, (B, T) if batched else (T,), device="cuda", dtype=torch.int32)
        pos.view(-1)[0] = -1
    got = px.norm_rope_backward(dy["q"], dy["rho"], dy["k"], x["q"], x["rho"], x["k"], cos, sin, pos, q_weight=w["q"],
                                rho_weight=w["rho"], k_weight=w["k"], eps=1e-5, norm=norm, interleaved=inter)
    h = _half_step(dtype)
    for i, name in enumerate(x):
        p = _row_positions(x[name], pos, batched)
        live = p >= 0
        X, DY = (_as_rows(t[name], batched)[live] for t in (x, dy))
        W = None if w[name] is None else to_f64(w[name])
        R = None if cos is None else S.rotation(cos.cpu().numpy(), sin.cpu().numpy(), p[live], d, inter)
        dx = _as_rows(got[i], batched)
        assert (dx[~live] == 0).all()
        ref, dw = S.norm_rope_grad(X, DY, W, R, 1e-5, norm)
        A = None if R is None else np.abs(R)
        dn = np.abs(DY) if A is None else np.einsum("nji,nhj->nhi", A, np.abs(DY))
        if norm:
            r = 1 / np.sqrt(np.mean(X * X, -1, keepdims=True) + 1e-5)
            g, unit = dn * (1 if W is None else np.abs(W)), np.abs(X) * r
            size = r * (g + unit * np.mean(g * unit, -1, keepdims=True))
            n = live.sum() * X.shape[1]
            _within(got[3 + i], dw if n else np.zeros(d), (n + d + 32) * U * (dn * unit).sum((0, 1)), "dw " + name)
        else:
            size = dn
            assert got[3 + i] is None
        _within(torch.from_numpy(dx[live]), ref, (3 * d + 64) * U * size * (1 + h) + h * np.abs(ref), "dx " + name)
    assert px.last_device_error() == 0


def test_norm_rope_backward_is_repeatable_and_in_a_graph(px):
    case = (True, 2, 4, 2, 300, 128, 128, False, True, torch.bfloat16)
    x, w, cos, sin = _rope_inputs(case, seed=5)
    dy = _rope_inputs(case, seed=6)[0]
    call = lambda: px.norm_rope_backward(dy["q"], dy["rho"], dy["k"], x["q"], x["rho"], x["k"], cos, sin,
                                         q_weight=w["q"], rho_weight=w["rho"], k_weight=w["k"])
    a, b = call(), call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = call()
    g.replay()
    for u, v, t in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(u, t)


@pytest.mark.parametrize("broadcast", [False, True])
def test_norm_rope_autograd(px, broadcast):
    # the node's gradients are norm_rope_backward's; a broadcast loss gradient (stride 0) is copied, not misread
    case = (False, 1, 4, 2, 70, 64, 64, False, True, torch.float32)
    x, w, cos, sin = _rope_inputs(case, seed=7)
    pos = torch.arange(70, device="cuda", dtype=torch.int32)
    pos[3] = -1
    leaves = [t.clone().requires_grad_() for t in (*x.values(), *w.values())]
    out = px.NormRope.apply(*leaves, cos, sin, pos, 1e-5, True, False)
    assert (out[0][3] == 0).all()
    if broadcast:
        dy = [torch.ones_like(o) for o in out]
        loss = sum(o.sum() for o in out)
    else:
        dy = [torch.randn_like(o) for o in out]
        loss = sum((o * g).sum() for o, g in zip(out, dy))
    got = torch.autograd.grad(loss, leaves)
    want = px.norm_rope_backward(*dy, *x.values(), cos, sin, pos, q_weight=w["q"], rho_weight=w["rho"],
                                 k_weight=w["k"], eps=1e-5)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_norm_rope_autograd_of_single_sets_and_captured(px):
    # probes absent, a rotation alone, and a captured backward pass (torch itself refuses to capture one of leaves
    # whose eager graph is still alive: their gradient nodes belong to the eager stream)
    case = (True, 2, 4, 2, 40, 64, 64, False, True, torch.bfloat16)
    x, w, cos, sin = _rope_inputs(case, seed=8)
    q, k = x["q"].clone().requires_grad_(), x["k"].clone().requires_grad_()
    qw = w["q"].clone().requires_grad_()

    def grads():
        y, none, z = px.NormRope.apply(q, None, k, qw, None, None, cos, sin)
        assert none is None
        return torch.autograd.grad(y.float().sum() + 2 * z.float().sum(), (q, k, qw))

    want = px.norm_rope_backward(torch.ones_like(q), None, torch.full_like(k, 2), q.detach(), None, k.detach(), cos, sin,
                                 q_weight=w["q"])
    got = grads()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        grads()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = grads()
    g.replay()
    for t in (got, cap):
        assert torch.equal(t[0], want[0]) and torch.equal(t[1], want[2]) and torch.equal(t[2], want[3].bfloat16())
    with pytest.raises(RuntimeError):      # no second derivatives, and no silence about it
        y = px.NormRope.apply(q, None, None, None, None, None, cos, sin)[0]
        (d,) = torch.autograd.grad(y.float().square().sum(), q, create_graph=True)
        d.float().sum().backward()
    r = px.NormRope.apply(q, None, None, None, None, None, cos, sin, None, 1e-6, False)[0]
    assert torch.equal(torch.autograd.grad(r, q, torch.ones_like(r))[0],
                       px.norm_rope_backward(torch.ones_like(q), None, None, q.detach(), None, None, cos, sin, norm=False)[0])


def test_norm_rope_without_tokens(px):
    q, w = torch.empty(0, 4, 64, device="cuda").bfloat16(), torch.ones(64, device="cuda").bfloat16()
    cos, sin = _tables(4, 64)
    y, none, z = px.norm_rope(q, None, q, cos, sin, q_weight=w)
    assert y.shape == q.shape and z.shape == q.shape and none is None
    g = px.norm_rope_backward(q, None, q, q, None, q, cos, sin, q_weight=w)
    assert g[0].shape == q.shape and (g[3] == 0).all() and g[4] is None and (g[5] == 0).all()
    b = torch.empty(2, 4, 0, 128, device="cuda")
    assert px.norm_rope(b, None, None, None, None)[0].shape == b.shape
    assert (px.norm_rope_backward(b, None, None, b, None, None, None, None)[3] == 0).all()


@pytest.mark.parametrize("B,T", [(20000, 1), (3001, 3), (1, 9000)])
@pytest.mark.parametrize("H", [1, 4, 9])
def test_norm_rope_backward_of_many_short_rows(px, B, T, H):
    # the batched rows are the packed ones with their positions written out
    x, dy = (torch.randn(B, H, T, 64, device="cuda").bfloat16() for _ in range(2))
    w, (cos, sin) = torch.randn(64, device="cuda").bfloat16(), _tables(T, 64)
    rows = lambda v: v.transpose(1, 2).reshape(B * T, H, 64)
    dx, _, _, dw, _, _ = px.norm_rope_backward(dy, None, None, x, None, None, cos, sin, q_weight=w)
    pos = torch.arange(T, device="cuda").repeat(B).int()
    px_, _, _, pw, _, _ = px.norm_rope_backward(rows(dy), None, None, rows(x), None, None, cos, sin, pos, q_weight=w)
    assert torch.equal(rows(dx), px_)
    # the same addends, which the same groups take in the same order
    assert torch.equal(dw, pw)


def test_norm_rope_past_32_bits(px):
    # more than 2^31 elements: rows on both sides of the border
    N, H, d = 4_300_000, 4, 128
    x = torch.empty(N, H, d, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, N // 2, 2 ** 31 // (H * d) - 1, 2 ** 31 // (H * d), N - 2, N - 1], device="cuda")
    x.zero_()
    x[rows] = torch.randn(len(rows), H, d, device="cuda").bfloat16()
    cos, sin = _tables(64, d)
    pos = (torch.arange(N, device="cuda") % 64).int()
    y = px.norm_rope(x, None, None, cos, sin, pos)[0]
    assert torch.equal(y[rows], px.norm_rope(x[rows], None, None, cos, sin, pos[rows])[0])
    assert not y[2:1000].any() and not y[N - 1000:N - 2].any()
    dx = px.norm_rope_backward(x, None, None, x, None, None, cos, sin, pos)
    want = px.norm_rope_backward(x[rows], None, None, x[rows], None, None, cos, sin, pos[rows])
    assert torch.equal(dx[0][rows], want[0]) and torch.allclose(dx[3], want[3], rtol=1e-5, atol=1e-5)


def test_rows_of_one_entry_have_any_stride(px):
    # torch leaves odd strides on dimensions of one entry; rows still start at 16 bytes
    base = torch.randn(4096, device="cuda").bfloat16()
    x = base.as_strided((1, 3, 64), (3, 64, 1))
    cos, sin = _tables(4, 64)
    assert torch.equal(px.norm_rope(x, None, None, cos, sin)[0], px.norm_rope(x.clone(), None, None, cos, sin)[0])
    one = base.as_strided((2, 1, 64), (128, 5, 1))
    slots = torch.tensor([3, 70], device="cuda")
    a, b = px.q4_cache(2, 1, 64), px.q4_cache(2, 1, 64)
    px.cache_append_q4(one, one, slots, a)
    px.cache_append_q4(one.clone(), one.clone(), slots, b)
    assert torch.equal(a, b)
    # keys broadcast over heads
    k = base[:640].view(5, 1, 128).expand(5, 4, 128)
    c, d = px.q4_cache(1, 4, 128), px.q4_cache(1, 4, 128)
    px.cache_append_q4(k, k, torch.arange(5, device="cuda"), c)
    px.cache_append_q4(k.contiguous(), k.contiguous(), torch.arange(5, device="cuda"), d)
    assert torch.equal(c, d)
    with pytest.raises(px.ParallaxError):     # written rows must not lie on one another
        px.norm_rope(k.contiguous(), None, None, None, None, out=(k, None, None))


# ------------------------------------------------------------------ cache rows
def _slots(N, pages, seed, skip=()):
    rng = np.random.default_rng(seed)
    s = rng.permutation(pages * 64)[:N].astype(np.int64)
    for i in skip:
        s[i] = -1
    return torch.tensor(s, device="cuda")


@pytest.mark.parametrize("N,Hkv,d,dtype", [(1, 1, 64, torch.bfloat16), (130, 3, 128, torch.bfloat16),
                                           (77, 2, 64, torch.float32), (40, 8, 128, torch.float32)])
def test_cache_append(px, N, Hkv, d, dtype):
    k, v = (torch.randn(N, Hkv, d, device="cuda").to(dtype) for _ in range(2))
    kc, vc = (torch.randn(5, Hkv, 64, d, device="cuda").to(dtype) for _ in range(2))
    slots = _slots(N, 5, N, skip=(N // 2,) if N > 1 else ())
    k_want, v_want = kc.clone(), vc.clone()
    live = slots >= 0
    k_want[slots[live] // 64, :, slots[live] % 64] = k[live]
    v_want[slots[live] // 64, :, slots[live] % 64] = v[live]
    px.cache_append(k, v, slots, kc, vc)
    assert torch.equal(kc, k_want) and torch.equal(vc, v_want) and px.last_device_error() == 0


def _q4_case(N, Hkv, d, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    k = scale * torch.randn(N, Hkv, d, device="cuda", generator=g) + torch.randn(Hkv, d, device="cuda", generator=g)
    v = scale * torch.randn(N, Hkv, d, device="cuda", generator=g)
    return k.bfloat16(), v.bfloat16()


def _check_q4(px, k, v, slots, pages):
    N, Hkv, d = k.shape
    cache = torch.randint(0, 256, (pages, Hkv, 72 * d), dtype=torch.uint8, device="cuda")
    rows_k, rows_v = (np.zeros((pages, Hkv, 64, d), np.float32) for _ in range(2))
    live = (slots >= 0).cpu().numpy()
    at = slots.cpu().numpy()[live]
    rows_k[at // 64, :, at % 64] = k.float().cpu().numpy()[live]
    rows_v[at // 64, :, at % 64] = v.float().cpu().numpy()[live]
    before = cache.cpu().numpy()
    px.cache_append_q4(k, v, slots, cache)
    after = cache.cpu().numpy()
    assert px.last_device_error() == 0
    # written codes and parameters are the definition's, everything else is as it was
    want = S.q4_blocks(rows_k, rows_v)
    (kb, ks), (vb, vs) = S._places(d)
    touched = np.zeros((pages, 64), bool)
    touched[at // 64, at % 64] = True
    touched = np.broadcast_to(touched[:, None], (pages, Hkv, 64))
    for byte, shift in ((kb, ks), (vb, vs)):
        nib = lambda x: (x[..., byte] >> shift.astype(np.uint8)) & 15
        assert np.array_equal(nib(after)[touched], nib(want)[touched])
        assert np.array_equal(nib(after)[~touched], nib(before)[~touched])
    par = lambda x: np.ascontiguousarray(x[..., 64 * d:]).view(np.uint32).reshape(pages, Hkv, 2, 64, d // 64)
    for i in (0, 1):
        a, b, w = (par(x)[:, :, i] for x in (after, before, want))
        same = a[touched] == w[touched]
        nan = np.isnan((w[touched] & 0xffff0000).astype(np.uint32).view(np.float32))
        assert (same | nan).all()
        assert np.isnan((a[touched] & 0xffff0000).astype(np.uint32).view(np.float32))[nan].all()
        assert np.array_equal(a[~touched], b[~touched])
    return cache, rows_k, rows_v


@pytest.mark.parametrize("N,Hkv,d", [(1, 1, 64), (1, 8, 128), (3, 3, 128), (130, 2, 64), (200, 5, 128)])
def test_cache_append_q4_and_gather(px, N, Hkv, d):
    k, v = _q4_case(N, Hkv, d, seed=N)
    slots = _slots(N, 4, N, skip=(N // 2,) if N > 1 else ())
    cache, _, _ = _check_q4(px, k, v, slots, 4)
    live = (slots >= 0).cpu().numpy()
    kq, vq = (S.q4_values(*S.q4_quantise(x.float().cpu().numpy())) for x in (k, v))
    for dtype in (torch.float32, torch.bfloat16):
        out = tuple(torch.full((N, Hkv, d), 9.0, dtype=dtype, device="cuda") for _ in range(2))
        px.cache_gather_q4(cache, slots, out=out)
        # fp32: s n is exact and the sum rounds once; bf16 rounds that again
        rel = U + (_half_step(dtype) if dtype == torch.bfloat16 else 0) * (1 + U)
        for got, want in zip(out, (kq, vq)):
            _within(got[slots >= 0], want[live], rel * np.abs(want[live]), "gather")
            assert (got[slots < 0] == 9).all()
    assert px.last_device_error() == 0


def test_cache_append_q4_consecutive_rows(px):
    # a prompt: neighbouring tokens share the words of their pair
    k, v = _q4_case(150, 2, 128, seed=11)
    _check_q4(px, k, v, torch.arange(13, 163, device="cuda"), 3)
    _check_q4(px, k, v, torch.arange(162, 12, -1, device="cuda"), 3)


def test_cache_append_q4_edges(px):
    k, v = _q4_case(8, 2, 128, seed=12)
    k[0] = 0
    k[1] = 2.5
    k[2, 0, 3] = float("inf")
    k[3, 1, 70] = float("nan")
    v[4, 0, 0], v[4, 0, 1] = 3e38, -3e38
    v[5] = 1e-40
    v[6, :, ::2] = 1e-39
    k[7] = torch.arange(128, device="cuda").bfloat16()
    _check_q4(px, k, v, torch.arange(8, device="cuda") * 7, 1)


def test_cache_append_q4_borders(px):
    # values that sit on the borders between codes (s = 1, m = 0): ties go to the even code
    x = torch.zeros(2, 1, 64, device="cuda")
    x[0, 0, :31] = torch.arange(31, device="cuda") / 2
    x[0, 0, 31] = 15
    x[1] = 3 * x[0] - 4
    _check_q4(px, x.bfloat16(), x.bfloat16(), torch.arange(2, device="cuda"), 1)


@pytest.mark.parametrize("seed", range(4))
def test_cache_append_q4_codes_are_the_quotients(px, seed):
    # many groups of every size of value: each code is the fp32 quotient rounded to nearest even
    g = torch.Generator(device="cuda")
    g.manual_seed(100 + seed)
    N, Hkv, d = 640, 4, 128
    size = torch.exp2(torch.randint(-110, 110, (N, Hkv, 1), device="cuda", generator=g).float())
    k = (size * torch.randn(N, Hkv, d, device="cuda", generator=g)).bfloat16()
    # few significant bits: quotients on and next to the borders
    v = (torch.randint(-200, 200, (N, Hkv, d), device="cuda", generator=g) * 2.0 ** (seed - 2)).bfloat16()
    cache, _, _ = _check_q4(px, k, v, torch.arange(N, device="cuda"), 10)
    kq, vq = px.cache_gather_q4(cache, torch.arange(N, device="cuda"), out_dtype=torch.float32)
    for got, x in ((kq, k), (vq, v)):
        want = S.q4_values(*S.q4_quantise(x.float().cpu().numpy()))
        _within(got, want, U * np.abs(want) + 2.0 ** -149, "values")


def test_cache_rows_take_slices_and_report_bad_slots(px):
    N, Hkv, d = 9, 2, 128
    x = torch.randn(N, 6 * Hkv * d, device="cuda").bfloat16()
    k, v = x[:, 2 * Hkv * d:3 * Hkv * d].view(N, Hkv, d), x[:, 5 * Hkv * d:].view(N, Hkv, d)
    slots = torch.arange(N, device="cuda") * 5
    a, b = px.q4_cache(2, Hkv, d), px.q4_cache(2, Hkv, d)
    px.cache_append_q4(k, v, slots, a)
    px.cache_append_q4(k.contiguous(), v.contiguous(), slots, b)
    assert torch.equal(a, b)
    px.last_device_error()
    slots[4] = 128
    slots[5] = 1 << 40
    c = px.q4_cache(2, Hkv, d)
    px.cache_append_q4(k, v, slots, c)
    assert px.last_device_error() == px.DEVERR_BAD_PAGE
    kc = torch.zeros(2, Hkv, 64, d, device="cuda").bfloat16()
    px.cache_append(k, v, slots, kc, kc.clone())
    assert px.last_device_error() == px.DEVERR_BAD_PAGE
    px.cache_gather_q4(c, slots)
    assert px.last_device_error() == px.DEVERR_BAD_PAGE
    empty = torch.zeros(0, Hkv, d, device="cuda").bfloat16()
    px.cache_append_q4(empty, empty, slots[:0], c)
    assert px.cache_gather_q4(c, slots[:0])[0].shape == (0, Hkv, d)
