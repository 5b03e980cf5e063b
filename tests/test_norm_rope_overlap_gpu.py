"""Layouts in which norm_rope's outputs lie in the gaps of what it reads: they do not overlap and are accepted."""

import pytest
import torch

from tests.test_serving_gpu import _tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from parallax_local_linear_b200 import binding
    return binding


def _views(kind, N, H, d):
    """q, rho, k and a place for each result, all in one storage."""
    if kind == "slices":            # [N, q rho k | results]
        s = torch.randn(N, 6 * H * d, device="cuda").bfloat16()
        part = [s[:, i * H * d:(i + 1) * H * d].view(N, H, d) for i in range(6)]
    elif kind == "heads":           # heads of the six taken in turn
        s = torch.randn(N, H, 6, d, device="cuda").bfloat16()
        part = [s[:, :, i] for i in range(6)]
    elif kind == "head major":      # results with heads outermost
        s = torch.randn(6 * H * N * d, device="cuda").bfloat16()
        part = [s[i * H * N * d:(i + 1) * H * N * d] for i in range(6)]
        part = [t.view(N, H, d) if i < 3 else t.view(H, N, d).transpose(0, 1) for i, t in enumerate(part)]
    else:                           # halves of wider rows
        s = torch.randn(3, N, H, 2 * d, device="cuda").bfloat16()
        part = [s[i % 3, :, :, (i // 3) * d:(i // 3 + 1) * d] for i in range(6)]
    return part[:3], part[3:]


@pytest.mark.parametrize("kind", ["slices", "heads", "head major", "halves"])
@pytest.mark.parametrize("N,H,d", [(1, 1, 64), (37, 3, 128)])
def test_outputs_between_inputs(px, kind, N, H, d):
    x, out = _views(kind, N, H, d)
    cos, sin = _tables(N, d)
    keep = [t.clone() for t in x]
    want = px.norm_rope(*keep, cos, sin)
    px.norm_rope(*x, cos, sin, out=tuple(out))
    for a, b, c, e in zip(want, out, keep, x):
        assert torch.equal(a, b) and torch.equal(c, e)
    px.norm_rope(*x, cos, sin, out=tuple(x))       # and in place
    for a, b in zip(want, x):
        assert torch.equal(a, b)


def test_batched_views_in_place(px):
    s = torch.randn(2, 19, 12, 64, device="cuda").bfloat16()      # [B, T, heads of q, rho, k, v]
    x = [s[:, :, i:i + n].transpose(1, 2) for i, n in ((0, 4), (4, 4), (8, 2))]
    cos, sin = _tables(19, 64)
    want, v = px.norm_rope(*[t.clone() for t in x], cos, sin), s[:, :, 10:].clone()
    px.norm_rope(*x, cos, sin, out=tuple(x))
    for a, b in zip(want, x):
        assert torch.equal(a, b)
    assert torch.equal(s[:, :, 10:], v)


def test_overlapping_outputs_are_refused(px):
    x = torch.randn(5, 4, 64, device="cuda").bfloat16()
    y = x.clone()
    cos, sin = _tables(5, 64)
    for out in ((y, y, None), (y, x, None)):
        with pytest.raises(px.ParallaxError):
            px.norm_rope(x, y.clone(), None, cos, sin, out=out)


def test_gather_into_gaps(px):
    # keys and values of a token side by side, as a fused [N, 2, Hkv, d] buffer holds them
    k, v = (torch.randn(70, 2, 128, device="cuda").bfloat16() for _ in range(2))
    cache, slots = px.q4_cache(2, 2, 128), torch.arange(70, device="cuda") + 13
    px.cache_append_q4(k, v, slots, cache)
    want = px.cache_gather_q4(cache, slots)
    both = torch.zeros(70, 2, 2, 128, device="cuda").bfloat16()
    px.cache_gather_q4(cache, slots, out=(both[:, 0], both[:, 1]))
    assert torch.equal(both[:, 0], want[0]) and torch.equal(both[:, 1], want[1])
    with pytest.raises(px.ParallaxError):
        px.cache_gather_q4(cache, slots, out=(both[:, 0], both[:, 0]))
