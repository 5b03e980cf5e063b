"""Columns that the rotation leaves alone: norm_rope and its backward past rot_dim.

They pass through, so a value there that is not finite stays in its own column,
and without the norm every column there comes out bit by bit as it went in
(negative zeros too).  Rounded columns are compared with
oracle.serving_oracle in float64; the bounds are those derived in
tests/test_serving_gpu.py.
"""

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from tests.helpers import to_f64
from tests.test_serving_gpu import U, _half_step, _rope_ref, _tables, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from parallax_local_linear_b200 import binding
    return binding


FORMS = [(d, rot, inter, dtype) for d, rot in ((64, 0), (64, 16), (64, 48), (128, 16), (128, 64), (128, 112))
         for inter in (False, True) for dtype in (torch.bfloat16, torch.float32)]


def _case(d, rot, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(37, 5, d, device="cuda", generator=g).to(dtype)
    x[3, :, rot:] = -0.0
    cos, sin = _tables(37, rot) if rot else (None, None)
    return x, cos, sin


def _bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("d,rot,inter,dtype", FORMS)
def test_rotation_alone(px, d, rot, inter, dtype):
    x, cos, sin = _case(d, rot, dtype, seed=d + rot)
    y = px.norm_rope(x, None, None, cos, sin, norm=False, interleaved=inter)[0]
    dx = px.norm_rope_backward(x, None, None, x, None, None, cos, sin, norm=False, interleaved=inter)[0]
    ref, bound = _rope_ref(to_f64(x), None, np.arange(37), cos, sin, 1e-6, False, inter, dtype)
    _within(y, ref, bound, "y")
    R = None if cos is None else S.rotation(cos.cpu().numpy(), sin.cpu().numpy(), np.arange(37), d, inter)
    size, h = np.abs(to_f64(x)), _half_step(dtype)
    if R is not None:
        size = np.einsum("nji,nhj->nhi", np.abs(R), size)
    dref, _ = S.norm_rope_grad(to_f64(x), to_f64(x), None, R, 1e-6, False)
    _within(dx, dref, (3 * d + 64) * U * size * (1 + h) + h * np.abs(dref), "dx")
    for out in (y, dx):
        assert torch.equal(_bits(out[..., rot:]), _bits(x[..., rot:]))


@pytest.mark.parametrize("d,rot,inter,dtype", FORMS)
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_not_finite_past_the_rotation_stays_in_its_column(px, d, rot, inter, dtype, value):
    x, cos, sin = _case(d, rot, dtype, seed=d + rot)
    want = px.norm_rope(x, None, None, cos, sin, norm=False, interleaved=inter)[0]
    back = px.norm_rope_backward(x, None, None, x, None, None, cos, sin, norm=False, interleaved=inter)[0]
    bad = x.clone()
    at = torch.randint(rot, d, (37, 5), device="cuda")
    hit = torch.nn.functional.one_hot(at, d).bool()
    hit[10:] = False       # in some of the rows
    bad[hit] = value
    y = px.norm_rope(bad, None, None, cos, sin, norm=False, interleaved=inter)[0]
    dx = px.norm_rope_backward(bad, None, None, bad, None, None, cos, sin, norm=False, interleaved=inter)[0]
    for got, ref in ((y, want), (dx, back)):
        assert torch.equal(_bits(got[~hit]), _bits(ref[~hit]))
        assert torch.equal(torch.nan_to_num(got[hit], 7.0), torch.nan_to_num(bad[hit], 7.0))


@pytest.mark.parametrize("d,rot,inter,dtype", FORMS)
def test_infinite_rows_with_the_norm(px, d, rot, inter, dtype):
    # the mean is infinite: x / inf is 0 in finite columns and NaN where the row is infinite, in no other column
    x, cos, sin = _case(d, rot, dtype, seed=d + rot + 1)
    at = torch.randint(rot, d, (37, 5), device="cuda")
    hit = torch.nn.functional.one_hot(at, d).bool()
    x[hit] = float("inf")
    w = (1 + 0.1 * torch.randn(d, device="cuda")).to(dtype)
    y = px.norm_rope(x, None, None, cos, sin, q_weight=w, interleaved=inter)[0]
    assert torch.isnan(y[hit]).all() and (y[~hit] == 0).all()


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_padding_rows_get_zero_gradients_whatever_the_weights(px, norm, dtype):
    x, cos, sin = _case(128, 64, dtype, seed=5)
    pos = torch.arange(37, device="cuda", dtype=torch.int32)
    pos[::3] = -1
    w = torch.ones(128, device="cuda", dtype=dtype)
    w[7], w[100] = float("inf"), float("nan")
    x[::3, :, 4] = float("nan")       # padding rows are not read
    dx, _, _, dw, _, _ = px.norm_rope_backward(x, None, None, x, None, None, cos, sin, pos,
                                               q_weight=w if norm else None, norm=norm)
    assert (dx[::3] == 0).all() and (not norm or torch.isfinite(dw).all())
