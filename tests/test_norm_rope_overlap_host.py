"""norm_rope refuses outputs that overlap what it reads or each other (no GPU needed).

Every call here is refused before anything touches a device: the addresses are
made up.  The layouts that are accepted are in test_norm_rope_overlap_gpu.py.
"""

import ctypes

import pytest

V = ctypes.c_void_p
T, D = 8, 128


@pytest.fixture(scope="module")
def px():
    from parallax_local_linear_b200 import binding
    return binding


def _call(px, sets, *, backward=False, dtype=1, pos=V(50 << 32), cos=V(51 << 32), sin=V(52 << 32)):
    """sets: dicts of x, y (or dy, dx, dw), w as addresses and xs, ys (or dys, dxs) strides, heads."""
    rows, grads = (px.HeadRows * 3)(), (px.HeadGrads * 3)()
    for r, g, s in zip(rows, grads, sets):
        h = s.get("heads", 4)
        dense = (0, h * D, D)
        r.x, r.y, r.w, r.heads = s["x"], s.get("y"), s.get("w"), h
        r.x_stride[:], r.y_stride[:] = s.get("xs", dense), s.get("ys", dense)
        g.dy, g.dx, g.dw = s.get("dy"), s.get("dx"), s.get("dw")
        g.dy_stride[:], g.dx_stride[:] = s.get("dys", dense), s.get("dxs", dense)
    p = px.NormRopeParams(1, T, D, D, 100, 0, 1, dtype, 1e-6, 0)
    if backward:
        return px.lib.parallax_norm_rope_backward(rows, grads, len(sets), pos, cos, sin, V(60 << 32), 1 << 20,
                                                  ctypes.byref(p), None)
    return px.lib.parallax_norm_rope(rows, len(sets), pos, cos, sin, ctypes.byref(p), None)


A, B, C, E = 1 << 32, 2 << 32, 3 << 32, 4 << 32
ROW = 4 * D * 2     # bytes of a token's four bf16 heads


@pytest.mark.parametrize("sets", [
    [dict(x=A, y=A + 16)],                                             # shifted by a vector
    [dict(x=A, y=A, ys=(0, 8 * D, D))],                                # in place with other strides
    [dict(x=A, y=B), dict(x=B, y=C)],                                  # the second set's rows
    [dict(x=A, y=C), dict(x=B, y=C)],                                  # both into one
    [dict(x=A, y=C), dict(x=B, y=C + 7 * ROW + 3 * D * 2)],            # their last and first head
    [dict(x=A, y=B, w=B + 7 * ROW)],                                   # the weights
    [dict(x=A, y=51 << 32)], [dict(x=A, y=(52 << 32) + 100 * 256 - 16)],   # cos, sin
    [dict(x=A, y=(50 << 32) - 8 * ROW + 16)],                          # positions
    # interleaved heads of one buffer, one head too far
    [dict(x=A, y=B, xs=(0, 8 * D, D), ys=(0, 8 * D, D)), dict(x=C, y=B + 3 * D * 2, xs=(0, 8 * D, D), ys=(0, 8 * D, D))],
    [dict(x=A, y=B, ys=(0, 8 * D, 2 * D)), dict(x=C, y=B + 2 * D * 2, ys=(0, 8 * D, 2 * D))],
])
def test_forward(px, sets):
    assert _call(px, sets) == 1


@pytest.mark.parametrize("sets", [
    [dict(x=A, dy=B, dx=B + 16)], [dict(x=A, dy=B, dx=A, dxs=(0, 8 * D, D))],
    [dict(x=A, dy=B, dx=C), dict(x=C, dy=E, dx=5 << 32)], [dict(x=A, dy=B, dx=C, dw=C + 64)],
    [dict(x=A, dy=B, dx=C, dw=A + 128)], [dict(x=A, dy=B, dx=C, dw=E), dict(x=5 << 32, dy=6 << 32, dx=7 << 32, dw=E + 256)],
    [dict(x=A, dy=B, dx=C, w=C + 256)], [dict(x=A, dy=B, dx=51 << 32)],
])
def test_backward(px, sets):
    assert _call(px, sets, backward=True) == 1
