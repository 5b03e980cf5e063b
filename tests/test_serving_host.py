"""Host-side refusals of the operators around attention: no GPU needed.

Every call below fails a check that runs before anything touches a device, so
made-up device addresses are never read.
"""

import ctypes

import pytest
import torch

V = ctypes.c_void_p


@pytest.fixture(scope="module")
def px():
    from parallax_local_linear_b200 import binding
    return binding


def _addr(i, off=0):
    return V((i << 32) + off)


# ------------------------------------------------------------------ page plan
def _plan(px, ptrs=None, **kw):
    base = dict(batch=4, num_rows=100, page_size=64, num_pages=50, max_pages_per_seq=8, num_free=10)
    base.update(kw)
    a = dict(cached=_addr(1), new=_addr(2), table=_addr(3), free=_addr(4), head=None, seq=_addr(5), cu=_addr(6),
             slots=_addr(7), pos=_addr(8), used=_addr(9))
    a.update(ptrs or {})
    p = px.PagePlanParams(**base)
    return px.lib.parallax_page_plan(*a.values(), ctypes.byref(p), None)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=0), 1), (dict(num_rows=-1), 1), (dict(num_pages=0), 1), (dict(max_pages_per_seq=0), 1),
    (dict(num_free=-1), 1), (dict(page_size=32), 2), (dict(batch=8193), 2), (dict(max_pages_per_seq=1 << 25), 2)])
def test_page_plan_parameters(px, kw, want):
    assert _plan(px, **kw) == want


@pytest.mark.parametrize("ptrs", [
    dict(cached=None), dict(new=None), dict(table=None), dict(free=None), dict(seq=None), dict(cu=None),
    dict(slots=None), dict(pos=None), dict(used=None), dict(slots=_addr(7, 4)), dict(cached=_addr(1, 2)),
    dict(seq=_addr(1)), dict(seq=_addr(2, 12)), dict(cu=_addr(5, 8)), dict(used=_addr(6, 16)), dict(pos=_addr(7, 796)),
    dict(table=_addr(4, 36)), dict(head=_addr(9))])
def test_page_plan_pointers(px, ptrs):
    assert _plan(px, ptrs) == 1


# ---------------------------------------------------------- norm and rotation
def _rope(px, ptrs=None, sets=1, heads=4, xs=(0, 512, 128), ys=(0, 512, 128), backward=False, g=None, **kw):
    base = dict(batch=1, tokens=8, head_dim=128, rot_dim=128, max_pos=100, interleaved=0, norm=1, dtype=1, eps=1e-6,
                pos_batch_stride=0)
    base.update(kw)
    a = dict(x=_addr(1), y=_addr(2), w=_addr(3), pos=_addr(4), cos=_addr(5), sin=_addr(6))
    a.update(ptrs or {})
    rows = (px.HeadRows * 4)()
    grads = (px.HeadGrads * 4)()
    for r, gr in zip(rows, grads):
        r.x, r.y, r.w = (a[n].value if a[n] else None for n in ("x", "y", "w"))
        r.heads = heads
        r.x_stride[:], r.y_stride[:] = xs, ys
        gr.dy, gr.dx, gr.dw = 7 << 32, 8 << 32, 9 << 32
        for name, value in (g or {}).items():
            setattr(gr, name, value)
        gr.dy_stride[:], gr.dx_stride[:] = xs, ys
    p = px.NormRopeParams(**base)
    if backward:
        return px.lib.parallax_norm_rope_backward(rows, grads, sets, a["pos"], a["cos"], a["sin"], None, 0,
                                                  ctypes.byref(p), None)
    return px.lib.parallax_norm_rope(rows, sets, a["pos"], a["cos"], a["sin"], ctypes.byref(p), None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(sets=0), 1), (dict(sets=4), 1), (dict(batch=0), 1), (dict(tokens=-1), 1), (dict(rot_dim=24), 1),
    (dict(rot_dim=144), 1), (dict(rot_dim=-16), 1), (dict(max_pos=0), 1), (dict(interleaved=2), 1), (dict(norm=2), 1),
    (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(dtype=5), 1), (dict(head_dim=96), 2), (dict(heads=0), 1),
    (dict(heads=1 << 20, tokens=1 << 12), 2), (dict(xs=(0, 512, 100)), 1), (dict(ys=(4, 512, 128)), 1),
    (dict(pos_batch_stride=-1), 1)])
def test_norm_rope_parameters(px, backward, kw, want):
    assert _rope(px, backward=backward, **kw) == want


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("ptrs,kw", [
    (dict(x=None), {}), (dict(x=_addr(1, 8)), {}), (dict(w=_addr(3, 2)), {}), (dict(cos=None), {}),
    (dict(sin=_addr(6, 4)), {}), (dict(pos=_addr(4, 1)), {}), (dict(pos=None), dict(tokens=101)), ({}, dict(norm=0))])
def test_norm_rope_pointers(px, backward, ptrs, kw):
    assert _rope(px, ptrs, backward=backward, **kw) == 1


def test_norm_rope_forward_and_backward_only(px):
    assert _rope(px, ys=(0, 512, 0)) == 1 and _rope(px, ys=(0, 0, 128)) == 1    # rows on top of each other
    assert _rope(px, backward=True, ys=(0, 0, 128)) == 1
    assert _append(px, "gather", ks=(0, 128)) == 1 and _append(px, "gather", vs=(512, 0)) == 1
    assert _rope(px, dict(y=None)) == 1 and _rope(px, dict(y=_addr(2, 2))) == 1
    assert _rope(px, dict(), tokens=0) == 0
    assert _rope(px, backward=True, g=dict(dy=None)) == 1
    assert _rope(px, backward=True, g=dict(dx=(8 << 32) + 8)) == 1
    assert _rope(px, dict(w=None), backward=True, norm=0) == 1    # dw without a norm
    p = px.NormRopeParams(1, 8, 128, 128, 100, 0, 1, 1, 1e-6, 0)
    assert px.lib.parallax_norm_rope_backward_workspace_size(ctypes.byref(p), 0) == px.SIZE_MAX
    assert px.lib.parallax_norm_rope_backward_workspace_size(None, 1) == px.SIZE_MAX


# ------------------------------------------------------------------ cache rows
def _append(px, which, ptrs=None, ks=(512, 128), vs=(512, 128), **kw):
    base = dict(num_rows=10, num_kv_heads=4, head_dim=128, page_size=64, num_pages=20, dtype=1)
    base.update(kw)
    a = dict(k=_addr(1), v=_addr(2), slots=_addr(3), cache=_addr(4), cache2=_addr(5))
    a.update(ptrs or {})
    p = px.AppendParams(**base)
    p.k_stride[:], p.v_stride[:] = ks, vs
    if which == "plain":
        return px.lib.parallax_cache_append(a["k"], a["v"], a["slots"], a["cache"], a["cache2"], ctypes.byref(p), None)
    if which == "q4":
        return px.lib.parallax_cache_append_q4(a["k"], a["v"], a["slots"], a["cache"], ctypes.byref(p), None)
    return px.lib.parallax_cache_gather_q4(a["cache"], a["slots"], a["k"], a["v"], ctypes.byref(p), None)


@pytest.mark.parametrize("which", ["plain", "q4", "gather"])
@pytest.mark.parametrize("kw,want", [
    (dict(num_rows=-1), 1), (dict(num_kv_heads=0), 1), (dict(num_pages=0), 1), (dict(dtype=3), 1),
    (dict(head_dim=80), 2), (dict(page_size=128), 2), (dict(ks=(512, 4)), 1), (dict(vs=(511, 128)), 1),
    (dict(num_rows=0), 0)])
def test_append_parameters(px, which, kw, want):
    assert _append(px, which, **kw) == want


@pytest.mark.parametrize("which", ["plain", "q4", "gather"])
@pytest.mark.parametrize("ptrs", [dict(k=None), dict(v=None), dict(slots=None), dict(cache=None), dict(k=_addr(1, 8)),
                                  dict(v=_addr(2, 2)), dict(slots=_addr(3, 4)), dict(cache=_addr(4, 8))])
def test_append_pointers(px, which, ptrs):
    assert _append(px, which, ptrs) == 1


def test_append_dtypes(px):
    assert _append(px, "q4", dtype=0) == 2     # only bf16 rows are quantised
    assert _append(px, "plain", dict(cache2=None)) == 1
    assert px.q4_block_bytes(64) == 4608 and px.q4_block_bytes(128) == 9216
    with pytest.raises(px.ParallaxError):
        px.q4_block_bytes(96)


# ---------------------------------------------------------------- 4-bit decode
def _decode(px, ptrs=None, **kw):
    base = dict(batch=8, num_q_heads=16, num_kv_heads=8, head_dim=128, kv_len=4096, page_size=64, num_pages=600,
                max_pages_per_seq=64, in_dtype=1, out_dtype=1, scale=0.088, num_ctas=0)
    base.update(kw)
    a = dict(q=_addr(1), rho=_addr(2), cache=_addr(3), table=_addr(4), lens=_addr(5), out=_addr(6))
    a.update(ptrs or {})
    p = px.DecodeParams(**base)
    return px.lib.parallax_decode_q4(*a.values(), None, 0, ctypes.byref(p), None), \
        px.lib.parallax_decode_q4_workspace_size(ctypes.byref(p), 148)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=0), 1), (dict(num_q_heads=12), 1), (dict(kv_len=-1), 1), (dict(in_dtype=7), 1), (dict(in_dtype=0), 2),
    (dict(out_dtype=9), 1), (dict(scale=float("inf")), 1), (dict(head_dim=96), 2), (dict(num_q_heads=72), 2),
    (dict(page_size=32), 2), (dict(batch=9000), 2), (dict(num_pages=0), 1), (dict(max_pages_per_seq=3), 1)])
def test_decode_q4_parameters(px, kw, want):
    assert _decode(px, **kw) == (want, px.SIZE_MAX)


@pytest.mark.parametrize("ptrs", [dict(q=None), dict(rho=None), dict(cache=None), dict(out=None), dict(table=None),
                                  dict(lens=None), dict(q=_addr(1, 2)), dict(cache=_addr(3, 8)), dict(lens=_addr(5, 2))])
def test_decode_q4_pointers(px, ptrs):
    assert _decode(px, ptrs)[0] == 1


def test_decode_q4_contiguous_takes_no_page_table(px):
    assert _decode(px, page_size=0, num_pages=0, max_pages_per_seq=0)[0] == 1


# ----------------------------------------------------------- the torch binding
def test_binding_refuses_shapes(px):
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    i32 = torch.int32
    with pytest.raises(ValueError):
        px.decode_q4(t(2, 4, 128), t(2, 4, 64), t(5, 2, 9216, dt=torch.uint8))
    with pytest.raises(ValueError):     # block bytes of another head_dim
        px.decode_q4(t(2, 4, 128), t(2, 4, 128), t(2, 2, 1, 4608, dt=torch.uint8))
    with pytest.raises(ValueError):     # 3 heads over 2
        px.decode_q4(t(2, 3, 64), t(2, 3, 64), t(2, 2, 1, 4608, dt=torch.uint8))
    with pytest.raises(ValueError):     # paged without seq_lens
        px.decode_q4(t(2, 4, 64), t(2, 4, 64), t(9, 2, 4608, dt=torch.uint8), page_table=t(2, 3, dt=i32))
    with pytest.raises(ValueError):     # kv_len leaves a page over
        px.decode_q4(t(2, 4, 64), t(2, 4, 64), t(2, 2, 3, 4608, dt=torch.uint8), kv_len=128)
    with pytest.raises(TypeError):
        px.cache_append_q4(t(3, 2, 64), t(3, 2, 64), t(3, dt=torch.int64), t(9, 2, 4608))
    with pytest.raises(ValueError):
        px.cache_append_q4(t(3, 2, 128), t(3, 2, 128), t(3, dt=torch.int64), t(9, 2, 4608, dt=torch.uint8))
    with pytest.raises(ValueError):
        px.cache_append(t(3, 2, 64), t(4, 2, 64), t(3, dt=torch.int64), t(9, 2, 64, 64), t(9, 2, 64, 64))
    with pytest.raises(ValueError):     # pages of another size
        px.cache_append(t(3, 2, 64), t(3, 2, 64), t(3, dt=torch.int64), t(9, 2, 32, 64), t(9, 2, 32, 64))
    with pytest.raises(ValueError):
        px.page_plan(t(4, dt=i32), t(5, dt=i32), t(4, 3, dt=i32), t(9, dt=i32), num_rows=5, num_pages=9)
    with pytest.raises(ValueError):
        px.page_plan(t(4, dt=i32), t(4, dt=i32), t(3, 3, dt=i32), t(9, dt=i32), num_rows=5, num_pages=9)
    cos = t(16, 32, dt=torch.float32)
    with pytest.raises(ValueError):
        px.norm_rope(t(5, 4, 64), t(5, 3, 64), None, cos, cos)
    with pytest.raises(ValueError):     # more tokens than angles
        px.norm_rope(t(17, 4, 64), None, None, cos, cos)
    with pytest.raises(ValueError):
        px.norm_rope(t(5, 4, 64), None, None, cos, None)
    with pytest.raises(ValueError):
        px.norm_rope(t(5, 4, 64), None, t(6, 2, 64), cos, cos)
    with pytest.raises(ValueError):
        px.norm_rope(t(2, 4, 5, 64), None, None, cos, cos, t(2, 4, dt=i32))
    with pytest.raises(ValueError):
        px.norm_rope(t(5, 4, 64), None, None, cos, cos, q_weight=t(64), norm=False)
    with pytest.raises(ValueError):     # host tensors
        px.norm_rope(t(5, 4, 64), None, None, cos, cos)
