"""The cache's writer and reader refuse outputs that overlap (no GPU needed: made-up addresses, refused before use)."""

import ctypes

import pytest

V = ctypes.c_void_p
A, B, C, E, F = (V(i << 32) for i in range(1, 6))
ROW = 4 * 128 * 2


@pytest.fixture(scope="module")
def px():
    from parallax_local_linear_b200 import binding
    return binding


def _params(px, ks=(512, 128), vs=(512, 128)):
    p = px.AppendParams(10, 4, 128, 64, 20, 1)
    p.k_stride[:], p.v_stride[:] = ks, vs
    return ctypes.byref(p)


@pytest.mark.parametrize("k_cache,v_cache,slots", [
    (E, E, C), (E, V(E.value + 20 * 4 * 64 * 128 * 2 - 16), C), (E, F, E), (E, F, V(F.value + 64))])
def test_append_pools(px, k_cache, v_cache, slots):
    assert px.lib.parallax_cache_append(A, B, slots, k_cache, v_cache, _params(px), None) == 1


@pytest.mark.parametrize("k,v,slots,kw", [
    (A, A, C, {}), (A, V(A.value + 9 * ROW), C, {}), (A, B, A, {}), (A, B, V(B.value + 9 * ROW), {}), (E, B, C, {}),
    (A, V(E.value + 9216), C, {}), (A, V(A.value + 256), C, dict(ks=(1024, 256), vs=(1024, 128)))])
def test_gather_results(px, k, v, slots, kw):
    assert px.lib.parallax_cache_gather_q4(E, slots, k, v, _params(px, **kw), None) == 1


@pytest.mark.parametrize("kw", [
    dict(out=V(A.value + 16)), dict(out=V(A.value - 16)), dict(out=A, out_dtype=0), dict(out=V(B.value + 16)),
    dict(out=V(C.value + 600 * 8 * 9216 - 16)), dict(out=E), dict(out=V(F.value - 16)), dict(out=V((6 << 32) + (1 << 22) - 16))])
def test_decode_q4_output(px, kw):
    kw = dict(out_dtype=1) | kw
    p = px.DecodeParams(8, 16, 8, 128, 4096, 64, 600, 64, 1, kw["out_dtype"], 0.088, 0)
    ws = V(6 << 32)
    st = px.lib.parallax_decode_q4(A, B, C, E, F, kw["out"], ws, 1 << 22, ctypes.byref(p), None)
    assert st == 1
