"""How exact the 4-bit decode is where few keys hold the weight, at every length.

The reference is the oracle's explicit float64 decode on the keys and values
that the cache's blocks stand for.  Rows of three kinds: near-uniform weights,
one key that lies `boost` above the others (an attention sink, a copied
token), and four such keys.

Two tolerances, of fp32 outputs, with u = 2^-24.

Per element, the worst case.  A score is off by at most ds_i = scale (d + 16)
2u sum |q_c| (s n + |m|)_c, a probe value by da_i = (d + 16) 2u sum |rho_c|
(s n + |m|)_c (2u: the tensor cores may truncate).  A weight is off by 2 max ds
of itself, 2^-21 for the exponential and the 22 bits in which e and e a enter
the value product, and (n + 64) 2u for the sums.  The output is formed from
two sums at a common offset a_ref of the probes, |a_ref| <= A = max |a_i|, so
it is off by at most
    sum_i w_i (1 + |abar| + |a_i| + 2 A) |V_i| e  +  sum_i w_i (da_i + sum_j w_j da_j) |V_i|
with e = 4 max ds + 2^-20 + (n + 64) 4u and |V_i| = (s n + |m|) of the value.

Per row, what the roundings come to when they do not conspire.  The output is
the difference of two terms, vbar and Sigma_KV^T rho, and where they nearly
cancel nothing is exact relative to the rest: with b one term's and the
other's root mean square added, an error of r b is r b / |out| of the output,
whatever computes it.  So the root mean square of a row's error is at most
2^-9 of b.  With probes of size 3 and keys of 128 columns |a_i - a_ref| stays
below 2^9 (a has a spread of about 50): weights of 22 bits enter times that,
so at 2^-13 of |v|, and fp32 sums at that offset at about 2^-13 too.  A score
of about 20 is 2^-18 off, which moves a weight w by w (1 - w) 2^-18 and the
output by that times 2^9: 2^-11.  Together they are below 2^-10; weights of 11
bits, at 2^-12 times the same 2^5 to 2^9, are over.
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


def _rows(px, n, H, d, rho, strong, boost, seed, qs=1.0, ks=1.0, vs=1.0):
    """A paged cache of two sequences of n keys of one KV head; every query points at the keys `strong` (places).
    qs, ks, vs: the sizes of queries, keys and values."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, device="cuda", generator=g)
    base = normal(2, 1, d)
    q = (qs * (base + 0.1 * normal(2, H, d))).bfloat16()
    k, v = normal(2, n, d), normal(2, n, d)
    for at in strong:
        k[:, at] += boost * d ** 0.5 / base.square().sum(-1) * base[:, 0]
    k, v = ks * k, vs * v
    pages = -(-n // 64)
    table = torch.tensor(np.random.default_rng(seed).permutation(2 * pages + 3)[:2 * pages].reshape(2, pages),
                         dtype=torch.int32, device="cuda")
    cache = px.q4_cache(2 * pages + 3, 1, d)
    t = torch.arange(n, device="cuda")
    for b in (0, 1):
        slots = table[b, t // 64].long() * 64 + t % 64
        px.cache_append_q4(k[b].bfloat16()[:, None], v[b].bfloat16()[:, None], slots, cache)
    return dict(q=q, rho=(rho * normal(2, H, d)).bfloat16(), cache=cache, table=table, n=n, d=d)


def _reference(x):
    q, rho, d, n = to_f64(x["q"]), to_f64(x["rho"]), x["d"], x["n"]
    cache = x["cache"].cpu().numpy()
    mag = cache.copy()
    par = np.ascontiguousarray(mag[..., 64 * d:]).view(np.uint16)
    par[..., 1::2] &= 0x7fff          # |m|
    mag[..., 64 * d:] = par.view(np.uint8)
    out, bound, size = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:2])
    for b in range(q.shape[0]):
        at = x["table"][b].cpu().numpy()
        (k, v), (ka, va) = (tuple(t.reshape(-1, d)[:n] for t in S.q4_unblock(c[at, 0], d)) for c in (cache, mag))
        for h in range(q.shape[1]):
            out[b, h] = oracle.parallax_query(q[b, h], rho[b, h], k, v, d ** -0.5)
            w = oracle.softmax_weights(d ** -0.5 * (k @ q[b, h]))
            a = k @ rho[b, h]
            ds = d ** -0.5 * (d + 16) * 2 * U * (ka @ np.abs(q[b, h])).max()
            da = (d + 16) * 2 * U * (ka @ np.abs(rho[b, h]))
            e = 4 * ds + 2.0 ** -20 + (n + 64) * 4 * U
            coef = w * (1 + abs(w @ a) + np.abs(a) + 2 * np.abs(a).max()) * e + w * (da + w @ da)
            bound[b, h] = coef @ va
            size[b, h] = _rms(w @ v) + _rms(w @ v - out[b, h])
    return out, bound, size


def _rms(y):
    return np.sqrt(np.mean(y * y, -1))


def _check(px, x, **kw):
    lens = torch.full((2,), x["n"], dtype=torch.int32, device="cuda")
    got = to_f64(px.decode_q4(x["q"], x["rho"], x["cache"], seq_lens=lens, page_table=x["table"], kv_len=x["n"],
                              out_dtype=torch.float32, **kw))
    ref, bound, size = _reference(x)
    over = np.abs(got - ref) - (bound * (1 + U) + U * np.abs(ref))
    assert np.isfinite(got).all()
    assert (over <= 0).all(), f"{over.max():.3e} over the worst case"
    rel = _rms(got - ref) / size
    assert (rel <= 2.0 ** -9).all(), f"a row is {rel.max():.2e} of its terms' size off"
    assert px.last_device_error() == 0


def _places(n):
    return {"first": [0], "last": [n - 1], "middle": [n // 2], "few": [n // 5, n // 3, n // 2, n - 2]}


@pytest.mark.parametrize("n", [127, 128, 200, 1000, 4096, 16384])
@pytest.mark.parametrize("where", ["first", "middle", "last", "few"])
@pytest.mark.parametrize("boost", [3.0, 9.0, 12.0])
def test_a_few_keys_hold_the_weight(px, n, where, boost):
    for rho in (0.3, 1.0, 3.0):
        _check(px, _rows(px, n, 4, 128, rho, _places(n)[where], boost, seed=n))


@pytest.mark.parametrize("n", [127, 128, 1000, 16384])
def test_flat_weights(px, n):
    for rho in (0.3, 1.0, 3.0):
        _check(px, _rows(px, n, 4, 128, rho, [], 0.0, seed=n))


@pytest.mark.parametrize("H,d", [(1, 128), (8, 128), (4, 64), (7, 64)])
def test_a_few_keys_hold_the_weight_in_every_form(px, H, d):
    for n in (128, 3000):
        for where in ("first", "few"):
            _check(px, _rows(px, n, H, d, 1.0, _places(n)[where], 12.0, seed=H + d))


@pytest.mark.parametrize("ctas", [1, 3, 148])
def test_a_long_row_and_other_grids(px, ctas):
    _check(px, _rows(px, 40000, 4, 128, 1.0, [23456], 12.0, seed=1), num_ctas=ctas)


@pytest.mark.parametrize("H,d", [(2, 128), (8, 64)])
def test_long_flat_rows_in_a_few_runs(px, H, d):
    # thousands of pages summed by one warp: what each step loses must not add up beside a row that averages out
    _check(px, _rows(px, 100_000, H, d, 0.1, [], 0.0, seed=2), num_ctas=1)


# sizes of queries, keys, values and probes, at both ends of the stated range: entries of q and rho below 2^114, value
# scales (about a quarter of a value) down to 2^-80, differences of probe values times a value scale up to 2^100
SIZES = [(1e-10, 1e10, 1e10, 1e5), (2.0 ** -30, 2.0 ** 30, 2.0 ** 30, 2.0 ** 30), (1.0, 1.0, 1e-3, 2.0 ** 100),
         (1.0, 1.0, 2.0 ** 60, 2.0 ** 30), (1.0, 1.0, 2.0 ** 97, 0.02), (1.0, 1.0, 2.0 ** -75, 1.0),
         (2.0 ** 75, 2.0 ** -75, 2.0 ** -75, 2.0 ** 70), (2.0 ** 105, 2.0 ** -105, 1.0, 2.0 ** 105),
         (2.0 ** -100, 2.0 ** 100, 1.0, 2.0 ** -100)]


@pytest.mark.parametrize("qs,ks,vs,rho", SIZES)
def test_sizes_at_the_ends_of_the_range(px, qs, ks, vs, rho):
    for n, strong in ((200, []), (100, [50]), (700, [7, 640])):
        _check(px, _rows(px, n, 4, 128, rho, strong, 9.0, seed=n, qs=qs, ks=ks, vs=vs))
