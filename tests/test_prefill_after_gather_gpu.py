"""A chunk of prompt over a prefix that is held in 4 bits.

There is no attention kernel for prompts over the 4-bit cache: the prefix comes
back as bf16 rows (cache_gather_q4), goes into bf16 pools (cache_append), the
chunk's own rows join it there, and prefill_paged reads the pools.  The chunk goes
into the 4-bit cache too, for the decode steps that follow.

What the path brings to prefill_paged has to be what the codes stand for, so its
output is bit by bit that of pools filled with those rows directly.  Against the
definition: prefill_paged rounds the weights e and e a of rows with 128 keys or
more to bf16, 2^-9 of each, and a row's output is
sum w_i (1 + abar - aref) v_i - sum w_i (a_i - aref) v_i over l, so it is off by
at most 2^-9 sum w_i (1 + |abar - aref| + |a_i - aref|) |v_i|, |aref| at most
A = max |a_i|, and as much again for what the fp32 sums, scores and l add (each
well below 2^-9 at these sizes).
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import serving_oracle as S
from tests.helpers import to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def px():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from parallax_local_linear_b200 import binding
    return binding


@pytest.mark.parametrize("prefix,chunk", [([130, 64], [70, 1]), ([0, 65], [20, 130])])
def test_chunk_over_a_gathered_prefix(px, prefix, chunk):
    torch.manual_seed(sum(prefix))
    B, H, Hkv, d, P = 2, 4, 2, 128, 16
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    normal = lambda *s: torch.randn(*s, device="cuda").bfloat16()
    cache = px.q4_cache(P, Hkv, d)
    table, free, head = torch.full((B, 6), -1, dtype=torch.int32, device="cuda"), torch.randperm(P, device="cuda").int(), 0
    # the prefix, quantised in an earlier step
    n0 = sum(prefix)
    plan = px.page_plan(i32([0, 0]), i32(prefix), table, free, num_rows=n0, num_pages=P)
    k0, v0 = normal(n0, Hkv, d), normal(n0, Hkv, d)
    px.cache_append_q4(k0, v0, plan.slot_map, cache)
    held = plan.slot_map
    # the chunk's step: the prefix into pools of the same pages, the chunk's rows into pools and cache
    n1 = sum(chunk)
    plan1 = px.page_plan(i32(prefix), i32(chunk), table, free, num_rows=n1, num_pages=P, free_head=plan.pages_used)
    q, rho, k1, v1 = normal(n1, H, d), normal(n1, H, d), normal(n1, Hkv, d), normal(n1, Hkv, d)
    kc, vc = (torch.full((P, Hkv, 64, d), float("nan"), device="cuda").bfloat16() for _ in range(2))
    kp, vp = px.cache_gather_q4(cache, held)
    px.cache_append(kp, vp, held, kc, vc)
    px.cache_append(k1, v1, plan1.slot_map, kc, vc)
    px.cache_append_q4(k1, v1, plan1.slot_map, cache)
    out = px.prefill_paged(q, rho, kc, vc, table, plan1.cu_seqlens, plan1.seq_lens, max_q_len=max(chunk),
                           out_dtype=torch.float32)
    kd, vd = (torch.full((P, Hkv, 64, d), float("nan"), device="cuda").bfloat16() for _ in range(2))
    for pool, old, new in ((kd, k0, k1), (vd, v0, v1)):
        pool[held // 64, :, held % 64] = torch.from_numpy(S.q4_values(*S.q4_quantise(old.float().cpu().numpy()))).float().bfloat16().cuda()
        pool[plan1.slot_map // 64, :, plan1.slot_map % 64] = new
    assert torch.equal(out, px.prefill_paged(q, rho, kd, vd, table, plan1.cu_seqlens, plan1.seq_lens,
                                             max_q_len=max(chunk), out_dtype=torch.float32))
    # the definition on the prefix as its codes stand for it, rounded to bf16 as the gather rounds
    deq = lambda x: to_f64(torch.from_numpy(S.q4_values(*S.q4_quantise(x.float().cpu().numpy()))).float().bfloat16())
    at0 = at1 = 0
    for b in range(B):
        keys = np.concatenate([deq(k0)[at0:at0 + prefix[b]], to_f64(k1)[at1:at1 + chunk[b]]])
        values = np.concatenate([deq(v0)[at0:at0 + prefix[b]], to_f64(v1)[at1:at1 + chunk[b]]])
        got = to_f64(out[at1:at1 + chunk[b]])
        for t in range(chunk[b]):
            n = prefix[b] + t + 1
            for h in range(H):
                qh, rh, k, v = to_f64(q[at1 + t, h]), to_f64(rho[at1 + t, h]), keys[:n, h // 2], values[:n, h // 2]
                ref = oracle.parallax_query(qh, rh, k, v, d ** -0.5)
                w, a = oracle.softmax_weights(d ** -0.5 * (k @ qh)), k @ rh
                bound = 2.0 ** -8 * (w * (1 + abs(w @ a) + np.abs(a) + 2 * np.abs(a).max())) @ np.abs(v)
                assert (np.abs(got[t, h] - ref) <= bound).all()
        at0, at1 = at0 + prefix[b], at1 + chunk[b]
    assert px.last_device_error() == 0
