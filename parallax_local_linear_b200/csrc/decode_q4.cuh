// Parallax decode over the 4-bit cache.
//
// One query head per CTA; each warp takes 32-token chunks, a lane per token
// for the scores and probe values and a lane per D/32 columns for the value
// sums, as the single-pass form of decode.cuh.
#pragma once

#include "cache_q4.cuh"
#include "decode.cuh"

namespace plx {

constexpr int kQ4Warps = 8;

struct DecodeQ4Args {
  const __nv_bfloat16* q;
  const __nv_bfloat16* rho;
  const uint8_t* cache;
  const int32_t* page_table;
  const int32_t* seq_lens;
  void* out;
  int B, Hq, Hkv, group, kv_len, paged, num_pages, max_pages;
  float scale_log2;
  int out_bf16;
};

template <int D>
__global__ void __launch_bounds__(kQ4Warps * 32) decode_q4_kernel(const DecodeQ4Args a) {
  using B = Q4Block<D>;
  constexpr int C = D / 32;
  __shared__ float s_q[2][D];
  __shared__ float s_m[kQ4Warps], s_l[kQ4Warps], s_c[kQ4Warps];
  __shared__ float s_o[kQ4Warps][2][D];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq, kvh = hq / a.group;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int len = a.seq_lens ? __ldg(a.seq_lens + b) : a.kv_len;
  if (len < 0 || len > a.kv_len) {
    if (tid == 0) report_error(4 /* PLX_DEVERR_BAD_LENGTH */);
    len = len < 0 ? 0 : a.kv_len;
  }
  for (int d = tid; d < D; d += kQ4Warps * 32) {
    s_q[0][d] = __bfloat162float(a.q[((size_t)b * a.Hq + hq) * D + d]);
    s_q[1][d] = __bfloat162float(a.rho[((size_t)b * a.Hq + hq) * D + d]);
  }
  __syncthreads();
  const int tiles_max = (a.kv_len + kQ4Page - 1) / kQ4Page;
  auto block_of = [&](int tile) {
    size_t i = ((size_t)b * a.Hkv + kvh) * tiles_max + tile;
    if (a.paged) {
      int p = __ldg(a.page_table + (size_t)b * a.max_pages + tile);
      if (p < 0 || p >= a.num_pages) {
        report_error(1 /* PLX_DEVERR_BAD_PAGE */);
        p = 0;
      }
      i = (size_t)p * a.Hkv + kvh;
    }
    return a.cache + i * B::kBytes;
  };
  float m = -INFINITY, l = 0.f, c = 0.f, o1[C], o2[C];
#pragma unroll
  for (int i = 0; i < C; ++i) o1[i] = o2[i] = 0.f;
  for (int t0 = warp * 32; t0 < len; t0 += kQ4Warps * 32) {
    const uint8_t* blk = block_of(t0 / kQ4Page);
    const int row = t0 % kQ4Page + lane;
    const bool ok = t0 + lane < len;
    float s = -INFINITY, av = 0.f;
    if (ok) {
      s = 0.f;
      const uint32_t* kr = reinterpret_cast<const uint32_t*>(blk + row * (D / 2));
      const uint32_t* kp = reinterpret_cast<const uint32_t*>(blk + B::kKParams) + row * B::kGroups;
      for (int w = 0; w < D / 8; ++w) {
        const int col = 32 * (w % B::kWords) + 8 * (w / B::kWords);
        const uint32_t word = kr[w], par = kp[col / 64];
        for (int i = 0; i < 8; ++i) {
          const float x = fmaf(bf16_lo_f(par), (float)((word >> (16 * (i & 1) + 4 * (i >> 1))) & 15u), bf16_hi_f(par));
          s = fmaf(s_q[0][col + i], x, s);
          av = fmaf(s_q[1][col + i], x, av);
        }
      }
      s *= a.scale_log2;
    }
    const float m_new = fmaxf(m, warp_max(s));
    const float alpha = ex2(m - m_new), p = ex2(s - m_new), pa = p * av;
    m = m_new;
    l = l * alpha + p;
    c = c * alpha + pa;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      o1[i] *= alpha;
      o2[i] *= alpha;
    }
    for (int j = 0; j < min(32, len - t0); ++j) {
      const float pj = __shfl_sync(0xffffffffu, p, j), paj = __shfl_sync(0xffffffffu, pa, j);
      const int r = t0 % kQ4Page + j;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int col = lane + 32 * i;
        const uint32_t word = reinterpret_cast<const uint32_t*>(blk + B::kV + (r / 2) * D)[B::kWords * (lane / 4) + i];
        const uint32_t par = reinterpret_cast<const uint32_t*>(blk + B::kVParams)[r * B::kGroups + col / 64];
        const float x = fmaf(bf16_lo_f(par), (float)((word >> (16 * (r & 1) + 4 * (lane % 4))) & 15u), bf16_hi_f(par));
        o1[i] = fmaf(pj, x, o1[i]);
        o2[i] = fmaf(paj, x, o2[i]);
      }
    }
  }
  l = warp_sum(l);
  c = warp_sum(c);
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
    s_c[warp] = c;
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
    s_o[warp][0][lane + 32 * i] = o1[i];
    s_o[warp][1][lane + 32 * i] = o2[i];
  }
  __syncthreads();
  for (int d = tid; d < D; d += kQ4Warps * 32) {
    float M = -INFINITY, L = 0.f, Cc = 0.f, O1 = 0.f, O2 = 0.f;
    for (int w = 0; w < kQ4Warps; ++w) M = fmaxf(M, s_m[w]);
    for (int w = 0; w < kQ4Warps; ++w) {
      const float al = s_m[w] == -INFINITY ? 0.f : ex2(s_m[w] - M);
      L += al * s_l[w];
      Cc += al * s_c[w];
      O1 += al * s_o[w][0][d];
      O2 += al * s_o[w][1][d];
    }
    const float val = len == 0 ? 0.f : finalize(O1, O2, L, Cc);
    const size_t idx = ((size_t)b * a.Hq + hq) * D + d;
    if (a.out_bf16)
      reinterpret_cast<__nv_bfloat16*>(a.out)[idx] = __float2bfloat16_rn(val);
    else
      reinterpret_cast<float*>(a.out)[idx] = val;
  }
}

}  // namespace plx
