// The paged cache's writers and the 4-bit cache's reader: cache append (plain
// pools and 4-bit blocks) and gather.  The block layout is in parallax.h.
//
// All three move rows between [N, Hkv, d] tensors and slots of the cache.  HBM
// bounds them on long prompts (the 4-bit append issues 69% of the time beside it) and
// launch latency on single tokens: append_q4 reads 4 d bytes of a token and head
// and writes 72 d / 64.  16382 tokens of 8 heads of 128 columns, appended and
// gathered in fp32 (239 MB): 46 us, 5.2 TB/s; 128 tokens of 4 heads: 3.8 us, device
// time.
#pragma once

#include "ptx.cuh"

namespace plx {

constexpr int kAppendThreads = 128;   // (256: 46.9 instead of 46.1 us for the prompts, 4.0 instead of 3.8 for the step)
constexpr int kQ4Page = 64;

// Byte offsets inside a block.
template <int D>
struct Q4Block {
  static constexpr int kGroups = D / 64;
  static constexpr int kWords = D / 32;                        // words of a lane's chunk
  static constexpr int kV = kQ4Page * D / 2;
  static constexpr int kKParams = kQ4Page * D;
  static constexpr int kParamBytes = kQ4Page * kGroups * 4;    // of K or of V
  static constexpr int kVParams = kKParams + kParamBytes;
  static constexpr int kBytes = kVParams + kParamBytes;        // 72 D
};

struct AppendArgs {
  const void* k;          // gather: written through k_out, v_out
  const void* v;
  void* k_out;
  void* v_out;
  const int64_t* slots;
  uint8_t* cache;         // 4-bit blocks
  void* k_pool;           // plain pools
  void* v_pool;
  long long ks[2], vs[2];
  int N, Hkv, num_pages;
};

// The slot of row r as (page, row in page); page -1 skips the row.
__device__ __forceinline__ void slot_of_row(const AppendArgs& a, int r, int& page, int& row) {
  const long long slot = __ldg(reinterpret_cast<const long long*>(a.slots) + r);
  page = -1;
  row = 0;
  if (slot < 0) return;
  if (slot >= (long long)a.num_pages * kQ4Page) {
    report_error(1 /* PLX_DEVERR_BAD_PAGE */);
    return;
  }
  page = (int)(slot / kQ4Page);
  row = (int)(slot % kQ4Page);
}

// ---------------------------------------------------------------- plain pools
// A vector per thread: row blockIdx.x.., head blockIdx.y, VPR 16-byte vectors of K
// and of V.
template <int VPR>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t i = blockIdx.x * kAppendThreads + threadIdx.x;
  const int vec = i % VPR, r = i / VPR, h = blockIdx.y;
  if (r >= a.N) return;
  int page, row;
  slot_of_row(a, r, page, row);
  if (page < 0) return;
  // strides in 16-byte vectors
  const uint4 kv = __ldg(static_cast<const uint4*>(a.k) + r * a.ks[0] + h * a.ks[1] + vec);
  const uint4 vv = __ldg(static_cast<const uint4*>(a.v) + r * a.vs[0] + h * a.vs[1] + vec);
  const size_t dst = (((size_t)page * a.Hkv + h) * kQ4Page + row) * VPR + vec;
  static_cast<uint4*>(a.k_pool)[dst] = kv;
  static_cast<uint4*>(a.v_pool)[dst] = vv;
}

// ------------------------------------------------------------------- quantise
// Minimum and maximum of three, NaN if one is.
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Codes of the lane's 8 columns and the parameter word of its group, which 8
// neighbouring lanes share.  kKeys: code i at bits 16 (i % 2) + 4 (i / 2) (a K
// word), otherwise at bits 4 i (two V half words).
//
// NaN wins the minimum and the maximum, so a group that is not finite ends up
// with a range that is not.  The format's quotients are fp32 quotients rounded
// to nearest; here each is a product with the rounded reciprocal and one
// correction by its exact remainder, which gives the same number (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000", 1990: with
// y = 1/b rounded to nearest, q = a y, r = a - q b, q + r y is a / b rounded to
// nearest; a reciprocal within one ulp is brought there by one Newton step
// unless b's significand is all ones, and a bf16's is not).  So a quotient that
// lies exactly between two codes, which bf16 rows have in one group of eight,
// rounds as it should.  Where the scale is below 2^-100 and the remainders could
// leave fp32's range, the lane divides.  Dividing throughout took 764
// instructions a pair of vectors; deciding the ties by their remainders
// afterwards 359, this takes 253.
template <bool kKeys>
__device__ __forceinline__ void quantise8(const uint4& vec, uint32_t& codes, uint32_t& param) {
  const uint32_t w[4] = {vec.x, vec.y, vec.z, vec.w};
  float2 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(bf16_lo_f(w[i]), bf16_hi_f(w[i]));
  float lo = min3_nan(min3_nan(x[0].x, x[0].y, x[1].x), min3_nan(x[1].y, x[2].x, x[2].y), min3_nan(x[3].x, x[3].y, x[3].y));
  float hi = max3_nan(max3_nan(x[0].x, x[0].y, x[1].x), max3_nan(x[1].y, x[2].x, x[2].y), max3_nan(x[3].x, x[3].y, x[3].y));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = min3_nan(lo, lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max3_nan(hi, hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float range = hi - lo;
  // A group that cannot be held reads back NaN: scale 0, minimum NaN.
  const bool finite = range < INFINITY;
  constexpr float k15th = 1.f / 15.f;
  float ratio = range * k15th;
  ratio = fmaf(fmaf(-ratio, 15.f, range), k15th, ratio);
  if (ratio < 0x1p-100f) ratio = __fdiv_rn(range, 15.f);
  const uint32_t s16 = pack_bf16(ratio, 0.f) & 0xffffu;
  const float s = __uint_as_float(s16 << 16);
  param = finite ? s16 | (__float_as_uint(lo) & 0xffff0000u) : 0x7fc00000u;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  inv = fmaf(fmaf(-s, inv, 1.f), inv, inv);
  // q + 1.5 2^23 holds round(q) in its low bits (ties to even); the constant's own
  // bits, as far as the shifts leave them in a word, are taken out at the end.
  constexpr uint32_t kMagicBits = 0x4b400000u;
  constexpr uint32_t kMagicSum = kMagicBits + (kMagicBits << 4) + (kMagicBits << 8) + (kMagicBits << 12) +
                                 (kMagicBits << 16) + (kMagicBits << 20) + (kMagicBits << 24) + (kMagicBits << 28);
  const float2 lo2 = make_float2(-lo, -lo), inv2 = make_float2(inv, inv), s2 = make_float2(-s, -s);
  const float2 magic = make_float2(12582912.f, 12582912.f);
  uint32_t sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = add2(x[i], lo2);
    const float2 q = mul2(x[i], inv2);
    const float2 t = add2(fma2(fma2(q, s2, x[i]), inv2, q), magic);
    const int p0 = kKeys ? 4 * i : 8 * i, p1 = kKeys ? 16 + 4 * i : 8 * i + 4;
    sum += (__float_as_uint(t.x) << p0) + (__float_as_uint(t.y) << p1);
  }
  codes = sum - kMagicSum;
  if (!finite || s < 0x1p-100f) {
    codes = 0;
    if (finite && s > 0.f) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float q = __fdiv_rn(k & 1 ? x[k / 2].y : x[k / 2].x, s);
        codes |= (uint32_t)fminf(rintf(q), 15.f) << (kKeys ? 4 * (k / 2) + 16 * (k & 1) : 4 * k);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) cache_append_q4_kernel(const AppendArgs a) {
  using B = Q4Block<D>;
  constexpr int LPR = D / 8;   // lanes of a row
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t i = blockIdx.x * kAppendThreads + threadIdx.x;
  const int l = i % LPR, r = i / LPR, h = blockIdx.y;
  const bool in = r < a.N;
  uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
  if (in) {   // beside the slot's load
    kv = __ldg(static_cast<const uint4*>(a.k) + r * a.ks[0] + h * a.ks[1] + l);
    vv = __ldg(static_cast<const uint4*>(a.v) + r * a.vs[0] + h * a.vs[1] + l);
  }
  int page = -1, row = 0;
  if (in) slot_of_row(a, r, page, row);
  uint32_t kc, kp, vc, vp;   // every lane of the warp takes part in the shuffles
  quantise8<true>(kv, kc, kp);
  quantise8<false>(vv, vc, vp);
  if (page < 0) return;
  uint8_t* block = a.cache + ((size_t)page * a.Hkv + h) * B::kBytes;
  // lane l holds columns 8 l ..: word c = l % 4, j = l / 4 of the K row, words
  // r = 2 (l % 4) + {0, 1} of the V row
  uint32_t* krow = reinterpret_cast<uint32_t*>(block + row * (D / 2));
  krow[B::kWords * (l % 4) + l / 4] = kc;
  uint16_t* vrow = reinterpret_cast<uint16_t*>(block + B::kV + (row / 2) * D) + (row & 1);
  vrow[2 * (B::kWords * (2 * (l % 4)) + l / 4)] = (uint16_t)vc;
  vrow[2 * (B::kWords * (2 * (l % 4) + 1) + l / 4)] = (uint16_t)(vc >> 16);
  if (l % 8 == 0) {
    reinterpret_cast<uint32_t*>(block + B::kKParams)[row * B::kGroups + l / 8] = kp;
    reinterpret_cast<uint32_t*>(block + B::kVParams)[row * B::kGroups + l / 8] = vp;
  }
}

// --------------------------------------------------------------------- gather
// A lane takes four neighbouring columns of a key and a value row, so that a
// row of results is written without gaps (with eight, an fp32 row is written
// 16 bytes of every 32 at a time: 38 against 24 us for 134 MB), and kGatherRows
// rows, so that their loads overlap.
constexpr int kGatherRows = 2;

// The low 4 bits as a number, without a conversion (a quarter-rate instruction).
__device__ __forceinline__ float code_value(uint32_t bits) {
  return __uint_as_float((bits & 15u) | 0x4b000000u) - 8388608.f;
}

template <int D, bool kBf16>
__global__ void __launch_bounds__(kAppendThreads) cache_gather_q4_kernel(const AppendArgs a) {
  using B = Q4Block<D>;
  constexpr int LPR = D / 4, RPC = kAppendThreads / LPR;   // lanes of a row, rows a CTA takes at once
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int l = threadIdx.x % LPR;
  const int first = blockIdx.x * (RPC * kGatherRows) + threadIdx.x / LPR, h = blockIdx.y;
  const uint8_t* block[kGatherRows];
  int row[kGatherRows];
#pragma unroll
  for (int u = 0; u < kGatherRows; ++u) {
    const int r = first + u * RPC;
    int page = -1;
    if (r < a.N) slot_of_row(a, r, page, row[u]);
    block[u] = page < 0 ? nullptr : a.cache + ((size_t)page * a.Hkv + h) * B::kBytes;
  }
  // columns 4 l .. 4 l + 3: a half of K's word l / 2 (columns 8 (l / 2) ..), and
  // a half word of V's
  const int kw = B::kWords * ((l / 2) % 4) + l / 8, kshift = 8 * (l % 2);
  const int vw = B::kWords * (l % 8) + l / 8;
  uint32_t kc[kGatherRows], vc[kGatherRows], kp[kGatherRows], vp[kGatherRows];
#pragma unroll
  for (int u = 0; u < kGatherRows; ++u) {
    if (block[u] == nullptr) continue;
    kc[u] = reinterpret_cast<const uint32_t*>(block[u] + row[u] * (D / 2))[kw] >> kshift;
    vc[u] = reinterpret_cast<const uint16_t*>(block[u] + B::kV + (row[u] / 2) * D)[2 * vw + (row[u] & 1)];
    kp[u] = reinterpret_cast<const uint32_t*>(block[u] + B::kKParams)[row[u] * B::kGroups + l / 16];
    vp[u] = reinterpret_cast<const uint32_t*>(block[u] + B::kVParams)[row[u] * B::kGroups + l / 16];
  }
#pragma unroll
  for (int u = 0; u < kGatherRows; ++u) {
    if (block[u] == nullptr) continue;
    float kx[4], vx[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      kx[e] = fmaf(bf16_lo_f(kp[u]), code_value(kc[u] >> (16 * (e & 1) + 4 * (e >> 1))), bf16_hi_f(kp[u]));
      vx[e] = fmaf(bf16_lo_f(vp[u]), code_value(vc[u] >> (4 * e)), bf16_hi_f(vp[u]));
    }
    // strides in 16-byte vectors
    uint4* ko = static_cast<uint4*>(a.k_out) + (first + u * RPC) * a.ks[0] + h * a.ks[1];
    uint4* vo = static_cast<uint4*>(a.v_out) + (first + u * RPC) * a.vs[0] + h * a.vs[1];
    if (kBf16) {
      __stcs(reinterpret_cast<uint2*>(ko) + l, make_uint2(pack_bf16(kx[0], kx[1]), pack_bf16(kx[2], kx[3])));
      __stcs(reinterpret_cast<uint2*>(vo) + l, make_uint2(pack_bf16(vx[0], vx[1]), pack_bf16(vx[2], vx[3])));
    } else {
      __stcs(reinterpret_cast<float4*>(ko) + l, make_float4(kx[0], kx[1], kx[2], kx[3]));
      __stcs(reinterpret_cast<float4*>(vo) + l, make_float4(vx[0], vx[1], vx[2], vx[3]));
    }
  }
}

}  // namespace plx
