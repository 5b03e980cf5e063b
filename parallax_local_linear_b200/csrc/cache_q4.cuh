// The paged cache's writers and the 4-bit cache's reader: cache append (plain
// pools and 4-bit blocks) and gather.  The block layout is in parallax.h.
//
// All three move rows between [N, Hkv, d] tensors and slots of the cache, one
// 16-byte vector (8 bf16 columns) per lane.  HBM bounds them on long prompts
// and launch latency on single tokens: append_q4 reads 4 d bytes of a token
// and head and writes 72 d / 64.
#pragma once

#include "ptx.cuh"

namespace plx {

constexpr int kAppendThreads = 256;
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
// A vector per thread: N * Hkv rows of VPR 16-byte vectors, K and V together.
template <int VPR>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long i = (long long)blockIdx.x * kAppendThreads + threadIdx.x;
  const long long rh = i / VPR;
  if (rh >= (long long)a.N * a.Hkv) return;
  const int vec = (int)(i % VPR), r = (int)(rh / a.Hkv), h = (int)(rh % a.Hkv);
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
// Codes of the lane's 8 columns (code i in bits 4 i) and the parameter word of
// its group, which 8 neighbouring lanes share.
__device__ __forceinline__ void quantise8(const uint4& vec, uint32_t& codes, uint32_t& param) {
  float x[8];
  const uint32_t w[4] = {vec.x, vec.y, vec.z, vec.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo_f(w[i]);
    x[2 * i + 1] = bf16_hi_f(w[i]);
  }
  float lo = x[0], hi = x[0];
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    finite = finite && fabsf(x[i]) < INFINITY;   // false for NaN too
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const uint32_t group = 0xffu << (threadIdx.x & 24);
  const float range = hi - lo;
  finite = (__ballot_sync(0xffffffffu, finite) & group) == group && range < INFINITY;
  const uint32_t s16 = pack_bf16(__fdiv_rn(range, 15.f), 0.f) & 0xffffu;
  const float s = __uint_as_float(s16 << 16);
  // A group that cannot be held reads back NaN: scale 0, minimum NaN.
  param = finite ? s16 | (__float_as_uint(lo) & 0xffff0000u) : 0x7fc00000u;
  codes = 0;
  if (!finite || !(s > 0.f)) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = rintf(__fdiv_rn(x[i] - lo, s));
    codes |= (uint32_t)fminf(q, 15.f) << (4 * i);
  }
}

// K's word order: column i of 8 at bits 16 (i % 2) + 4 (i / 2).
__device__ __forceinline__ uint32_t k_word(uint32_t c) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= ((c >> (4 * i)) & 15u) << (16 * (i & 1) + 4 * (i >> 1));
  return w;
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) cache_append_q4_kernel(const AppendArgs a) {
  using B = Q4Block<D>;
  constexpr int LPR = D / 8;   // lanes of a row
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long i = (long long)blockIdx.x * kAppendThreads + threadIdx.x;
  const long long rh = i / LPR;
  const int l = (int)(i % LPR);
  const bool in = rh < (long long)a.N * a.Hkv;
  const int r = in ? (int)(rh / a.Hkv) : 0, h = in ? (int)(rh % a.Hkv) : 0;
  int page = -1, row = 0;
  if (in) slot_of_row(a, r, page, row);
  uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
  if (page >= 0) {
    kv = __ldg(static_cast<const uint4*>(a.k) + r * a.ks[0] + h * a.ks[1] + l);
    vv = __ldg(static_cast<const uint4*>(a.v) + r * a.vs[0] + h * a.vs[1] + l);
  }
  uint32_t kc, kp, vc, vp;   // every lane of the warp takes part in the shuffles
  quantise8(kv, kc, kp);
  quantise8(vv, vc, vp);
  if (page < 0) return;
  uint8_t* block = a.cache + ((size_t)page * a.Hkv + h) * B::kBytes;
  // lane l holds columns 8 l ..: word c = l % 4, j = l / 4 of the K row, words
  // r = 2 (l % 4) + {0, 1} of the V row
  uint32_t* krow = reinterpret_cast<uint32_t*>(block + row * (D / 2));
  krow[B::kWords * (l % 4) + l / 4] = k_word(kc);
  uint16_t* vrow = reinterpret_cast<uint16_t*>(block + B::kV + (row / 2) * D) + (row & 1);
  vrow[2 * (B::kWords * (2 * (l % 4)) + l / 4)] = (uint16_t)vc;
  vrow[2 * (B::kWords * (2 * (l % 4) + 1) + l / 4)] = (uint16_t)(vc >> 16);
  if (l % 8 == 0) {
    reinterpret_cast<uint32_t*>(block + B::kKParams)[row * B::kGroups + l / 8] = kp;
    reinterpret_cast<uint32_t*>(block + B::kVParams)[row * B::kGroups + l / 8] = vp;
  }
}

// --------------------------------------------------------------------- gather
template <int D, bool kBf16>
__global__ void __launch_bounds__(kAppendThreads) cache_gather_q4_kernel(const AppendArgs a) {
  using B = Q4Block<D>;
  constexpr int LPR = D / 8;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long i = (long long)blockIdx.x * kAppendThreads + threadIdx.x;
  const long long rh = i / LPR;
  if (rh >= (long long)a.N * a.Hkv) return;
  const int l = (int)(i % LPR), r = (int)(rh / a.Hkv), h = (int)(rh % a.Hkv);
  int page, row;
  slot_of_row(a, r, page, row);
  if (page < 0) return;
  const uint8_t* block = a.cache + ((size_t)page * a.Hkv + h) * B::kBytes;
  const uint32_t kw = reinterpret_cast<const uint32_t*>(block + row * (D / 2))[B::kWords * (l % 4) + l / 4];
  const uint16_t* vrow = reinterpret_cast<const uint16_t*>(block + B::kV + (row / 2) * D) + (row & 1);
  const uint32_t vw = vrow[2 * (B::kWords * (2 * (l % 4)) + l / 4)] |
                      (uint32_t)vrow[2 * (B::kWords * (2 * (l % 4) + 1) + l / 4)] << 16;
  const uint32_t kp = reinterpret_cast<const uint32_t*>(block + B::kKParams)[row * B::kGroups + l / 8];
  const uint32_t vp = reinterpret_cast<const uint32_t*>(block + B::kVParams)[row * B::kGroups + l / 8];
  float kx[8], vx[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    kx[e] = fmaf(bf16_lo_f(kp), (float)((kw >> (16 * (e & 1) + 4 * (e >> 1))) & 15u), bf16_hi_f(kp));
    vx[e] = fmaf(bf16_lo_f(vp), (float)((vw >> (4 * e)) & 15u), bf16_hi_f(vp));
  }
  // strides in 16-byte vectors
  if (kBf16) {
    static_cast<uint4*>(a.k_out)[r * a.ks[0] + h * a.ks[1] + l] =
        make_uint4(pack_bf16(kx[0], kx[1]), pack_bf16(kx[2], kx[3]), pack_bf16(kx[4], kx[5]), pack_bf16(kx[6], kx[7]));
    static_cast<uint4*>(a.v_out)[r * a.vs[0] + h * a.vs[1] + l] =
        make_uint4(pack_bf16(vx[0], vx[1]), pack_bf16(vx[2], vx[3]), pack_bf16(vx[4], vx[5]), pack_bf16(vx[6], vx[7]));
  } else {
    float4* ko = static_cast<float4*>(a.k_out) + r * a.ks[0] + h * a.ks[1] + 2 * l;
    float4* vo = static_cast<float4*>(a.v_out) + r * a.vs[0] + h * a.vs[1] + 2 * l;
    ko[0] = make_float4(kx[0], kx[1], kx[2], kx[3]);
    ko[1] = make_float4(kx[4], kx[5], kx[6], kx[7]);
    vo[0] = make_float4(vx[0], vx[1], vx[2], vx[3]);
    vo[1] = make_float4(vx[4], vx[5], vx[6], vx[7]);
  }
}

}  // namespace plx
