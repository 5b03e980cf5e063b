// Parallax decode over the 4-bit cache: 144 bytes a token and KV head at d = 128,
// so the arithmetic per byte is 3.6 times the bf16 decode's.  While the clock is up
// the latencies of three warps a sub-partition bound it (57% of the issue slots, 52% of the
// integer pipe in use at 1.65 GHz), in sustained runs, at 1.3 GHz, the issue slots
// (1080 instructions a page).
//
// The sums are those of the single-pass form in decode.cuh,
//     l = sum e_i,  c = sum e_i a_i,  O1 = sum e_i v_i,  O2 = sum e_i a_i v_i,
// on k = s n + m and v = s n + m (codes n, scales s and minima m, one pair per
// token and group of 64 columns).  Scales and minima stay out of the products:
//     q.k   = sum_g s_g (q_g . n_g) + m_g (sum of q_g)
//     O1_d  = sum_i (e_i s_i) n_id + sum_i e_i m_i        (d in group g of i's row)
// so the tensor cores multiply bare codes.  A code masked out of its word is
// already an fp16 number: bits 0..3 of a half are the subnormal n 2^-24 and bits
// 4..7 are n 2^-20.  One AND makes two operands; the powers of two are taken
// out of the queries on one side and of the results on the other.
//
// Operands (mma.sync m16n8k16, fp16 in, fp32 sums; the contraction has 8 columns
// for 4 heads, far below what a tcgen05 tile needs, and its operands would have
// to be written back to shared memory):
//     [S A] (16 tokens x 8) = K (16 x d) . [q_0 rho_0 q_1 rho_1 ..] (d x 8)
//     [O1 O2] (16 columns x 8) += V^T (16 x 16 tokens) . [p_0 pa_0 p_1 pa_1 ..] (16 x 8)
// Codes are the A operand both times, read from shared memory with one 16-byte
// load per row and lane in the block's own layout.  A lane's accumulators
// belong to one head (lane % 4) throughout: scores and probes of tokens r and
// r + 8, r = lane / 4, then O1 and O2 of d/8 columns.  The weights change
// from accumulator to operand by a transposing move (movmatrix).
//
// Ranges.  q and rho are scaled by a power of two to at most 2^14 per row
// (exact: they are bf16; up to 2^114).  e s and e a s have to fit fp16: the
// running reference is not the largest score alone but
//     M = max_i x_i + log2(max_i,g s_ig max_i(1, |a_i|)),      p_i = 2^(x_i - M + 10)
// with x_i the score in powers of two (maxima of a page).  M stays until a page
// needs it to be more than 5 larger, so every product is at most 2^15, nothing
// above 2^-34 of the largest is lost, and after a unit's first page the
// sums are hardly ever rescaled (1.5% of the time).  Probe values above 2^10 are
// taken in a larger unit.
//
// Exactness.  The output is the difference of two sums whose terms are w_i
// |a_i - aref| |v_i|, so what is rounded in them comes back |a - aref| times.
//   - The weights enter with their low halves in a second product (22 bits
//     together), as in decode.cuh.
//   - aref is the probe value of the key with the largest score so far, or of one
//     within 2^5 of it in weight (any constant leaves the output unchanged):
//     the sums are shifted when a page brings a larger one, and merging
//     shifts c and O2 of the pieces to a common one.  So where one key holds the
//     weight its own term is about zero.  This also keeps the tensor cores' grid
//     harmless: they add the terms of a product in steps set by the largest exponents,
//     where a subnormal code counts as 2^-14, so beside one heavy weight the other
//     15 tokens' terms are cut at 2^-14 of it (measured: 1.1e-4 of the heavy
//     weight, always downwards).
//   - The tensor cores truncate, and sums of codes (0 to 15) grow with every page, so what
//     each step loses would add up: 0.07% of a flat row after 170 pages, percents of it
//     after thousands. As a group's columns share their minima's sums, any
//     constant may go from the former to the latter: every 16 pages one column's sums
//     do, and the rest are differences of columns.
// With 11 bits and the first key's probe value a row with one key 12 above 1000
// others was up to 6% off, with 22 bits alone 0.4%, with both 0.01%.
//
// Work.  The pages of every (sequence, KV head) unit are laid end to end and
// cut into equal runs, one per warp: no warp waits for another until its run
// is done.  A warp keeps its own ring of asynchronous copies (one page and head
// is one contiguous block) and refills a slot as it leaves it; copies by all
// lanes cost it 9 issue slots a slot, where a bulk copy from one lane held it up
// for about 450 cycles.  Units that lie
// inside a run are finished in registers; pieces of cut units are merged in
// the CTA after one barrier, and across CTAs in the workspace, by the last CTA
// that finishes a piece (a counter per unit, which that CTA takes back to zero).
//
// Measured (device time in a graph, full clock): 32 sequences of 32768 keys, 32/8 heads, d =
// 128 (1.21 GB) 222 us, 5.4 TB/s (269 us a call sustained for seconds under the power
// cap); 8 of 4096, 16/8 heads (38 MB) 18.3 us, of which set-up, first pages and
// merge take about 8; 16 of 16384 and 4 KV heads (151 MB) 39 us with 4 query heads
// each and 60 us with 8.
#pragma once

#include <type_traits>

#include <cuda_fp16.h>

#include "cache_q4.cuh"
#include "decode.cuh"

namespace plx {

struct DecodeQ4Args {
  const __nv_bfloat16* q;
  const __nv_bfloat16* rho;
  const uint8_t* cache;
  const int32_t* page_table;       // [B, max_pages] or null: blocks [B, Hkv, pages of kv_len]
  const int32_t* seq_lens;         // [B] or null
  void* out;
  float* slots;                    // [2 * gridDim.x][group][2 D + 4]
  int32_t* counters;               // [B * Hkv]
  int B, Hq, Hkv, group, kv_len, num_pages, max_pages;
  float scale_log2;
  int out_bf16;
  int min_pages;                   // a CTA takes at least this many pages
};

// Weights against a new reference are at most 2^kQ4Top, and 2^kQ4Slack times
// that before it moves: together below fp16's 2^16.  A key 2^kQ4Slack above the
// one that gave aref takes its place.
constexpr float kQ4Top = 10.f, kQ4Slack = 5.f;

// Probe values (from aref, in their unit) are at most this: p s, which is smaller by
// them than p a s, keeps its low half.
constexpr float kQ4MaxProbe = 1024.f;

// Pages after which a unit's sums of codes are taken back to about zero: with 8, 16
// and 32 decode_long's shape takes 223.6, 221.5 and 220.5 us, and rows of 32768 keys in
// runs of 170 pages are 2.5e-5, 3.4e-5 and 6.6e-5 of themselves off (6.7e-4 without).
constexpr int kQ4Settle = 16;

// Warps of a CTA (one CTA per SM) and its shared memory.  A ring slot holds
// one half of a block, K's or V's codes and parameters.
template <int D, int NT>
struct Q4Smem {
  static constexpr int kWarps = NT == 1 ? 12 : 8;                  // 168 and 255 registers a thread (d = 128: 4 and 20 bytes spilled)
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCodes = kQ4Page * D / 2;
  static constexpr int kPart = kCodes + Q4Block<D>::kParamBytes;
  static constexpr int kSlots = 2 * (128 / D);                     // per warp (3 for d = 128 measured 0 to 4% slower)
  static constexpr int kRing = kSlots * kPart;                     // per warp
  static constexpr int kRow = 2 * D + 4;                           // a head's state: m l c aref O1 O2
  static constexpr int kState = 4 * NT * kRow * 4;                 // bytes of a piece
  static constexpr int kStateOff = kWarps * kRing;
  static constexpr int kQRow = 2 * D + 16;                         // a staged q or rho row (16 bytes apart in the banks)
  static constexpr int kQ = 8 * NT * kQRow;                        // per warp
  static constexpr int kQOff = kStateOff + kWarps * kState;
  static constexpr int kMetaOff = kQOff + kWarps * kQ;
  static constexpr int kPreOff = kMetaOff + kWarps * 8 * 4;
  static constexpr int kBytes = kPreOff + (kThreads + 4) * 4;
  static_assert(kState <= kRing, "a warp's last piece fits in its ring");
  static_assert(2 * kWarps <= 32 && kWarps % 4 == 0, "a lane for every piece of a CTA");
  static_assert(kMaxBatch <= 32 * kThreads, "a lane for every sequence of a share");
};

// D += A * B, m16n8k16, fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of the 8 x 8 matrix of halves that the warp holds two to a lane.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// 16 bytes from global to shared memory, not through L1.
__device__ __forceinline__ void q4_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
// Zeros instead where !read.
__device__ __forceinline__ void q4_copy16(uint32_t dst, const void* src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
               "r"(read ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void q4_copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void q4_copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// N consecutive words of shared memory.
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    static_assert(N == 1, "1, 2 or 4 words");
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// ---------------------------------------------------------------- the page space
// pre[i]: pages (of all heads) of the sequences before thread i's share of
// `per` sequences.
struct Q4Space {
  const DecodeQ4Args& a;
  const int* pre;
  int shares, per;
  uint32_t T, G, W;      // pages, CTAs with work, warps of those
  uint32_t quot, rem;    // T / W, T % W

  __device__ __forceinline__ int len(int b) const {
    if (a.seq_lens == nullptr) return a.kv_len;
    return min(max(__ldg(a.seq_lens + b), 0), a.kv_len);
  }
  __device__ __forceinline__ int pages(int b) const { return (len(b) + kQ4Page - 1) / kQ4Page; }
  // First page of warp w's run, floor(w T / W): W < 2^16, so 32 bits are enough.
  __device__ __forceinline__ uint32_t start(uint32_t w) const { return w * quot + w * rem / W; }
  // The CTA whose runs hold page x.
  __device__ __forceinline__ uint32_t owner(uint32_t x) const {
    return (uint32_t)(((uint64_t)(x + 1) * G - 1) / T);
  }
};

// A place in the page space: page `local` of unit (b, hu), which starts at page
// `ua` of the space and has `tiles` pages.
struct Q4Cursor {
  int b, hu, local, tiles, len, ua;

  // The whole warp calls this together.
  __device__ __forceinline__ void seek(const Q4Space& s, int x) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    if (s.a.seq_lens == nullptr) {
      const int per_seq = s.pages(0) * s.a.Hkv;
      b = x / per_seq;
      base = b * per_seq;
    } else {
      // last share with pre <= x (it is not empty): first among every 32nd part's first, then in that part
      const int part = s.shares / 32;
      int lo = __popc(__ballot_sync(0xffffffffu, s.pre[lane * part] <= x)) - 1;
      lo = lo * part + __popc(__ballot_sync(0xffffffffu, lane < part && s.pre[lo * part + min(lane, part - 1)] <= x)) - 1;
      if (s.per == 1) {
        b = lo;
        base = s.pre[lo];
      } else {
        const int i = lo * s.per + lane;
        const int n = lane < s.per && i < s.a.B ? s.pages(i) * s.a.Hkv : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const int first = __ffs(__ballot_sync(0xffffffffu, s.pre[lo] + inc > x)) - 1;
        b = lo * s.per + first;
        base = s.pre[lo] + __shfl_sync(0xffffffffu, inc - n, first);
      }
    }
    len = s.len(b);
    tiles = (len + kQ4Page - 1) / kQ4Page;
    hu = (x - base) / tiles;
    local = (x - base) % tiles;
    ua = base + hu * tiles;
  }
  __device__ __forceinline__ void next_page(const Q4Space& s) {
    if (++local < tiles) return;
    local = 0;
    ua += tiles;
    if (++hu < s.a.Hkv) return;
    hu = 0;
    tiles = 0;
    while (++b < s.a.B) {
      len = s.len(b);
      tiles = (len + kQ4Page - 1) / kQ4Page;
      if (tiles > 0) return;
    }
  }
  // The page's entry in the page table, and from it its block.
  __device__ __forceinline__ int entry(const Q4Space& s) const {
    return s.a.page_table == nullptr ? 0 : __ldg(s.a.page_table + (size_t)b * s.a.max_pages + local);
  }
  __device__ __forceinline__ size_t block(const Q4Space& s, int page) const {
    const DecodeQ4Args& a = s.a;
    if (a.page_table == nullptr)
      return ((size_t)b * a.Hkv + hu) * (size_t)((a.kv_len + kQ4Page - 1) / kQ4Page) + local;
    if (page < 0 || page >= a.num_pages) {
      report_error(1 /* PLX_DEVERR_BAD_PAGE */);
      page = 0;
    }
    return (size_t)page * a.Hkv + hu;
  }
};

// Writes four neighbouring columns of one output row.
__device__ __forceinline__ void store_out4(const DecodeQ4Args& a, size_t idx, float v0, float v1, float v2, float v3) {
  if (a.out_bf16)
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + idx) =
        make_uint2(pack_bf16(v0, v1), pack_bf16(v2, v3));
  else
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + idx) = make_float4(v0, v1, v2, v3);
}

// The running state of a warp for one unit, in registers: lane (r, c) =
// (lane / 4, lane % 4) holds heads c + 4 t and of each the columns 32 j + 4 r
// + 0 .. 3.
template <int D, int NT>
struct Q4WarpState {
  static constexpr int G = D / 64, J = D / 32;
  float o[NT][2 * J][4];       // codes' sums: [2 j + h]: columns +2 h, +2 h + 1 (O1, O2 each)
  float pm[NT][G][2];          // sum p m, sum pa m of the lane's tokens
  float m[NT], l[NT], c[NT], aref[NT];
  float xref[NT];              // score of the key whose probe value is aref
  float unit[NT];              // aref, c and O2 are in this many ones (a power of two)

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < 2 * J; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) pm[t][g][0] = pm[t][g][1] = 0.f;
      m[t] = xref[t] = -INFINITY;
      l[t] = c[t] = aref[t] = 0.f;
      unit[t] = 1.f;
    }
  }
  // Moves one column's sums of codes, of every column of its group, into the
  // minima's sums (which all columns share).
  __device__ __forceinline__ void settle() {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float d0 = __shfl_sync(0xffffffffu, o[t][4 * g][0], lane & 3);
        const float d1 = __shfl_sync(0xffffffffu, o[t][4 * g][1], lane & 3);
#pragma unroll
        for (int i = 4 * g; i < 4 * g + 4; ++i) {
          o[t][i][0] -= d0;
          o[t][i][1] -= d1;
          o[t][i][2] -= 16.f * d0;
          o[t][i][3] -= 16.f * d1;
        }
        if (lane < 4) {
          pm[t][g][0] = fmaf(d0, 16777216.f, pm[t][g][0]);
          pm[t][g][1] = fmaf(d1, 16777216.f, pm[t][g][1]);
        }
      }
  }
  // Sums over the lanes that hold other tokens of the same heads; the codes'
  // powers of two, the minima's sums and the unit go in.  l becomes 1 to 2
  // first (and m what that took), so that c and O2 are no larger than the probe
  // values make them.
  __device__ __forceinline__ void close() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l[t] += __shfl_xor_sync(0xffffffffu, l[t], off);
        c[t] += __shfl_xor_sync(0xffffffffu, c[t], off);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          pm[t][g][0] += __shfl_xor_sync(0xffffffffu, pm[t][g][0], off);
          pm[t][g][1] += __shfl_xor_sync(0xffffffffu, pm[t][g][1], off);
        }
      }
      const int e = min(max((int)(__float_as_uint(l[t]) >> 23) - 127, -126), 126);
      const float f = __uint_as_float((uint32_t)(127 - e) << 23);
      m[t] += e;
      l[t] *= f;
      c[t] = c[t] * f * unit[t];
#pragma unroll
      for (int i = 0; i < 2 * J; ++i) {
        o[t][i][0] = fmaf(o[t][i][0], 16777216.f, pm[t][i / 4][0]) * f;
        o[t][i][1] = fmaf(o[t][i][1], 16777216.f, pm[t][i / 4][1]) * f * unit[t];
        o[t][i][2] = fmaf(o[t][i][2], 1048576.f, pm[t][i / 4][0]) * f;
        o[t][i][3] = fmaf(o[t][i][3], 1048576.f, pm[t][i / 4][1]) * f * unit[t];
      }
      aref[t] *= unit[t];
    }
  }
  // After close(): the finished output rows.
  __device__ __forceinline__ void write_out(const DecodeQ4Args& a, int b, int hu) const {
    const int r = (threadIdx.x & 31) >> 2, hc = threadIdx.x & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int h = 4 * t + hc;
      if (h >= a.group) continue;
      const size_t row = ((size_t)b * a.Hq + (size_t)hu * a.group + h) * D;
#pragma unroll
      for (int j = 0; j < J; ++j)
        store_out4(a, row + 32 * j + 4 * r, finalize(o[t][2 * j][0], o[t][2 * j][1], l[t], c[t]),
                   finalize(o[t][2 * j][2], o[t][2 * j][3], l[t], c[t]),
                   finalize(o[t][2 * j + 1][0], o[t][2 * j + 1][1], l[t], c[t]),
                   finalize(o[t][2 * j + 1][2], o[t][2 * j + 1][3], l[t], c[t]));
    }
  }
  // After close(): the piece, as [head][m l c aref O1 O2].
  __device__ __forceinline__ void deposit(float* dst) const {
    const int r = (threadIdx.x & 31) >> 2, hc = threadIdx.x & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float* row = dst + (4 * t + hc) * (2 * D + 4);
      if (r == 0) *reinterpret_cast<float4*>(row) = make_float4(m[t], l[t], c[t], aref[t]);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        *reinterpret_cast<float4*>(row + 4 + 32 * j + 4 * r) =
            make_float4(o[t][2 * j][0], o[t][2 * j][2], o[t][2 * j + 1][0], o[t][2 * j + 1][2]);
        *reinterpret_cast<float4*>(row + 4 + D + 32 * j + 4 * r) =
            make_float4(o[t][2 * j][1], o[t][2 * j][3], o[t][2 * j + 1][1], o[t][2 * j + 1][3]);
      }
    }
  }
};

// Adds a page's tokens to the sums: weights from the scores fs x and probe
// values av against the reference st.m, 16 tokens at a time.  `slot`: the page's value
// codes and parameters.  Weights are fp16 pairs: rounded, and what that left.
template <int D, int NT>
__device__ __forceinline__ void q4_value_sums(Q4WarpState<D, NT>& st, const uint8_t* slot, const float (&fs)[NT],
                                              const float (&x)[NT][8], const float (&av)[NT][8]) {
  using SM = Q4Smem<D, NT>;
  constexpr int G = D / 64, J = D / 32;
  const int lane = threadIdx.x & 31, r = lane >> 2, hc = lane & 3;
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    uint32_t bh[NT][G][2], bl[NT][G][2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int e = 2 * kk + half;
      uint32_t vp[G];
      lds_words<G>(slot + SM::kCodes + (16 * kk + r + 8 * half) * (4 * G), vp);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float p = ex2(fmaf(fs[t], x[t][e], kQ4Top - st.m[t])), pa = p * av[t][e];
        st.l[t] += p;
        st.c[t] += pa;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float s = bf16_lo_f(vp[g]), mn = bf16_hi_f(vp[g]);
          st.pm[t][g][0] = fmaf(p, mn, st.pm[t][g][0]);
          st.pm[t][g][1] = fmaf(pa, mn, st.pm[t][g][1]);
          const float ps = p * s, pas = pa * s;
          const uint32_t hi = pack_half(ps, pas);
          bh[t][g][half] = transpose_8x8(hi);
          const float2 hf = unpack_half(hi);
          bl[t][g][half] = transpose_8x8(pack_half(ps - hf.x, pas - hf.y));
        }
      }
    }
    uint32_t w0[J], w1[J];
    lds_words<J>(slot + (8 * kk + hc) * D + r * (D / 8), w0);
    lds_words<J>(slot + (8 * kk + hc + 4) * D + r * (D / 8), w1);
#pragma unroll
    for (int j = 0; j < J; j += 2) {   // the two words of a group: four products, then their low halves
      uint32_t av4[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t u0 = w0[j + q / 2] >> (8 * (q & 1)), u1 = w1[j + q / 2] >> (8 * (q & 1));
        av4[q][0] = u0 & 0x000f000fu;
        av4[q][1] = u0 & 0x00f000f0u;
        av4[q][2] = u1 & 0x000f000fu;
        av4[q][3] = u1 & 0x00f000f0u;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          mma_f16_16816(st.o[t][2 * j + q], av4[q][0], av4[q][1], av4[q][2], av4[q][3], bh[t][j / 2][0], bh[t][j / 2][1]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          mma_f16_16816(st.o[t][2 * j + q], av4[q][0], av4[q][1], av4[q][2], av4[q][3], bl[t][j / 2][0], bl[t][j / 2][1]);
      }
    }
  }
}

// The running sum of a unit's pieces for four columns of one head.
struct Q4Merged {
  float m = -INFINITY, l = 0.f, c = 0.f, aref = 0.f;
  float4 o1 = make_float4(0.f, 0.f, 0.f, 0.f), o2 = make_float4(0.f, 0.f, 0.f, 0.f);

  // Adds the piece (head = m, l, c, aref; p1, p2 its columns): both sides at
  // the larger reference, the piece's probe values from this sum's offset.
  __device__ __forceinline__ void add(const float4& head, const float4& p1, const float4& p2) {
    const bool first = l == 0.f && m == -INFINITY;
    const float mx = fmaxf(m, head.x), al = first ? 0.f : ex2(m - mx), be = ex2(head.x - mx);
    if (first) aref = head.w;
    const float shift = head.w - aref;
    m = mx;
    l = fmaf(be, head.y, al * l);
    c = fmaf(be, fmaf(shift, head.y, head.z), al * c);
    o1.x = fmaf(be, p1.x, al * o1.x);
    o1.y = fmaf(be, p1.y, al * o1.y);
    o1.z = fmaf(be, p1.z, al * o1.z);
    o1.w = fmaf(be, p1.w, al * o1.w);
    o2.x = fmaf(be, fmaf(shift, p1.x, p2.x), al * o2.x);
    o2.y = fmaf(be, fmaf(shift, p1.y, p2.y), al * o2.y);
    o2.z = fmaf(be, fmaf(shift, p1.z, p2.z), al * o2.z);
    o2.w = fmaf(be, fmaf(shift, p1.w, p2.w), al * o2.w);
  }
  __device__ __forceinline__ void write_out(const DecodeQ4Args& a, size_t idx) const {
    store_out4(a, idx, finalize(o1.x, o2.x, l, c), finalize(o1.y, o2.y, l, c), finalize(o1.z, o2.z, l, c),
               finalize(o1.w, o2.w, l, c));
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(Q4Smem<D, NT>::kThreads, 1) decode_q4_kernel(const DecodeQ4Args a) {
  using SM = Q4Smem<D, NT>;
  using B = Q4Block<D>;
  constexpr int S = SM::kSlots, G = D / 64, J = D / 32, kWarps = SM::kWarps, kThreads = SM::kThreads;
  extern __shared__ __align__(128) uint8_t q4_smem[];
  int* meta = reinterpret_cast<int*>(q4_smem + SM::kMetaOff);   // [warp]: first piece's unit, ua, ub; last piece's
  int* pre = reinterpret_cast<int*>(q4_smem + SM::kPreOff);
  __shared__ int s_last[kWarps / 4];
  __shared__ int s_part[kWarps];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, hc = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- the page space
  Q4Space sp{a, pre, kThreads, (a.B + kThreads - 1) / kThreads};
  if (a.seq_lens == nullptr) {
    sp.T = (uint32_t)a.B * a.Hkv * ((a.kv_len + kQ4Page - 1) / kQ4Page);
  } else {
    int sum = 0;
    const int b0 = min(a.B, tid * sp.per), b1 = min(a.B, b0 + sp.per);
    for (int b = b0; b < b1; ++b) {
      const int n = __ldg(a.seq_lens + b);
      if ((n < 0 || n > a.kv_len) && blockIdx.x == 0) report_error(4 /* PLX_DEVERR_BAD_LENGTH */);
      sum += sp.pages(b) * a.Hkv;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) s_part[warp] = inc;
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) base = total;
      total += s_part[w];
    }
    pre[tid] = base + inc - sum;
    sp.T = total;
  }
  __syncthreads();
  sp.G = min((uint32_t)gridDim.x, (sp.T + a.min_pages - 1) / a.min_pages);
  // Sequences without tokens have no pages: their rows are zero.
  auto zero_rows = [&] {
    if (a.seq_lens == nullptr) return;
    for (int b = blockIdx.x; b < a.B; b += gridDim.x)
      if (sp.len(b) == 0)
        for (int i = tid; i < a.Hq * D / 4; i += kThreads) store_out4(a, (size_t)b * a.Hq * D + 4 * i, 0.f, 0.f, 0.f, 0.f);
  };
  if (blockIdx.x >= sp.G) {
    zero_rows();
    return;
  }
  sp.W = sp.G * kWarps;
  sp.quot = sp.T / sp.W;
  sp.rem = sp.T % sp.W;

  const uint32_t gw = blockIdx.x * kWarps + warp;
  const int y0 = (int)sp.start(gw), y1 = (int)sp.start(gw + 1), n = y1 - y0;
  uint8_t* ring = q4_smem + warp * SM::kRing;
  uint8_t* q_rows = q4_smem + SM::kQOff + warp * SM::kQ;
  float* first_state = reinterpret_cast<float*>(q4_smem + SM::kStateOff + warp * SM::kState);
  if (lane < 8) meta[warp * 8 + lane] = -1;
  __syncwarp();

  if (n > 0) {
    Q4Cursor cur, ahead;
    cur.seek(sp, y0);
    ahead = cur;
    // The q and rho rows of a unit come the same way, into q_rows: row 8 t + 2 i
    // is q and row 8 t + 2 i + 1 rho of head 4 t + i (zeros past the group).  They
    // are asked for before the unit's first pages (behind those they waited for
    // 2.5 us of page copies), the next unit's as soon as the warp has made its
    // operands of the current one's.
    auto fetch_q = [&](int b, int hu) {
#pragma unroll
      for (int k = lane; k < 8 * NT * (D / 8); k += 32) {
        const int n = k / (D / 8), v = k % (D / 8), h = n / 2;
        const bool live = h < a.group;
        const __nv_bfloat16* src = ((n & 1) ? a.rho : a.q) +
                                   ((size_t)b * a.Hq + (size_t)hu * a.group + (live ? h : 0)) * D + 8 * v;
        q4_copy16(smem_u32(q_rows + n * SM::kQRow + 16 * v), src, live);
      }
    };
    fetch_q(cur.b, cur.hu);
    // Part 2 i is the keys of the run's page i, part 2 i + 1 its values; part k
    // goes to slot k % S.  A page's entry in the page table is read when the
    // part before it is issued and looked at when its own keys are.  Every
    // part is one group of 16-byte asynchronous copies, 512 bytes a step of
    // the warp (past the run's end the groups are empty), so that part k has
    // landed once at most S - 1 groups are on their way.
    int issued = 0, entry = ahead.entry(sp);
    const uint8_t* src = nullptr;
    const uint32_t ring_lane = smem_u32(ring) + 16 * lane;
    uint32_t fill = ring_lane;        // where the next part goes
    auto issue = [&](auto part) {     // part: 0 for keys, 1 for values (of the page that is due)
      constexpr bool kValues = decltype(part)::value;
      if (issued < 2 * n) {
        if (!kValues) src = a.cache + ahead.block(sp, entry) * B::kBytes + 16 * lane;
        constexpr int kFrom = kValues ? B::kV : 0, kParams = kValues ? B::kVParams : B::kKParams;
#pragma unroll
        for (int c = 0; c < SM::kCodes; c += 512) q4_copy16(fill + c, src + kFrom + c);
        if (B::kParamBytes == 512 || lane < B::kParamBytes / 16) q4_copy16(fill + SM::kCodes, src + kParams);
        ++issued;
        fill = fill == ring_lane + (S - 1) * SM::kPart ? ring_lane : fill + SM::kPart;
        if (kValues && issued < 2 * n) {
          ahead.next_page(sp);
          entry = ahead.entry(sp);
        }
      }
      q4_copy_commit();
    };
    using Keys = std::integral_constant<bool, false>;
    using Values = std::integral_constant<bool, true>;
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if (k % 2 == 0) issue(Keys{}); else issue(Values{});
    }

    Q4WarpState<D, NT> st;
    uint32_t qf[NT][D / 16][2];     // [q rho ..] operand
    float fs[NT], fa[NT];           // factors of a score (in powers of two; positive) and of a probe value
    float qs[NT][G], rs[NT][G];     // group sums of q (over fs) and rho
    int seg = 0;                    // pages of the current unit done by this warp
    uint8_t* slot = ring;
    auto landed = [&] {             // the slot's part is there, for every lane
      q4_copy_wait<S - 1>();
      __syncwarp();
    };
    auto leave = [&](auto part) {   // done with the slot: refill it, go to the next one
      __syncwarp();
      issue(part);
      slot = slot == ring + (S - 1) * SM::kPart ? ring : slot + SM::kPart;
    };
    // A value page's parameters of tokens past the sequence's end become zero
    // (they may be NaN).
    auto clear_tail = [&](int nvalid) {
      for (int tok = nvalid + lane; tok < kQ4Page; tok += 32)
#pragma unroll
        for (int g = 0; g < G; ++g) reinterpret_cast<uint32_t*>(slot + SM::kCodes)[tok * G + g] = 0;
      __syncwarp();
    };

    for (int i = 0; i < n; ++i) {
      landed();
      const int nvalid = cur.len - cur.local * kQ4Page;   // tokens of this page (>= 1; 64 or more: all)
      if (seg == 0) {
        // The unit's rows went out with the part that followed the previous
        // unit's first keys, at the latest the last but one so far.
        if constexpr (S > 2) {
          q4_copy_wait<1>();
          __syncwarp();
        }
        st.reset();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          uint4 v[J];
#pragma unroll
          for (int j = 0; j < J; ++j)
            v[j] = *reinterpret_cast<const uint4*>(q_rows + (8 * t + r) * SM::kQRow + 64 * j + 16 * hc);
          float f[J][8], mx = 0.f, gsum[G];
#pragma unroll
          for (int g = 0; g < G; ++g) gsum[g] = 0.f;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[j][2 * e] = bf16_lo_f(w[e]);
              f[j][2 * e + 1] = bf16_hi_f(w[e]);
              mx = fmaxf(mx, fmaxf(fabsf(f[j][2 * e]), fabsf(f[j][2 * e + 1])));
              gsum[j / 2] += f[j][2 * e] + f[j][2 * e + 1];
            }
          }
#pragma unroll
          for (int off = 1; off < 4; off <<= 1) {
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
#pragma unroll
            for (int g = 0; g < G; ++g) gsum[g] += __shfl_xor_sync(0xffffffffu, gsum[g], off);
          }
          // 2^up takes the row's largest entry into [2^13, 2^14); clamped so
          // that the power and its inverse times 2^24 are normal numbers
          const int up = min(120, max(-100, 13 - ((int)(__float_as_uint(mx) >> 23) - 127)));
          const float inv = __uint_as_float((uint32_t)(24 - up + 127) << 23);
          // (a negative scale turns q around)
          const float sc = __uint_as_float((uint32_t)(up + 127) << 23 | (a.scale_log2 < 0.f && !(r & 1) ? 0x80000000u : 0u));
          const float unit = __uint_as_float((uint32_t)(up - 24 + 127) << 23 | (__float_as_uint(sc) & 0x80000000u));
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const float lo = sc * 0.0625f;   // the codes of odd pairs are 2^4 larger
            qf[t][2 * j][0] = pack_half(f[j][0] * sc, f[j][1] * sc);
            qf[t][2 * j][1] = pack_half(f[j][2] * lo, f[j][3] * lo);
            qf[t][2 * j + 1][0] = pack_half(f[j][4] * sc, f[j][5] * sc);
            qf[t][2 * j + 1][1] = pack_half(f[j][6] * lo, f[j][7] * lo);
          }
          // rows 2 hc and 2 hc + 1 are this lane's head's q and rho
          fs[t] = fmaxf(__shfl_sync(0xffffffffu, inv, 8 * hc) * fabsf(a.scale_log2), 0x1p-126f);   // (-inf stays -inf at scale 0)
          fa[t] = __shfl_sync(0xffffffffu, inv, 8 * hc + 4);
#pragma unroll
          for (int g = 0; g < G; ++g) {
            qs[t][g] = __shfl_sync(0xffffffffu, gsum[g] * unit, 8 * hc);
            rs[t][g] = __shfl_sync(0xffffffffu, gsum[g], 8 * hc + 4);
          }
        }
        if (i + cur.tiles - cur.local < n) {   // the run goes on past this unit
          Q4Cursor next = cur;
          next.local = next.tiles - 1;
          next.next_page(sp);
          __syncwarp();   // every lane has read the rows
          fetch_q(next.b, next.hu);
        }
      }

      // ---- scores and probe values of tokens 16 mt + r and + 8
      float x[NT][8], av[NT][8];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        uint32_t w0[J], w1[J];
        lds_words<J>(slot + (16 * mt + r) * (D / 2) + hc * (D / 8), w0);
        lds_words<J>(slot + (16 * mt + r + 8) * (D / 2) + hc * (D / 8), w1);
        float acc[NT][G][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int g = 0; g < G; ++g) acc[t][g][0] = acc[t][g][1] = acc[t][g][2] = acc[t][g][3] = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t u0 = w0[j] >> (8 * h), u1 = w1[j] >> (8 * h);
#pragma unroll
            for (int t = 0; t < NT; ++t)
              mma_f16_16816(acc[t][j / 2], u0 & 0x000f000fu, u1 & 0x000f000fu, u0 & 0x00f000f0u, u1 & 0x00f000f0u,
                            qf[t][2 * j + h][0], qf[t][2 * j + h][1]);
          }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t kp[G];
          lds_words<G>(slot + SM::kCodes + (16 * mt + r + 8 * half) * (4 * G), kp);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float s = 0.f, p = 0.f, pmn = -st.aref[t];   // (aref is 0 until the unit's first page has given it)
#pragma unroll
            for (int g = 0; g < G; ++g) {
              s = fmaf(bf16_lo_f(kp[g]), acc[t][g][2 * half], s);
              p = fmaf(bf16_lo_f(kp[g]), acc[t][g][2 * half + 1], p);
              s = fmaf(bf16_hi_f(kp[g]), qs[t][g], s);
              pmn = fmaf(bf16_hi_f(kp[g]), rs[t][g], pmn);
            }
            x[t][2 * mt + half] = s;   // over fs
            av[t][2 * mt + half] = fmaf(fa[t], p, pmn);
          }
        }
      }
      leave(std::integral_constant<bool, S % 2 != 0>{});   // part 2 i + S

      landed();
      if (nvalid < kQ4Page) {   // tokens past the sequence's end weigh nothing, whatever their parameters
        clear_tail(nvalid);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (16 * (e >> 1) + r + 8 * (e & 1) >= nvalid) {
              x[t][e] = -INFINITY;
              av[t][e] = 0.f;
            }
      }

      // ---- the running reference: the page's largest score, probe value and scale
      float mx[NT], ma[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mx[t] = max3(max3(x[t][0], x[t][1], x[t][2]), max3(x[t][3], x[t][4], x[t][5]), fmaxf(x[t][6], x[t][7]));
        ma[t] = max3(max3(fabsf(av[t][0]), fabsf(av[t][1]), fabsf(av[t][2])),
                     max3(fabsf(av[t][3]), fabsf(av[t][4]), fabsf(av[t][5])),
                     max3(fabsf(av[t][6]), fabsf(av[t][7]), 1.f));
      }
      float vbig;   // log2 of the largest scale, or of what keeps the sums of p m (below 2^99) in fp32's range where it is smaller
      {
        uint32_t w[2 * G];
        lds_words<2 * G>(slot + SM::kCodes + lane * (8 * G), w);
        __nv_bfloat162 m2 = __habs2(*reinterpret_cast<__nv_bfloat162*>(&w[0]));
#pragma unroll
        for (int k = 1; k < 2 * G; ++k) m2 = __hmax2(m2, __habs2(*reinterpret_cast<__nv_bfloat162*>(&w[k])));
        const uint32_t both = *reinterpret_cast<uint32_t*>(&m2);   // scales are in the low half
        const float v = max3(bf16_lo_f(both), bf16_hi_f(both) * 0x1p-40f, 0x1p-84f);
        vbig = lg2(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v))));
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          mx[t] = fmaxf(mx[t], __shfl_xor_sync(0xffffffffu, mx[t], off));
          ma[t] = fmaxf(ma[t], __shfl_xor_sync(0xffffffffu, ma[t], off));
        }
      float need[NT];
      bool due = false;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        need[t] = fs[t] * mx[t] + fminf(lg2(ma[t]) + vbig, 100.f);
        due = due || need[t] > st.m[t] + kQ4Slack || fs[t] * mx[t] > st.xref[t] + kQ4Slack || ma[t] > kQ4MaxProbe;
      }
      due = due || seg % kQ4Settle == kQ4Settle - 1;
      if (__any_sync(0xffffffffu, due)) {   // (settling apart from this, each page waited for its products: 4% of the time)
        st.settle();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          // aref goes to the key with the page's largest score
          bool mine = false;
          float here = 0.f;
#pragma unroll
          for (int e = 7; e >= 0; --e)
            if (x[t][e] == mx[t]) {
              mine = true;
              here = av[t][e];
            }
          const uint32_t holders = __ballot_sync(0xffffffffu, mine) & (0x11111111u << hc);
          float shift = __shfl_sync(0xffffffffu, here, holders ? __ffs(holders) - 1 : 0);
          if (!(fs[t] * mx[t] > st.xref[t] + kQ4Slack) || holders == 0) shift = 0.f;
          else st.xref[t] = fs[t] * mx[t];
          ma[t] = 1.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (x[t][e] > -INFINITY) av[t][e] -= shift;   // (tokens past the end keep theirs, 0)
            ma[t] = fmaxf(ma[t], fabsf(av[t][e]));
          }
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) ma[t] = fmaxf(ma[t], __shfl_xor_sync(0xffffffffu, ma[t], off));
          // large probe values get a larger unit
          const int up = ma[t] > kQ4MaxProbe ? min((int)(__float_as_uint(ma[t]) >> 23) - 127, 126) : 0;
          const float f = __uint_as_float((uint32_t)(127 - up) << 23);
          st.unit[t] *= __uint_as_float((uint32_t)(127 + up) << 23);
          fa[t] *= f;
          ma[t] = fmaxf(ma[t] * f, 1.f);
#pragma unroll
          for (int g = 0; g < G; ++g) rs[t][g] *= f;
#pragma unroll
          for (int e = 0; e < 8; ++e) av[t][e] *= f;
          // and the reference moves if it still has to
          need[t] = fs[t] * mx[t] + fminf(lg2(ma[t]) + vbig, 100.f);
          const float m_new = need[t] > st.m[t] + kQ4Slack ? need[t] : st.m[t];
          const float alpha = m_new == st.m[t] ? 1.f : ex2(st.m[t] - m_new), alpha2 = alpha * f;
          st.m[t] = m_new;
          st.aref[t] = (st.aref[t] + shift) * f;
          st.c[t] = fmaf(-shift, st.l[t], st.c[t]) * alpha2;
          st.l[t] *= alpha;
#pragma unroll
          for (int k = 0; k < 2 * J; ++k) {
            st.o[t][k][1] = fmaf(-shift, st.o[t][k][0], st.o[t][k][1]) * alpha2;
            st.o[t][k][3] = fmaf(-shift, st.o[t][k][2], st.o[t][k][3]) * alpha2;
            st.o[t][k][0] *= alpha;
            st.o[t][k][2] *= alpha;
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            st.pm[t][g][1] = fmaf(-shift, st.pm[t][g][0], st.pm[t][g][1]) * alpha2;
            st.pm[t][g][0] *= alpha;
          }
        }
      }

      q4_value_sums<D, NT>(st, slot, fs, x, av);
      leave(std::integral_constant<bool, S % 2 == 0>{});
      ++seg;

      if (cur.local + 1 == cur.tiles && (i + 1 < n || seg == cur.tiles)) {
        // the unit ends here: finish it, or leave the run's first piece
        st.close();
        if (seg == cur.tiles) {
          st.write_out(a, cur.b, cur.hu);
        } else {
          st.deposit(first_state);
          if (lane == 0) {
            meta[warp * 8 + 0] = cur.b * a.Hkv + cur.hu;
            meta[warp * 8 + 1] = cur.ua;
            meta[warp * 8 + 2] = cur.ua + cur.tiles;
          }
        }
        seg = 0;
      }
      if (i + 1 < n) cur.next_page(sp);
    }
    if (seg > 0) {   // the run's last piece, into the ring, which holds no copy any more
      st.close();
      st.deposit(reinterpret_cast<float*>(ring));
      if (lane == 0) {
        meta[warp * 8 + 3] = cur.b * a.Hkv + cur.hu;
        meta[warp * 8 + 4] = cur.ua;
        meta[warp * 8 + 5] = cur.ua + cur.tiles;
      }
    }
  }
  zero_rows();
  __syncthreads();

  // ---- merge the CTA's pieces.  A team of four warps takes every kTeams-th
  // unit: a thread four columns of a head.  Lane k knows piece k of the CTA:
  // warp k / 2's first (even k) or last one; pieces of a unit are in order.
  constexpr int kTeams = kWarps / 4;
  const int team = warp / 4, tt = tid % 128;
  const int x0 = (int)sp.start(blockIdx.x * kWarps), x1 = (int)sp.start((blockIdx.x + 1) * kWarps);
  const int my_unit = lane < 2 * kWarps ? meta[(lane >> 1) * 8 + 3 * (lane & 1)] : -1;
  uint32_t todo = __ballot_sync(0xffffffffu, my_unit >= 0);
  auto team_bar = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + team) : "memory"); };
  for (int k = 0; todo != 0; ++k) {
    const int first = __ffs(todo) - 1, unit = __shfl_sync(0xffffffffu, my_unit, first);
    const uint32_t pieces = __ballot_sync(0xffffffffu, my_unit == unit);
    todo &= ~pieces;
    if (k % kTeams != team) continue;
    const int ua = meta[(first >> 1) * 8 + 3 * (first & 1) + 1], ub = meta[(first >> 1) * 8 + 3 * (first & 1) + 2];
    const bool whole = ua >= x0 && ub <= x1;
    const size_t out_row = ((size_t)(unit / a.Hkv) * a.Hq + (size_t)(unit % a.Hkv) * a.group) * D;
    const int items = a.group * (D / 4);
    const size_t slot_stride = (size_t)a.group * SM::kRow;
    const uint32_t c0 = whole ? 0 : sp.owner(ua), c1 = whole ? 0 : sp.owner(ub - 1);
    // Slot 2 c holds a piece of a unit that goes on from CTA c - 1 (or starts
    // with c), slot 2 c + 1 one that starts inside c; of a unit's CTAs only the
    // first can hold it in the second.
    const bool inside = !whole && (int)sp.start(c0 * kWarps) < ua;
    auto slot_of = [&](uint32_t c) { return a.slots + (2 * c + (c == c0 && inside ? 1 : 0)) * slot_stride; };
    for (int i = tt; i < items; i += 128) {
      const int h = i / (D / 4), d = 4 * (i % (D / 4));
      Q4Merged s;
      for (uint32_t left = pieces; left; left &= left - 1) {
        const int q = __ffs(left) - 1;
        const float* p = reinterpret_cast<const float*>((q & 1) ? q4_smem + (q >> 1) * SM::kRing
                                                                : q4_smem + SM::kStateOff + (q >> 1) * SM::kState) +
                         h * SM::kRow;
        s.add(*reinterpret_cast<const float4*>(p), *reinterpret_cast<const float4*>(p + 4 + d),
              *reinterpret_cast<const float4*>(p + 4 + D + d));
      }
      if (whole) {
        s.write_out(a, out_row + (size_t)h * D + d);
      } else {
        float* p = slot_of(blockIdx.x) + h * SM::kRow;
        *reinterpret_cast<float4*>(p + 4 + d) = s.o1;
        *reinterpret_cast<float4*>(p + 4 + D + d) = s.o2;
        if (d == 0) *reinterpret_cast<float4*>(p) = make_float4(s.m, s.l, s.c, s.aref);
      }
    }
    if (whole) continue;
    team_bar();
    if (tt == 0) {   // (the barrier puts the team's writes before this thread's fence, and its fence before their reads)
      __threadfence();
      const bool last = atomicAdd(a.counters + unit, 1) == (int)(c1 - c0);
      s_last[team] = last;
      if (last) atomicExch(a.counters + unit, 0);
      __threadfence();
    }
    team_bar();
    if (s_last[team]) {
      for (int i = tt; i < items; i += 128) {
        const int h = i / (D / 4), d = 4 * (i % (D / 4));
        Q4Merged s;
#pragma unroll 4
        for (uint32_t c = c0; c <= c1; ++c) {
          const float* p = slot_of(c) + h * SM::kRow;
          s.add(__ldcg(reinterpret_cast<const float4*>(p)), __ldcg(reinterpret_cast<const float4*>(p + 4 + d)),
                __ldcg(reinterpret_cast<const float4*>(p + 4 + D + d)));
        }
        s.write_out(a, out_row + (size_t)h * D + d);
      }
    }
    team_bar();   // s_last can be written again
  }
}

}  // namespace plx
