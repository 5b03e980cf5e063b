// RMS norm of head rows with the position rotation, forward and backward (the
// definition is at parallax_norm_rope in parallax.h).
//
//     n = x r w,  r = (mean x^2 + eps)^(-1/2),   y = R n
// with R the rotation of column pairs.  R is orthogonal, so with dn = R^T dy
// and g = dn w
//     dx = r (g - x r^2 mean(g x)),   dw = sum over rows dn x r.
//
// Both directions read each row once and write one row: HBM bounds them.  A
// row lies in the 16-byte vectors of LPR neighbouring lanes (16 lanes for 128
// bf16 columns), so its sums are butterfly shuffles among them and the row
// never leaves registers.  A lane's columns are two runs of 8 bytes, one on
// each side of the pairs it turns (column f and f + rot/2; next to each other
// when interleaved or past rot), so that a pair never lies in two lanes: with
// whole 16-byte vectors the partner's came by four shuffles and was unpacked a
// second time.  A group of lanes takes several heads of one token, so a
// token's cos and sin are read once for them.
//
// Measured (device time in a graph, full clock, bf16, d = 128): 4 x 8192 tokens of 3 x 16
// heads forward (810 MB) 134 us, 6.0 TB/s; 4 x 8192 of 16 + 16 + 4 heads backward (910 MB)
// 150 us, 6.1 TB/s (138 to 141 and 168 to 171 us a call sustained for seconds); 8 tokens
// forward 2.1 us.
#pragma once

#include "ptx.cuh"

namespace plx {

constexpr int kNrFwdThreads = 64;   // (810 MB: 133.4 us; 134.4 with 128 threads, 136.1 with 256)
constexpr int kNrThreads = 256;     // backward (128: 1% slower on long rows, 15% on short ones)
constexpr int kNrMaxSets = 3;
constexpr int kNrBwdCtasPerSm = 3;
constexpr int kNrBwdHeads = 4;                                    // rows of an item
constexpr int kNrBwdSmem = 2 * kNrBwdHeads * 2 * kNrThreads * 16;  // two items' vectors
constexpr int kNrDwThreads = 1024;

struct NormRopeSet {
  const void* x;
  void* y;                // backward: dx
  const void* dy;         // backward only
  const void* w;
  float* dw;              // backward only
  int heads, chunks;      // chunks of `hpg` heads
  int ctas, first_cta;    // backward: its share of the grid
  long long xs[3], ys[3], ds[3];   // element strides of batch entry, token, head
};

struct NormRopeArgs {
  NormRopeSet set[kNrMaxSets];
  const int32_t* positions;
  const float* cos;
  const float* sin;
  float* partial;         // backward: [gridDim.x][D]
  long long pos_batch_stride;
  int sets, B, T, rot, max_pos, norm, hpg;
  float eps;
};

// Rows are read once and written once: neither way through L1, and out of L2
// first (810 MB forward: 147 to 133 us).
__device__ __forceinline__ uint2 load_row(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p)
               : "memory");   // (y may be x itself)
  return v;
}
__device__ __forceinline__ void store_row(void* p, uint32_t v0, uint32_t v1) {
  asm volatile("st.global.cs.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(v0), "r"(v1) : "memory");
}
// 16 bytes into shared memory as they arrive; zeros where !read.
__device__ __forceinline__ void copy_row(uint32_t dst, const void* src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
               "r"(read ? 16 : 0)
               : "memory");
}

// A lane's share of a row: E values from two runs of 8 bytes, in pairs (the
// packed fp32 arithmetic takes two at an instruction).
template <typename T>
struct RowVec;
template <>
struct RowVec<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float2 (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(bf16_lo_f(w[i]), bf16_hi_f(w[i]));
  }
  static __device__ __forceinline__ uint4 pack(const float2 (&f)[4]) {
    return make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y), pack_bf16(f[2].x, f[2].y),
                      pack_bf16(f[3].x, f[3].y));
  }
};
template <>
struct RowVec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float2 (&f)[2]) {
    f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ uint4 pack(const float2 (&f)[2]) {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                      __float_as_uint(f[1].y));
  }
};

// cos and sin of the lane's pairs at one position: pairs i and i + P/2 of its
// columns turn by (c, s)[i], or with kInter the two columns of pair i do.
// (1, 0) past rot.
template <int P, bool kInter>
struct Turn {
  static constexpr int N = kInter ? P : P / 2;
  float2 c[N], s[N];
};

template <int P, bool kInter>
__device__ __forceinline__ void load_turn(const NormRopeArgs& a, int pos, int col0, Turn<P, kInter>& t) {
  if (col0 >= a.rot) {
#pragma unroll
    for (int i = 0; i < t.N; ++i) {
      t.c[i] = make_float2(1.f, 1.f);
      t.s[i] = make_float2(0.f, 0.f);
    }
    return;
  }
  const size_t row = (size_t)pos * (a.rot / 2);
#pragma unroll
  for (int i = 0; i < t.N; ++i) {
    if (kInter) {
      const float c = __ldg(a.cos + row + col0 / 2 + i), s = __ldg(a.sin + row + col0 / 2 + i);
      t.c[i] = make_float2(c, c);
      t.s[i] = make_float2(s, s);
    } else {
      t.c[i] = __ldg(reinterpret_cast<const float2*>(a.cos + row + col0) + i);
      t.s[i] = __ldg(reinterpret_cast<const float2*>(a.sin + row + col0) + i);
    }
  }
}

__device__ __forceinline__ float2 neg2(float2 v) { return make_float2(-v.x, -v.y); }

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T, int D, bool kInter>
struct NrLane {
  static constexpr int E = RowVec<T>::E, P = E / 2, H = P / 2, LPR = D / E;
  int col0, col1;      // first columns of the two runs

  __device__ __forceinline__ explicit NrLane(const NormRopeArgs& a) {
    const int l = (threadIdx.x & 31) % LPR, turning = kInter ? 0 : a.rot / E;   // lanes with a run on each side
    col0 = l < turning ? l * (E / 2) : l * E;
    col1 = col0 + (l < turning ? a.rot / 2 : E / 2);
  }
  __device__ __forceinline__ uint4 weights(const void* w) const {
    if (w == nullptr) return make_uint4(0, 0, 0, 0);
    const uint2 v0 = __ldg(reinterpret_cast<const uint2*>(static_cast<const T*>(w) + col0));
    const uint2 v1 = __ldg(reinterpret_cast<const uint2*>(static_cast<const T*>(w) + col1));
    return make_uint4(v0.x, v0.y, v1.x, v1.y);
  }
  // The other column of each pair of columns.
  static __device__ __forceinline__ float2 partner(const float2 (&f)[P], int i) {
    return kInter ? make_float2(f[i].y, f[i].x) : f[(i + H) % P];
  }
  // Zeros where `zero`.
  __device__ __forceinline__ void store(T* row, const float2 (&o)[P], bool zero = false) const {
    const uint4 v = zero ? make_uint4(0, 0, 0, 0) : RowVec<T>::pack(o);
    store_row(row + col0, v.x, v.y);
    store_row(row + col1, v.z, v.w);
  }
};

// The position of a token, or -1 for padding (a bad one is reported).
__device__ __forceinline__ int nr_position(const NormRopeArgs& a, int b, int t) {
  if (a.positions == nullptr && t < a.max_pos) return t;
  const int pos = a.positions ? __ldg(a.positions + b * a.pos_batch_stride + t) : t;
  if (a.rot > 0 && pos >= 0 && pos < a.max_pos) return pos;
  if (a.rot == 0 && pos >= 0) return pos;
  if (pos != -1) report_error(32 /* PLX_DEVERR_BAD_POSITION */);
  return -1;
}

// A group of LPR lanes takes the rows of chunk blockIdx.y (a set's next `hpg`
// heads) of one token; neighbouring groups take neighbouring tokens.  20 CTAs an
// SM hold the bf16, not interleaved kernels to 48 registers and spill 32 bytes of set-up
// (810 MB: 134.1 us; 135.0 without the bound, on 56 registers, and 144.2 with 16 CTAs,
// on 61; 128 packed tokens of 40 heads the other way round, 3.9, 3.6 and 3.7).
template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kNrFwdThreads, 20) norm_rope_kernel(const NormRopeArgs a) {
  using L = NrLane<T, D, kInter>;
  constexpr int P = L::P;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const L ln(a);
  int chunk = blockIdx.y, si = 0;
  while (chunk >= a.set[si].chunks) chunk -= a.set[si++].chunks;
  const NormRopeSet& set = a.set[si];
  const int tok = (int)((blockIdx.x * kNrFwdThreads + threadIdx.x) / L::LPR);
  const int b = a.B == 1 ? 0 : tok / a.T, t = tok - b * a.T;
  const int h0 = chunk * a.hpg;
  const int pos = b < a.B && t < a.T ? nr_position(a, b, t) : -1;
  const bool live = pos >= 0, turns = ln.col0 < a.rot;
  // y = r (x wc + partner(x) ws) with the weights taken into the rotation
  float2 wc[P], ws[P];
  {
    Turn<P, kInter> tn;
    load_turn<P, kInter>(a, live ? pos : 0, live ? ln.col0 : D, tn);
    float2 w[P];
    RowVec<T>::unpack(ln.weights(set.w), w);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (set.w == nullptr) w[i] = make_float2(1.f, 1.f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 c = tn.c[i % tn.N], sn = tn.s[i % tn.N];
      wc[i] = mul2(w[i], c);
      ws[i] = mul2(L::partner(w, i), kInter ? make_float2(-sn.x, sn.y) : i < L::H ? neg2(sn) : sn);
    }
  }
  const T* x = static_cast<const T*>(set.x) + b * set.xs[0] + t * set.xs[1] + h0 * set.xs[2];
  T* y = static_cast<T*>(set.y) + b * set.ys[0] + t * set.ys[1] + h0 * set.ys[2];
  const int heads = live ? min(a.hpg, set.heads - h0) : 0;
  constexpr int U = 2;   // rows in flight (four, on 24 warps an SM instead of 40, are 1% slower, and more in small calls)
  for (int j = 0; j < a.hpg; j += U) {
    uint2 v0[U], v1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v0[u] = v1[u] = make_uint2(0, 0);
      if (j + u < heads) {
        v0[u] = load_row(x + (j + u) * set.xs[2] + ln.col0);
        v1[u] = load_row(x + (j + u) * set.xs[2] + ln.col1);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 f[P], o[P];
      RowVec<T>::unpack(make_uint4(v0[u].x, v0[u].y, v1[u].x, v1[u].y), f);
      float r = 1.f;
      if (a.norm) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) ss = fma2(mul2(f[i], make_float2(1.f / D, 1.f / D)), f[i], ss);   // (overflows only with the mean itself)
        r = rsqrtf(row_sum<L::LPR>(ss.x + ss.y) + a.eps);
      }
      // (past rot a column passes through: no term of a partner that may not be finite)
#pragma unroll
      for (int i = 0; i < P; ++i)
        o[i] = mul2(turns ? fma2(f[i], wc[i], mul2(L::partner(f, i), ws[i])) : mul2(f[i], wc[i]), make_float2(r, r));
      if (j + u < heads) ln.store(y + (j + u) * set.ys[2], o);
    }
  }
}

// Backward.  Every set has a share of the grid's CTAs by its number of heads;
// each CTA walks over its set's rows and leaves its sum for dw in
// partial[blockIdx.x].
template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kNrThreads, kNrBwdCtasPerSm) norm_rope_bwd_kernel(const NormRopeArgs a) {
  using L = NrLane<T, D, kInter>;
  constexpr int P = L::P;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const L ln(a);
  int si = 0;
  while (si + 1 < a.sets && (int)blockIdx.x >= a.set[si + 1].first_cta) ++si;
  const NormRopeSet& set = a.set[si];
  float2 w[P], acc[P];
  RowVec<T>::unpack(ln.weights(set.w), w);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (set.w == nullptr) w[i] = make_float2(1.f, 1.f);
    acc[i] = make_float2(0.f, 0.f);
  }
  const bool turns = ln.col0 < a.rot;   // (past rot a column passes through)
  const int groups = set.ctas * (kNrThreads / L::LPR), tokens = a.B * a.T;
  const uint32_t items = (uint32_t)tokens * set.chunks;
  const uint32_t group = (blockIdx.x - set.first_cta) * (kNrThreads / L::LPR) + threadIdx.x / L::LPR;

  // An item is kNrBwdHeads heads of a token.  The next item's rows come into the
  // warp's own part of shared memory while it works on the current one (loading
  // two rows at a time into registers left 24 warps waiting: 231 against 177 us
  // for 910 MB).
  struct Item {
    const T* x;
    const T* dy;
    T* dx;
    int heads, pos;      // rows to write; position, or -1
  };
  // The group's items are `groups` tokens apart, chunk after chunk; stepping
  // through long rows needs no division.
  int chunk = items > 0 ? 0 : set.chunks, b = 0;
  uint32_t t = group;
  auto settle = [&] {
    if (t >= (uint32_t)a.T) {
      t -= a.T;
      ++b;
      if (t >= (uint32_t)a.T) {
        b += t / a.T;
        t %= a.T;
      }
    }
    if (b >= a.B) {
      b -= a.B;
      ++chunk;
      if (b >= a.B) {
        chunk += b / a.B;
        b %= a.B;
      }
    }
  };
  if (items > 0) settle();
  auto here = [&] {
    Item it;
    const bool in = chunk < set.chunks;
    const int h0 = in ? chunk * kNrBwdHeads : 0, bb = in ? b : 0, tt = in ? (int)t : 0;
    it.pos = in ? nr_position(a, bb, tt) : -1;
    it.x = static_cast<const T*>(set.x) + bb * set.xs[0] + tt * set.xs[1] + h0 * set.xs[2];
    it.dy = static_cast<const T*>(set.dy) + bb * set.ds[0] + tt * set.ds[1] + h0 * set.ds[2];
    it.dx = static_cast<T*>(set.y) + bb * set.ys[0] + tt * set.ys[1] + h0 * set.ys[2];
    it.heads = in ? min(kNrBwdHeads, set.heads - h0) : 0;   // (padding rows of a token read nothing and write zeros)
    return it;
  };
  // [2][kNrBwdHeads][x, dy][group]: rows as they are in memory
  extern __shared__ __align__(16) uint8_t nr_smem[];
  const int lane_row = (threadIdx.x & 31) % L::LPR;
  auto slot = [&](int buf, int j, int which) {
    return nr_smem + ((buf * kNrBwdHeads + j) * 2 + which) * (kNrThreads * 16) + (threadIdx.x / L::LPR) * (L::LPR * 16);
  };
  auto fetch = [&](const Item& it, int buf) {
    const T* x = it.x + lane_row * L::E;
    const T* dy = it.dy + lane_row * L::E;
    const int reads = it.pos >= 0 ? it.heads : 0;
#pragma unroll
    for (int j = 0; j < kNrBwdHeads; ++j) {   // (nothing is read where the size is 0)
      copy_row(smem_u32(slot(buf, j, 0) + lane_row * 16), x, j < reads && a.norm);
      copy_row(smem_u32(slot(buf, j, 1) + lane_row * 16), dy, j < reads);
      x += set.xs[2];
      dy += set.ds[2];
    }
  };
  auto take = [&](int buf, int j, int which) {
    const T* row = reinterpret_cast<const T*>(slot(buf, j, which));
    const uint2 v0 = *reinterpret_cast<const uint2*>(row + ln.col0), v1 = *reinterpret_cast<const uint2*>(row + ln.col1);
    return make_uint4(v0.x, v0.y, v1.x, v1.y);
  };
  Item next = here();
  fetch(next, 0);
  asm volatile("cp.async.commit_group;" ::: "memory");
  int buf = 0;
  // Every lane of a warp makes the same number of rounds: the sums' shuffles need all of them.
  for (uint32_t base = 0; base < items; base += groups, buf ^= 1) {
    const Item it = next;
    __syncwarp();   // every lane has read the slots that are filled next
    if (base + groups < items) {
      t += groups;
      settle();
      next = here();
      fetch(next, buf ^ 1);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    Turn<P, kInter> tn;
    load_turn<P, kInter>(a, max(it.pos, 0), it.pos >= 0 ? ln.col0 : D, tn);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kNrBwdHeads; ++j) {
      float2 f[P], e[P], d[P], g[P];
      RowVec<T>::unpack(take(buf, j, 0), f);
      RowVec<T>::unpack(take(buf, j, 1), e);
      float2 ss = make_float2(0.f, 0.f), gx = ss;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        // dn: the transposed rotation
        const float2 sn = tn.s[i % tn.N];
        d[i] = turns ? fma2(e[i], tn.c[i % tn.N],
                            mul2(L::partner(e, i), kInter ? make_float2(sn.x, -sn.y) : i < L::H ? sn : neg2(sn)))
                     : e[i];
        g[i] = mul2(d[i], w[i]);
        const float2 fd = mul2(f[i], make_float2(1.f / D, 1.f / D));
        ss = fma2(fd, f[i], ss);
        gx = fma2(g[i], fd, gx);
      }
      if (a.norm) {
        const float r = rsqrtf(row_sum<L::LPR>(ss.x + ss.y) + a.eps);
        const float k = -r * r * row_sum<L::LPR>(gx.x + gx.y);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          g[i] = mul2(fma2(f[i], make_float2(k, k), g[i]), make_float2(r, r));
          acc[i] = fma2(d[i], mul2(f[i], make_float2(r, r)), acc[i]);
        }
      }
      if (j < it.heads) ln.store(it.dx + j * set.ys[2], g, it.pos < 0);   // (a weight may not be finite)
    }
  }
  if (set.dw == nullptr) return;
  float (*part)[D] = reinterpret_cast<float (*)[D]>(nr_smem);   // [kNrThreads / LPR][D]
  static_assert(kNrThreads / L::LPR * D * 4 <= kNrBwdSmem, "the groups' sums fit");
  __syncthreads();   // (each thread has read its own vectors)
#pragma unroll
  for (int i = 0; i < P; ++i)
    *reinterpret_cast<float2*>(&part[threadIdx.x / L::LPR][(i < L::H ? ln.col0 : ln.col1) + 2 * (i % L::H)]) = acc[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < kNrThreads / L::LPR; ++g) sum += part[g][threadIdx.x];
    a.partial[(size_t)blockIdx.x * D + threadIdx.x] = sum;
  }
}

// dw of set blockIdx.x: the sum of its CTAs' partial rows, in a fixed order.
template <int D>
__global__ void __launch_bounds__(kNrDwThreads) norm_rope_dw_kernel(const NormRopeArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const NormRopeSet& set = a.set[blockIdx.x];
  float* dw = set.dw;
  if (dw == nullptr) return;
  constexpr int kWays = kNrDwThreads / D;
  __shared__ float part[kWays][D];
  const int d = threadIdx.x % D, way = threadIdx.x / D;
  const float* p = a.partial + (size_t)set.first_cta * D + d;
  const int n = set.ctas;
  float sum = 0.f;
#pragma unroll 8
  for (int i = way; i < n; i += kWays) sum += p[(size_t)i * D];
  part[way][d] = sum;
  __syncthreads();
  if (way == 0) {
#pragma unroll
    for (int k = 1; k < kWays; ++k) sum += part[k][d];
    dw[d] = sum;
  }
}

}  // namespace plx
