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
// never leaves registers.  A lane's rotation partner holds the pair's other
// column (another lane of the row, or the lane itself when interleaved), and
// the lane forms only its own column of the pair: the partner's raw vector
// comes by four shuffles.  A group of lanes takes several heads of one token,
// so a token's cos and sin are read once for them.
#pragma once

#include "ptx.cuh"

namespace plx {

constexpr int kNrThreads = 256;
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
// first (rope_prefill 147 to 133 us).
__device__ __forceinline__ uint4 load_row(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");   // (y may be x itself)
  return v;
}
__device__ __forceinline__ void store_row(void* p, const uint4& v) {
  asm volatile("st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// 16 bytes into shared memory as they arrive; zeros where !read.
__device__ __forceinline__ void copy_row(uint32_t dst, const void* src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
               "r"(read ? 16 : 0)
               : "memory");
}

// A lane's share of a row: E values from one 16-byte vector, in pairs (the
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

// The lane's own columns of the rotation at one position:
//     y_e = n_e c[e] + partner(n)_e s[e].
// (c, s) is (cos, -sin) for the first column of a pair, (cos, sin) for the
// second and (1, 0) past rot.
template <int P>
struct Turn {
  float2 c[P], s[P];
};

template <int P, bool kInter>
__device__ __forceinline__ void load_turn(const NormRopeArgs& a, int pos, int col0, Turn<P>& t) {
  const int half = a.rot / 2;
  if (col0 >= a.rot) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      t.c[i] = make_float2(1.f, 1.f);
      t.s[i] = make_float2(0.f, 0.f);
    }
    return;
  }
  const size_t row = (size_t)pos * half;
  if (kInter) {
    const float* cp = a.cos + row + col0 / 2;
    const float* sp = a.sin + row + col0 / 2;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float c = __ldg(cp + i), s = __ldg(sp + i);
      t.c[i] = make_float2(c, c);
      t.s[i] = make_float2(-s, s);
    }
  } else {
    const bool second = col0 >= half;   // rot is a multiple of 16: a lane's columns lie in one half
    const int f0 = second ? col0 - half : col0;
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(a.cos + row + f0) + i);
      const float4 s = __ldg(reinterpret_cast<const float4*>(a.sin + row + f0) + i);
      t.c[2 * i] = make_float2(c.x, c.y);
      t.c[2 * i + 1] = make_float2(c.z, c.w);
      t.s[2 * i] = second ? make_float2(s.x, s.y) : make_float2(-s.x, -s.y);
      t.s[2 * i + 1] = second ? make_float2(s.z, s.w) : make_float2(-s.z, -s.w);
    }
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T, int D, bool kInter>
struct NrLane {
  static constexpr int E = RowVec<T>::E, P = E / 2, LPR = D / E, RPW = 32 / LPR;
  int col0, src;       // first column, lane of the rotation partner

  __device__ __forceinline__ explicit NrLane(const NormRopeArgs& a) {
    const int lane = threadIdx.x & 31, l = lane % LPR;
    col0 = l * E;
    const int shift = a.rot / 2 / E;
    src = col0 >= a.rot || kInter ? lane : (col0 < a.rot / 2 ? lane + shift : lane - shift);
  }
  // The partner columns of a vector of the lane's row.  Every lane takes part.
  __device__ __forceinline__ void partner(const uint4& v, float2 (&f)[P]) const {
    if (kInter) {   // the partner of column e is e ^ 1
      RowVec<T>::unpack(v, f);
#pragma unroll
      for (int i = 0; i < P; ++i) f[i] = make_float2(f[i].y, f[i].x);
    } else {
      RowVec<T>::unpack(make_uint4(__shfl_sync(0xffffffffu, v.x, src), __shfl_sync(0xffffffffu, v.y, src),
                                   __shfl_sync(0xffffffffu, v.z, src), __shfl_sync(0xffffffffu, v.w, src)),
                        f);
    }
  }
  __device__ __forceinline__ uint4 load_weights(const void* w) const {
    return w == nullptr ? make_uint4(0, 0, 0, 0)
                        : __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(w) + col0));
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
// heads) of one token; neighbouring groups take neighbouring tokens.
template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NormRopeArgs a) {
  using L = NrLane<T, D, kInter>;
  constexpr int P = L::P;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const L ln(a);
  int chunk = blockIdx.y, si = 0;
  while (chunk >= a.set[si].chunks) chunk -= a.set[si++].chunks;
  const NormRopeSet& set = a.set[si];
  const int tok = (int)((blockIdx.x * kNrThreads + threadIdx.x) / L::LPR);
  const int b = a.B == 1 ? 0 : tok / a.T, t = tok - b * a.T;
  const int h0 = chunk * a.hpg;
  const int pos = b < a.B && t < a.T ? nr_position(a, b, t) : -1;
  const bool live = pos >= 0;
  // y = r (x wc + partner(x) ws) with the weights taken into the rotation
  float2 wc[P], ws[P];
  {
    Turn<P> tn;
    load_turn<P, kInter>(a, live ? pos : 0, live ? ln.col0 : D, tn);
    const uint4 wv = ln.load_weights(set.w);
    float2 w[P], wp[P];
    RowVec<T>::unpack(wv, w);
    ln.partner(wv, wp);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      wc[i] = set.w == nullptr ? tn.c[i] : mul2(w[i], tn.c[i]);
      ws[i] = set.w == nullptr ? tn.s[i] : mul2(wp[i], tn.s[i]);
    }
  }
  const T* x = static_cast<const T*>(set.x) + b * set.xs[0] + t * set.xs[1] + h0 * set.xs[2] + ln.col0;
  T* y = static_cast<T*>(set.y) + b * set.ys[0] + t * set.ys[1] + h0 * set.ys[2] + ln.col0;
  const int heads = live ? min(a.hpg, set.heads - h0) : 0;
  constexpr int U = 4;   // rows in flight
  for (int j = 0; j < a.hpg; j += U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = make_uint4(0, 0, 0, 0);
      if (j + u < heads) v[u] = load_row(x + (j + u) * set.xs[2]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 f[P], p[P], o[P];
      RowVec<T>::unpack(v[u], f);
      ln.partner(v[u], p);
      float r = 1.f;
      if (a.norm) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) ss = fma2(mul2(f[i], make_float2(1.f / D, 1.f / D)), f[i], ss);   // (overflows only with the mean itself)
        r = rsqrtf(row_sum<L::LPR>(ss.x + ss.y) + a.eps);
      }
#pragma unroll
      for (int i = 0; i < P; ++i) o[i] = mul2(fma2(f[i], wc[i], mul2(p[i], ws[i])), make_float2(r, r));
      if (j + u < heads) store_row(y + (j + u) * set.ys[2], RowVec<T>::pack(o));
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
  RowVec<T>::unpack(ln.load_weights(set.w), w);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (set.w == nullptr) w[i] = make_float2(1.f, 1.f);
    acc[i] = make_float2(0.f, 0.f);
  }
  const uint32_t groups = set.ctas * (kNrThreads / L::LPR), tokens = a.B * a.T, items = tokens * set.chunks;
  const uint32_t group = (blockIdx.x - set.first_cta) * (kNrThreads / L::LPR) + threadIdx.x / L::LPR;

  // An item is kNrBwdHeads heads of a token.  The next item's vectors come into
  // this thread's own part of shared memory while it works on the current one
  // (loading two rows at a time into registers left 24 warps waiting: 268
  // against 231 us for rope_grad at its best chunk).
  struct Item {
    const T* x;
    const T* dy;
    T* dx;
    int heads, pos;      // rows to write; position, or -1
  };
  auto decode = [&](uint32_t item) {
    Item it;
    const bool in = item < items;
    const int chunk = in ? item / tokens : 0, tok = in ? item - chunk * tokens : 0;
    const int b = a.B == 1 ? 0 : tok / a.T, t = tok - b * a.T, h0 = chunk * kNrBwdHeads;
    it.pos = in ? nr_position(a, b, t) : -1;
    it.x = static_cast<const T*>(set.x) + b * set.xs[0] + t * set.xs[1] + h0 * set.xs[2] + ln.col0;
    it.dy = static_cast<const T*>(set.dy) + b * set.ds[0] + t * set.ds[1] + h0 * set.ds[2] + ln.col0;
    it.dx = static_cast<T*>(set.y) + b * set.ys[0] + t * set.ys[1] + h0 * set.ys[2] + ln.col0;
    it.heads = in ? min(kNrBwdHeads, set.heads - h0) : 0;   // (padding rows of a token read nothing and write zeros)
    return it;
  };
  extern __shared__ __align__(16) uint8_t nr_smem[];   // [2][kNrBwdHeads][x, dy][thread]
  auto slot = [&](int buf, int j, int which) {
    return nr_smem + (((buf * kNrBwdHeads + j) * 2 + which) * kNrThreads + threadIdx.x) * 16;
  };
  auto fetch = [&](const Item& it, int buf) {
#pragma unroll
    for (int j = 0; j < kNrBwdHeads; ++j) {
      const bool read = it.pos >= 0 && j < it.heads;
      copy_row(smem_u32(slot(buf, j, 0)), read && a.norm ? it.x + j * set.xs[2] : static_cast<const T*>(set.dy), read && a.norm);
      copy_row(smem_u32(slot(buf, j, 1)), read ? it.dy + j * set.ds[2] : static_cast<const T*>(set.dy), read);
    }
  };
  Item next = decode(group);
  fetch(next, 0);
  asm volatile("cp.async.commit_group;" ::: "memory");
  int buf = 0;
  // Every lane of a warp makes the same number of rounds: the sums' shuffles need all of them.
  for (uint32_t base = 0; base < items; base += groups, buf ^= 1) {
    const Item it = next;
    if (base + groups < items) {
      next = decode(base + groups + group);
      fetch(next, buf ^ 1);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    Turn<P> tn;
    load_turn<P, kInter>(a, max(it.pos, 0), it.pos >= 0 ? ln.col0 : D, tn);
#pragma unroll
    for (int i = 0; i < P; ++i) tn.s[i] = make_float2(-tn.s[i].x, -tn.s[i].y);   // the transposed rotation
    asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll
    for (int j = 0; j < kNrBwdHeads; ++j) {
      const uint4 vd = *reinterpret_cast<const uint4*>(slot(buf, j, 1));
      float2 f[P], d[P], p[P], g[P];
      RowVec<T>::unpack(*reinterpret_cast<const uint4*>(slot(buf, j, 0)), f);
      RowVec<T>::unpack(vd, d);
      ln.partner(vd, p);
      float2 ss = make_float2(0.f, 0.f), gx = ss;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        d[i] = fma2(d[i], tn.c[i], mul2(p[i], tn.s[i]));   // dn
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
      if (j < it.heads) store_row(it.dx + j * set.ys[2], RowVec<T>::pack(g));
    }
  }
  if (set.dw == nullptr) return;
  float (*part)[D] = reinterpret_cast<float (*)[D]>(nr_smem);   // [kNrThreads / LPR][D]
  static_assert(kNrThreads / L::LPR * D * 4 <= kNrBwdSmem, "the groups' sums fit");
  __syncthreads();   // (each thread has read its own vectors)
#pragma unroll
  for (int i = 0; i < P; ++i) *reinterpret_cast<float2*>(&part[threadIdx.x / L::LPR][ln.col0 + 2 * i]) = acc[i];
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
