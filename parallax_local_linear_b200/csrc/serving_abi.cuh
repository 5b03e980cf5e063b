// C entry points of the operators around attention: page plan, head norm with
// rotation, cache append and gather, and the 4-bit decode.  Included by
// parallax.cu after its host helpers.
#pragma once

#include <atomic>

namespace {

using namespace plx;

// Raises a kernel's dynamic shared-memory limit to `bytes`, once per device
// (every call of the kernel asks for as much: 2 us of host time otherwise).
template <auto kKernel>
cudaError_t set_smem_once(int bytes) {
  static std::atomic<bool> done[kMaxDevices];
  int dev = 0;
  if (note(cudaGetDevice(&dev)) != cudaSuccess) return cudaErrorInvalidDevice;
  if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = set_smem(kKernel, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
  return e;
}

// -------------------------------------------------------------- page plan
plx_status validate_page_plan(const plx_page_plan_params* p) {
  if (p == nullptr) return PLX_ERR_INVALID_ARG;
  if (p->batch < 1 || p->num_rows < 0 || p->num_pages < 1 || p->max_pages_per_seq < 1 || p->num_free < 0)
    return PLX_ERR_INVALID_ARG;
  if (p->page_size != kPage || p->batch > kPlanMaxBatch) return PLX_ERR_UNSUPPORTED;
  if ((int64_t)p->max_pages_per_seq * kPage >= (int64_t)INT32_MAX) return PLX_ERR_UNSUPPORTED;
  return PLX_OK;
}

// ------------------------------------------------------- norm and rotation
bool strides_ok(const int64_t* s, int n, int elt) {
  for (int i = 0; i < n; ++i)
    if (s[i] % (16 / elt) != 0) return false;
  return true;
}

// Rows that are written have places of their own: no stride of 0 over several.
bool distinct(const int64_t* s, const int64_t* count, int n) {
  for (int i = 0; i < n; ++i)
    if (s[i] == 0 && count[i] > 1) return false;
  return true;
}

// Strided runs of bytes: at base + sum k_i stride_i, k_i < count_i, `run` bytes
// each, all within lo .. hi - 1.
using Wide = __int128;   // (strides are the caller's)
struct Runs {
  const void* base;
  Wide stride[3];
  int64_t count[3], run;
  Wide lo, hi;
};

Runs head_runs(const void* base, const int64_t* stride, const int64_t* count, int d, int elt) {
  Runs r{base, {}, {}, (int64_t)d * elt, (Wide)reinterpret_cast<uintptr_t>(base), 0};
  r.hi = r.lo + r.run;
  for (int i = 0; i < 3; ++i) {
    r.stride[i] = (Wide)stride[i] * elt;
    r.count[i] = count[i];
    const Wide last = r.stride[i] * (count[i] - 1);
    (last < 0 ? r.lo : r.hi) += last;
  }
  return r;
}
Runs flat_run(const void* base, int64_t bytes) {
  const Wide at = (Wide)reinterpret_cast<uintptr_t>(base);
  return {base, {0, 0, 0}, {1, 1, 1}, bytes, at, at + bytes};
}
bool same_runs(const Runs& a, const Runs& b) {
  bool same = a.base == b.base && a.run == b.run;
  for (int i = 0; i < 3; ++i) same = same && a.count[i] == b.count[i] && (a.stride[i] == b.stride[i] || a.count[i] == 1);
  return same;
}

// Do runs of a and b share a byte?  Exact, so that slices of one fused
// projection, which lie in each other's gaps, do not count: is there a difference
// of places sum k_i stride_i + (a - b) within (-a.run, b.run)?  Dimensions are
// taken from the largest stride down; what the smaller ones can still add leaves
// one or two k for each (where strides lie so that there are many, the answer
// after kMaxSteps is yes).
bool runs_overlap(const Runs& a, const Runs& b) {
  if (a.hi <= b.lo || b.hi <= a.lo) return false;
  struct Dim {
    Wide stride, lo, hi;   // k in lo .. hi
  };
  if (a.base == nullptr || b.base == nullptr || a.run <= 0 || b.run <= 0) return false;
  Dim dim[6];
  int n = 0;
  auto put = [&](Wide stride, Wide lo, Wide hi) {
    if (stride == 0 || lo == hi) return;
    if (stride < 0) {
      stride = -stride;
      const Wide t = lo;
      lo = -hi;
      hi = -t;
    }
    int at = 0;
    while (at < n && dim[at].stride > stride) ++at;
    if (at < n && dim[at].stride == stride) {
      dim[at].lo += lo;
      dim[at].hi += hi;
      return;
    }
    for (int i = n++; i > at; --i) dim[i] = dim[i - 1];
    dim[at] = {stride, lo, hi};
  };
  for (int i = 0; i < 3; ++i) {
    if (a.count[i] <= 0 || b.count[i] <= 0) return false;
    put(a.stride[i], 0, a.count[i] - 1);
    put(b.stride[i], -(b.count[i] - 1), 0);
  }
  constexpr int kMaxSteps = 4096;
  int steps = 0;
  auto meet = [&](auto&& self, int i, Wide delta) -> bool {
    Wide lo = 0, hi = 0;   // what dimensions i and on can add
    for (int k = i; k < n; ++k) {
      lo += dim[k].lo * dim[k].stride;
      hi += dim[k].hi * dim[k].stride;
    }
    if (delta + hi <= -a.run || delta + lo >= b.run) return false;
    if (i == n || ++steps > kMaxSteps) return true;
    const Wide s = dim[i].stride, rest_lo = lo - dim[i].lo * s, rest_hi = hi - dim[i].hi * s;
    // k s in (-a.run - delta - rest_hi, b.run - delta - rest_lo)
    Wide k = (-a.run - delta - rest_hi) / s - 1, end = (b.run - delta - rest_lo) / s + 1;
    if (k < dim[i].lo) k = dim[i].lo;
    if (end > dim[i].hi) end = dim[i].hi;
    for (; k <= end; ++k)
      if (self(self, i + 1, delta + k * s)) return true;
    return false;
  };
  return meet(meet, 0, (Wide)reinterpret_cast<uintptr_t>(a.base) - (Wide)reinterpret_cast<uintptr_t>(b.base));
}

// Outputs of a norm + rotation call lie apart from each other and from what it
// reads; one may be its own set's rows, place by place.
bool norm_rope_apart(const plx_head_rows* rows, const plx_head_grads* grads, int32_t num_sets, const float* cos,
                     const float* sin, const int32_t* positions, const plx_norm_rope_params* p) {
  const int elt = p->dtype == PLX_BF16 ? 2 : 4, d = p->head_dim;
  if (p->tokens == 0) return true;
  Runs in[2 * kNrMaxSets], out[2 * kNrMaxSets], flat[kNrMaxSets + 3];
  int n_in = 0, n_out = 0, n_flat = 0;
  for (int i = 0; i < num_sets; ++i) {
    const int64_t count[3] = {p->batch, p->tokens, rows[i].heads};
    out[n_out++] = grads ? head_runs(grads[i].dx, grads[i].dx_stride, count, d, elt)
                         : head_runs(rows[i].y, rows[i].y_stride, count, d, elt);
    if (!grads || p->norm) in[n_in++] = head_runs(rows[i].x, rows[i].x_stride, count, d, elt);
    if (grads) in[n_in++] = head_runs(grads[i].dy, grads[i].dy_stride, count, d, elt);
    if (rows[i].w) flat[n_flat++] = flat_run(rows[i].w, (int64_t)d * elt);
  }
  const int rows_out = n_out;
  const int per_set = n_in / num_sets;
  if (grads)
    for (int i = 0; i < num_sets; ++i)
      if (grads[i].dw) out[n_out++] = flat_run(grads[i].dw, (int64_t)d * 4);
  if (p->rot_dim > 0) {
    flat[n_flat++] = flat_run(cos, (int64_t)p->max_pos * p->rot_dim * 2);
    flat[n_flat++] = flat_run(sin, (int64_t)p->max_pos * p->rot_dim * 2);
  }
  if (positions) flat[n_flat++] = flat_run(positions, 4 * (p->pos_batch_stride * (p->batch - 1) + p->tokens));
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (!(i < rows_out && j / per_set == i && same_runs(out[i], in[j])) && runs_overlap(out[i], in[j])) return false;
    for (int j = 0; j < n_flat; ++j)
      if (runs_overlap(out[i], flat[j])) return false;
    for (int j = 0; j < i; ++j)
      if (runs_overlap(out[i], out[j])) return false;
  }
  return true;
}

plx_status validate_norm_rope(const plx_head_rows* rows, const plx_head_grads* grads, int32_t num_sets,
                              const float* cos, const float* sin, const int32_t* positions,
                              const plx_norm_rope_params* p) {
  if (p == nullptr || rows == nullptr || num_sets < 1 || num_sets > kNrMaxSets) return PLX_ERR_INVALID_ARG;
  if (p->batch < 1 || p->tokens < 0 || p->rot_dim < 0 || p->max_pos < 0) return PLX_ERR_INVALID_ARG;
  if (p->dtype != PLX_F32 && p->dtype != PLX_BF16) return PLX_ERR_INVALID_ARG;
  if ((p->interleaved != 0 && p->interleaved != 1) || (p->norm != 0 && p->norm != 1)) return PLX_ERR_INVALID_ARG;
  if (p->norm && !(std::isfinite(p->eps) && p->eps > 0.f)) return PLX_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return PLX_ERR_UNSUPPORTED;
  if (p->rot_dim > p->head_dim || p->rot_dim % 16 != 0) return PLX_ERR_INVALID_ARG;
  if (p->rot_dim > 0) {
    if (cos == nullptr || sin == nullptr || !aligned(cos, 16) || !aligned(sin, 16) || p->max_pos < 1)
      return PLX_ERR_INVALID_ARG;
    if (positions == nullptr && p->tokens > p->max_pos) return PLX_ERR_INVALID_ARG;
  }
  if (positions && (!aligned(positions, 4) || p->pos_batch_stride < 0)) return PLX_ERR_INVALID_ARG;
  const int elt = p->dtype == PLX_BF16 ? 2 : 4;
  for (int i = 0; i < num_sets; ++i) {
    const plx_head_rows& r = rows[i];
    if (r.heads < 1) return PLX_ERR_INVALID_ARG;
    // a set's rows and the grid's threads are counted in 32 bits; blockIdx.y has 16
    if ((int64_t)r.heads * p->batch * p->tokens >= (int64_t)INT32_MAX || r.heads > 16384) return PLX_ERR_UNSUPPORTED;
    if ((int64_t)p->batch * p->tokens >= (int64_t)INT32_MAX / 32) return PLX_ERR_UNSUPPORTED;
    if (r.w && (!p->norm || !aligned(r.w, 16))) return PLX_ERR_INVALID_ARG;
    const bool any = p->tokens > 0;   // (an empty tensor has no address)
    if (!aligned(r.x, 16) || !strides_ok(r.x_stride, 3, elt)) return PLX_ERR_INVALID_ARG;
    const int64_t count[3] = {p->batch, p->tokens, r.heads};
    if (any && !distinct(grads ? grads[i].dx_stride : r.y_stride, count, 3)) return PLX_ERR_INVALID_ARG;
    if (grads == nullptr) {
      if ((any && (!r.x || !r.y)) || !aligned(r.y, 16) || !strides_ok(r.y_stride, 3, elt)) return PLX_ERR_INVALID_ARG;
    } else {
      const plx_head_grads& g = grads[i];
      if (any && ((!r.x && p->norm) || !g.dy || !g.dx)) return PLX_ERR_INVALID_ARG;
      if (!aligned(g.dy, 16) || !aligned(g.dx, 16)) return PLX_ERR_INVALID_ARG;
      if (!strides_ok(g.dy_stride, 3, elt) || !strides_ok(g.dx_stride, 3, elt)) return PLX_ERR_INVALID_ARG;
      if (g.dw && (!p->norm || !aligned(g.dw, 4))) return PLX_ERR_INVALID_ARG;
    }
  }
  return norm_rope_apart(rows, grads, num_sets, cos, sin, positions, p) ? PLX_OK : PLX_ERR_INVALID_ARG;
}

// The backward's grid: one CTA per set at least.
int norm_rope_bwd_ctas(int num_sms, int num_sets) {
  const int n = num_sms * kNrBwdCtasPerSm;
  return n < num_sets ? num_sets : n;
}

// Shares it out by the sets' numbers of heads (a set's rows are its work).
void norm_rope_bwd_shares(NormRopeArgs* a, int ctas) {
  long long heads = 0, before = 0;
  for (int i = 0; i < a->sets; ++i) heads += a->set[i].heads;
  int at = 0;
  for (int i = 0; i < a->sets; ++i) {
    before += a->set[i].heads;
    int end = (int)(before * ctas / heads);
    if (end < at + 1) end = at + 1;                                   // at least one for this set
    if (end > ctas - (a->sets - 1 - i)) end = ctas - (a->sets - 1 - i);   // and for each after it
    a->set[i].first_cta = at;
    a->set[i].ctas = end - at;
    at = end;
  }
}

NormRopeArgs norm_rope_args(const plx_head_rows* rows, int32_t num_sets, const int32_t* positions, const float* cos,
                            const float* sin, const plx_norm_rope_params* p, int hpg) {
  NormRopeArgs a{};
  a.positions = positions;
  a.cos = cos;
  a.sin = sin;
  a.pos_batch_stride = p->pos_batch_stride;
  a.sets = num_sets;
  a.B = p->batch;
  a.T = p->tokens;
  a.rot = p->rot_dim;
  a.max_pos = p->max_pos;
  a.norm = p->norm;
  a.eps = p->eps;
  a.hpg = hpg;
  for (int i = 0; i < num_sets; ++i) {
    NormRopeSet& s = a.set[i];
    s.x = rows[i].x;
    s.y = rows[i].y;
    s.w = rows[i].w;
    s.heads = rows[i].heads;
    s.chunks = (rows[i].heads + hpg - 1) / hpg;
    for (int k = 0; k < 3; ++k) {
      s.xs[k] = rows[i].x_stride[k];
      s.ys[k] = rows[i].y_stride[k];
    }
  }
  return a;
}

template <typename T, int D, bool kInter>
plx_status launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  constexpr int per_cta = kNrFwdThreads / NrLane<T, D, kInter>::LPR;
  long long chunks = 0;
  for (int i = 0; i < a.sets; ++i) chunks += a.set[i].chunks;
  const long long tokens = (long long)a.B * a.T;
  return launch_pdl(norm_rope_kernel<T, D, kInter>, dim3((unsigned)((tokens + per_cta - 1) / per_cta), (unsigned)chunks),
                    dim3(kNrFwdThreads), 0, stream, a) == cudaSuccess
             ? PLX_OK
             : PLX_ERR_CUDA;
}

template <typename T, int D, bool kInter>
plx_status launch_norm_rope_bwd(const NormRopeArgs& a, int ctas, bool dw, cudaStream_t stream) {
  if (set_smem_once<norm_rope_bwd_kernel<T, D, kInter>>(kNrBwdSmem) != cudaSuccess ||
      launch_pdl(norm_rope_bwd_kernel<T, D, kInter>, dim3(ctas), dim3(kNrThreads), kNrBwdSmem, stream, a) != cudaSuccess)
    return PLX_ERR_CUDA;
  if (!dw) return PLX_OK;
  return launch_pdl(norm_rope_dw_kernel<D>, dim3(a.sets), dim3(kNrDwThreads), 0, stream, a) == cudaSuccess ? PLX_OK
                                                                                                       : PLX_ERR_CUDA;
}

// Heads that a group of lanes takes for one token: enough to have its cos and
// sin once for several rows, few enough that every SM has groups.
int norm_rope_heads_per_group(const plx_head_rows* rows, int32_t num_sets, const plx_norm_rope_params* p) {
  const int lanes = p->head_dim * (p->dtype == PLX_BF16 ? 2 : 4) / 16;
  long long heads = 0;
  for (int i = 0; i < num_sets; ++i) heads += rows[i].heads;
  const int sms = current_device_sms();
  const long long fill = (long long)(sms > 0 ? sms : 148) * 16 * kNrFwdThreads / lanes;   // 16 of the 20 CTAs that an SM holds
  // 4 x 8192 tokens of 3 x 16 heads (810 MB): 134.1 us; 137.1 with 8, 147.0 with 4, 205.7 with 2.  4 x 512 tokens: 13.7,
  // 13.7, 12.5, 15.5.
  int hpg = 16;
  while (hpg > 1 && (long long)p->batch * p->tokens * heads / hpg < fill) hpg /= 2;
  return hpg;
}

// ------------------------------------------------------------ cache append
plx_status validate_append(const plx_append_params* p) {
  if (p == nullptr) return PLX_ERR_INVALID_ARG;
  if (p->num_rows < 0 || p->num_kv_heads < 1 || p->num_pages < 1) return PLX_ERR_INVALID_ARG;
  if (p->dtype != PLX_F32 && p->dtype != PLX_BF16) return PLX_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return PLX_ERR_UNSUPPORTED;
  if (p->page_size != kQ4Page) return PLX_ERR_UNSUPPORTED;
  if (p->num_rows >= INT32_MAX / 32 || p->num_kv_heads > 65535) return PLX_ERR_UNSUPPORTED;   // the grid's limits
  const int elt = p->dtype == PLX_BF16 ? 2 : 4;
  if (!strides_ok(p->k_stride, 2, elt) || !strides_ok(p->v_stride, 2, elt)) return PLX_ERR_INVALID_ARG;
  return PLX_OK;
}

// Two pools, or two results of a gather, apart from each other and from the slots
// (and results from the cache).
bool rows_apart(const Runs& k, const Runs& v, const int64_t* slots, const plx_append_params* p,
                const Runs& cache = flat_run(nullptr, 0)) {
  const Runs s = flat_run(slots, 8 * (int64_t)p->num_rows);
  return !runs_overlap(k, v) && !runs_overlap(k, s) && !runs_overlap(v, s) && !runs_overlap(k, cache) &&
         !runs_overlap(v, cache);
}
int64_t pool_bytes(const plx_append_params* p, int64_t block) { return (int64_t)p->num_pages * p->num_kv_heads * block; }

AppendArgs append_args(const int64_t* slots, const plx_append_params* p) {
  AppendArgs a{};
  a.slots = slots;
  a.N = p->num_rows;
  a.Hkv = p->num_kv_heads;
  a.num_pages = p->num_pages;
  const int vec = p->dtype == PLX_BF16 ? 8 : 4;   // elements of a 16-byte vector
  for (int i = 0; i < 2; ++i) {
    a.ks[i] = p->k_stride[i] / vec;
    a.vs[i] = p->v_stride[i] / vec;
  }
  return a;
}

// `lanes` threads for `rows` rows of one KV head (blockIdx.y).
template <typename Kernel>
plx_status launch_rows(Kernel kern, const AppendArgs& a, int lanes, cudaStream_t stream, int rows = 1) {
  const int per_cta = kAppendThreads / lanes * rows;
  const dim3 grid((unsigned)((a.N + per_cta - 1) / per_cta), (unsigned)a.Hkv);
  return launch_pdl(kern, grid, dim3(kAppendThreads), 0, stream, a) == cudaSuccess ? PLX_OK : PLX_ERR_CUDA;
}

// -------------------------------------------------------------- 4-bit decode
plx_status validate_decode_q4(const plx_decode_params* p) {
  plx_status st = validate_decode(p);
  if (st != PLX_OK) return st;
  if (p->in_dtype != PLX_BF16) return PLX_ERR_UNSUPPORTED;
  return PLX_OK;
}

// A default grid gives every CTA at least this many pages.
constexpr int kQ4MinPages = 4;
// The kernel counts its warps (12 a CTA) in 16 bits.
constexpr int kQ4MaxCtas = 4096;

struct DecodeQ4Plan {
  int ctas;
  size_t counter_bytes, slot_bytes;
};

DecodeQ4Plan plan_decode_q4(const plx_decode_params* p, int num_sms) {
  DecodeQ4Plan pl{};
  const int64_t units = (int64_t)p->batch * p->num_kv_heads;
  const int64_t pages = units * ((p->kv_len + kQ4Page - 1) / kQ4Page);
  const int64_t least = p->num_ctas > 0 ? 1 : kQ4MinPages;
  int64_t ctas = p->num_ctas > 0 ? p->num_ctas : num_sms;
  if (ctas > (pages + least - 1) / least) ctas = (pages + least - 1) / least;
  if (ctas < 1) ctas = 1;
  if (ctas > kQ4MaxCtas) ctas = kQ4MaxCtas;
  pl.ctas = (int)ctas;
  pl.counter_bytes = ((size_t)units * 4 + 255) & ~size_t(255);
  pl.slot_bytes = ((size_t)2 * pl.ctas * (p->num_q_heads / p->num_kv_heads) * (2 * p->head_dim + 4) * 4 + 255) &
                  ~size_t(255);
  return pl;
}

template <int D, int NT>
cudaError_t launch_decode_q4(const DecodeQ4Args& a, int ctas, cudaStream_t stream) {
  const cudaError_t e = set_smem_once<decode_q4_kernel<D, NT>>(Q4Smem<D, NT>::kBytes);
  return e != cudaSuccess ? e : launch_pdl(decode_q4_kernel<D, NT>, dim3(ctas), dim3(Q4Smem<D, NT>::kThreads),
                                               Q4Smem<D, NT>::kBytes, stream, a);
}

}  // namespace

extern "C" {

plx_status parallax_page_plan(const int32_t* cached_lens, const int32_t* new_lens, int32_t* page_table,
                              const int32_t* free_pages, const int32_t* free_head, int32_t* seq_lens,
                              int32_t* cu_seqlens, int64_t* slot_map, int32_t* positions, int32_t* pages_used,
                              const plx_page_plan_params* p, cudaStream_t stream) {
  plx_status st = validate_page_plan(p);
  if (st != PLX_OK) return st;
  if (!cached_lens || !new_lens || !page_table || !seq_lens || !cu_seqlens || !pages_used) return PLX_ERR_INVALID_ARG;
  if (p->num_free > 0 && !free_pages) return PLX_ERR_INVALID_ARG;
  if (p->num_rows > 0 && (!slot_map || !positions)) return PLX_ERR_INVALID_ARG;
  const size_t B = p->batch, R = p->num_rows;
  struct Range {
    const void* p;
    size_t n, align;
  };
  const Range in[] = {{cached_lens, 4 * B, 4}, {new_lens, 4 * B, 4}, {free_pages, 4 * (size_t)p->num_free, 4},
                      {free_head, (size_t)(free_head ? 4 : 0), 4}};
  const Range out[] = {{page_table, 4 * B * p->max_pages_per_seq, 4}, {seq_lens, 4 * B, 4}, {cu_seqlens, 4 * B + 4, 4},
                       {slot_map, 8 * R, 8}, {positions, 4 * R, 4}, {pages_used, 4, 4}};
  for (const Range& o : out) {
    if (!aligned(o.p, o.align)) return PLX_ERR_INVALID_ARG;
    for (const Range& i : in)
      if (i.n > 0 && o.n > 0 && overlaps(o.p, o.n, i.p, i.n)) return PLX_ERR_INVALID_ARG;
    for (const Range& q : out)
      if (&q != &o && q.n > 0 && o.n > 0 && overlaps(o.p, o.n, q.p, q.n)) return PLX_ERR_INVALID_ARG;
  }
  for (const Range& i : in)
    if (!aligned(i.p, i.align)) return PLX_ERR_INVALID_ARG;
  const int num_sms = current_device_sms();
  if (num_sms <= 0) return PLX_ERR_CUDA;
  PagePlanArgs a{};
  a.cached = cached_lens;
  a.fresh = new_lens;
  a.table = page_table;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.seq_lens = seq_lens;
  a.cu = cu_seqlens;
  a.slots = slot_map;
  a.positions = positions;
  a.used = pages_used;
  a.B = p->batch;
  a.rows = p->num_rows;
  a.num_pages = p->num_pages;
  a.max_pages = p->max_pages_per_seq;
  a.num_free = p->num_free;
  // one CTA per two rows a thread, and one per 64 requests (a warp takes four)
  const int64_t by_rows = ((int64_t)p->num_rows + 2 * kPlanThreads - 1) / (2 * kPlanThreads);
  const int64_t by_requests = ((int64_t)p->batch + 63) / 64;
  int64_t ctas = by_rows > by_requests ? by_rows : by_requests;
  if (ctas > num_sms) ctas = num_sms;
  const int smem = plan_smem_bytes(a.B);
  if (smem > 48 * 1024 && set_smem_once<page_plan_kernel>(plan_smem_bytes(kPlanMaxBatch)) != cudaSuccess)
    return PLX_ERR_CUDA;
  return launch_pdl(page_plan_kernel, dim3((unsigned)ctas), dim3(kPlanThreads), smem, stream, a) == cudaSuccess
             ? PLX_OK
             : PLX_ERR_CUDA;
}

plx_status parallax_norm_rope(const plx_head_rows* rows, int32_t num_sets, const int32_t* positions,
                              const float* cos, const float* sin, const plx_norm_rope_params* p,
                              cudaStream_t stream) {
  plx_status st = validate_norm_rope(rows, nullptr, num_sets, cos, sin, positions, p);
  if (st != PLX_OK) return st;
  if (p->tokens == 0) return PLX_OK;
  const NormRopeArgs a = norm_rope_args(rows, num_sets, positions, cos, sin, p,
                                        norm_rope_heads_per_group(rows, num_sets, p));
  const bool il = p->interleaved != 0;
  if (p->dtype == PLX_BF16) {
    if (p->head_dim == 64)
      return il ? launch_norm_rope<__nv_bfloat16, 64, true>(a, stream)
                : launch_norm_rope<__nv_bfloat16, 64, false>(a, stream);
    return il ? launch_norm_rope<__nv_bfloat16, 128, true>(a, stream)
              : launch_norm_rope<__nv_bfloat16, 128, false>(a, stream);
  }
  if (p->head_dim == 64)
    return il ? launch_norm_rope<float, 64, true>(a, stream) : launch_norm_rope<float, 64, false>(a, stream);
  return il ? launch_norm_rope<float, 128, true>(a, stream) : launch_norm_rope<float, 128, false>(a, stream);
}

size_t parallax_norm_rope_backward_workspace_size(const plx_norm_rope_params* p, int32_t num_sets) {
  if (p == nullptr || num_sets < 1 || num_sets > kNrMaxSets) return (size_t)-1;
  if (p->head_dim != 64 && p->head_dim != 128) return (size_t)-1;
  const int num_sms = current_device_sms();
  if (num_sms <= 0) return (size_t)-1;
  return (size_t)norm_rope_bwd_ctas(num_sms, num_sets) * p->head_dim * sizeof(float);
}

plx_status parallax_norm_rope_backward(const plx_head_rows* rows, const plx_head_grads* grads, int32_t num_sets,
                                       const int32_t* positions, const float* cos, const float* sin,
                                       void* workspace, size_t workspace_bytes, const plx_norm_rope_params* p,
                                       cudaStream_t stream) {
  if (grads == nullptr) return PLX_ERR_INVALID_ARG;
  plx_status st = validate_norm_rope(rows, grads, num_sets, cos, sin, positions, p);
  if (st != PLX_OK) return st;
  bool dw = false;
  for (int i = 0; i < num_sets; ++i) dw = dw || grads[i].dw != nullptr;
  const int num_sms = current_device_sms();
  if (num_sms <= 0) return PLX_ERR_CUDA;
  const int ctas = norm_rope_bwd_ctas(num_sms, num_sets);
  if (dw && (workspace == nullptr || !aligned(workspace, 16) ||
             workspace_bytes < (size_t)ctas * p->head_dim * sizeof(float)))
    return PLX_ERR_WORKSPACE;
  NormRopeArgs a = norm_rope_args(rows, num_sets, positions, cos, sin, p, kNrBwdHeads);
  a.partial = static_cast<float*>(workspace);
  for (int i = 0; i < num_sets; ++i) {
    NormRopeSet& s = a.set[i];
    s.dy = grads[i].dy;
    s.y = grads[i].dx;
    s.dw = grads[i].dw;
    for (int k = 0; k < 3; ++k) {
      s.ds[k] = grads[i].dy_stride[k];
      s.ys[k] = grads[i].dx_stride[k];
    }
  }
  norm_rope_bwd_shares(&a, ctas);
  const bool il = p->interleaved != 0;
  if (p->dtype == PLX_BF16) {
    if (p->head_dim == 64)
      return il ? launch_norm_rope_bwd<__nv_bfloat16, 64, true>(a, ctas, dw, stream)
                : launch_norm_rope_bwd<__nv_bfloat16, 64, false>(a, ctas, dw, stream);
    return il ? launch_norm_rope_bwd<__nv_bfloat16, 128, true>(a, ctas, dw, stream)
              : launch_norm_rope_bwd<__nv_bfloat16, 128, false>(a, ctas, dw, stream);
  }
  if (p->head_dim == 64)
    return il ? launch_norm_rope_bwd<float, 64, true>(a, ctas, dw, stream)
              : launch_norm_rope_bwd<float, 64, false>(a, ctas, dw, stream);
  return il ? launch_norm_rope_bwd<float, 128, true>(a, ctas, dw, stream)
            : launch_norm_rope_bwd<float, 128, false>(a, ctas, dw, stream);
}

plx_status parallax_cache_append(const void* k, const void* v, const int64_t* slot_map, void* k_cache,
                                 void* v_cache, const plx_append_params* p, cudaStream_t stream) {
  plx_status st = validate_append(p);
  if (st != PLX_OK) return st;
  if (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return PLX_ERR_INVALID_ARG;
  if (p->num_rows == 0) return PLX_OK;
  if (!k || !v || !slot_map || !aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 8)) return PLX_ERR_INVALID_ARG;
  const int64_t block = (int64_t)kQ4Page * p->head_dim * (p->dtype == PLX_BF16 ? 2 : 4);
  if (!rows_apart(flat_run(k_cache, pool_bytes(p, block)), flat_run(v_cache, pool_bytes(p, block)), slot_map, p))
    return PLX_ERR_INVALID_ARG;
  AppendArgs a = append_args(slot_map, p);
  a.k = k;
  a.v = v;
  a.k_pool = k_cache;
  a.v_pool = v_cache;
  const int vpr = p->head_dim * (p->dtype == PLX_BF16 ? 2 : 4) / 16;
  if (vpr == 8) return launch_rows(cache_append_kernel<8>, a, 8, stream);
  if (vpr == 16) return launch_rows(cache_append_kernel<16>, a, 16, stream);
  return launch_rows(cache_append_kernel<32>, a, 32, stream);
}

size_t parallax_q4_block_bytes(int32_t head_dim) {
  return head_dim == 64 ? Q4Block<64>::kBytes : head_dim == 128 ? Q4Block<128>::kBytes : 0;
}

plx_status parallax_cache_append_q4(const void* k, const void* v, const int64_t* slot_map, void* kv_cache,
                                    const plx_append_params* p, cudaStream_t stream) {
  plx_status st = validate_append(p);
  if (st != PLX_OK) return st;
  if (p->dtype != PLX_BF16) return PLX_ERR_UNSUPPORTED;
  if (!kv_cache || !aligned(kv_cache, 16)) return PLX_ERR_INVALID_ARG;
  if (p->num_rows == 0) return PLX_OK;
  if (!k || !v || !slot_map || !aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 8)) return PLX_ERR_INVALID_ARG;
  AppendArgs a = append_args(slot_map, p);
  a.k = k;
  a.v = v;
  a.cache = static_cast<uint8_t*>(kv_cache);
  return p->head_dim == 64 ? launch_rows(cache_append_q4_kernel<64>, a, 8, stream)
                           : launch_rows(cache_append_q4_kernel<128>, a, 16, stream);
}

plx_status parallax_cache_gather_q4(const void* kv_cache, const int64_t* slot_map, void* k, void* v,
                                    const plx_append_params* p, cudaStream_t stream) {
  plx_status st = validate_append(p);
  if (st != PLX_OK) return st;
  if (!kv_cache || !aligned(kv_cache, 16)) return PLX_ERR_INVALID_ARG;
  if (p->num_rows == 0) return PLX_OK;
  if (!k || !v || !slot_map || !aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 8)) return PLX_ERR_INVALID_ARG;
  const int64_t count[2] = {p->num_rows, p->num_kv_heads};
  if (!distinct(p->k_stride, count, 2) || !distinct(p->v_stride, count, 2)) return PLX_ERR_INVALID_ARG;
  const int elt = p->dtype == PLX_BF16 ? 2 : 4;
  const int64_t rows[3] = {1, count[0], count[1]}, ks[3] = {0, p->k_stride[0], p->k_stride[1]},
                vs[3] = {0, p->v_stride[0], p->v_stride[1]};
  if (!rows_apart(head_runs(k, ks, rows, p->head_dim, elt), head_runs(v, vs, rows, p->head_dim, elt), slot_map, p,
                  flat_run(kv_cache, pool_bytes(p, parallax_q4_block_bytes(p->head_dim)))))
    return PLX_ERR_INVALID_ARG;
  AppendArgs a = append_args(slot_map, p);
  a.k_out = k;
  a.v_out = v;
  a.cache = const_cast<uint8_t*>(static_cast<const uint8_t*>(kv_cache));
  const int lanes = p->head_dim / 4;
  auto kern = p->head_dim == 64 ? (p->dtype == PLX_BF16 ? cache_gather_q4_kernel<64, true> : cache_gather_q4_kernel<64, false>)
                                : (p->dtype == PLX_BF16 ? cache_gather_q4_kernel<128, true>
                                                        : cache_gather_q4_kernel<128, false>);
  return launch_rows(kern, a, lanes, stream, kGatherRows);
}

size_t parallax_decode_q4_workspace_size(const plx_decode_params* p, int32_t num_sms) {
  if (validate_decode_q4(p) != PLX_OK) return (size_t)-1;
  if (num_sms <= 0) num_sms = current_device_sms();
  if (num_sms <= 0) return (size_t)-1;
  const DecodeQ4Plan pl = plan_decode_q4(p, num_sms);
  return pl.counter_bytes + pl.slot_bytes;
}

plx_status parallax_decode_q4(const void* q, const void* rho, const void* kv_cache, const int32_t* page_table,
                              const int32_t* seq_lens, void* out, void* workspace, size_t workspace_bytes,
                              const plx_decode_params* p, cudaStream_t stream) {
  plx_status st = validate_decode_q4(p);
  if (st != PLX_OK) return st;
  if (!q || !rho || !kv_cache || !out) return PLX_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(rho, 16) || !aligned(kv_cache, 16) || !aligned(out, 16)) return PLX_ERR_INVALID_ARG;
  const bool paged = p->page_size != 0;
  if (paged && (page_table == nullptr || seq_lens == nullptr)) return PLX_ERR_INVALID_ARG;
  if (!paged && page_table != nullptr) return PLX_ERR_INVALID_ARG;
  if ((page_table && !aligned(page_table, 4)) || (seq_lens && !aligned(seq_lens, 4))) return PLX_ERR_INVALID_ARG;
  // (a unit's queries and probes are read before its rows are written, by all that read them)
  const bool in_place = p->out_dtype == PLX_BF16;
  const size_t rows = (size_t)p->batch * p->num_q_heads * p->head_dim, n = rows * (in_place ? 2 : 4);
  const size_t pages = paged ? p->num_pages : (size_t)p->batch * ((p->kv_len + kQ4Page - 1) / kQ4Page);
  if ((!(in_place && out == q) && overlaps(out, n, q, 2 * rows)) ||
      (!(in_place && out == rho) && overlaps(out, n, rho, 2 * rows)) ||
      overlaps(out, n, kv_cache, pages * p->num_kv_heads * parallax_q4_block_bytes(p->head_dim)) ||
      (workspace && overlaps(out, n, workspace, workspace_bytes)) ||
      (page_table && overlaps(out, n, page_table, 4 * (size_t)p->batch * p->max_pages_per_seq)) ||
      (seq_lens && overlaps(out, n, seq_lens, 4 * (size_t)p->batch)))
    return PLX_ERR_INVALID_ARG;
  const int num_sms = current_device_sms();
  if (num_sms <= 0) return PLX_ERR_CUDA;
  const DecodeQ4Plan pl = plan_decode_q4(p, num_sms);
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes % 256 != 0 ||
      workspace_bytes < pl.counter_bytes + pl.slot_bytes)
    return PLX_ERR_WORKSPACE;
  if (p->kv_len == 0) {   // every sequence is empty: the output is zero
    return note(cudaMemsetAsync(out, 0, n, stream)) == cudaSuccess ? PLX_OK : PLX_ERR_CUDA;
  }
  DecodeQ4Args a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.rho = static_cast<const __nv_bfloat16*>(rho);
  a.cache = static_cast<const uint8_t*>(kv_cache);
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.B = p->batch;
  a.Hq = p->num_q_heads;
  a.Hkv = p->num_kv_heads;
  a.group = p->num_q_heads / p->num_kv_heads;
  a.kv_len = p->kv_len;
  a.num_pages = paged ? p->num_pages : 0;
  a.max_pages = paged ? p->max_pages_per_seq : 0;
  a.scale_log2 = p->scale * 1.4426950408889634f;
  a.out_bf16 = p->out_dtype == PLX_BF16 ? 1 : 0;
  a.slots = static_cast<float*>(workspace);
  a.counters = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + workspace_bytes - pl.counter_bytes);
  a.min_pages = p->num_ctas > 0 ? 1 : kQ4MinPages;
  const bool one = a.group <= 4;   // four heads fill the 8 columns of a product
  const cudaError_t e = p->head_dim == 64 ? (one ? launch_decode_q4<64, 1>(a, pl.ctas, stream)
                                                 : launch_decode_q4<64, 2>(a, pl.ctas, stream))
                                          : (one ? launch_decode_q4<128, 1>(a, pl.ctas, stream)
                                                 : launch_decode_q4<128, 2>(a, pl.ctas, stream));
  return e == cudaSuccess ? PLX_OK : PLX_ERR_CUDA;
}

}  // extern "C"
