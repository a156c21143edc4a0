// Per-adapter gradient norms over many tensors, clipping, and AdamW on the
// clipped gradient, on gfx950.
//
//   s_a = sum over adapter a's tensors of g^2,  norm_a = sqrt(s_a),
//   c_a = min(1, max_norm / (norm_a + 1e-6));   g <- c_a g, or one AdamW step on c_a g.
//
// Three launches: partial sums of one 8192-element chunk each (64-bit sums, so
// no square of a finite gradient overflows), one block a group that joins its
// chunks' sums in a fixed order and derives the group's factors, and the pass
// that uses them.  A group is skipped exactly when its sum is not finite, that
// is when any of its elements is NaN or +-Inf, so the norm's pass over g is also
// the scan that decides the skip.  Both passes are bound by HBM.  The chunks of
// one group are consecutive, since the table is sorted by group.
#include "common.hpp"
#include "sgmv.hpp"

namespace lora {

constexpr int GRAD_THREADS = 256;
constexpr int GRAD_CHUNK = LORA_GRAD_CHUNK;
static_assert(GRAD_CHUNK % (GRAD_THREADS * 4) == 0, "whole 16-byte rounds per chunk");

// A group's factors, written by the join and read by the pass that follows.
// c_a = coef 2^exp2: applied with ldexp it rounds as one fp32 product, and keeps its
// bits where c_a itself would be an fp32 subnormal (gradients near the fp32 range).
struct GradFactors {
  float coef;          // 0.5 2^1 for a skipped group
  int32_t exp2;
  float step_size;     // lr / (1 - beta1^step)
  float inv_sqrt_bc2;  // 1 / sqrt(1 - beta2^step)
  int32_t skip;
};

__device__ __forceinline__ float clipped(float g, const GradFactors& f) {
  return __builtin_amdgcn_ldexpf(g * f.coef, f.exp2);
}

// The part of a tensor that chunk `c` covers; count 0 if the table is not what
// it has to be there (flagged: the chunk is then read and written by nobody).
struct GradSpan {
  int64_t begin;
  int32_t count;
  int32_t group;
};

// Called by whole waves with a uniform c in [0, n_chunks).
__device__ __forceinline__ GradSpan grad_span(const grad_shape& sh, const grad_tensor* tab, int c,
                                              int32_t* status) {
  // the last tensor whose first_chunk is <= c
  const int lane = (int)(threadIdx.x & 63);
  int lo = 0, end = sh.n_tensors;
  while (end - lo > 1) {
    const int step = (end - lo + 63) / 64;
    const int j = lo + lane * step;
    const uint64_t m = __ballot(j < end && (j == lo || tab[j].first_chunk <= c));
    const int k = 63 - __clzll(m);   // lane 0 always votes
    lo += k * step;
    end = min(end, lo + step);
  }
  const grad_tensor t = tab[lo];
  const int64_t at = (int64_t)(c - t.first_chunk) * GRAD_CHUNK;
  const bool ok = t.first_chunk >= 0 && t.first_chunk <= c && t.offset >= 0 && t.count >= 0 &&
                  t.offset <= sh.n_elems && t.count <= sh.n_elems - t.offset && at < t.count &&
                  t.group >= 0 && t.group < sh.n_groups;
  if (!ok) {
    if (lane == 0) set_flag(status, LORA_FLAG_BAD_DESC);
    return GradSpan{0, 0, 0};
  }
  return GradSpan{t.offset + at, (int32_t)min((int64_t)GRAD_CHUNK, t.count - at), t.group};
}

// A chunk's sum of squares, read in 16-byte pieces where the span is 16-byte
// aligned and element by element elsewhere.
__global__ __launch_bounds__(GRAD_THREADS) void grad_partial_kernel(
    grad_shape sh, const grad_tensor* __restrict__ tab, const float* __restrict__ g,
    double* __restrict__ partial, int32_t* __restrict__ status) {
  __shared__ double red[GRAD_THREADS / kWave];
  const int c = blockIdx.x;
  const GradSpan sp = grad_span(sh, tab, c, status);
  const float* p = g + sp.begin;
  double s = 0.0;
  if (((uintptr_t)p & 15) == 0) {
    const int n4 = sp.count / 4;
    float4 v[GRAD_CHUNK / (GRAD_THREADS * 4)];
#pragma unroll
    for (int q = 0; q < GRAD_CHUNK / (GRAD_THREADS * 4); ++q) {
      const int i = q * GRAD_THREADS + threadIdx.x;
      v[q] = i < n4 ? ((const float4*)p)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int q = 0; q < GRAD_CHUNK / (GRAD_THREADS * 4); ++q)
      s += (double)v[q].x * v[q].x + (double)v[q].y * v[q].y + (double)v[q].z * v[q].z +
           (double)v[q].w * v[q].w;
    const int i = n4 * 4 + threadIdx.x;
    if (i < sp.count) s += (double)p[i] * p[i];
  } else {
    for (int i = threadIdx.x; i < sp.count; i += GRAD_THREADS) s += (double)p[i] * p[i];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, kWave);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) partial[c] = (red[0] + red[1]) + (red[2] + red[3]);
}

struct GradAdam {
  int64_t* steps;   // null: no optimizer step follows
  double lr, beta1, beta2;
};

// One block a group: its chunks' sums, the norm and the factors.
__global__ __launch_bounds__(GRAD_THREADS) void grad_join_kernel(
    grad_shape sh, const grad_tensor* __restrict__ tab, const double* __restrict__ partial,
    float max_norm, GradAdam ad, float* __restrict__ norms, GradFactors* __restrict__ out,
    int32_t* __restrict__ status) {
  __shared__ double red[GRAD_THREADS / kWave];
  const int a = blockIdx.x;
  // first tensors of groups a and a + 1
  int lim[2];
  for (int k = 0; k < 2; ++k) {
    int lo = 0, hi = sh.n_tensors;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (tab[mid].group < a + k) lo = mid + 1; else hi = mid;
    }
    lim[k] = lo;
  }
  int c0 = lim[0] < sh.n_tensors ? tab[lim[0]].first_chunk : sh.n_chunks;
  int c1 = lim[1] < sh.n_tensors ? tab[lim[1]].first_chunk : sh.n_chunks;
  c0 = max(c0, 0);
  c1 = min(c1, sh.n_chunks);
  double s = 0.0;
  for (int c = c0 + threadIdx.x; c < c1; c += GRAD_THREADS) s += partial[c];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, kWave);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  s = (red[0] + red[1]) + (red[2] + red[3]);
  const double norm = sqrt(s);
  const bool bad = !__builtin_isfinite(s);
  GradFactors f{0.5f, 1, 0.f, 0.f, bad ? 1 : 0};
  if (bad) set_flag(status, LORA_FLAG_NONFINITE_GRAD);
  else f.coef = (float)frexp(fmin(1.0, (double)max_norm / (norm + 1e-6)), &f.exp2);
  if (ad.steps && !bad) {
    const int64_t step = ad.steps[a] + 1;
    ad.steps[a] = step;
    f.step_size = (float)(ad.lr / (1.0 - pow(ad.beta1, (double)step)));
    f.inv_sqrt_bc2 = (float)(1.0 / sqrt(1.0 - pow(ad.beta2, (double)step)));
  }
  if (norms) norms[a] = (float)norm;
  out[a] = f;
}

// out = c_a g over one chunk; a skipped group's gradient is copied as it is.
__global__ __launch_bounds__(GRAD_THREADS) void grad_scale_kernel(
    grad_shape sh, const grad_tensor* __restrict__ tab, const float* g,
    const GradFactors* __restrict__ fac, float* out, int32_t* __restrict__ status) {
  const GradSpan sp = grad_span(sh, tab, blockIdx.x, status);
  if (sp.count == 0) return;
  const GradFactors f = fac[sp.group];
  const float* p = g + sp.begin;
  float* o = out + sp.begin;
  if ((((uintptr_t)p | (uintptr_t)o) & 15) == 0) {
    const int n4 = sp.count / 4;
    float4 v[GRAD_CHUNK / (GRAD_THREADS * 4)];
#pragma unroll
    for (int q = 0; q < GRAD_CHUNK / (GRAD_THREADS * 4); ++q) {
      const int i = q * GRAD_THREADS + threadIdx.x;
      if (i < n4) v[q] = ((const float4*)p)[i];
    }
#pragma unroll
    for (int q = 0; q < GRAD_CHUNK / (GRAD_THREADS * 4); ++q) {
      const int i = q * GRAD_THREADS + threadIdx.x;
      if (i < n4)
        ((float4*)o)[i] = make_float4(clipped(v[q].x, f), clipped(v[q].y, f), clipped(v[q].z, f),
                                      clipped(v[q].w, f));
    }
    const int i = n4 * 4 + threadIdx.x;
    if (i < sp.count) o[i] = clipped(p[i], f);
  } else {
    for (int i = threadIdx.x; i < sp.count; i += GRAD_THREADS) o[i] = clipped(p[i], f);
  }
}

// The step's constants, each rounded to fp32 from its 64-bit value: 1 - beta2
// taken from an fp32 beta2 = 0.999 would be off by 1.3e-5.
struct AdamConst {
  float b1, a1, b2, a2, decay, eps;   // a = 1 - b, decay = lr weight_decay
};

__device__ __forceinline__ void adam_elem(float& p, float g, float& m, float& v,
                                          const AdamConst& k, const GradFactors& f) {
  g = clipped(g, f);
  m = k.b1 * m + k.a1 * g;
  v = k.b2 * v + k.a2 * (g * g);
  p = p - k.decay * p;
  p = p - f.step_size * __fdiv_rn(m, __fsqrt_rn(v) * f.inv_sqrt_bc2 + k.eps);
}

// One AdamW step on c_a g over one chunk; a skipped group keeps every value.
__global__ __launch_bounds__(GRAD_THREADS) void grad_adam_kernel(
    grad_shape sh, const grad_tensor* __restrict__ tab, const GradFactors* __restrict__ fac,
    float* __restrict__ p, const float* __restrict__ g, float* __restrict__ m,
    float* __restrict__ v, AdamConst k, uint16_t* __restrict__ pb, int32_t* __restrict__ status) {
  const GradSpan sp = grad_span(sh, tab, blockIdx.x, status);
  if (sp.count == 0) return;
  const GradFactors f = fac[sp.group];
  if (f.skip) return;
  p += sp.begin;
  g += sp.begin;
  m += sp.begin;
  v += sp.begin;
  if (pb) pb += sp.begin;
  const bool vec = (((uintptr_t)p | (uintptr_t)g | (uintptr_t)m | (uintptr_t)v) & 15) == 0 &&
                   ((uintptr_t)pb & 7) == 0;
  int done = 0;
  if (vec) {
    const int n4 = sp.count / 4;
    done = n4 * 4;
#pragma unroll 2
    for (int i = threadIdx.x; i < n4; i += GRAD_THREADS) {
      float4 pp = ((float4*)p)[i], mm = ((float4*)m)[i], vv = ((float4*)v)[i];
      const float4 gg = ((const float4*)g)[i];
      adam_elem(pp.x, gg.x, mm.x, vv.x, k, f);
      adam_elem(pp.y, gg.y, mm.y, vv.y, k, f);
      adam_elem(pp.z, gg.z, mm.z, vv.z, k, f);
      adam_elem(pp.w, gg.w, mm.w, vv.w, k, f);
      ((float4*)p)[i] = pp;
      ((float4*)m)[i] = mm;
      ((float4*)v)[i] = vv;
      if (pb) ((uint2*)pb)[i] = make_uint2(pack2bf(pp.x, pp.y), pack2bf(pp.z, pp.w));
    }
  }
  for (int i = done + threadIdx.x; i < sp.count; i += GRAD_THREADS) {
    float pp = p[i], mm = m[i], vv = v[i];
    adam_elem(pp, g[i], mm, vv, k, f);
    p[i] = pp;
    m[i] = mm;
    v[i] = vv;
    if (pb) pb[i] = f2bf(pp);
  }
}

}  // namespace lora

namespace lora_host {
using namespace lora;

struct GradWs {
  int32_t* status;
  GradFactors* fac;
  double* partial;
  size_t total;
};
static GradWs carve_grads(const grad_shape& sh, void* ws) {
  Carve cv(ws, 0);
  GradWs w{};
  w.status = cv.take<int32_t>(64);
  w.fac = cv.take<GradFactors>((size_t)sh.n_groups);
  w.partial = cv.take<double>((size_t)sh.n_chunks);
  w.total = cv.used;
  return w;
}
size_t grad_ws_bytes(const grad_shape& sh) { return carve_grads(sh, nullptr).total; }

static lora_status norms_and_factors(const grad_shape& sh, const grad_tensor* tab, const float* g,
                                     float max_norm, const GradAdam& ad, float* norms,
                                     const GradWs& w, hipStream_t s) {
  if (sh.n_chunks > 0) {
    hipLaunchKernelGGL(grad_partial_kernel, dim3((unsigned)sh.n_chunks), dim3(GRAD_THREADS), 0, s,
                       sh, tab, g, w.partial, w.status);
    lora_status st = launch_check("grad_partial");
    if (st != LORA_OK) return st;
  }
  hipLaunchKernelGGL(grad_join_kernel, dim3((unsigned)sh.n_groups), dim3(GRAD_THREADS), 0, s, sh,
                     tab, w.partial, max_norm, ad, norms, w.fac, w.status);
  return launch_check("grad_join");
}

lora_status launch_grad_norm(const grad_shape& sh, const grad_tensor* tab, const float* g,
                             float* norms, void* ws, hipStream_t s) {
  return norms_and_factors(sh, tab, g, INFINITY, GradAdam{}, norms, carve_grads(sh, ws), s);
}

lora_status launch_grad_clip(const grad_shape& sh, const grad_tensor* tab, const float* g,
                             float max_norm, float* out, float* norms, void* ws, hipStream_t s) {
  const GradWs w = carve_grads(sh, ws);
  lora_status st = norms_and_factors(sh, tab, g, max_norm, GradAdam{}, norms, w, s);
  if (st != LORA_OK || sh.n_chunks == 0) return st;
  hipLaunchKernelGGL(grad_scale_kernel, dim3((unsigned)sh.n_chunks), dim3(GRAD_THREADS), 0, s, sh,
                     tab, g, w.fac, out, w.status);
  return launch_check("grad_scale");
}

lora_status launch_adam_clipped(const grad_shape& sh, const grad_tensor* tab, int64_t* steps,
                                float* p, const float* g, float* m, float* v, float max_norm,
                                double lr, double beta1, double beta2, double eps, double wd,
                                uint16_t* p_bf16, float* norms, void* ws, hipStream_t s) {
  const GradWs w = carve_grads(sh, ws);
  lora_status st = norms_and_factors(sh, tab, g, max_norm, GradAdam{steps, lr, beta1, beta2}, norms,
                                     w, s);
  if (st != LORA_OK || sh.n_chunks == 0) return st;
  const AdamConst k{(float)beta1, (float)(1.0 - beta1), (float)beta2,
                    (float)(1.0 - beta2), (float)(lr * wd), (float)eps};
  hipLaunchKernelGGL(grad_adam_kernel, dim3((unsigned)sh.n_chunks), dim3(GRAD_THREADS), 0, s, sh,
                     tab, w.fac, p, g, m, v, k, p_bf16, w.status);
  return launch_check("grad_adam");
}

}  // namespace lora_host
