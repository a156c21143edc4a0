// Per-adapter gradient norms over many tensors, clipping, and AdamW on the
// clipped gradient, on gfx950.
//
//   s_a = sum over adapter a's tensors of g^2,  norm_a = sqrt(s_a),
//   c_a = min(1, max_norm / (norm_a + 1e-6));   g <- c_a g, or one AdamW step on c_a g.
//
// Two launches.  The first walks the chunks (8192 elements of one tensor) and
// leaves, per block and group, the sum of squares in 64 bits, so that no square of
// a finite gradient overflows.  In the second every block joins its group's sums
// again, in block order -- at most 4096 of them, read from L2 while its own first
// elements are on their way -- instead of a launch between the two that would
// only add its latency, and then scales or steps its chunks.  A group is skipped
// when its sum is not finite, that is when any of its elements is NaN or +-Inf, so the
// norm's pass over g is also the scan that decides the skip (AdamW skips a group with a
// counter that counts no steps as well).  Both passes are bound by HBM.
#include "common.hpp"
#include "sgmv.hpp"

namespace lora {

constexpr int GRAD_THREADS = 256;
constexpr int GRAD_CHUNK = LORA_GRAD_CHUNK;
static_assert(GRAD_CHUNK % (GRAD_THREADS * 4) == 0, "whole 16-byte rounds per chunk");

// A group's factors.  c_a = coef 2^exp2, with exp2 = 0 wherever c_a is a normal fp32
// number: one product, and c_a = 1 leaves every g as it is, subnormals too.  A smaller
// c_a (gradients near the fp32 range) keeps its bits in coef, and ldexp rounds only
// where the result is subnormal.
struct GradFactors {
  float coef;          // 1 for a group whose gradient is not finite
  int32_t exp2;
  float step_size;     // lr / (1 - beta1^step)
  float inv_sqrt_bc2;  // 1 / sqrt(1 - beta2^step)
  int32_t skip;        // a gradient that is not finite, or a counter that counts no steps
};

__device__ __forceinline__ float clipped(float g, const GradFactors& f) {
  return __builtin_amdgcn_ldexpf(g * f.coef, f.exp2);
}

// The part of a tensor that a chunk covers; count 0 if the table is not what it
// has to be there (flagged: the chunk is then read and written by nobody).
struct GradSpan {
  int64_t begin;
  int32_t count;
  int32_t group;
};

// Workspace of one call (all written before they are read).
struct GradWs {
  int32_t* status;
  GradSpan* span;      // [n_chunks]
  double* slot;        // [blocks + n_groups]: block b's part of group a at b + a.  Both only
                       // grow along the chunks, so no two parts share a slot.
  int32_t* start;      // [n_groups + 1] first chunk of each group
  int64_t* steps;      // [n_groups] the step counters before the call
  int32_t per;         // chunks per block of the first launch
};

// The last tensor whose first_chunk is <= c, by a whole wave with a uniform c.
__device__ __forceinline__ int grad_find(const grad_shape& sh, const grad_tensor* tab, int c) {
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
  return __builtin_amdgcn_readfirstlane(lo);
}

// Entry i by itself, in order, and with the chunks it has to have.
__device__ __forceinline__ bool grad_entry_ok(const grad_shape& sh, const grad_tensor* tab, int i) {
  const grad_tensor t = tab[i];
  if (t.offset < 0 || t.count < 0 || t.offset > sh.n_elems || t.count > sh.n_elems - t.offset ||
      t.group < (i > 0 ? tab[i - 1].group : 0) || t.group < 0 || t.group >= sh.n_groups)
    return false;
  const int end = i + 1 < sh.n_tensors ? tab[i + 1].first_chunk : sh.n_chunks;
  return (i > 0 || t.first_chunk == 0) &&
         end - (int64_t)t.first_chunk == (t.count + GRAD_CHUNK - 1) / GRAD_CHUNK;
}

__device__ __forceinline__ GradSpan grad_span(const grad_shape& sh, const grad_tensor& t, int c,
                                              int32_t* status) {
  const int64_t at = (int64_t)(c - t.first_chunk) * GRAD_CHUNK;
  const bool ok = t.first_chunk >= 0 && t.first_chunk <= c && t.offset >= 0 && t.count >= 0 &&
                  t.offset <= sh.n_elems && t.count <= sh.n_elems - t.offset && at < t.count &&
                  t.group >= 0 && t.group < sh.n_groups;
  if (!ok) {
    if (threadIdx.x == 0) set_flag(status, LORA_FLAG_BAD_DESC);
    return GradSpan{0, 0, 0};
  }
  return GradSpan{t.offset + at, (int32_t)min((int64_t)GRAD_CHUNK, t.count - at), t.group};
}

// Sum over the block, the same value in every thread.
__device__ __forceinline__ double grad_block_sum(double s, double* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, kWave);
  __syncthreads();   // red may still be read from the last call
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

constexpr int GRAD_ROUNDS = GRAD_CHUNK / (GRAD_THREADS * 4);   // 16-byte pieces per thread

// A chunk's pieces into registers (zeros past its end and where it is not 16-byte
// aligned), and their sum of squares with what the pieces leave out.
struct GradPieces {
  float4 v[GRAD_ROUNDS];
};
__device__ __forceinline__ void grad_fetch(GradPieces& r, const float* g, const GradSpan& sp) {
  const float* p = g + sp.begin;
  const int n4 = ((uintptr_t)p & 15) == 0 ? sp.count / 4 : 0;
#pragma unroll
  for (int q = 0; q < GRAD_ROUNDS; ++q) {
    const int i = q * GRAD_THREADS + threadIdx.x;
    r.v[q] = i < n4 ? ((const float4*)p)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}
__device__ __forceinline__ double grad_squares(const GradPieces& r, const float* g,
                                               const GradSpan& sp) {
  double s = 0.0;
#pragma unroll
  for (int q = 0; q < GRAD_ROUNDS; ++q)
    s += (double)r.v[q].x * r.v[q].x + (double)r.v[q].y * r.v[q].y +
         (double)r.v[q].z * r.v[q].z + (double)r.v[q].w * r.v[q].w;
  const float* p = g + sp.begin;
  const int done = ((uintptr_t)p & 15) == 0 ? sp.count & ~3 : 0;
  for (int i = done + threadIdx.x; i < sp.count; i += GRAD_THREADS) s += (double)p[i] * p[i];
  return s;
}

// Whether a counter of steps made has a next one, at least 1: others would divide by
// 1 - beta^0 or count past 64 bits.
__device__ __forceinline__ bool grad_counts(int64_t made) { return made >= 0 && made < INT64_MAX; }

// First launch.  Block b takes chunks b per .. (b + 1) per - 1, the next chunk's
// elements in flight while one is summed.
__global__ __launch_bounds__(GRAD_THREADS) void grad_partial_kernel(
    grad_shape sh, const grad_tensor* __restrict__ tab, const float* __restrict__ g,
    const int64_t* __restrict__ steps, GradWs ws) {
  __shared__ double red[GRAD_THREADS / kWave];
  // the groups' first chunks, the step counters and the table's check, by the grid's threads
  const int threads = gridDim.x * GRAD_THREADS, id = blockIdx.x * GRAD_THREADS + threadIdx.x;
  for (int i = id; i < max(sh.n_tensors, 1); i += threads) {
    const int before = i > 0 ? min(tab[i - 1].group, sh.n_groups) : -1;
    const int here = sh.n_tensors > 0 ? min(tab[i].group, sh.n_groups) : -1;
    if (sh.n_tensors > 0 && !grad_entry_ok(sh, tab, i)) set_flag(ws.status, LORA_FLAG_BAD_DESC);
    for (int a = max(before + 1, 0); a <= min(here, sh.n_groups - 1); ++a)
      ws.start[a] = tab[i].first_chunk;
    if (i + 1 >= sh.n_tensors)
      for (int a = max(here + 1, 0); a <= sh.n_groups; ++a) ws.start[a] = sh.n_chunks;
  }
  if (steps)
    for (int a = id; a < sh.n_groups; a += threads) {
      ws.steps[a] = steps[a];
      if (!grad_counts(steps[a])) set_flag(ws.status, LORA_FLAG_BAD_DESC);
    }

  const int c0 = blockIdx.x * ws.per, c1 = min(sh.n_chunks, c0 + ws.per);
  if (c0 >= c1) return;
  int ti = grad_find(sh, tab, c0);
  GradSpan sp = grad_span(sh, tab[ti], c0, ws.status);
  GradPieces cur, nxt;
  grad_fetch(cur, g, sp);
  double s = 0.0;
  for (int c = c0; c < c1; ++c) {
    GradSpan ns{0, 0, -1};
    if (c + 1 < c1) {
      while (ti + 1 < sh.n_tensors && tab[ti + 1].first_chunk <= c + 1) ++ti;
      ns = grad_span(sh, tab[ti], c + 1, ws.status);
      grad_fetch(nxt, g, ns);
    }
    s += grad_squares(cur, g, sp);
    if (threadIdx.x == 0) ws.span[c] = sp;
    if (ns.group != sp.group) {   // uniform: the group ends here for this block
      const double t = grad_block_sum(s, red);
      if (threadIdx.x == 0) ws.slot[blockIdx.x + sp.group] = t;
      s = 0.0;
    }
    sp = ns;
    cur = nxt;
  }
}

struct GradAdam {
  int64_t* steps;   // null: no optimizer step follows
  double lr, beta1, beta2;
};

// b^n by squaring: the relative error of b^n is n 2^-53, so that of 1 - b^n, of
// size 1 / (1 - b) at most where b^n counts, stays below fp32's.
__device__ __forceinline__ double power(double b, int64_t n) {
  double r = 1.0;
  for (; n > 0; n >>= 1) {
    if (n & 1) r *= b;
    b *= b;
  }
  return r;
}

// Group a's sum, by the whole block in block order; the factors that follow from it.
__device__ __forceinline__ GradFactors grad_factors(const grad_shape& sh, const GradWs& ws, int a,
                                                    float max_norm, const GradAdam& ad,
                                                    double* red, double& norm) {
  const int c0 = max(ws.start[a], 0), c1 = min(ws.start[a + 1], sh.n_chunks);
  double s = 0.0;
  if (c0 < c1)
    for (int b = c0 / ws.per + (int)threadIdx.x; b <= (c1 - 1) / ws.per; b += GRAD_THREADS)
      s += ws.slot[b + a];
  s = grad_block_sum(s, red);
  norm = sqrt(s);
  GradFactors f{1.f, 0, 0.f, 0.f, 0};
  if (!__builtin_isfinite(s)) {
    f.skip = 1;
    return f;
  }
  const double c = fmin(1.0, (double)max_norm / (norm + 1e-6));
  f.coef = (float)c;
  if (c < 0x1p-126) f.coef = (float)frexp(c, &f.exp2);
  if (ad.steps) {
    f.skip = !grad_counts(ws.steps[a]);
    const int64_t step = f.skip ? 1 : ws.steps[a] + 1;
    f.step_size = (float)(ad.lr / (1.0 - power(ad.beta1, step)));
    f.inv_sqrt_bc2 = (float)(1.0 / sqrt(1.0 - power(ad.beta2, step)));
  }
  return f;
}

// What one block a group reports: the norm, the flag, the step counter.
__device__ __forceinline__ void grad_report(const GradWs& ws, int a, double norm,
                                            const GradFactors& f, const GradAdam& ad,
                                            float* norms) {
  if (threadIdx.x != 0) return;
  if (norms) norms[a] = (float)norm;
  if (!__builtin_isfinite(norm)) set_flag(ws.status, LORA_FLAG_NONFINITE_GRAD);
  if (ad.steps && !f.skip) ad.steps[a] = ws.steps[a] + 1;
}

// grad_norm's second launch: one block a group.
__global__ __launch_bounds__(GRAD_THREADS) void grad_norm_kernel(grad_shape sh, GradWs ws,
                                                                 float* __restrict__ norms) {
  __shared__ double red[GRAD_THREADS / kWave];
  double norm;
  const GradFactors f = grad_factors(sh, ws, blockIdx.x, INFINITY, GradAdam{}, red, norm);
  grad_report(ws, blockIdx.x, norm, f, GradAdam{}, norms);
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

struct GradOut {
  float* out;          // grad_clip's result; null: the AdamW step below
  float* p;
  float* m;
  float* v;
  uint16_t* pb;
  AdamConst k;
};

// The second launch's accesses are non-temporal: each value is used once, and with
// ordinary ones the lines of p, m and v push out the g that the first launch left in
// the last-level cache and are written back under the next call's reads (87 M
// parameters, one call after another: 647 us with ordinary accesses, 575 us without).
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ f32x4 nt_load(const float* p) {
  return __builtin_nontemporal_load((const f32x4*)p);
}
__device__ __forceinline__ void nt_store(float* p, f32x4 v) {
  __builtin_nontemporal_store(v, (f32x4*)p);
}

// Four elements of every array that the second launch touches.
struct GradQuad {
  f32x4 g, p, m, v;
};
template <bool ADAM>
__device__ __forceinline__ GradQuad grad_load4(const float* g, const GradOut& o, int64_t at) {
  GradQuad q;
  q.g = nt_load(g + at);
  if (ADAM) {
    q.p = nt_load(o.p + at);
    q.m = nt_load(o.m + at);
    q.v = nt_load(o.v + at);
  }
  return q;
}
template <bool ADAM>
__device__ __forceinline__ void grad_store4(GradQuad q, const GradOut& o, int64_t at,
                                            const GradFactors& f) {
  if (!ADAM) {
    nt_store(o.out + at, f32x4{clipped(q.g[0], f), clipped(q.g[1], f), clipped(q.g[2], f),
                               clipped(q.g[3], f)});
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float p = q.p[i], m = q.m[i], v = q.v[i];
    adam_elem(p, q.g[i], m, v, o.k, f);
    q.p[i] = p;
    q.m[i] = m;
    q.v[i] = v;
  }
  nt_store(o.p + at, q.p);
  nt_store(o.m + at, q.m);
  nt_store(o.v + at, q.v);
  if (o.pb)
    __builtin_nontemporal_store(u32x2{pack2bf(q.p[0], q.p[1]), pack2bf(q.p[2], q.p[3])},
                                (u32x2*)(o.pb + at));
}

// Second launch: out = c_a g (a skipped group's gradient as it is), or one AdamW
// step on c_a g (a skipped group keeps every value).  The chunks are taken in PARTS
// parts each, block b parts b, b + blocks, ...: all of a part's accesses are in flight
// at once, and blocks that run together touch neighbouring memory (ranges of chunks
// per block instead cost 5%).
// g and out may be the same buffer: a thread reads an element before it writes it.
template <bool ADAM, int PARTS>
__global__ __launch_bounds__(GRAD_THREADS) void grad_apply_kernel(grad_shape sh, GradWs ws,
                                                                  const float* g, float max_norm,
                                                                  GradAdam ad, GradOut o,
                                                                  float* __restrict__ norms) {
  __shared__ double red[GRAD_THREADS / kWave];
  constexpr int PART = GRAD_CHUNK / PARTS;
  constexpr int AHEAD = PART / (GRAD_THREADS * 4);   // 16-byte pieces per thread
  GradFactors f{};
  int group = -1;
  const int units = sh.n_chunks * PARTS;   // < 2^26
  GradSpan sp = blockIdx.x < units ? ws.span[blockIdx.x / PARTS] : GradSpan{0, 0, 0};
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t begin = sp.begin + (int64_t)(u % PARTS) * PART;
    const int count = min(sp.count - u % PARTS * PART, PART);
    const int a = sp.group;
    if (u + gridDim.x < units) sp = ws.span[(u + gridDim.x) / PARTS];
    if (count <= 0) continue;
    bool vec = ((uintptr_t)(g + begin) & 15) == 0;
    if (ADAM)
      vec = vec && ((((uintptr_t)(o.p + begin)) | ((uintptr_t)(o.m + begin)) |
                     ((uintptr_t)(o.v + begin))) & 15) == 0 &&
            (((uintptr_t)(o.pb ? o.pb + begin : nullptr)) & 7) == 0;
    else
      vec = vec && ((uintptr_t)(o.out + begin) & 15) == 0;
    const int n4 = vec ? count / 4 : 0;
    GradQuad q[AHEAD];
#pragma unroll
    for (int r = 0; r < AHEAD; ++r) {
      const int i = r * GRAD_THREADS + (int)threadIdx.x;
      if (i < n4) q[r] = grad_load4<ADAM>(g, o, begin + 4 * (int64_t)i);
    }
    if (a != group) {   // the factors are found while the first pieces arrive
      group = a;
      double norm;
      f = grad_factors(sh, ws, a, max_norm, ad, red, norm);
      if (u == ws.start[a] * PARTS) grad_report(ws, a, norm, f, ad, norms);
    }
    if (ADAM && f.skip) continue;
#pragma unroll
    for (int r = 0; r < AHEAD; ++r) {
      const int i = r * GRAD_THREADS + (int)threadIdx.x;
      if (i < n4) grad_store4<ADAM>(q[r], o, begin + 4 * (int64_t)i, f);
    }
    for (int i = n4 * 4 + threadIdx.x; i < count; i += GRAD_THREADS) {
      const int64_t at = begin + i;
      if (ADAM) {
        float pp = o.p[at], mm = o.m[at], vv = o.v[at];
        adam_elem(pp, g[at], mm, vv, o.k, f);
        o.p[at] = pp;
        o.m[at] = mm;
        o.v[at] = vv;
        if (o.pb) o.pb[at] = f2bf(pp);
      } else {
        o.out[at] = clipped(g[at], f);
      }
    }
  }
  // groups without a chunk have a norm of zero and step over nothing
  for (int a = blockIdx.x * GRAD_THREADS + threadIdx.x; a < sh.n_groups;
       a += gridDim.x * GRAD_THREADS)
    if (ws.start[a] >= ws.start[a + 1]) {
      if (norms) norms[a] = 0.f;
      if (ad.steps && grad_counts(ws.steps[a])) ad.steps[a] = ws.steps[a] + 1;
    }
}

}  // namespace lora

namespace lora_host {
using namespace lora;

// Most blocks of the first launch: its blocks' sums of a group are read at once by
// every block of the second.
constexpr int GRAD_BLOCKS = 4096;

static GradWs carve_grads(const grad_shape& sh, void* ws, size_t* bytes = nullptr) {
  Carve cv(ws, 0);
  GradWs w{};
  w.per = (int)std::max<int64_t>(1, cdiv(sh.n_chunks, GRAD_BLOCKS));
  w.status = cv.take<int32_t>(64);
  w.span = cv.take<GradSpan>((size_t)sh.n_chunks);
  w.slot = cv.take<double>((size_t)cdiv(sh.n_chunks, w.per) + sh.n_groups);
  w.start = cv.take<int32_t>((size_t)sh.n_groups + 1);
  w.steps = cv.take<int64_t>((size_t)sh.n_groups);
  if (bytes) *bytes = cv.used;
  return w;
}
size_t grad_ws_bytes(const grad_shape& sh) {
  size_t n = 0;
  carve_grads(sh, nullptr, &n);
  return n;
}

static lora_status partial_sums(const grad_shape& sh, const grad_tensor* tab, const float* g,
                                const int64_t* steps, const GradWs& w, hipStream_t s) {
  const unsigned grid = (unsigned)std::max<int64_t>(1, cdiv(sh.n_chunks, w.per));
  hipLaunchKernelGGL(grad_partial_kernel, dim3(grid), dim3(GRAD_THREADS), 0, s, sh, tab, g, steps, w);
  return launch_check("grad_partial");
}

// Parts of a chunk a block takes at a time, and the most blocks.  AdamW moves four
// arrays: a quarter keeps 32 KB in flight, and 16384 blocks ran best (87 M parameters,
// both launches: 537 us, with 4096 blocks 583, with one block per quarter 566; 5.5 TB/s
// in the second launch).  Clipping moves two: a whole chunk keeps them busy (18 M
// elements: 38.6 us, in quarters 45) unless there are too few chunks for the CUs
// (0.14 M elements: 7.8 us, in quarters 7.0).
template <bool ADAM, int PARTS>
static lora_status apply(const grad_shape& sh, const GradWs& w, const float* g, float max_norm,
                         const GradAdam& ad, const GradOut& o, float* norms, hipStream_t s) {
  constexpr int most = ADAM ? 16384 : 8192;
  const unsigned grid = (unsigned)std::max(1, std::min(sh.n_chunks * PARTS, most));
  hipLaunchKernelGGL((grad_apply_kernel<ADAM, PARTS>), dim3(grid), dim3(GRAD_THREADS), 0, s, sh, w,
                     g, max_norm, ad, o, norms);
  return launch_check("grad_apply");
}

lora_status launch_grad_norm(const grad_shape& sh, const grad_tensor* tab, const float* g,
                             float* norms, void* ws, hipStream_t s) {
  const GradWs w = carve_grads(sh, ws);
  lora_status st = partial_sums(sh, tab, g, nullptr, w, s);
  if (st != LORA_OK) return st;
  hipLaunchKernelGGL(grad_norm_kernel, dim3((unsigned)sh.n_groups), dim3(GRAD_THREADS), 0, s, sh, w,
                     norms);
  return launch_check("grad_norm");
}

lora_status launch_grad_clip(const grad_shape& sh, const grad_tensor* tab, const float* g,
                             float max_norm, float* out, float* norms, void* ws, hipStream_t s) {
  const GradWs w = carve_grads(sh, ws);
  lora_status st = partial_sums(sh, tab, g, nullptr, w, s);
  if (st != LORA_OK) return st;
  GradOut o{};
  o.out = out;
  return sh.n_chunks >= 4 * device_cus() ? apply<false, 1>(sh, w, g, max_norm, GradAdam{}, o, norms, s)
                                         : apply<false, 4>(sh, w, g, max_norm, GradAdam{}, o, norms, s);
}

lora_status launch_adam_clipped(const grad_shape& sh, const grad_tensor* tab, int64_t* steps,
                                float* p, const float* g, float* m, float* v, float max_norm,
                                double lr, double beta1, double beta2, double eps, double wd,
                                uint16_t* p_bf16, float* norms, void* ws, hipStream_t s) {
  const GradWs w = carve_grads(sh, ws);
  lora_status st = partial_sums(sh, tab, g, steps, w, s);
  if (st != LORA_OK) return st;
  const AdamConst k{(float)beta1, (float)(1.0 - beta1), (float)beta2,
                    (float)(1.0 - beta2), (float)(lr * wd), (float)eps};
  const GradOut o{nullptr, p, m, v, p_bf16, k};
  return apply<true, 4>(sh, w, g, max_norm, GradAdam{steps, lr, beta1, beta2}, o, norms, s);
}

}  // namespace lora_host
