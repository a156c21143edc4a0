// RMS norm with the residual's addition on gfx950: forward (bf16 or 8-bit
// block-scaled output) and backward.
//
//   h = bf16(x + residual),  rstd = 1 / sqrt(mean_j h_j^2 + eps),
//   v_j = h_j rstd w_j;      y = bf16(v), or per 32 columns
//   e = the least integer with max|v| <= 448 2^e,  q = e4m3(v 2^-e).
//   backward, with xh = h rstd and g = dy w:
//   dx = bf16(dh + rstd (g - xh mean_j(g xh))),   dw_j = sum_t dy_tj xh_tj.
//
// Everything is bound by HBM: a row is read once, kept in registers across its
// reduction and written once (but for the backward of rows past 16384 columns, which
// does not fit them: see there).  In a captured graph, launches included, 8192 x 4096
// with the residual takes 46.4 us (5.8 TB/s), its backward 44.6 us (6.0 TB/s) and 51.6
// with the weight's gradient; 4097 x 2048 in 8 bits 11.7 us (5.0 TB/s).
// A team of lanes owns a row and lane l of it holds the 8-column vectors l, l + team, ...:
// rows of up to 512 columns take part of a wave (several rows a wave, shuffles only),
// longer ones whole waves of one block that join their sums through LDS.  Teams step over
// the rows with the grid's stride, so a block reads the weight once.  The team of a row
// depends on `hidden` alone: a row's bits do not change with the batch.
#include <type_traits>

#include "common.hpp"
#include "sgmv.hpp"

namespace lora {

constexpr int NORM_MAX_VPL = 4;      // vectors of 8 columns a lane holds
constexpr int NORM_SMALL_BLOCK = 256;

// Columns c..c+7 of a row: one 16-byte access where every row is 16-byte
// aligned (hidden a multiple of 8), else element by element up to column H.
// NT: a non-temporal access, see norm_streams.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <bool VEC, bool NT = false>
__device__ __forceinline__ uint4 norm_load8(const uint16_t* row, int c, int H) {
  if (VEC && NT) {
    const u32x4 v = __builtin_nontemporal_load((const u32x4*)(row + c));
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
  if (VEC) return *(const uint4*)(row + c);
  uint32_t r[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < H) r[i >> 1] |= (uint32_t)row[c + i] << (16 * (i & 1));
  return make_uint4(r[0], r[1], r[2], r[3]);
}
template <bool VEC, bool NT>
__device__ __forceinline__ void norm_store8(uint16_t* row, int c, int H, uint4 v) {
  if (VEC && NT) {
    __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, (u32x4*)(row + c));
    return;
  }
  if (VEC) {
    *(uint4*)(row + c) = v;
    return;
  }
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < H) row[c + i] = (uint16_t)(r[i >> 1] >> (16 * (i & 1)));
}
__device__ __forceinline__ void unpack8(uint4 v, float* f) {
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = bf2f_lo(r[q]);
    f[2 * q + 1] = bf2f_hi(r[q]);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack2bf(f[0], f[1]), pack2bf(f[2], f[3]), pack2bf(f[4], f[5]),
                    pack2bf(f[6], f[7]));
}

// Sum over the row's team, the same value in each of its lanes: shuffles within
// the wave, then the waves' sums in wave order.  `red` alternates between two
// halves by `turn`, so one barrier a row suffices.
__device__ __forceinline__ float team_sum(float s, int team, float (*red)[16], int turn) {
  const int in_wave = team < kWave ? team : kWave;
  for (int o = in_wave >> 1; o > 0; o >>= 1) s += __shfl_xor(s, o, kWave);
  if (team <= kWave) return s;
  if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = s;
  __syncthreads();
  float t = 0.f;
  for (int w = 0; w < team / kWave; ++w) t += red[turn][w];
  return t;
}

__device__ __forceinline__ float norm_rstd(float ss, int H, float eps) {
  return __fdiv_rn(1.f, __fsqrt_rn(ss / (float)H + eps));
}

// The 8-bit form of the 32 columns that lanes 4i..4i+3 hold: the scale's biased
// exponent byte from the largest finite magnitude's bits (the least power of two
// with max <= 448 scale, so no finite value saturates), at least 1 (2^-126) and
// by the finite range at most 247, so that the scale and its reciprocal are
// normal fp32 numbers; then e4m3 codes, rounded to nearest even.  NaN and
// +-Inf become the NaN code.
__device__ __forceinline__ uint2 quantize8(const float* v, int& scale_byte) {
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(v[i]);
    mx = (a <= 3.4028234663852886e38f && a > mx) ? a : mx;
  }
  mx = fmaxf(mx, __shfl_xor(mx, 1, kWave));
  mx = fmaxf(mx, __shfl_xor(mx, 2, kWave));
  const int bits = __float_as_int(mx);
  const int b = max((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000 ? 1 : 0), 1);
  scale_byte = b;
  const float mul = __int_as_float((254 - b) << 23);   // 2^(127 - b)
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = v[i] * mul;
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(s[4], s[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(s[6], s[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

template <int VPL, bool VEC, bool NT, bool Q8>
__global__ __launch_bounds__(VPL == 1 ? NORM_SMALL_BLOCK : 1024) void rmsnorm_fwd_kernel(
    int64_t n, int H, int team, const uint16_t* x, const uint16_t* res,
    const uint16_t* __restrict__ weight, float eps, uint16_t* h, uint16_t* y,
    uint8_t* __restrict__ q, uint8_t* __restrict__ qs, float* __restrict__ rstd_out) {
  __shared__ float red[2][16];
  const int lane = threadIdx.x % team;
  const int64_t per_block = blockDim.x / team;
  const int64_t stride = per_block * gridDim.x;
  uint4 wv[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = (lane + v * team) * 8;
    wv[v] = c < H ? norm_load8<VEC>(weight, c, H) : make_uint4(0, 0, 0, 0);
  }
  int turn = 0;
  // every lane of a block runs the same number of rounds (the barriers below)
  for (int64_t r0 = (int64_t)blockIdx.x * per_block; r0 < n; r0 += stride, turn ^= 1) {
    const int64_t row = r0 + threadIdx.x / team, base = row * H;
    const bool live = row < n;
    uint4 xv[VPL], rv[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c = (lane + v * team) * 8;
      const bool on = live && c < H;
      xv[v] = on ? norm_load8<VEC, NT>(x + base, c, H) : make_uint4(0, 0, 0, 0);
      if (res) rv[v] = on ? norm_load8<VEC, NT>(res + base, c, H) : make_uint4(0, 0, 0, 0);
    }
    float f[VPL][8];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c = (lane + v * team) * 8;
      unpack8(xv[v], f[v]);
      if (res) {
        float g[8];
        unpack8(rv[v], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[v][i] += g[i];
        const uint4 hv = pack8(f[v]);
        if (live && c < H) norm_store8<VEC, NT>(h + base, c, H, hv);
        unpack8(hv, f[v]);   // the statistics are those of the stored h
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += f[v][i] * f[v][i];
    }
    ss = team_sum(ss, team, red, turn);
    const float rstd = norm_rstd(ss, H, eps);
    if (rstd_out && lane == 0 && live) rstd_out[row] = rstd;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c = (lane + v * team) * 8;
      float w[8], o[8];
      unpack8(wv[v], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = f[v][i] * rstd * w[i];
      if (Q8) {
        int b;
        const uint2 code = quantize8(o, b);
        if (live && c < H) {
          *(uint2*)(q + base + c) = code;
          if ((lane & 3) == 0) qs[base / 32 + c / 32] = (uint8_t)b;
        }
      } else if (live && c < H) {
        norm_store8<VEC, NT>(y + base, c, H, pack8(o));
      }
    }
  }
}

// Backward.  With `partial`, each lane keeps its columns' dw terms over the
// rows its team visits; the block's teams are joined through LDS in team order
// and the block writes one row of partial [gridDim.x][H].  A row of more than
// 16384 columns does not fit the registers beside dw: it is read again, from the
// caches, once its sum is known, and 42 registers a lane still spill to scratch, with a
// frozen weight too (2048 x 20480: 203 us without dw, 185 with it, 1.7 to 1.8 TB/s).
template <int VPL, bool VEC, bool NT>
__global__ __launch_bounds__(VPL == 1 ? NORM_SMALL_BLOCK : 1024) void rmsnorm_bwd_kernel(
    int64_t n, int H, int team, const uint16_t* dy, const uint16_t* dh,
    const uint16_t* __restrict__ h, const uint16_t* __restrict__ weight,
    const float* __restrict__ rstd_in, uint16_t* dx, float* __restrict__ partial) {
  constexpr bool AGAIN = VPL == NORM_MAX_VPL;
  __shared__ float red[2][16];
  __shared__ float join[NORM_SMALL_BLOCK * 8];
  const int lane = threadIdx.x % team;
  const int64_t per_block = blockDim.x / team;
  const int64_t stride = per_block * gridDim.x;
  uint4 wv[VPL];
  float dw[VPL][8];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int c = (lane + v * team) * 8;
    if (!AGAIN) wv[v] = c < H ? norm_load8<VEC>(weight, c, H) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v][i] = 0.f;
  }
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * per_block; r0 < n; r0 += stride, turn ^= 1) {
    const int64_t row = r0 + threadIdx.x / team, base = row * H;
    const bool live = row < n;
    const float rstd = live ? rstd_in[row] : 0.f;
    uint4 dv[VPL], hv[VPL], uv[VPL];
    auto load = [&](int v) {
      const int c = (lane + v * team) * 8;
      const bool on = live && c < H;
      dv[v] = on ? norm_load8<VEC, NT && !AGAIN>(dy + base, c, H) : make_uint4(0, 0, 0, 0);
      hv[v] = on ? norm_load8<VEC, NT && !AGAIN>(h + base, c, H) : make_uint4(0, 0, 0, 0);
      if (AGAIN) wv[v] = c < H ? norm_load8<VEC>(weight, c, H) : make_uint4(0, 0, 0, 0);
    };
    auto load_dh = [&](int v) {
      const int c = (lane + v * team) * 8;
      if (dh)
        uv[v] = live && c < H ? norm_load8<VEC, NT>(dh + base, c, H) : make_uint4(0, 0, 0, 0);
    };
    if (!AGAIN)
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        load(v);
        load_dh(v);
      }
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      if (AGAIN) {
        asm volatile("" ::: "memory");   // not all of the row's loads at once
        load(v);
      }
      float d[8], x[8], w[8];
      unpack8(dv[v], d);
      unpack8(hv[v], x);
      unpack8(wv[v], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = x[i] * rstd;
        s += d[i] * w[i] * xh;
        dw[v][i] += d[i] * xh;
      }
    }
    const float c1 = team_sum(s, team, red, turn) / (float)H;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      if (AGAIN) {
        asm volatile("" ::: "memory");   // a second read, not a kept register
        load(v);
        load_dh(v);
      }
      const int c = (lane + v * team) * 8;
      float d[8], x[8], w[8], u[8], o[8];
      unpack8(dv[v], d);
      unpack8(hv[v], x);
      unpack8(wv[v], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = rstd * (d[i] * w[i] - x[i] * rstd * c1);
      if (dh) {
        unpack8(uv[v], u);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += u[i];
      }
      if (live && c < H) norm_store8<VEC, NT>(dx + base, c, H, pack8(o));
    }
  }
  if (!partial) return;
  float* out = partial + (int64_t)blockIdx.x * H;
  if (per_block == 1) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int c = (lane + v * team) * 8;
      if (VEC) {
        if (c < H) {
          *(f32x4*)(out + c) = f32x4{dw[v][0], dw[v][1], dw[v][2], dw[v][3]};
          *(f32x4*)(out + c + 4) = f32x4{dw[v][4], dw[v][5], dw[v][6], dw[v][7]};
        }
        continue;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < H) out[c + i] = dw[v][i];
    }
    return;
  }
  // several teams a block (VPL is 1 here): join[team index][column]
#pragma unroll
  for (int i = 0; i < 8; ++i) join[threadIdx.x * 8 + i] = dw[0][i];
  __syncthreads();
  const int cols = team * 8;
  for (int c = threadIdx.x; c < H; c += blockDim.x) {
    float t = 0.f;
    for (int k = 0; k < (int)per_block; ++k) t += join[k * cols + c];
    out[c] = t;
  }
}

// dw[c] (+)= sum over blocks of partial[b][c].  A block takes 32 columns (whole
// 128-byte lines); its 128 groups of 8 lanes sum every 128th row, and the groups are
// joined in a fixed order.
constexpr int COLSUM_COLS = 32, COLSUM_GROUPS = 128;

__global__ __launch_bounds__(1024) void norm_colsum_kernel(const float* __restrict__ partial,
                                                           int blocks, int H,
                                                           float* __restrict__ dw, int accumulate) {
  __shared__ float s[COLSUM_GROUPS][COLSUM_COLS];
  __shared__ float s2[32][COLSUM_COLS];
  const int group = threadIdx.x / 8, c4 = (threadIdx.x % 8) * 4;
  const int c = blockIdx.x * COLSUM_COLS + c4;
  float t[4] = {0.f, 0.f, 0.f, 0.f};
  const bool vec = (H & 3) == 0;   // rows 16-byte aligned
#pragma unroll 4
  for (int b = group; b < blocks; b += COLSUM_GROUPS) {
    const float* p = partial + (int64_t)b * H + c;
    if (vec && c < H) {
      const f32x4 v = *(const f32x4*)p;
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] += v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < H) t[i] += p[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s[group][c4 + i] = t[i];
  __syncthreads();
  const int col = threadIdx.x % COLSUM_COLS, part = threadIdx.x / COLSUM_COLS;
  float a = 0.f;
#pragma unroll
  for (int k = 0; k < COLSUM_GROUPS / 32; ++k) a += s[part * (COLSUM_GROUPS / 32) + k][col];
  s2[part][col] = a;
  __syncthreads();
  const int out = blockIdx.x * COLSUM_COLS + col;
  if (part != 0 || out >= H) return;
  a = 0.f;
#pragma unroll
  for (int k = 0; k < 32; ++k) a += s2[k][col];
  dw[out] = accumulate ? dw[out] + a : a;
}

}  // namespace lora

namespace lora_host {
using namespace lora;

// The team of a row of H columns, the vectors a lane holds and the block.
struct NormPlan {
  int team, vpl, block;
};
static NormPlan norm_plan(int64_t H) {
  const int64_t vecs = cdiv(H, 8);
  if (vecs <= kWave) {
    int team = 4;   // at least the four lanes of a 32-column scale block
    while (team < vecs) team *= 2;
    return {team, 1, NORM_SMALL_BLOCK};
  }
  const int vpl = vecs <= 2 * 1024 ? 2 : NORM_MAX_VPL;
  const int team = (int)align_up(cdiv(vecs, vpl), kWave);
  return {team, vpl, team};
}

static unsigned norm_grid(int64_t n, const NormPlan& p, int64_t cap) {
  return (unsigned)std::max<int64_t>(1, std::min(cdiv(n, p.block / p.team), cap));
}

// Blocks of a pass that keeps nothing: 2^20 threads in all, more than run at once.
static unsigned norm_free_grid(int64_t n, const NormPlan& p) {
  return norm_grid(n, p, std::max<int64_t>(1, (1 << 20) / p.block));
}

// Blocks that keep dw partials: 2^17 threads in all (8 waves a CU), which the whole
// multiples of the CUs below raise to as many as 2^18.  The partials, written and read
// again, are 8 MB at 1024, 2048, 4096 and 8192 columns, 14 MB at 7168, 16 at 16384 and 32
// at 32768 (at 8192 x 4096 51.6 us; with twice the blocks 56.5, with half of them 69.7).  As
// many on every CU: rounded up to whole multiples of 256, or down where that would leave
// blocks without a row (2790 x 7168: 512 blocks 35.6 us, 256 43.0, 292 40.3; 500 x 7168:
// 256 blocks 13.6, 500 15.3).
int64_t rmsnorm_bwd_blocks(int64_t n, int64_t hidden) {
  const NormPlan p = norm_plan(hidden);
  const int64_t most = (1 << 17) / p.block, up = align_up(most, 256);
  return norm_grid(n, p, n >= up * (p.block / p.team) ? up : std::max<int64_t>(256, most / 256 * 256));
}

// Calls that move more than 96 MB, three eighths of the last-level cache, make
// non-temporal accesses: little of theirs would be found there again, and lines that
// others wrote are not pushed out under their reads.  Forward / backward at 8192 x
// 4096 (268 MB): 46.4 / 44.9 us, 50.0 / 50.5 with ordinary accesses; at 4096 rows 24.8 /
// 23.7 against 26.3 / 26.6; at 2048 rows (67 MB, inputs in the cache) 13.7 / 13.7
// against 12.2 / 13.0.
static bool norm_streams(int64_t n, int64_t H, int arrays) {
  return n * H * 2 * arrays > (int64_t)96 << 20;
}

template <int VPL, bool Q8>
static void fwd_launch(const NormPlan& p, unsigned grid, int64_t n, int64_t H, const uint16_t* x,
                       const uint16_t* res, const uint16_t* w, float eps, uint16_t* h, uint16_t* y,
                       uint8_t* q, uint8_t* qs, float* rstd, hipStream_t s) {
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(p.block), 0, s, n, (int)H, p.team, x, res, w, eps, h,
                       y, q, qs, rstd);
  };
  if (H % 8 != 0) go(rmsnorm_fwd_kernel<VPL, false, false, false>);
  else if (norm_streams(n, H, res ? 4 : 2)) go(rmsnorm_fwd_kernel<VPL, true, true, Q8>);
  else go(rmsnorm_fwd_kernel<VPL, true, false, Q8>);
}

lora_status launch_rmsnorm_fwd(int64_t n, int64_t H, const uint16_t* x, const uint16_t* res,
                               const uint16_t* w, float eps, uint16_t* h, uint16_t* y, uint8_t* q,
                               uint8_t* qs, float* rstd, hipStream_t s) {
  const NormPlan p = norm_plan(H);
  const unsigned grid = norm_free_grid(n, p);
  const auto go = [&](auto vpl) {
    constexpr int V = decltype(vpl)::value;
    if (q) fwd_launch<V, true>(p, grid, n, H, x, res, w, eps, h, y, q, qs, rstd, s);
    else fwd_launch<V, false>(p, grid, n, H, x, res, w, eps, h, y, q, qs, rstd, s);
  };
  if (p.vpl == 1) go(std::integral_constant<int, 1>{});
  else if (p.vpl == 2) go(std::integral_constant<int, 2>{});
  else go(std::integral_constant<int, NORM_MAX_VPL>{});
  return launch_check("rmsnorm_fwd");
}

template <int VPL>
static void bwd_launch(const NormPlan& p, unsigned grid, int64_t n, int64_t H, const uint16_t* dy,
                       const uint16_t* dh, const uint16_t* h, const uint16_t* w, const float* rstd,
                       uint16_t* dx, float* partial, hipStream_t s) {
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(p.block), 0, s, n, (int)H, p.team, dy, dh, h, w, rstd,
                       dx, partial);
  };
  if (H % 8 != 0) go(rmsnorm_bwd_kernel<VPL, false, false>);
  else if (norm_streams(n, H, dh ? 4 : 3)) go(rmsnorm_bwd_kernel<VPL, true, true>);
  else go(rmsnorm_bwd_kernel<VPL, true, false>);
}

lora_status launch_rmsnorm_bwd(int64_t n, int64_t H, const uint16_t* dy, const uint16_t* dh,
                               const uint16_t* h, const uint16_t* w, const float* rstd,
                               uint16_t* dx, float* dw, int accumulate, float* partial,
                               hipStream_t s) {
  const NormPlan p = norm_plan(H);
  const unsigned grid = dw ? (unsigned)rmsnorm_bwd_blocks(n, H) : norm_free_grid(n, p);
  float* part = dw ? partial : nullptr;
  if (p.vpl == 1) bwd_launch<1>(p, grid, n, H, dy, dh, h, w, rstd, dx, part, s);
  else if (p.vpl == 2) bwd_launch<2>(p, grid, n, H, dy, dh, h, w, rstd, dx, part, s);
  else bwd_launch<NORM_MAX_VPL>(p, grid, n, H, dy, dh, h, w, rstd, dx, part, s);
  lora_status st = launch_check("rmsnorm_bwd");
  if (st != LORA_OK || !dw) return st;
  hipLaunchKernelGGL(norm_colsum_kernel, dim3((unsigned)cdiv(H, COLSUM_COLS)), dim3(1024), 0, s, partial,
                     (int)grid, (int)H, dw, accumulate);
  return launch_check("norm_colsum");
}

}  // namespace lora_host
