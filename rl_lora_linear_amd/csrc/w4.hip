// Few-token products with 4-bit frozen weights on gfx950, plain and with the
// mixed-adapter LoRA delta, and the quantiser that lays the weights out.
//
//   W_ik = e2m1(code_ik) 2^(s_{i, k/32} - 127),   y_t = W x_t (+ s_a B_a A_a x_t).
//
// A wave takes 16 R weight rows, 16 T tokens and a slice of k; the block's
// eight waves split k and are joined through LDS in wave order.  Each lane
// reads 16 bytes of codes -- one scale's 32 weights -- turns them into bf16
// pairs with the conversion unit (exact: a 2-bit significand times a power of
// two) and feeds v_mfma_f32_16x16x32_bf16 four times.  k may be met in any order
// as long as weights and x agree, so lane group g of the MFMA simply takes
// scale block 4c + g and both operands load whole 16-byte pieces in memory
// order: no shuffle, no LDS on the way in.  8-bit x is widened to bf16 in
// registers (exact as well).  Sums are fp32 throughout, y is rounded once.
// The scaled 4-bit MFMA would take the codes as they are, but it aligns the 128
// products of a step to the largest of them and drops what lies ~2^-14 below.
#include "common.hpp"
#include "sgmv.hpp"

namespace lora {

constexpr int W4_WAVES = 8;
constexpr int W4_CHUNK = 128;   // k of one step: four scale blocks, one per lane group

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float e8m0(int byte) {   // 0 is 2^-127 (a subnormal), 255 is NaN
  return __int_as_float(byte == 0 ? 0x400000 : byte == 255 ? 0x7FC00000 : byte << 23);
}
// Codes 2i, 2i + 1 of four bytes as a bf16 pair, times 2^(byte - 127); `scale` has the
// scale byte as its exponent field.
template <int I>
__device__ __forceinline__ uint32_t w4_pair(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, I));
}
__device__ __forceinline__ bf16x8 w4_widen(uint32_t codes, float scale) {
  return as_bf16x8(make_uint4(w4_pair<0>(codes, scale), w4_pair<1>(codes, scale),
                              w4_pair<2>(codes, scale), w4_pair<3>(codes, scale)));
}
// Eight e4m3 codes (OCP) times `scale` as bf16.
__device__ __forceinline__ bf16x8 x8_widen(uint32_t lo, uint32_t hi, float scale) {
  uint32_t r[4];
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true));
  return as_bf16x8(make_uint4(r[0], r[1], r[2], r[3]));
}

// Where a token's adapter factors lie, resolved and checked by the shrink.
struct W4Token {
  int64_t b_off;
  int32_t rank;   // 0: no delta for this token
  int32_t pad;
};

// ------------------------------------------------------------------ shrink
// u_t = s_a A_a x_t in fp32, one wave per (token, rank row); rows past the
// adapter's rank and rows of tokens without one are zero.  Block (0, t) writes
// token t's W4Token; the grid together checks every descriptor of the table.
constexpr int W4S_WAVES = 4;

struct W4Adapters {
  const uint16_t* A_pack;
  const lora_adapter_desc* desc;
  const int32_t* ids;
  int64_t a_elems, b_elems;
  int32_t n_ad, max_rank, sorted;
};

__device__ __forceinline__ bool w4_desc_ok(const lora_adapter_desc& d, const W4Adapters& a, int d_in,
                                           int d_out) {
  const int64_t r = d.rank;
  return r >= 8 && r <= 64 && (r % 8) == 0 && r <= a.max_rank && d.a_off >= 0 && d.b_off >= 0 &&
         (d.a_off % 8) == 0 && (d.b_off % 8) == 0 && d.a_off + r * d_in <= a.a_elems &&
         d.b_off + r * d_out <= a.b_elems;
}

template <bool X8>
__global__ __launch_bounds__(64 * W4S_WAVES) void w4_shrink_kernel(
    int n, int d_in, int d_out, const void* __restrict__ x_, const uint8_t* __restrict__ xs,
    W4Adapters ad, float* __restrict__ u, W4Token* __restrict__ tok, int32_t* __restrict__ status) {
  const int lane = threadIdx.x & 63;
  const int j = blockIdx.x * W4S_WAVES + (threadIdx.x >> 6);   // rank row, wave-uniform
  const int t = blockIdx.y;
  const int64_t gid = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x;
  for (int64_t k = gid; k < ad.n_ad; k += (int64_t)gridDim.x * gridDim.y * blockDim.x) {
    const lora_adapter_desc d = ad.desc[k];
    if (d.rank != 0 && !w4_desc_ok(d, ad, d_in, d_out)) set_flag(status, LORA_FLAG_BAD_DESC);
  }
  const int id = ad.ids[t];
  lora_adapter_desc d{0, 0, 0, 0.f};
  if (id >= 0 && id < ad.n_ad) d = ad.desc[id];
  const bool on = d.rank != 0 && w4_desc_ok(d, ad, d_in, d_out);
  const int rank = on ? d.rank : 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    tok[t] = W4Token{on ? d.b_off : 0, rank, 0};
    if (id < 0 || id >= ad.n_ad) set_flag(status, LORA_FLAG_ID_RANGE);
    if (ad.sorted && t > 0 && ad.ids[t - 1] > id) set_flag(status, LORA_FLAG_UNSORTED);
  }
  if (j >= ad.max_rank) return;
  float s = 0.f;
  if (j < rank) {
    const uint16_t* a = ad.A_pack + d.a_off + (int64_t)j * d_in;
#pragma unroll 4
    for (int k = lane * 8; k < d_in; k += 512) {
      const uint4 av = *(const uint4*)(a + k);
      uint4 xv;
      if (X8) {
        const uint2 c = *(const uint2*)((const uint8_t*)x_ + (int64_t)t * d_in + k);
        const float sc = e8m0(xs[((int64_t)t * d_in + k) / 32]);
        const bf16x8 w = x8_widen(c.x, c.y, sc);
        xv = __builtin_bit_cast(uint4, w);
      } else {
        xv = *(const uint4*)((const uint16_t*)x_ + (int64_t)t * d_in + k);
      }
      const uint32_t aw[4] = {av.x, av.y, av.z, av.w}, xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        s += bf2f_lo(aw[q]) * bf2f_lo(xw[q]);
        s += bf2f_hi(aw[q]) * bf2f_hi(xw[q]);
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, kWave);
    s *= d.scale;
  }
  if (lane == 0) u[(int64_t)t * ad.max_rank + j] = s;
}

// ------------------------------------------------------------------ product
struct W4Delta {
  const uint16_t* B_pack;   // null: no adapters
  const float* u;
  const W4Token* tok;
  int32_t max_rank;
};

template <int R, int T, bool X8>
__global__ __launch_bounds__(64 * W4_WAVES) void w4_product_kernel(
    int n, int d_in, int d_out, const void* __restrict__ x_, const uint8_t* __restrict__ xs,
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, W4Delta dl,
    uint16_t* __restrict__ y) {
  extern __shared__ f32x4 join[];   // [W4_WAVES][R * T][64]
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int l = lane & 15, g = lane >> 4;
  const int row0 = blockIdx.x * 16 * R, tok0 = blockIdx.y * 16 * T;
  const int chunks = (d_in + W4_CHUNK - 1) / W4_CHUNK;
  const int per = (chunks + W4_WAVES - 1) / W4_WAVES;
  const int c0 = w * per, c1 = min(chunks, c0 + per);
  f32x4 acc[R][T];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};

#pragma unroll 2
  for (int c = c0; c < c1; ++c) {
    const int k = c * W4_CHUNK + g * 32;
    const bool kin = k < d_in;   // d_in is a multiple of 64: the last step may be half
    uint4 wc[R];
    float ws[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = row0 + 16 * i + l;
      wc[i] = kin ? *(const uint4*)(codes + (row * d_in + k) / 2) : make_uint4(0, 0, 0, 0);
      ws[i] = __int_as_float((kin ? (int)scales[(row * d_in + k) / 32] : 127) << 23);
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int64_t tk = tok0 + 16 * t + l;
      uint4 xv[4];
      if (tk < n && kin) {
        if (X8) {
          const uint4* p = (const uint4*)((const uint8_t*)x_ + tk * d_in + k);
          const float sc = e8m0(xs[(tk * d_in + k) / 32]);
          const uint4 a = p[0], b = p[1];
          xv[0] = __builtin_bit_cast(uint4, x8_widen(a.x, a.y, sc));
          xv[1] = __builtin_bit_cast(uint4, x8_widen(a.z, a.w, sc));
          xv[2] = __builtin_bit_cast(uint4, x8_widen(b.x, b.y, sc));
          xv[3] = __builtin_bit_cast(uint4, x8_widen(b.z, b.w, sc));
        } else {
          const uint4* p = (const uint4*)((const uint16_t*)x_ + tk * d_in + k);
#pragma unroll
          for (int q = 0; q < 4; ++q) xv[q] = p[q];
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) xv[q] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint32_t cw[4] = {wc[i].x, wc[i].y, wc[i].z, wc[i].w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[i][t] = mfma16(w4_widen(cw[q], ws[i]), as_bf16x8(xv[q]), acc[i][t]);
      }
    }
  }

  // the LoRA delta's part of wave w: rank columns 8w .. 8w + 7
  if (dl.B_pack) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int tk = tok0 + 16 * t + l;
      if (tk >= n) continue;
      const W4Token tm = dl.tok[tk];
      if (8 * w >= tm.rank) continue;
      const float4* up = (const float4*)(dl.u + (int64_t)tk * dl.max_rank + 8 * w);
      const float4 ua = up[0], ub = up[1];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t row = row0 + 16 * i + 4 * g + e;
          const uint4 b = *(const uint4*)(dl.B_pack + tm.b_off + row * tm.rank + 8 * w);
          float s = ua.x * bf2f_lo(b.x);
          s += ua.y * bf2f_hi(b.x);
          s += ua.z * bf2f_lo(b.y);
          s += ua.w * bf2f_hi(b.y);
          s += ub.x * bf2f_lo(b.z);
          s += ub.y * bf2f_hi(b.z);
          s += ub.z * bf2f_lo(b.w);
          s += ub.w * bf2f_hi(b.w);
          acc[i][t][e] += s;
        }
    }
  }

#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int t = 0; t < T; ++t) join[(w * R * T + i * T + t) * 64 + lane] = acc[i][t];
  __syncthreads();
  for (int it = threadIdx.x; it < R * T * 64; it += 64 * W4_WAVES) {
    f32x4 s = join[it];
#pragma unroll
    for (int v = 1; v < W4_WAVES; ++v) s += join[v * R * T * 64 + it];
    const int ln = it & 63, i = (it >> 6) / T, t = (it >> 6) % T;
    const int64_t tk = tok0 + 16 * t + (ln & 15);
    if (tk < n)
      *(uint2*)(y + tk * d_out + row0 + 16 * i + 4 * (ln >> 4)) =
          make_uint2(pack2bf(s[0], s[1]), pack2bf(s[2], s[3]));
  }
}

// ------------------------------------------------------------------ quantiser
// 32 weights per four lanes: the least power of two with max|w| <= 6 scale (no
// finite weight saturates), then the nearest e2m1 magnitude, ties to the even
// code.  NaN and +-Inf do not take part in the scale; NaN becomes 0.
__global__ __launch_bounds__(256) void w4_quantize_kernel(int64_t n8, const uint16_t* __restrict__ W,
                                                          uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  for (int64_t v0 = (int64_t)blockIdx.x * 256; v0 < n8; v0 += (int64_t)gridDim.x * 256) {
    const int64_t v = v0 + threadIdx.x;   // n8 is a multiple of 4: whole groups of lanes
    const bool on = v < n8;
    const uint4 a = on ? ((const uint4*)W)[v] : make_uint4(0, 0, 0, 0);
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
    float f[8];
    float mx = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[2 * q] = bf2f_lo(aw[q]);
      f[2 * q + 1] = bf2f_hi(aw[q]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float m = fabsf(f[i]);
      mx = (__builtin_isfinite(f[i]) && m > mx) ? m : mx;
    }
    mx = fmaxf(mx, __shfl_xor(mx, 1, kWave));
    mx = fmaxf(mx, __shfl_xor(mx, 2, kWave));
    const int bits = __float_as_int(mx);
    const int b = max((bits >> 23) - 2 + ((bits & 0x7FFFFF) > 0x400000 ? 1 : 0), 1);
    const float inv = __int_as_float((254 - b) << 23);
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float m = fabsf(f[i]) * inv;
      uint32_t c = (m > 0.25f) + (m >= 0.75f) + (m > 1.25f) + (m >= 1.75f) + (m > 2.5f) +
                   (m >= 3.5f) + (m > 5.f);
      if (f[i] < 0.f) c |= 8;
      out |= c << (4 * i);
    }
    if (on) {
      ((uint32_t*)codes)[v] = out;
      if ((threadIdx.x & 3) == 0) scales[v / 4] = (uint8_t)b;
    }
  }
}

}  // namespace lora

namespace lora_host {
using namespace lora;

lora_status launch_w4_quantize(const uint16_t* W, int64_t rows, int64_t cols, uint8_t* codes,
                               uint8_t* scales, hipStream_t s) {
  const int64_t n8 = rows * cols / 8;
  hipLaunchKernelGGL(w4_quantize_kernel, dim3((unsigned)std::min<int64_t>(cdiv(n8, 256), 8192)),
                     dim3(256), 0, s, n8, W, codes, scales);
  return launch_check("w4_quantize");
}

size_t w4_ws_bytes(int64_t n, int max_rank) {
  Carve cv(nullptr, 0);
  cv.take<int32_t>(64);
  cv.take<float>((size_t)n * max_rank);
  cv.take<W4Token>((size_t)n);
  return cv.used;
}

template <int R, int T, bool X8>
static lora_status product(int n, int d_in, int d_out, const void* x, const uint8_t* xs,
                           const uint8_t* codes, const uint8_t* scales, const W4Delta& dl,
                           uint16_t* y, hipStream_t s) {
  constexpr int lds = W4_WAVES * R * T * 64 * (int)sizeof(f32x4);
  static const hipError_t attr = hipFuncSetAttribute((const void*)w4_product_kernel<R, T, X8>,
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  TRY_HIP(attr);
  hipLaunchKernelGGL((w4_product_kernel<R, T, X8>),
                     dim3((unsigned)(d_out / (16 * R)), (unsigned)cdiv(n, 16 * T)),
                     dim3(64 * W4_WAVES), lds, s, n, d_in, d_out, x, xs, codes, scales, dl, y);
  return launch_check("w4_product");
}

template <bool X8>
static lora_status product_for(int n, int d_in, int d_out, const void* x, const uint8_t* xs,
                               const uint8_t* codes, const uint8_t* scales, const W4Delta& dl,
                               uint16_t* y, hipStream_t s) {
  if (n <= 16) return product<1, 1, X8>(n, d_in, d_out, x, xs, codes, scales, dl, y, s);
  if (n <= 32) return product<1, 2, X8>(n, d_in, d_out, x, xs, codes, scales, dl, y, s);
  if (n <= 64) return product<1, 4, X8>(n, d_in, d_out, x, xs, codes, scales, dl, y, s);
  return product<4, 4, X8>(n, d_in, d_out, x, xs, codes, scales, dl, y, s);
}

lora_status launch_w4_linear(int64_t n, int64_t d_in, int64_t d_out, const void* x,
                             const uint8_t* xs, const uint8_t* codes, const uint8_t* scales,
                             uint16_t* y, hipStream_t s) {
  const W4Delta none{};
  return xs ? product_for<true>((int)n, (int)d_in, (int)d_out, x, xs, codes, scales, none, y, s)
            : product_for<false>((int)n, (int)d_in, (int)d_out, x, xs, codes, scales, none, y, s);
}

lora_status launch_lora_w4(const lora_shape& sh, const void* x, const uint8_t* xs,
                           const uint8_t* codes, const uint8_t* scales, const uint16_t* A_pack,
                           const uint16_t* B_pack, const lora_adapter_desc* desc,
                           const int32_t* ids, uint16_t* y, void* ws, hipStream_t s) {
  const int n = (int)sh.n_tokens, d_in = (int)sh.d_in, d_out = (int)sh.d_out;
  Carve cv(ws, 0);
  int32_t* status = cv.take<int32_t>(64);
  float* u = cv.take<float>((size_t)n * sh.max_rank);
  W4Token* tok = cv.take<W4Token>((size_t)n);
  const W4Adapters ad{A_pack, desc, ids, sh.a_pack_elems, sh.b_pack_elems, sh.n_adapters, sh.max_rank,
                      sh.order == LORA_IDS_SORTED};
  const dim3 grid((unsigned)cdiv(sh.max_rank, W4S_WAVES), (unsigned)n);
  if (xs)
    hipLaunchKernelGGL(w4_shrink_kernel<true>, grid, dim3(64 * W4S_WAVES), 0, s, n, d_in, d_out, x,
                       xs, ad, u, tok, status);
  else
    hipLaunchKernelGGL(w4_shrink_kernel<false>, grid, dim3(64 * W4S_WAVES), 0, s, n, d_in, d_out, x,
                       xs, ad, u, tok, status);
  lora_status st = launch_check("w4_shrink");
  if (st != LORA_OK) return st;
  const W4Delta dl{B_pack, u, tok, sh.max_rank};
  return xs ? product_for<true>(n, d_in, d_out, x, xs, codes, scales, dl, y, s)
            : product_for<false>(n, d_in, d_out, x, xs, codes, scales, dl, y, s);
}

}  // namespace lora_host
