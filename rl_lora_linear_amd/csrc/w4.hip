// Few-token products with 4-bit frozen weights on gfx950, plain and with the
// mixed-adapter LoRA delta, and the quantiser that lays the weights out.
//
//   W_ik = e2m1(code_ik) 2^(s_{i, k/32} - 127),   y_t = W x_t (+ s_a B_a A_a x_t).
//
// One persistent block per CU keeps its tokens' x in registers as MFMA fragments and
// streams 16-row tiles of codes past it; the block's waves split k and are joined
// through LDS in wave order.  A lane turns 16 bytes of codes -- one scale's 32 weights
// -- into bf16 pairs with the conversion unit (exact for scale bytes up to 252: a 2-bit
// significand times a power of two, where that is below bf16's normal numbers a
// subnormal, which the matrix unit keeps) and feeds v_mfma_f32_16x16x32_bf16 four times.
// k may be met in any order as long as weights and x agree, so lane group g of the MFMA
// simply takes scale block 4 c + g and both operands are read as whole 16-byte pieces in
// memory order, without shuffles.  8-bit x is widened to bf16 in registers (exact for
// scale bytes 3 to 246; below, multiples of 2^-133).  Sums are fp32 throughout, y is
// rounded once.  The scaled 4-bit MFMA would take the codes as they are, but it aligns
// the 128 products of a step to the largest of them and drops what lies ~2^-14 below.
// Bound by the codes' bytes where there are many (one token's 151936 x 4096, 331 MB:
// 54 to 57 us, 5.8 to 6.1 TB/s of the 7.1 that plain reads reach), by launch, first
// access and the join where there are few (4096 x 4096 4.2 us, a launch alone 3.9;
// 12288 x 4096 8.6), by LDS traffic and conversions in large batches of long rows (64
// tokens 12288 -> 4096 17.1 us).  The adapters' shrink is a launch of its own, 3 us
// with one token; times in a captured graph.
#include "common.hpp"
#include "desc.hpp"
#include "sgmv.hpp"

namespace lora {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a),
                                         __builtin_bit_cast(bf16x2, b), c, false);
}
// Codes 2i, 2i + 1 of four bytes as a bf16 pair, times 2^(byte - 127); `scale` has the
// scale byte as its exponent field (the unit takes that field alone: 0 is 2^-127, 255 NaN);
// a value of 2^128 or more becomes infinite.
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
// Bound by reading A, eight 16-byte pieces a lane in flight: 64 tokens of 64 adapters
// with 12288 columns 10 us, 3.9 TB/s of distinct A (more waves that split k, or one
// wave for all tokens of an adapter, were slower).
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
  return desc_ok(d, a.max_rank, d_in, d_out, a.a_elems, a.b_elems);
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
  float s = 0.f, s1 = 0.f;
  if (j < rank) {
    const uint16_t* a = ad.A_pack + d.a_off + (int64_t)j * d_in;
#pragma unroll 8
    for (int k = lane * 8; k < d_in; k += 512) {
      const uint4 av = *(const uint4*)(a + k);
      uint4 xv;
      if (X8) {
        const uint2 c = *(const uint2*)((const uint8_t*)x_ + (int64_t)t * d_in + k);
        const float sc = __int_as_float((int)xs[((int64_t)t * d_in + k) / 32] << 23);
        xv = __builtin_bit_cast(uint4, x8_widen(c.x, c.y, sc));
      } else {
        xv = *(const uint4*)((const uint16_t*)x_ + (int64_t)t * d_in + k);
      }
      // two exact products and an fp32 sum per instruction
      s = dot2(av.x, xv.x, s);
      s1 = dot2(av.y, xv.y, s1);
      s = dot2(av.z, xv.z, s);
      s1 = dot2(av.w, xv.w, s1);
    }
    s += s1;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, kWave);
    s *= d.scale;
  }
  if (lane == 0) u[(int64_t)t * ad.max_rank + j] = s;
}

// ------------------------------------------------------------------ product
// One block per CU holds 16 tokens (32 where T is 2) and streams row tiles of 16 past
// them.  The waves split k in pieces of 256 columns ("pairs": two steps of four
// scale blocks): wave w keeps its pairs' x as MFMA fragments in registers for all
// of its tiles and moves its own pairs of codes through a ring of its own in LDS,
// so the pairs need no barrier.  LDS-DMA fills the ring two pairs ahead, five with
// eight waves (73 KB and more in flight per CU).  Loading the fragments straight into registers would
// touch 16 rows per quarter wave: the texture path then serves 16 bytes a clock,
// a quarter of what it does for the whole 128-byte lines that the DMA asks for.
// At the end of a tile the waves' sums are joined through LDS (one barrier); a
// wave owns one token's LoRA delta (two where a block has 8 waves or T is 2, four where
// it has 4), whose factor rows are one more ring entry.
constexpr int W4_PAIR = 256;                     // columns of one ring entry
// Up to four tokens read x's fragments straight from memory (bf16 4096 -> 12288: one
// token 8.7 us, through LDS 9.5; 8 -> 9.4 and 9.6, 16 -> 10.7 and 10.0; in 8 bits four
// tokens 9.3 and 9.1).
constexpr int W4_DIRECT_TOKENS = 4;
constexpr int W4_SCALES = 2048;                  // entry: 16 rows x 128 B of codes, then
constexpr int W4_ENTRY = 2048 + 256;             // 16 rows x 12 B holding 8 B of scales
// LDS of a block of NW waves in TEAMS teams and T token tiles: the rings ([slot][wave]),
// the waves' sums (of two rounds in turn where T is 1), the deltas likewise; at the end
// the tokens' u.  Before the rings start, x passes through all before u but the first
// EARLY slots, which fill meanwhile: as many as leave the number of x's rounds as it is (16
// tokens in 8 bits 4096 -> 12288 9.4 us, 10.0 with the rings begun after x).
// LONG: an entry holds its pair's x too.
template <int NW, int TEAMS, int P, int T, bool X8, bool LONG>
struct W4Lds {
  static constexpr int X_PAIR = 16 * W4_PAIR * (X8 ? 1 : 2);   // bytes of a pair of 16 tokens' x
  static constexpr int ENTRY = W4_ENTRY + (LONG ? X_PAIR + (X8 ? 256 : 0) : 0);
  static constexpr int OPS = 3 + (LONG ? X_PAIR / 1024 + X8 : 0);   // DMA instructions per entry
  static constexpr int DEPTH = LONG ? (X8 ? 5 : 3) : 48 / NW;  // entries per wave
  static constexpr int SLOT = NW * ENTRY;
  static constexpr int TURNS = T == 1 ? 2 : 1;
  static constexpr int JOIN = DEPTH * SLOT;                    // [TURNS][NW][T][64] f32x4
  static constexpr int DELTA = JOIN + TURNS * NW * T * 64 * 16;
                                                               // [TURNS][TEAMS][16 T tokens][16 rows] f32
  static constexpr int END = DELTA + TURNS * TEAMS * T * 16 * 16 * 4;
  static constexpr int BYTES = 160 * 1024;                     // one block a CU
  static constexpr int U = BYTES - T * 16 * 64 * 4;            // [16 T tokens][64] f32
  static constexpr int x_pairs(int early) { return std::min((U - early * SLOT) / NW / X_PAIR, T * P); }
  static constexpr int x_rounds(int early) {
    return x_pairs(early) > 0 ? (T * P + x_pairs(early) - 1) / x_pairs(early) : 1 << 20;
  }
  static constexpr int early() {
    int e = 0;
    while (e < DEPTH && x_rounds(e + 1) == x_rounds(0)) ++e;
    return e;
  }
  static constexpr int EARLY = early();
  static constexpr int X_PAIRS = x_pairs(EARLY);
  static_assert(END <= U && (LONG || (X_PAIRS > 0 && EARLY * SLOT + NW * X_PAIRS * X_PAIR <= U)));
};

struct W4Delta {
  const uint16_t* B_pack;   // null: no adapters
  const float* u;
  const W4Token* tok;
  int32_t max_rank;
};

__device__ __forceinline__ uint32_t lds_at(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
// One LDS-DMA per lane, global (base + voff) -> LDS (m0v + lane * size).
__device__ __forceinline__ void dma16(uint32_t voff, const void* base, uint32_t m0v) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(m0v), "v"(voff), "s"(base)
               : "memory");
}
__device__ __forceinline__ void dma16_nt(uint32_t voff, const void* base, uint32_t m0v) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(m0v), "v"(voff), "s"(base)
               : "memory");
}
__device__ __forceinline__ void dma4(uint32_t voff, const void* base, uint32_t m0v) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, %2" ::"s"(m0v), "v"(voff), "s"(base)
               : "memory");
}
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}
struct W4Args {
  const uint8_t* x;        // bf16, or e4m3 codes
  const uint8_t* xs;
  const uint8_t* codes;
  const uint8_t* scales;
  uint16_t* y;
  W4Delta dl;
  int32_t n, d_in, d_out;
  int32_t row_blocks;      // blocks that split the row tiles; the grid is these times the token tiles
};

// NW waves, each holding the x of P pairs of 16 T tokens.  The waves form TEAMS teams
// that take a row tile each at a time and split k among themselves.  LONG: d_in beyond
// what the waves can hold of x; a pair's x then comes through the ring with its codes,
// for every tile again.  DELTA: with adapters.  STREAM: the codes are read
// non-temporally, see product_for.
template <int NW, int TEAMS, int P, int T, bool X8, bool LONG, bool DELTA, bool STREAM = false>
__global__ __launch_bounds__(64 * NW) void w4_product_kernel(W4Args a) {
  using M = W4Lds<NW, TEAMS, P, T, X8, LONG>;
  __shared__ __attribute__((aligned(16))) char lds[M::BYTES];
  constexpr int WT = NW / TEAMS;                 // waves of a team
  constexpr int TOKS = (16 * T + WT - 1) / WT;   // tokens whose delta a wave owns
  static_assert(!LONG || T == 1);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & 15, g = lane >> 4, team = wave / WT, w = wave % WT;
  // this block's rounds of TEAMS tiles: rb, rb + row_blocks, ... (blocks that run
  // together read neighbouring rows)
  const int rb = blockIdx.x % a.row_blocks, tok0 = (blockIdx.x / a.row_blocks) * 16 * T;
  const int n_tiles = (a.d_out / (16 * TEAMS) - rb + a.row_blocks - 1) / a.row_blocks;
  const int toks = min(a.n - tok0, 16 * T);
  const int half = a.d_in / 2;          // bytes of a row of codes
  const int blocks = a.d_in / 32;       // scale bytes of a row
  const int pairs = (a.d_in + W4_PAIR - 1) / W4_PAIR;
  // this wave's pairs: w P .. w P + P - 1; LONG: w, w + WT, ...
  const int mine = LONG ? (pairs - w + WT - 1) / WT : min(max(pairs - w * P, 0), P);

  // The adapters of the delta's tokens, w + i WT, and their u are asked for before all
  // else: nothing waits for them until the first delta.
  float* u = (float*)(lds + M::U);
  i32x4 tm[TOKS];   // W4Token, by scalar loads
#pragma unroll
  for (int i = 0; i < TOKS; ++i) {
    const int t = w + i * WT;
    tm[i] = i32x4{0, 0, 0, 0};
    if (DELTA && t < toks) {
      tm[i] = ((const __attribute__((address_space(4))) i32x4*)(uintptr_t)a.dl.tok)[tok0 + t];
      dma4(min(lane, a.dl.max_rank - 1) * 4, a.dl.u + (int64_t)(tok0 + t) * a.dl.max_rank,
           lds_at(u + t * 64));
    }
  }

  // x fragments: lane (l, g) of chunk h of a pair holds scale block 8 q + 4 h + g of
  // token l of a token tile.  Lanes past the last token take the last one's (their
  // columns of the product are separate and never stored); blocks past d_in are zeros.
  bf16x8 xf[T][P][2][4];
  auto put_x = [&](int t, int i, int h, bool in, const uint4* v, float sc) {
    if constexpr (X8) {
      xf[t][i][h][0] = x8_widen(v[0].x, v[0].y, sc);
      xf[t][i][h][1] = x8_widen(v[0].z, v[0].w, sc);
      xf[t][i][h][2] = x8_widen(v[1].x, v[1].y, sc);
      xf[t][i][h][3] = x8_widen(v[1].z, v[1].w, sc);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) xf[t][i][h][q] = as_bf16x8(v[q]);
    }
    if (!in) {
#pragma unroll
      for (int q = 0; q < 4; ++q) xf[t][i][h][q] = as_bf16x8(make_uint4(0, 0, 0, 0));
    }
  };
  constexpr int XB = X8 ? 32 : 64;      // bytes of a scale block of x
  auto x_scale = [&](int64_t t, int blk) {
    return X8 ? __int_as_float((int)a.xs[t * blocks + blk] << 23) : 1.f;
  };
  auto load_x = [&]() {                 // straight from memory
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int64_t tk = tok0 + min(16 * t + l, toks - 1);
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int blk = (w * P + i) * 8 + h * 4 + g;
          const int at = min(blk, blocks - 1);
          const uint4* p = (const uint4*)(a.x + (tk * blocks + at) * XB);
          uint4 v[XB / 16];
#pragma unroll
          for (int q = 0; q < XB / 16; ++q) v[q] = p[q];
          put_x(t, i, h, blk < blocks, v, x_scale(tk, at));
        }
    }
  };
  constexpr int PIECES = 8 * XB / 16;   // 16-byte pieces of a token's x in a pair
  constexpr int X_ROWS = kWave / PIECES;   // tokens that one instruction fetches of
  // piece (h, k) of token l in a pair's x in LDS: swizzled by token so that the 16 lanes
  // of a group read 16 different banks
  auto x_piece = [&](const char* mem, int h, int k) {
    return *(const uint4*)(mem + (l * PIECES + (((h * 4 + g) * (XB / 16) + k) ^ l)) * 16);
  };
  const uint32_t x_end = (uint32_t)blocks * XB - 16;
  // what this lane fetches of pair q by the instruction for tokens m X_ROWS ..
  auto x_off = [&](int t0, int m, int q) {
    const int t = m * X_ROWS + lane / PIECES;
    return min(t0 + t, toks - 1) * (uint32_t)(blocks * XB) +
           min((uint32_t)(q * PIECES + ((lane % PIECES) ^ t)) * 16, x_end);
  };
  const uint8_t* xbase = a.x + (int64_t)tok0 * blocks * XB;
  // x's scales (LONG): the words that hold a token's 8 bytes, wherever they begin
  const uint32_t xs_low = X8 && LONG ? (uint32_t)(uintptr_t)(a.xs + (int64_t)tok0 * blocks) & 3 : 0;
  const uint8_t* xsbase = a.xs + (int64_t)tok0 * blocks - xs_low;

  char* ring = lds + wave * M::ENTRY;
  const uint32_t ring0 = lds_at(ring);
  // what this lane fetches of an entry: the 16-byte pieces of row r8 (+ 8) that its
  // slot holds (pieces are swizzled by row, see lds_sw), and a word of scales
  const uint32_t r8 = lane >> 3;
  const uint32_t off0 = r8 * half + ((lane & 7) ^ lds_sw(r8)) * 16;
  const uint32_t off1 = (r8 + 8) * half + ((lane & 7) ^ lds_sw(r8 + 8)) * 16;
  const int srow = min(lane / 3, 15);
  const uint32_t soff = ((srow * blocks) & ~3) + min(lane - srow * 3, 2) * 4;
  const uint32_t xsoff = ((min(srow, toks - 1) * blocks + xs_low) & ~3) + min(lane - srow * 3, 2) * 4;
  const uint32_t xs_end = (toks * blocks - 1 + xs_low) & ~3;
  int rank[TOKS];
  const uint16_t* B[TOKS];
  int per_tile = mine, total = mine * n_tiles;     // (deltas are added below)
  int it = 0, ij = 0, issued = 0;                  // the next entry to issue
  uint32_t islot = ring0;
  const uint8_t* cbase = a.codes + (int64_t)(rb * TEAMS + team) * 16 * half;
  const uint8_t* sbase = a.scales + (int64_t)(rb * TEAMS + team) * 16 * blocks;
  const int64_t cstep = (int64_t)a.row_blocks * TEAMS * 16 * half;
  const int64_t sstep = (int64_t)a.row_blocks * TEAMS * 16 * blocks;
  const uint32_t row_end = half - 16, scale_end = 16 * blocks - 4;
  auto issue_next = [&]() {
    if (!DELTA || ij < mine) {
      const uint32_t q = LONG ? ij * WT + w : w * P + ij;
      // (pieces past the row's end take its last one: their x is zero)
      const uint32_t v0 = min(off0 + q * 128, r8 * half + row_end);
      const uint32_t v1 = min(off1 + q * 128, (r8 + 8) * half + row_end);
      if (STREAM) {
        dma16_nt(v0, cbase, islot);
        dma16_nt(v1, cbase, islot + 1024);
      } else {
        dma16(v0, cbase, islot);
        dma16(v1, cbase, islot + 1024);
      }
      dma4(min(soff + q * 8, scale_end), sbase, islot + W4_SCALES);
      if (LONG) {
#pragma unroll
        for (int m = 0; m < 16 / X_ROWS; ++m) dma16(x_off(0, m, q), xbase, islot + W4_ENTRY + m * 1024);
        if (X8) dma4(min(xsoff + q * 8, xs_end), xsbase, islot + W4_ENTRY + M::X_PAIR);
      }
    } else {   // a token's 16 factor rows: at most 2 KB
      int r = 0, left = ij - mine;
      const uint16_t* b = nullptr;
#pragma unroll
      for (int i = 0; i < TOKS; ++i) {   // the wave's token with `left` others before it
        if (rank[i] != 0 && left-- == 0) {
          r = rank[i];
          b = B[i];
        }
      }
      const uint16_t* base = b + ((rb + (int64_t)it * a.row_blocks) * TEAMS + team) * 16 * r;
      dma16(min(lane * 16, r * 32 - 16), base, islot);
      dma16(min(lane * 16 + 1024, r * 32 - 16), base, islot + 1024);
#pragma unroll
      for (int i = 2; i < M::OPS; ++i) dma4(0, base, islot + W4_SCALES);   // (an entry's count)
    }
    ++issued;
    islot = islot == ring0 + (M::DEPTH - 1) * M::SLOT ? ring0 : islot + M::SLOT;
    const bool wrap = ++ij == per_tile;
    ij = wrap ? 0 : ij;
    it += wrap ? 1 : 0;
    cbase += wrap ? cstep : 0;
    sbase += wrap ? sstep : 0;
  };
  // the first tile's codes are on their way before the adapters are looked up
  if (DELTA) {
    per_tile = mine + TOKS;   // (no next tile yet)
    total = min(total, mine);
  }
  // through LDS, some pairs at a time: whole lines of a token's row
  auto stage_x = [&](auto&& meanwhile) {
    constexpr int PAIR = M::X_PAIR, ROUND = M::X_PAIRS;
    char* mem = lds + M::EARLY * M::SLOT + wave * (ROUND * PAIR);
    const uint32_t m0v = lds_at(mem);
#pragma unroll
    for (int i0 = 0; i0 < T * P; i0 += ROUND) {
#pragma unroll
      for (int i = i0; i < T * P && i < i0 + ROUND; ++i)
#pragma unroll
        for (int m = 0; m < 16 / X_ROWS; ++m)
          dma16(x_off(i / P * 16, m, w * P + i % P), xbase, m0v + (i - i0) * PAIR + m * 1024);
      if (i0 == 0 && meanwhile())
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(M::OPS * M::EARLY) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
      for (int i = i0; i < T * P && i < i0 + ROUND; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int blk = (w * P + i % P) * 8 + h * 4 + g;
          uint4 v[XB / 16];
#pragma unroll
          for (int k = 0; k < XB / 16; ++k) v[k] = x_piece(mem + (i - i0) * PAIR, h, k);
          put_x(i / P, i % P, h, blk < blocks, v,
                x_scale(tok0 + min(i / P * 16 + l, toks - 1), min(blk, blocks - 1)));
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
    asm volatile("s_barrier" ::: "memory");        // the rings overlap other waves' parts
  };
  const bool staged = !LONG && toks > W4_DIRECT_TOKENS;
  if (staged)
    stage_x([&]() {
      while (issued < M::EARLY && issued < total) issue_next();
      return issued == M::EARLY;
    });
  while (issued < M::DEPTH && issued < total) issue_next();

  int deltas = 0;
  float* delta = (float*)(lds + M::DELTA);
#pragma unroll
  for (int i = 0; i < TOKS; ++i) {
    const int t = w + i * WT;
    rank[i] = __builtin_amdgcn_readfirstlane(tm[i][2]);
    B[i] = a.dl.B_pack + uniform64((int64_t)(uint32_t)tm[i][0] | (int64_t)tm[i][1] << 32);
    deltas += rank[i] > 0 ? 1 : 0;
    if (DELTA && t < 16 * T && lane < 16 * M::TURNS)   // zeros stay where a token has no delta
      delta[(((lane >> 4) * TEAMS + team) * 16 * T + t) * 16 + (lane & 15)] = 0.f;
  }
  per_tile = mine + deltas;
  if (DELTA) {
    if (ij == per_tile) {   // no delta here
      ij = 0;
      ++it;
      cbase += cstep;
      sbase += sstep;
    }
    total = per_tile * n_tiles;
    while (issued < M::DEPTH && issued < total) issue_next();
  }
  if (!LONG && !staged) {
    load_x();
    // x has landed here, by a vmcnt(0) that the compiler sees: a wait of its own at the
    // first use, in the loop, would drain the ring there in every round
    __builtin_amdgcn_s_waitcnt(0x0F70);
  }

  float* join = (float*)(lds + M::JOIN);
  const char* e = ring;
  // Before an entry is read: while entries remain to be issued, exactly DEPTH - 1
  // younger ones are in flight; at the end all that remain are waited for.  FULL: all
  // of the tile's pairs are there and as many entries remain to be issued.
  auto wait_entry = [&](bool full) {
    if (full || issued < total)
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(M::OPS * (M::DEPTH - 1)) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  };
  auto next_entry = [&](bool full) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before the slot is refilled
    e = e == ring + (M::DEPTH - 1) * M::SLOT ? ring : e + M::SLOT;
    if (full || issued < total) issue_next();
  };
  // teams: a pair's sum by itself, see the join
  constexpr int SUMS = TEAMS > 1 ? P : 1;
  f32x4 acc[SUMS][T][2];
  auto take_pair = [&](int i, int q, bool full) {
    wait_entry(full);
    uint4 cw[2];
    int sc[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      cw[h] = *(const uint4*)(e + (l * 8 + ((4 * h + g) ^ lds_sw(l))) * 16);
      // a row's own bytes only: those past its end may be another row's NaN
      sc[h] = *(const uint8_t*)(e + W4_SCALES + l * 12 + ((l * blocks) & 2) +
                                min(4 * h + g, blocks - 1 - q * 8));
      if (LONG) {
        const int blk = q * 8 + 4 * h + g;
        uint4 v[XB / 16];
#pragma unroll
        for (int k = 0; k < XB / 16; ++k) v[k] = x_piece(e + W4_ENTRY, h, k);
        float xsc = 1.f;
        if (X8)
          xsc = __int_as_float(
              (int)*(const uint8_t*)(e + W4_ENTRY + M::X_PAIR + l * 12 +
                                     ((min(l, toks - 1) * blocks + xs_low) & 3) + 4 * h + g) << 23);
        put_x(0, 0, h, blk < blocks, v, xsc);
      }
    }
    next_entry(full);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t code[4] = {cw[h].x, cw[h].y, cw[h].z, cw[h].w};
        const bf16x8 wf = w4_widen(code[k], __int_as_float(sc[h] << 23));
#pragma unroll
        for (int t = 0; t < T; ++t) {
          f32x4& c = acc[SUMS > 1 ? i : 0][t][h];
          c = mfma16(wf, xf[t][LONG ? 0 : i][h][k], c);
        }
      }
  };
  for (int tile = 0; tile < n_tiles; ++tile) {
    const int turn = M::TURNS == 2 ? tile & 1 : 0;
#pragma unroll
    for (int i = 0; i < SUMS * T * 2; ++i) acc[i / (2 * T)][i / 2 % T][i % 2] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (!LONG && mine == P && issued + per_tile <= total) {
#pragma unroll
      for (int i = 0; i < P; ++i) take_pair(i, w * P + i, true);
    } else if (LONG) {
      for (int i = 0; i < mine; ++i) take_pair(0, i * WT + w, false);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (i >= mine) break;
        take_pair(i, w * P + i, false);
      }
    }
    if (DELTA) {
#pragma unroll
      for (int i = 0; i < TOKS; ++i) {
        // a token's delta: four lanes a row, 8 ranks and the 8 that lie 32 further each
        if (rank[i] == 0) continue;
        wait_entry(false);
        const int row = lane >> 2, j = (lane & 3) * 8;
        const float* ui = u + (w + i * WT) * 64;
        float s = 0.f;
#pragma unroll 1
        for (int k = j; k < rank[i]; k += 32) {
          const uint4 b = *(const uint4*)(e + (row * rank[i] + k) * 2);
          const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            s += ui[k + 2 * q] * bf2f_lo(bw[q]);
            s += ui[k + 2 * q + 1] * bf2f_hi(bw[q]);
          }
        }
        next_entry(false);
        s += __shfl_xor(s, 1, kWave);
        s += __shfl_xor(s, 2, kWave);
        if ((lane & 3) == 0) delta[((turn * TEAMS + team) * 16 * T + w + i * WT) * 16 + row] = s;
      }
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
      f32x4 sum = acc[0][t][0] + acc[0][t][1];
#pragma unroll
      for (int i = 1; i < SUMS; ++i) sum += acc[i][t][0] + acc[i][t][1];
      ((f32x4*)join)[((turn * NW + wave) * T + t) * 64 + lane] = sum;
    }
    // writes of this tile visible to all; the other buffer is free again after it.
    // The DMA in flight is not waited for.
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    // output 64 (w % 4) + lane of a team's token tile: accumulator lane i / 4's row i % 4
    static_assert(WT >= 4 * T, "waves to sum a team's tiles");
    if (w < 4 * T) {
      const int t = w / 4, i = (w % 4) * 64 + lane, al = i >> 2;
      const float* p = join + ((turn * NW + team * WT) * T + t) * 256 + i;
      // Waves of one pair are added two and two, as a wave of two teams adds its two pairs:
      // a token's sum has one order for a given d_in, whatever the batch.
      constexpr int STEP = P == 1 && !LONG ? 2 : 1;
      float s = 0.f;
#pragma unroll 4
      for (int v = 0; v < WT; v += STEP) s += STEP == 2 ? p[v * T * 256] + p[(v + 1) * T * 256] : p[v * T * 256];
      const int tk = 16 * t + (al & 15), row = 4 * (al >> 4) + (i & 3);
      if (DELTA) s += delta[((turn * TEAMS + team) * 16 * T + tk) * 16 + row];
      const float s1 = __shfl_xor(s, 1, kWave);
      const int64_t tile_row = ((int64_t)(rb + tile * a.row_blocks) * TEAMS + team) * 16;
      if ((lane & 1) == 0 && tk < toks)
        *(uint32_t*)(a.y + (int64_t)(tok0 + tk) * a.d_out + tile_row + row) = pack2bf(s, s1);
    }
    if (M::TURNS == 1) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }
}

// ------------------------------------------------------------------ quantiser
// 32 weights per four lanes: the least power of two with max|w| <= 6 scale (no
// finite weight saturates), then the nearest e2m1 magnitude, ties to the even
// code.  NaN and +-Inf do not take part in the scale; NaN becomes 0.  Run once per
// frozen matrix: 151936 x 4096 392 us (4.0 TB/s read and written), 12288 x 4096 34.5.
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

template <int NW, int TEAMS, int P, int T, bool X8, bool LONG, bool DELTA, bool STREAM = false>
static lora_status product(W4Args a, hipStream_t s) {
  // One block per CU: the token tiles times as many row blocks as that leaves, a
  // multiple of 8 (the XCDs) where there is more than one token tile, so that the
  // token tiles of the same rows share an XCD's L2.
  const int64_t tok_tiles = cdiv(a.n, 16 * T);
  int64_t rb = std::max<int64_t>(1, device_cus() / tok_tiles);
  if (tok_tiles > 1 && rb >= 8) rb &= ~(int64_t)7;
  a.row_blocks = (int)std::min<int64_t>(rb, a.d_out / (16 * TEAMS));
  hipLaunchKernelGGL((w4_product_kernel<NW, TEAMS, P, T, X8, LONG, DELTA, STREAM>),
                     dim3((unsigned)(a.row_blocks * tok_tiles)), dim3(64 * NW), 0, s, a);
  return launch_check("w4_product");
}

// The fewest registers of x that hold d_in: 16 waves with one or two pairs each, 8 with
// five or six (64 tokens 10240 -> 5120: five 17.9 us, six 19.0).  Where one pair leaves
// room, a block takes two token tiles from 81 tokens on: half the blocks would read and
// convert the codes twice (256 tokens 4096 -> 12288 39.1 us against 47.9; 96 19.9
// against 22.6), but fewer tokens leave them too few row tiles (48 tokens 14.6 against
// 14.1, with 64 adapters 27.5 against 24.5).  Longer rows stream x (one token 14336 ->
// 4096 10.2 us, 64 tokens 32; kept in registers phase by phase 11.5 and 66), which reads
// x again for every tile: at 12288 -> 4096 1, 16 and 64 tokens take 9.3, 10.0 and 28.2 us
// so and 10.0, 12.1 and 17.2 from registers.  The choice has to follow from d_in alone: it
// sets the order of a token's sum.
template <bool X8, bool DELTA>
static lora_status product_for(const W4Args& a, hipStream_t s) {
  const int64_t pairs = cdiv(a.d_in, W4_PAIR);
  // Codes of more than 96 MB, three eighths of the last-level cache, are read
  // non-temporally where one token tile reads them once: 151936 x 4096 54.2 us against
  // 60.8, 32768 x 8192 28.3 against 30.6; 12288 x 4096 (25 MB, found in that cache) 9.2
  // against 8.8.
  const bool streams = !DELTA && a.n <= 16 && (int64_t)a.d_out * a.d_in / 2 > (int64_t)96 << 20;
  // Up to 2048 columns one row tile would leave half of the waves without a pair: two
  // teams take two tiles, where there are more tiles than CUs (one token 1024 -> 49152
  // 9.5 us against 13.0, 2048 -> 49152 12.3 against 13.9; 64 tokens 2048 -> 25600 16.9
  // against 21.1; 2048 -> 4096, 256 tiles, 4.2 against 4.0), and up to 1024 columns four
  // (64 tokens 1024 -> 25600 11.7 against 13.5 with two; two token tiles as well serve
  // more than 80 tokens better: 256 28.2 against 29.3).  With adapters a wave of two teams
  // has two tokens' deltas, which sixteen tokens do not gain from (2048 -> 12288 14.7 us
  // against 13.7; 64 tokens 1024 -> 25600 35.2 against 39.0), and with two token tiles four,
  // for which the registers do not suffice.
  const int64_t tiles = a.d_out / 16 * cdiv(a.n, 16);
  if constexpr (!DELTA) {
    if (pairs <= 4 && !streams && a.n <= 80 && tiles > 2 * device_cus())
      return product<16, 4, 1, 1, X8, false, false>(a, s);
    if (streams && pairs <= 8) return product<16, 2, 1, 1, X8, false, false, true>(a, s);
    if (streams && pairs <= 16) {
      // up to 4096 columns two teams halve the rounds (one token's 151936 x 4096 57.0 us
      // against 60.3), but read x twice (sixteen tokens 67.0 against 63.0)
      return a.n <= W4_DIRECT_TOKENS ? product<16, 2, 2, 1, X8, false, false, true>(a, s)
                                     : product<16, 1, 1, 1, X8, false, false, true>(a, s);
    }
    if (streams && pairs <= 32) return product<16, 1, 2, 1, X8, false, false, true>(a, s);
  }
  if (pairs <= 8 && tiles > device_cus()) {
    if (a.n <= 80 && (!DELTA || a.n > 16)) return product<16, 2, 1, 1, X8, false, DELTA>(a, s);
    if constexpr (!DELTA)
      if (a.n > 80) return product<16, 2, 1, 2, X8, false, false>(a, s);
  }
  if (pairs <= 16)
    return a.n > 80 ? product<16, 1, 1, 2, X8, false, DELTA>(a, s)
                    : product<16, 1, 1, 1, X8, false, DELTA>(a, s);
  if (pairs <= 32) return product<16, 1, 2, 1, X8, false, DELTA>(a, s);
  if (pairs <= 40) return product<8, 1, 5, 1, X8, false, DELTA>(a, s);
  if (pairs <= 48) return product<8, 1, 6, 1, X8, false, DELTA>(a, s);
  return product<4, 1, 1, 1, X8, true, DELTA>(a, s);
}

static lora_status launch_product(int64_t n, int64_t d_in, int64_t d_out, const void* x,
                                  const uint8_t* xs, const uint8_t* codes, const uint8_t* scales,
                                  const W4Delta& dl, uint16_t* y, hipStream_t s) {
  const W4Args a{(const uint8_t*)x, xs, codes, scales, y, dl, (int)n, (int)d_in, (int)d_out, 0};
  if (dl.B_pack) return xs ? product_for<true, true>(a, s) : product_for<false, true>(a, s);
  return xs ? product_for<true, false>(a, s) : product_for<false, false>(a, s);
}

lora_status launch_w4_linear(int64_t n, int64_t d_in, int64_t d_out, const void* x,
                             const uint8_t* xs, const uint8_t* codes, const uint8_t* scales,
                             uint16_t* y, hipStream_t s) {
  return launch_product(n, d_in, d_out, x, xs, codes, scales, W4Delta{}, y, s);
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
  return launch_product(n, d_in, d_out, x, xs, codes, scales, dl, y, s);
}

}  // namespace lora_host
