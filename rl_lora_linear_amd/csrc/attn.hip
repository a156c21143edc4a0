// Attention over packed prompts on gfx950, forward and backward.
//
//   s_ij = scale q_i.k_j over the keys that query i sees, lse_i = log sum_j exp(s_ij),
//   p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j;
//   ds_ij = p_ij (do_i.v_j - delta_i),  delta_i = do_i.o_i,
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i.
//
// All three kernels have one form.  A wave owns 32 rows of one side (queries, or keys for
// dk and dv) as columns of v_mfma_f32_32x32x16_bf16, its operands of them in registers;
// the other side passes in tiles through LDS.  The first product's result X (S^T, dP^T, S,
// dP) then has a wave's own row in each lane: lane (l, h) = (lane & 31, lane >> 5) holds
// column l and rows 8 (r / 4) + 4 h + r % 4 of the 32.  As bf16, eight of these in turn are
// already an operand of the second product (O^T += V^T P^T, dQ^T += K^T dS^T, dV^T +=
// dO^T P, dK^T += Q^T dS): the sum over the tile's rows may run in any order, so its place
// 8 h + j stands for row 8 (j / 4) + 4 h + j % 4, and the other operand is read from LDS in
// that order by transposing reads.  Nothing is shuffled between lanes but a row's maximum.
// The rows of a result are a lane's own column, so maxima, sums, lse and delta apply
// without a broadcast.
// dk and dv, and dq, are made by two kernels that each recompute the scores (7 products in
// place of 5): every sum then has one owner and a fixed order, with no atomics and no
// partial results in memory.  (Adding dq up from the key side would write and read fp32 dq
// once for each 128 keys, and in an order that changes.)
// Roundings: s, lse, delta and all sums are fp32; p and ds are rounded to bf16 where they
// become operands (half a step, 2^-8 of a weight or less, signs as they come), as the
// matrix instruction asks; outputs once at the end.
#include <type_traits>

#include "attn.hpp"

namespace lora {

constexpr float AT_LOG2E = 1.4426950408889634f, AT_LN2 = 0.6931471805599453f;
constexpr int AT_TILE = 64;   // rows of a tile in LDS

struct AttnArgs {
  const uint16_t *q, *k, *v, *o, *dout;
  uint16_t *out, *dq, *dk, *dv;
  float* lse;     // [heads][n_q]
  float* stats;   // [heads][2][n_q]: lse in powers of two, delta; from the dq kernel for the other
  const int32_t *cu_q, *cu_k;
  int32_t* status;
  int64_t q_stride, k_stride, v_stride, o_stride, n_q, n_k;
  int32_t n_seqs, n_heads, n_kv, group, causal, tiles;
  int32_t wpr, shift;   // forward: waves of a block in one head; log2 of its rows
  float scale, scale_log2;
};

// A block's sequence and tile of 2^shift rows, from its number and the offsets alone: the
// n_rows / 2^shift + n_seqs numbers of a launch are enough for any offsets, and a number that
// is left over has nothing to do.
struct AttnSeq {
  int64_t q0, k0;
  int lq, lk, tile;   // tile < 0: nothing to do
};
__device__ __forceinline__ bool read_sequence(const AttnArgs& a, int b, AttnSeq& s) {
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  s = {q0, k0, q1 - q0, k1 - k0, -1};
  return q0 >= 0 && q1 >= q0 && q1 <= a.n_q && k0 >= 0 && k1 >= k0 && k1 <= a.n_k;
}
// Up to 24 sequences, one to a lane: the one with the most rows on the other side first, and
// its tiles with the most work first (of keys the first tiles, of queries the last), so that
// the launch does not end on a long block.  Each lane sums the tiles of the sequences before
// its own, which with many sequences costs more than the order gives.  Forward in order of
// length over forward in order of the offsets, the mean of six shapes (2500 to 10010 tokens; one
// shape's figures scatter by 5 %): 10 sequences 0.98, 16 0.95, 20 0.95, 24 0.98, 28 1.03,
// 32 1.04; whole backward 0.96, 0.98, 0.98, 1.01, 0.99, 0.96.  8192 tokens of 64: 67 -> 82 us.
constexpr int AT_SORTED = 24;
template <bool KEYS>
__device__ __forceinline__ AttnSeq find_sorted(const AttnArgs& a, int id, int shift) {
  const int lane = threadIdx.x & 63;
  AttnSeq s{0, 0, 0, 0, -1};
  int tiles = 0, work = 0;
  if (lane < a.n_seqs && read_sequence(a, lane, s))
    tiles = ((KEYS ? s.lk : s.lq) + (1 << shift) - 1) >> shift, work = KEYS ? s.lq : s.lk;
  int first = 0;
  for (int j = 0; j < a.n_seqs; ++j) {
    const int t = __builtin_amdgcn_readlane(tiles, j), w = __builtin_amdgcn_readlane(work, j);
    if (w > work || (w == work && j < lane)) first += t;
  }
  const int n = id - first;
  const uint64_t mine = __ballot(n >= 0 && n < tiles);
  if (!mine) return {0, 0, 0, 0, -1};
  const int b = __builtin_ctzll(mine);
  s.tile = KEYS ? n : tiles - 1 - n;
  s.q0 = __builtin_amdgcn_readlane((int)s.q0, b), s.k0 = __builtin_amdgcn_readlane((int)s.k0, b);
  s.lq = __builtin_amdgcn_readlane(s.lq, b), s.lk = __builtin_amdgcn_readlane(s.lk, b);
  s.tile = __builtin_amdgcn_readlane(s.tile, b);
  return s;
}
// Any number of them: sequence b owns the numbers from cu[b] / 2^shift + b on (rounded down),
// which leaves room for its last, partial tile; a number behind its last tile is empty.
template <bool KEYS>
__device__ __forceinline__ AttnSeq find_sequence(const AttnArgs& a, int id, int shift) {
  if (a.n_seqs <= AT_SORTED) return find_sorted<KEYS>(a, id, shift);
  if (!KEYS) id = a.tiles - 1 - id;
  const int32_t* const cu = KEYS ? a.cu_k : a.cu_q;
  const int lane = threadIdx.x & 63;
  const auto first = [&](int b) { return (cu[b] >> shift) + b; };
  int lo = 0, end = a.n_seqs;
  while (end - lo > 1) {
    const int step = (end - lo + 63) / 64, j = lo + lane * step;
    const uint64_t m = __ballot(j < end && first(j) <= id);
    if (!m) break;
    lo += (63 - __clzll(m)) * step;
    end = min(end, lo + step);
  }
  AttnSeq s;
  const int b = __builtin_amdgcn_readfirstlane(lo);
  if (!read_sequence(a, b, s)) return s;
  s.tile = id - first(b);
  if (s.tile < 0 || (int64_t)s.tile << shift >= (KEYS ? s.lk : s.lq)) s.tile = -1;
  return s;
}

// Every sequence's offsets, checked by the first block of a launch.
__device__ __forceinline__ void check_sequences(const AttnArgs& a) {
  bool bad = false;
  for (int b = threadIdx.x; b < a.n_seqs; b += blockDim.x) {
    AttnSeq s;
    bad |= !read_sequence(a, b, s);
  }
  if (bad) set_flag(a.status, LORA_FLAG_BAD_LENGTH);
}

// LDS rows of D columns: 16-byte chunk c of row r lies at chunk c ^ at_swz(r).  The direct
// reads (16 rows, one chunk) and the transposing ones (4 rows, 64 bytes) then both spread
// over all banks.
template <int D>
__device__ __forceinline__ int at_swz(int r) {
  return D == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : ((r >> 1 & 1) << 2) | ((r >> 2) & 3);
}
template <int D>
__device__ __forceinline__ uint32_t at_lds(int r, int chunk) {
  return (uint32_t)(r * (D * 2) + ((chunk ^ at_swz<D>(r)) << 4));
}

// Where a lane's operands lie in a tile.  Direct: row l, columns 16 kk + 8 h on.
// Transposed: columns 32 dt .. 32 dt + 31 as rows, over 16 rows in the order above, by two
// transposing reads.  The swizzle is a XOR, so one base each gives all of them; OPAQUE
// keeps the compiler from holding them all in registers.
struct AttnPlaces {
  uint32_t direct, transposed;
};
template <int D>
__device__ __forceinline__ AttnPlaces attn_places(int lane) {
  const int i = lane & 15, r = 4 * (lane >> 5) + (i >> 2), c = (lane >> 4 & 1) * 2 + ((i & 3) >> 1);
  return {at_lds<D>(lane & 31, lane >> 5), at_lds<D>(r, c) + (i & 1) * 8};
}
__device__ __forceinline__ AttnPlaces opaque(AttnPlaces p) {
  asm volatile("" : "+v"(p.direct), "+v"(p.transposed));
  return p;
}
__device__ __forceinline__ bf16x8 direct_op(const char* rows, AttnPlaces p, int kk) {
  return as_bf16x8(*(const uint4*)(rows + (p.direct ^ (kk << 5))));
}
template <int D>
__device__ __forceinline__ bf16x8 transposed_op(const char* rows, AttnPlaces p, int dt) {
  const uint2 a = tr_read((const uint4*)rows, p.transposed ^ (dt << 6));
  const uint2 b = tr_read((const uint4*)(rows + 8 * D * 2), p.transposed ^ (dt << 6) ^ 32);
  return as_bf16x8(make_uint4(a.x, a.y, b.x, b.y));
}

// LDS-DMA, 16 bytes a lane from base + voff, the lanes' one behind the other from LDS byte
// `to` on.  Issued by hand: the compiler would wait for it before every LDS read.
// M0 holds the LDS address: an operand, so that the compiler writes it and knows it; the hardware
// asks for one wait state between that write and the load.
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
__device__ __forceinline__ void dma16(uint32_t voff, const void* base, uint32_t to) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(to), "v"(voff), "s"(base) : "memory");
}
__device__ __forceinline__ void dma4_at(const void* p, uint32_t to) {   // 4 bytes a lane, each from its own address
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, off" ::"{m0}"(to), "v"(p) : "memory");
}
// Rows r0 .. r0 + ROWS - 1 of a [rows][D] matrix to LDS, by NW waves.  Rows past the end
// are copies of the last one: their weights are 0.
template <int D, int NW, int ROWS = AT_TILE>
__device__ __forceinline__ void dma_tile(const uint16_t* src, int64_t stride, int r0, int rows, uint32_t to, int wave,
                                         int lane) {
  constexpr int CH = D / 8, PER = 64 / CH, N = ROWS / PER;   // rows of an instruction; instructions
  const uint16_t* const base = src + r0 * stride;
#pragma unroll
  for (int j = 0; j < (N + NW - 1) / NW; ++j) {
    const int n = j * NW + wave, r = n * PER + lane / CH;
    if (N % NW && n >= N) break;
    const uint32_t at = (uint32_t)min(r, rows - 1 - r0) * (uint32_t)(stride * 2) + (((lane % CH) ^ at_swz<D>(r)) << 4);
    dma16(at, base, to + n * 1024);
  }
}

// A wave's own 32 rows as operand: lane (l, h) holds columns 16 kk + 8 h + 0..7 of row l.
template <int D>
__device__ __forceinline__ void load_rows(bf16x8* f, const uint16_t* row, int h) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) f[kk] = as_bf16x8(*(const uint4*)(row + kk * 16 + h * 8));
}

// Waits for the rows here: else the compiler does where they are used, in the loop, each
// time, and there the wait would be for the tiles on their way as well.
template <int N>
__device__ __forceinline__ void settle(bf16x8 (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint4 u = __builtin_bit_cast(uint4, f[i]);
    asm volatile("" : "+v"(u.x), "+v"(u.y), "+v"(u.z), "+v"(u.w));
    f[i] = as_bf16x8(u);
  }
}

// The order of the products before this point in a block of instructions: the LDS reads of
// four, then each product with the reads of the fourth one on.
template <int PRODUCTS, int READS>
__device__ __forceinline__ void feed_products() {
  constexpr int AHEAD = 4;
  __builtin_amdgcn_sched_group_barrier(0x100, READS * AHEAD, 0);
#pragma unroll
  for (int i = 0; i < PRODUCTS - AHEAD; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, AHEAD, 0);
}

__device__ __forceinline__ bf16x8 pack_op(const f32x16& x, int half) {
  const int o = half * 8;
  return as_bf16x8(make_uint4(pack2bf(x[o], x[o + 1]), pack2bf(x[o + 2], x[o + 3]), pack2bf(x[o + 4], x[o + 5]),
                              pack2bf(x[o + 6], x[o + 7])));
}
__device__ __forceinline__ int result_row(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// A lane's column of D results as bf16: four neighbouring columns of the row at a time.
template <int D>
__device__ __forceinline__ void store_row(uint16_t* row, const f32x16* x, float mul, int h) {
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      *(uint2*)(row + dt * 32 + result_row(r, h)) =
          make_uint2(pack2bf(x[dt][r] * mul, x[dt][r + 1] * mul), pack2bf(x[dt][r + 2] * mul, x[dt][r + 3] * mul));
}

// The halves of a word that hold NaN or Inf, as a mask.
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
  return ((w & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u) | ((w & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u);
}
__device__ __forceinline__ bool not_finite(bf16x8 x) {
  const uint4 u = __builtin_bit_cast(uint4, x);
  return (odd_halves(u.x) | odd_halves(u.y) | odd_halves(u.z) | odd_halves(u.w)) != 0;
}

// Whether what this lane fetched of a tile by dma_tile holds NaN or Inf.
template <int D, int NW, int ROWS = AT_TILE>
__device__ __forceinline__ bool dma_not_finite(const char* tile, int wave, int lane) {
  constexpr int N = ROWS * D * 2 / 1024;
  bool odd = false;
#pragma unroll
  for (int j = 0; j < (N + NW - 1) / NW; ++j) {
    const int n = j * NW + wave;
    if (N % NW && n >= N) break;
    odd |= not_finite(as_bf16x8(*(const uint4*)(tile + n * 1024 + lane * 16)));
  }
  return odd;
}

// acc += V^T P^T over 16 keys (key0 .. in the order above) where V may hold NaN or Inf:
// these are taken out and added key by key, for the queries that see the key.  (A weight
// of 0 would not keep them out; what other queries get has the bits of the plain product.)
__device__ __forceinline__ f32x16 product_seen(bf16x8 v, bf16x8 p, f32x16 acc, int key0, int last_key) {
  const int h = threadIdx.x >> 5 & 1;
  const uint4 u = __builtin_bit_cast(uint4, v);
  const uint4 m = make_uint4(odd_halves(u.x), odd_halves(u.y), odd_halves(u.z), odd_halves(u.w));
  acc = mfma32(as_bf16x8(make_uint4(u.x & ~m.x, u.y & ~m.y, u.z & ~m.z, u.w & ~m.w)), p, acc);
#pragma unroll 1
  for (int i = 0; i < 16; ++i) {
    const int j = i & 7, hi = i >> 3;
    const uint32_t keep = h != hi ? 0u : j & 1 ? 0xFFFF0000u : 0xFFFFu;
    uint4 w;
    w.x = (j >> 1) == 0 ? u.x & m.x & keep : 0u;
    w.y = (j >> 1) == 1 ? u.y & m.y & keep : 0u;
    w.z = (j >> 1) == 2 ? u.z & m.z & keep : 0u;
    w.w = (j >> 1) == 3 ? u.w & m.w & keep : 0u;
    const f32x16 with = mfma32(as_bf16x8(w), p, acc);
    const bool seen = key0 + 8 * (j >> 2) + 4 * hi + (j & 3) <= last_key;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = seen ? with[r] : acc[r];
  }
  return acc;
}

// ---------------------------------------------------------------- forward
// NW waves of 32 query rows: `wpr` of them behind one another in one head, the rest in the
// next heads of the same group, which read the same tiles.  Tiles of 64 keys pass through
// two LDS stages by LDS-DMA, one barrier a tile; the tiles that no query of the block masks
// in a loop of their own, whose stages are compile-time offsets.  Two waves on each SIMD
// take turns: while one computes its weights the other's products run.
// The weights are powers of two relative to a reference that follows the row's maximum
// only when that has passed it by 2^6: they stay below 2^6, exact as any float, and the
// output is hardly ever rescaled.
// Bound by the matrix units and the clock that their power leaves: 16384 tokens, 32 heads of
// 128 over 8, causal (2.2 TFLOP): 1.96-2.08 ms, 1.06-1.12 PFLOP/s, the units busy in 59 % of
// the cycles at 1.9 GHz (a large library matrix product: 1.37 PFLOP/s).  LDS is read
// without conflicts and for a third of the cycles; 0.43 GB come from memory, 0.20 of
// them the operands once.  Tried without gain: wave priorities around the products (the same), two
// groups of waves half a tile apart (2088 against 1980 us).
// Short prompts pay for a block's start (offsets, q, first tile: three round trips, in about
// four rounds of blocks) and for the tiles behind the last pair of whole ones, whose v is looked
// through before it is used (a fifth of the tiles; the masked halves are a tenth of the work):
// 8192 tokens of 16, 98-101 us for 59.5 GFLOP.
constexpr float AT_SLACK = 6.f;

template <int D, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2, 2))) void attention_fwd_kernel(AttnArgs a) {
  constexpr int ND = D / 32, NK = D / 16;
  constexpr int TILE = AT_TILE * D * 2;            // bytes of one operand of a stage
  __shared__ __attribute__((aligned(16))) char lds[4 * TILE];
  __shared__ int odd_tile[2];                      // of a stage: one more than the tile where v holds NaN or Inf
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & 31, h = lane >> 5;
  if (blockIdx.x == 0) check_sequences(a);
  const int per_block = NW / a.wpr, columns = a.n_heads / per_block;   // heads of a block; blocks of a row tile
  const int hx = blockIdx.x % columns, kvh = hx % a.n_kv;
  const int head = kvh * a.group + hx / a.n_kv * per_block + wave / a.wpr;
  const AttnSeq s = find_sequence<false>(a, blockIdx.x / columns, a.shift);
  if (s.tile < 0) return;
  const int row0 = s.tile << a.shift, w0 = row0 + wave % a.wpr * 32, i = w0 + l;   // query row
  const int ahead = s.lk - s.lq;
  // the last key that this lane's query, the wave and the block see
  const int last = a.causal ? min(i + ahead, s.lk - 1) : s.lk - 1;
  const int wave_first = a.causal ? w0 + ahead : s.lk - 1;
  const int wave_last = w0 >= s.lq ? -1 : a.causal ? min(w0 + 31 + ahead, s.lk - 1) : s.lk - 1;
  const int keys = a.causal ? min(row0 + (1 << a.shift) + ahead, s.lk) : s.lk;
  const int tiles = keys > 0 ? (keys + AT_TILE - 1) / AT_TILE : 0;

  const uint16_t* const kp = a.k + s.k0 * a.k_stride + kvh * D;
  const uint16_t* const vp = a.v + s.k0 * a.v_stride + kvh * D;
  const uint32_t lds0 = lds_offset(lds);
  const auto stage = [&](int t, int st) {
    dma_tile<D, NW>(kp, a.k_stride, t * AT_TILE, s.lk, lds0 + st * 2 * TILE, wave, lane);
    dma_tile<D, NW>(vp, a.v_stride, t * AT_TILE, s.lk, lds0 + st * 2 * TILE + TILE, wave, lane);
  };

  if (threadIdx.x < 2) odd_tile[threadIdx.x] = 0;
  if (tiles) stage(0, 0);   // (on its way while q's rows are)
  // a negative scale turns q's signs, a scale of 0 makes q 0: the maximum of the products
  // is then that of the scores
  bf16x8 qf[NK];
  load_rows<D>(qf, a.q + (s.q0 + min(i, s.lq - 1)) * a.q_stride + head * D, h);
  const float c = a.scale == 0.f ? 1.f : fabsf(a.scale_log2);
  if (a.scale <= 0.f) {
    const uint32_t turn = a.scale < 0.f ? 0x80008000u : 0u, keep = a.scale < 0.f ? ~0u : 0u;
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) {
      const uint4 u = __builtin_bit_cast(uint4, qf[kk]);
      qf[kk] = as_bf16x8(make_uint4((u.x ^ turn) & keep, (u.y ^ turn) & keep, (u.z ^ turn) & keep, (u.w ^ turn) & keep));
    }
  }
  settle(qf);
  __syncthreads();
  f32x16 acc[ND];
#pragma unroll
  for (int dt = 0; dt < ND; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[dt][r] = 0.f;
  float ref = -INFINITY, sum = 0.f;

  const AttnPlaces places = attn_places<D>(lane);

  const auto step = [&](int t, auto st, auto masked) {   // masked: false_type, or whether to mask
    const int K0 = st * 2 * TILE, V0 = K0 + TILE;
    const int t0 = t * AT_TILE;
    const AttnPlaces at = opaque(places);
    f32x16 x[2];
#pragma unroll
    for (int r = 0; r < 16; ++r) x[0][r] = x[1][r] = 0.f;
    // (two sums in turn: a product that adds to the one before it waits for it)
#pragma unroll
    for (int kk = 0; kk < NK; ++kk)
#pragma unroll
      for (int u = 0; u < 2; ++u) x[u] = mfma32(direct_op(lds + K0 + u * 32 * D * 2, at, kk), qf[kk], x[u]);
    feed_products<2 * NK, 1>();
    if (masked) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (t0 + u * 32 + result_row(r, h) > last) x[u][r] = -INFINITY;
    }
    float top = fmaxf(x[0][0], x[1][0]);
#pragma unroll
    for (int r = 1; r < 16; ++r) top = fmaxf(fmaxf(top, x[0][r]), x[1][r]);
    top = fmaxf(top, __shfl_xor(top, 32, kWave)) * c;
    // (each row by its own scores alone: no other query's keys show in its bits)
    const bool rise = top > ref + AT_SLACK;
    if (__any(rise)) {
      const float next = rise ? top : ref, scale = rise ? __builtin_amdgcn_exp2f(ref - next) : 1.f;
      ref = next;
      sum *= scale;
#pragma unroll
      for (int dt = 0; dt < ND; ++dt)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[dt][r] *= scale;
    }
    const float base = ref == -INFINITY ? 0.f : ref;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        x[u][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[u][r], c, -base));
        sum += x[u][r];
      }
    if (masked) {
      if (__builtin_amdgcn_readfirstlane(odd_tile[st]) == t + 1) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const bf16x8 p = pack_op(x[b >> 1], b & 1);
#pragma unroll
          for (int dt = 0; dt < ND; ++dt)
            acc[dt] = product_seen(transposed_op<D>(lds + V0 + b * 16 * D * 2, at, dt), p, acc[dt], t0 + b * 16, last);
        }
        return;
      }
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const bf16x8 p = pack_op(x[b >> 1], b & 1);
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) acc[dt] = mfma32(transposed_op<D>(lds + V0 + b * 16 * D * 2, at, dt), p, acc[dt]);
    }
  };
  // tile t has landed for every wave, and every wave is done with the other stage; where a
  // tile is masked, each wave has looked through the part of v that it fetched
  const auto arrive = [&](int t, int st, bool look) {
    if (look) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      if (__any(dma_not_finite<D, NW>(lds + st * 2 * TILE + TILE, wave, lane))) odd_tile[st] = t + 1;
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (t + 1 < tiles) stage(t + 1, 1 - st);
  };
  // the tiles that no query of the block has to mask, in pairs; then the rest
  const int whole = min(a.causal ? row0 + ahead + 1 : s.lk, s.lk);
  const int pairs = max(whole, 0) / (2 * AT_TILE);
  const bool on = w0 < s.lq;
  int t = 0;
  for (; t < 2 * pairs; t += 2) {
    arrive(t, 0, false);
    if (on) step(t, std::integral_constant<int, 0>{}, std::false_type{});
    arrive(t + 1, 1, false);
    if (on) step(t + 1, std::integral_constant<int, 1>{}, std::false_type{});
  }
  for (; t < tiles; ++t) {
    arrive(t, t & 1, true);
    const int t0 = t * AT_TILE;
    if (t0 <= wave_last) step(t, t & 1, t0 + AT_TILE - 1 > wave_first || t0 + AT_TILE > s.lk);
  }
  if (i >= s.lq) return;
  sum += __shfl_xor(sum, 32, kWave);
  store_row<D>(a.out + (s.q0 + i) * a.o_stride + head * D, acc, sum == 0.f ? 0.f : 1.f / sum, h);
  if (h == 0) a.lse[head * a.n_q + s.q0 + i] = sum == 0.f ? -INFINITY : (ref + __log2f(sum)) * AT_LN2;
}

// ---------------------------------------------------------------- dq
// Waves, tiles and stages as in the forward, three products a tile in place of two.  8192
// tokens of 6, 32 heads of 128 over 8 (11.3 M pairs a head), in blocks of four heads by 32
// rows: 287-294 us, 0.94-0.96 PFLOP/s; the matrix units are busy in 55 % of the cycles.
template <int D, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2, 2))) void attention_dq_kernel(AttnArgs a) {
  constexpr int ND = D / 32, NK = D / 16;
  constexpr int TILE = AT_TILE * D * 2;
  __shared__ __attribute__((aligned(16))) char lds[4 * TILE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & 31, h = lane >> 5;
  if (blockIdx.x == 0) check_sequences(a);
  const int per_block = NW / a.wpr, columns = a.n_heads / per_block;
  const int hx = blockIdx.x % columns, kvh = hx % a.n_kv;
  const int head = kvh * a.group + hx / a.n_kv * per_block + wave / a.wpr;
  const AttnSeq s = find_sequence<false>(a, blockIdx.x / columns, a.shift);
  if (s.tile < 0) return;
  const int row0 = s.tile << a.shift, w0 = row0 + wave % a.wpr * 32, i = w0 + l;
  const int ahead = s.lk - s.lq;
  const int last = a.causal ? min(i + ahead, s.lk - 1) : s.lk - 1;
  const int wave_first = a.causal ? w0 + ahead : s.lk - 1;
  const int wave_last = w0 >= s.lq ? -1 : a.causal ? min(w0 + 31 + ahead, s.lk - 1) : s.lk - 1;
  const int keys = a.causal ? min(row0 + (1 << a.shift) + ahead, s.lk) : s.lk;
  const int tiles = keys > 0 ? (keys + AT_TILE - 1) / AT_TILE : 0;

  const uint16_t* const kp = a.k + s.k0 * a.k_stride + kvh * D;
  const uint16_t* const vp = a.v + s.k0 * a.v_stride + kvh * D;
  const uint32_t lds0 = lds_offset(lds);
  const auto stage = [&](int t, int st) {
    dma_tile<D, NW>(kp, a.k_stride, t * AT_TILE, s.lk, lds0 + st * 2 * TILE, wave, lane);
    dma_tile<D, NW>(vp, a.v_stride, t * AT_TILE, s.lk, lds0 + st * 2 * TILE + TILE, wave, lane);
  };
  if (tiles) stage(0, 0);
  const int64_t row = s.q0 + min(i, s.lq - 1);
  bf16x8 qf[NK], df[NK];
  load_rows<D>(qf, a.q + row * a.q_stride + head * D, h);
  load_rows<D>(df, a.dout + row * a.o_stride + head * D, h);
  // delta, the diagonal of dO O^T, by the instruction and in the order of dO V^T: where o is
  // v (a single key) ds is 0, as it should be
  float delta = 0.f;
  {
    bf16x8 of[NK];
    load_rows<D>(of, a.o + row * a.o_stride + head * D, h);
    f32x16 z;
#pragma unroll
    for (int r = 0; r < 16; ++r) z[r] = 0.f;
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) z = mfma32(of[kk], df[kk], z);
#pragma unroll
    for (int r = 0; r < 16; ++r) delta = result_row(r, h) == l ? z[r] : delta;
    delta += __shfl_xor(delta, 32, kWave);
  }
  settle(qf);
  settle(df);
  const float lse = a.lse[head * a.n_q + row] * AT_LOG2E;
  if (i < s.lq) a.stats[((int64_t)head * 2 + h) * a.n_q + row] = h ? delta : lse;
  f32x16 acc[ND];
#pragma unroll
  for (int dt = 0; dt < ND; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[dt][r] = 0.f;

  const AttnPlaces places = attn_places<D>(lane);

  const auto step = [&](int t, auto st, auto masked) {   // masked: false_type, or whether to mask
    const int K0 = st * 2 * TILE, V0 = K0 + TILE;
    const int t0 = t * AT_TILE;
    const AttnPlaces at = places;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f32x16 x, y;
#pragma unroll
      for (int r = 0; r < 16; ++r) x[r] = y[r] = 0.f;
#pragma unroll
      for (int kk = 0; kk < NK; ++kk) {
        x = mfma32(direct_op(lds + K0 + u * 32 * D * 2, at, kk), qf[kk], x);
        y = mfma32(direct_op(lds + V0 + u * 32 * D * 2, at, kk), df[kk], y);
      }
      feed_products<2 * NK, 1>();
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(x[r], a.scale_log2, -lse));
        x[r] = p * (y[r] - delta);
      }
      if (masked) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (t0 + u * 32 + result_row(r, h) > last) x[r] = 0.f;
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const bf16x8 ds = pack_op(x, b);
#pragma unroll
        for (int dt = 0; dt < ND; ++dt)
          acc[dt] = mfma32(transposed_op<D>(lds + K0 + (u * 32 + b * 16) * D * 2, at, dt), ds, acc[dt]);
      }
    }
  };
  // tile t has landed for every wave, and every wave is done with the other stage
  const auto arrive = [&](int t, int st) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (t + 1 < tiles) stage(t + 1, 1 - st);
  };
  // the tiles that no query of the block has to mask, in pairs; then the rest
  const int whole = min(a.causal ? row0 + ahead + 1 : s.lk, s.lk);
  const int pairs = max(whole, 0) / (2 * AT_TILE);
  const bool on = w0 < s.lq;
  int t = 0;
  for (; t < 2 * pairs; t += 2) {
    arrive(t, 0);
    if (on) step(t, std::integral_constant<int, 0>{}, std::false_type{});
    arrive(t + 1, 1);
    if (on) step(t + 1, std::integral_constant<int, 1>{}, std::false_type{});
  }
  for (; t < tiles; ++t) {
    arrive(t, t & 1);
    const int t0 = t * AT_TILE;
    if (t0 <= wave_last) step(t, t & 1, t0 + AT_TILE - 1 > wave_first || t0 + AT_TILE > s.lk);
  }
  if (i < s.lq) store_row<D>(a.dq + (s.q0 + i) * a.q_stride + head * D, acc, a.scale, h);
}

// ---------------------------------------------------------------- dk, dv
// A wave owns 32 keys, KW waves 32 KW of them in a row, and the block's NW / KW phases
// share out what those keys have to see: tiles of 32 queries of a head, with their dout,
// lse and delta, head after head of the group, phase p taking every (NW / KW)-th.  Each
// phase has two LDS stages of its own, filled by its own waves, the DMA a tile ahead.  At the
// end the phases' sums are added in order, through LDS.
// Four products a tile, two waves on a SIMD (256 registers each: the two sums alone are 128).
// 8192 tokens of 6 as above: 420-490 us, 0.75-0.87 PFLOP/s, the matrix units busy in 41 % of
// the cycles: the waves of a block go in step from tile to tile, and the longest block holds
// the end up (a block's work goes from 4020 queries of four heads down to 64).  Phases of a
// single wave need no barrier (2048 tokens 183 -> 173 us).
constexpr int DKV_TILE = 32;

template <int D, int NW, int KW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(NW / 4, NW / 4))) void attention_dkv_kernel(AttnArgs a) {
  constexpr int ND = D / 32, NK = D / 16, P = NW / KW;
  constexpr int TILE = DKV_TILE * D * 2, STAGE = 2 * TILE;   // q's rows, then dout's
  static_assert(P * 2 * STAGE >= (NW - KW) * TILE * 2);      // room for the other phases' dk or dv in fp32
  __shared__ __attribute__((aligned(16))) char lds[P * 2 * STAGE];
  __shared__ __attribute__((aligned(16))) float stats[P][2][2][DKV_TILE];   // of a stage: lse in powers of two, delta
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & 31, h = lane >> 5, phase = wave / KW, kw = wave % KW;
  const int kvh = blockIdx.x % a.n_kv;
  const AttnSeq s = find_sequence<true>(a, blockIdx.x / a.n_kv, a.shift);
  if (s.tile < 0) return;
  const int row0 = s.tile << a.shift, w0 = row0 + kw * 32, j = w0 + l;   // key row
  const int ahead = s.lk - s.lq;
  // the first query that sees this lane's key, one of the wave's, all of the wave's
  const int first = a.causal ? j - ahead : 0;
  const int wave_first = w0 >= s.lk ? 1 << 30 : a.causal ? w0 - ahead : 0, wave_all = a.causal ? w0 + 31 - ahead : 0;
  const int begin = a.causal ? max(row0 - ahead, 0) / DKV_TILE : 0;
  const int end = (s.lq + DKV_TILE - 1) / DKV_TILE, per_head = max(end - begin, 0);
  const int tiles = per_head * a.group, steps = (tiles + P - 1) / P;

  // the phase's tile: head of the group and tile of the head
  struct At {
    int head, tile;
  };
  const auto skip = [&](At& t, int n) {
    for (t.tile += n; t.tile >= end && t.head < a.group; t.tile -= per_head) ++t.head;
  };
  const uint32_t lds0 = lds_offset(lds) + phase * 2 * STAGE, stats0 = lds_offset(stats) + phase * (int)sizeof(stats[0]);
  At ask{0, begin};
  const auto stage = [&](int st) {
    if (ask.head >= a.group) return;
    const int t0 = ask.tile * DKV_TILE, head = kvh * a.group + ask.head;
    dma_tile<D, KW, DKV_TILE>(a.q + s.q0 * a.q_stride + head * D, a.q_stride, t0, s.lq, lds0 + st * STAGE, kw, lane);
    dma_tile<D, KW, DKV_TILE>(a.dout + s.q0 * a.o_stride + head * D, a.o_stride, t0, s.lq, lds0 + st * STAGE + TILE, kw, lane);
    // the lower lanes fetch the tile's lse, the upper ones its delta (each wave the same)
    dma4_at(a.stats + ((int64_t)head * 2 + h) * a.n_q + s.q0 + min(t0 + l, s.lq - 1), stats0 + st * (int)sizeof(stats[0][0]));
    skip(ask, P);
  };
  At now{0, begin};
  if (per_head) {
    skip(now, phase);
    ask = now;
    stage(0);
  }
  bf16x8 kf[NK], vf[NK];
  const int64_t row = s.k0 + min(j, s.lk - 1);
  load_rows<D>(kf, a.k + row * a.k_stride + kvh * D, h);
  load_rows<D>(vf, a.v + row * a.v_stride + kvh * D, h);
  settle(kf);
  settle(vf);
  f32x16 dk[ND], dv[ND];
#pragma unroll
  for (int dt = 0; dt < ND; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) dk[dt][r] = dv[dt][r] = 0.f;
  const AttnPlaces places = attn_places<D>(lane);

  const auto step = [&](int t0, int st, const bool masked) {
    const char *const qt = lds, *const gt = qt + TILE;
    const float* const stat = &stats[phase][st][0][0];
    const uint32_t off = (phase * 2 + st) * STAGE;   // (above the bits that the swizzle turns)
    const AttnPlaces at = opaque({places.direct + off, places.transposed + off});
    f32x16 x, y;
#pragma unroll
    for (int r = 0; r < 16; ++r) x[r] = y[r] = 0.f;
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) {
      x = mfma32(direct_op(qt, at, kk), kf[kk], x);
      y = mfma32(direct_op(gt, at, kk), vf[kk], y);
    }
    feed_products<2 * NK, 1>();
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const f32x4 ls = *(const f32x4*)&stat[8 * r4 + 4 * h];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int r = r4 * 4 + c;
        x[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[r], a.scale_log2, -ls[c]));
      }
    }
    if (masked) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int q = t0 + result_row(r, h);
        if (q < first || q >= s.lq) x[r] = 0.f;
      }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const bf16x8 p = pack_op(x, b);
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) dv[dt] = mfma32(transposed_op<D>(gt + b * 16 * D * 2, at, dt), p, dv[dt]);
    }
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const f32x4 de = *(const f32x4*)&stat[DKV_TILE + 8 * r4 + 4 * h];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int r = r4 * 4 + c;
        y[r] = x[r] * (y[r] - de[c]);
      }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const bf16x8 ds = pack_op(y, b);
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) dk[dt] = mfma32(transposed_op<D>(qt + b * 16 * D * 2, at, dt), ds, dk[dt]);
    }
  };
  for (int n = 0, st = 0; n < steps; ++n) {
    // the tile has landed, every wave of the phase is done with the stage before it (a wave
    // that is a phase by itself waits for nobody)
    if constexpr (KW == 1) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    stage(1 - st);
    const int t0 = now.tile * DKV_TILE;
    if (now.head < a.group && t0 + DKV_TILE - 1 >= wave_first) step(t0, st, t0 < wave_all || t0 + DKV_TILE > s.lq);
    skip(now, P);
    st = 1 - st;
  }
  const auto add_phases = [&](f32x16* x) {
    if (P == 1) return;
    f32x4* const part = (f32x4*)lds + ((phase - 1) * KW + kw) * (ND * 4 * 64);
    __syncthreads();
    if (phase)
#pragma unroll
      for (int i = 0; i < ND * 4; ++i) part[i * 64 + lane] = f32x4{x[i / 4][i % 4 * 4], x[i / 4][i % 4 * 4 + 1], x[i / 4][i % 4 * 4 + 2], x[i / 4][i % 4 * 4 + 3]};
    __syncthreads();
    if (phase == 0)
#pragma unroll
      for (int p = 1; p < P; ++p)
#pragma unroll
        for (int i = 0; i < ND * 4; ++i) {
          const f32x4 v = ((const f32x4*)lds)[((p - 1) * KW + kw) * (ND * 4 * 64) + i * 64 + lane];
#pragma unroll
          for (int c = 0; c < 4; ++c) x[i / 4][i % 4 * 4 + c] += v[c];
        }
  };
  add_phases(dk);
  add_phases(dv);
  if (phase || j >= s.lk) return;
  store_row<D>(a.dk + (s.k0 + j) * a.k_stride + kvh * D, dk, a.scale, h);
  store_row<D>(a.dv + (s.k0 + j) * a.v_stride + kvh * D, dv, 1.f, h);
}

}  // namespace lora

// ---------------------------------------------------------------- launches
namespace lora_host {

using namespace lora;

static AttnArgs attn_args(const attn_shape& sh, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                          const int32_t* cu_q, const int32_t* cu_k, void* ws) {
  AttnArgs a{};
  a.q = q, a.k = k, a.v = v, a.cu_q = cu_q, a.cu_k = cu_k, a.status = (int32_t*)ws;
  a.stats = (float*)((char*)ws + 256);
  a.q_stride = sh.q_stride, a.k_stride = sh.k_stride, a.v_stride = sh.v_stride, a.o_stride = sh.o_stride;
  a.n_q = sh.n_q, a.n_k = sh.n_k, a.n_seqs = sh.n_seqs, a.n_heads = sh.n_heads, a.n_kv = sh.n_kv_heads;
  a.group = sh.n_heads / sh.n_kv_heads, a.causal = sh.causal;
  a.scale = sh.scale, a.scale_log2 = sh.scale * AT_LOG2E;
  return a;
}

// The blocks of the kernels whose waves own queries.  Four waves: two such blocks share a CU
// and fill each other's waits at a block's start and end.  Eight (two heads of a group by 128
// rows, or 256 rows): a tile that comes through LDS serves twice the queries, which pays where
// blocks live long.  Forward, four / eight waves, us:
//   16384 tokens, 32 heads of 128       2057 / 1982      4096 tokens             157 / 148
//   2048 tokens                           53 /   61      8192 tokens of 16       101 / 108
//   8192 tokens of 6                     165 /  164      10010 of 8, heads of 64  92 /  97
// Four waves of up to four heads of a group where there are blocks enough: fewer rows behind
// a sequence's last, and waves that need the same keys.  128 rows of one head / 32 of four:
//   8192 tokens of 100                  80.5 / 64.7      4096 tokens of 8       47.9 / 46.5
//   8192 of 64, heads of 64             30.4 / 26.9      300 tokens             11.8 / 12.6
struct QueryGrid {
  dim3 blocks;
  int waves;
};
static QueryGrid query_grid(AttnArgs& a, const attn_shape& sh) {
  const auto tiles = [&](int shift) { return (sh.n_q >> shift) + sh.n_seqs; };
  int waves = 8, heads = a.group % 2 == 0 ? 2 : 1;
  a.shift = heads == 2 ? 7 : 8;
  const bool few = tiles(a.shift) * (a.n_heads / heads) < 2 * device_cus();
  if (few || sh.n_q / 2048 < sh.n_seqs) {
    waves = 4, heads = few || a.group % 2 ? 1 : a.group % 4 ? 2 : 4;
    a.shift = heads == 4 ? 5 : heads == 2 ? 6 : 7;
  }
  a.wpr = waves / heads;
  a.tiles = (int)tiles(a.shift);
  return {dim3((unsigned)((int64_t)a.tiles * (a.n_heads / heads))), waves};
}

lora_status launch_attention_fwd(const attn_shape& sh, const uint16_t* q, const uint16_t* k,
                                 const uint16_t* v, const int32_t* cu_q, const int32_t* cu_k,
                                 uint16_t* o, float* lse, void* ws, hipStream_t s) {
  AttnArgs a = attn_args(sh, q, k, v, cu_q, cu_k, ws);
  a.out = o, a.lse = lse;
  const QueryGrid g = query_grid(a, sh);
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, g.blocks, dim3(64 * g.waves), 0, s, a); };
  if (sh.head_dim == 128) g.waves == 8 ? go(attention_fwd_kernel<128, 8>) : go(attention_fwd_kernel<128, 4>);
  else g.waves == 8 ? go(attention_fwd_kernel<64, 8>) : go(attention_fwd_kernel<64, 4>);
  return launch_check("attention_forward");
}

lora_status launch_attention_bwd(const attn_shape& sh, const uint16_t* dout, const uint16_t* q,
                                 const uint16_t* k, const uint16_t* v, const uint16_t* o,
                                 const float* lse, const int32_t* cu_q, const int32_t* cu_k,
                                 uint16_t* dq, uint16_t* dk, uint16_t* dv, void* ws, hipStream_t s) {
  AttnArgs a = attn_args(sh, q, k, v, cu_q, cu_k, ws);
  a.dout = dout, a.o = o, a.lse = const_cast<float*>(lse), a.dq = dq, a.dk = dk, a.dv = dv;
  // dq first: it also leaves delta for the other kernel
  const QueryGrid g = query_grid(a, sh);
  const auto go_q = [&](auto kernel) { hipLaunchKernelGGL(kernel, g.blocks, dim3(64 * g.waves), 0, s, a); };
  if (sh.head_dim == 128) g.waves == 8 ? go_q(attention_dq_kernel<128, 8>) : go_q(attention_dq_kernel<128, 4>);
  else g.waves == 8 ? go_q(attention_dq_kernel<64, 8>) : go_q(attention_dq_kernel<64, 4>);
  lora_status st = launch_check("attention_backward dq");
  if (st != LORA_OK) return st;
  // Keys of a block, by the blocks that 128 of them make.  128: each tile that comes through
  // LDS serves most keys; 64 and 32: the longest block, which a causal batch may end up
  // waiting for, is half and a quarter as long.  Whole backward, 128 / 64 / 32 keys, us:
  //   16384 tokens, 8 key heads (1032 blocks)    6890 / 7028 / 8566
  //   4096 tokens, 32 key heads (1056)            476 /  537 /  695
  //   8192 tokens of 16, 8 key heads (640)        479 /  426 /  502
  //   4096 tokens, 8 key heads (264)              622 /  476 /  573
  //   4096 tokens of 8, 4 key heads (160)         390 /  256 /  189
  //   2048 tokens, 8 key heads (136)              297 /  207 /  173
  // (Each sequence counts for a block, so batches of many short ones take 128 keys, of which their
  // last blocks own few: 8192 tokens of 100, 227 us, and the other sizes are not measured there.)
  // With 32 keys a wave is a phase by itself; eight of them, where LDS has room for their
  // stages (heads of 64), make the block half as long as four (5000 tokens, 4 key heads:
  // 294 -> 246 us; 200 tokens: 16.4 -> 17.8).
  const auto key_blocks = [&](int shift) { return ((sh.n_k >> shift) + sh.n_seqs) * sh.n_kv_heads; };
  a.shift = key_blocks(7) >= 4 * device_cus() ? 7 : key_blocks(7) >= device_cus() ? 6 : 5;
  a.tiles = (int)((sh.n_k >> a.shift) + sh.n_seqs);
  const auto go_k = [&](auto kernel, int waves) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)key_blocks(a.shift)), dim3(64 * waves), 0, s, a);
  };
  const auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    a.shift == 7   ? go_k(attention_dkv_kernel<D, 8, 4>, 8)
    : a.shift == 6 ? go_k(attention_dkv_kernel<D, 8, 2>, 8)
                   : go_k(attention_dkv_kernel<D, D == 64 ? 8 : 4, 1>, D == 64 ? 8 : 4);
  };
  if (sh.head_dim == 128) pick(std::integral_constant<int, 128>{});
  else pick(std::integral_constant<int, 64>{});
  return launch_check("attention_backward dk, dv");
}

}  // namespace lora_host
