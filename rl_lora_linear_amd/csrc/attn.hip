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
// partial results in memory.
#include <type_traits>

#include "attn.hpp"

namespace lora {

constexpr float AT_LOG2E = 1.4426950408889634f, AT_LN2 = 0.6931471805599453f;
constexpr int AT_WAVES = 4, AT_ROWS = 32 * AT_WAVES;   // rows of a block
constexpr int AT_SHIFT = 7;                            // log2(AT_ROWS)
constexpr int AT_TILE = 64;                            // rows of a tile in LDS
static_assert(1 << AT_SHIFT == AT_ROWS);

struct AttnArgs {
  const uint16_t *q, *k, *v, *o, *dout;
  uint16_t *out, *dq, *dk, *dv;
  float *lse, *delta;   // [heads][n_q]
  const int32_t *cu_q, *cu_k;
  int32_t* status;
  int64_t q_stride, k_stride, v_stride, o_stride, n_q, n_k;
  int32_t n_seqs, n_heads, n_kv, group, causal, tiles;
  int32_t wpr, shift;   // forward: waves of a block in one head; log2 of its rows
  float scale, scale_log2;
};

// Tiles of a packed batch: sequence b owns the tile numbers from cu[b] / rows + b on
// (rounded down), which leaves room for its last, partial tile; a number behind its last
// tile is empty.  So a block finds its sequence from cu alone.
struct AttnSeq {
  int64_t q0, k0;
  int lq, lk, tile;   // tile < 0: nothing to do
};
__device__ __forceinline__ AttnSeq find_sequence(const AttnArgs& a, const int32_t* cu, int id,
                                                 int shift = AT_SHIFT) {
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
  AttnSeq s{0, 0, 0, 0, -1};
  const int b = __builtin_amdgcn_readfirstlane(lo);
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  if (q0 < 0 || q1 < q0 || q1 > a.n_q || k0 < 0 || k1 < k0 || k1 > a.n_k) return s;
  s.q0 = q0, s.k0 = k0, s.lq = q1 - q0, s.lk = k1 - k0;
  s.tile = id - first(b);
  if (s.tile < 0 || (int64_t)s.tile << shift >= (cu == a.cu_q ? s.lq : s.lk)) s.tile = -1;
  return s;
}

// Every sequence's offsets, checked by the first block of a launch.
__device__ __forceinline__ void check_sequences(const AttnArgs& a) {
  bool bad = false;
  for (int b = threadIdx.x; b < a.n_seqs; b += blockDim.x) {
    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
    bad |= q0 < 0 || q1 < q0 || q1 > a.n_q || k0 < 0 || k1 < k0 || k1 > a.n_k;
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

// A tile of rows r0 .. r0 + AT_TILE - 1 of a [rows][D] matrix into LDS, zeros past `rows`.
template <int D>
__device__ __forceinline__ void stage_tile(char* dst, const uint16_t* src, int64_t stride, int r0, int rows) {
  constexpr int CH = D / 8;
#pragma unroll
  for (int i = 0; i < AT_TILE * CH / (64 * AT_WAVES); ++i) {
    const int j = i * 64 * AT_WAVES + threadIdx.x, r = j / CH, c = j % CH;
    const uint4 x = r0 + r < rows ? *(const uint4*)(src + (int64_t)(r0 + r) * stride + c * 8) : make_uint4(0, 0, 0, 0);
    *(uint4*)(dst + at_lds<D>(r, c)) = x;
  }
}

// Operand of 32 rows, columns 16 kk .. 16 kk + 15.
template <int D>
__device__ __forceinline__ bf16x8 direct_op(const char* tile, int row0, int kk, int l, int h) {
  return as_bf16x8(*(const uint4*)(tile + at_lds<D>(row0 + l, 2 * kk + h)));
}
// Transposed operand: columns 32 dt .. 32 dt + 31 as its rows, over rows row0 .. row0 + 15
// in the order above.
template <int D>
__device__ __forceinline__ bf16x8 transposed_op(const char* tile, int row0, int dt, int lane) {
  const int i = lane & 15, r = row0 + 4 * (lane >> 5) + (i >> 2);
  const int c = dt * 4 + (lane >> 4 & 1) * 2 + ((i & 3) >> 1), lo = (i & 1) * 8;
  const uint2 a = tr_read((const uint4*)tile, at_lds<D>(r, c) + lo);
  const uint2 b = tr_read((const uint4*)tile, at_lds<D>(r + 8, c) + lo);
  return as_bf16x8(make_uint4(a.x, a.y, b.x, b.y));
}

// The same from addresses worked out before: two rows' places in a tile.
template <int D>
__device__ __forceinline__ void transposed_at(uint32_t* at, int dt, int lane) {
  const int i = lane & 15, r = 4 * (lane >> 5) + (i >> 2);
  const int c = dt * 4 + (lane >> 4 & 1) * 2 + ((i & 3) >> 1), lo = (i & 1) * 8;
  at[0] = at_lds<D>(r, c) + lo;
  at[1] = at_lds<D>(r + 8, c) + lo;
}
__device__ __forceinline__ bf16x8 transposed_pair(const char* tile, const uint32_t* at) {
  const uint2 a = tr_read((const uint4*)tile, at[0]), b = tr_read((const uint4*)tile, at[1]);
  return as_bf16x8(make_uint4(a.x, a.y, b.x, b.y));
}

// LDS-DMA, 16 bytes a lane from base + voff, the lanes' one behind the other from LDS byte
// `to` on.  Issued by hand: the compiler would wait for it before every LDS read.
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
__device__ __forceinline__ void dma16(uint32_t voff, const void* base, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(voff), "s"(base) : "memory");
}
// Rows r0 .. r0 + AT_TILE - 1 of a [rows][D] matrix to LDS, by NW waves.  Rows past the end
// are copies of the last one: their weights are 0.
template <int D, int NW>
__device__ __forceinline__ void dma_tile(const uint16_t* src, int64_t stride, int r0, int rows, uint32_t to, int wave,
                                         int lane) {
  constexpr int CH = D / 8, PER = 64 / CH, N = AT_TILE / PER / NW;   // rows of an instruction; instructions
  const uint16_t* const base = src + r0 * stride;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int n = wave * N + j, r = n * PER + lane / CH;
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
// two LDS stages by LDS-DMA, one barrier a tile.  Two waves on each SIMD take turns: while
// one computes its weights the other's products run.
// The weights are powers of two relative to a reference that follows the row's maximum
// only when that has passed it by 2^6: they stay below 2^6, exact as any float, and the
// output is hardly ever rescaled.
constexpr float AT_SLACK = 6.f;

template <int D, int NW>
__global__ __launch_bounds__(64 * NW) void attention_fwd_kernel(AttnArgs a) {
  constexpr int ND = D / 32, NK = D / 16;
  constexpr int TILE = AT_TILE * D * 2;            // bytes of one operand of a stage
  __shared__ __attribute__((aligned(16))) char lds[4 * TILE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & 31, h = lane >> 5;
  if (blockIdx.x == 0) check_sequences(a);
  const int per_block = NW / a.wpr, columns = a.n_heads / per_block;   // heads of a block; blocks of a row tile
  const int hx = blockIdx.x % columns, kvh = hx % a.n_kv;
  const int head = kvh * a.group + hx / a.n_kv * per_block + wave / a.wpr;
  const AttnSeq s = find_sequence(a, a.cu_q, a.tiles - 1 - blockIdx.x / columns, a.shift);
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
  if (tiles) stage(0, 0);
  f32x16 acc[ND];
#pragma unroll
  for (int dt = 0; dt < ND; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[dt][r] = 0.f;
  float ref = -INFINITY, sum = 0.f;

  // where this lane's operands lie in a tile
  uint32_t ka[NK], va[ND][2];
#pragma unroll
  for (int kk = 0; kk < NK; ++kk) ka[kk] = at_lds<D>(l, 2 * kk + h);
#pragma unroll
  for (int dt = 0; dt < ND; ++dt) transposed_at<D>(va[dt], dt, lane);

  const auto step = [&](int t, auto stage_c, auto masked_c) {
    constexpr int K0 = decltype(stage_c)::value * 2 * TILE, V0 = K0 + TILE;
    constexpr bool MASKED = decltype(masked_c)::value;
    const int t0 = t * AT_TILE;
    f32x16 x[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int r = 0; r < 16; ++r) x[u][r] = 0.f;
#pragma unroll
      for (int kk = 0; kk < NK; ++kk)
        x[u] = mfma32(as_bf16x8(*(const uint4*)(lds + K0 + u * 32 * D * 2 + ka[kk])), qf[kk], x[u]);
    }
    if (MASKED) {
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
    if (__any(top > ref + AT_SLACK)) {
      const float next = fmaxf(ref, top), scale = next == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(ref - next);
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
    if (MASKED) {
      bool odd = false;
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) odd |= not_finite(transposed_pair(lds + V0 + b * 16 * D * 2, va[dt]));
      if (__any(odd)) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const bf16x8 p = pack_op(x[b >> 1], b & 1);
#pragma unroll
          for (int dt = 0; dt < ND; ++dt)
            acc[dt] = product_seen(transposed_pair(lds + V0 + b * 16 * D * 2, va[dt]), p, acc[dt], t0 + b * 16, last);
        }
        return;
      }
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const bf16x8 p = pack_op(x[b >> 1], b & 1);
#pragma unroll
      for (int dt = 0; dt < ND; ++dt) acc[dt] = mfma32(transposed_pair(lds + V0 + b * 16 * D * 2, va[dt]), p, acc[dt]);
    }
  };
  // tile t has landed for every wave, and every wave is done with the other stage
  const auto turn = [&](int t, auto stage_c) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (t + 1 < tiles) stage(t + 1, 1 - decltype(stage_c)::value);
    const int t0 = t * AT_TILE;
    if (t0 > wave_last) return;
    if (t0 + AT_TILE - 1 > wave_first || t0 + AT_TILE > s.lk) step(t, stage_c, std::true_type{});
    else step(t, stage_c, std::false_type{});
  };
  for (int t = 0; t < tiles; t += 2) {
    turn(t, std::integral_constant<int, 0>{});
    if (t + 1 < tiles) turn(t + 1, std::integral_constant<int, 1>{});
  }
  if (i >= s.lq) return;
  sum += __shfl_xor(sum, 32, kWave);
  store_row<D>(a.out + (s.q0 + i) * a.o_stride + head * D, acc, sum == 0.f ? 0.f : 1.f / sum, h);
  if (h == 0) a.lse[head * a.n_q + s.q0 + i] = sum == 0.f ? -INFINITY : (ref + __log2f(sum)) * AT_LN2;
}

// ---------------------------------------------------------------- dq
template <int D>
__global__ __launch_bounds__(64 * AT_WAVES) void attention_dq_kernel(AttnArgs a) {
  constexpr int ND = D / 32, NK = D / 16;
  __shared__ uint4 lds[2 * AT_TILE * D / 8];
  char *const kt = (char*)lds, *const vt = kt + AT_TILE * D * 2;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & 31, h = lane >> 5;
  if (blockIdx.x == 0) check_sequences(a);
  const int hx = blockIdx.x % a.n_heads, kvh = hx % a.n_kv, head = kvh * a.group + hx / a.n_kv;
  const AttnSeq s = find_sequence(a, a.cu_q, a.tiles - 1 - blockIdx.x / a.n_heads);
  if (s.tile < 0) return;
  const int row0 = s.tile * AT_ROWS, w0 = row0 + wave * 32, i = w0 + l;
  const int ahead = s.lk - s.lq;
  const int last = a.causal ? min(i + ahead, s.lk - 1) : s.lk - 1;
  const int wave_first = a.causal ? w0 + ahead : s.lk - 1, wave_last = a.causal ? min(w0 + 31 + ahead, s.lk - 1) : s.lk - 1;
  const int keys = a.causal ? min(row0 + AT_ROWS + ahead, s.lk) : s.lk;

  const int64_t row = s.q0 + min(i, s.lq - 1);
  bf16x8 qf[NK], df[NK];
  load_rows<D>(qf, a.q + row * a.q_stride + head * D, h);
  load_rows<D>(df, a.dout + row * a.o_stride + head * D, h);
  float delta = 0.f;
  {
    bf16x8 of[NK];
    load_rows<D>(of, a.o + row * a.o_stride + head * D, h);
#pragma unroll
    for (int kk = 0; kk < NK; ++kk)
#pragma unroll
      for (int j = 0; j < 8; ++j) delta += (float)of[kk][j] * (float)df[kk][j];
    delta += __shfl_xor(delta, 32, kWave);
  }
  const float lse = a.lse[head * a.n_q + row] * AT_LOG2E;
  if (i < s.lq && h == 0) a.delta[head * a.n_q + row] = delta;
  f32x16 acc[ND];
#pragma unroll
  for (int dt = 0; dt < ND; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[dt][r] = 0.f;
  const uint16_t* const kp = a.k + s.k0 * a.k_stride + kvh * D;
  const uint16_t* const vp = a.v + s.k0 * a.v_stride + kvh * D;

  for (int t0 = 0; t0 < keys; t0 += AT_TILE) {
    __syncthreads();
    stage_tile<D>(kt, kp, a.k_stride, t0, s.lk);
    stage_tile<D>(vt, vp, a.v_stride, t0, s.lk);
    __syncthreads();
    if (t0 > wave_last || w0 >= s.lq) continue;
    const bool masked = t0 + AT_TILE - 1 > wave_first || t0 + AT_TILE > s.lk;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      f32x16 x, y;
#pragma unroll
      for (int r = 0; r < 16; ++r) x[r] = y[r] = 0.f;
#pragma unroll
      for (int kk = 0; kk < NK; ++kk) {
        x = mfma32(direct_op<D>(kt, t * 32, kk, l, h), qf[kk], x);
        y = mfma32(direct_op<D>(vt, t * 32, kk, l, h), df[kk], y);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float p = __builtin_amdgcn_exp2f(x[r] * a.scale_log2 - lse);
        x[r] = p * (y[r] - delta);
        if (masked && t0 + t * 32 + result_row(r, h) > last) x[r] = 0.f;
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const bf16x8 ds = pack_op(x, b);
#pragma unroll
        for (int dt = 0; dt < ND; ++dt) acc[dt] = mfma32(transposed_op<D>(kt, t * 32 + b * 16, dt, lane), ds, acc[dt]);
      }
    }
  }
  if (i < s.lq) store_row<D>(a.dq + (s.q0 + i) * a.q_stride + head * D, acc, a.scale, h);
}

// ---------------------------------------------------------------- dk, dv
template <int D>
__global__ __launch_bounds__(64 * AT_WAVES) void attention_dkv_kernel(AttnArgs a) {
  constexpr int ND = D / 32, NK = D / 16;
  __shared__ uint4 lds[2 * AT_TILE * D / 8];
  __shared__ __attribute__((aligned(16))) float lse_s[AT_TILE], delta_s[AT_TILE];
  char *const qt = (char*)lds, *const dt_ = qt + AT_TILE * D * 2;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & 31, h = lane >> 5;
  const int kvh = blockIdx.x % a.n_kv;
  // the first keys are seen by the most queries
  const AttnSeq s = find_sequence(a, a.cu_k, blockIdx.x / a.n_kv);
  if (s.tile < 0) return;
  const int row0 = s.tile * AT_ROWS, w0 = row0 + wave * 32, j = w0 + l;   // key row
  const int ahead = s.lk - s.lq;
  // the first query that sees this lane's key, one of the wave's, one of the block's
  const int first = a.causal ? j - ahead : 0;
  const int wave_first = a.causal ? w0 - ahead : 0, wave_all = a.causal ? w0 + 31 - ahead : 0;
  const int begin = a.causal ? max(row0 - ahead, 0) / AT_TILE * AT_TILE : 0;

  bf16x8 kf[NK], vf[NK];
  const int64_t row = s.k0 + min(j, s.lk - 1);
  load_rows<D>(kf, a.k + row * a.k_stride + kvh * D, h);
  load_rows<D>(vf, a.v + row * a.v_stride + kvh * D, h);
  f32x16 dk[ND], dv[ND];
#pragma unroll
  for (int dt = 0; dt < ND; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) dk[dt][r] = dv[dt][r] = 0.f;

  for (int gh = 0; gh < a.group; ++gh) {
    const int head = kvh * a.group + gh;
    const uint16_t* const qp = a.q + s.q0 * a.q_stride + head * D;
    const uint16_t* const dp = a.dout + s.q0 * a.o_stride + head * D;
    for (int t0 = begin; t0 < s.lq; t0 += AT_TILE) {
      __syncthreads();
      stage_tile<D>(qt, qp, a.q_stride, t0, s.lq);
      stage_tile<D>(dt_, dp, a.o_stride, t0, s.lq);
      if (threadIdx.x < AT_TILE) {
        const bool in = t0 + (int)threadIdx.x < s.lq;
        const int64_t at = head * a.n_q + s.q0 + t0 + threadIdx.x;
        // rows that do not exist, and queries that see no key, weigh 0
        const float v = in ? a.lse[at] : INFINITY;
        lse_s[threadIdx.x] = v == -INFINITY ? INFINITY : v * AT_LOG2E;
        delta_s[threadIdx.x] = in ? a.delta[at] : 0.f;
      }
      __syncthreads();
      if (t0 + AT_TILE - 1 < wave_first || w0 >= s.lk) continue;
      const bool masked = t0 < wave_all;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x16 x, y;
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = y[r] = 0.f;
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
          x = mfma32(direct_op<D>(qt, t * 32, kk, l, h), kf[kk], x);
          y = mfma32(direct_op<D>(dt_, t * 32, kk, l, h), vf[kk], y);
        }
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const f32x4 ls = *(const f32x4*)(lse_s + t * 32 + 8 * r4 + 4 * h), de = *(const f32x4*)(delta_s + t * 32 + 8 * r4 + 4 * h);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int r = r4 * 4 + c;
            x[r] = __builtin_amdgcn_exp2f(x[r] * a.scale_log2 - ls[c]);
            y[r] = x[r] * (y[r] - de[c]);
            if (masked && t0 + t * 32 + result_row(r, h) < first) x[r] = y[r] = 0.f;
          }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const bf16x8 p = pack_op(x, b), ds = pack_op(y, b);
#pragma unroll
          for (int dt = 0; dt < ND; ++dt) {
            dv[dt] = mfma32(transposed_op<D>(dt_, t * 32 + b * 16, dt, lane), p, dv[dt]);
            dk[dt] = mfma32(transposed_op<D>(qt, t * 32 + b * 16, dt, lane), ds, dk[dt]);
          }
        }
      }
    }
  }
  if (j >= s.lk) return;
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
  a.delta = (float*)((char*)ws + 256);
  a.q_stride = sh.q_stride, a.k_stride = sh.k_stride, a.v_stride = sh.v_stride, a.o_stride = sh.o_stride;
  a.n_q = sh.n_q, a.n_k = sh.n_k, a.n_seqs = sh.n_seqs, a.n_heads = sh.n_heads, a.n_kv = sh.n_kv_heads;
  a.group = sh.n_heads / sh.n_kv_heads, a.causal = sh.causal;
  a.scale = sh.scale, a.scale_log2 = sh.scale * AT_LOG2E;
  return a;
}
static int attn_tiles(int64_t n, int n_seqs) { return (int)(n / AT_ROWS) + n_seqs; }

lora_status launch_attention_fwd(const attn_shape& sh, const uint16_t* q, const uint16_t* k,
                                 const uint16_t* v, const int32_t* cu_q, const int32_t* cu_k,
                                 uint16_t* o, float* lse, void* ws, hipStream_t s) {
  AttnArgs a = attn_args(sh, q, k, v, cu_q, cu_k, ws);
  a.out = o, a.lse = lse;
  const auto tiles = [&](int shift) { return (sh.n_q >> shift) + sh.n_seqs; };
  // eight waves where that leaves a block for each CU: two heads of a group, or 256 rows
  int waves = 8, heads = a.group % 2 == 0 ? 2 : 1;
  a.shift = heads == 2 ? 7 : 8;
  if (tiles(a.shift) * (a.n_heads / heads) < device_cus()) waves = 4, heads = 1, a.shift = 7;
  a.wpr = waves / heads;
  a.tiles = (int)tiles(a.shift);
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((int64_t)a.tiles * (a.n_heads / heads))), dim3(64 * waves), 0, s, a);
  };
  if (sh.head_dim == 128) waves == 8 ? go(attention_fwd_kernel<128, 8>) : go(attention_fwd_kernel<128, 4>);
  else waves == 8 ? go(attention_fwd_kernel<64, 8>) : go(attention_fwd_kernel<64, 4>);
  return launch_check("attention_forward");
}

lora_status launch_attention_bwd(const attn_shape& sh, const uint16_t* dout, const uint16_t* q,
                                 const uint16_t* k, const uint16_t* v, const uint16_t* o,
                                 const float* lse, const int32_t* cu_q, const int32_t* cu_k,
                                 uint16_t* dq, uint16_t* dk, uint16_t* dv, void* ws, hipStream_t s) {
  AttnArgs a = attn_args(sh, q, k, v, cu_q, cu_k, ws);
  a.dout = dout, a.o = o, a.lse = const_cast<float*>(lse), a.dq = dq, a.dk = dk, a.dv = dv;
  a.tiles = attn_tiles(sh.n_q, sh.n_seqs);
  const dim3 block(64 * AT_WAVES), grid_q((unsigned)((int64_t)a.tiles * a.n_heads));
  // dq first: it also leaves delta for the other kernel
  if (sh.head_dim == 128) hipLaunchKernelGGL(attention_dq_kernel<128>, grid_q, block, 0, s, a);
  else hipLaunchKernelGGL(attention_dq_kernel<64>, grid_q, block, 0, s, a);
  lora_status st = launch_check("attention_backward dq");
  if (st != LORA_OK) return st;
  a.tiles = attn_tiles(sh.n_k, sh.n_seqs);
  const dim3 grid_k((unsigned)((int64_t)a.tiles * a.n_kv));
  if (sh.head_dim == 128) hipLaunchKernelGGL(attention_dkv_kernel<128>, grid_k, block, 0, s, a);
  else hipLaunchKernelGGL(attention_dkv_kernel<64>, grid_k, block, 0, s, a);
  return launch_check("attention_backward dk, dv");
}

}  // namespace lora_host
