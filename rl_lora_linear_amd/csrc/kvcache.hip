// The paged key-value cache on gfx950: block tables and slot maps from request lengths,
// new rows into the pages, and the attention of one new token of each request.
#include <cmath>

#include "attn.hpp"
#include "q8.hpp"

namespace lora {

constexpr float KV_LOG2E = 1.4426950408889634f, KV_LN2 = 0.6931471805599453f;

// ---------------------------------------------------------------- block tables and slots
// All of it follows from running sums over the requests of three counts: new rows, pages
// needed, pages put back.  Requests number at most some thousands, so every block sums
// them itself (a few per thread) and keeps the sums in LDS; then new rows, new table
// entries and returned pages are independent items, each found by a binary search.  One
// launch does all: of one block, or of a grid where outputs do not lie on inputs.  Where
// they do (seq_lens over cached_lens, the state over itself) no block of a grid may see
// them changed, so a second launch of one block writes them.
// Bound by the chain of a launch, the lengths' loads, the scan's barriers and the dependent
// loads of an item (its request, its page): 64 requests 6.7-7.0 us, 1000 requests with 104 000
// new rows 9.5-9.8 us (1.3 MB; 15.7 as two launches).  Scans kept in memory between launches, or
// one block that hands them to others, would wait for a launch or a flag instead.
constexpr int TAB_THREADS = 1024;

struct TableArgs {
  const int32_t* cached;
  const int32_t* fresh;
  int32_t* seq_lens;
  int32_t* table;
  int32_t* ring;
  const int64_t* state;
  int64_t* state_out;
  int32_t* cu_new;
  int32_t* slots;
  int32_t* positions;
  int32_t* token_seqs;
  int32_t* status;
  int64_t n_slots;
  int32_t n, page_shift, n_pages, max_pages;
  int32_t items, lengths;   // which halves this launch does (the second by its first block)
};

// What one request asks for.
struct Request {
  int32_t cached, rows, owned, need, back;
  bool bad;
};
__device__ __forceinline__ Request request_of(const TableArgs& a, int b) {
  const int64_t cached = a.cached[b], fresh = a.fresh[b];
  const int64_t room = (int64_t)a.max_pages << a.page_shift;
  const int64_t pad = (1 << a.page_shift) - 1;
  Request r;
  r.rows = (int32_t)max(fresh, (int64_t)0);
  r.bad = cached < 0 || cached + r.rows > room;
  r.cached = (int32_t)cached;
  r.owned = r.bad ? 0 : (int32_t)((cached + pad) >> a.page_shift);
  r.need = r.bad || fresh < 0 ? 0 : (int32_t)((cached + r.rows + pad) >> a.page_shift) - r.owned;
  r.back = fresh < 0 ? r.owned : 0;
  return r;
}

struct Sums {
  int64_t rows, need, back;
};

// Exclusive running sums over the block's threads; `total` is the block's.
__device__ __forceinline__ Sums block_scan(Sums v, Sums& total, Sums* waves) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Sums s = v;
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t x = __shfl_up(s.rows, o, kWave), y = __shfl_up(s.need, o, kWave),
                  z = __shfl_up(s.back, o, kWave);
    if (lane >= o) s.rows += x, s.need += y, s.back += z;
  }
  if (lane == 63) waves[wave] = s;
  __syncthreads();
  Sums before{0, 0, 0};
  total = {0, 0, 0};
  for (int w = 0; w < TAB_THREADS / 64; ++w) {
    const Sums t = waves[w];
    if (w < wave) before.rows += t.rows, before.need += t.need, before.back += t.back;
    total.rows += t.rows, total.need += t.need, total.back += t.back;
  }
  return {before.rows + s.rows - v.rows, before.need + s.need - v.need, before.back + s.back - v.back};
}

// The largest b in [lo, hi] with pre[b] <= i.
__device__ __forceinline__ int last_at_most(const int32_t* pre, int lo, int hi, int32_t i) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// PRE: the running sums [n] of rows, pages taken and pages put, in LDS; they stop at
// values that no valid item reaches, so 32 bits hold them.
__global__ __launch_bounds__(TAB_THREADS) void kv_tables_kernel(TableArgs a) {
  extern __shared__ int32_t pre[];
  __shared__ Sums waves[TAB_THREADS / 64];
  __shared__ int32_t taken_s, flags_s;
  int32_t *rows_at = pre, *take_at = pre + a.n, *back_at = pre + 2 * a.n;
  const int tid = threadIdx.x;
  if (tid == 0) taken_s = flags_s = 0;
  int64_t head = a.state[0], tail = a.state[1];
  const bool state_ok = head >= 0 && tail >= head && tail - head <= a.n_pages;
  const int64_t avail = state_ok ? tail - head : 0;
  const int per = (a.n + TAB_THREADS - 1) / TAB_THREADS;
  const int b0 = min(tid * per, a.n), b1 = min(b0 + per, a.n);

  Sums mine{0, 0, 0}, total;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(a, b);
    mine.rows += r.rows, mine.need += r.need, mine.back += r.back;
  }
  Sums at = block_scan(mine, total, waves);
  const int64_t cap = a.n_slots;
  int32_t flags = state_ok ? 0 : LORA_FLAG_BAD_PAGE, taken = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(a, b);
    // the sums are clamped where they pass every item: rows at n_slots, pages at n_pages + 1
    rows_at[b] = (int32_t)min(at.rows, cap);
    back_at[b] = (int32_t)min(at.back, (int64_t)a.n_pages + 1);
    const bool fits = !r.bad && (r.rows == 0 || at.rows + r.rows <= cap);
    const bool paged = r.need == 0 || at.need + r.need <= avail;
    // a request left out takes no page: the sign bit of its sum says so
    const int32_t t = (int32_t)min(at.need, (int64_t)a.n_pages + 1);
    take_at[b] = fits && paged ? t : ~t;
    if (fits && paged && r.need) taken = (int32_t)(at.need + r.need);
    if (!fits) flags |= LORA_FLAG_BAD_LENGTH;
    else if (!paged) flags |= LORA_FLAG_NO_PAGES;
    at.rows += r.rows, at.need += r.need, at.back += r.back;
  }
  // pages taken: up to the last served request that needs some
  for (int o = 32; o; o >>= 1) {
    taken = max(taken, __shfl_xor(taken, o, kWave));
    flags |= __shfl_xor(flags, o, kWave);
  }
  if ((tid & 63) == 0) {
    atomicMax(&taken_s, taken);
    if (flags) atomicOr(&flags_s, flags);
  }
  __syncthreads();
  taken = taken_s;
  // pages put must leave alone the ring's entries that are free, those taken now included
  const bool put_ok = state_ok && total.back <= a.n_pages - avail;
  const int32_t n_put = put_ok ? (int32_t)total.back : 0;
  const int32_t n_rows = (int32_t)min(total.rows, cap);
  const int32_t head0 = state_ok ? (int32_t)(head % a.n_pages) : 0, tail0 = state_ok ? (int32_t)(tail % a.n_pages) : 0;
  const auto ring_at = [&](int32_t from, int32_t i) {
    const int64_t j = (int64_t)from + i;
    return (int32_t)(j >= a.n_pages ? j - a.n_pages : j);
  };
  int32_t bad = 0;

  if (a.items) {
    const int64_t step = (int64_t)gridDim.x * TAB_THREADS, first = (int64_t)blockIdx.x * TAB_THREADS + tid;
    for (int64_t t = first; t < a.n_slots; t += step) {
      int32_t slot = -1, pos = -1, seq = -1;
      if (t < n_rows) {
        seq = last_at_most(rows_at, 0, a.n - 1, (int32_t)t);
        const Request r = request_of(a, seq);
        if (!r.bad) pos = r.cached + (int32_t)t - rows_at[seq];
        if (take_at[seq] >= 0) {
          const int32_t p = pos >> a.page_shift;
          const int32_t page = p < r.owned ? a.table[(int64_t)seq * a.max_pages + p]
                                           : a.ring[ring_at(head0, take_at[seq] + p - r.owned)];
          if ((uint32_t)page < (uint32_t)a.n_pages) slot = (page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
          else bad = LORA_FLAG_BAD_PAGE;
        }
      }
      a.slots[t] = slot;
      if (a.positions) a.positions[t] = pos;
      if (a.token_seqs) a.token_seqs[t] = seq;
    }
    if (a.cu_new)
      for (int64_t b = first; b <= a.n; b += step) a.cu_new[b] = b < a.n ? rows_at[b] : n_rows;
    // table entries and returned pages: a wave goes through a request's pages
    const int lane = tid & 63;
    const int64_t wave = (int64_t)blockIdx.x * (TAB_THREADS / 64) + (tid >> 6);
    for (int64_t b = wave; b < a.n; b += (int64_t)gridDim.x * (TAB_THREADS / 64)) {
      const Request r = request_of(a, (int)b);
      if (take_at[b] >= 0)
        for (int32_t j = lane; j < r.need; j += 64) {
          const int32_t page = a.ring[ring_at(head0, take_at[b] + j)];
          a.table[b * a.max_pages + r.owned + j] = page;
          if ((uint32_t)page >= (uint32_t)a.n_pages) bad = LORA_FLAG_BAD_PAGE;
        }
      if (n_put)
        for (int32_t j = lane; j < r.back; j += 64) {
          const int32_t page = a.table[b * a.max_pages + j];
          a.ring[ring_at(tail0, back_at[b] + j)] = page;
          if ((uint32_t)page >= (uint32_t)a.n_pages) bad = LORA_FLAG_BAD_PAGE;
        }
    }
  }
  if (bad) set_flag(a.status, bad);
  if (!a.lengths || blockIdx.x) return;
  // every thread has read what these overwrite; each rewrites its own requests
  __syncthreads();
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(a, b);
    const bool ended = a.fresh[b] < 0;
    a.seq_lens[b] = take_at[b] < 0 ? r.cached : ended ? 0 : r.cached + r.rows;
  }
  if (tid == 0) {
    const int32_t f = flags_s | (put_ok || total.back == 0 ? 0 : LORA_FLAG_BAD_PAGE);
    if (f) set_flag(a.status, f);
    a.state_out[0] = head + taken;
    a.state_out[1] = tail + n_put;
  }
}

// ---------------------------------------------------------------- new rows into the pages
// A lane moves 8 columns: 16 bytes in, 16 (or 8 and, from one lane of four, a scale) out.
// Bound by memory: in 8 bits 16381 rows of 8 heads of 128, 67 MB in and 34 out, 20-21.5 us,
// 4.7-5.0 TB/s (a large copy: 5.2); 64 rows in bf16 2.6 us, a launch.
// The codes are the norm's 8-bit form, so that its rounding (half a step of e4m3, 2^-4 of a
// value) is the only one.
struct WriteArgs {
  const uint16_t *k, *v;
  const int32_t* slots;
  void *kc, *vc;
  uint8_t *ks, *vs;
  int32_t* status;
  int64_t k_stride, v_stride, n;
  int32_t n_kv, page_shift;
  int32_t n_slots;   // of the cache
};

template <int D, bool X8>
__global__ __launch_bounds__(256) void kv_write_kernel(WriteArgs a) {
  constexpr int PIECES = D / 8;
  const int per_row = a.n_kv * PIECES;
  const int64_t end = a.n * 2 * per_row;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < end; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / (2 * per_row);
    const int j = (int)(i - t * 2 * per_row);
    const bool is_v = j >= per_row;
    const int c = is_v ? j - per_row : j, head = c / PIECES, piece = c % PIECES;
    const int32_t slot = a.slots[t];
    if (slot < 0 || slot >= a.n_slots) {
      if (slot != -1 && j == 0) set_flag(a.status, LORA_FLAG_BAD_PAGE);
      continue;   // (the four lanes that share a scale share a row: all go or none)
    }
    const uint4 x = *(const uint4*)((is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + c * 8);
    const int64_t page = slot >> a.page_shift, row = slot & ((1 << a.page_shift) - 1);
    const int64_t at = (((page * a.n_kv + head) << a.page_shift) + row) * PIECES + piece;
    if (!X8) {
      ((uint4*)(is_v ? a.vc : a.kc))[at] = x;
      continue;
    }
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float f[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) f[2 * q] = bf2f_lo(w[q]), f[2 * q + 1] = bf2f_hi(w[q]);
    int b;
    const uint2 code = quantize8(f, b);
    ((uint2*)(is_v ? a.vc : a.kc))[at] = code;
    if ((piece & 3) == 0) (is_v ? a.vs : a.ks)[at >> 2] = (uint8_t)b;
  }
}

// ---------------------------------------------------------------- one token of each request
// A block takes a run of a request's keys for one key head (and up to 16 of its query
// heads: the columns of a 16x16x32 matrix instruction, so a group of any size costs one
// pass over the cache).  Its four waves take tiles of 32 keys in turn.
//   S^T = K Q^T: lane (l, g) = (lane & 15, lane >> 4) holds key l's chunk as operand and
//   ends with column (query head) l, keys 4g .. 4g+3 of the 16;
//   O^T += V^T P^T: those are the operand of P as they lie, where the instruction's key
//   8g + j means key 4g + j of the tile's first 16 keys (j < 4) or second (j >= 4).  V's
//   operand for the same order comes from LDS by transposing reads.
// So nothing but the maximum and the sum crosses lanes, and each lane rescales the output
// of its own query head.
//
// Where the length is cut must not show in the result, or a request's bits would change
// with the batch.  So the sums have one shape, by the request's length alone: units of
// DEC_UNIT keys (more where that makes more than 32 of them), in which each wave keeps a
// running maximum, sum and output and the four are added; and the units' results
// (maximum, sum, output) joined two by two, neighbours first, as the leaves of a binary
// tree.  A block takes an aligned run of 2^k units, a subtree, whatever k suits the batch;
// what is left of the tree is joined by a second kernel.
//
// Scores, weights' sums and outputs are fp32; the weights are rounded to bf16 to be an operand
// (half a step, 2^-8 of a weight), and the output once at the end.
// Bound by memory where the batch is large: 64 requests of 2500 to 8000 tokens, 8 key heads of
// 128 in bf16 (1.37 GB): 237-250 us and 5 to join, 5.5-5.8 TB/s, the rate of a large copy.  In 8
// bits, 250 requests of 900 to 3000, 4 key heads (0.51 GB): 101-107 us and 5, 4.8-5 TB/s: the
// conversion of two codes at a time and the V tile's way through LDS take turns with the
// loads of 12 waves.  One request of 4001: 7.0-7.4 us and 2.6-3.5, each a launch and a chain of
// three loads (length, page, rows).  Asking two tiles ahead, and loads past the caches, were
// no faster.
// Units of 256 keys are two tiles a wave before the four waves' sums are joined (128: 250
// requests of 1000 in bf16 152 us against 145, 16 of 1000 16 against 14; one of 4001 9.3 against
// 10.3), and 32 of them the most that a second kernel joins in one step.
constexpr int DEC_WAVES = 4, DEC_TILE = 32, DEC_STRIPE = DEC_WAVES * DEC_TILE, DEC_UNIT = 256, DEC_MAX_UNITS = 32;
constexpr float DEC_SLACK = 6.f;
constexpr int DEC_MAX_SPAN = 8;      // units of a block that takes its request whole, at most
constexpr int DEC_CUT_SPAN = 4;      // of one that takes a part; see decode_plan
constexpr int DEC_CU_BLOCKS = 9;     // blocks of a CU that so long a block has to leave

__host__ __device__ __forceinline__ int decode_unit(int len) {
  int s = DEC_UNIT;
  while ((int64_t)s * DEC_MAX_UNITS < len) s *= 2;
  return s;
}

// A piece of the result: four columns of an output, with its row's maximum (in powers of
// two) and sum, relative to which it stands.
struct DecNode {
  f32x4 o;
  float m, sum;
};
__device__ __forceinline__ DecNode dec_join(const DecNode& x, const DecNode& y) {
  const float m = fmaxf(x.m, y.m), ref = m == -INFINITY ? 0.f : m;
  const float a = __builtin_amdgcn_exp2f(x.m - ref), b = __builtin_amdgcn_exp2f(y.m - ref);
  DecNode r;
  r.m = m;
  r.sum = __builtin_fmaf(x.sum, a, y.sum * b);
#pragma unroll
  for (int i = 0; i < 4; ++i) r.o[i] = __builtin_fmaf(x.o[i], a, y.o[i] * b);
  return r;
}

struct DecodeArgs {
  const uint16_t* q;
  const void *kc, *vc;
  const uint8_t *ks, *vs;
  const int32_t *table, *lens;
  uint16_t* o;
  float* lse;
  float* part;       // [n][heads][nodes][D] outputs of the blocks' runs
  float2* stat;      // [n][heads][nodes] their maxima and sums
  int32_t* status;
  int64_t q_stride;
  int32_t n_heads, n_kv, group, page_shift, n_pages, max_pages, max_len, nodes, span, col_groups;
  float scale_log2;
  uint32_t q_turn, q_keep;
};

// Four columns from c on of a row's output, and with the first its lse.
__device__ __forceinline__ void dec_store(const DecodeArgs& a, int64_t row, int D, int c, const DecNode& v) {
  const float mul = v.sum == 0.f ? 0.f : 1.f / v.sum;
  *(uint2*)(a.o + row * D + c) = make_uint2(pack2bf(v.o[0] * mul, v.o[1] * mul), pack2bf(v.o[2] * mul, v.o[3] * mul));
  if (a.lse && c == 0) a.lse[row] = v.sum == 0.f ? -INFINITY : (v.m + __log2f(v.sum)) * KV_LN2;
}

__device__ __forceinline__ bf16x8 kv_widen(uint32_t lo, uint32_t hi, float scale) {
  uint32_t r[4];
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true));
  return as_bf16x8(make_uint4(r[0], r[1], r[2], r[3]));
}

// V rows in LDS, D columns of bf16: 16-byte chunk c of row r lies at chunk c ^ swz(r), so
// that the 8 rows by 32 bytes that half a wave reads transposed lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t dec_v_at(int row, int chunk) {
  const int s = D == 128 ? (row & 7) << 1 : ((row >> 1) & 3) << 1;
  return (uint32_t)(row * (D * 2) + ((chunk ^ s) << 4));
}

// What a wave holds of a tile on its way: the lane's pieces of K as operands, and of V as
// they go to LDS.  In 8 bits a piece is 16 codes, and its scale rides along.
template <int D, bool X8>
struct DecTile {
  static constexpr int KP = D / (X8 ? 64 : 32);                 // pieces of a key row per lane
  static constexpr int VP = DEC_TILE * D * (X8 ? 1 : 2) / 1024; // pieces of the V rows per lane
  uint4 k[2][KP], v[VP];
  uint32_t ks[X8 ? 2 : 1], vs[X8 ? VP : 1];
  int n[2];   // keys that exist among the first 16 and the second 16
};

// The pages of a tile's two halves (a page holds 16 rows at least, so a half lies in one);
// asked for a tile ahead of its rows.
struct DecPages {
  int32_t p[2];
};
__device__ __forceinline__ DecPages dec_pages(const DecodeArgs& a, const int32_t* table, int t0, int k1) {
  DecPages r{{0, 0}};
#pragma unroll
  for (int t = 0; t < 2; ++t)
    if (t0 + 16 * t < k1) r.p[t] = table[(t0 + 16 * t) >> a.page_shift];
  return r;
}

// Asks for all rows of tile t0.  Rows behind the request's last one lie in its last page and
// are fetched like the others; for a half that has no page, rows of page 0 are.
template <int D, bool X8>
__device__ __forceinline__ void dec_ask(const DecodeArgs& a, DecPages pages, int kvh, int t0, int k1, int lane,
                                        DecTile<D, X8>& x, bool& bad) {
  using T = DecTile<D, X8>;
  constexpr int ROW = D * (X8 ? 1 : 2);
  const int l = lane & 15, g = lane >> 4;
  int64_t row[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int key = t0 + 16 * t;
    x.n[t] = min(max(k1 - key, 0), 16);
    uint32_t page = 0;
    if (x.n[t]) {
      page = (uint32_t)__builtin_amdgcn_readfirstlane(pages.p[t]);
      if (page >= (uint32_t)a.n_pages) bad = true, x.n[t] = 0, page = 0;
    }
    row[t] = (((int64_t)page * a.n_kv + kvh) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const char* const at = (const char*)a.kc + row[t] * ROW;
#pragma unroll
    for (int i = 0; i < T::KP; ++i) x.k[t][i] = *(const uint4*)(at + (uint32_t)(l * ROW + i * 64 + g * 16));
    if (X8) {
      const uint8_t* const sc = a.ks + row[t] * (D / 32) + (uint32_t)(l * (D / 32));
      x.ks[t] = D == 128 ? *(const uint32_t*)sc : *(const uint16_t*)sc;
    }
  }
  constexpr int LPR = ROW / 16, PER = 64 / LPR;    // lanes of a row, rows of an instruction
#pragma unroll
  for (int i = 0; i < T::VP; ++i) {
    const int r = i * PER % 16;                    // first row within its half
    const int64_t r0 = row[i * PER / 16] + r;
    x.v[i] = *(const uint4*)((const char*)a.vc + r0 * ROW + (uint32_t)(lane * 16));
    if (X8) x.vs[i] = *(a.vs + r0 * (D / 32) + (uint32_t)(lane >> 1));
  }
}

// ITEMS: pieces of the result per thread (1: up to 8 heads of 128 columns).
template <int D, bool X8, int ITEMS>
__global__ __launch_bounds__(64 * DEC_WAVES, X8 ? 3 : 2) void decode_kernel(DecodeArgs a) {
  using T = DecTile<D, X8>;
  constexpr int NK = D / 32;            // steps of 32 columns
  constexpr int ND = D / 16;            // output tiles of 16 columns
  constexpr int V_BYTES = DEC_TILE * D * 2;
  __shared__ uint4 lds[DEC_WAVES * V_BYTES / 16];
  __shared__ float2 ms[DEC_WAVES][16];
  __shared__ f32x4 left_o[3][ITEMS][64 * DEC_WAVES];    // of a subtree that waits for its neighbour: the thread's own
  __shared__ float2 left_ms[3][ITEMS][64 * DEC_WAVES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & 15, g = lane >> 4;
  const int heads_at = blockIdx.x % (a.n_kv * a.col_groups);
  const int rest = blockIdx.x / (a.n_kv * a.col_groups);
  const int node = rest % a.nodes, b = rest / a.nodes;
  const int kvh = heads_at / a.col_groups, cols0 = heads_at % a.col_groups * 16;
  const int cols = min(16, a.group - cols0);
  int len = a.lens[b];
  if ((uint32_t)len > (uint32_t)a.max_len) {
    if (node == 0 && heads_at == 0 && threadIdx.x == 0) set_flag(a.status, LORA_FLAG_BAD_LENGTH);
    len = 0;
  }
  const int unit = decode_unit(len), run = unit * a.span;
  const int k0 = node * run, k1 = min(k0 + run, len);
  if (k0 >= len && node > 0) return;   // the first also writes a request without keys
  const bool only = len <= run;

  // Q as operand: lane (l, g) holds 8 columns of query head l for each step.  In 8 bits
  // a lane's 16 codes are the columns of two steps.
  const auto col_of = [&](int kk) { return X8 ? (kk >> 1) * 64 + g * 16 + (kk & 1) * 8 : kk * 32 + g * 8; };
  bf16x8 qf[NK];
  const int head0 = kvh * a.group + cols0;
  // a negative scale turns q's signs, a scale of 0 makes q 0 (scale_log2 is positive)
#pragma unroll
  for (int kk = 0; kk < NK; ++kk) {
    const uint4 u = l < cols ? *(const uint4*)(a.q + b * a.q_stride + (int64_t)(head0 + l) * D + col_of(kk)) : make_uint4(0, 0, 0, 0);
    qf[kk] = as_bf16x8(make_uint4((u.x ^ a.q_turn) & a.q_keep, (u.y ^ a.q_turn) & a.q_keep, (u.z ^ a.q_turn) & a.q_keep,
                                  (u.w ^ a.q_turn) & a.q_keep));
  }
  const int32_t* const table = a.table + (int64_t)b * a.max_pages;
  bool bad = false;
  T x;
  const int first = k0 + wave * DEC_TILE;
  dec_ask<D, X8>(a, dec_pages(a, table, first, k1), kvh, first, k1, lane, x, bad);
  DecPages pages = dec_pages(a, table, first + DEC_STRIPE, k1);

  f32x4 acc[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, sum = 0.f;
  char* const vl = (char*)lds + wave * V_BYTES;

  const auto tile = [&](int t0) {
    // ---- scores of 32 keys
    f32x4 s[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < T::KP; ++i) {
        if (X8) {
          const float sc = e8m0(x.ks[t] >> (8 * (2 * i + (g >> 1))) & 255);
          s[t] = mfma16(kv_widen(x.k[t][i].x, x.k[t][i].y, sc), qf[2 * i], s[t]);
          s[t] = mfma16(kv_widen(x.k[t][i].z, x.k[t][i].w, sc), qf[2 * i + 1], s[t]);
        } else {
          s[t] = mfma16(as_bf16x8(x.k[t][i]), qf[i], s[t]);
        }
      }
    }
    const int n0 = x.n[0], n1 = x.n[1];
    const bool whole = n0 + n1 == DEC_TILE;
    // ---- V rows into LDS: rows that do not exist as zeros, whatever lies there
    constexpr int LPR = X8 ? D / 16 : D / 8, PER = 64 / LPR;
    if (!whole) {
#pragma unroll
      for (int i = 0; i < T::VP; ++i) {
        const int r = i * PER + lane / LPR;
        const bool live = (r & 15) < (r < 16 ? n0 : n1);
        x.v[i] = live ? x.v[i] : make_uint4(0, 0, 0, 0);
        if (X8) x.vs[i] = live ? x.vs[i] : 127;
      }
    }
#pragma unroll
    for (int i = 0; i < T::VP; ++i) {
      const int r = i * PER + lane / LPR, c = lane % LPR;
      const uint4 w = x.v[i];
      if (X8) {
        const float sc = e8m0(x.vs[i]);
        *(bf16x8*)(vl + dec_v_at<D>(r, 2 * c)) = kv_widen(w.x, w.y, sc);
        *(bf16x8*)(vl + dec_v_at<D>(r, 2 * c + 1)) = kv_widen(w.z, w.w, sc);
      } else {
        *(uint4*)(vl + dec_v_at<D>(r, c)) = w;
      }
    }
    if (t0 + DEC_STRIPE < k1) dec_ask<D, X8>(a, pages, kvh, t0 + DEC_STRIPE, k1, lane, x, bad);
    pages = dec_pages(a, table, t0 + 2 * DEC_STRIPE, k1);
    // ---- softmax: weights relative to a reference that follows the maximum only when that
    // has passed it by 2^6
    if (!whole) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (4 * g + r >= (t ? n1 : n0)) s[t][r] = -INFINITY;
    }
    float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])), fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
    top = fmaxf(top, __shfl_xor(top, 16, kWave));
    top = fmaxf(top, __shfl_xor(top, 32, kWave)) * a.scale_log2;
    const bool rise = top > m + DEC_SLACK;
    if (__any(rise)) {
      const float next = rise ? top : m, keep = rise ? __builtin_amdgcn_exp2f(m - next) : 1.f;
      m = next;
      sum *= keep;
#pragma unroll
      for (int i = 0; i < ND; ++i) acc[i] *= keep;
    }
    const float ref = m == -INFINITY ? 0.f : m;
    uint32_t p[4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float e[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) sum += e[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][r], a.scale_log2, -ref));
      p[2 * t] = pack2bf(e[0], e[1]);
      p[2 * t + 1] = pack2bf(e[2], e[3]);
    }
    const bf16x8 pf = as_bf16x8(make_uint4(p[0], p[1], p[2], p[3]));
    // ---- output
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      const int r = 4 * g + (l >> 2), c = 2 * i + ((l & 3) >> 1), lo = (l & 1) * 8;
      const uint2 v0 = tr_read((const uint4*)vl, dec_v_at<D>(r, c) + lo);
      const uint2 v1 = tr_read((const uint4*)vl, dec_v_at<D>(r + 16, c) + lo);
      acc[i] = mfma16(as_bf16x8(make_uint4(v0.x, v0.y, v1.x, v1.y)), pf, acc[i]);
    }
    __builtin_amdgcn_wave_barrier();
  };

  // ---- the waves' results of a unit, added in wave order (its V tiles are done with);
  // thread t holds piece t of the 16 D / 4
  DecNode value[ITEMS];
  const auto join_waves = [&]() {
    sum += __shfl_xor(sum, 16, kWave);
    sum += __shfl_xor(sum, 32, kWave);
    if (g == 0) ms[wave][l] = make_float2(m, sum);
    float* const of = (float*)lds + wave * (16 * D);
#pragma unroll
    for (int i = 0; i < ND; ++i) *(f32x4*)(of + l * D + ((i * 16 + 4 * g) ^ ((l & 7) << 2))) = acc[i];
    __syncthreads();
#pragma unroll
    for (int t = 0; t < ITEMS; ++t) {
      const int i = t * 64 * DEC_WAVES + threadIdx.x, h = i / (D / 4) & 15, c = i % (D / 4) * 4;
      const float* const src = (const float*)lds + h * D + (c ^ ((h & 7) << 2));
      DecNode v;
      v.m = fmaxf(fmaxf(ms[0][h].x, ms[1][h].x), fmaxf(ms[2][h].x, ms[3][h].x));
      v.sum = 0.f;
      v.o = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < DEC_WAVES; ++w) {
        const float f = __builtin_amdgcn_exp2f(ms[w][h].x - (v.m == -INFINITY ? 0.f : v.m));
        v.sum = __builtin_fmaf(ms[w][h].y, f, v.sum);
        const f32x4 p = *(const f32x4*)(src + w * 16 * D);
#pragma unroll
        for (int q = 0; q < 4; ++q) v.o[q] = __builtin_fmaf(p[q], f, v.o[q]);
      }
      value[t] = v;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ND; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    m = -INFINITY, sum = 0.f;
  };

  int units = 0;   // whole units so far: bit k says that left[k] waits for its neighbour
  for (int u0 = k0; u0 < k1;) {
    const int end = min(u0 + unit, k1);
    for (int s0 = u0; s0 < end; s0 += DEC_STRIPE)
      if (s0 + wave * DEC_TILE < k1) tile(s0 + wave * DEC_TILE);
    join_waves();
    u0 = end;
    if (u0 == k1) break;
    bool open = true;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (!open) continue;
      open = units >> k & 1;
#pragma unroll
      for (int t = 0; t < ITEMS; ++t) {
        if (open) value[t] = dec_join(DecNode{left_o[k][t][threadIdx.x], left_ms[k][t][threadIdx.x].x, left_ms[k][t][threadIdx.x].y}, value[t]);
        else left_o[k][t][threadIdx.x] = value[t].o, left_ms[k][t][threadIdx.x] = make_float2(value[t].m, value[t].sum);
      }
    }
    ++units;
  }
  if (k0 >= k1) join_waves();
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (units >> k & 1) {
#pragma unroll
      for (int t = 0; t < ITEMS; ++t)
        value[t] = dec_join(DecNode{left_o[k][t][threadIdx.x], left_ms[k][t][threadIdx.x].x, left_ms[k][t][threadIdx.x].y}, value[t]);
    }
  if (bad) set_flag(a.status, LORA_FLAG_BAD_PAGE);

  const int64_t bh = (int64_t)b * a.n_heads + head0;
#pragma unroll
  for (int t = 0; t < ITEMS; ++t) {
    const int i = t * 64 * DEC_WAVES + threadIdx.x, h = i / (D / 4), c = i % (D / 4) * 4;
    if (h >= cols) continue;
    if (only) dec_store(a, bh + h, D, c, value[t]);
    else {
      *(f32x4*)(a.part + ((bh + h) * a.nodes + node) * D + c) = value[t].o;
      if (c == 0) a.stat[(bh + h) * a.nodes + node] = make_float2(value[t].m, value[t].sum);
    }
  }
}

// What is left of the trees: GROUPS groups of D / 4 threads a row (request and head), each
// thread with four neighbouring nodes' pieces, then the groups' through LDS.
template <int D, int GROUPS>
__global__ __launch_bounds__(256) void decode_join_kernel(DecodeArgs a, int64_t rows) {
  constexpr int LANES = D / 4, ROWS = 256 / LANES / GROUPS;
  __shared__ DecNode lds[GROUPS > 1 ? 256 : 1];
  const int grp = threadIdx.x / LANES % GROUPS, c = threadIdx.x % LANES;
  const int64_t bh = (int64_t)blockIdx.x * ROWS + threadIdx.x / (LANES * GROUPS);
  int n = 0;
  if (bh < rows) {
    const int len = a.lens[bh / a.n_heads];
    if ((uint32_t)len <= (uint32_t)a.max_len) n = (int)cdiv(len, (int64_t)decode_unit(len) * a.span);
  }
  if (n <= 1) n = 0;   // written before
  DecNode v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = bh * a.nodes + grp * 4 + i;
    if (grp * 4 + i >= n) continue;
    v[i].o = ((const f32x4*)a.part)[at * LANES + c];
    const float2 st = a.stat[at];
    v[i].m = st.x, v[i].sum = st.y;
  }
  const int mine = n - grp * 4;
  if (mine > 1) v[0] = dec_join(v[0], v[1]);
  if (mine > 3) v[2] = dec_join(v[2], v[3]);
  if (mine > 2) v[0] = dec_join(v[0], v[2]);
#pragma unroll
  for (int k = 1; k < GROUPS; k *= 2) {
    __syncthreads();
    if (mine > 0) lds[threadIdx.x] = v[0];
    __syncthreads();
    if (grp % (2 * k) == 0 && mine > 4 * k) v[0] = dec_join(v[0], lds[threadIdx.x + k * LANES]);
  }
  if (n && grp == 0) dec_store(a, bh, D, c * 4, v[0]);
}

}  // namespace lora

// ---------------------------------------------------------------- launches
namespace lora_host {

using namespace lora;

static int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

lora_status launch_kv_tables(const kv_shape& sh, const int32_t* cached, const int32_t* fresh,
                             int32_t* seq_lens, int32_t* table, int32_t* ring, const int64_t* state,
                             int64_t* state_out, int32_t* cu_new, int64_t n_slots, int32_t* slots,
                             int32_t* positions, int32_t* token_seqs, void* ws, hipStream_t s) {
  TableArgs a{cached, fresh, seq_lens, table, ring, state, state_out, cu_new, slots, positions,
              token_seqs, (int32_t*)ws, n_slots, sh.n_seqs, log2_of(sh.page_size), sh.n_pages,
              sh.max_pages, 1, 1};
  const size_t lds = 3 * sizeof(int32_t) * (size_t)std::max(sh.n_seqs, 1);
  if (n_slots <= 4 * TAB_THREADS && sh.n_seqs <= TAB_THREADS) {
    hipLaunchKernelGGL(kv_tables_kernel, dim3(1), dim3(TAB_THREADS), lds, s, a);
    return launch_check("kv_tables");
  }
  const int64_t items = std::max<int64_t>(n_slots, (int64_t)sh.n_seqs * 64);
  const unsigned grid = (unsigned)std::min<int64_t>(cdiv(items, TAB_THREADS), device_cus());
  const auto meet = [&](const void* p, const void* q, size_t bytes) {
    return (const char*)p < (const char*)q + bytes && (const char*)q < (const char*)p + bytes;
  };
  const bool in_place = meet(seq_lens, cached, 4 * (size_t)sh.n_seqs) || meet(state_out, state, 16);
  a.lengths = !in_place;
  hipLaunchKernelGGL(kv_tables_kernel, dim3(grid), dim3(TAB_THREADS), lds, s, a);
  lora_status st = launch_check("kv_tables");
  if (st != LORA_OK || !in_place) return st;
  a.lengths = 1;
  a.items = 0;
  hipLaunchKernelGGL(kv_tables_kernel, dim3(1), dim3(TAB_THREADS), lds, s, a);
  return launch_check("kv_tables lengths");
}

lora_status launch_kv_write(const kv_shape& sh, int64_t n, const uint16_t* k, int64_t k_stride,
                            const uint16_t* v, int64_t v_stride, const int32_t* slots, void* k_cache,
                            void* v_cache, uint8_t* k_scales, uint8_t* v_scales, void* ws,
                            hipStream_t s) {
  const WriteArgs a{k, v, slots, k_cache, v_cache, k_scales, v_scales, (int32_t*)ws, k_stride,
                    v_stride, n, sh.n_kv_heads, log2_of(sh.page_size), sh.n_pages * sh.page_size};
  const int64_t pieces = n * 2 * sh.n_kv_heads * (sh.head_dim / 8);
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(cdiv(pieces, 256), 1 << 20)), dim3(256), 0, s, a);
  };
  if (sh.head_dim == 128) k_scales ? go(kv_write_kernel<128, true>) : go(kv_write_kernel<128, false>);
  else k_scales ? go(kv_write_kernel<64, true>) : go(kv_write_kernel<64, false>);
  return launch_check("kv_write");
}

// How a batch is cut: units of a block, and nodes that a request of up to max_len keys has
// then.  A block that can take its request whole (up to eight units) does where the requests
// make a block for each CU: no partial results, no second launch.  Longer requests are cut into
// runs of up to four units as long as nine blocks are left for each CU (three are resident).
// Runs of eight end a launch on long blocks however many there are.  Requests of 0.3 to 1
// times a length, 32 heads of 128; runs of 1, 2, 4 and 8 units, us (* what the rule takes):
//   400 x 3000, 4 key heads                373   351  *318   397    (1600 blocks by 12 units)
//   400 x 3000, 4 key heads, 8 bits        212   199  *178   224
//   200 x 3000, 4 key heads, 8 bits        109   102  * 94   122    (2400 blocks of four)
//   170 x 3000, 4 key heads, 8 bits         93  * 87    82   104    (2040)
//   64 x 8000, 8 key heads                 266   254  *252   276
//   32 x 8000, 8 key heads                 127  *124   131   142    (2048)
//   64 x 4000, 8 key heads                 139  *133   144   141    (2048)
//   16 x 31000, 8 key heads, 8 bits      * 150   155   160   150    (2048 of two)
// (over 580 such batches the time is within 2.3 % of the best run's on average).  Whole requests
// against the best cut:
//   32 x 300, 8 key heads                 10.6 / 13.5      31 x 300 (248 blocks)   10.3 / 13.0
//   32 x 1000                             20.6 / 20.4      250 x 1000               123 /  146
//   32 x 2000, 8 bits (256 blocks)        30.2 / 25.0      64 x 2000, 8 bits       43.9 / 48.7
//   100 x 1500                            89.8 / 88.5      128 x 2000, 2 key heads 44.5 / 45.8
struct DecodePlan {
  int span, nodes;
};
static DecodePlan decode_plan(int64_t columns, int64_t max_len) {   // columns: requests by key heads by 16 query heads
  const int64_t units = std::min<int64_t>(DEC_MAX_UNITS, std::max<int64_t>(1, cdiv(max_len, DEC_UNIT)));
  int span = 1;
  const int64_t cus = device_cus();
  const bool one = units <= DEC_MAX_SPAN && columns >= cus;
  while (one ? span < units : span < DEC_CUT_SPAN && columns * cdiv(units, 2 * span) >= DEC_CU_BLOCKS * cus) span *= 2;
  return {span, (int)cdiv(units, span)};
}
static int64_t decode_columns(const kv_shape& sh, int32_t n_heads) {
  return (int64_t)sh.n_kv_heads * cdiv(n_heads / sh.n_kv_heads, 16);
}
static size_t decode_part_bytes(size_t parts, const kv_shape& sh) {
  return parts ? 256 + align_up(parts * sizeof(float2), 256) + parts * sh.head_dim * sizeof(float) : 256;
}

size_t decode_ws_bytes(const kv_shape& sh, int32_t n_heads, int64_t max_len) {
  const DecodePlan p = decode_plan(sh.n_seqs * decode_columns(sh, n_heads), max_len);
  return decode_part_bytes(p.nodes == 1 ? 0 : (size_t)sh.n_seqs * n_heads * p.nodes, sh);
}

// The most of them over smaller batches and bounds, which may be cut into more parts.  For
// requests of u units the parts grow with the batch until the cut gets coarser: the largest
// batch before each coarser cut, and the whole one, are all there is to look at.
size_t decode_ws_bound(const kv_shape& sh, int32_t n_heads, int64_t max_len) {
  size_t most = 0;
  const int64_t units = std::min<int64_t>(DEC_MAX_UNITS, cdiv(max_len, DEC_UNIT));
  const int64_t columns = decode_columns(sh, n_heads), cus = device_cus();
  for (int64_t u = 2; u <= units; ++u) {
    const auto look = [&](int64_t most_columns) {   // the largest batch with fewer columns than that
      const int64_t n = std::min<int64_t>(sh.n_seqs, (most_columns - 1) / columns);
      const DecodePlan p = decode_plan(n * columns, u * DEC_UNIT);
      if (p.nodes > 1) most = std::max(most, (size_t)n * n_heads * p.nodes);
    };
    look(sh.n_seqs * columns + 1);
    if (u <= DEC_MAX_SPAN) look(cus);
    for (int span = 2; span <= DEC_CUT_SPAN; span *= 2) look(cdiv(DEC_CU_BLOCKS * cus, cdiv(u, span)));
  }
  return decode_part_bytes(most, sh);
}

lora_status launch_decode(const kv_shape& sh, int32_t n_heads, const uint16_t* q, int64_t q_stride,
                          const void* k_cache, const void* v_cache, const uint8_t* k_scales,
                          const uint8_t* v_scales, const int32_t* table, const int32_t* seq_lens,
                          int64_t max_len, float scale, uint16_t* o, float* lse, void* ws,
                          hipStream_t s) {
  const DecodePlan p = decode_plan(sh.n_seqs * decode_columns(sh, n_heads), max_len);
  DecodeArgs a{};
  a.q = q, a.kc = k_cache, a.vc = v_cache, a.ks = k_scales, a.vs = v_scales;
  a.table = table, a.lens = seq_lens, a.o = o, a.lse = lse, a.status = (int32_t*)ws;
  a.q_stride = q_stride, a.n_heads = n_heads, a.n_kv = sh.n_kv_heads, a.group = n_heads / sh.n_kv_heads;
  a.page_shift = log2_of(sh.page_size), a.n_pages = sh.n_pages, a.max_pages = sh.max_pages;
  a.max_len = (int32_t)max_len, a.nodes = p.nodes, a.span = p.span, a.col_groups = (int)cdiv(a.group, 16);
  a.scale_log2 = scale == 0.f ? 1.f : std::fabs(scale) * KV_LOG2E;
  a.q_turn = scale < 0.f ? 0x80008000u : 0u, a.q_keep = scale == 0.f ? 0u : ~0u;
  const int64_t rows = (int64_t)sh.n_seqs * n_heads;
  a.stat = (float2*)((char*)ws + 256);
  a.part = (float*)((char*)ws + 256 + align_up(rows * a.nodes * (int64_t)sizeof(float2), 256));
  const int64_t blocks = (int64_t)sh.n_seqs * a.nodes * a.n_kv * a.col_groups;
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(64 * DEC_WAVES), 0, s, a);
  };
  if (sh.head_dim == 64) k_scales ? go(decode_kernel<64, true, 1>) : go(decode_kernel<64, false, 1>);
  else if (a.group <= 8) k_scales ? go(decode_kernel<128, true, 1>) : go(decode_kernel<128, false, 1>);
  else k_scales ? go(decode_kernel<128, true, 2>) : go(decode_kernel<128, false, 2>);
  lora_status st = launch_check("decode");
  if (st != LORA_OK || a.nodes == 1) return st;
  const auto join = [&](auto kernel, int per_block) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)cdiv(rows, per_block)), dim3(256), 0, s, a, rows);
  };
  if (sh.head_dim == 128) a.nodes <= 4 ? join(decode_join_kernel<128, 1>, 8) : join(decode_join_kernel<128, 8>, 1);
  else a.nodes <= 4 ? join(decode_join_kernel<64, 1>, 16) : join(decode_join_kernel<64, 8>, 2);
  return launch_check("decode_join");
}

}  // namespace lora_host
