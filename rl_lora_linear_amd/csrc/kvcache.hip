// The paged key-value cache on gfx950: block tables and slot maps from request lengths,
// new rows into the pages, and the attention of one new token of each request.
#include "attn.hpp"
#include "q8.hpp"

namespace lora {

constexpr float KV_LOG2E = 1.4426950408889634f, KV_LN2 = 0.6931471805599453f;

// ---------------------------------------------------------------- block tables and slots
// All of it follows from running sums over the requests of three counts: new rows, pages
// needed, pages put back.  Requests number at most some thousands, so every block sums
// them itself (a few per thread) and keeps the sums in LDS; then new rows, new table
// entries and returned pages are independent items, each found by a binary search.  One
// launch does all where one block suffices.  Else a grid does the items, and a second
// launch of one block writes what a caller may have passed in place (seq_lens over
// cached_lens, the state over itself), which no block of the first may see changed.
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
  int32_t items, lengths;   // which halves this launch does
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
        pos = r.cached + (int32_t)t - rows_at[seq];
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
  if (!a.lengths) return;
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
// A block takes one split of a request's length for one key head (and up to 16 of its
// query heads: the columns of a 16x16x32 matrix instruction, so a group of any size costs
// one pass over the cache).  Its four waves take the split's tiles of 32 keys in turn,
// each with its own running maximum, sum and output, and join at the end; the splits of
// a request are joined by a second kernel.
//   S^T = K Q^T: lane (l, g) = (lane & 15, lane >> 4) holds key l's chunk as operand and
//   ends with column (query head) l, keys 4g .. 4g+3 of the 16;
//   O^T += V^T P^T: those are the operand of P as they lie, where the instruction's key
//   8g + j means key 4g + j of the tile's first 16 keys (j < 4) or second (j >= 4).  V's
//   operand for the same order comes from LDS by transposing reads.
// So nothing but the maximum and the sum crosses lanes, and each lane rescales the output
// of its own query head.
constexpr int DEC_WAVES = 4, DEC_TILE = 32, DEC_MIN_SPLIT = 128, DEC_MAX_SPLITS = 32;

// The split's length for a request of `len` keys: a power of two, so that a request has
// at most 32 splits; by its own length alone.
__host__ __device__ __forceinline__ int decode_split(int len) {
  int s = DEC_MIN_SPLIT;
  while ((int64_t)s * DEC_MAX_SPLITS < len) s *= 2;
  return s;
}

struct DecodeArgs {
  const uint16_t* q;
  const void *kc, *vc;
  const uint8_t *ks, *vs;
  const int32_t *table, *lens;
  uint16_t* o;
  float* lse;
  float* part;       // [n][heads][splits][D] outputs over their sums
  float2* stat;      // [n][heads][splits] (maximum in powers of two, sum)
  int32_t* status;
  int64_t q_stride;
  int32_t n_heads, n_kv, group, page_shift, n_pages, max_pages, max_len, splits, col_groups;
  float scale_log2;
};

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

template <int D, bool X8>
__global__ __launch_bounds__(64 * DEC_WAVES) void decode_kernel(DecodeArgs a) {
  constexpr int NK = D / 32;            // steps of 32 columns
  constexpr int ND = D / 16;            // output tiles of 16 columns
  constexpr int V_BYTES = DEC_TILE * D * 2;
  __shared__ uint4 lds[DEC_WAVES * V_BYTES / 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane & 15, g = lane >> 4;
  const int heads_at = blockIdx.x % (a.n_kv * a.col_groups);
  const int rest = blockIdx.x / (a.n_kv * a.col_groups);
  const int split = rest % a.splits, b = rest / a.splits;
  const int kvh = heads_at / a.col_groups, cols0 = heads_at % a.col_groups * 16;
  const int cols = min(16, a.group - cols0);
  int len = a.lens[b];
  if ((uint32_t)len > (uint32_t)a.max_len) {
    if (split == 0 && heads_at == 0 && threadIdx.x == 0) set_flag(a.status, LORA_FLAG_BAD_LENGTH);
    len = 0;
  }
  const int per = decode_split(len);
  const int k0 = split * per, k1 = min(k0 + per, len);
  if (k0 >= len && split > 0) return;   // split 0 also writes a request without keys
  const bool only = len <= per;

  // Q as operand: lane (l, g) holds 8 columns of query head l for each step.  In 8 bits
  // a lane loads 16 codes at once, the columns of two steps.
  const auto col_of = [&](int kk) { return X8 ? (kk >> 1) * 64 + g * 16 + (kk & 1) * 8 : kk * 32 + g * 8; };
  bf16x8 qf[NK];
  const int head0 = kvh * a.group + cols0;
#pragma unroll
  for (int kk = 0; kk < NK; ++kk)
    qf[kk] = as_bf16x8(l < cols ? *(const uint4*)(a.q + b * a.q_stride + (int64_t)(head0 + l) * D + col_of(kk))
                                : make_uint4(0, 0, 0, 0));

  f32x4 acc[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, sum = 0.f;
  char* const vl = (char*)lds + wave * V_BYTES;
  const int32_t* const table = a.table + (int64_t)b * a.max_pages;
  const int page_mask = (1 << a.page_shift) - 1;
  bool bad = false;

  // a row of the cache: its index in rows, or -1 where there is none
  const auto row_of = [&](int key) -> int64_t {
    if (key >= k1) return -1;
    const int32_t page = table[key >> a.page_shift];
    if ((uint32_t)page >= (uint32_t)a.n_pages) {
      bad = true;
      return -1;
    }
    return (((int64_t)page * a.n_kv + kvh) << a.page_shift) + (key & page_mask);
  };

  for (int t0 = k0 + wave * DEC_TILE; t0 < k1; t0 += DEC_WAVES * DEC_TILE) {
    // ---- scores of 32 keys
    f32x4 s[2];
    bool live[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t row = row_of(t0 + t * 16 + l);
      live[t] = row >= 0;
      s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (X8) {
        const uint8_t* kr = (const uint8_t*)a.kc + row * D;
#pragma unroll
        for (int kk = 0; kk < NK; kk += 2) {
          const uint4 c = live[t] ? *(const uint4*)(kr + col_of(kk)) : make_uint4(0, 0, 0, 0);
          const float sc = live[t] ? e8m0(a.ks[row * (D / 32) + col_of(kk) / 32]) : 1.f;
          s[t] = mfma16(kv_widen(c.x, c.y, sc), qf[kk], s[t]);
          s[t] = mfma16(kv_widen(c.z, c.w, sc), qf[kk + 1], s[t]);
        }
      } else {
        const uint16_t* kr = (const uint16_t*)a.kc + row * D;
#pragma unroll
        for (int kk = 0; kk < NK; ++kk)
          s[t] = mfma16(as_bf16x8(live[t] ? *(const uint4*)(kr + col_of(kk)) : make_uint4(0, 0, 0, 0)), qf[kk], s[t]);
      }
    }
    // ---- V rows into LDS: rows that do not exist as zeros, whatever lies there
    constexpr int LPR = X8 ? D / 16 : D / 8;    // lanes of a row, 16 bytes each
#pragma unroll
    for (int i = 0; i < DEC_TILE * LPR / 64; ++i) {
      const int r = (i * 64 + lane) / LPR, c = (i * 64 + lane) % LPR;
      const int64_t row = row_of(t0 + r);
      const uint4 x = row >= 0 ? *(const uint4*)((const char*)a.vc + row * D * (X8 ? 1 : 2) + c * 16) : make_uint4(0, 0, 0, 0);
      if (X8) {
        const float sc = row >= 0 ? e8m0(a.vs[row * (D / 32) + c / 2]) : 1.f;
        *(bf16x8*)(vl + dec_v_at<D>(r, 2 * c)) = kv_widen(x.x, x.y, sc);
        *(bf16x8*)(vl + dec_v_at<D>(r, 2 * c + 1)) = kv_widen(x.z, x.w, sc);
      } else {
        *(uint4*)(vl + dec_v_at<D>(r, c)) = x;
      }
    }
    // ---- softmax: which of the lane's 8 keys exist is known to the lanes that loaded them
    const uint64_t on[2] = {__ballot(live[0]), __ballot(live[1])};
    float top = -INFINITY;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[t][r] = on[t] >> (4 * g + r) & 1 ? s[t][r] * a.scale_log2 : -INFINITY;
        top = fmaxf(top, s[t][r]);
      }
    top = fmaxf(top, __shfl_xor(top, 16, kWave));
    top = fmaxf(top, __shfl_xor(top, 32, kWave));
    const float m_new = fmaxf(m, top), ref = m_new == -INFINITY ? 0.f : m_new;
    const float keep = __builtin_amdgcn_exp2f(m - ref);
    m = m_new;
    sum *= keep;
    uint32_t p[4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float e[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) sum += e[r] = __builtin_amdgcn_exp2f(s[t][r] - ref);
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
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) acc[i][r4] *= keep;
      acc[i] = mfma16(as_bf16x8(make_uint4(v0.x, v0.y, v1.x, v1.y)), pf, acc[i]);
    }
    __builtin_amdgcn_wave_barrier();
  }
  if (bad) set_flag(a.status, LORA_FLAG_BAD_PAGE);

  // ---- the waves' results, joined in wave order (the V tiles are done with)
  sum += __shfl_xor(sum, 16, kWave);
  sum += __shfl_xor(sum, 32, kWave);
  __shared__ float2 ms[DEC_WAVES][16];
  if (g == 0) ms[wave][l] = make_float2(m, sum);
  __syncthreads();
  float big = -INFINITY;
#pragma unroll
  for (int w = 0; w < DEC_WAVES; ++w) big = fmaxf(big, ms[w][l].x);
  const float ref = big == -INFINITY ? 0.f : big;
  float all = 0.f;
#pragma unroll
  for (int w = 0; w < DEC_WAVES; ++w) all += ms[w][l].y * __builtin_amdgcn_exp2f(ms[w][l].x - ref);
  const float mul = __builtin_amdgcn_exp2f(m - ref) * (all > 0.f || all != all ? 1.f / all : 0.f);
  float* const of = (float*)lds + wave * (16 * D);   // [16 heads][D], a wave's V tile: 32 D bf16
#pragma unroll
  for (int i = 0; i < ND; ++i)
    *(f32x4*)(of + l * D + ((i * 16 + 4 * g) ^ ((l & 7) << 2))) = acc[i] * mul;
  __syncthreads();
  const int64_t bh = (int64_t)b * a.n_heads + head0;
  for (int i = threadIdx.x; i < cols * (D / 4); i += 64 * DEC_WAVES) {
    const int h = i / (D / 4), c = i % (D / 4) * 4;
    const float* src = (const float*)lds + h * D + (c ^ ((h & 7) << 2));
    f32x4 v = *(const f32x4*)src;
#pragma unroll
    for (int w = 1; w < DEC_WAVES; ++w) v += *(const f32x4*)(src + w * 16 * D);
    if (only) *(uint2*)(a.o + (bh + h) * D + c) = make_uint2(pack2bf(v[0], v[1]), pack2bf(v[2], v[3]));
    else *(f32x4*)(a.part + ((bh + h) * a.splits + split) * D + c) = v;
  }
  if (threadIdx.x < cols) {   // (lane l of wave 0: its own head's sums)
    if (!only) a.stat[(bh + l) * a.splits + split] = make_float2(big, all);
    else if (a.lse) a.lse[bh + l] = all == 0.f ? -INFINITY : (big + __log2f(all)) * KV_LN2;
  }
}

// The splits of a request and head, joined in order: a wave each.
template <int D>
__global__ __launch_bounds__(256) void decode_join_kernel(DecodeArgs a, int64_t rows) {
  const int64_t bh = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (bh >= rows) return;
  const int len = a.lens[bh / a.n_heads];
  if ((uint32_t)len > (uint32_t)a.max_len) return;
  const int per = decode_split(len), n = (len + per - 1) / per;
  if (n <= 1) return;
  const float2 st = lane < n ? a.stat[bh * a.splits + lane] : make_float2(-INFINITY, 0.f);
  float big = st.x;
  for (int o = 32; o; o >>= 1) big = fmaxf(big, __shfl_xor(big, o, kWave));
  const float ref = big == -INFINITY ? 0.f : big;
  const float w = st.y * __builtin_amdgcn_exp2f(st.x - ref);
  float all = w;
  for (int o = 32; o; o >>= 1) all += __shfl_xor(all, o, kWave);
  const float mul = w * (all > 0.f || all != all ? 1.f / all : 0.f);
  constexpr int C = D / 64;
  float v[C] = {};
  const float* part = a.part + bh * a.splits * D + lane * C;
#pragma unroll 8
  for (int i = 0; i < n; ++i) {
    const float f = __shfl(mul, i, kWave);
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] += part[i * D + c] * f;
  }
  if (C == 2) *(uint32_t*)(a.o + bh * D + lane * 2) = pack2bf(v[0], v[C - 1]);
  else a.o[bh * D + lane] = f2bf(v[0]);
  if (a.lse && lane == 0) a.lse[bh] = all == 0.f ? -INFINITY : (big + __log2f(all)) * KV_LN2;
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
  a.lengths = 0;
  hipLaunchKernelGGL(kv_tables_kernel, dim3(grid), dim3(TAB_THREADS), lds, s, a);
  lora_status st = launch_check("kv_tables");
  if (st != LORA_OK) return st;
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

// Splits that a request of up to max_len keys may have.
static int decode_splits(int64_t max_len) {
  return (int)std::min<int64_t>(DEC_MAX_SPLITS, std::max<int64_t>(1, cdiv(max_len, DEC_MIN_SPLIT)));
}

size_t decode_ws_bytes(const kv_shape& sh, int32_t n_heads, int64_t max_len) {
  const int splits = decode_splits(max_len);
  if (splits == 1) return 256;
  const size_t parts = (size_t)sh.n_seqs * n_heads * splits;
  return 256 + align_up(parts * sizeof(float2), 256) + parts * sh.head_dim * sizeof(float);
}

lora_status launch_decode(const kv_shape& sh, int32_t n_heads, const uint16_t* q, int64_t q_stride,
                          const void* k_cache, const void* v_cache, const uint8_t* k_scales,
                          const uint8_t* v_scales, const int32_t* table, const int32_t* seq_lens,
                          int64_t max_len, float scale, uint16_t* o, float* lse, void* ws,
                          hipStream_t s) {
  DecodeArgs a{};
  a.q = q, a.kc = k_cache, a.vc = v_cache, a.ks = k_scales, a.vs = v_scales;
  a.table = table, a.lens = seq_lens, a.o = o, a.lse = lse, a.status = (int32_t*)ws;
  a.q_stride = q_stride, a.n_heads = n_heads, a.n_kv = sh.n_kv_heads, a.group = n_heads / sh.n_kv_heads;
  a.page_shift = log2_of(sh.page_size), a.n_pages = sh.n_pages, a.max_pages = sh.max_pages;
  a.max_len = (int32_t)max_len, a.splits = decode_splits(max_len), a.col_groups = (int)cdiv(a.group, 16);
  a.scale_log2 = scale * KV_LOG2E;
  const int64_t rows = (int64_t)sh.n_seqs * n_heads;
  a.stat = (float2*)((char*)ws + 256);
  a.part = (float*)((char*)ws + 256 + align_up(rows * a.splits * (int64_t)sizeof(float2), 256));
  const int64_t blocks = (int64_t)sh.n_seqs * a.splits * a.n_kv * a.col_groups;
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(64 * DEC_WAVES), 0, s, a);
  };
  if (sh.head_dim == 128) k_scales ? go(decode_kernel<128, true>) : go(decode_kernel<128, false>);
  else k_scales ? go(decode_kernel<64, true>) : go(decode_kernel<64, false>);
  lora_status st = launch_check("decode");
  if (st != LORA_OK || a.splits == 1) return st;
  const dim3 grid((unsigned)cdiv(rows, 4));
  if (sh.head_dim == 128) hipLaunchKernelGGL(decode_join_kernel<128>, grid, dim3(256), 0, s, a, rows);
  else hipLaunchKernelGGL(decode_join_kernel<64>, grid, dim3(256), 0, s, a, rows);
  return launch_check("decode_join");
}

}  // namespace lora_host
