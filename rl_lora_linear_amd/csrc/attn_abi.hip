// C-ABI entry points of the attention and key-value cache calls: host-side validation,
// then their launches on the caller's stream.
#include <cmath>

#include "attn.hpp"

using namespace lora_host;
using lora::cdiv;

#define TRY(expr)                  \
  do {                             \
    lora_status _st = (expr);      \
    if (_st != LORA_OK) return _st; \
  } while (0)

namespace {

hipStream_t S(void* p) { return (hipStream_t)p; }
bool aligned(const void* p, unsigned to) { return ((uintptr_t)p & (to - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }

lora_status unsupported(const char* what, const char* rule) {
  set_error("%s: %s", what, rule);
  return LORA_E_UNSUPPORTED;
}

// The bytes of `rows` rows of `cols` bf16 elements at a stride.
struct Span {
  const char *from, *to;
};
Span span(const void* p, int64_t rows, int64_t stride, int64_t cols) {
  const char* c = (const char*)p;
  return {c, rows > 0 ? c + ((rows - 1) * stride + cols) * 2 : c};
}
bool meet(Span a, Span b) {
  return a.from && b.from && a.from < a.to && b.from < b.to && a.from < b.to && b.from < a.to;
}
Span bytes(const void* p, int64_t n) { return {(const char*)p, (const char*)p + n}; }
// The first of `out` that lies on another buffer, of `in` or of the other outputs; -1: none.
template <size_t N, size_t M>
int clash(const Span (&out)[N], const Span (&in)[M]) {
  for (size_t i = 0; i < N; ++i) {
    for (const Span& s : in)
      if (meet(out[i], s)) return (int)i;
    for (size_t j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return (int)i;
  }
  return -1;
}
// Whether rows of two strided matrices share bytes.  Slices of one buffer (the same stride)
// lie between one another: they meet where their columns do.
bool rows_meet(const void* a, int64_t a_rows, int64_t a_stride, int64_t a_cols, const void* b,
               int64_t b_rows, int64_t b_stride, int64_t b_cols) {
  if (!meet(span(a, a_rows, a_stride, a_cols), span(b, b_rows, b_stride, b_cols))) return false;
  if (a_stride != b_stride) return true;
  const int64_t row = a_stride * 2;
  int64_t gap = ((const char*)b - (const char*)a) % row;
  if (gap < 0) gap += row;
  return gap < a_cols * 2 || gap + b_cols * 2 > row;
}

// (the kernels multiply it by log2 e)
bool scale_ok(float s) { return std::fabs(s) < 0x1p127f; }

lora_status check_attn(const attn_shape* p, const char* what) {
  LORA_ARG_CHECK(p != nullptr, "%s: shape is NULL", what);
  const attn_shape& s = *p;
  LORA_ARG_CHECK(s.n_q >= 0 && s.n_q < (1 << 30) && s.n_k >= 0 && s.n_k < (1 << 30),
                 "%s: n_q %lld or n_k %lld outside [0, 2^30)", what, (long long)s.n_q, (long long)s.n_k);
  LORA_ARG_CHECK(s.n_seqs >= 0 && s.n_seqs <= 65536, "%s: n_seqs %d outside [0, 65536]", what, s.n_seqs);
  LORA_ARG_CHECK(s.n_kv_heads >= 1 && s.n_heads >= 1 && s.n_heads <= 1024 && s.n_heads % s.n_kv_heads == 0,
                 "%s: n_heads %d must be a multiple of n_kv_heads %d, at most 1024", what, s.n_heads, s.n_kv_heads);
  LORA_ARG_CHECK(s.causal == 0 || s.causal == 1, "%s: causal must be 0 or 1", what);
  LORA_ARG_CHECK(scale_ok(s.scale), "%s: scale must be below 2^127 in magnitude", what);
  if (s.head_dim != 64 && s.head_dim != 128) return unsupported(what, "head_dim must be 64 or 128");
  const int64_t q = (int64_t)s.n_heads * s.head_dim, k = (int64_t)s.n_kv_heads * s.head_dim;
  for (int64_t st : {s.q_stride, s.k_stride, s.v_stride, s.o_stride})
    LORA_ARG_CHECK(st % 8 == 0 && st < (1 << 24), "%s: stride %lld must be a multiple of 8 below 2^24",
                   what, (long long)st);
  LORA_ARG_CHECK(s.q_stride >= q && s.o_stride >= q && s.k_stride >= k && s.v_stride >= k,
                 "%s: a stride is shorter than its row", what);
  // a launch takes fewer than 2^32 threads, and a block has 512
  const auto fits = [&](int64_t rows, int64_t heads) { return (rows / 128 + s.n_seqs + 1) * heads < (1 << 23); };
  if (!fits(s.n_q, s.n_heads) || !fits(s.n_k, s.n_kv_heads))
    return unsupported(what, "too many rows times heads for one launch");
  return LORA_OK;
}

lora_status check_ws(const void* ws, size_t have, size_t need, const char* what) {
  if (!ws || have < need) {
    set_error("%s: workspace %zu bytes < %zu needed", what, have, need);
    return LORA_E_WORKSPACE;
  }
  LORA_ARG_CHECK(aligned16(ws), "%s: the workspace must be 16-byte aligned", what);
  return LORA_OK;
}

size_t attn_ws(const attn_shape& s) { return 256 + (size_t)s.n_heads * s.n_q * 2 * sizeof(float); }

lora_status check_kv(const kv_shape* p, const char* what) {
  LORA_ARG_CHECK(p != nullptr, "%s: shape is NULL", what);
  const kv_shape& s = *p;
  LORA_ARG_CHECK(s.n_seqs >= 0 && s.n_seqs <= 4096, "%s: n_seqs %d outside [0, 4096]", what, s.n_seqs);
  LORA_ARG_CHECK(s.n_kv_heads >= 1 && s.n_kv_heads <= 1024, "%s: n_kv_heads %d outside [1, 1024]", what, s.n_kv_heads);
  LORA_ARG_CHECK(s.n_pages >= 1 && s.max_pages >= 1, "%s: n_pages and max_pages must be positive", what);
  if (s.head_dim != 64 && s.head_dim != 128) return unsupported(what, "head_dim must be 64 or 128");
  if (s.page_size < 16 || s.page_size > 256 || (s.page_size & (s.page_size - 1)))
    return unsupported(what, "page_size must be 16, 32, 64, 128 or 256");
  if ((int64_t)s.n_pages * s.page_size >= ((int64_t)1 << 31) || (int64_t)s.max_pages * s.page_size >= ((int64_t)1 << 31))
    return unsupported(what, "n_pages and max_pages times page_size must be below 2^31");
  return LORA_OK;
}

int64_t cache_rows(const kv_shape& s) { return (int64_t)s.n_pages * s.page_size * s.n_kv_heads; }

lora_status check_caches(const kv_shape& s, const void* kc, const void* vc, const uint8_t* ks, const uint8_t* vs,
                         const char* what) {
  LORA_ARG_CHECK(kc && vc && aligned16(kc) && aligned16(vc), "%s: k_cache or v_cache NULL or not 16-byte aligned", what);
  LORA_ARG_CHECK((ks == nullptr) == (vs == nullptr), "%s: k_scales and v_scales go together", what);
  LORA_ARG_CHECK(aligned(ks, 4) && aligned(vs, 4), "%s: scales must be 4-byte aligned", what);
  return LORA_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ packed prompts
size_t attention_workspace_bytes(const attn_shape* shape) {
  if (check_attn(shape, "attention") != LORA_OK) return 0;
  return attn_ws(*shape);
}

lora_status attention_forward(const attn_shape* shape, const uint16_t* q, const uint16_t* k,
                              const uint16_t* v, const int32_t* cu_q, const int32_t* cu_k,
                              uint16_t* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_attn(shape, "attention_forward"));
  const attn_shape& s = *shape;
  LORA_ARG_CHECK(s.n_q == 0 || (q && o && lse), "attention_forward: q, o and lse must be non-NULL");
  LORA_ARG_CHECK(s.n_k == 0 || (k && v), "attention_forward: k and v must be non-NULL");
  LORA_ARG_CHECK(s.n_seqs == 0 || (cu_q && cu_k), "attention_forward: cu_q and cu_k must be non-NULL");
  LORA_ARG_CHECK(aligned16(q) && aligned16(k) && aligned16(v) && aligned16(o),
                 "attention_forward: q, k, v and o must be 16-byte aligned");
  LORA_ARG_CHECK(aligned(lse, 4) && aligned(cu_q, 4) && aligned(cu_k, 4), "attention_forward: lse, cu_q and cu_k must be 4-byte aligned");
  TRY(check_ws(ws, ws_bytes, attn_ws(s), "attention_forward"));
  const int64_t qc = (int64_t)s.n_heads * s.head_dim, kc = (int64_t)s.n_kv_heads * s.head_dim;
  LORA_ARG_CHECK(!rows_meet(o, s.n_q, s.o_stride, qc, q, s.n_q, s.q_stride, qc) &&
                     !rows_meet(o, s.n_q, s.o_stride, qc, k, s.n_k, s.k_stride, kc) &&
                     !rows_meet(o, s.n_q, s.o_stride, qc, v, s.n_k, s.v_stride, kc),
                 "attention_forward: o overlaps q, k or v");
  const int64_t cu = 4 * ((int64_t)s.n_seqs + 1);
  const Span out[] = {bytes(lse, 4 * (int64_t)s.n_heads * s.n_q), bytes(ws, (int64_t)attn_ws(s))};
  const Span in[] = {span(q, s.n_q, s.q_stride, qc), span(k, s.n_k, s.k_stride, kc), span(v, s.n_k, s.v_stride, kc),
                     span(o, s.n_q, s.o_stride, qc), bytes(cu_q, cu), bytes(cu_k, cu)};
  LORA_ARG_CHECK(clash(out, in) < 0, "attention_forward: lse or the workspace overlaps another operand");
  LORA_ARG_CHECK(!meet(in[3], in[4]) && !meet(in[3], in[5]), "attention_forward: o overlaps cu_q or cu_k");
  if (s.n_q == 0 || s.n_seqs == 0) return LORA_OK;
  return launch_attention_fwd(s, q, k, v, cu_q, cu_k, o, lse, ws, S(stream));
}

lora_status attention_backward(const attn_shape* shape, const uint16_t* dout, const uint16_t* q,
                               const uint16_t* k, const uint16_t* v, const uint16_t* o,
                               const float* lse, const int32_t* cu_q, const int32_t* cu_k,
                               uint16_t* dq, uint16_t* dk, uint16_t* dv, void* ws,
                               size_t ws_bytes, void* stream) {
  TRY(check_attn(shape, "attention_backward"));
  const attn_shape& s = *shape;
  LORA_ARG_CHECK(s.n_q == 0 || (dout && q && o && lse && dq), "attention_backward: dout, q, o, lse and dq must be non-NULL");
  LORA_ARG_CHECK(s.n_k == 0 || (k && v && dk && dv), "attention_backward: k, v, dk and dv must be non-NULL");
  LORA_ARG_CHECK(s.n_seqs == 0 || (cu_q && cu_k), "attention_backward: cu_q and cu_k must be non-NULL");
  for (const void* p : {(const void*)dout, (const void*)q, (const void*)k, (const void*)v, (const void*)o,
                        (const void*)dq, (const void*)dk, (const void*)dv})
    LORA_ARG_CHECK(aligned16(p), "attention_backward: bf16 operands must be 16-byte aligned");
  LORA_ARG_CHECK(aligned(lse, 4) && aligned(cu_q, 4) && aligned(cu_k, 4), "attention_backward: lse, cu_q and cu_k must be 4-byte aligned");
  TRY(check_ws(ws, ws_bytes, attn_ws(s), "attention_backward"));
  const int64_t qc = (int64_t)s.n_heads * s.head_dim, kc = (int64_t)s.n_kv_heads * s.head_dim;
  struct Rows {
    const void* p;
    int64_t rows, stride, cols;
  };
  const Rows out[3] = {{dq, s.n_q, s.q_stride, qc}, {dk, s.n_k, s.k_stride, kc}, {dv, s.n_k, s.v_stride, kc}};
  const Rows in[5] = {{dout, s.n_q, s.o_stride, qc}, {o, s.n_q, s.o_stride, qc}, {q, s.n_q, s.q_stride, qc},
                      {k, s.n_k, s.k_stride, kc}, {v, s.n_k, s.v_stride, kc}};
  const auto meets = [](const Rows& a, const Rows& b) {
    return rows_meet(a.p, a.rows, a.stride, a.cols, b.p, b.rows, b.stride, b.cols);
  };
  for (int i = 0; i < 3; ++i) {
    for (const Rows& r : in) LORA_ARG_CHECK(!meets(out[i], r), "attention_backward: dq, dk or dv overlaps an input");
    for (int j = 0; j < i; ++j) LORA_ARG_CHECK(!meets(out[i], out[j]), "attention_backward: dq, dk and dv overlap");
  }
  const int64_t cu = 4 * ((int64_t)s.n_seqs + 1);
  const Span work[] = {bytes(ws, (int64_t)attn_ws(s))};
  Span rest[11];
  int n = 0;
  for (const Rows& r : in) rest[n++] = span(r.p, r.rows, r.stride, r.cols);
  for (const Rows& r : out) rest[n++] = span(r.p, r.rows, r.stride, r.cols);
  rest[n++] = bytes(lse, 4 * (int64_t)s.n_heads * s.n_q);
  rest[n++] = bytes(cu_q, cu);
  rest[n++] = bytes(cu_k, cu);
  LORA_ARG_CHECK(clash(work, rest) < 0, "attention_backward: the workspace overlaps another operand");
  for (int i = 0; i < 3; ++i)
    LORA_ARG_CHECK(!meet(rest[5 + i], rest[8]) && !meet(rest[5 + i], rest[9]) && !meet(rest[5 + i], rest[10]),
                   "attention_backward: dq, dk or dv overlaps lse, cu_q or cu_k");
  if (s.n_seqs == 0 || (s.n_q == 0 && s.n_k == 0)) return LORA_OK;
  return launch_attention_bwd(s, dout, q, k, v, o, lse, cu_q, cu_k, dq, dk, dv, ws, S(stream));
}

// ------------------------------------------------------------------ key-value cache
size_t kv_tables_workspace_bytes(const kv_shape* shape) {
  return check_kv(shape, "kv_tables") == LORA_OK ? 256 : 0;
}

lora_status kv_tables(const kv_shape* shape, const int32_t* cached_lens, const int32_t* new_lens,
                      int32_t* seq_lens, int32_t* block_table, int32_t* ring,
                      const int64_t* ring_state, int64_t* ring_state_out, int32_t* cu_new,
                      int64_t n_slots, int32_t* slots, int32_t* positions, int32_t* token_seqs,
                      void* ws, size_t ws_bytes, void* stream) {
  TRY(check_kv(shape, "kv_tables"));
  const kv_shape& s = *shape;
  LORA_ARG_CHECK(n_slots >= 0 && n_slots < (1 << 30), "kv_tables: n_slots %lld outside [0, 2^30)", (long long)n_slots);
  LORA_ARG_CHECK(s.n_seqs == 0 || (cached_lens && new_lens && seq_lens && block_table),
                 "kv_tables: cached_lens, new_lens, seq_lens and block_table must be non-NULL");
  LORA_ARG_CHECK(ring && ring_state && ring_state_out, "kv_tables: ring, ring_state and ring_state_out must be non-NULL");
  LORA_ARG_CHECK(n_slots == 0 || slots, "kv_tables: slots must be non-NULL");
  LORA_ARG_CHECK(aligned(ring_state, 8) && aligned(ring_state_out, 8), "kv_tables: the ring's state must be 8-byte aligned");
  for (const void* p : {(const void*)cached_lens, (const void*)new_lens, (const void*)seq_lens, (const void*)block_table,
                        (const void*)ring, (const void*)cu_new, (const void*)slots, (const void*)positions, (const void*)token_seqs})
    LORA_ARG_CHECK(aligned(p, 4), "kv_tables: int32 operands must be 4-byte aligned");
  TRY(check_ws(ws, ws_bytes, 256, "kv_tables"));
  const int64_t n4 = 4 * (int64_t)s.n_seqs, s4 = 4 * n_slots;
  // in place, or apart: seq_lens and cached_lens, the two states
  const Span lens = bytes(seq_lens != cached_lens ? cached_lens : nullptr, n4),
             state = bytes(ring_state_out != ring_state ? ring_state : nullptr, 16);
  const Span out[] = {bytes(seq_lens, n4), bytes(block_table, n4 * s.max_pages), bytes(ring, 4 * (int64_t)s.n_pages),
                      bytes(ring_state_out, 16), bytes(cu_new, n4 + 4), bytes(slots, s4), bytes(positions, s4),
                      bytes(token_seqs, s4), bytes(ws, 256)};
  const Span in[] = {lens, bytes(new_lens, n4), state};
  LORA_ARG_CHECK(clash(out, in) < 0, "kv_tables: an output overlaps another operand");
  return launch_kv_tables(s, cached_lens, new_lens, seq_lens, block_table, ring, ring_state, ring_state_out, cu_new,
                          n_slots, slots, positions, token_seqs, ws, S(stream));
}

lora_status kv_write(const kv_shape* shape, int64_t n, const uint16_t* k, int64_t k_stride,
                     const uint16_t* v, int64_t v_stride, const int32_t* slots, void* k_cache,
                     void* v_cache, uint8_t* k_scales, uint8_t* v_scales, void* ws,
                     size_t ws_bytes, void* stream) {
  TRY(check_kv(shape, "kv_write"));
  const kv_shape& s = *shape;
  const int64_t cols = (int64_t)s.n_kv_heads * s.head_dim;
  LORA_ARG_CHECK(n >= 0 && n < (1 << 30), "kv_write: n %lld outside [0, 2^30)", (long long)n);
  LORA_ARG_CHECK(n == 0 || (k && v && slots), "kv_write: k, v and slots must be non-NULL");
  LORA_ARG_CHECK(aligned16(k) && aligned16(v) && aligned(slots, 4), "kv_write: k and v must be 16-byte aligned, slots 4-byte");
  for (int64_t st : {k_stride, v_stride})
    LORA_ARG_CHECK(st % 8 == 0 && st >= cols && st < ((int64_t)1 << 31),
                   "kv_write: stride %lld must be a multiple of 8 in [%lld, 2^31)", (long long)st, (long long)cols);
  TRY(check_caches(s, k_cache, v_cache, k_scales, v_scales, "kv_write"));
  TRY(check_ws(ws, ws_bytes, 256, "kv_write"));
  const int64_t rows = cache_rows(s), half = k_scales ? s.head_dim / 2 : s.head_dim;   // of two bytes
  for (const void* c : {k_cache, v_cache})
    LORA_ARG_CHECK(!meet(span(c, rows, half, half), span(k, n, k_stride, cols)) &&
                       !meet(span(c, rows, half, half), span(v, n, v_stride, cols)),
                   "kv_write: a cache overlaps k or v");
  LORA_ARG_CHECK(!meet(span(k_cache, rows, half, half), span(v_cache, rows, half, half)), "kv_write: the caches overlap");
  const int64_t sb = rows * (s.head_dim / 32);
  const Span out[] = {bytes(k_scales, sb), bytes(v_scales, sb), bytes(ws, 256)};
  const Span in[] = {span(k, n, k_stride, cols), span(v, n, v_stride, cols), span(k_cache, rows, half, half),
                     span(v_cache, rows, half, half), bytes(slots, 4 * n)};
  LORA_ARG_CHECK(clash(out, in) < 0, "kv_write: the scales or the workspace overlap another operand");
  LORA_ARG_CHECK(!meet(in[2], in[4]) && !meet(in[3], in[4]), "kv_write: a cache overlaps slots");
  if (n == 0) return LORA_OK;
  return launch_kv_write(s, n, k, k_stride, v, v_stride, slots, k_cache, v_cache, k_scales, v_scales, ws, S(stream));
}

static lora_status check_decode(const kv_shape* shape, int32_t n_heads, int64_t max_len) {
  TRY(check_kv(shape, "attention_decode"));
  const kv_shape& s = *shape;
  LORA_ARG_CHECK(n_heads >= 1 && n_heads <= 1024 && n_heads % s.n_kv_heads == 0,
                 "attention_decode: n_heads %d must be a multiple of n_kv_heads %d, at most 1024", n_heads, s.n_kv_heads);
  LORA_ARG_CHECK(max_len >= 0 && max_len <= (int64_t)s.max_pages * s.page_size,
                 "attention_decode: max_len %lld outside [0, max_pages * page_size]", (long long)max_len);
  if (max_len > (1 << 30)) return unsupported("attention_decode", "max_len must not pass 2^30");
  // a launch takes fewer than 2^32 threads
  if ((int64_t)s.n_seqs * 32 * s.n_kv_heads * cdiv(n_heads / s.n_kv_heads, 16) >= 1 << 24)
    return unsupported("attention_decode", "too many requests times heads for one launch");
  return LORA_OK;
}

size_t attention_decode_workspace_bytes(const kv_shape* shape, int32_t n_heads, int64_t max_len) {
  if (check_decode(shape, n_heads, max_len) != LORA_OK) return 0;
  return decode_ws_bound(*shape, n_heads, max_len);
}

lora_status attention_decode(const kv_shape* shape, int32_t n_heads, const uint16_t* q,
                             int64_t q_stride, const void* k_cache, const void* v_cache,
                             const uint8_t* k_scales, const uint8_t* v_scales,
                             const int32_t* block_table, const int32_t* seq_lens,
                             int64_t max_len, float scale, uint16_t* o, float* lse, void* ws,
                             size_t ws_bytes, void* stream) {
  TRY(check_decode(shape, n_heads, max_len));
  const kv_shape& s = *shape;
  const int64_t cols = (int64_t)n_heads * s.head_dim;
  LORA_ARG_CHECK(scale_ok(scale), "attention_decode: scale must be below 2^127 in magnitude");
  LORA_ARG_CHECK(s.n_seqs == 0 || (q && o && block_table && seq_lens),
                 "attention_decode: q, o, block_table and seq_lens must be non-NULL");
  LORA_ARG_CHECK(aligned16(q) && aligned16(o), "attention_decode: q and o must be 16-byte aligned");
  LORA_ARG_CHECK(aligned(block_table, 4) && aligned(seq_lens, 4) && aligned(lse, 4),
                 "attention_decode: block_table, seq_lens and lse must be 4-byte aligned");
  LORA_ARG_CHECK(q_stride % 8 == 0 && q_stride >= cols && q_stride < ((int64_t)1 << 31),
                 "attention_decode: q_stride %lld must be a multiple of 8 in [%lld, 2^31)", (long long)q_stride, (long long)cols);
  TRY(check_caches(s, k_cache, v_cache, k_scales, v_scales, "attention_decode"));
  TRY(check_ws(ws, ws_bytes, decode_ws_bytes(s, n_heads, max_len), "attention_decode"));
  LORA_ARG_CHECK(!meet(span(o, s.n_seqs, cols, cols), span(q, s.n_seqs, q_stride, cols)), "attention_decode: o overlaps q");
  const int64_t rows = cache_rows(s), half = k_scales ? s.head_dim / 2 : s.head_dim, sb = rows * (s.head_dim / 32);
  const Span out[] = {span(o, s.n_seqs, cols, cols), bytes(lse, 4 * (int64_t)s.n_seqs * n_heads),
                      bytes(ws, (int64_t)decode_ws_bytes(s, n_heads, max_len))};
  const Span in[] = {span(q, s.n_seqs, q_stride, cols), span(k_cache, rows, half, half), span(v_cache, rows, half, half),
                     bytes(k_scales, sb), bytes(v_scales, sb), bytes(block_table, 4 * (int64_t)s.n_seqs * s.max_pages),
                     bytes(seq_lens, 4 * (int64_t)s.n_seqs)};
  LORA_ARG_CHECK(clash(out, in) < 0, "attention_decode: an output overlaps another operand");
  if (s.n_seqs == 0) return LORA_OK;
  return launch_decode(s, n_heads, q, q_stride, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, max_len,
                       scale, o, lse, ws, S(stream));
}

}  // extern "C"
