// Launches of the attention and key-value cache kernels.
#pragma once

#include "common.hpp"

namespace lora_host {

// attn.hip
lora_status launch_attention_fwd(const attn_shape& sh, const uint16_t* q, const uint16_t* k,
                                 const uint16_t* v, const int32_t* cu_q, const int32_t* cu_k,
                                 uint16_t* o, float* lse, void* ws, hipStream_t s);
lora_status launch_attention_bwd(const attn_shape& sh, const uint16_t* dout, const uint16_t* q,
                                 const uint16_t* k, const uint16_t* v, const uint16_t* o,
                                 const float* lse, const int32_t* cu_q, const int32_t* cu_k,
                                 uint16_t* dq, uint16_t* dk, uint16_t* dv, void* ws, hipStream_t s);

// kvcache.hip
lora_status launch_kv_tables(const kv_shape& sh, const int32_t* cached, const int32_t* fresh,
                             int32_t* seq_lens, int32_t* table, int32_t* ring, const int64_t* state,
                             int64_t* state_out, int32_t* cu_new, int64_t n_slots, int32_t* slots,
                             int32_t* positions, int32_t* token_seqs, void* ws, hipStream_t s);
lora_status launch_kv_write(const kv_shape& sh, int64_t n, const uint16_t* k, int64_t k_stride,
                            const uint16_t* v, int64_t v_stride, const int32_t* slots, void* k_cache,
                            void* v_cache, uint8_t* k_scales, uint8_t* v_scales, void* ws,
                            hipStream_t s);
size_t decode_ws_bytes(const kv_shape& sh, int32_t n_heads, int64_t max_len);
size_t decode_ws_bound(const kv_shape& sh, int32_t n_heads, int64_t max_len);
lora_status launch_decode(const kv_shape& sh, int32_t n_heads, const uint16_t* q, int64_t q_stride,
                          const void* k_cache, const void* v_cache, const uint8_t* k_scales,
                          const uint8_t* v_scales, const int32_t* table, const int32_t* seq_lens,
                          int64_t max_len, float scale, uint16_t* o, float* lse, void* ws,
                          hipStream_t s);

}  // namespace lora_host
