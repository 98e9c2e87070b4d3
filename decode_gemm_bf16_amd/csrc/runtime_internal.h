// Internal entry points of runtime.cpp shared with other sources of the library.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/uw.h"
#include "attention.h"

namespace uw {

// The SwiGLU layer behind uw_mlp_forward, with fused_only restricting every
// projection to the fused direct-palette kernels (no allocation anywhere).
uw_status mlp_forward_impl(uw_handle gate, uw_handle up, uw_handle down, const int32_t* pipelines,
                           const uint16_t* x_dev, float* y_dev, int64_t tokens, void* work_dev, size_t work_bytes,
                           bool fused_only);

// uw_route's checks and its launch (routing.cpp).
uw_status route_check(const void* logits, int32_t type, int64_t ld, int64_t tokens, const float* bias,
                      const uw_route_config* c, const int32_t* experts, const float* weights);
uw_status route_launch(const void* logits, int32_t type, int64_t ld, int64_t tokens, const float* bias,
                       const uw_route_config* c, int32_t* experts, float* weights, hipStream_t s);

// The sizes that uw_attend_workspace_bytes and uw_attention_workspace_bytes take (attention.cpp).
uw_status attention_sizes_check(const uw_cache_config* config, int64_t tokens, int64_t seqs, int64_t max_tokens,
                                int64_t max_length);
// uw_cache_write's and uw_attend's checks, and their kernels' arguments (attention.cpp).
uw_status cache_write_prepare(const uw_cache_config* config, const uw_rotary* rotary, const void* q_dev,
                          int64_t ldq, const void* k_dev, int64_t ldk, const void* v_dev, int64_t ldv, int32_t type,
                          const int32_t* positions_dev, const float* freqs_dev, const int32_t* axis_dev,
                          const int32_t* slots_dev, int64_t tokens, uint16_t* q_out_dev, int64_t ldq_out,
                          uint16_t* k_cache_dev, uint16_t* v_cache_dev, CacheWriteArgs* out);
uw_status attend_prepare(const uw_cache_config* config, const uw_attend_config* options, const uint16_t* q_dev,
                          int64_t ldq, const uint16_t* k_cache_dev, const uint16_t* v_cache_dev,
                          const int32_t* offsets_dev, const int32_t* lengths_dev, const int32_t* tables_dev,
                          int64_t ldt, int64_t max_pages, const float* slopes_dev, const int32_t* prefix_dev,
                          const int32_t* first_dev, const uint64_t* mask_dev, int32_t mask_words, int64_t tokens,
                          int64_t seqs, int64_t max_tokens, int64_t max_length, void* y_dev, int64_t ldy,
                          int32_t y_type, float* lse_dev, void* work_dev, size_t work_bytes, AttendArgs* out,
                          AttendPlan* plan_out);

// Sets the thread-local error text read by uw_last_error and returns st.
uw_status set_error(uw_status st, const char* msg);

}  // namespace uw
