// host_util.h -- host helpers that the C entry points share (defined in host.cu).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime_api.h>

#include "gqa_decode.h"

namespace gqa {

// Sets this thread's gqa_last_error() text and returns s.
gqa_status fail(gqa_status s, const char* fmt, ...);
gqa_status cuda_fail(cudaError_t e, const char* what);
bool aligned16(const void* p);
// Shapes that do not depend on the device.
gqa_status check_shape(int n_tok, int n_heads, int n_kv_heads, int head_dim, int max_kv_len,
                       int kind);
// SM count of the current device, cached per device id; <= 0 and *st set when it cannot be had.
int current_sm_count(gqa_status* st);

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // null when the driver has none
gqa_status encode_f16_cache(const void* kc, const void* vc, int n_seq, int64_t cache_cap,
                            int n_kv_heads, int head_dim, int tile, CUtensorMap* tk,
                            CUtensorMap* tv);

// The plan of the calls with a visible set (visible_host.cu): budget is the most positions a row
// sees (-1: all of them).
gqa_status plan_visible(int n_tok, int n_seq, int n_heads, int n_kv_heads, int head_dim,
                        int max_kv_len, int budget, int kind, int num_sms, gqa_plan* plan);

}  // namespace gqa
