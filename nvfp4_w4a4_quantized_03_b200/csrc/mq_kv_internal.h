// mq_kv_internal.h -- launchers of the attention block's calls and of the linear
// with bf16 activation, shared by the CUDA translation units (not part of the
// public C ABI, which is include/mq.h).
#pragma once
#include "../../include/mq.h"
#include "mq_internal.h"

namespace mq {

// mq_rope_kv_append and mq_kv_attention (checked arguments of include/mq.h).
struct KvAppendArgs {
    const void* qkv;
    int64_t T, row_stride;
    int q_heads, rot_dim, interleaved;
    const float* rope;
    int64_t max_pos;
    const mq_kv_cache* cache;
    const mq_kv_batch* batch;
    void* q_out;
    int* status;             // may be null
};
cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream);

struct KvAttentionArgs {
    const void* q;
    int64_t T, q_row_stride;
    int q_heads;
    const mq_kv_cache* cache;
    const mq_kv_batch* batch;
    int64_t max_q, max_len;
    float scale;
    void* out;
    void* ws;
};
cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t stream);
struct KvAttendParams;
cudaError_t launch_kv_prefill(const KvAttendParams& p, int head_dim, int64_t blocks, cudaStream_t stream);

// mq_linear_w4a16: M <= 64 rows of bf16 X against an NVFP4 weight.
cudaError_t launch_linear_w4a16(const void* x, int64_t M, int64_t K, const uint8_t* w_codes, const uint8_t* w_scales,
                                const float* alpha_w, int64_t N, void* y, int num_sms, cudaStream_t stream);

// Debug build (MQ_DEBUG): bounds-check hits of each translation unit since
// its last read (0 in the release build).
namespace kv_append { unsigned long long debug_hits_kv_append(); }
namespace kv_attend { unsigned long long debug_hits_kv_attend(); }
namespace kv_prefill { unsigned long long debug_hits_kv_prefill(); }
namespace w4a16 { unsigned long long debug_hits_w4a16(); }

}  // namespace mq
