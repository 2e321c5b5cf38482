// mq_kv.cuh -- what the append to the paged E4M3 cache and the two forms of the
// attention over it share: the page scale's range, the attention's parameters,
// and the join of a cell's chunks.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "mq_debug.cuh"
#include "mq_ptx.cuh"

namespace mq {

// A page's scale is 2^e, e in this range: 448 * 2^119 is the largest bf16's
// binade, and 2^96 * (number of tokens) still fits binary32, which the
// attention's sums of 2^-e-weighted terms need.
constexpr int KV_E_MIN = -96, KV_E_MAX = 119;

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two binary32 operations per instruction
__device__ __forceinline__ uint64_t pack2u(uint32_t x, uint32_t y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ uint64_t pack2(float x, float y) { return pack2u(__float_as_uint(x), __float_as_uint(y)); }
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Of each half of a pair: the larger of a and |b|; a NaN in b counts as nothing.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %2;\n\tmax.bf16x2 %0, %1, t;\n\t}" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

struct KvAttendParams {
    const __nv_bfloat16* q;              // [T, q_stride]
    const int* cu;
    const int* lens;
    const int* table;
    const uint8_t* k_codes;
    const uint8_t* v_codes;
    const float* k_scales;
    const float* v_scales;
    __nv_bfloat16* out;                  // [T, q_heads, D]
    int* status;
    int* tickets;                        // one per (sequence, row tile, kv head)
    float* part;                         // partial results
    int64_t T, q_stride, num_pages, max_pages, max_len;
    int batch, q_heads, kv_heads, group, page_log2, max_q;
    int row_tiles, chunks, chunk_tokens;
    int by_length;                       // tcgen05 form: blocks in the order of the keys they see
    float scale_log2;
};

// out of row `ri` (new token x head of the group) of the sequence at c0, four elements from 4 c4:
// acc / lsum, zero for a row that saw nothing.
template <int D>
__device__ __forceinline__ void kv_write_out(const KvAttendParams& p, int c0, int64_t ri, int head, int c4,
                                             const float4& acc, float lsum) {
    const float inv = lsum > 0.f || lsum != lsum ? __fdiv_rn(1.f, lsum) : 0.f;
    const int64_t at = ((c0 + ri / p.group) * p.q_heads + head * p.group + ri % p.group) * D + c4 * 4;
    if (MQ_CHECK(at + 4 <= p.T * p.q_heads * (int64_t)D))
        *reinterpret_cast<uint2*>(p.out + at) =
            make_uint2(cvt_bf16x2(acc.y * inv, acc.x * inv), cvt_bf16x2(acc.w * inv, acc.z * inv));
}

// A cell's partial results: [chunk][row][D] values, then [chunk][row] pairs (M, l),
// for p.chunks chunks of rows_cap rows.
template <int D>
__device__ __forceinline__ float* kv_part_ml(const KvAttendParams& p, float* part, int rows_cap) {
    return part + (int64_t)p.chunks * rows_cap * D;
}

// Joins the first `chunks` of them in their order; `weights`: shared memory of nrows * chunks floats.
template <int D>
__device__ __forceinline__ void kv_join(const KvAttendParams& p, float* part, int chunks, int rows_cap,
                                        int nrows, int c0, int64_t row0, int head, int tid, int threads,
                                        float* weights) {
    constexpr int V4 = D / 4;
    const int64_t step = (int64_t)rows_cap * D;
    const float2* ml = reinterpret_cast<const float2*>(kv_part_ml<D>(p, part, rows_cap));
    // each row's maximum and the chunks' weights 2^(M - max) / sum: by a warp per
    // row where rows are few, by a thread per row where they are many
    const int width = nrows <= 64 ? 32 : 1, lane = tid % width;
    for (int r = tid / width; r < nrows; r += threads / width) {
        float top = -INFINITY;
#pragma unroll 4
        for (int c = lane; c < chunks; c += width) top = fmaxf(top, __ldcg(&ml[c * rows_cap + r].x));
        if (width == 32) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
        float lsum = 0.f;
#pragma unroll 4
        for (int c = lane; c < chunks; c += width) {
            const float2 v = __ldcg(&ml[c * rows_cap + r]);
            const float f = v.x == -INFINITY ? 0.f : ex2(v.x - top);
            weights[r * chunks + c] = f;
            lsum = __fmaf_rn(v.y, f, lsum);
        }
        if (width == 32) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, o);
        }
        // a row that saw nothing: zero
        const float inv = lsum > 0.f || lsum != lsum ? __fdiv_rn(1.f, lsum) : 0.f;
        for (int c = lane; c < chunks; c += width) weights[r * chunks + c] *= inv;
    }
    __syncthreads();
    for (int i = tid; i < nrows * V4; i += threads) {
        const int r = i / V4, c4 = i % V4;
        const float4* src = reinterpret_cast<const float4*>(part + (int64_t)r * D + c4 * 4);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 16
        for (int c = 0; c < chunks; ++c) {
            const float4 x = __ldcg(src + c * (step / 4));
            const float f = weights[r * chunks + c];
            acc.x = __fmaf_rn(x.x, f, acc.x);
            acc.y = __fmaf_rn(x.y, f, acc.y);
            acc.z = __fmaf_rn(x.z, f, acc.z);
            acc.w = __fmaf_rn(x.w, f, acc.w);
        }
        kv_write_out<D>(p, c0, row0 + r, head, c4, acc, 1.f);
    }
}

}  // namespace mq
