// mq_kv_append.cu -- rotary positions on Q and K of a fused QKV product, and
// the append of K and V to a paged cache of E4M3 codes (mq_rope_kv_append).
//
// Mathematics, for a token at position p and a head row x of D elements whose
// first r are rotated (pairs (a, b) = (x_j, x_{j + r/2}), or (x_2j, x_2j+1)
// interleaved; c, s the table's cosine and sine of pair j at p):
//     a' = fl32(fl32(a c) - fl32(b s)),   b' = fl32(fl32(b c) + fl32(a s))
// every step one binary32 operation, so the result does not depend on how the
// work is split.  Q leaves rounded to bf16.  K and V of the tokens that fall
// into one page become E4M3 codes under the page's scale for their head,
//     2^e,  e = least integer with max|x| <= 448 * 2^e  (clamped to [-96, 119]),
// a power of two: E4M3 keeps its four significant bits wherever in its range
// the values lie, and when later tokens need a larger scale the earlier codes
// are rescaled by an exact power of two (only codes that become subnormal
// round, once per growth).
//
// Bound: memory.  One block per (page, kv head) holds the page's new rows in
// registers between the maximum and the codes, so K and V are read once and
// written once; the Q rows ride in the same launch.  8192 tokens of 32 + 2 x 8
// heads of 128 (189 MB algorithmic): figures beside launch_kv_append.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/mq.h"
#include "mq_debug.cuh"
#include "mq_internal.h"
#include "mq_kv.cuh"
#include "mq_ptx.cuh"

namespace mq {
namespace kv_append {

constexpr int Q_ROWS = 2;                 // rows of Q per block

struct Params {
    const __nv_bfloat16* qkv;     // [T, row_stride]
    const float* rope;            // [max_pos, rot_dim], cosines then sines
    const int* cu;                // [batch + 1]
    const int* lens;              // [batch]
    const int* table;             // [batch, max_pages]
    uint8_t* k_codes;
    uint8_t* v_codes;
    float* k_scales;
    float* v_scales;
    __nv_bfloat16* q_out;         // [T, q_heads, D]
    int* status;
    int64_t T, row_stride, max_pos, num_pages, max_pages;
    int batch, q_heads, kv_heads, rot_dim, interleaved;
    int kv_blocks;                // blocks [0, kv_blocks) append, the rest rotate Q
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// The cosines and sines that the 8 elements from d0 need (d0 < rot_dim).
struct CosSin {
    float c[8], s[8];
};
__device__ __forceinline__ void load_cos_sin(const float* row, int d0, int rot_dim, int interleaved, CosSin& cs) {
    const int half = rot_dim >> 1;
    if (interleaved) {
        const float4 c = *reinterpret_cast<const float4*>(row + (d0 >> 1));
        const float4 s = *reinterpret_cast<const float4*>(row + half + (d0 >> 1));
        cs.c[0] = c.x; cs.c[1] = c.y; cs.c[2] = c.z; cs.c[3] = c.w;
        cs.s[0] = s.x; cs.s[1] = s.y; cs.s[2] = s.z; cs.s[3] = s.w;
    } else {
        const int j = d0 < half ? d0 : d0 - half;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 c = *reinterpret_cast<const float4*>(row + j + i);
            const float4 s = *reinterpret_cast<const float4*>(row + half + j + i);
            cs.c[i] = c.x; cs.c[i + 1] = c.y; cs.c[i + 2] = c.z; cs.c[i + 3] = c.w;
            cs.s[i] = s.x; cs.s[i + 1] = s.y; cs.s[i + 2] = s.z; cs.s[i + 3] = s.w;
        }
    }
}

// x: the 8 elements from d0; y: the 8 elements half a rotation away (half layout).
__device__ __forceinline__ void rotate8(float (&x)[8], const uint4& partner, int d0, int rot_dim, int interleaved,
                                        const CosSin& cs) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(a, cs.c[i]), __fmul_rn(b, cs.s[i]));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(b, cs.c[i]), __fmul_rn(a, cs.s[i]));
        }
    } else {
        float y[8];
        unpack8(partner, y);
        const bool lo = d0 < (rot_dim >> 1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = __fmul_rn(x[i], cs.c[i]), v = __fmul_rn(y[i], cs.s[i]);
            x[i] = lo ? __fsub_rn(u, v) : __fadd_rn(u, v);
        }
    }
}

__device__ __forceinline__ int partner_offset(int d0, int rot_dim) {
    const int half = rot_dim >> 1;
    return d0 < half ? half : -half;
}

// Least e in [KV_E_MIN, KV_E_MAX] with amax <= 448 * 2^e; 448 = 1.75 * 2^8.
__device__ __forceinline__ int page_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return max(KV_E_MIN, min(KV_E_MAX, e));
}

__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = cvt_e4m3x2(x[2 * i + 1] * inv, x[2 * i] * inv);
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ void decode8(const uint2& v, float (&x)[8]) {
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = cvt_e4m3x2_to_f16x2((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
        const __half2 p = *reinterpret_cast<const __half2*>(&h);
        x[2 * i] = __low2float(p);
        x[2 * i + 1] = __high2float(p);
    }
}

// D / 8 threads hold one token's row, 8 elements each.
template <int D, int P>
struct Shape {
    static constexpr int LANES = D / 8;
    static constexpr int PASSES = P * LANES >= 256 ? 2 : 1;
    static constexpr int THREADS = P * LANES / PASSES;
    static constexpr int TOKENS = P / PASSES;            // per pass
    static_assert(TOKENS * PASSES == P && THREADS % 32 == 0, "page shape");
};

// One page of one sequence, one kv head.
template <int D, int P>
__device__ __forceinline__ void append_page(const Params& p, int block) {
    using S = Shape<D, P>;
    __shared__ int s_seq;
    __shared__ uint32_t s_top[2][32];
    const int tid = threadIdx.x;
    const int slot = block / p.kv_heads, head = block % p.kv_heads;
    // Slots of sequence b start at cu[b] / P + 2 b: its n new tokens touch at
    // most floor(n / P) + 2 pages, which is what the next start leaves room for.
    if (tid == 0) s_seq = -1;
    __syncthreads();
    for (int b = tid; b < p.batch; b += S::THREADS) {
        const int c0 = p.cu[b], c1 = p.cu[b + 1];
        if (c1 > c0 && c0 >= 0) {
            const int base = c0 / P + 2 * b, next = c1 / P + 2 * (b + 1);
            if (slot >= base && slot < next) s_seq = b;
        }
    }
    __syncthreads();
    const int b = s_seq;
    if (b < 0) return;
    const int c0 = p.cu[b], n = p.cu[b + 1] - c0;
    const int64_t len = p.lens[b], start = len - n;           // position of the first new token
    const int64_t page0 = start > 0 ? start / P : 0;
    const int64_t pi = page0 + (slot - (c0 / P + 2 * b));
    if (pi * P >= len) return;
    const int first = pi == page0 && start > 0 ? (int)(start % P) : 0;   // earlier tokens in this page
    // tables that do not hold what the batch names: nothing is written
    const int64_t last = min(len, (pi + 1) * P) - 1;
    bool ok = pi < p.max_pages && (int64_t)c0 + n <= p.T && (p.rot_dim == 0 || last < p.max_pos);
    const int64_t page = ok ? p.table[(int64_t)b * p.max_pages + pi] : -1;
    ok = ok && page >= 0 && page < p.num_pages;
    if (!ok) {
        if (tid == 0 && p.status) atomicExch(p.status, MQ_ERR_INVALID_ARG);
        return;
    }
    const int lane = tid % S::LANES, d0 = lane * 8;
    const bool rotated = d0 < p.rot_dim;
    const int partner = !p.interleaved && rotated ? partner_offset(d0, p.rot_dim) : 0;
    const __nv_bfloat16* kcol = p.qkv + (int64_t)(p.q_heads + head) * D + d0;
    const __nv_bfloat16* vcol = kcol + (int64_t)p.kv_heads * D;

    float k[S::PASSES][8];
    uint4 v[S::PASSES];
    float ktop = 0.f, vtop = 0.f;
#pragma unroll
    for (int i = 0; i < S::PASSES; ++i) {
        const int64_t pos = pi * P + i * S::TOKENS + tid / S::LANES;
        const bool mine = pos >= start && pos < len && MQ_CHECK(c0 + pos - start >= 0 && c0 + pos - start < p.T);
        uint4 kw = make_uint4(0, 0, 0, 0), kp = kw;
        v[i] = kw;
        if (mine) {
            const int64_t off = (c0 + pos - start) * p.row_stride;
            kw = *reinterpret_cast<const uint4*>(kcol + off);
            v[i] = *reinterpret_cast<const uint4*>(vcol + off);
            if (partner) kp = *reinterpret_cast<const uint4*>(kcol + off + partner);
        }
        unpack8(kw, k[i]);
        if (mine && rotated) {
            CosSin cs;
            load_cos_sin(p.rope + pos * p.rot_dim, d0, p.rot_dim, p.interleaved, cs);
            rotate8(k[i], kp, d0, p.rot_dim, p.interleaved, cs);
        }
        float x[8];
        unpack8(v[i], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {          // fmaxf: a NaN leaves the scale as it is
            ktop = fmaxf(ktop, fabsf(k[i][j]));
            vtop = fmaxf(vtop, fabsf(x[j]));
        }
    }
    const uint32_t kb = __reduce_max_sync(0xffffffffu, __float_as_uint(ktop));
    const uint32_t vb = __reduce_max_sync(0xffffffffu, __float_as_uint(vtop));
    if (tid % 32 == 0) {
        s_top[0][tid / 32] = kb;
        s_top[1][tid / 32] = vb;
    }
    const int64_t cell = page * p.kv_heads + head;
    float old_k = 0.f, old_v = 0.f;
    if (first > 0) {
        old_k = p.k_scales[cell];
        old_v = p.v_scales[cell];
    }
    __syncthreads();
    uint32_t kt = 0, vt = 0;
#pragma unroll
    for (int w = 0; w < S::THREADS / 32; ++w) {
        kt = max(kt, s_top[0][w]);
        vt = max(vt, s_top[1][w]);
    }
    const float scale_k = fmaxf(old_k, exp2i(page_exponent(__uint_as_float(kt))));
    const float scale_v = fmaxf(old_v, exp2i(page_exponent(__uint_as_float(vt))));
    const float inv_k = __fdiv_rn(1.f, scale_k), inv_v = __fdiv_rn(1.f, scale_v);
    if (tid == 0) {                            // every thread has read the old ones: they passed the barrier
        p.k_scales[cell] = scale_k;
        p.v_scales[cell] = scale_v;
    }
    uint8_t* kout = p.k_codes + cell * (P * D) + d0;
    uint8_t* vout = p.v_codes + cell * (P * D) + d0;
    const bool grow_k = first > 0 && scale_k > old_k, grow_v = first > 0 && scale_v > old_v;
    const float down_k = __fdiv_rn(old_k, scale_k), down_v = __fdiv_rn(old_v, scale_v);
#pragma unroll
    for (int i = 0; i < S::PASSES; ++i) {
        const int tok = i * S::TOKENS + tid / S::LANES;
        const int64_t pos = pi * P + tok;
        const bool mine = pos >= start && pos < len;
        if (tok < first) {
            // earlier tokens of the page, brought to the grown scale
            float x[8];
            if (grow_k) {
                decode8(*reinterpret_cast<const uint2*>(kout + tok * D), x);
                *reinterpret_cast<uint2*>(kout + tok * D) = encode8(x, down_k);
            }
            if (grow_v) {
                decode8(*reinterpret_cast<const uint2*>(vout + tok * D), x);
                *reinterpret_cast<uint2*>(vout + tok * D) = encode8(x, down_v);
            }
        }
        // A NaN in V would reach every row of a later product with the page,
        // also rows that do not see the token; stored in K it reaches the
        // token's score, so exactly the rows that see the token become NaN.
        float x[8];
        unpack8(v[i], x);
        bool nan = false;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (x[j] != x[j]) {
                nan = true;
                x[j] = 0.f;
            }
        const uint32_t votes = __ballot_sync(0xffffffffu, nan);
        const uint32_t group = (votes >> (tid % 32 / S::LANES * S::LANES)) & ((S::LANES == 32) ? ~0u : (1u << S::LANES) - 1u);
        if (mine) {
            uint2 kc = encode8(k[i], inv_k);
            if (group && lane == 0) kc.x |= 0x7Fu;
            *reinterpret_cast<uint2*>(kout + tok * D) = kc;
            *reinterpret_cast<uint2*>(vout + tok * D) = encode8(x, inv_v);
        }
    }
}

// Two rows of Q: a thread keeps 8 columns of one head at a time, the loads of
// both rows in flight together.
template <int D>
__device__ __forceinline__ void rotate_q(const Params& p, int block, int threads) {
    constexpr int LANES = D / 8;
    __shared__ int64_t s_pos[Q_ROWS];
    const int tid = threadIdx.x;
    const int64_t r0 = (int64_t)block * Q_ROWS;
    if (tid < Q_ROWS) s_pos[tid] = -1;
    __syncthreads();
    for (int b = tid; b < p.batch; b += threads) {
        const int64_t c0 = p.cu[b], c1 = p.cu[b + 1];
        const int64_t lo = max(c0, r0), hi = min(min(c1, r0 + Q_ROWS), p.T);
        if (lo < hi) {
            const int64_t shift = (int64_t)p.lens[b] - c1;
            for (int64_t r = lo; r < hi; ++r) s_pos[r - r0] = r + shift;
        }
    }
    __syncthreads();
    const int lane = tid % LANES, d0 = lane * 8, groups = threads / LANES;
    const bool rotated = d0 < p.rot_dim;
    const int partner = !p.interleaved && rotated ? partner_offset(d0, p.rot_dim) : 0;
    int64_t pos[Q_ROWS];
#pragma unroll
    for (int r = 0; r < Q_ROWS; ++r) {
        pos[r] = s_pos[r];                        // negative: padding, the row stays as it was
        if (rotated && pos[r] >= p.max_pos) {
            if (p.status) atomicExch(p.status, MQ_ERR_INVALID_ARG);
            pos[r] = -1;
        }
    }
    for (int h = tid / LANES; h < p.q_heads; h += groups) {
        const __nv_bfloat16* src = p.qkv + r0 * p.row_stride + h * D + d0;
        uint4 w[Q_ROWS], y[Q_ROWS];
#pragma unroll
        for (int r = 0; r < Q_ROWS; ++r) {
            w[r] = y[r] = make_uint4(0, 0, 0, 0);
            if (pos[r] >= 0) {
                w[r] = *reinterpret_cast<const uint4*>(src + r * p.row_stride);
                if (partner) y[r] = *reinterpret_cast<const uint4*>(src + r * p.row_stride + partner);
            }
        }
#pragma unroll
        for (int r = 0; r < Q_ROWS; ++r) {
            if (pos[r] < 0) continue;
            if (rotated) {
                CosSin cs;
                load_cos_sin(p.rope + pos[r] * p.rot_dim, d0, p.rot_dim, p.interleaved, cs);
                float x[8];
                unpack8(w[r], x);
                rotate8(x, y[r], d0, p.rot_dim, p.interleaved, cs);
                w[r] = make_uint4(cvt_bf16x2(x[1], x[0]), cvt_bf16x2(x[3], x[2]), cvt_bf16x2(x[5], x[4]),
                                  cvt_bf16x2(x[7], x[6]));
            }
            if (MQ_CHECK(r0 + r < p.T && h < p.q_heads))
                *reinterpret_cast<uint4*>(p.q_out + ((r0 + r) * p.q_heads + h) * D + d0) = w[r];
        }
    }
}

template <int D, int P>
__global__ void __launch_bounds__(Shape<D, P>::THREADS, 1024 / Shape<D, P>::THREADS) k_kv_append(Params p) {
    pdl_launch_dependents();
    pdl_wait();
    if ((int)blockIdx.x < p.kv_blocks)
        append_page<D, P>(p, blockIdx.x);
    else
        rotate_q<D>(p, blockIdx.x - p.kv_blocks, Shape<D, P>::THREADS);
}

MQ_DEBUG_READER(debug_hits_kv_append)

template <int D, int P>
cudaError_t launch(const Params& p, int64_t blocks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    int nattr = 0;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(Shape<D, P>::THREADS);
    cfg.stream = stream;
    set_pdl_attr(attr, &nattr);
    cfg.attrs = attr;
    cfg.numAttrs = nattr;
    return cudaLaunchKernelEx(&cfg, k_kv_append<D, P>, p);
}

}  // namespace kv_append

// ---------------------------------------------------------------- host side
cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
    using namespace kv_append;
    const mq_kv_cache& c = *a.cache;
    const mq_kv_batch& s = *a.batch;
    Params p{};
    p.qkv = static_cast<const __nv_bfloat16*>(a.qkv);
    p.rope = a.rope;
    p.cu = s.cu_rows;
    p.lens = s.lens;
    p.table = s.page_table;
    p.k_codes = c.k_codes;
    p.v_codes = c.v_codes;
    p.k_scales = c.k_scales;
    p.v_scales = c.v_scales;
    p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
    p.status = a.status;
    p.T = a.T;
    p.row_stride = a.row_stride;
    p.max_pos = a.max_pos;
    p.num_pages = c.num_pages;
    p.max_pages = s.max_pages;
    p.batch = s.batch;
    p.q_heads = a.q_heads;
    p.kv_heads = c.kv_heads;
    p.rot_dim = a.rot_dim;
    p.interleaved = a.interleaved;
    const int64_t slots = a.T / c.page_size + 2 * (int64_t)s.batch;
    const int64_t kv_blocks = slots * c.kv_heads;
    const int64_t q_blocks = (a.T + Q_ROWS - 1) / Q_ROWS;
    if (kv_blocks + q_blocks > 0x7fffffff) return cudaErrorInvalidValue;
    p.kv_blocks = (int)kv_blocks;
    const int64_t blocks = kv_blocks + q_blocks;
#define MQ_KV_APPEND(D_, P_) \
    if (c.head_dim == D_ && c.page_size == P_) return launch<D_, P_>(p, blocks, stream);
    MQ_KV_APPEND(64, 16) MQ_KV_APPEND(64, 32) MQ_KV_APPEND(64, 64) MQ_KV_APPEND(64, 128)
    MQ_KV_APPEND(128, 16) MQ_KV_APPEND(128, 32) MQ_KV_APPEND(128, 64) MQ_KV_APPEND(128, 128)
#undef MQ_KV_APPEND
    return cudaErrorInvalidValue;
}

}  // namespace mq
