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
// Bound: memory (one read of the product, one write of Q and of the codes).  One
// block per (page, kv head) finds the page's maximum and then writes its codes;
// the Q rows ride in the same launch.  8192 tokens of 32 + 2 x 8 heads of 128
// (189 MB algorithmic): 42 us, 4.5 TB/s (the Q rows alone take 31 us, K and V
// alone 18); one token of one sequence 3.1 us, of 64 sequences 4.1 us (in a graph).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "mq_debug.cuh"
#include "mq_kv.cuh"
#include "mq_kv_internal.h"
#include "mq_ptx.cuh"

namespace mq {
namespace kv_append {

constexpr int Q_ROWS_MAX = 8;

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
    int batch, q_heads, kv_heads, rot_dim;
    int q_rows;                   // rows of Q per block
    int by_row;                   // what the slots are (append_page)
    int kv_blocks;                // blocks [0, kv_blocks) append, the rest rotate Q
};

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// D / 16 threads hold one row, two vectors of 8 elements each, so placed that
// neighbouring threads read neighbouring vectors: half layout, rotated part:
// the two halves of 8 pairs (a row is read once, 8 cosines and sines serve 16
// elements); interleaved: vectors D / 2 apart, 4 pairs each.
struct Place {
    int at[2];                // first elements of the vectors
    bool rotated[2];
};
template <int D, bool INTERLEAVED>
__device__ __forceinline__ Place place_of(int lane, int rot_dim) {
    const int half = rot_dim >> 1;
    Place q;
    if (INTERLEAVED) {
        q.at[0] = 8 * lane;
        q.at[1] = 8 * lane + D / 2;
    } else if (8 * lane < half) {
        q.at[0] = 8 * lane;
        q.at[1] = 8 * lane + half;
    } else {
        q.at[0] = 16 * lane;                       // behind the rotated elements
        q.at[1] = 16 * lane + 8;
    }
    q.rotated[0] = q.at[0] < rot_dim;
    q.rotated[1] = q.at[1] < rot_dim;
    return q;
}

// Cosines and sines: of 8 pairs (half layout), of 4 pairs of either vector (interleaved).
struct CosSin {
    float c[8], s[8];
};
template <bool INTERLEAVED>
__device__ __forceinline__ void load_cos_sin(const float* row, const Place& at, int half, CosSin& cs) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const int column = INTERLEAVED ? at.at[i / 4] / 2 : at.at[0] + i;
        float4 c = make_float4(0.f, 0.f, 0.f, 0.f), s = c;
        if (!INTERLEAVED || at.rotated[i / 4]) {
            c = *reinterpret_cast<const float4*>(row + column);
            s = *reinterpret_cast<const float4*>(row + half + column);
        }
        cs.c[i] = c.x; cs.c[i + 1] = c.y; cs.c[i + 2] = c.z; cs.c[i + 3] = c.w;
        cs.s[i] = s.x; cs.s[i + 1] = s.y; cs.s[i + 2] = s.z; cs.s[i + 3] = s.w;
    }
}

// x: the two vectors, the first of them rotated.  One operation at a time: as
// pairs (mul and add .f32x2) the assembler joined product and sum into one
// rounding.
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate(float (&x)[16], const Place& at, const CosSin& cs) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (INTERLEAVED && i >= 4 && !at.rotated[1]) break;
        const int ia = INTERLEAVED ? 2 * i : i, ib = INTERLEAVED ? 2 * i + 1 : i + 8;
        const float a = x[ia], b = x[ib];
        x[ia] = __fsub_rn(__fmul_rn(a, cs.c[i]), __fmul_rn(b, cs.s[i]));
        x[ib] = __fadd_rn(__fmul_rn(b, cs.c[i]), __fmul_rn(a, cs.s[i]));
    }
}

// Least e in [KV_E_MIN, KV_E_MAX] with amax <= 448 * 2^e; 448 = 1.75 * 2^8.
__device__ __forceinline__ int page_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return max(KV_E_MIN, min(KV_E_MAX, e));
}

__device__ __forceinline__ bool any_nan_bf16x2(const uint4& v) {
    uint32_t r;
    asm("{\n\t.reg .b32 a, b;\n\tmax.NaN.bf16x2 a, %1, %2;\n\tmax.NaN.bf16x2 b, %3, %4;\n\tmax.NaN.bf16x2 %0, a, b;\n\t}"
        : "=r"(r) : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
    return (r & 0x7FFFu) > 0x7F80u || (r & 0x7FFF0000u) > 0x7F800000u;
}

__device__ __forceinline__ uint2 encode8(const float* x, float inv) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack2(mul2(pack2(x[2 * i], x[2 * i + 1]), pack2(inv, inv)), lo, hi);
        h[i] = cvt_e4m3x2(hi, lo);
    }
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ void decode8(const uint2& v, float* x) {
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = cvt_e4m3x2_to_f16x2((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
        const __half2 p = *reinterpret_cast<const __half2*>(&h);
        x[2 * i] = __low2float(p);
        x[2 * i + 1] = __high2float(p);
    }
}

constexpr int THREADS = 256;

// The part of a block that holds one kv head of a page: whole warps, the block
// where the page is large enough for it.
template <int D, int P>
struct Part {
    static constexpr int LANES = D / 16;                                      // threads of a token
    static constexpr int SIZE = P * LANES < THREADS ? P * LANES : THREADS;
    static constexpr int TOKENS = SIZE / LANES;                               // tokens at a time
    static constexpr int HEADS = THREADS / SIZE;                              // kv heads of a block
};

// One page of one sequence, Part::HEADS kv heads.
template <int D, int P, bool INTERLEAVED>
__device__ __forceinline__ void append_page(const Params& p, int block) {
    using S = Part<D, P>;
    constexpr int LANES = S::LANES, TOKENS = S::TOKENS, WARPS = S::SIZE / 32;
    __shared__ int s_seq;
    __shared__ uint32_t s_top[2][THREADS / 32];
    const int tid = threadIdx.x, part = tid / S::SIZE;
    const int groups = (p.kv_heads + S::HEADS - 1) / S::HEADS;
    const int slot = block / groups, head = block % groups * S::HEADS + part;
    const bool active = head < p.kv_heads;
    // Which page a slot is: with many rows, slots of sequence b start at cu[b] / P
    // + 2 b (its n new tokens touch at most floor(n / P) + 2 pages, which is what
    // the next start leaves room for); with few, a slot is a row, and the first
    // row of each page stands for it.
    if (tid == 0) s_seq = -1;
    __syncthreads();
    for (int b = tid; b < p.batch; b += THREADS) {
        const int c0 = p.cu[b], c1 = p.cu[b + 1];
        if (c1 > c0 && c0 >= 0) {
            const int base = p.by_row ? c0 : c0 / P + 2 * b, next = p.by_row ? c1 : c1 / P + 2 * (b + 1);
            if (slot >= base && slot < next) s_seq = b;
        }
    }
    __syncthreads();
    const int b = s_seq;
    if (b < 0) return;
    const int c0 = p.cu[b], n = p.cu[b + 1] - c0;
    const int64_t len = p.lens[b], start = len - n;           // position of the first new token
    int64_t pi = (start > 0 ? start / P : 0) + (slot - (c0 / P + 2 * b));
    if (p.by_row) {
        const int64_t pos = start + (slot - c0);
        if (pos < 0 || (slot != c0 && pos % P != 0)) return;
        pi = pos / P;
    }
    if (pi * P >= len) return;
    // the page's tokens [0, first) are earlier ones, [first, last) new
    const int first = (int)max((int64_t)0, start - pi * P);
    const int last = (int)min(len - pi * P, (int64_t)P);
    // tables that do not hold what the batch names: nothing is written
    bool ok = pi < p.max_pages && (int64_t)c0 + n <= p.T && (p.rot_dim == 0 || pi * P + last <= p.max_pos);
    const int64_t page = ok ? p.table[(int64_t)b * p.max_pages + pi] : -1;
    ok = ok && page >= 0 && page < p.num_pages;
    if (!ok) {
        if (tid == 0 && p.status) atomicExch(p.status, MQ_ERR_INVALID_ARG);
        return;
    }
    const int lane = tid % LANES, tok0 = tid % S::SIZE / LANES;
    const Place at = place_of<D, INTERLEAVED>(lane, p.rot_dim);
    const __nv_bfloat16* kcol =
        p.qkv + (c0 + pi * P - start) * p.row_stride + (int64_t)(p.q_heads + head) * D;           // of the page's token 0
    const int64_t v_off = (int64_t)p.kv_heads * D;

    // The page's new rows are read twice, the second time from L1 or L2: held
    // in registers between the maximum and the codes they cost the occupancy
    // that hides the first read.
    float k[16];
    uint4 v[2];
    auto load = [&](int tok) {
        const bool mine = active && tok < last && MQ_CHECK(c0 + pi * P + tok - start >= 0 && c0 + pi * P + tok - start < p.T);
        uint4 kw[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[i] = kw[i] = make_uint4(0, 0, 0, 0);
            if (mine) {
                const __nv_bfloat16* src = kcol + tok * p.row_stride + at.at[i];
                kw[i] = *reinterpret_cast<const uint4*>(src);
                v[i] = *reinterpret_cast<const uint4*>(src + v_off);
            }
        }
        unpack8(kw[0], k);
        unpack8(kw[1], k + 8);
        if (mine && at.rotated[0]) {
            CosSin cs;
            load_cos_sin<INTERLEAVED>(p.rope + (pi * P + tok) * p.rot_dim, at, p.rot_dim >> 1, cs);
            rotate<INTERLEAVED>(k, at, cs);
        }
    };
    float ktop = 0.f;                              // the head's maximum of K, of V (a bf16 pair)
    uint32_t vtop = 0;
    for (int base = first; base < last; base += TOKENS) {
        load(base + tok0);
#pragma unroll
        for (int j = 0; j < 16; ++j) ktop = fmaxf(ktop, fabsf(k[j]));       // a NaN leaves the scale as it is
#pragma unroll
        for (int i = 0; i < 2; ++i)
            vtop = max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(vtop, v[i].x), v[i].y), v[i].z), v[i].w);
    }
    const uint32_t kb = __reduce_max_sync(0xffffffffu, __float_as_uint(ktop));
    const uint32_t vb = __reduce_max_sync(0xffffffffu, max(vtop << 16, vtop & 0xFFFF0000u));
    if (tid % 32 == 0) {
        s_top[0][tid / 32] = kb;
        s_top[1][tid / 32] = vb;
    }
    const int64_t cell = page * p.kv_heads + head;
    float old[2] = {0.f, 0.f}, scale[2], inv[2];   // of K, of V
    if (first > 0 && active) {
        old[0] = p.k_scales[cell];
        old[1] = p.v_scales[cell];
    }
    __syncthreads();
    if (!active) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < WARPS; ++j) w = max(w, s_top[i][part * WARPS + j]);
        scale[i] = fmaxf(old[i], exp2i(page_exponent(__uint_as_float(w))));
        inv[i] = __fdiv_rn(1.f, scale[i]);
    }
    if (tid % S::SIZE == 0) {                      // every thread has read the old ones: they passed the barrier
        p.k_scales[cell] = scale[0];
        p.v_scales[cell] = scale[1];
    }
    uint8_t* out[2] = {p.k_codes + cell * (P * D), p.v_codes + cell * (P * D)};
    if (first > 0) {
        // earlier tokens of the page, brought to a scale that has grown
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (scale[i] <= old[i]) continue;
            const float down = __fdiv_rn(old[i], scale[i]);
            for (int tok = tok0; tok < first; tok += TOKENS)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint2* code = reinterpret_cast<uint2*>(out[i] + tok * D + at.at[e]);
                    float x[8];
                    decode8(*code, x);
                    *code = encode8(x, down);
                }
        }
    }
    const bool held = last - first <= TOKENS;
    for (int base = first; base < last; base += TOKENS) {
        const int tok = base + tok0;
        if (!held) load(tok);
        // A NaN in V would reach every row of a later product with the page,
        // also rows that do not see the token; stored in K it reaches the
        // token's score, so exactly the rows that see the token become NaN.
        float x[16];
        unpack8(v[0], x);
        unpack8(v[1], x + 8);
        const bool nan = any_nan_bf16x2(v[0]) || any_nan_bf16x2(v[1]);
        if (nan) {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = x[j] != x[j] ? 0.f : x[j];
        }
        const uint32_t votes = __ballot_sync(0xffffffffu, nan);
        const uint32_t token_votes = (votes >> (tid % 32 / LANES * LANES)) & ((1u << LANES) - 1u);
        if (tok < last) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint2 kc = encode8(k + 8 * i, inv[0]);
                if (i == 0 && token_votes && lane == 0) kc.x |= 0x7Fu;
                *reinterpret_cast<uint2*>(out[0] + tok * D + at.at[i]) = kc;
                *reinterpret_cast<uint2*>(out[1] + tok * D + at.at[i]) = encode8(x + 8 * i, inv[1]);
            }
        }
    }
}

// `q_rows` rows of Q, a few at a time: a thread keeps 16 columns of a row and
// walks heads two by two, so a row's cosines and sines are loaded once for
// all of them.  The first rows' X does not wait for the positions.
template <int D, bool INTERLEAVED>
__device__ __forceinline__ void rotate_q(const Params& p, int block) {
    constexpr int LANES = D / 16, WALK = 2;
    __shared__ int64_t s_pos[Q_ROWS_MAX];
    const int tid = threadIdx.x;
    const int64_t r0 = (int64_t)block * p.q_rows;
    const int rows = (int)min((int64_t)p.q_rows, p.T - r0);
    const int lane = tid % LANES, groups = THREADS / LANES, group = tid / LANES;
    const int at_once = max(1, min(rows, groups / ((p.q_heads + WALK - 1) / WALK)));   // rows at a time
    const int per_row = groups / at_once;                                      // groups of a row
    const int sub = group / per_row, h0 = group % per_row;
    const bool idle = sub >= at_once;                                          // groups left over
    const Place at = place_of<D, INTERLEAVED>(lane, p.rot_dim);
    uint4 w[WALK][2];
    auto load = [&](int r, int h) {
#pragma unroll
        for (int i = 0; i < WALK; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                w[i][e] = make_uint4(0, 0, 0, 0);
                if (r < rows && h + i * per_row < p.q_heads)
                    w[i][e] = *reinterpret_cast<const uint4*>(p.qkv + (r0 + r) * p.row_stride + (h + i * per_row) * D + at.at[e]);
            }
    };
    if (!idle) load(sub, h0);
    if (tid < Q_ROWS_MAX) s_pos[tid] = -1;
    __syncthreads();
    for (int b = tid; b < p.batch; b += THREADS) {
        const int64_t c0 = p.cu[b], c1 = p.cu[b + 1];
        const int64_t lo = max(c0, r0), hi = min(c1, r0 + rows);
        if (lo < hi) {
            const int64_t shift = (int64_t)p.lens[b] - c1;
            for (int64_t r = lo; r < hi; ++r) s_pos[r - r0] = r + shift;
        }
    }
    __syncthreads();
    if (idle) return;
    for (int r = sub; r < rows; r += at_once) {
        int64_t pos = s_pos[r];                       // negative: padding, the row stays as it was
        if (p.rot_dim > 0 && pos >= p.max_pos) {
            if (p.status) atomicExch(p.status, MQ_ERR_INVALID_ARG);
            pos = -1;
        }
        if (pos < 0) continue;
        CosSin cs;
        if (at.rotated[0]) load_cos_sin<INTERLEAVED>(p.rope + pos * p.rot_dim, at, p.rot_dim >> 1, cs);
        for (int h = h0; h < p.q_heads; h += WALK * per_row) {
            if (r != sub || h != h0) load(r, h);
#pragma unroll
            for (int i = 0; i < WALK; ++i) {
                if (h + i * per_row >= p.q_heads) continue;
                if (at.rotated[0]) {
                    float f[16];
                    unpack8(w[i][0], f);
                    unpack8(w[i][1], f + 8);
                    rotate<INTERLEAVED>(f, at, cs);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        w[i][e] = make_uint4(cvt_bf16x2(f[8 * e + 1], f[8 * e]), cvt_bf16x2(f[8 * e + 3], f[8 * e + 2]),
                                             cvt_bf16x2(f[8 * e + 5], f[8 * e + 4]), cvt_bf16x2(f[8 * e + 7], f[8 * e + 6]));
                }
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (MQ_CHECK(r0 + r < p.T))
                        *reinterpret_cast<uint4*>(p.q_out + ((r0 + r) * p.q_heads + h + i * per_row) * D + at.at[e]) = w[i][e];
            }
        }
    }
}

template <int D, int P, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS, 4) k_kv_append(Params p) {
    pdl_launch_dependents();
    pdl_wait();
    if ((int)blockIdx.x < p.kv_blocks)
        append_page<D, P, INTERLEAVED>(p, blockIdx.x);
    else
        rotate_q<D, INTERLEAVED>(p, blockIdx.x - p.kv_blocks);
}

MQ_DEBUG_READER(debug_hits_kv_append)

template <int D, int P, bool INTERLEAVED>
cudaError_t launch(const Params& p, int64_t blocks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    int nattr = 0;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    set_pdl_attr(attr, &nattr);
    cfg.attrs = attr;
    cfg.numAttrs = nattr;
    return cudaLaunchKernelEx(&cfg, k_kv_append<D, P, INTERLEAVED>, p);
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
    const int64_t pages = a.T / c.page_size + 2 * (int64_t)s.batch;
    p.by_row = a.T <= pages;
    const int64_t slots = p.by_row ? a.T : pages;
    const int heads = std::max(1, THREADS / (c.page_size * (c.head_dim / 16)));        // Part::HEADS
    const int64_t kv_blocks = slots * ((c.kv_heads + heads - 1) / heads);
    // two rows of Q per block while the rows are few (latency), eight once they fill the device
    p.q_rows = a.T >= 2048 ? Q_ROWS_MAX : 2;
    const int64_t q_blocks = (a.T + p.q_rows - 1) / p.q_rows;
    if (kv_blocks + q_blocks > 0x7fffffff) return cudaErrorInvalidValue;
    p.kv_blocks = (int)kv_blocks;
    const int64_t blocks = kv_blocks + q_blocks;
#define MQ_KV_APPEND(D_, P_) \
    if (c.head_dim == D_ && c.page_size == P_) \
        return a.interleaved ? launch<D_, P_, true>(p, blocks, stream) : launch<D_, P_, false>(p, blocks, stream);
    MQ_KV_APPEND(64, 16) MQ_KV_APPEND(64, 32) MQ_KV_APPEND(64, 64) MQ_KV_APPEND(64, 128)
    MQ_KV_APPEND(128, 16) MQ_KV_APPEND(128, 32) MQ_KV_APPEND(128, 64) MQ_KV_APPEND(128, 128)
#undef MQ_KV_APPEND
    return cudaErrorInvalidValue;
}

}  // namespace mq
