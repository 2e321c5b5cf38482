// mq_kv_attention.cu -- softmax attention of a batch's new tokens over the
// paged E4M3 cache (mq_kv_attention): the form for few rows per kv head.
//
// Mathematics.  For a row with query q and the keys j <= its position, with
// page exponents ek, ev of key j's page and codes ck_j, cv_j:
//     u_j = scale * log2(e) * 2^ek * (q . ck_j) + ev
//     out = sum_j 2^(u_j - M) cv_j / sum_j 2^(u_j - M) 2^(-ev)
// i.e. V's scale goes into the exponent, so the weights of the product with
// V's codes are at most 2^8 (M follows the running maximum of u, and is moved
// only when a weight would pass 2^8), and the denominator takes the scale out
// again.  Every factor 2^e is exact.  E4M3 codes are exact in f16, and q goes
// to f16 after division by its row's power of two, which loses nothing above
// 2^-38 of the row's maximum; so the f16 products are those of the exact
// operands, and the one rounding is that of the weights to f16 (2^-12).
// Scores, weights, sums and outputs are held in binary32.  A weight below 2^-126
// is zero: a key is lost, from the denominator too, where 2^(u_j) is less than
// 2^-118 of the row's largest (6 + 8 bits of room above the maximum); with V's
// page scales within 2^100 of one another that is a key of no weight.
//
// Bound: the cache is read once per kv head (2 D bytes per token), at HBM
// rate: 64 sequences of up to 8K tokens, 32 / 8 heads of 128, 106 us (4.8 TB/s,
// 0.73 of the measured copy), 4 of 131K 197 to 207 us (box to box, 5.2 to 5.4
// TB/s); at D = 64 the instructions per byte double, 3.0 TB/s.  One sequence of
// 4K takes 12 us, most of it the chain of dependent loads (lengths, page, codes)
// and the join.  A warp takes 16 tokens at a time straight from global memory
// into the fragments of mma.m16n8k16: K's codes as the left operand (tokens x
// d), V's as the left operand of the second product (d x tokens); the order of
// d inside a fragment is free, so each lane loads 16 consecutive bytes of a
// token.  The transposition of the weights between the two products is one
// movmatrix per 8 x 8.  Nothing goes through shared memory but the merge of
// the warps' partial results.
#include <cuda_bf16.h>
#include <cuda_fp16.h>


#include "mq_debug.cuh"
#include "mq_kv.cuh"
#include "mq_kv_internal.h"
#include "mq_kv_plan.h"
#include "mq_ptx.cuh"

namespace mq {
namespace kv_attend {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int STEP = 16;                 // tokens of one warp step
constexpr float LAZY = 8.f;              // M moves when a weight would pass 2^LAZY
constexpr float BIAS = 6.f;              // weights are held times 2^BIAS: 2^14 at most, f16 holds 2^16

using Params = KvAttendParams;

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16(float hi, float lo) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// 16 or 8 bytes of codes, streamed: the cache is larger than L2 in earnest (a
// plain load: the append before it may still have been writing when this grid began)
template <int N>
__device__ __forceinline__ void load_codes(uint32_t (&w)[N], const uint8_t* p) {
    if constexpr (N == 4) {
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
    } else {
        asm volatile("ld.global.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(THREADS, NT == 1 ? (D == 64 ? 5 : 4) : (D == 64 ? 4 : 3)) k_kv_attend(Params p) {
    constexpr int ROWS = 8 * NT;
    constexpr int KH = D / 64;               // 16-byte pieces of a K row per lane
    constexpr int VW = D / 32;               // words of a V row per lane
    constexpr int MT = D / 16;               // 16-wide slices of d
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    pdl_wait();

    // chunk fastest, then kv head, row tile (last rows first: they see most), sequence
    int id = blockIdx.x;
    const int chunk = id % p.chunks;
    id /= p.chunks;
    const int head = id % p.kv_heads;
    id /= p.kv_heads;
    const int tile = p.row_tiles - 1 - id % p.row_tiles, b = id / p.row_tiles;
    const int c0 = p.cu[b], n = p.cu[b + 1] - c0;
    const int64_t len = max(p.lens[b], 0);
    const int page_tokens = 1 << p.page_log2;
    if (n <= 0) return;
    // lengths that the call's arguments or the table do not cover: the rows stay as they were
    if (c0 < 0 || (int64_t)c0 + n > p.T || n > p.max_q || len > p.max_len || len > p.max_pages << p.page_log2) {
        if (tid == 0 && p.status) atomicExch(p.status, MQ_ERR_INVALID_ARG);
        return;
    }
    // positions and rows stay below 2^31 - 2^16 (checked by the entry point)
    const int rows = n * p.group, row0 = tile * ROWS;
    if (row0 >= rows) return;
    const int start = (int)len - n;                             // position of the first new token
    const int last_row = min(rows, row0 + ROWS) - 1;
    const int end = max(0, min((int)len, start + last_row / p.group + 1));   // keys that some row sees
    const int chunks = max(1, (int)(((int64_t)end + p.chunk_tokens - 1) / p.chunk_tokens));
    if (chunk >= chunks) return;
    const int k0 = chunk * p.chunk_tokens, k1 = (int)min((int64_t)end, (int64_t)k0 + p.chunk_tokens);
    const int sees_all = start + row0 / p.group;                // keys up to this position: every row sees them

    // The warp's steps of 16 keys: the page of the step after the next is
    // looked up while the codes and scales of the next are on their way.
    const int* table = p.table + (int64_t)b * p.max_pages;
    auto page_of = [&](int tok0) { return tok0 < k1 ? table[tok0 >> p.page_log2] : -1; };
    int page = page_of(k0 + warp * STEP);

    // Q: row g of each n-tile, the d that the K fragments hold: 16 t .. 16 t + 15 (+ 64)
    uint32_t qf[NT][4 * KH][2];
    float fac[NT][2];                        // scale * log2(e) * 2^(row's exponent) of rows 2t, 2t + 1
    int pos[NT][2];                          // their positions (-1: no row)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = row0 + nt * 8 + g;
        float x[KH][16];
        float top = 0.f;
#pragma unroll
        for (int h = 0; h < KH; ++h) {
            uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            if (r < rows) {
                const uint4* src = reinterpret_cast<const uint4*>(
                    p.q + (int64_t)(c0 + r / p.group) * p.q_stride + (int64_t)(head * p.group + r % p.group) * D +
                    h * 64 + t * 16);
                w[0] = src[0];
                w[1] = src[1];
            }
            const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[h][2 * i] = __uint_as_float(u[i] << 16);
                x[h][2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
                top = fmaxf(top, fmaxf(fabsf(x[h][2 * i]), fabsf(x[h][2 * i + 1])));
            }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // to a maximum in [2^13, 2^14): the power of two comes back in `fac`
        const int e = max(-100, (int)(__float_as_uint(top) >> 23) - 127) - 13;
        const float down = exp2i(-e), up = exp2i(e);
#pragma unroll
        for (int h = 0; h < KH; ++h)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                qf[nt][4 * h + s][0] = pack_f16(x[h][4 * s + 1] * down, x[h][4 * s] * down);
                qf[nt][4 * h + s][1] = pack_f16(x[h][4 * s + 3] * down, x[h][4 * s + 2] * down);
            }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int ri = row0 + nt * 8 + 2 * t + i;
            fac[nt][i] = p.scale_log2 * __shfl_sync(0xffffffffu, up, (2 * t + i) * 4);
            pos[nt][i] = ri < rows ? start + ri / p.group : -1;
        }
    }

    float o[NT][MT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nt][j][i] = 0.f;
    }

    uint32_t kw[2][KH][4], vw[4][VW];
    float sk = 0.f, sv = 1.f;                // the pages' scales of the step whose codes are on their way
    bool valid = false;
    int64_t base = 0;                        // byte offset of its first code
    [[maybe_unused]] const int64_t pool = (p.num_pages * p.kv_heads << p.page_log2) * D;
    auto load_k = [&](int tok0) {
        valid = page >= 0 && page < p.num_pages;
        if (!valid && p.status && lane == 0) atomicExch(p.status, MQ_ERR_INVALID_ARG);
        const int64_t cell = valid ? (int64_t)page * p.kv_heads + head : 0;
        base = ((cell << p.page_log2) + (tok0 & (page_tokens - 1))) * D;
        sk = p.k_scales[cell];
        sv = p.v_scales[cell];
        const uint8_t* src = p.k_codes + base + g * D + t * 16;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < KH; ++h) {
                if (MQ_CHECK(base + (g + 8 * i) * D + h * 64 + t * 16 + 16 <= pool)) load_codes(kw[i][h], src + i * 8 * D + h * 64);
            }
        page = page_of(tok0 + WARPS * STEP);
    };
    auto load_v = [&](int tok0) {
        const uint8_t* src = p.v_codes + base + 2 * t * D + g * (VW * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (MQ_CHECK(base + (2 * t + (i & 1) + 8 * (i >> 1)) * D + (g + 1) * (VW * 4) <= pool))
                load_codes(vw[i], src + ((i & 1) + 8 * (i >> 1)) * D);
        if (tok0 + STEP > k1 || !valid) {
            // behind the last token a page holds whatever was there, and so does
            // the pool's first page in place of one that is none: a NaN code
            // times a zero weight is no zero
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (tok0 + 2 * t + (i & 1) + 8 * (i >> 1) >= k1 || !valid) {
#pragma unroll
                    for (int w = 0; w < VW; ++w) vw[i][w] = 0;
                }
        }
    };

    int tok0 = k0 + warp * STEP;
    if (tok0 < k1) {
        load_k(tok0);
        load_v(tok0);
    }
    for (; tok0 < k1; tok0 += WARPS * STEP) {
        const int next = tok0 + WARPS * STEP;
        const float ck = sk, ev = (float)((int)(__float_as_uint(sv) >> 23) - 127);
        const float iev = __uint_as_float((254u << 23) - (__float_as_uint(sv) & 0x7F800000u));
        const bool here = valid;
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int h = 0; h < KH; ++h)
#pragma unroll
            for (int st = 0; st < 4; ++st) {
                const uint32_t a[4] = {cvt_e4m3x2_to_f16x2((uint16_t)kw[0][h][st]), cvt_e4m3x2_to_f16x2((uint16_t)kw[1][h][st]),
                                       cvt_e4m3x2_to_f16x2((uint16_t)(kw[0][h][st] >> 16)),
                                       cvt_e4m3x2_to_f16x2((uint16_t)(kw[1][h][st] >> 16))};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(s[nt], a, qf[nt][4 * h + st][0], qf[nt][4 * h + st][1]);
            }
        if (next < k1) load_k(next);

        // s[nt]: tokens g (0, 1) and g + 8 (2, 3), rows 2t and 2t + 1
        const bool masked = tok0 + STEP - 1 > sees_all || !here;
        bool higher = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float u = __fmaf_rn(s[nt][i], fac[nt][i & 1] * ck, ev);
                if (masked) {
                    const int at = tok0 + g + 8 * (i >> 1);
                    u = at <= pos[nt][i & 1] && at < k1 && here ? u : -INFINITY;
                }
                s[nt][i] = u;
                higher |= u > m[nt][i & 1] + LAZY;
            }
        }
        if (__any_sync(0xffffffffu, higher)) {
            // move the maxima: over the 8 lanes that hold a row's tokens
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float top = fmaxf(m[nt][i], fmaxf(s[nt][i], s[nt][i + 2]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    const float f = top > m[nt][i] ? ex2(m[nt][i] - top) : 1.f;     // m = -inf: nothing to keep
                    m[nt][i] = top;
                    l[nt][i] *= f;
#pragma unroll
                    for (int j = 0; j < MT; ++j) {
                        o[nt][j][i] *= f;
                        o[nt][j][i + 2] *= f;
                    }
                }
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float mm = m[nt][i & 1] == -INFINITY ? 0.f : m[nt][i & 1];
                w[i] = ex2(s[nt][i] - mm + BIAS);
                l[nt][i & 1] = __fmaf_rn(w[i], iev, l[nt][i & 1]);
            }
            pf[nt][0] = movmatrix(pack_f16(w[1], w[0]));
            pf[nt][1] = movmatrix(pack_f16(w[3], w[2]));
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            // d = g D/8 + 2 j and + 1: two bytes of each of the four tokens' pieces
            const uint32_t sel = j & 1 ? 0x7362u : 0x5140u;
            const uint32_t a01 = __byte_perm(vw[0][j >> 1], vw[1][j >> 1], sel);
            const uint32_t a23 = __byte_perm(vw[2][j >> 1], vw[3][j >> 1], sel);
            const uint32_t a[4] = {cvt_e4m3x2_to_f16x2((uint16_t)a01), cvt_e4m3x2_to_f16x2((uint16_t)(a01 >> 16)),
                                   cvt_e4m3x2_to_f16x2((uint16_t)a23), cvt_e4m3x2_to_f16x2((uint16_t)(a23 >> 16))};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][j], a, pf[nt][0], pf[nt][1]);
        }
        if (next < k1) load_v(next);
    }

    // ---- merge the warps: lane (g, t) holds rows 8 nt + 2 t and + 1, d = g D/8 ...
    float* mm = reinterpret_cast<float*>(smem);                // [WARPS][ROWS]
    float* ll = mm + WARPS * ROWS;                             // [WARPS][ROWS]
    float* oo = ll + WARPS * ROWS;                             // [WARPS][ROWS][D]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float sum = l[nt][i];
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            const int r = nt * 8 + 2 * t + i;
            if (g == 0) {
                mm[warp * ROWS + r] = m[nt][i];
                ll[warp * ROWS + r] = sum;
            }
            float* dst = oo + ((size_t)warp * ROWS + r) * D + g * (D / 8);
#pragma unroll
            for (int j = 0; j < MT; ++j) *reinterpret_cast<float2*>(dst + 2 * j) = make_float2(o[nt][j][i], o[nt][j][i + 2]);
        }
    __syncthreads();
    constexpr int V4 = D / 4;
    const int64_t cell = ((int64_t)b * p.row_tiles + tile) * p.kv_heads + head;
    float* part = p.part ? p.part + cell * p.chunks * (int64_t)(ROWS * (D + 2)) : nullptr;
    const int nrows = last_row - row0 + 1;
    for (int i = tid; i < nrows * V4; i += THREADS) {
        const int r = i / V4, c4 = i % V4;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) top = fmaxf(top, mm[w * ROWS + r]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float lsum = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float mw = mm[w * ROWS + r];
            const float f = mw == -INFINITY ? 0.f : ex2(mw - top);
            const float4 v = *reinterpret_cast<const float4*>(oo + ((size_t)w * ROWS + r) * D + c4 * 4);
            acc.x = __fmaf_rn(v.x, f, acc.x);
            acc.y = __fmaf_rn(v.y, f, acc.y);
            acc.z = __fmaf_rn(v.z, f, acc.z);
            acc.w = __fmaf_rn(v.w, f, acc.w);
            lsum = __fmaf_rn(ll[w * ROWS + r], f, lsum);
        }
        if (chunks == 1) {
            kv_write_out<D>(p, c0, row0 + r, head, c4, acc, lsum);
        } else {
            *reinterpret_cast<float4*>(part + ((int64_t)chunk * ROWS + r) * D + c4 * 4) = acc;
            if (c4 == 0)
                reinterpret_cast<float2*>(kv_part_ml<D>(p, part, ROWS))[chunk * ROWS + r] = make_float2(top, lsum);
        }
    }
    if (chunks == 1) return;
    // ---- the last chunk to finish joins them, in chunk order
    __shared__ int s_last;
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        const int done = atomicAdd(p.tickets + cell, 1);
        s_last = done == chunks - 1;
        if (s_last) p.tickets[cell] = 0;                        // as it was found
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    kv_join<D>(p, part, chunks, ROWS, nrows, c0, row0, head, tid, THREADS, reinterpret_cast<float*>(smem));
}

MQ_DEBUG_READER(debug_hits_kv_attend)

template <int D, int NT>
cudaError_t launch(const Params& p, int64_t blocks, cudaStream_t stream) {
    constexpr int SMEM = WARPS * 8 * NT * (D + 2) * 4;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    const int d = dev < 64 ? dev : 63;
    if (!attr_set[d]) {
        cudaError_t e = cudaFuncSetAttribute(k_kv_attend<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        attr_set[d] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    int nattr = 0;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = stream;
    set_pdl_attr(attr, &nattr);
    cfg.attrs = attr;
    cfg.numAttrs = nattr;
    return cudaLaunchKernelEx(&cfg, k_kv_attend<D, NT>, p);
}

}  // namespace kv_attend

// ---------------------------------------------------------------- host side
cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t stream) {
    using namespace kv_attend;
    const mq_kv_cache& c = *a.cache;
    const mq_kv_batch& s = *a.batch;
    const KvPlan plan = kv_plan(s.batch, a.q_heads, c.kv_heads, c.head_dim, a.max_q, a.max_len);
    Params p{};
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.cu = s.cu_rows;
    p.lens = s.lens;
    p.table = s.page_table;
    p.k_codes = c.k_codes;
    p.v_codes = c.v_codes;
    p.k_scales = c.k_scales;
    p.v_scales = c.v_scales;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    p.status = reinterpret_cast<int*>(ws) + WS_STATUS;
    p.tickets = reinterpret_cast<int*>(ws + plan.tickets_off);
    p.part = plan.chunks > 1 ? reinterpret_cast<float*>(ws + plan.part_off) : nullptr;
    p.T = a.T;
    p.q_stride = a.q_row_stride;
    p.num_pages = c.num_pages;
    p.max_pages = s.max_pages;
    p.max_len = a.max_len;
    p.batch = s.batch;
    p.q_heads = a.q_heads;
    p.kv_heads = c.kv_heads;
    p.group = a.q_heads / c.kv_heads;
    p.page_log2 = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
    p.max_q = (int)a.max_q;
    p.row_tiles = (int)plan.row_tiles;
    p.chunks = (int)plan.chunks;
    p.chunk_tokens = (int)plan.chunk_tokens;
    p.by_length = plan.by_length;
    p.scale_log2 = a.scale * 1.44269504088896340736f;
    const int64_t blocks = plan.cells * plan.chunks;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    if (plan.prefill) return launch_kv_prefill(p, c.head_dim, blocks, stream);
#define MQ_KV_ATTEND(D_, NT_) \
    if (c.head_dim == D_ && plan.nt == NT_) return launch<D_, NT_>(p, blocks, stream);
    MQ_KV_ATTEND(64, 1) MQ_KV_ATTEND(64, 2)
    MQ_KV_ATTEND(128, 1) MQ_KV_ATTEND(128, 2)
#undef MQ_KV_ATTEND
    return cudaErrorInvalidValue;
}

}  // namespace mq
