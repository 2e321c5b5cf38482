// mq_kv_prefill.cu -- the attention of mq_kv_attention where a kv head has many
// rows (prompts and chunks of them): tcgen05 form, 256 rows per CTA.
//
// The mathematics is that of mq_kv_attention.cu: scores u = scale log2(e) 2^ek
// (q . ck) + ev, weights 2^(u - M) in f16, V's codes in f16, the denominator
// without ev.  Codes are exact in f16, so both products are kind::f16 with the
// exact operands and binary32 accumulators in tensor memory.
//
// A CTA holds two tiles of 128 rows (rows = new token x head of the group, so
// the heads of a group share K and V) and walks the keys in blocks of 128:
//   warps 0-3, 4-7   softmax of tile 0 and 1: a thread owns a row.  It reads
//                    the row's scores from tensor memory, moves the maximum M
//                    only when a weight would pass 2^8 (then rescales its row
//                    of O there), and writes the weights over the scores, as
//                    the left operand of the second product
//   warps 8-11       converters: E4M3 codes from global memory to f16 in shared
//                    memory (128-byte swizzle), one block ahead in registers
//   warp 13          looks up the pages and scales of the blocks to come; a group
//                    of 16 keys without a page is read from zeros and gets no
//                    weight (addresses from here on: zeroing in the converters
//                    cost 3% of a prompt's time, they are short of registers)
//   warp 12          issues the products: S_t = Q_t K^T, then O_t += P_t V, the
//                    two tiles alternating, so that one tile's softmax runs
//                    under the other's products
// V needs no transposition: [token][d] is the MN-major right operand.
//
// Bound: per block and CTA the two tiles' products take 2048 cycles of the
// tensor pipe at D = 128 and their 32768 exponentials 2048 cycles of the SFU;
// a tile's own chain (products 1420 cycles, scores and maximum 550, weights
// 1750, hand-overs) is ~4000, and two tiles in turn leave either pipe about
// half idle: 8192-token prompt, 32 heads of 128: 0.60 ms, 920 TFLOP/s.
// Measured against this form and dropped (same prompt): two threads per row
// (0.69 ms), the weights under the last block's maximum, computed again where it
// rose (0.65 ms), an issuer of its own for each tile (0.73 ms; 0.63 ms with the
// tiles taking turns), Q in tensor memory at D = 64 (3% slower).  With neither
// softmax nor conversions the products run at 2050 cycles per block, with the
// conversions at 3350: the converters' stores and the tensor pipe's reads share
// the bandwidth of shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "mq_debug.cuh"
#include "mq_kv.cuh"
#include "mq_kv_internal.h"
#include "mq_kv_plan.h"
#include "mq_ptx.cuh"

namespace mq {
namespace kv_prefill {

constexpr int TILE = 128;                       // rows per tile
constexpr int ROWS = 2 * TILE;
constexpr int BLOCK = 128;                      // keys per block
constexpr int GROUPS = BLOCK / 16;              // a page holds whole groups of 16 keys
constexpr int CONV_WARP = 8, MMA_WARP = 12, TABLE_WARP = 13;
constexpr int THREADS = 16 * 32;               // four warpgroups (warps 14 and 15 only hand back registers)
constexpr int STAGES = 2;                       // of K and of V
constexpr int TABLES = 4;                       // of the blocks' pages and their scales
constexpr float LAZY = 8.f, BIAS = 6.f;         // as in mq_kv_attention.cu
constexpr float FACTOR_MIN = 1.17549435e-38f;   // 2^-126
constexpr long long TIMEOUT_CYCLES = 4000000000LL;

struct Smem {
    uint64_t q_full, k_full[STAGES], k_empty[STAGES], v_full[STAGES], v_empty[STAGES];
    uint64_t s_full[2], p_full[2], o_full[2], t_full[TABLES], t_empty[TABLES], drained;
    const uint8_t* k_at[TABLES][GROUPS];        // a group's codes in the pool; g_zeros where it has no page
    const uint8_t* v_at[TABLES][GROUPS];
    float ck[TABLES][GROUPS], ev[TABLES][GROUPS], iev[TABLES][GROUPS];
    uint32_t tmem_base;
    int abort_flag;
    int last;
    int seq, tile;                              // by_length
};

// What a group without a page is read from: zeros (what the pool holds in its
// place may be a NaN code, which times a zero weight is no zero).
__device__ uint4 g_zeros[16 * 128 / 16];

template <int D>
struct Layout {
    static constexpr int HALVES = D / 64;                    // 64 f16 = one 128-byte swizzle row
    static constexpr int TILE_BYTES = 128 * D * 2;           // 128 rows of Q, K or V
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = 2 * TILE_BYTES;
    static constexpr int V_OFF = K_OFF + STAGES * TILE_BYTES;
    static constexpr int BYTES = V_OFF + STAGES * TILE_BYTES + 1024;
    // more than half of the SM's shared memory, whatever D: tensor memory is
    // allocated whole, so two CTAs of an SM would only wait for one another
    static constexpr int SMEM = BYTES > 120 * 1024 ? BYTES : 120 * 1024;
    static constexpr uint32_t S_COL = 0, O_COL = 256;
};

__device__ __forceinline__ uint32_t pack_f16(float hi, float lo) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// The products of one block, K = 16 per instruction, issued as one sequence:
// operands by the low words of their shared-memory descriptors (in 16 bytes)
// or their tensor-memory columns, the offsets of the steps as immediates, so
// that the issuing lane keeps no table of descriptors.
//   S = Q K^T: steps of 32 bytes inside the 128-byte swizzle row, then the next 64 d
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t hi) {
#define MQ_STEP(off, p) \
    "add.u32 ra, %1, " off ";\n\tadd.u32 rb, %2, " off ";\n\tmov.b64 da, {ra, %4};\n\tmov.b64 db, {rb, %4};\n\t" \
    "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, " p ";\n\t"
    if constexpr (D == 128) {
        asm volatile(
            "{\n\t.reg .pred f, t;\n\t.reg .b32 ra, rb;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
            MQ_STEP("0", "f") MQ_STEP("2", "t") MQ_STEP("4", "t") MQ_STEP("6", "t")
            MQ_STEP("1024", "t") MQ_STEP("1026", "t") MQ_STEP("1028", "t") MQ_STEP("1030", "t")
            "}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(hi) : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred f, t;\n\t.reg .b32 ra, rb;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
            MQ_STEP("0", "f") MQ_STEP("2", "t") MQ_STEP("4", "t") MQ_STEP("6", "t")
            "}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(hi) : "memory");
    }
#undef MQ_STEP
}
//   O (+)= P V: 8 columns of P and 16 tokens (2048 bytes) of V per step
__device__ __forceinline__ void mma_outputs(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t hi, uint32_t acc) {
#define MQ_STEP(aoff, boff, p) \
    "add.u32 ra, %1, " aoff ";\n\tadd.u32 rb, %2, " boff ";\n\tmov.b64 db, {rb, %4};\n\t" \
    "tcgen05.mma.cta_group::1.kind::f16 [%0], [ra], db, %3, " p ";\n\t"
    asm volatile(
        "{\n\t.reg .pred f, t;\n\t.reg .b32 ra, rb;\n\t.reg .b64 db;\n\tsetp.ne.b32 f, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        MQ_STEP("0", "0", "f") MQ_STEP("8", "128", "t") MQ_STEP("16", "256", "t") MQ_STEP("24", "384", "t")
        MQ_STEP("32", "512", "t") MQ_STEP("40", "640", "t") MQ_STEP("48", "768", "t") MQ_STEP("56", "896", "t")
        "}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(hi), "r"(acc) : "memory");
#undef MQ_STEP
}
// ex2 that keeps its place among the other volatile instructions
__device__ __forceinline__ float ex2v(float x) {
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^x of a pair, x <= 120, on the FMA pipe: x = i + f with i the nearest integer
// (it appears in the low bits of x + 1.5 * 2^23), 2^f = 1 + f (c1 + f (c2 + f (c3 + f c4)))
// with coefficients fitted here to the least largest relative error on
// [-1/2, 1/2], 2^-18.4; i goes into the exponent.  Below 2^-126 the result
// runs out towards 0, which it is from -127 on (-inf too).  Of a NaN it makes a
// number: the row's sum has it from the maximum.
__device__ __forceinline__ void exp2_pair(float& x, float& y) {
    const uint64_t v = pack2(fmaxf(x, -127.f), fmaxf(y, -127.f));
    const uint64_t t = add2(v, pack2(12582912.f, 12582912.f));
    const uint64_t f = fma2(add2(t, pack2(-12582912.f, -12582912.f)), pack2(-1.f, -1.f), v);
    uint64_t q = fma2(f, pack2(0x1.3a02ccp-7f, 0x1.3a02ccp-7f), pack2(0x1.c9fc46p-5f, 0x1.c9fc46p-5f));
    q = fma2(f, q, pack2(0x1.ec0378p-3f, 0x1.ec0378p-3f));
    q = fma2(f, q, pack2(0x1.62e12cp-1f, 0x1.62e12cp-1f));
    q = fma2(f, q, pack2(1.f, 1.f));
    float a, b, c, d;
    unpack2(t, a, b);
    unpack2(q, c, d);
    x = __uint_as_float(__float_as_uint(c) + (__float_as_uint(a) << 23));
    y = __uint_as_float(__float_as_uint(d) + (__float_as_uint(b) << 23));
}
// the larger, a NaN before all others
__device__ __forceinline__ float max2(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max3(uint32_t a, uint32_t b, uint32_t c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return r;
}
__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// The row tiles of the whole batch in the order of the keys they see (in units
// of 64), most first, so that the last blocks to start are short ones: warp 0
// finds tile `job` of that order.  A sequence's tiles from tmin(v) on see 64 v
// keys or more; a search over v with a sum over the batch gives the v of tile
// `job`.  N: sequences per lane.
template <int N>
__device__ __forceinline__ void by_length(const KvAttendParams& p, int job, Smem* s) {
    const int lane = threadIdx.x % 32;
    int start[N], len[N], own[N], longest = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int b = lane + 32 * i;
        start[i] = len[i] = own[i] = 0;
        if (b < p.batch) {
            const int64_t c0 = p.cu[b], n = p.cu[b + 1] - c0;
            const int l = max(p.lens[b], 0);
            if (n <= 0) continue;
            own[i] = 1;                                      // of a sequence that is refused: the block that reports it
            if (c0 < 0 || c0 + n > p.T || n > p.max_q || l > p.max_len || l > p.max_pages << p.page_log2) continue;
            own[i] = (int)((n * p.group + ROWS - 1) / ROWS);
            start[i] = l - (int)n;
            len[i] = l;
            longest = max(longest, l);
        }
    }
    if (lane == 0) s->seq = -1;
    __syncwarp();
    // sequences alike need no search
    const int own0 = __shfl_sync(0xffffffffu, own[0], 0), len0 = __shfl_sync(0xffffffffu, len[0], 0);
    bool alike = true;
#pragma unroll
    for (int i = 0; i < N; ++i) alike = alike && (lane + 32 * i >= p.batch || (own[i] == own0 && len[i] == len0));
    if (__all_sync(0xffffffffu, alike)) {
        if (lane == 0 && job / p.batch < own0) {
            s->seq = job % p.batch;
            s->tile = own0 - 1 - job / p.batch;
        }
        return;
    }
    auto tmin = [&](int i, int v) {
        return v <= 0 ? 0 : v > len[i] >> 6 ? own[i] : max(0, (v << 6) - 1 - start[i]) * p.group / ROWS;
    };
    auto count = [&](int v) {
        int sum = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) sum += own[i] - tmin(i, v);
        return __reduce_add_sync(0xffffffffu, sum);
    };
    int lo = 0, hi = (__reduce_max_sync(0xffffffffu, longest) >> 6) + 1;
    if (count(0) <= job) return;                             // no such tile
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (count(mid) > job)
            lo = mid;
        else
            hi = mid;
    }
    int left = job - count(hi);                              // among the tiles that see 64 lo .. 64 lo + 63 keys
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int first = tmin(i, lo), mine = tmin(i, hi) - first;
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        if (left >= upto - mine && left < upto) {
            s->seq = lane + 32 * i;
            s->tile = first + left - (upto - mine);
        }
        left -= __shfl_sync(0xffffffffu, upto, 31);
    }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1) k_kv_prefill(KvAttendParams p) {
    using L = Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ Smem sm;
    Smem* s = &sm;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    pdl_launch_dependents();
    pdl_wait();

    // chunk fastest, then kv head, sequence; the last row tiles (they see most)
    // first, those of a ragged batch by what they see
    int id = blockIdx.x;
    const int chunk = id % p.chunks;
    id /= p.chunks;
    const int head = id % p.kv_heads;
    id /= p.kv_heads;
    int b = id % p.batch, tile = p.row_tiles - 1 - id / p.batch;
    if (p.by_length) {
        if (warp == 0) {
            if (p.batch <= 32)
                by_length<1>(p, id, s);
            else
                by_length<KV_BY_LENGTH_MAX / 32>(p, id, s);
        }
        __syncthreads();
        b = s->seq;
        tile = s->tile;
        if (b < 0) return;
    }
    const int c0 = p.cu[b], n = p.cu[b + 1] - c0;
    const int64_t len = max(p.lens[b], 0);
    const int page_tokens = 1 << p.page_log2;
    if (n <= 0) return;
    if (c0 < 0 || (int64_t)c0 + n > p.T || n > p.max_q || len > p.max_len || len > p.max_pages << p.page_log2) {
        if (tid == 0 && p.status) atomicExch(p.status, MQ_ERR_INVALID_ARG);
        return;
    }
    // positions and rows stay below 2^31 - 2^16 (checked by the entry point)
    const int rows = n * p.group, row0 = tile * ROWS;
    if (row0 >= rows) return;
    const int start = (int)len - n;
    const int last_row = min(rows, row0 + ROWS) - 1;
    const int end = max(0, min((int)len, start + last_row / p.group + 1));
    const int chunks = max(1, (int)(((int64_t)end + p.chunk_tokens - 1) / p.chunk_tokens));
    if (chunk >= chunks) return;
    const int k0 = chunk * p.chunk_tokens, k1 = (int)min((int64_t)end, (int64_t)k0 + p.chunk_tokens);
    const int blocks = k1 > k0 ? (k1 - k0 + BLOCK - 1) / BLOCK : 0;
    const bool two = row0 + TILE < rows;                     // the second tile has rows

    if (tid == 0) {
        mbar_init(&s->q_full, 8);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&s->k_full[i], 4);
            mbar_init(&s->v_full[i], 4);
            mbar_init(&s->k_empty[i], 1);
            mbar_init(&s->v_empty[i], 1);
        }
        for (int i = 0; i < TABLES; ++i) {
            mbar_init(&s->t_full[i], 1);
            mbar_init(&s->t_empty[i], two ? 12 : 8);
        }
        mbar_init(&s->drained, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->s_full[i], 1);
            mbar_init(&s->p_full[i], 4);
            mbar_init(&s->o_full[i], 1);
        }
        s->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == MMA_WARP) {
        tmem_alloc(&s->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s->tmem_base;
    const uint32_t sbase = smem_u32(base);
    const volatile int* abort_flag = &s->abort_flag;
    auto raise = [&]() {
        *(volatile int*)&s->abort_flag = 1;
        if (p.status) atomicExch(p.status, MQ_ERR_TIMEOUT);
    };
    // all lanes wait; false (for the whole warp) once a wait has run out
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, TIMEOUT_CYCLES, abort_flag));
        if (!ok && lane == 0) raise();
        return ok;
    };

    // 512 threads start with 128 registers each; the softmax warpgroups take
    // what the others leave: 2 x 176 + 80 + 80 = 4 x 128
    if (warp < CONV_WARP)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    else if (warp < MMA_WARP)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");

    float m = -INFINITY, l = 0.f;                            // softmax threads: their row's
    if (blocks == 0) {
        // a chunk without keys (rows of padding): nothing to add up
    } else if (warp < CONV_WARP) {
        // ------------------------------------------------------------ softmax
        const int t = warp / 4;                              // tile
        const int r = tid % TILE;                            // row of the tile
        const int row = row0 + t * TILE + r;
        const bool mine = row < rows;
        float fac = 0.f;
        int pos = -1;
        {
            uint4 w[D / 8];
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) w[i] = make_uint4(0, 0, 0, 0);
            if (mine) {
                pos = start + row / p.group;
                const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)(c0 + row / p.group) * p.q_stride +
                                                                  (head * p.group + row % p.group) * D);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) w[i] = src[i];
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xFFFF0000u))));
            }
            const int e = max(-100, (int)(__float_as_uint(top) >> 23) - 127) - 13;
            const float down = exp2i(-e);
            fac = p.scale_log2 * exp2i(e);
            const uint32_t qrow = sbase + L::Q_OFF + t * L::TILE_BYTES + r * 128;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    h[j] = pack_f16(__uint_as_float(u[j] & 0xFFFF0000u) * down, __uint_as_float(u[j] << 16) * down);
                st_shared_v4(qrow + (i / 8) * (TILE * 128) + (((i & 7) ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s->q_full);
        }
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lanes + L::S_COL + t * BLOCK;
        const uint32_t o_addr = tmem + lanes + L::O_COL + t * D;
        const int sees_all = start + (row0 + t * TILE) / p.group;     // keys every row of the tile sees
        if (t == 0 || two) {
            for (int j = 0; j < blocks; ++j) {
                const int kb = k0 + j * BLOCK;
                if (!wait(&s->t_full[j % TABLES], (j / TABLES) & 1) || !wait(&s->s_full[t], j & 1)) break;
                tc_fence_after();
                const bool masked = kb + BLOCK - 1 > min(sees_all, k1 - 1);
                if (masked) {
                    const int limit = min(pos, k1 - 1) - kb;     // last key of the block the row sees
#pragma unroll
                    for (int c = 0; c < BLOCK; c += 32) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(s_addr + c, v);
                        tmem_ld_wait_regs(v);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i > limit) v[i] = 0xFF800000u;                        // -inf
                        tmem_st_32x32b_x32(s_addr + c, v);
                    }
                    tmem_st_wait();
                }
                // the block's maximum
                float top = -INFINITY, fck[GROUPS], sh[GROUPS], iev[GROUPS];
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    // a factor of 0 would make NaN of -inf: it underflows only where the scores are 0 all the same
                    fck[g] = fmaxf(fac * s->ck[j % TABLES][g], FACTOR_MIN);
                    sh[g] = s->ev[j % TABLES][g];
                    iev[g] = s->iev[j % TABLES][g];
                }
                {
                    uint32_t v[2][32];
                    tmem_ld_32x32b_x32(s_addr, v[0]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        tmem_ld_wait_regs(v[c & 1]);
                        if (c < 3) tmem_ld_32x32b_x32(s_addr + 32 * (c + 1), v[1 - (c & 1)]);
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const uint32_t* x = v[c & 1] + 16 * g;
                            float g0 = max3(x[0], x[1], x[2]), g1 = max3(x[3], x[4], x[5]);
#pragma unroll
                            for (int i = 6; i < 14; i += 4) {
                                g0 = max3(__float_as_uint(g0), x[i], x[i + 1]);
                                g1 = max3(__float_as_uint(g1), x[i + 2], x[i + 3]);
                            }
                            g0 = max2(max3(__float_as_uint(g0), x[14], x[15]), g1);
                            top = max2(top, __fmaf_rn(g0, fck[2 * c + g], sh[2 * c + g]));
                        }
                    }
                }
                // A NaN among the scores the row sees, or an infinite one, is
                // a NaN in its sum from here on, and so in its output:
                // exp2_pair would make a number of it.
                if (!(top < INFINITY)) l = NAN;
                if (__any_sync(0xffffffffu, top > m + LAZY)) {
                    const float f = top > m + LAZY ? ex2(m - top) : 1.f;
                    if (top > m + LAZY) m = top;
                    l *= f;
                    if (j > 0) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16(o_addr + c, o);
                            tmem_ld_wait_regs16(o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st_32x32b_x16(o_addr + c, o);
                        }
                    }
                }
                // The weights, group by group: the exponentials of one beside
                // the sums and conversions of the one before (a result of the
                // SFU that is needed at once stalls the warp: 2514 -> 1329
                // cycles per 128 keys of a lone warp).
                const float shift = BIAS - (m == -INFINITY ? 0.f : m);
                uint32_t v[2][16];
                uint64_t u[2][8];
                float e[2][16];
                auto exponents = [&](int g) {
                    const uint32_t* x = v[g & 1];
                    tmem_ld_wait_regs16(v[g & 1]);
                    if (g + 1 < GROUPS) tmem_ld_32x32b_x16(s_addr + 16 * (g + 1), v[1 - (g & 1)]);
                    const uint64_t fck2 = pack2(fck[g], fck[g]), sh2 = pack2(sh[g] + shift, sh[g] + shift);
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[g & 1][i] = fma2(pack2u(x[2 * i], x[2 * i + 1]), fck2, sh2);
                };
                tmem_ld_32x32b_x16(s_addr, v[0]);
                exponents(0);
#pragma unroll
                for (int g = 0; g <= GROUPS; ++g) {
                    if (g < GROUPS) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float w0, w1;
                            unpack2(u[g & 1][i], w0, w1);
                            // D = 64: three pairs of eight on the FMA pipe (448 ->
                            // 425 us for an 8192-token prompt of 28 heads; at
                            // D = 128, where the products are longer, no gain)
                            if (D == 64 && (i == 1 || i == 4 || i == 6)) {
                                exp2_pair(w0, w1);
                            } else {
                                w0 = ex2v(w0);
                                w1 = ex2v(w1);
                            }
                            e[g & 1][2 * i] = w0;
                            e[g & 1][2 * i + 1] = w1;
                        }
                        if (g + 1 < GROUPS) exponents(g + 1);
                    }
                    if (g > 0) {
                        const float* w = e[1 - (g & 1)];
                        uint64_t sum = pack2(w[0], w[1]);
                        uint32_t h[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (i > 0) sum = add2(sum, pack2(w[2 * i], w[2 * i + 1]));
                            h[i] = pack_f16(w[2 * i + 1], w[2 * i]);
                        }
                        float w0, w1;
                        unpack2(sum, w0, w1);
                        l = __fmaf_rn(w0 + w1, iev[g - 1], l);
                        // group g - 1's weights lie over scores of groups that were read before
                        tmem_st_32x32b_x8(s_addr + 8 * (g - 1), h);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&s->p_full[t]);
                    mbar_arrive(&s->t_empty[j % TABLES]);
                }
            }
        }
    } else if (warp < MMA_WARP) {
        // ------------------------------------------------------------ converters
        constexpr int PIECES = D / 16;                       // 16-byte pieces of a token
        constexpr int TOKENS = 128 / PIECES;                 // tokens per pass of the 128 threads
        constexpr int PASSES = BLOCK / TOKENS;
        // Thread -> (token, piece): eight consecutive threads store four pieces
        // of two neighbouring tokens, whose swizzles differ in the lowest bit,
        // so a 16-byte store of theirs meets every bank once.
        const int i = tid - CONV_WARP * 32;
        const int piece = D == 64 ? i & 3 : (i & 3) | (i >> 1 & 4);
        const int tok = D == 64 ? i >> 2 : (i >> 2 & 1) | (i >> 3 & 14);
        const uint32_t row = (piece >> 2) * (BLOCK * 128) + tok * 128;
        const uint32_t at0 = row + ((((piece & 3) * 2) ^ (tok & 7)) << 4);
        const uint32_t at1 = row + ((((piece & 3) * 2 + 1) ^ (tok & 7)) << 4);
        const int within = (tok & 15) * D + piece * 16;
        [[maybe_unused]] const int64_t pool = (p.num_pages * p.kv_heads << p.page_log2) * D;
        uint4 kc[PASSES], vc[PASSES];
        auto load = [&](uint4 (&c)[PASSES], const uint8_t* const (&groups)[TABLES][GROUPS],
                        [[maybe_unused]] const uint8_t* codes, int j) {
#pragma unroll
            for (int q = 0; q < PASSES; ++q) {
                const uint8_t* at = groups[j % TABLES][q * TOKENS / 16 + (TOKENS == 32 ? tok >> 4 : 0)] + within;
                c[q] = make_uint4(0, 0, 0, 0);
                if (MQ_CHECK(at - within == reinterpret_cast<const uint8_t*>(g_zeros) || (at >= codes && at + 16 <= codes + pool)))
                    c[q] = load_codes(at);
            }
            // behind the last key a page holds whatever was there, a NaN code
            // times a zero weight is no zero: zeros instead
            const int left = k1 - (k0 + j * BLOCK);
            if (left < BLOCK) {
#pragma unroll
                for (int q = 0; q < PASSES; ++q)
                    if (q * TOKENS + tok >= left) c[q] = make_uint4(0, 0, 0, 0);
            }
        };
        auto store = [&](uint32_t dst, const uint4 (&c)[PASSES]) {
#pragma unroll
            for (int q = 0; q < PASSES; ++q) {
                const uint32_t w[4] = {c[q].x, c[q].y, c[q].z, c[q].w};
                uint32_t h[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h[2 * e] = cvt_e4m3x2_to_f16x2((uint16_t)w[e]);
                    h[2 * e + 1] = cvt_e4m3x2_to_f16x2((uint16_t)(w[e] >> 16));
                }
                st_shared_v4(dst + at0 + q * TOKENS * 128, h[0], h[1], h[2], h[3]);
                st_shared_v4(dst + at1 + q * TOKENS * 128, h[4], h[5], h[6], h[7]);
            }
            fence_proxy_async_shared();
            __syncwarp();
        };
        bool ok = wait(&s->t_full[0], 0);
        if (ok) {
            load(kc, s->k_at, p.k_codes, 0);
            load(vc, s->v_at, p.v_codes, 0);
            if (lane == 0) mbar_arrive(&s->t_empty[0]);
        }
        for (int j = 0; ok && j < blocks; ++j) {
            const int st = j % STAGES, nt = (j + 1) % TABLES;
            const uint32_t phase = (j / STAGES) & 1;
            const bool more = j + 1 < blocks;
            ok = wait(&s->k_empty[st], phase ^ 1);
            if (!ok) break;
            store(sbase + L::K_OFF + st * L::TILE_BYTES, kc);
            if (lane == 0) mbar_arrive(&s->k_full[st]);
            if (more) {
                ok = wait(&s->t_full[nt], ((j + 1) / TABLES) & 1);
                if (!ok) break;
                load(kc, s->k_at, p.k_codes, j + 1);
            }
            ok = wait(&s->v_empty[st], phase ^ 1);
            if (!ok) break;
            store(sbase + L::V_OFF + st * L::TILE_BYTES, vc);
            if (lane == 0) mbar_arrive(&s->v_full[st]);
            if (more) {
                load(vc, s->v_at, p.v_codes, j + 1);
                __syncwarp();
                if (lane == 0) mbar_arrive(&s->t_empty[nt]);
            }
        }
    } else if (warp == TABLE_WARP) {
        // ------------------------------------------------------------ tables
        // of the blocks to come: lane g looks up K's side of group g, lane g + 8 V's
        for (int j = 0; j < blocks; ++j) {
            const int tb = j % TABLES;
            int64_t off = -1;
            const uint8_t* zeros = reinterpret_cast<const uint8_t*>(g_zeros);
            float scale = 1.f;
            const int g = lane % GROUPS, at = k0 + j * BLOCK + g * 16;
            if (lane < 2 * GROUPS && at < k1) {
                const int64_t page = p.table[(int64_t)b * p.max_pages + (at >> p.page_log2)];
                if (page >= 0 && page < p.num_pages) {
                    const int64_t cell = page * p.kv_heads + head;
                    off = ((cell << p.page_log2) + (at & (page_tokens - 1))) * D;
                    scale = (lane < GROUPS ? p.k_scales : p.v_scales)[cell];
                } else if (p.status) {
                    atomicExch(p.status, MQ_ERR_INVALID_ARG);
                }
            }
            __syncwarp();
            if (!wait(&s->t_empty[tb], ((j / TABLES) & 1) ^ 1)) break;
            if (lane < GROUPS) {
                s->k_at[tb][g] = off < 0 ? zeros : p.k_codes + off;
                s->ck[tb][g] = off < 0 ? 0.f : scale;
            } else if (lane < 2 * GROUPS) {
                s->v_at[tb][g] = off < 0 ? zeros : p.v_codes + off;
                s->ev[tb][g] = off < 0 ? -INFINITY : (float)((int)(__float_as_uint(scale) >> 23) - 127);
                s->iev[tb][g] = __uint_as_float((254u << 23) - (__float_as_uint(scale) & 0x7F800000u));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s->t_full[tb]);
        }
    } else if (warp == MMA_WARP) {
        // ------------------------------------------------------------ products
        // S = Q K^T: 128 x 128 x D, both operands K-major in shared memory;
        // O += P V: 128 x D x 128, P in tensor memory, V MN-major
        constexpr uint32_t ID_S = (1u << 4) | ((uint32_t)(BLOCK >> 3) << 17) | ((uint32_t)(TILE >> 4) << 24);
        constexpr uint32_t ID_O = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(TILE >> 4) << 24);
        const bool leader = elect_one();
        // high words of the descriptors: 1024 bytes between groups of 8 rows,
        // version 1, 128-byte swizzle; V's low word also holds the 16 KB between
        // its halves of 64 d
        constexpr uint32_t HI = (1024u >> 4) | 1u << 14 | 2u << 29;
        const uint32_t q_lo = ((sbase + L::Q_OFF) >> 4 & 0x3FFF) | 1u << 16, k_lo = ((sbase + L::K_OFF) >> 4 & 0x3FFF) | 1u << 16;
        const uint32_t v_lo = ((sbase + L::V_OFF) >> 4 & 0x3FFF) | (uint32_t)(BLOCK * 128 >> 4) << 16;
        auto scores = [&](int t, int st) {
            if (leader) {
                mma_scores<D>(tmem + L::S_COL + t * BLOCK, q_lo + t * (L::TILE_BYTES >> 4), k_lo + st * (L::TILE_BYTES >> 4), ID_S, HI);
                mma_commit(&s->s_full[t]);
            }
            __syncwarp();
        };
        auto outputs = [&](int t, int st, bool first) {
            if (leader)
                mma_outputs(tmem + L::O_COL + t * D, tmem + L::S_COL + t * BLOCK, v_lo + st * (L::TILE_BYTES >> 4), ID_O, HI, !first);
            __syncwarp();
        };
        auto run = [&]() {
            if (!wait(&s->q_full, 0) || !wait(&s->k_full[0], 0)) return;
            tc_fence_after();
            scores(0, 0);
            if (two) scores(1, 0);
            if (leader) mma_commit(&s->k_empty[0]);
            __syncwarp();
            for (int j = 0; j < blocks; ++j) {
                const int st = j % STAGES, nst = (j + 1) % STAGES;
                const bool more = j + 1 < blocks;
                if (!wait(&s->v_full[st], (j / STAGES) & 1)) return;
                for (int t = 0; t < (two ? 2 : 1); ++t) {
                    if (!wait(&s->p_full[t], j & 1)) return;
                    tc_fence_after();
                    outputs(t, st, j == 0);
                    if (t == 0 && more && !wait(&s->k_full[nst], ((j + 1) / STAGES) & 1)) return;
                    tc_fence_after();
                    if (more) {
                        scores(t, nst);
                    } else {
                        if (leader) mma_commit(&s->o_full[t]);
                        __syncwarp();
                    }
                }
                if (leader) {
                    mma_commit(&s->v_empty[st]);
                    if (more) mma_commit(&s->k_empty[nst]);
                }
                __syncwarp();
            }
        };
        run();
        // also after a wait that ran out: what was issued ends before tensor memory is given back
        if (leader) mma_commit(&s->drained);
        __syncwarp();
        mbar_wait_bounded(&s->drained, 0, TIMEOUT_CYCLES, nullptr);
    }

    // ---------------------------------------------------------------- output
    const int64_t cell = ((int64_t)b * p.row_tiles + tile) * p.kv_heads + head;
    float* part = p.part ? p.part + cell * p.chunks * (int64_t)(ROWS * (D + 2)) : nullptr;
    if (warp < CONV_WARP && !(warp >= 4 && !two)) {
        const int t = warp / 4;
        const int row = row0 + tid;                          // tid = 128 t + row of the tile
        const uint32_t o_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16) + L::O_COL + t * D;
        const bool have = blocks > 0 && wait(&s->o_full[t], 0);
        tc_fence_after();
        const float inv = l > 0.f || l != l ? __fdiv_rn(1.f, l) : 0.f;       // a row that sees nothing: zero
        const int64_t at = ((int64_t)(c0 + row / p.group) * p.q_heads + head * p.group + row % p.group) * D;
        float* dst = part ? part + ((int64_t)chunk * ROWS + tid) * D : nullptr;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            uint32_t v[32];
            if (have) {
                tmem_ld_32x32b_x32(o_addr + c, v);
                tmem_ld_wait_regs(v);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0u;
            }
            if (row < rows) {
                if (chunks == 1) {
                    if (l == 0.f) {                          // its weights were all zero: so is the sum, NaN codes or not
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0u;
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t h[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            h[k] = cvt_bf16x2(__uint_as_float(v[i + 2 * k + 1]) * inv, __uint_as_float(v[i + 2 * k]) * inv);
                        if (MQ_CHECK(at + c + i + 8 <= p.T * p.q_heads * (int64_t)D))
                            *reinterpret_cast<uint4*>(p.out + at + c + i) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<uint4*>(dst + c + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
        }
        if (chunks > 1 && row < rows)
            reinterpret_cast<float2*>(kv_part_ml<D>(p, part, ROWS))[chunk * ROWS + tid] = make_float2(m, l);
        tc_fence_before();
    }
    __threadfence();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (chunks == 1) return;
    // ---- the last chunk to finish joins them, in chunk order
    if (tid == 0) {
        const int done = atomicAdd(p.tickets + cell, 1);
        s->last = done == chunks - 1;
        if (s->last) p.tickets[cell] = 0;
    }
    __syncthreads();
    if (!s->last) return;
    __threadfence();
    kv_join<D>(p, part, chunks, ROWS, last_row - row0 + 1, c0, row0, head, tid, THREADS, reinterpret_cast<float*>(base));
}

MQ_DEBUG_READER(debug_hits_kv_prefill)

template <int D>
cudaError_t launch(const KvAttendParams& p, int64_t blocks, cudaStream_t stream) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    const int d = dev < 64 ? dev : 63;
    if (!attr_set[d]) {
        cudaError_t e = cudaFuncSetAttribute(k_kv_prefill<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::SMEM);
        if (e != cudaSuccess) return e;
        attr_set[d] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    int nattr = 0;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = Layout<D>::SMEM;
    cfg.stream = stream;
    set_pdl_attr(attr, &nattr);
    cfg.attrs = attr;
    cfg.numAttrs = nattr;
    return cudaLaunchKernelEx(&cfg, k_kv_prefill<D>, p);
}

}  // namespace kv_prefill

// ---------------------------------------------------------------- host side
cudaError_t launch_kv_prefill(const KvAttendParams& p, int head_dim, int64_t blocks, cudaStream_t stream) {
    return head_dim == 64 ? kv_prefill::launch<64>(p, blocks, stream) : kv_prefill::launch<128>(p, blocks, stream);
}

}  // namespace mq
