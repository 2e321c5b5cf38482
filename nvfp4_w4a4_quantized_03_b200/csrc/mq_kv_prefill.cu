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
//   warp 12          issues the products: S_t = Q_t K^T, then O_t += P_t V, the
//                    two tiles alternating, so that one tile's softmax runs
//                    under the other's products
// V needs no transposition: [token][d] is the MN-major right operand.
//
// Bound: per block and CTA the two tiles' products take 2048 cycles of the
// tensor pipe at D = 128, their 32768 exponentials 2048 cycles of the SFU, and
// shared memory moves 256 KB, 2048 cycles: three resources near balance, so
// the tensor pipe cannot be filled; figures beside launch_kv_prefill.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/mq.h"
#include "mq_debug.cuh"
#include "mq_internal.h"
#include "mq_kv.cuh"
#include "mq_kv_plan.h"
#include "mq_ptx.cuh"

namespace mq {
namespace kv_prefill {

constexpr int TILE = 128;                       // rows per tile
constexpr int ROWS = 2 * TILE;
constexpr int BLOCK = 128;                      // keys per block
constexpr int GROUPS = BLOCK / 16;              // a page holds whole groups of 16 keys
constexpr int CONV_WARP = 8, MMA_WARP = 12;
constexpr int THREADS = 16 * 32;               // four warpgroups (warps 13-15 only hand back registers)
constexpr int STAGES = 2;                       // of K and of V
constexpr int TABLES = 4;                       // of the blocks' page scales
constexpr float LAZY = 8.f, BIAS = 6.f;         // as in mq_kv_attention.cu
constexpr long long TIMEOUT_CYCLES = 4000000000LL;

struct Smem {
    uint64_t q_full, k_full[STAGES], k_empty[STAGES], v_full[STAGES], v_empty[STAGES];
    uint64_t s_full[2], p_full[2], o_full[2], t_full[TABLES], drained;
    float ck[TABLES][GROUPS], ev[TABLES][GROUPS], iev[TABLES][GROUPS];
    uint32_t tmem_base;
    int abort_flag;
    int last;
};

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
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// 16 codes -> 16 f16, two 16-byte stores
__device__ __forceinline__ void store_f16(uint32_t addr, int chunk, int swz, int odd_first, const uint4& c) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[2 * i] = cvt_e4m3x2_to_f16x2((uint16_t)w[i]);
        h[2 * i + 1] = cvt_e4m3x2_to_f16x2((uint16_t)(w[i] >> 16));
    }
    // the two halves of a row are a multiple of 128 bytes apart: their lanes
    // start with different chunks, so that a store meets no bank twice
    const uint32_t a0 = addr + ((chunk ^ swz) << 4), a1 = addr + (((chunk + 1) ^ swz) << 4);
    if (!odd_first) {
        st_shared_v4(a0, h[0], h[1], h[2], h[3]);
        st_shared_v4(a1, h[4], h[5], h[6], h[7]);
    } else {
        st_shared_v4(a1, h[4], h[5], h[6], h[7]);
        st_shared_v4(a0, h[0], h[1], h[2], h[3]);
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

    // chunk fastest, then kv head, sequence; the last row tiles (they see most) first
    int id = blockIdx.x;
    const int chunk = id % p.chunks;
    id /= p.chunks;
    const int head = id % p.kv_heads;
    id /= p.kv_heads;
    const int b = id % p.batch, tile = p.row_tiles - 1 - id / p.batch;
    const int c0 = p.cu[b], n = p.cu[b + 1] - c0;
    const int64_t len = p.lens[b];
    const int page_tokens = 1 << p.page_log2;
    if (n <= 0) return;
    if (c0 < 0 || (int64_t)c0 + n > p.T || n > p.max_q || len > p.max_len || len > p.max_pages << p.page_log2) {
        if (tid == 0 && p.status) atomicExch(p.status, MQ_ERR_INVALID_ARG);
        return;
    }
    const int64_t rows = (int64_t)n * p.group, row0 = (int64_t)tile * ROWS;
    if (row0 >= rows) return;
    const int64_t start = len - n;
    const int64_t last_row = min(rows, row0 + ROWS) - 1;
    const int64_t end = max((int64_t)0, min(len, start + last_row / p.group + 1));
    const int chunks = max(1, (int)((end + p.chunk_tokens - 1) / p.chunk_tokens));
    if (chunk >= chunks) return;
    const int64_t k0 = (int64_t)chunk * p.chunk_tokens, k1 = min(end, k0 + p.chunk_tokens);
    const int blocks = k1 > k0 ? (int)((k1 - k0 + BLOCK - 1) / BLOCK) : 0;
    const bool two = row0 + TILE < rows;                     // the second tile has rows

    if (tid == 0) {
        mbar_init(&s->q_full, 8);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&s->k_full[i], 4);
            mbar_init(&s->v_full[i], 4);
            mbar_init(&s->k_empty[i], 1);
            mbar_init(&s->v_empty[i], 1);
        }
        for (int i = 0; i < TABLES; ++i) mbar_init(&s->t_full[i], 1);
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
    // what the others leave: 2 x 176 + 96 + 64 = 4 x 128
    if (warp < CONV_WARP)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    else if (warp < MMA_WARP)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");

    float m = -INFINITY, l = 0.f;                            // softmax threads: their row's
    if (blocks == 0) {
        // a chunk without keys (rows of padding): nothing to add up
    } else if (warp < CONV_WARP) {
        // ------------------------------------------------------------ softmax
        const int t = warp / 4;                              // tile
        const int r = tid % TILE;                            // row of the tile
        const int64_t row = row0 + t * TILE + r;
        const bool mine = row < rows;
        float fac = 0.f;
        int64_t pos = -1;
        {
            uint4 w[D / 8];
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) w[i] = make_uint4(0, 0, 0, 0);
            if (mine) {
                pos = start + row / p.group;
                const uint4* src = reinterpret_cast<const uint4*>(p.q + (c0 + row / p.group) * p.q_stride +
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
        const int64_t sees_all = start + (row0 + t * TILE) / p.group;     // keys every row of the tile sees
        if (t == 0 || two) {
            for (int j = 0; j < blocks; ++j) {
                const int64_t kb = k0 + (int64_t)j * BLOCK;
                if (!wait(&s->t_full[j % TABLES], (j / TABLES) & 1) || !wait(&s->s_full[t], j & 1)) break;
                tc_fence_after();
                const float* ck = s->ck[j % TABLES];
                const float* ev = s->ev[j % TABLES];
                const float* iev = s->iev[j % TABLES];
                const bool masked = kb + BLOCK - 1 > min(sees_all, k1 - 1);
                const int limit = (int)min((int64_t)BLOCK, min(pos, k1 - 1) - kb);   // last key of the block it sees
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < BLOCK; c += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(s_addr + c, v);
                    tmem_ld_wait_regs(v);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        float gm = -INFINITY;
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x = __uint_as_float(v[g * 16 + i]);
                            if (masked) x = c + g * 16 + i <= limit ? x : -INFINITY;
                            gm = fmaxf(gm, x);
                        }
                        // -inf stays -inf where the factor is 0 (an empty row of Q has fac > 0 all the same)
                        const float u = __fmaf_rn(gm, fac * ck[c / 16 + g], ev[c / 16 + g]);
                        top = fmaxf(top, gm == -INFINITY ? -INFINITY : u);
                    }
                }
                float f = 1.f;
                if (top > m + LAZY) {
                    f = ex2(m - top);
                    m = top;
                    l *= f;
                }
                if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
                    for (int c = 0; c < D; c += 32) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(o_addr + c, v);
                        tmem_ld_wait_regs(v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                        tmem_st_32x32b_x32(o_addr + c, v);
                    }
                }
                const float shift = BIAS - (m == -INFINITY ? 0.f : m);
#pragma unroll
                for (int c = 0; c < BLOCK; c += 32) {
                    uint32_t v[32], h[16];
                    tmem_ld_32x32b_x32(s_addr + c, v);
                    tmem_ld_wait_regs(v);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float fck = fac * ck[c / 16 + g], sh = ev[c / 16 + g] + shift;
                        float sum = 0.f;
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float x = ex2(__fmaf_rn(__uint_as_float(v[g * 16 + i]), fck, sh));
                            float y = ex2(__fmaf_rn(__uint_as_float(v[g * 16 + i + 1]), fck, sh));
                            if (masked) {
                                x = c + g * 16 + i <= limit ? x : 0.f;
                                y = c + g * 16 + i + 1 <= limit ? y : 0.f;
                            }
                            sum += x + y;
                            h[g * 8 + i / 2] = pack_f16(y, x);
                        }
                        l = __fmaf_rn(sum, iev[c / 16 + g], l);
                    }
                    tmem_st_32x32b_x16(s_addr + c / 2, h);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s->p_full[t]);
            }
        }
    } else if (warp < MMA_WARP) {
        // ------------------------------------------------------------ converters
        constexpr int PIECES = D / 16;                       // 16-byte pieces of a token
        constexpr int TOKENS = 128 / PIECES;                 // tokens per pass of the 128 threads
        constexpr int PASSES = BLOCK / TOKENS;
        const int i = tid - CONV_WARP * 32;
        const int piece = i % PIECES, tok = i / PIECES;
        const uint32_t half = (piece >> 2) * (BLOCK * 128);
        const int chunk16 = (piece & 3) * 2;
        const int odd = piece >> 2;
        const int64_t head_bytes = (int64_t)page_tokens * D;
        [[maybe_unused]] const int64_t pool = p.num_pages * p.kv_heads * head_bytes;
        // lane g of each warp: group g of a block, its byte offset in the pool (-1: nothing to read)
        int64_t off = -1;
        float gk = 0.f, gv = 1.f;
        auto find = [&](int j) {
            off = -1;
            gk = 0.f;
            gv = 1.f;
            const int64_t at = k0 + (int64_t)j * BLOCK + lane * 16;
            if (lane < GROUPS && j < blocks && at < k1) {
                const int64_t page = p.table[(int64_t)b * p.max_pages + (at >> p.page_log2)];
                if (page >= 0 && page < p.num_pages) {
                    const int64_t cell = page * p.kv_heads + head;
                    off = cell * head_bytes + (at & (page_tokens - 1)) * D;
                    gk = p.k_scales[cell];
                    gv = p.v_scales[cell];
                } else if (p.status) {
                    atomicExch(p.status, MQ_ERR_INVALID_ARG);
                }
            }
        };
        uint4 kc[PASSES], vc[PASSES];
        auto load = [&](uint4 (&c)[PASSES], const uint8_t* codes, int64_t o, int j) {
#pragma unroll
            for (int q = 0; q < PASSES; ++q) {
                const int token = q * TOKENS + tok;
                const int64_t go = __shfl_sync(0xffffffffu, o, token >> 4);
                const int64_t at = go + (token & 15) * D + piece * 16;
                c[q] = make_uint4(0, 0, 0, 0);
                // behind the last key a page holds whatever was there: zeros instead
                if (go >= 0 && k0 + (int64_t)j * BLOCK + token < k1 && MQ_CHECK(at + 16 <= pool)) c[q] = load_codes(codes + at);
            }
        };
        find(0);
        load(kc, p.k_codes, off, 0);
        load(vc, p.v_codes, off, 0);
        for (int j = 0; j < blocks; ++j) {
            const int st = j % STAGES;
            const uint32_t phase = (j / STAGES) & 1;
            if (!wait(&s->k_empty[st], phase ^ 1)) break;
            // The block's scales.  Table j % 4 is free: the stage just freed was
            // block j - 2's, whose scores needed both tiles' weights of block j - 3.
            if (warp == CONV_WARP) {
                if (lane < GROUPS) {
                    s->ck[j % TABLES][lane] = gk;
                    s->ev[j % TABLES][lane] = (float)((int)(__float_as_uint(gv) >> 23) - 127);
                    s->iev[j % TABLES][lane] = __uint_as_float((254u << 23) - (__float_as_uint(gv) & 0x7F800000u));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s->t_full[j % TABLES]);
            }
            find(j + 1);
            const uint32_t kdst = sbase + L::K_OFF + st * L::TILE_BYTES + half;
#pragma unroll
            for (int q = 0; q < PASSES; ++q) {
                const int token = q * TOKENS + tok;
                store_f16(kdst + token * 128, chunk16, token & 7, odd, kc[q]);
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s->k_full[st]);
            if (j + 1 < blocks) load(kc, p.k_codes, off, j + 1);
            if (!wait(&s->v_empty[st], phase ^ 1)) break;
            const uint32_t vdst = sbase + L::V_OFF + st * L::TILE_BYTES + half;
#pragma unroll
            for (int q = 0; q < PASSES; ++q) {
                const int token = q * TOKENS + tok;
                store_f16(vdst + token * 128, chunk16, token & 7, odd, vc[q]);
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s->v_full[st]);
            if (j + 1 < blocks) load(vc, p.v_codes, off, j + 1);
        }
    } else if (warp == MMA_WARP) {
        // ------------------------------------------------------------ products
        // S = Q K^T: 128 x 128 x D, both operands K-major in shared memory;
        // O += P V: 128 x D x 128, P in tensor memory, V MN-major
        constexpr uint32_t ID_S = (1u << 4) | ((uint32_t)(BLOCK >> 3) << 17) | ((uint32_t)(TILE >> 4) << 24);
        constexpr uint32_t ID_O = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(TILE >> 4) << 24);
        const bool leader = elect_one();
        auto scores = [&](int t, int st) {
            const uint64_t a = smem_desc(sbase + L::Q_OFF + t * L::TILE_BYTES, 16, 1024, 2);
            const uint64_t bd = smem_desc(sbase + L::K_OFF + st * L::TILE_BYTES, 16, 1024, 2);
            if (leader) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t step = (uint64_t)((k / 4) * (TILE * 128) + (k % 4) * 32) >> 4;
                    mma_ss(tmem + L::S_COL + t * BLOCK, a + step, bd + step, ID_S, k != 0);
                }
                mma_commit(&s->s_full[t]);
            }
            __syncwarp();
        };
        auto outputs = [&](int t, int st, bool first) {
            const uint64_t bd = smem_desc(sbase + L::V_OFF + st * L::TILE_BYTES, BLOCK * 128, 1024, 2);
            if (leader) {
#pragma unroll
                for (int k = 0; k < BLOCK / 16; ++k)
                    mma_ts(tmem + L::O_COL + t * D, tmem + L::S_COL + t * BLOCK + k * 8, bd + (uint64_t)(k * 2048 >> 4),
                           ID_O, !(first && k == 0));
            }
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
        const int64_t row = row0 + tid;                      // tid = 128 t + row of the tile
        const uint32_t o_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16) + L::O_COL + t * D;
        const bool have = blocks > 0 && wait(&s->o_full[t], 0);
        tc_fence_after();
        const float inv = l > 0.f || l != l ? __fdiv_rn(1.f, l) : 0.f;       // a row that sees nothing: zero
        const int64_t at = ((c0 + row / p.group) * p.q_heads + head * p.group + row % p.group) * D;
        float* dst = part ? part + ((int64_t)chunk * ROWS + tid) * (D + 2) : nullptr;
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
                    for (int i = 0; i < 32; i += 2)
                        *reinterpret_cast<float2*>(dst + c + i) =
                            make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                }
            }
        }
        if (chunks > 1 && row < rows) *reinterpret_cast<float2*>(dst + D) = make_float2(m, l);
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
    kv_join<D>(p, part, chunks, ROWS, (int)(last_row - row0 + 1), c0, row0, head, tid, THREADS);
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
