// mq_w4a16.cu -- y = x W^T with x in bf16 and W in NVFP4 (mq_linear_w4a16): the
// projection of a decode step whose activation stays unquantized.
//
// Mathematics: y[m, n] = bf16(alpha * sum over the K slices of 2^e[m] sum_k (2^-e[m] x[m, k]) (sigma q)[n, k]).
// sigma q has at most six significant bits and lies in 2^-10 .. 2688: exact in
// f16.  x goes to f16 under a power of two per token that brings the largest
// magnitude so far of its K slice to [2^13, 2^14): eight significant bits stay
// exact down to 2^-28 of that maximum, below it an error of 2^-39 of it is
// left.  So the f16 products of mma.m16n8k16 are those of the exact operands;
// sums are binary32, with one rounding to bf16 at the end.
// (bf16 operands would spare x its conversion, but an E2M1 pair goes to f16 in
// one instruction and to bf16 in five.)
//
// Bound: the weight is read once (0.5625 bytes per element), but its decoding
// keeps up with memory only just: ~180 instructions per 16 rows x 128 columns
// of a warp, 2 cycles each on the ALU.  Measured: 1 x 4096 x 4096 5.1 us, 1 x
// 6144 x 4096 6.8, 1 x 24576 x 4096 18.0 (3.2 TB/s; 14.6 with the arithmetic
// left out, 12.3 with the loads left out), 5 x 24576 x 4096 19.3, 32 x 4096 x
// 12288 22.2.  A block holds 128 rows of W and one slice of K, the blocks of a
// cluster the slices of the same rows; a block's partial sums are added through
// distributed shared memory in rank order.  Each lane reads 16 bytes (32
// elements, two scale blocks) of a row at a time, four steps ahead, and the
// order of K inside a fragment is free, so what a lane loads is what it
// multiplies.  A warp's 16 rows are four runs of four, 32 rows apart: that is
// where the stored scales of one 64-byte piece belong, so no scale sector is
// read twice.  Dropped: one persistent block per SM with rings of its own for
// every warp (17.3 and 19.0 us for 1 and 5 x 24576 x 4096, slower below).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mq_debug.cuh"
#include "mq_kv_internal.h"
#include "mq_kv.cuh"
#include "mq_ptx.cuh"

namespace mq {
namespace w4a16 {

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int STEP = 128;                 // K elements of one warp step
constexpr int SUB = 512;                  // K elements of x converted at a time: a warp's 16 per lane
constexpr int STEPS = SUB / STEP;

struct Params {
    const __nv_bfloat16* x;               // [M, K]
    const uint8_t* w_codes;               // [N, K / 2]
    const uint8_t* w_scales;              // atoms of 128 rows x 4 scales
    const float* alpha;
    __nv_bfloat16* y;                     // [M, N]
    int M, N, K, katoms, slice, split;    // slice: K elements per block, a multiple of SUB
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float hi, float lo) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// A bf16 pair times a power of two (exact above 2^-126), to f16.
__device__ __forceinline__ uint32_t to_f16x2(uint32_t x, uint32_t pow2) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(pow2));
    return pack_f16(__uint_as_float(r & 0xFFFF0000u), __uint_as_float(r << 16));
}
__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// Eight E2M1 codes -> four f16 pairs (exact), element 0 in the low half of h[0].
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

template <int NT>
struct Shape {
    static constexpr int MP = 8 * NT, ROWS = 128;
    static constexpr int X_BYTES = 2 * MP * SUB * 2;     // two turns
    static constexpr int AHEAD = 4;                      // steps of W in registers
    static constexpr int TOKENS = MP / WARPS;            // tokens a warp converts
    static constexpr int PER_SM = 2;                     // blocks, by registers
    static constexpr int PART_BYTES = MP * ROWS * 4;
    static constexpr int SMEM = X_BYTES > PART_BYTES ? X_BYTES : PART_BYTES;
};

template <int NT>
__global__ void __launch_bounds__(THREADS, Shape<NT>::PER_SM) k_linear_w4a16(Params p) {
    using S = Shape<NT>;
    constexpr int MP = S::MP, ROWS = S::ROWS, AHEAD = S::AHEAD, TOKENS = S::TOKENS;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float s_ratio[2][MP];                   // what a token's sums so far are to be multiplied with
    __shared__ float s_up[MP];                         // 2^e of each token
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane >> 2, t = lane & 3;
    const uint32_t rank = cluster_ctarank();
    const int block = blockIdx.x / p.split;            // rows [block ROWS, ...)
    const int k_lo = (int)rank * p.slice, k_hi = min(p.K, k_lo + p.slice);

    // the first columns of W's rows toward L2 before the wait for the previous
    // grid (a prefetch leaves nothing visible; of the whole slice it took
    // bandwidth from the loads: 18.3 -> 20.0 us for 1 x 24576 x 4096)
    if (tid < ROWS && block * ROWS + tid < p.N && k_hi > k_lo)
        bulk_prefetch_l2(p.w_codes + (int64_t)(block * ROWS + tid) * (p.K / 2) + k_lo / 2, min(SUB, k_hi - k_lo) / 2);

    // the warp's tile of the block's 128 rows: rows 4 warp + (r & 3) + 32 (r >> 2)
    const uint8_t* codes[2];
    const uint8_t* scales[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = g + 8 * h, in = warp * 4 + (r & 3);
        const int row = min(block * ROWS + in + 32 * (r >> 2), p.N - 1);                  // behind N: read, not written
        codes[h] = p.w_codes + (int64_t)row * (p.K / 2) + k_lo / 2 + t * 16;
        scales[h] = p.w_scales + ((int64_t)block * p.katoms + k_lo / 64 + (t >> 1)) * 512 + in * 16 + (r >> 2) * 4 + 2 * (t & 1);
    }
    // K is a multiple of 64: where the slice ends in half a step, its upper
    // lanes read what the lower ones do; X is zero there
    const int steps = (k_hi - k_lo + STEP - 1) / STEP;
    const bool half_end = (k_hi - k_lo) % STEP != 0;
    pdl_launch_dependents();
    pdl_wait();

    uint4 cw[AHEAD][2];
    uint16_t sw[AHEAD][2];
    auto load = [&](int a, int step, int at) {             // `at`: steps from where the pointers stand
        if (step < steps) {
            int ch = at * (STEP / 2), sh = at * (STEP / 64 * 512);
            if (half_end && step == steps - 1 && t >= 2) {
                ch -= 32;
                sh -= 512;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                cw[a][h] = load_stream(codes[h] + ch);
                sw[a][h] = *reinterpret_cast<const uint16_t*>(scales[h] + sh);
            }
        }
    };
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) load(a, a, a);

    // X, 512 columns at a time: a warp converts tokens warp, warp + 8, ..., 16
    // elements per lane, under the largest exponent of the token so far
    int e_run[TOKENS];
    uint4 xw[TOKENS][2];
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) e_run[i] = -113;
    auto load_x = [&](int k0) {
#pragma unroll
        for (int i = 0; i < TOKENS; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int m = warp + WARPS * i, k = k0 + h * 256 + lane * 8;
                xw[i][h] = make_uint4(0, 0, 0, 0);
                if (m < p.M && k < k_hi) xw[i][h] = *reinterpret_cast<const uint4*>(p.x + (int64_t)m * p.K + k);
            }
    };
    auto convert = [&](int turn) {
#pragma unroll
        for (int i = 0; i < TOKENS; ++i) {
            const int m = warp + WARPS * i;
            if (m >= p.M) break;
            uint32_t top = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4& w = xw[i][h];
                top = max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(top, w.x), w.y), w.z), w.w);
            }
            const uint32_t bits = __reduce_max_sync(0xffffffffu, max(top << 16, top & 0xFFFF0000u));
            const int e = max(e_run[i], (int)(bits >> 23) - 127 - 13);        // the maximum to [2^13, 2^14)
            if (lane == 0) {
                s_ratio[turn][m] = exp2i(max(-126, e_run[i] - e));
                s_up[m] = exp2i(e);
            }
            e_run[i] = e;
            const uint32_t d = cvt_bf16x2(exp2i(-e), exp2i(-e));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 w = xw[i][h];
                const uint4 f = make_uint4(to_f16x2(w.x, d), to_f16x2(w.y, d), to_f16x2(w.z, d), to_f16x2(w.w, d));
                // as the fragments are read: [step][8 elements of a lane's 32][token][lane quarter]
                const int v = h * 32 + lane;
                *reinterpret_cast<uint4*>(smem + turn * (MP * SUB * 2) +
                                          ((((v >> 4) * 4 + (v & 3)) * MP + m) * 4 + ((v >> 2) & 3)) * 16) = f;
            }
        }
    };
    load_x(k_lo);

    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;

    int turn = 0;
    for (int k0 = k_lo, step0 = 0; k0 < k_hi; k0 += SUB, step0 += STEPS, turn ^= 1) {
        // Two turns of shared memory and one barrier: whoever writes a turn has
        // passed the barrier behind which the other one was read last.
        convert(turn);
        if (k0 + SUB < k_hi) load_x(k0 + SUB);
        __syncthreads();
        if (k0 > k_lo) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float r = s_ratio[turn][n * 8 + 2 * t + e];
                    acc[n][e] *= r;
                    acc[n][e + 2] *= r;
                }
        }
        const uint8_t* xs = smem + turn * (MP * SUB * 2);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            if (step0 + s >= steps) break;
            const int a = s % AHEAD;
            uint32_t sf[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t v = cvt_e4m3x2_to_f16x2(sw[a][h]);
                sf[h][0] = __byte_perm(v, v, 0x1010);
                sf[h][1] = __byte_perm(v, v, 0x3232);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {              // words of eight codes; scale block j / 2 of the lane's two
                uint4 b[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    b[n] = *reinterpret_cast<const uint4*>(xs + (((s * 4 + j) * MP + n * 8 + g) * 4 + t) * 16);
                const uint4 &c0 = cw[a][0], &c1 = cw[a][1];
                const uint32_t w0 = j == 0 ? c0.x : j == 1 ? c0.y : j == 2 ? c0.z : c0.w;
                const uint32_t w1 = j == 0 ? c1.x : j == 1 ? c1.y : j == 2 ? c1.z : c1.w;
                uint32_t h0[4], h1[4];
                decode8(w0, h0);
                decode8(w1, h1);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    h0[q] = mul_f16x2(h0[q], sf[0][j >> 1]);
                    h1[q] = mul_f16x2(h1[q], sf[1][j >> 1]);
                }
                const uint32_t a0[4] = {h0[0], h1[0], h0[1], h1[1]}, a1[4] = {h0[2], h1[2], h0[3], h1[3]};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_f16(acc[n], a0, b[n].x, b[n].y);
                    mma_f16(acc[n], a1, b[n].z, b[n].w);
                }
            }
            load(a, step0 + s + AHEAD, s + AHEAD);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            codes[h] += SUB / 2;
            scales[h] += SUB / 64 * 512;
        }
    }
    // acc: rows g (0, 1) and g + 8 (2, 3) of a tile, tokens 2t and 2t + 1, to [token][row of the block]
    __syncthreads();
    float* part = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int m = n * 8 + 2 * t + (e & 1), r = g + 8 * (e >> 1);
            if (m < p.M) part[m * ROWS + warp * 4 + (r & 3) + 32 * (r >> 2)] = k_hi > k_lo ? acc[n][e] * s_up[m] : 0.f;
        }
    if (p.split > 1)
        cluster_sync();
    else
        __syncthreads();
    // the cluster's blocks finish a share of the outputs each, partial sums added in rank order
    const float alpha = *p.alpha;
    const float* peer[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) peer[q] = q < p.split ? map_shared_rank(part, (uint32_t)q) : part;
    for (int i = (int)rank * THREADS + tid; i < p.M * ROWS; i += p.split * THREADS) {
        float sum = peer[0][i];
#pragma unroll
        for (int q = 1; q < 8; ++q)
            if (q < p.split) sum += peer[q][i];
        const int m = i / ROWS, n = block * ROWS + i % ROWS;
        if (n < p.N && MQ_CHECK((int64_t)m * p.N + n < (int64_t)p.M * p.N))
            p.y[(int64_t)m * p.N + n] = __float2bfloat16_rn(sum * alpha);
    }
    if (p.split > 1) cluster_sync();                   // peers' shared memory is read until here
}

MQ_DEBUG_READER(debug_hits_w4a16)

template <int NT>
cudaError_t launch(Params p, int num_sms, cudaStream_t stream) {
    using S = Shape<NT>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    const int d = dev < 64 ? dev : 63;
    if (!attr_set[d]) {
        cudaError_t e = cudaFuncSetAttribute(k_linear_w4a16<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        attr_set[d] = true;
    }
    const int blocks = (p.N + S::ROWS - 1) / S::ROWS;
    // split K (a power of two, at most 8) while a block keeps 512 columns and
    // all blocks run at once (a second wave of few blocks costs as much as the first)
    int split = 1;
    while (split < 8 && (int64_t)blocks * split * 2 <= S::PER_SM * (int64_t)num_sms && (p.K + SUB - 1) / SUB >= 2 * split) split *= 2;
    p.split = split;
    p.slice = ((p.K + SUB - 1) / SUB + split - 1) / split * SUB;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    int nattr = 1;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(blocks * split);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = stream;
    set_pdl_attr(attr, &nattr);
    cfg.attrs = attr;
    cfg.numAttrs = nattr;
    return cudaLaunchKernelEx(&cfg, k_linear_w4a16<NT>, p);
}

}  // namespace w4a16

// ---------------------------------------------------------------- host side
cudaError_t launch_linear_w4a16(const void* x, int64_t M, int64_t K, const uint8_t* w_codes, const uint8_t* w_scales,
                                const float* alpha_w, int64_t N, void* y, int num_sms, cudaStream_t stream) {
    using namespace w4a16;
    Params p{static_cast<const __nv_bfloat16*>(x), w_codes, w_scales, alpha_w, static_cast<__nv_bfloat16*>(y),
             (int)M, (int)N, (int)K, (int)scale_atom_cols(K), 0, 1};
    if (M <= 8) return launch<1>(p, num_sms, stream);
    if (M <= 16) return launch<2>(p, num_sms, stream);
    // 32 tokens at a time: eight n-tiles do not fit the registers, and reading W
    // a second time costs less (64 x 4096 x 12288: 98 us as one)
    for (int64_t m = 0; m < M; m += 32) {
        p.x = static_cast<const __nv_bfloat16*>(x) + m * K;
        p.y = static_cast<__nv_bfloat16*>(y) + m * N;
        p.M = (int)(M - m < 32 ? M - m : 32);
        const cudaError_t e = launch<4>(p, num_sms, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace mq
