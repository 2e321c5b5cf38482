// mq_w4a16.cu -- y = x W^T with x in bf16 and W in NVFP4 (mq_linear_w4a16): the
// projection of a decode step whose activation stays unquantized.
//
// Mathematics: y[m, n] = bf16(alpha * 2^12 * sum_k x[m, k] (2^-12 sigma[n, k/16] q[n, k])).
// sigma q has at most six significant bits, so (2^-12 sigma q) is exact in
// bf16; the products of mma.m16n8k16 are exact and summed in binary32; one
// rounding to bf16 at the end.
//
// An E2M1 code S EE M placed at bits 15, 8..6 of a bf16 is q 2^-126 (the
// subnormal 0.5 included); times the bf16 sigma 2^114 it is 2^-12 sigma q.
//
// Bound: the weight is read once (0.5625 bytes per element).  A block holds
// 16 RT rows, its warps split K, each lane reads 16 bytes (32 elements, two
// scale blocks) of a row at a time, and the order of K inside a fragment is
// free, so what a lane loads is what it multiplies.  The 16 rows of a tile
// are four runs of four, 32 rows apart: that is where the stored scales of one
// 64-byte piece belong, so no scale sector is read twice.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/mq.h"
#include "mq_debug.cuh"
#include "mq_internal.h"
#include "mq_ptx.cuh"

namespace mq {
namespace w4a16 {

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int STEP = 128;                 // K elements of one warp step

struct Params {
    const __nv_bfloat16* x;               // [M, K]
    const uint8_t* w_codes;               // [N, K / 2]
    const uint8_t* w_scales;              // atoms of 128 rows x 4 scales
    const float* alpha;
    __nv_bfloat16* y;                     // [M, N]
    int M, N, K, katoms;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// Elements i and i + 4 of a word of eight codes, as bf16 pair q 2^-126.
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    const uint32_t top = I == 3 ? w : w << (12 - 4 * I);
    const uint32_t mag = I < 2 ? w << (6 - 4 * I) : w >> (4 * I - 6);
    return (top & 0x80008000u) | (mag & 0x01C001C0u);
}
// Two E4M3 scales -> each twice in a bf16 pair, times 2^114 (exact).
__device__ __forceinline__ void scale_pairs(uint16_t s, uint32_t (&f)[2]) {
    const uint32_t h = cvt_e4m3x2_to_f16x2(s);
    const __half2 v = *reinterpret_cast<const __half2*>(&h);
    const float k = __uint_as_float((114u + 127u) << 23);
    const float lo = __low2float(v) * k, hi = __high2float(v) * k;
    f[0] = cvt_bf16x2(lo, lo);
    f[1] = cvt_bf16x2(hi, hi);
}

template <int NT, int RT>
__global__ void __launch_bounds__(THREADS) k_linear_w4a16(Params p) {
    constexpr int ROWS = 16 * RT, MP = 8 * NT;
    extern __shared__ float part[];                    // [WARPS][MP][ROWS]
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane >> 2, t = lane & 3;
    // tile rows: base + (r & 3) + 32 (r >> 2)
    const int tiles = blockIdx.x * RT;
    int row[RT][2];
    const uint8_t* codes[RT][2];
    const uint8_t* scales[RT][2];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int tile = tiles + i, r = g + 8 * h;
            const int atom = tile >> 3, in = (tile & 7) * 4 + (r & 3);     // row % 32
            row[i][h] = atom * 128 + in + 32 * (r >> 2);
            const int rc = min(row[i][h], p.N - 1);                        // rows behind N: read, not written
            codes[i][h] = p.w_codes + (int64_t)rc * (p.K / 2) + t * 16;
            const int atom_c = min(atom, (p.N + 127) / 128 - 1);
            scales[i][h] = p.w_scales + ((int64_t)atom_c * p.katoms + (t >> 1)) * 512 + in * 16 + (r >> 2) * 4 + 2 * (t & 1);
        }
    pdl_launch_dependents();
    pdl_wait();

    float acc[RT][NT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[i][n][0] = acc[i][n][1] = acc[i][n][2] = acc[i][n][3] = 0.f;

    uint4 cw[RT][2];
    uint16_t sw[RT][2];
    auto load = [&](int k0) {
        // K is a multiple of 64: of the last step the upper lanes may hold nothing
        const bool in = k0 + 32 * t < p.K;
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                cw[i][h] = make_uint4(0, 0, 0, 0);
                sw[i][h] = 0;
                if (in) {
                    cw[i][h] = load_stream(codes[i][h] + k0 / 2);
                    sw[i][h] = *reinterpret_cast<const uint16_t*>(scales[i][h] + (int64_t)(k0 / 64) * 512);
                }
            }
    };
    int k0 = warp * STEP;
    if (k0 < p.K) load(k0);
    for (; k0 < p.K; k0 += WARPS * STEP) {
        uint4 c[RT][2];
        uint32_t sf[RT][2][2];
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                c[i][h] = cw[i][h];
                scale_pairs(sw[i][h], sf[i][h]);
            }
        if (k0 + WARPS * STEP < p.K) load(k0 + WARPS * STEP);
        const bool in = k0 + 32 * t < p.K;
#pragma unroll
        for (int j = 0; j < 4; ++j) {                  // words of eight codes; scale block j / 2 of the lane's two
            uint32_t b[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint4 xv = make_uint4(0, 0, 0, 0);
                if (in && n * 8 + g < p.M)
                    xv = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)(n * 8 + g) * p.K + k0 + 32 * t + 8 * j));
                b[n][0] = __byte_perm(xv.x, xv.z, 0x5410);     // elements 0, 4
                b[n][1] = __byte_perm(xv.x, xv.z, 0x7632);     // 1, 5
                b[n][2] = __byte_perm(xv.y, xv.w, 0x5410);     // 2, 6
                b[n][3] = __byte_perm(xv.y, xv.w, 0x7632);     // 3, 7
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const uint32_t w0 = j == 0 ? c[i][0].x : j == 1 ? c[i][0].y : j == 2 ? c[i][0].z : c[i][0].w;
                const uint32_t w1 = j == 0 ? c[i][1].x : j == 1 ? c[i][1].y : j == 2 ? c[i][1].z : c[i][1].w;
                const uint32_t s0 = sf[i][0][j >> 1], s1 = sf[i][1][j >> 1];
                const uint32_t a0[4] = {mul_bf16x2(code_pair<0>(w0), s0), mul_bf16x2(code_pair<0>(w1), s1),
                                        mul_bf16x2(code_pair<1>(w0), s0), mul_bf16x2(code_pair<1>(w1), s1)};
                const uint32_t a1[4] = {mul_bf16x2(code_pair<2>(w0), s0), mul_bf16x2(code_pair<2>(w1), s1),
                                        mul_bf16x2(code_pair<3>(w0), s0), mul_bf16x2(code_pair<3>(w1), s1)};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_bf16(acc[i][n], a0, b[n][0], b[n][1]);
                    mma_bf16(acc[i][n], a1, b[n][2], b[n][3]);
                }
            }
        }
    }
    // acc: rows g (0, 1) and g + 8 (2, 3) of a tile, tokens 2t and 2t + 1
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                part[(warp * MP + n * 8 + 2 * t + (e & 1)) * ROWS + i * 16 + g + 8 * (e >> 1)] = acc[i][n][e];
    __syncthreads();
    const float scale = __fmul_rn(__ldg(p.alpha), 4096.f);
    for (int i = tid; i < p.M * ROWS; i += THREADS) {
        const int m = i / ROWS, r = i % ROWS;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) sum += part[(w * MP + m) * ROWS + r];
        const int tile = tiles + r / 16, rr = r % 16;
        const int n = (tile >> 3) * 128 + (tile & 7) * 4 + (rr & 3) + 32 * (rr >> 2);
        if (n < p.N && MQ_CHECK((int64_t)m * p.N + n < (int64_t)p.M * p.N))
            p.y[(int64_t)m * p.N + n] = __float2bfloat16_rn(sum * scale);
    }
}

MQ_DEBUG_READER(debug_hits_w4a16)

template <int NT, int RT>
cudaError_t launch(const Params& p, cudaStream_t stream) {
    constexpr int SMEM = WARPS * 8 * NT * 16 * RT * 4;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    const int d = dev < 64 ? dev : 63;
    if (!attr_set[d]) {
        cudaError_t e = cudaFuncSetAttribute(k_linear_w4a16<NT, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        attr_set[d] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    int nattr = 0;
    const int tiles = (p.N + 127) / 128 * 8;
    cfg.gridDim = dim3((tiles + RT - 1) / RT);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = stream;
    set_pdl_attr(attr, &nattr);
    cfg.attrs = attr;
    cfg.numAttrs = nattr;
    return cudaLaunchKernelEx(&cfg, k_linear_w4a16<NT, RT>, p);
}

}  // namespace w4a16

// ---------------------------------------------------------------- host side
cudaError_t launch_linear_w4a16(const void* x, int64_t M, int64_t K, const uint8_t* w_codes, const uint8_t* w_scales,
                                const float* alpha_w, int64_t N, void* y, int num_sms, cudaStream_t stream) {
    using namespace w4a16;
    (void)num_sms;
    Params p{static_cast<const __nv_bfloat16*>(x), w_codes, w_scales, alpha_w, static_cast<__nv_bfloat16*>(y),
             (int)M, (int)N, (int)K, (int)scale_atom_cols(K)};
    if (M <= 8) return launch<1, 1>(p, stream);
    if (M <= 16) return launch<2, 1>(p, stream);
    if (M <= 32) return launch<4, 2>(p, stream);
    return launch<8, 2>(p, stream);
}

}  // namespace mq
