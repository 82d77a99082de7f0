// Matrix-vector products with an int4 group-32 matrix: y[t, n] = sum_k x[t, k] W[n, k] for
// 1..32 token rows x, W[n, k] = scale[n, k / 32] (nibble - 8) (the expert weights' format).
//
// What bounds it is reading W (0.5625 bytes a weight): at the copy bandwidth of a B200 that is
// 11.7 T weights a second, 41 a clock and SM, so a weight may cost about three lane operations.
// Multiply-adds on the CUDA cores alone would spend one per weight and token beside the
// decoding; here the products go to the tensor cores (mma m16n8k16, bf16 operands, fp32 sums):
//
//   A  16 rows of W as bf16 nibble - 8, exact: nibbles i and i + 4 of a word, or'ed into the
//      mantissas of the bf16 pair (128, 128), are 128 + nibble; subtracting 136 leaves the code.
//   B  x in the matching order of k (any order will do as long as both operands have it).
//   C  the sums of one scale group, multiplied by its scale and added in fp32: the scale never
//      touches an operand, so nothing is rounded before the sums.
//
// A lane reads 16-byte chunks, one whole group of one row; the quad of lanes that shares a row
// reads four consecutive groups. An mma sums over its quad, so it must not mix groups:
//
//   few rows (x has 1 or 2): the quad's four groups stay apart in the columns of B. Column
//      4 token + group holds x for the lane of that group and zero for the other three: eight
//      products make the sums of four groups and two tokens.
//   more rows: the quad transposes its 4 x 4 words, after which a lane holds its quarter of each
//      group in turn, and the eight columns of B are eight tokens.
//
// A warp owns 16 rows of W (a tile) and every KS-th step of 128 columns; the KS warps of a tile
// add their sums through shared memory in warp order, so results do not depend on timing.
#include "common.cuh"
#include "internal.h"

#include <cuda_bf16.h>

namespace redmoe {
namespace {

constexpr int GV_WARPS = 8;
constexpr int GV_THREADS = 32 * GV_WARPS;
constexpr int GV_MAX_T = 32;
constexpr int GV_STEP = 128;     // columns of a step: four groups
constexpr int GV_MAX_K = 65536;
constexpr int GV_PAD = 64;       // bytes between token rows in shared memory (bank offset)

struct GemvParams {
    const uint8_t* w;      // [N, K/2]
    const uint16_t* s;     // [N, K/32] bf16
    const uint16_t* x;     // [T, K] bf16
    void* y;               // [T, N]
    int N, K, T;
    int ks;                // warps of a tile, a power of two
    int slab;              // columns of x in shared memory at a time, a multiple of 128
};

__device__ __forceinline__ uint32_t dequant2(uint32_t w) {
    uint32_t v;
    asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(v) : "r"(w));  // (w & a) | b
    const __nv_bfloat162 off = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));  // 136
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), off);
    return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Copy columns [k0, k0 + cols) of x's T rows to shared memory, every run of eight in the order
// (0,4) (1,5) (2,6) (3,7) in which dequant2 yields a word's nibbles; zeros beyond K.
__device__ __forceinline__ void stage_x(const GemvParams& p, int k0, int cols, int stride, unsigned char* xs) {
    const int runs = cols / 8;
    for (int i = threadIdx.x; i < p.T * runs; i += GV_THREADS) {
        const int t = i / runs, r = i - t * runs, k = k0 + 8 * r;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (k < p.K) v = __ldg(reinterpret_cast<const uint4*>(p.x + size_t(t) * p.K + k));
        *reinterpret_cast<uint4*>(xs + size_t(t) * stride + 16 * r) =
            make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                       __byte_perm(v.y, v.w, 0x7632));
    }
}

// The 4 x 4 words of a quad, transposed: lane t ends with word t of the four lanes' chunks.
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int t) {
    const bool odd = t & 1, high = t & 2;
    {
        const uint32_t a = __shfl_xor_sync(FULL, odd ? w[0] : w[1], 1), b = __shfl_xor_sync(FULL, odd ? w[2] : w[3], 1);
        if (odd) { w[0] = a; w[2] = b; } else { w[1] = a; w[3] = b; }
    }
    {
        const uint32_t a = __shfl_xor_sync(FULL, high ? w[0] : w[2], 2), b = __shfl_xor_sync(FULL, high ? w[1] : w[3], 2);
        if (high) { w[0] = a; w[1] = b; } else { w[2] = a; w[3] = b; }
    }
}

template <bool F32>
__device__ __forceinline__ void put(void* y, size_t i, float v) {
    if (F32) static_cast<float*>(y)[i] = v;
    else static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
}

// NT = 0: one or two tokens; otherwise NT blocks of eight tokens.
template <int NT, bool F32>
__global__ void __launch_bounds__(GV_THREADS) gemv_kernel(const GemvParams p) {
    extern __shared__ __align__(16) unsigned char sm[];
    constexpr int NA = NT ? 4 * NT : 2;   // sums a lane holds
    const int stride = p.slab * 2 + GV_PAD;
    unsigned char* zero = sm;             // 64 bytes of zeros: x of absent tokens and other groups
    unsigned char* xs = sm + 64;
    float* red = reinterpret_cast<float*>(xs + size_t(p.T) * stride);  // [GV_WARPS][NA][32]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, q = lane & 3;
    const int tiles_cta = GV_WARPS / p.ks;
    const int wk = warp % p.ks;
    const int ntiles = (p.N + 15) / 16;
    const int groups = p.K / 32;
    if (threadIdx.x < 4) reinterpret_cast<uint4*>(zero)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
    const bool one_slab = p.slab >= p.K;
    if (one_slab) stage_x(p, 0, p.slab, stride, xs);
    __syncthreads();

    for (int tile0 = blockIdx.x * tiles_cta; tile0 < ntiles; tile0 += gridDim.x * tiles_cta) {
        const int tile = tile0 + warp / p.ks;
        const int r0 = min(tile * 16 + g, p.N - 1), r1 = min(tile * 16 + g + 8, p.N - 1);
        const uint8_t* w0 = p.w + size_t(r0) * (p.K / 2);
        const uint8_t* w1 = p.w + size_t(r1) * (p.K / 2);
        const uint16_t* s0 = p.s + size_t(r0) * groups;
        const uint16_t* s1 = p.s + size_t(r1) * groups;
        float acc[NA] = {};
        for (int k0 = 0; k0 < p.K; k0 += p.slab) {
            if (!one_slab) {
                __syncthreads();
                stage_x(p, k0, p.slab, stride, xs);
                __syncthreads();
            }
            const int steps = (min(p.slab, p.K - k0) + GV_STEP - 1) / GV_STEP;
            for (int st = wk; st < steps; st += p.ks) {
                const int k = k0 + st * GV_STEP, gr = k / 32;  // the step's first column and group
                uint32_t a[4] = {}, b[4] = {};                 // this lane's group of rows r0 and r1
                if (gr + q < groups) {
                    const uint4 u = ld_stream(w0 + k / 2 + 16 * q), v = ld_stream(w1 + k / 2 + 16 * q);
                    a[0] = u.x; a[1] = u.y; a[2] = u.z; a[3] = u.w;
                    b[0] = v.x; b[1] = v.y; b[2] = v.z; b[3] = v.w;
                }
                if (NT == 0) {
                    // scales of this lane's two columns: groups 2 (q & 1) and 2 (q & 1) + 1
                    const int c = gr + 2 * (q & 1);
                    float sc[4];
                    sc[0] = c < groups ? bf16f(__ldg(s0 + c)) : 0.0f;
                    sc[1] = c + 1 < groups ? bf16f(__ldg(s0 + c + 1)) : 0.0f;
                    sc[2] = c < groups ? bf16f(__ldg(s1 + c)) : 0.0f;
                    sc[3] = c + 1 < groups ? bf16f(__ldg(s1 + c + 1)) : 0.0f;
                    const bool mine = (g & 3) == q && (g >> 2) < p.T;
                    const unsigned char* xp = mine ? xs + size_t(g >> 2) * stride + st * (2 * GV_STEP) + 64 * q : zero;
                    float cc[4] = {};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 x = reinterpret_cast<const uint4*>(xp)[i];
                        mma_bf16(cc, dequant2(a[i]), dequant2(b[i]), dequant2(a[i] >> 4), dequant2(b[i] >> 4), x.x, x.y);
                        mma_bf16(cc, dequant2(a[i] >> 8), dequant2(b[i] >> 8), dequant2(a[i] >> 12), dequant2(b[i] >> 12),
                                 x.z, x.w);
                    }
                    acc[0] = fmaf(cc[0], sc[0], fmaf(cc[1], sc[1], acc[0]));
                    acc[1] = fmaf(cc[2], sc[2], fmaf(cc[3], sc[3], acc[1]));
                } else {
                    quad_transpose(a, q);
                    quad_transpose(b, q);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // group gr + i; beyond the last group a and b are zero codes' words
                        const float sa = gr + i < groups ? bf16f(__ldg(s0 + gr + i)) : 0.0f;
                        const float sb = gr + i < groups ? bf16f(__ldg(s1 + gr + i)) : 0.0f;
                        const uint32_t a0 = dequant2(a[i]), a1 = dequant2(b[i]), a2 = dequant2(a[i] >> 4),
                                       a3 = dequant2(b[i] >> 4), a4 = dequant2(a[i] >> 8), a5 = dequant2(b[i] >> 8),
                                       a6 = dequant2(a[i] >> 12), a7 = dequant2(b[i] >> 12);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const int t = nt * 8 + g;
                            const unsigned char* xp =
                                t < p.T ? xs + size_t(t) * stride + st * (2 * GV_STEP) + 64 * i + 16 * q : zero;
                            const uint4 x = *reinterpret_cast<const uint4*>(xp);
                            float cc[4] = {};
                            mma_bf16(cc, a0, a1, a2, a3, x.x, x.y);
                            mma_bf16(cc, a4, a5, a6, a7, x.z, x.w);
                            acc[4 * nt + 0] = fmaf(cc[0], sa, acc[4 * nt + 0]);
                            acc[4 * nt + 1] = fmaf(cc[1], sa, acc[4 * nt + 1]);
                            acc[4 * nt + 2] = fmaf(cc[2], sb, acc[4 * nt + 2]);
                            acc[4 * nt + 3] = fmaf(cc[3], sb, acc[4 * nt + 3]);
                        }
                    }
                }
            }
        }
        if (NT == 0) {  // the two lanes of a token
            acc[0] += __shfl_xor_sync(FULL, acc[0], 1);
            acc[1] += __shfl_xor_sync(FULL, acc[1], 1);
        }
        if (p.ks > 1) {
            __syncthreads();  // the sums of the tile before have been read
#pragma unroll
            for (int i = 0; i < NA; ++i) red[(warp * NA + i) * 32 + lane] = acc[i];
            __syncthreads();
            if (wk != 0) continue;
            for (int w = 1; w < p.ks; ++w) {
#pragma unroll
                for (int i = 0; i < NA; ++i) acc[i] += red[((warp + w) * NA + i) * 32 + lane];
            }
        }
        const int n0 = tile * 16 + g, n1 = n0 + 8;
        if (NT == 0) {
            const int t = q >> 1;
            if ((q & 1) == 0 && t < p.T) {
                if (n0 < p.N) put<F32>(p.y, size_t(t) * p.N + n0, acc[0]);
                if (n1 < p.N) put<F32>(p.y, size_t(t) * p.N + n1, acc[1]);
            }
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = nt * 8 + 2 * q + (i & 1), n = i < 2 ? n0 : n1;
                    if (t < p.T && n < p.N) put<F32>(p.y, size_t(t) * p.N + n, acc[4 * nt + i]);
                }
            }
        }
    }
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
    return a && b && x < y + bn && y < x + an;
}

using GemvKernel = void (*)(GemvParams);

GemvKernel pick_gemv(int T, bool f32) {
    if (T <= 2) return f32 ? gemv_kernel<0, true> : gemv_kernel<0, false>;
    if (T <= 8) return f32 ? gemv_kernel<1, true> : gemv_kernel<1, false>;
    if (T <= 16) return f32 ? gemv_kernel<2, true> : gemv_kernel<2, false>;
    return f32 ? gemv_kernel<4, true> : gemv_kernel<4, false>;
}

}  // namespace
}  // namespace redmoe

using namespace redmoe;

extern "C" redmoe_status redmoe_gemv(const redmoe_matrix* W, const void* x, int32_t x_dtype, int32_t T, void* y,
                                     int32_t y_dtype, void* stream) {
    if (!W || T < 0) return REDMOE_ERR_INVALID_ARG;
    const int dts[] = {W->dtype, x_dtype, y_dtype};
    for (int d : dts)
        if (d < 0 || d > DT_INT2) return REDMOE_ERR_INVALID_ARG;
    if (W->rows <= 0 || W->cols <= 0 || W->cols % 32) return REDMOE_ERR_INVALID_ARG;
    if (W->dtype != DT_INT4 || x_dtype != DT_BF16 || (y_dtype != DT_F32 && y_dtype != DT_BF16))
        return REDMOE_ERR_UNSUPPORTED;
    if (T > GV_MAX_T || W->cols > GV_MAX_K || W->rows > (1 << 28)) return REDMOE_ERR_UNSUPPORTED;
    if (!W->w || !W->s || !aligned(W->w, 16) || !aligned(W->s, 16)) return REDMOE_ERR_INVALID_ARG;
    if (T == 0) return REDMOE_OK;
    if (!x || !y || !aligned(x, 16) || !aligned(y, y_dtype == DT_F32 ? 4 : 2)) return REDMOE_ERR_INVALID_ARG;
    const size_t N = W->rows, K = W->cols, yb = size_t(T) * N * (y_dtype == DT_F32 ? 4 : 2);
    if (overlap(y, yb, x, size_t(T) * K * 2) || overlap(y, yb, W->w, N * K / 2) || overlap(y, yb, W->s, N * K / 16))
        return REDMOE_ERR_INVALID_ARG;
    DevInfo di;
    if (!get_dev_info(&di)) return REDMOE_ERR_CUDA;
    GemvParams p;
    p.w = static_cast<const uint8_t*>(W->w);
    p.s = static_cast<const uint16_t*>(W->s);
    p.x = static_cast<const uint16_t*>(x);
    p.y = y;
    p.N = W->rows;
    p.K = W->cols;
    p.T = T;
    const int na = T <= 2 ? 2 : (T <= 8 ? 4 : (T <= 16 ? 8 : 16));
    const int red = GV_WARPS * na * 32 * 4;
    // x whole in shared memory where two blocks of an SM can hold it, else a slab at a time
    const int room = 100 * 1024 - 64 - red;
    const int whole = (p.K + GV_STEP - 1) / GV_STEP * GV_STEP;
    const int fits = ((room / T) - GV_PAD) / 2 / GV_STEP * GV_STEP;
    p.slab = whole < fits ? whole : fits;
    const int steps = p.slab / GV_STEP, tiles = (p.N + 15) / 16;
    p.ks = 1;
    while (p.ks < GV_WARPS && 2 * p.ks <= steps && tiles * p.ks < 16 * di.sm_count) p.ks *= 2;
    const int need = (tiles + GV_WARPS / p.ks - 1) / (GV_WARPS / p.ks), most = 2 * di.sm_count;
    const int smem = 64 + T * (p.slab * 2 + GV_PAD) + red;
    const GemvKernel kern = pick_gemv(T, y_dtype == DT_F32);
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return REDMOE_ERR_CUDA;
    kern<<<need < most ? need : most, GV_THREADS, smem, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? REDMOE_OK : REDMOE_ERR_CUDA;
}
