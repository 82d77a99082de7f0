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
// A step is 16 rows of W (a tile) by 128 columns. A block has a run of whole tiles, its warps
// equal shares of that run's steps; a tile whose steps fall to several warps is added up through
// shared memory in warp order, so results do not depend on timing. Loads run two steps ahead
// in registers.
#include "common.cuh"
#include "internal.h"

#include <cuda_bf16.h>

namespace redmoe {
namespace {

constexpr int GV_MAX_T = 32;
constexpr int GV_STEP = 128;     // columns of a step: four groups
constexpr int GV_MAX_K = 65536;
constexpr int GV_PAD = 64;       // bytes between token rows in shared memory (bank offset)
constexpr int GV_AHEAD = 2;      // steps of a load batch; one batch is in flight while one is used
constexpr int GV_ZERO = 256;     // bytes of zeros: one step of an absent token

struct GemvParams {
    const uint8_t* w;      // [N, K/2]
    const uint16_t* s;     // [N, K/32] bf16
    const uint16_t* x;     // [T, K] bf16
    void* y;               // [T, N]
    int N, K, T;
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

// Copy x's T rows to shared memory, every run of eight columns in the order (0,4) (1,5) (2,6)
// (3,7) in which dequant2 yields a word's nibbles; zeros beyond K, and a step of zeros behind.
template <int THREADS>
__device__ __forceinline__ void stage_x(const GemvParams& p, int steps, int stride, unsigned char* xs) {
    const int runs = steps * (GV_STEP / 8);
    for (int i = threadIdx.x; i < p.T * runs; i += THREADS) {
        const int t = i / runs, r = i - t * runs;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (8 * r < p.K) v = __ldg(reinterpret_cast<const uint4*>(p.x + size_t(t) * p.K + 8 * r));
        *reinterpret_cast<uint4*>(xs + size_t(t) * stride + 16 * r) =
            make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                       __byte_perm(v.y, v.w, 0x7632));
    }
    if (threadIdx.x < GV_ZERO / 16)
        *reinterpret_cast<uint4*>(xs + size_t(p.T) * stride + 16 * threadIdx.x) = make_uint4(0u, 0u, 0u, 0u);
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

// One step's operands as they come from memory: this lane's group of rows r0 and r1 and the
// scales that its sums need.
template <int NT>
struct Step {
    static constexpr int NS = NT ? 4 : 2;
    uint32_t a[4], b[4], s[NS];
};

// Position in a run of steps: 128 columns `s` of tile `tile`, with the lane's addresses there.
struct Cursor {
    const uint8_t *w0, *w1;
    const uint16_t *s0, *s1;
    int tile, s;
    __device__ __forceinline__ void at(const GemvParams& p, int tile_, int s_, int g, int q) {
        tile = tile_;
        s = s_;
        const int r0 = min(tile * 16 + g, p.N - 1), r1 = min(tile * 16 + g + 8, p.N - 1);
        w0 = p.w + size_t(r0) * (p.K / 2) + size_t(s) * 64 + 16 * q;
        w1 = p.w + size_t(r1) * (p.K / 2) + size_t(s) * 64 + 16 * q;
        s0 = p.s + size_t(r0) * (p.K / 32) + 4 * s;
        s1 = p.s + size_t(r1) * (p.K / 32) + 4 * s;
    }
    __device__ __forceinline__ void next(const GemvParams& p, int steps, int g, int q) {
        if (++s == steps) {
            at(p, tile + 1, 0, g, q);
            return;
        }
        w0 += 64;
        w1 += 64;
        s0 += 4;
        s1 += 4;
    }
};

// A pair of bf16 scales; ALIGNED: K % 128 == 0, every step has four groups and starts on 8 bytes.
__device__ __forceinline__ uint32_t scale2(const uint16_t* s, int i, int left) {
    const uint32_t lo = i < left ? __ldg(s + i) : 0, hi = i + 1 < left ? __ldg(s + i + 1) : 0;
    return lo | (hi << 16);
}

template <int NT, bool ALIGNED>
__device__ __forceinline__ void load_step(const GemvParams& p, const Cursor& c, int q, Step<NT>& st) {
    const int left = p.K / 32 - 4 * c.s;  // groups from this step's first to the row's end
    uint4 u = make_uint4(0u, 0u, 0u, 0u), v = u;
    if (ALIGNED || q < left) {
        u = ld_stream(c.w0);
        v = ld_stream(c.w1);
    }
    st.a[0] = u.x; st.a[1] = u.y; st.a[2] = u.z; st.a[3] = u.w;
    st.b[0] = v.x; st.b[1] = v.y; st.b[2] = v.z; st.b[3] = v.w;
    if (NT == 0) {  // this lane's two columns: groups 2 (q & 1) and 2 (q & 1) + 1
        const int i = 2 * (q & 1);
        st.s[0] = ALIGNED ? __ldg(reinterpret_cast<const uint32_t*>(c.s0 + i)) : scale2(c.s0, i, left);
        st.s[1] = ALIGNED ? __ldg(reinterpret_cast<const uint32_t*>(c.s1 + i)) : scale2(c.s1, i, left);
    } else if (ALIGNED) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(c.s0)), y = __ldg(reinterpret_cast<const uint2*>(c.s1));
        st.s[0] = x.x; st.s[1] = x.y; st.s[2 % Step<NT>::NS] = y.x; st.s[3 % Step<NT>::NS] = y.y;
    } else {
        st.s[0] = scale2(c.s0, 0, left);
        st.s[1] = scale2(c.s0, 2, left);
        st.s[2 % Step<NT>::NS] = scale2(c.s1, 0, left);
        st.s[3 % Step<NT>::NS] = scale2(c.s1, 2, left);
    }
}

// acc += the step's products. xp: this lane's x at the step's first column, of its token and
// group (few rows) or of each of its NT tokens.
__device__ __forceinline__ void few_step(const Step<0>& st, const unsigned char* xp, float (&acc)[2]) {
    float cc[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 x = reinterpret_cast<const uint4*>(xp)[i];
        const uint32_t a = st.a[i], b = st.b[i];
        mma_bf16(cc, dequant2(a), dequant2(b), dequant2(a >> 4), dequant2(b >> 4), x.x, x.y);
        mma_bf16(cc, dequant2(a >> 8), dequant2(b >> 8), dequant2(a >> 12), dequant2(b >> 12), x.z, x.w);
    }
    acc[0] = fmaf(cc[0], bf16lo(st.s[0]), fmaf(cc[1], bf16hi(st.s[0]), acc[0]));
    acc[1] = fmaf(cc[2], bf16lo(st.s[1]), fmaf(cc[3], bf16hi(st.s[1]), acc[1]));
}

template <int NT>
__device__ __forceinline__ void row_step(Step<NT>& st, const unsigned char* const (&xp)[NT], int q, float (&acc)[4 * NT]) {
    quad_transpose(st.a, q);
    quad_transpose(st.b, q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float sa = i & 1 ? bf16hi(st.s[i / 2]) : bf16lo(st.s[i / 2]);
        const float sb = i & 1 ? bf16hi(st.s[2 + i / 2]) : bf16lo(st.s[2 + i / 2]);
        const uint32_t a = st.a[i], b = st.b[i];
        const uint32_t a0 = dequant2(a), a1 = dequant2(b), a2 = dequant2(a >> 4), a3 = dequant2(b >> 4),
                       a4 = dequant2(a >> 8), a5 = dequant2(b >> 8), a6 = dequant2(a >> 12), a7 = dequant2(b >> 12);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint4 x = *reinterpret_cast<const uint4*>(xp[nt] + 64 * i);
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

// Results of one tile: NT = 0 after adding the two lanes of a token.
template <int NT, bool F32, int NA>
__device__ __forceinline__ void put_tile(const GemvParams& p, int tile, int g, int q, const float (&acc)[NA]) {
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
                if (t < p.T && n < p.N) put<F32>(p.y, size_t(t) * p.N + n, acc[(4 * nt + i) % NA]);
            }
        }
    }
}

// NT = 0: one or two tokens; otherwise NT blocks of eight tokens. All of x in shared memory.
template <int NT, bool F32, bool ALIGNED, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 8 ? 3 : 1) gemv_kernel(const GemvParams p) {
    extern __shared__ __align__(16) unsigned char sm[];
    constexpr int NA = NT ? 4 * NT : 2;   // sums a lane holds
    const int steps = (p.K + GV_STEP - 1) / GV_STEP;
    const int stride = steps * (2 * GV_STEP) + GV_PAD;
    unsigned char* xs = sm;
    unsigned char* zero = xs + size_t(p.T) * stride;  // x of absent tokens and of other groups
    float* red = reinterpret_cast<float*>(zero + GV_ZERO);  // [WARPS][NA][32]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, q = lane & 3;
    const int ntiles = (p.N + 15) / 16;
    const int ta = int((long long)ntiles * blockIdx.x / gridDim.x), tb = int((long long)ntiles * (blockIdx.x + 1) / gridDim.x);
    // at most 2^24 tiles over 148 blocks or more, of 512 steps: total * WARPS < 2^30
    const int total = (tb - ta) * steps;
    auto begin = [&](int w) { return total * w / WARPS; };
    const int za = begin(warp), zb = begin(warp + 1);

    Cursor in;
    in.at(p, ta + za / steps, za % steps, g, q);
    int tile = in.tile, s = in.s;
    int zin = za;
    Step<NT> st[2][GV_AHEAD];
    auto fetch = [&](Step<NT> (&to)[GV_AHEAD]) {
#pragma unroll
        for (int i = 0; i < GV_AHEAD; ++i) {
            if (zin < zb) {
                load_step<NT, ALIGNED>(p, in, q, to[i]);
                in.next(p, steps, g, q);
            }
            ++zin;
        }
    };
    fetch(st[0]);
    stage_x<32 * WARPS>(p, steps, stride, xs);
    __syncthreads();

    constexpr int NX = NT ? NT : 1;
    const unsigned char* x0[NX];  // this lane's x in step 0, and what a step adds
    int xstep[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        const int t = NT ? 8 * i + g : g >> 2;
        const bool mine = t < p.T && (NT || (g & 3) == q);
        x0[i] = (mine ? xs + size_t(t) * stride : zero) + (NT ? 16 * q : (mine ? 64 * q : 0));
        xstep[i] = mine ? 2 * GV_STEP : 0;
    }
    float acc[NA] = {};
    bool whole = s == 0;  // the segment at hand starts at its tile's first step
    auto finish = [&](bool last) {  // the segment ends: behind its tile's last step, or (last) before it
        if (NT == 0) {
            acc[0] += __shfl_xor_sync(FULL, acc[0], 1);
            acc[1] += __shfl_xor_sync(FULL, acc[1], 1);
        }
        if (whole && !last) put_tile<NT, F32, NA>(p, tile, g, q, acc);
        if (!whole) {
#pragma unroll
            for (int i = 0; i < NA; ++i) red[(warp * NA + i) * 32 + lane] = acc[i];
        }
    };
    auto use = [&](Step<NT> (&from)[GV_AHEAD], int z) {
#pragma unroll
        for (int i = 0; i < GV_AHEAD; ++i) {
            if (z + i >= zb) break;
            const unsigned char* xp[NX];
#pragma unroll
            for (int j = 0; j < NX; ++j) xp[j] = x0[j] + s * xstep[j];
            if constexpr (NT == 0) few_step(from[i], xp[0], acc);
            else row_step<NT>(from[i], xp, q, acc);
            if (++s == steps) {
                finish(false);
                ++tile;
                s = 0;
                whole = true;
#pragma unroll
                for (int j = 0; j < NA; ++j) acc[j] = 0.0f;
            }
        }
    };
    for (int z = za; z < zb; z += 2 * GV_AHEAD) {
        fetch(st[1]);
        use(st[0], z);
        fetch(st[0]);
        use(st[1], z + GV_AHEAD);
    }
    const bool open = zb > za && s != 0;  // the last segment ends inside its tile
    if (open) finish(true);
    __syncthreads();
    if (!open || !whole) return;
    // this warp has the tile's first steps: the rest lies with the warps behind it
    const int end = (tile - ta + 1) * steps;
    for (int w = warp + 1; w < WARPS && begin(w) < end; ++w) {
        if (begin(w) == begin(w + 1)) continue;
#pragma unroll
        for (int i = 0; i < NA; ++i) acc[i] += red[(w * NA + i) * 32 + lane];
    }
    put_tile<NT, F32, NA>(p, tile, g, q, acc);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
    return a && b && x < y + bn && y < x + an;
}

using GemvKernel = void (*)(GemvParams);

struct GemvPlan {
    GemvKernel kern;
    int warps, sums, blocks;  // warps a block, sums a lane, blocks an SM
};

template <bool F32, bool ALIGNED>
GemvPlan plan_for(int T) {
    if (T <= 2) return {gemv_kernel<0, F32, ALIGNED, 8>, 8, 2, 3};
    if (T <= 8) return {gemv_kernel<1, F32, ALIGNED, 16>, 16, 4, 1};
    if (T <= 16) return {gemv_kernel<2, F32, ALIGNED, 16>, 16, 8, 1};
    return {gemv_kernel<4, F32, ALIGNED, 16>, 16, 16, 1};
}
GemvPlan plan_gemv(int T, bool f32, bool aligned) {
    return f32 ? (aligned ? plan_for<true, true>(T) : plan_for<true, false>(T))
               : (aligned ? plan_for<false, true>(T) : plan_for<false, false>(T));
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
    p.N = W->rows;
    p.K = W->cols;
    // Token rows at a time: as many as fit in shared memory (all, at 32 rows of up to 2,944
    // columns or 8 of up to 13,000), in whole blocks of eight where that is less than T. Each
    // pass over W serves one such share.
    const bool f32 = y_dtype == DT_F32, aligned128 = p.K % GV_STEP == 0;
    const int steps = (p.K + GV_STEP - 1) / GV_STEP, tiles = (p.N + 15) / 16;
    const int stride = steps * (2 * GV_STEP) + GV_PAD;
    const int room = di.max_smem_optin - GV_ZERO - 16 * 16 * 32 * 4;
    int most = room / stride;
    if (most < T && most > 8) most -= most % 8;
    if (most < 1) return REDMOE_ERR_UNSUPPORTED;
    for (int t = 0; t < T; t += most) {
        p.T = T - t < most ? T - t : most;
        p.x = static_cast<const uint16_t*>(x) + size_t(t) * p.K;
        p.y = static_cast<char*>(y) + size_t(t) * p.N * (f32 ? 4 : 2);
        const GemvPlan plan = plan_gemv(p.T, f32, aligned128);
        const int smem = p.T * stride + GV_ZERO + plan.warps * plan.sums * 32 * 4;
        if (smem > 48 * 1024 &&
            cudaFuncSetAttribute(plan.kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return REDMOE_ERR_CUDA;
        const int slots = plan.blocks * di.sm_count;
        plan.kern<<<tiles < slots ? tiles : slots, 32 * plan.warps, smem, static_cast<cudaStream_t>(stream)>>>(p);
        if (cudaGetLastError() != cudaSuccess) return REDMOE_ERR_CUDA;
    }
    return REDMOE_OK;
}
