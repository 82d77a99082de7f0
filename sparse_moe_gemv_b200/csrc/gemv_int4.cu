// Matrix-vector products with an int4 group-32 matrix: y[t, n] = sum_k x[t, k] W[n, k] for
// 1..32 token rows x, W[n, k] = scale[n, k / 32] (nibble - 8) (the expert weights' format).
//
// What bounds it is reading W (0.5625 bytes a weight): at the copy bandwidth of a B200 that is
// 11.7 T weights a second, 41 a clock and SM, so a weight may cost about three lane operations.
// Multiply-adds on the CUDA cores alone would spend one per weight and token beside the
// decoding; here the products go to the tensor cores (mma m16n8k16, bf16 operands, fp32 sums)
// and a nibble is decoded by one AND:
//
//   A  16 rows of W. The bf16 bit patterns 0 .. 255 are the numbers 0 .. 255 times 2^-133 (the
//      subnormals and the first binade share their step, and mma takes both as they are), so a
//      word's nibbles under the masks 0x000F000F and 0x00F000F0, and those of the word shifted by
//      eight, already are pairs of bf16 numbers nibble 2^-133 and 16 nibble 2^-133.
//   B  x in the matching order of k (any order will do as long as both operands have it), every
//      second pair divided by 16, scaled by a power of two per token that puts its largest
//      element just under the largest bf16: products come out near one. All of that is exact.
//   C  starts at -8 times the group's sum of x and takes the products: the sum over a scale group
//      of x (nibble - 8). It is multiplied by the group's scale and added up in fp32; the scale
//      never touches an operand.
//
// Products are exact (down to 2^-116 of a row's largest x). The sums of a group run over nibbles
// of 0 .. 15, so their rounding is in proportion to 16 scale sum |x|, about three times what sums
// of the codes -8 .. 7 would have. An infinite x makes its row NaN (infinity - infinity).
//
// An mma sums over the quad of lanes that shares its rows, so the quad must not mix groups:
//
//   one or two rows of x: the eight columns of B are eight groups. A lane holds one whole group
//      (16 bytes) of one row; column j of B is x in the lane slots of group j and zero in the
//      others, so one chain of eight products makes eight groups' sums of eight W rows.
//   more rows: the eight columns of B are eight tokens, and a lane holds its quarter (4 bytes) of
//      one group after the other.
//
// A step is 16 rows of W (a tile) by 256 columns. A block has a run of whole tiles, its warps
// equal shares of that run's steps; a tile whose steps fall to several warps is added up through
// shared memory in warp order, so results do not depend on timing. Each warp copies its steps
// into a ring of its own with asynchronous copies (128-byte lines asked for whole), so no warp
// waits for another until the end, and the loads in flight need no registers.
#include "common.cuh"
#include "internal.h"

#include <cuda_bf16.h>

namespace redmoe {
namespace {

constexpr int GV_WARPS = 16;
constexpr int GV_MAX_T = 32;
constexpr int GV_MAX_K = 65536;
constexpr int GV_COLS = 256;     // columns of a step
constexpr int GV_PAD = 64;       // bytes between token rows of x in shared memory (bank offset)
constexpr int GV_ZERO = 256;     // bytes of zeros: half a step of an absent token
constexpr int GV_WROW = GV_COLS / 2 + 16;                  // bytes of a slot's row of W (bank offset)
constexpr int GV_SROW = GV_COLS / 16;                      // bytes of a slot's row of scales
constexpr int GV_SLOT = 16 * (GV_WROW + GV_SROW);
constexpr int GV_SLOTS = 4;      // of a warp's ring: three steps in flight while one is used
constexpr int GV_RING = GV_SLOTS * GV_SLOT;

struct GemvParams {
    const uint8_t* w;      // [N, K/2]
    const uint16_t* s;     // [N, K/32] bf16
    const uint16_t* x;     // [T, K] bf16
    void* y;               // [T, N]
    int N, K, T;
};

__host__ __device__ __forceinline__ int row_stride(int K) { return (K + GV_COLS - 1) / GV_COLS * (2 * GV_COLS) + GV_PAD; }

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
// d = c0 c1 in both rows + the products of one word of two rows with eight columns of x.
__device__ __forceinline__ void mma_word(float (&d)[4], uint32_t a, uint32_t b, const uint4& x, float c0, float c1,
                                         float c2, float c3) {
    constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u;
    mma_bf16(d, a & LO, b & LO, a & HI, b & HI, x.x, x.y, c0, c1, c2, c3);
    mma_bf16(d, (a >> 8) & LO, (b >> 8) & LO, (a >> 8) & HI, (b >> 8) & HI, x.z, x.w, d[0], d[1], d[2], d[3]);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// The exponent that a row's largest x is scaled to: the largest with room for rounding sums.
constexpr int GV_TOP = 126;

// x's T rows in shared memory as B wants them: every run of eight columns in the order (0,4)
// (1,5)/16 (2,6) (3,7)/16, times 2^(GV_TOP - e) with e the exponent of the row's largest finite
// element; zeros beyond K, and GV_ZERO of them behind. gsum: -8 times the sum of each group, in
// the units of the products (FEW: [token][group], else [group][token]). exps[t] = e.
template <bool FEW, int TOK>
__device__ __forceinline__ void stage_x(const GemvParams& p, int stride, unsigned char* xs, float* gsum, int* exps) {
    const int runs = (stride - GV_PAD) / 16;  // a multiple of 32: a warp's lanes are in one row
    for (int i = threadIdx.x; i < TOK; i += blockDim.x) exps[i] = 0;
    if (threadIdx.x < GV_ZERO / 16)
        *reinterpret_cast<uint4*>(xs + size_t(p.T) * stride + 16 * threadIdx.x) = make_uint4(0u, 0u, 0u, 0u);
    if (!FEW) {  // absent tokens
        for (int i = threadIdx.x; i < runs / 4 * TOK; i += blockDim.x)
            if (i % TOK >= p.T) gsum[i] = 0.0f;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * runs; i += blockDim.x) {
        const int t = i / runs, r = i - t * runs;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (8 * r < p.K) v = __ldg(reinterpret_cast<const uint4*>(p.x + size_t(t) * p.K + 8 * r));
        *reinterpret_cast<uint4*>(xs + size_t(t) * stride + 16 * r) = v;
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t top = 0;  // largest magnitude as a bit pattern; infinities and NaN do not count
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
            if (lo < 0x7f80u) top = max(top, lo);
            if (hi < 0x7f80u) top = max(top, hi);
        }
        top = __reduce_max_sync(FULL, top);
        if ((threadIdx.x & 31) == 0) atomicMax(&exps[t], int(top));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * runs; i += blockDim.x) {
        const int t = i / runs, r = i - t * runs;
        // the scale 2^(GV_TOP - e) as two factors: e is -126 .. 127 (rows of subnormals: -126)
        const int e = max(exps[t] >> 7, 1) - 127, up = GV_TOP - e;
        const float f0 = __int_as_float((127 + up / 2) << 23), f1 = __int_as_float((127 + up - up / 2) << 23);
        const uint4 v = *reinterpret_cast<const uint4*>(xs + size_t(t) * stride + 16 * r);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float f[8], s = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = bf16lo(w[j]) * f0 * f1;
            f[2 * j + 1] = bf16hi(w[j]) * f0 * f1;
            s += f[2 * j] * 0x1p-64f + f[2 * j + 1] * 0x1p-64f;
        }
        s += __shfl_xor_sync(FULL, s, 1);
        s += __shfl_xor_sync(FULL, s, 2);
        const float k = 0.0625f;
        auto pair = [](float lo, float hi) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
            return *reinterpret_cast<const uint32_t*>(&h);
        };
        *reinterpret_cast<uint4*>(xs + size_t(t) * stride + 16 * r) =
            make_uint4(pair(f[0], f[4]), pair(f[1] * k, f[5] * k), pair(f[2], f[6]), pair(f[3] * k, f[7] * k));
        if ((r & 3) == 0) gsum[FEW ? t * (runs / 4) + r / 4 : (r / 4) * TOK + t] = s * -0x1p-66f;  // -8 2^(64 - 133)
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.T; i += blockDim.x) exps[i] = max(exps[i] >> 7, 1) - 127;
    __syncthreads();
}

// Position in a warp's share of steps, with the lane's first address there: eight lanes read 128
// bytes of a row, lane l chunk l % 8 of rows l / 8 + 4 j.
struct Cursor {
    const uint8_t* w;
    const uint16_t* sc;  // scales of row lane % 16
    int tile, s;
    __device__ __forceinline__ void at(const GemvParams& p, int tile_, int s_, int lane) {
        tile = tile_;
        s = s_;
        w = p.w + size_t(tile * 16 + lane / 8) * (p.K / 2) + size_t(s) * (GV_COLS / 2) + 16 * (lane % 8);
        sc = p.s + size_t(tile * 16 + lane % 16) * (p.K / 32) + s * (GV_COLS / 32);
    }
    __device__ __forceinline__ void next(const GemvParams& p, int steps, int lane) {
        w += GV_COLS / 2;
        sc += GV_COLS / 32;
        if (++s == steps) at(p, tile + 1, 0, lane);
    }
};

// Ask for one step. Rows beyond N and columns beyond K keep what the slot holds: any code is
// finite and meets a zero x or an output that is not stored. Scales beyond K are zeroed (what
// lies there need not be finite). WHOLE: K % 256 == 0, a row's scales of a step are 16 bytes.
template <bool WHOLE>
__device__ __forceinline__ void fetch(const GemvParams& p, const Cursor& c, int lane, unsigned char* slot) {
    const uint32_t dst = smem_u32(slot) + (lane / 8) * GV_WROW + 16 * (lane % 8);
    const int groups = p.K / 32 - c.s * (GV_COLS / 32);  // groups left in the row
    const size_t step4 = size_t(p.K) * 2;  // bytes of four rows
    if (WHOLE || lane % 8 < groups) {
        if (c.tile * 16 + 16 <= p.N) {
#pragma unroll
            for (int j = 0; j < 4; ++j) cp_async16(dst + 4 * j * GV_WROW, c.w + j * step4);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c.tile * 16 + lane / 8 + 4 * j < p.N) cp_async16(dst + 4 * j * GV_WROW, c.w + j * step4);
        }
    }
    unsigned char* ss = slot + 16 * GV_WROW + (lane % 16) * GV_SROW;
    if (c.tile * 16 + lane % 16 < p.N) {
        if (WHOLE) {
            if (lane < 16) cp_async16(smem_u32(ss), c.sc);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = 4 * (lane / 16) + i;
                reinterpret_cast<uint16_t*>(ss)[k] = k < groups ? __ldg(c.sc + k) : uint16_t(0);
            }
        }
    }
}

// One or two tokens, 16 rows by 256 columns: lane (g, q) reads chunk q + 4 (g & 1) of rows
// g / 2 + 4 j. The rows g of an mma are a W row's first four groups (g even) and its last four
// (g odd): columns 2 q, 2 q + 1 of a lane's sums count where they are that half's.
// w: the lane's first chunk, s: the first row's scales, x: the lane's column of B (zeros in the
// lanes that hold other groups), xrow bytes from one token's to the next.
// gs: this lane's pair of group sums, grow floats from one token's to the next.
template <int TOK>
__device__ __forceinline__ void few_step(const unsigned char* w, const unsigned char* s, const unsigned char* x, int xrow,
                                         const float* gs, int grow, float (&acc)[4 * TOK]) {
    float cc[TOK][2][4];
    uint4 v[4];
    uint32_t sc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = *reinterpret_cast<const uint4*>(w + 4 * j * GV_WROW);
        sc[j] = *reinterpret_cast<const uint32_t*>(s + 4 * j * GV_SROW);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            const uint4 xv = *reinterpret_cast<const uint4*>(x + t * xrow + 16 * i);
            const float2 c = i == 0 ? *reinterpret_cast<const float2*>(gs + t * grow) : make_float2(0.0f, 0.0f);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 va = v[2 * h], vb = v[2 * h + 1];
                const uint32_t a = i == 0 ? va.x : i == 1 ? va.y : i == 2 ? va.z : va.w;
                const uint32_t b = i == 0 ? vb.x : i == 1 ? vb.y : i == 2 ? vb.z : vb.w;
                float(&d)[4] = cc[t][h];
                if (i == 0) mma_word(d, a, b, xv, c.x, c.y, c.x, c.y);
                else mma_word(d, a, b, xv, d[0], d[1], d[2], d[3]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float s0 = bf16lo(sc[j]), s1 = bf16hi(sc[j]);
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            const int k = 4 * t + j, c = 2 * (j & 1);
            acc[k] = fmaf(cc[t][j / 2][c], s0, fmaf(cc[t][j / 2][c + 1], s1, acc[k]));
        }
    }
}

// Eight NT tokens, 16 rows by 128 columns: lane (g, q) reads its quarter of the four groups of
// rows g and g + 8; x holds the lane's token of each block of eight, gs the group sums of the
// lane's two tokens of C in the first block.
template <int NT>
__device__ __forceinline__ void row_step(const unsigned char* w, const unsigned char* s, const unsigned char* const (&x)[NT],
                                         const float* gs, float (&acc)[4 * NT]) {
    const uint2 sa = *reinterpret_cast<const uint2*>(s), sb = *reinterpret_cast<const uint2*>(s + 8 * GV_SROW);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = *reinterpret_cast<const uint32_t*>(w + 16 * i);
        const uint32_t b = *reinterpret_cast<const uint32_t*>(w + 8 * GV_WROW + 16 * i);
        const uint32_t ua = i < 2 ? sa.x : sa.y, ub = i < 2 ? sb.x : sb.y;
        const float fa = i & 1 ? bf16hi(ua) : bf16lo(ua), fb = i & 1 ? bf16hi(ub) : bf16lo(ub);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint4 v = *reinterpret_cast<const uint4*>(x[nt] + 64 * i);
            const float2 c = *reinterpret_cast<const float2*>(gs + i * (8 * NT) + 8 * nt);
            float cc[4];
            mma_word(cc, a, b, v, c.x, c.y, c.x, c.y);
            acc[4 * nt + 0] = fmaf(cc[0], fa, acc[4 * nt + 0]);
            acc[4 * nt + 1] = fmaf(cc[1], fa, acc[4 * nt + 1]);
            acc[4 * nt + 2] = fmaf(cc[2], fb, acc[4 * nt + 2]);
            acc[4 * nt + 3] = fmaf(cc[3], fb, acc[4 * nt + 3]);
        }
    }
}

template <bool F32>
__device__ __forceinline__ void put(void* y, size_t i, float v) {
    if (F32) static_cast<float*>(y)[i] = v;
    else static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
}

// NT < 0: -NT tokens (one or two); otherwise NT blocks of eight. All of x in shared memory.
template <int NT, bool F32, bool WHOLE>
__global__ void __launch_bounds__(32 * GV_WARPS, 1) gemv_kernel(const GemvParams p) {
    extern __shared__ __align__(16) unsigned char sm[];
    constexpr bool FEW = NT <= 0;
    constexpr int TOK = FEW ? -NT : 8 * NT;
    constexpr int NA = FEW ? 4 * TOK : 4 * NT;  // sums a lane holds
    const int steps = (p.K + GV_COLS - 1) / GV_COLS, stride = row_stride(p.K);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int g = lane >> 2, q = lane & 3;
    unsigned char* xs = sm;
    unsigned char* zero = xs + size_t(p.T) * stride;
    int* exps = reinterpret_cast<int*>(zero + GV_ZERO);     // [TOK], in 128 bytes
    float* gsum = reinterpret_cast<float*>(exps + 32);      // [TOK][8 steps] or [8 steps][TOK]
    float* red = gsum + TOK * 8 * steps;                    // [warps][NA][32]
    unsigned char* ring = reinterpret_cast<unsigned char*>(red + warps * NA * 32) + warp * GV_RING;

    const int ntiles = (p.N + 15) / 16;
    const int ta = int((long long)ntiles * blockIdx.x / gridDim.x), tb = int((long long)ntiles * (blockIdx.x + 1) / gridDim.x);
    // at most 2^24 tiles over 148 blocks or more, of 256 steps: total * warps < 2^30
    const int total = (tb - ta) * steps;
    auto begin = [&](int w) { return total * w / warps; };
    const int za = begin(warp), zb = begin(warp + 1);

    Cursor in;
    in.at(p, ta + za / steps, za % steps, lane);
    int tile = in.tile, s = in.s, zin = za, sin = 0;
    auto ask = [&]() {  // one group per call, an empty one behind the last step
        if (zin < zb) {
            fetch<WHOLE>(p, in, lane, ring + sin);
            in.next(p, steps, lane);
            sin = sin + GV_SLOT == GV_RING ? 0 : sin + GV_SLOT;
            ++zin;
        }
        cp_commit();
    };
    #pragma unroll
    for (int i = 0; i < GV_SLOTS - 1; ++i) ask();
    stage_x<FEW, TOK>(p, stride, xs, gsum, exps);

    const int xrow = FEW && (g & 3) == q ? stride : 0;
    constexpr int NX = FEW ? 1 : NT;
    const unsigned char* x0[NX];
    int xstep[NX];  // bytes a step adds
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        const bool there = FEW ? (g & 3) == q : 8 * i + g < p.T;  // few tokens: this lane is its column's group
        x0[i] = (there ? xs + (FEW ? 64 * g : (8 * i + g) * stride) : zero) + (FEW ? 0 : 16 * q);
        xstep[i] = there ? 2 * GV_COLS : 0;
    }
    const unsigned char* my_w = ring + (FEW ? (lane / 8) * GV_WROW + 16 * (lane % 8) : g * GV_WROW + 4 * q);
    const unsigned char* my_s = ring + 16 * GV_WROW + (FEW ? (lane / 8) * GV_SROW + 4 * q : g * GV_SROW);
    const float* my_g = gsum + 2 * q;

    float acc[NA] = {};
    auto put_tile = [&](int tl, const float (&v)[NA]) {
        if constexpr (FEW) {
            const int m = lane % 8;  // the sums are in all eight lanes of a row: lane m stores sum m
            float u = v[0];
#pragma unroll
            for (int i = 1; i < NA; ++i) u = m == i ? v[i] : u;
            const int n = tl * 16 + lane / 8 + 4 * (m & 3), t = m >> 2;
            if (m < NA && n < p.N) put<F32>(p.y, size_t(t) * p.N + n, ldexpf(u, exps[t] + 133 - GV_TOP));
        } else {
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                const int t = 8 * (i / 4) + 2 * q + (i & 1), n = tl * 16 + g + 8 * ((i >> 1) & 1);
                if (t < p.T && n < p.N) put<F32>(p.y, size_t(t) * p.N + n, ldexpf(v[i], exps[t] + 133 - GV_TOP));
            }
        }
    };
    bool whole = s == 0;  // the segment at hand starts at its tile's first step
    auto finish = [&](bool ended) {
        if constexpr (FEW) {  // add the four lanes that hold the row's groups; the other four hold none of it
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                float v = (q >> 1) == (g & 1) ? acc[i] : 0.0f;
                v += __shfl_xor_sync(FULL, v, 1);
                v += __shfl_xor_sync(FULL, v, 2);
                acc[i] = v + __shfl_xor_sync(FULL, v, 4);
            }
        }
        if (whole && ended) put_tile(tile, acc);
        if (!whole) {
#pragma unroll
            for (int i = 0; i < NA; ++i) red[(warp * NA + i) * 32 + lane] = acc[i];
        }
    };
    int slot = 0;
    for (int z = za; z < zb; ++z) {
        cp_wait<GV_SLOTS - 2>();
        __syncwarp();
        const unsigned char *w = my_w + slot, *sc = my_s + slot;
        if constexpr (FEW) {
            few_step<TOK>(w, sc, x0[0] + s * xstep[0], xrow, my_g + 8 * s, 8 * steps, acc);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const unsigned char* xp[NX];
#pragma unroll
                for (int i = 0; i < NX; ++i) xp[i] = x0[i] + s * xstep[i] + h * (xstep[i] / 2);
                row_step<NT>(w + 64 * h, sc + 8 * h, xp, my_g + (8 * s + 4 * h) * TOK, acc);
            }
        }
        __syncwarp();  // the slot has been read
        ask();
        slot = slot + GV_SLOT == GV_RING ? 0 : slot + GV_SLOT;
        if (++s == steps) {
            finish(true);
            ++tile;
            s = 0;
            whole = true;
#pragma unroll
            for (int i = 0; i < NA; ++i) acc[i] = 0.0f;
        }
    }
    const bool open = zb > za && s != 0;  // the last segment ends inside its tile
    if (open) finish(false);
    __syncthreads();
    if (!open || !whole) return;
    // this warp has the tile's first steps: the rest lies with the warps behind it
    const int end = (tile - ta + 1) * steps;
    for (int w = warp + 1; w < warps && begin(w) < end; ++w) {
        if (begin(w) == begin(w + 1)) continue;
#pragma unroll
        for (int i = 0; i < NA; ++i) acc[i] += red[(w * NA + i) * 32 + lane];
    }
    put_tile(tile, acc);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
    return a && b && x < y + bn && y < x + an;
}

using GemvKernel = void (*)(GemvParams);

template <bool F32>
GemvKernel pick_gemv(int T, bool whole) {
    if (T == 1) return whole ? gemv_kernel<-1, F32, true> : gemv_kernel<-1, F32, false>;
    if (T == 2) return whole ? gemv_kernel<-2, F32, true> : gemv_kernel<-2, F32, false>;
    if (T <= 8) return whole ? gemv_kernel<1, F32, true> : gemv_kernel<1, F32, false>;
    if (T <= 16) return whole ? gemv_kernel<2, F32, true> : gemv_kernel<2, F32, false>;
    return whole ? gemv_kernel<4, F32, true> : gemv_kernel<4, F32, false>;
}

int kept(int T) { return T <= 2 ? T : (T <= 8 ? 8 : (T <= 16 ? 16 : 32)); }    // tokens
int sums(int T) { return T <= 2 ? 4 * T : (T <= 8 ? 4 : (T <= 16 ? 8 : 16)); }  // of a lane

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
    const bool f32 = y_dtype == DT_F32;
    const int tiles = (p.N + 15) / 16, stride = row_stride(p.K);
    // Token rows at a time: all, or as many as leave room for the shortest rings, in whole blocks of
    // eight if more than that. Each pass over W serves one such share.
    const int groups = (p.K + GV_COLS - 1) / GV_COLS * (GV_COLS / 32);
    auto fixed_bytes = [&](int n) {
        return n * stride + GV_ZERO + 128 + 4 * groups * kept(n) + GV_WARPS * sums(n) * 32 * 4;
    };
    int most = T;
    while (most > 1 && fixed_bytes(most) + 8 * GV_RING > di.max_smem_optin)
        most = most > 8 ? (most - 1) / 8 * 8 : most - 1;
    for (int t = 0; t < T; t += most) {
        p.T = T - t < most ? T - t : most;
        p.x = static_cast<const uint16_t*>(x) + size_t(t) * p.K;
        p.y = static_cast<char*>(y) + size_t(t) * p.N * (f32 ? 4 : 2);
        const int fixed = fixed_bytes(p.T), room = (di.max_smem_optin - fixed) / GV_RING;
        const int warps = room < GV_WARPS ? room : GV_WARPS;
        const int smem = fixed + warps * GV_RING;
        const GemvKernel kern = f32 ? pick_gemv<true>(p.T, p.K % GV_COLS == 0) : pick_gemv<false>(p.T, p.K % GV_COLS == 0);
        if (smem > 48 * 1024 &&
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return REDMOE_ERR_CUDA;
        kern<<<tiles < di.sm_count ? tiles : di.sm_count, 32 * warps, smem, static_cast<cudaStream_t>(stream)>>>(p);
        if (cudaGetLastError() != cudaSuccess) return REDMOE_ERR_CUDA;
    }
    return REDMOE_OK;
}
