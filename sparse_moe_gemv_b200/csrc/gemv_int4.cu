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
//   one row of x: the eight columns of B are eight groups. A lane holds one whole group (16 bytes)
//      of one row; column j of B is x in the lane slots of group j and zero in the others, so one
//      chain of eight products makes eight groups' sums of eight W rows.
//   more rows: the eight columns of B are eight tokens, and a lane holds its quarter (4 bytes) of
//      one group after the other.
//
// A step is 16 rows of W (a tile) by 256 columns. A block has a run of whole tiles, its warps
// equal shares of that run's steps; a tile whose steps fall to several warps is added up through
// shared memory in warp order, so results do not depend on timing. Each warp copies its steps
// into a ring of its own with asynchronous copies (128-byte lines asked for whole), so no warp
// waits for another until the end, and the loads in flight need no registers.
//
// Measured on a B200: 151936 x 2048 at one token 33.1 us (26.7 at the copy bandwidth; the steady rate
// is 93% of it, four to five us are the launch, x and the last steps). 24571 x 4096 at 13 tokens 23.9
// us (8.6): 60% of the copy bandwidth in the steady state, where the reads of x from shared memory
// keep that four fifths busy, and ten us for the launch, x (1.7 to fetch, 2.5 to shape) and the tail.
#include "common.cuh"
#include "internal.h"
#include "launch.h"

#include <cuda_bf16.h>

namespace redmoe {
namespace {

constexpr int GV_MAX_T = 32;
constexpr int GV_MAX_K = 65536;
constexpr int GV_COLS = 256;     // columns of a slice, the unit of x's layout
constexpr int GV_PAD = 64;       // bytes between token rows of x in shared memory (bank offset)
constexpr int GV_ZERO = 256;     // bytes of zeros: half a step of an absent token

struct GemvParams {
    const uint8_t* w;      // [N, K/2]
    const uint16_t* s;     // [N, K/32] bf16
    const uint16_t* x;     // [T, K] bf16
    void* y;               // [T, N]
    int N, K, T;
    int share;             // tokens of a row of blocks: row blockIdx.y has those from share * blockIdx.y on
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

// The exponent that a row's largest x is scaled to: the largest with room for its sums.
constexpr int GV_TOP = 126;

// How the block's warps share x's rows while it is prepared: `parts` warps a row (one, and several
// rows a warp, where there are more rows than warps), warp `part` of them on runs of eight columns
// 32 part + lane, + 32 parts, ...
struct RowShare {
    int parts, part, first, step;
    __device__ __forceinline__ explicit RowShare(int T) {
        const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
        parts = max(warps / T, 1);
        part = warps >= T ? warp / T : 0;
        first = warps >= T ? warp % T : warp;
        if (part >= parts) first = T;  // a warp too many
        step = warps >= T ? T : warps;
    }
};

// Ask for x's T rows in shared memory (zeros beyond K).
__device__ __forceinline__ void fetch_x(const GemvParams& p, const RowShare& sh, int stride, unsigned char* xs) {
    const int runs = (stride - GV_PAD) / 16, lane = threadIdx.x & 31;
    for (int t = sh.first; t < p.T; t += sh.step) {
#pragma unroll 4
        for (int r = 32 * sh.part + lane; r < runs; r += 32 * sh.parts) {
            unsigned char* dst = xs + t * stride + 16 * r;
            if (8 * r < p.K) cp_async16(smem_u32(dst), p.x + size_t(t) * p.K + 8 * r);
            else *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pow2_pair(int e) { return uint32_t(127 + e) * 0x00800080u; }  // bf16 (2^e, 2^e)

// Once this thread's part of fetch_x has arrived: x as B wants it. Every run of eight columns in
// the order (0,4) (1,5)/16 (2,6) (3,7)/16, times 2^(GV_TOP - e) with e the exponent of the row's
// largest element; exps[t] = e. gsum: -8 times the sum of each group in the units of the products
// (ONE: [group], else [group][token]), made by the products themselves with a tile of
// eights. tops: scratch, one word for each warp of each row.
template <bool ONE, int TOK>
__device__ __forceinline__ void shape_x(const GemvParams& p, const RowShare& sh, int stride, unsigned char* xs, const unsigned char* zero,
                                        float* gsum, int* exps, uint32_t* tops) {
    const int runs = (stride - GV_PAD) / 16, steps = runs / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    constexpr int BATCH = ONE ? 1 : 4;  // one token: hardly a run or a group for every warp
    for (int t = sh.first; t < p.T; t += sh.step) {  // the runs this thread asked for
        uint32_t m = 0;
#pragma unroll 4
        for (int r = 32 * sh.part + lane; r < runs; r += 32 * sh.parts) {
            const uint4 v = *reinterpret_cast<const uint4*>(xs + t * stride + 16 * r);
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                     __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
        }
        const uint32_t top = __reduce_max_sync(FULL, max(m & 0xffffu, m >> 16));
        if (lane == 0) tops[sh.part * p.T + t] = top;
    }
    __syncthreads();
    for (int t = sh.first; t < p.T; t += sh.step) {
        const uint32_t top = __reduce_max_sync(FULL, lane < sh.parts ? tops[lane * p.T + t] : 0u);
        // e is -126 (also for rows of subnormals) .. 128 (infinity or NaN); the scale as two factors
        const int e = max(int(top >> 7), 1) - 127, up = GV_TOP - e, f0 = up / 2, f1 = up - f0;
        const uint32_t a = pow2_pair(f0), b = pow2_pair(f1), c = pow2_pair(f1 - 4);
        uint4* row = reinterpret_cast<uint4*>(xs + t * stride);
        for (int r0 = 32 * sh.part + lane; r0 < runs; r0 += 32 * BATCH * sh.parts) {
            uint4 in[BATCH];  // several at a time: in place, a load would wait for the store before it
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (r0 + 32 * i * sh.parts < runs) in[i] = row[r0 + 32 * i * sh.parts];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const uint4 v = in[i];
                if (r0 + 32 * i * sh.parts < runs)
                    row[r0 + 32 * i * sh.parts] =
                        make_uint4(mul2(mul2(__byte_perm(v.x, v.z, 0x5410), a), b), mul2(mul2(__byte_perm(v.x, v.z, 0x7632), a), c),
                                   mul2(mul2(__byte_perm(v.y, v.w, 0x5410), a), b), mul2(mul2(__byte_perm(v.y, v.w, 0x7632), a), c));
            }
        }
        if (lane == 0 && sh.part == 0) exps[t] = e;
    }
    __syncthreads();
    constexpr int NB = ONE ? 1 : TOK / 8;  // blocks of eight tokens
    const int g = lane >> 2, q = lane & 3;
    for (int i = warp; i < 8 / BATCH * steps * NB; i += warps) {  // groups of a block of eight tokens
        const int first = BATCH * (i / NB), t0 = 8 * (i % NB);
        const unsigned char* from = (t0 + g < p.T ? xs + (t0 + g) * stride + 64 * first : zero) + 16 * q;
        const int next = t0 + g < p.T ? 64 : 0;
        uint4 x[BATCH];
        float d[BATCH][4];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) x[j] = *reinterpret_cast<const uint4*>(from + j * next);
#pragma unroll
        for (int j = 0; j < BATCH; ++j) mma_word(d[j], 0x88888888u, 0x88888888u, x[j], 0.0f, 0.0f, 0.0f, 0.0f);
        if (g == 0) {  // every row of the sums is the same; this lane has tokens t0 + 2 q and the next
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                if (!ONE) *reinterpret_cast<float2*>(gsum + (first + j) * TOK + t0 + 2 * q) = make_float2(-d[j][0], -d[j][1]);
                else if (q == 0) gsum[first + j] = -d[j][0];
            }
        }
    }
    __syncthreads();
}

// What a pass over NT blocks of eight tokens, or (NT = 0) over one token, uses. Two tokens already
// take the block of eight: 18.5 us where a kernel for two like the one for one took 20.6 (24571 x
// 4096). Each number against its neighbours, in us, the two sides of a choice in one state of the kernel (later
// steps moved both: compare within a line only):
//   M      two tiles a step up to eight tokens, see two_tiles; with more blocks of eight, steps of two
//          tiles of 256 or 128 columns take 31.9 and 29.7, one tile 24.5 (T = 13, 24571 x 4096)
//   WARPS  20 and 16: 34.2 (T = 1, 151936 x 2048) and 16.4 (T = 4); 12 warps 37.8 and 18.0
//   COLS   512 at one token 35.1 (151936 x 2048), 256 37.5
//   SLOTS  2: 34.2, 16.4, 24.4, 26.3 us (T = 1, 4, 13; T = 32 at 24571 x 2048), 3: 36.8, 17.7, 26.5,
//          30.2: what a third slot asks for first costs more than the second leaves open
template <int NT, int M_ = 1> struct Plan {
    static constexpr bool ONE = NT == 0;
    static constexpr int TOK = ONE ? 1 : 8 * NT;    // tokens that sums are kept for
    static constexpr int M = M_;                    // tiles of 16 rows in a step: x is read once for them
    static constexpr int WARPS = ONE ? 20 : 16;                    // at most
    static constexpr int ROWS = 16 * M;
    static constexpr int COLS = ONE ? 512 : 256;    // columns of a step: one or two slices
    static constexpr int WROW = COLS / 2 + 16;      // bytes of a slot's row of W (bank offset)
    static constexpr int SROW = COLS / 16;          // bytes of a slot's row of scales
    static constexpr int NA = M * 4 * (ONE ? 1 : NT);              // sums a lane holds
    static constexpr int SLOTS = 2;                                // of a warp's ring
    static constexpr int SLOT = ROWS * (WROW + SROW);
    static constexpr int WARP_BYTES = SLOTS * SLOT + NA * 32 * 4;  // shared memory of a warp
    static constexpr int fixed_bytes(int T, int K) {               // and of a block besides
        return T * row_stride(K) + GV_ZERO + 128 + 128 + 4 * 8 * TOK * ((K + GV_COLS - 1) / GV_COLS);
    }
};

// Eight scales of a row that starts anywhere, as the two aligned 16-byte pieces that hold them (a load for
// each scale takes 26.0 and 22.4 us where this takes 22.4 and 20.6, 24571 x 4064 at T = 4 and 1).
struct Scales {
    uint4 a, b;
    int first, need;  // where the eight begin in a, in scales; how many of them count (the others are zero)
    __device__ __forceinline__ void load(const GemvParams& p, size_t i) {
        const size_t end = size_t(p.N) * (p.K / 32), from = i & ~size_t(7);
        if (from + 16 <= end) {
            first = int(i - from);
            const uint4* q = reinterpret_cast<const uint4*>(p.s + from);
            a = q[0];
            b = q[1];
        } else {  // the matrix's last scales, one at a time
            uint32_t w[4] = {};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < need) w[k / 2] |= uint32_t(p.s[i + k]) << 16 * (k & 1);
            first = 0;
            a = make_uint4(w[0], w[1], w[2], w[3]);
            b = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    __device__ __forceinline__ uint4 get() const {
        uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int k = 0; k < 6; ++k) w[k] = first & 4 ? w[k + 2] : w[k];
#pragma unroll
        for (int k = 0; k < 5; ++k) w[k] = first & 2 ? w[k + 1] : w[k];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[k] = __funnelshift_r(w[k], w[k + 1], 16 * (first & 1));
            w[k] = need >= 2 * k + 2 ? w[k] : need == 2 * k + 1 ? w[k] & 0xffffu : 0u;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Position in a warp's share of steps, with the lane's first address there: eight lanes read 128
// bytes of a row, lane l chunk l % 8 of rows l / 8 + 4 j.
template <class P>
struct Cursor {
    const uint8_t* w;
    const uint16_t* sc;
    int tile, s;
    __device__ __forceinline__ void at(const GemvParams& p, int tile_, int s_, int lane) {
        tile = tile_;
        s = s_;
        w = p.w + size_t(tile * P::ROWS + lane / 8) * (p.K / 2) + size_t(s) * (P::COLS / 2) + 16 * (lane % 8);
        sc = p.s + size_t(tile * P::ROWS + lane % P::ROWS) * (p.K / 32) + s * (P::COLS / 32);
    }
    __device__ __forceinline__ void next(const GemvParams& p, int steps, int lane) {
        w += P::COLS / 2;
        sc += P::COLS / 32;
        if (++s == steps) at(p, tile + 1, 0, lane);
    }
};

// Ask for one step. Rows beyond N and columns beyond K keep what the slot holds: any code is
// finite and meets a zero x or an output that is not stored. Scales beyond K are not used (whole
// slices) or zeroed: what lies there need not be finite. WHOLE: K % 256 == 0, a row's scales of a
// slice are 16 bytes.
template <bool WHOLE, class P>
__device__ __forceinline__ void fetch(const GemvParams& p, const Cursor<P>& c, int lane, unsigned char* slot,
                                      Scales& later) {
    constexpr int SLICES = P::COLS / GV_COLS;
    const uint32_t dst = smem_u32(slot) + (lane / 8) * P::WROW + 16 * (lane % 8);
    const int groups = p.K / 32 - c.s * (P::COLS / 32);  // groups left in the row
    const size_t step4 = size_t(p.K) * 2;                // bytes of four rows
    const bool full = c.tile * P::ROWS + P::ROWS <= p.N;
#pragma unroll
    for (int h = 0; h < SLICES; ++h) {
        if (WHOLE ? h > 0 && groups <= 8 * h : groups <= 8 * h + lane % 8) continue;
        if (full) {
#pragma unroll
            for (int j = 0; j < P::ROWS / 4; ++j) cp_async16(dst + 4 * j * P::WROW + 128 * h, c.w + j * step4 + 128 * h);
        } else {
#pragma unroll
            for (int j = 0; j < P::ROWS / 4; ++j)
                if (c.tile * P::ROWS + lane / 8 + 4 * j < p.N)
                    cp_async16(dst + 4 * j * P::WROW + 128 * h, c.w + j * step4 + 128 * h);
        }
    }
    const int h = lane / P::ROWS;  // lane: slice h of row lane % ROWS
    const bool there = h < SLICES && groups > 8 * h && (full || c.tile * P::ROWS + lane % P::ROWS < p.N);
    if constexpr (WHOLE) {
        if (there) cp_async16(smem_u32(slot + P::ROWS * P::WROW + (lane % P::ROWS) * P::SROW) + 16 * h, c.sc + 8 * h);
    } else {
        later.need = there ? groups - 8 * h : 0;
        if (there) later.load(p, size_t(c.sc - p.s) + 8 * h);
    }
}
// The scales that fetch left in registers, when their step begins.
template <class P>
__device__ __forceinline__ void settle(int lane, unsigned char* slot, const Scales& later) {
    if (lane < P::ROWS * (P::COLS / GV_COLS))
        *reinterpret_cast<uint4*>(slot + P::ROWS * P::WROW + (lane % P::ROWS) * P::SROW + 16 * (lane / P::ROWS)) = later.get();
}

// One token, 16 rows by 256 columns: lane (g, q) reads chunk q + 4 (g & 1) of rows g / 2 + 4 j. The
// rows g of an mma are a W row's first four groups (g even) and its last four (g odd): columns
// 2 q, 2 q + 1 of a lane's sums count where they are that half's.
// w: the lane's first chunk, s: the first row's scales; `release` is called once they are read.
// x: the lane's column of B (zeros in the lanes that hold other groups). gs: its two group sums.
template <class P, class Release>
__device__ __forceinline__ void one_step(const unsigned char* w, const unsigned char* s, Release release,
                                         const unsigned char* x, const float* gs, float (&acc)[4]) {
    uint4 v[4];
    uint32_t sc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint4*>(w + 4 * j * P::WROW);
#pragma unroll
    for (int j = 0; j < 4; ++j) sc[j] = *reinterpret_cast<const uint32_t*>(s + 4 * j * P::SROW);
    release();
    float cc[2][4];
    const float2 c = *reinterpret_cast<const float2*>(gs);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 xv = *reinterpret_cast<const uint4*>(x + 16 * i);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 va = v[2 * h], vb = v[2 * h + 1];
            const uint32_t a = i == 0 ? va.x : i == 1 ? va.y : i == 2 ? va.z : va.w;
            const uint32_t b = i == 0 ? vb.x : i == 1 ? vb.y : i == 2 ? vb.z : vb.w;
            float(&d)[4] = cc[h];
            if (i == 0) mma_word(d, a, b, xv, c.x, c.y, c.x, c.y);
            else mma_word(d, a, b, xv, d[0], d[1], d[2], d[3]);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int e = 2 * (j & 1);
        acc[j] = fmaf(cc[j / 2][e], bf16lo(sc[j]), fmaf(cc[j / 2][e + 1], bf16hi(sc[j]), acc[j]));
    }
}

// Eight NT tokens, M tiles of 16 rows by 128 columns: lane (g, q) reads its quarter of the four
// groups of rows g and g + 8; x holds the lane's token of each block of eight, gs the group sums
// that the lane's part of C starts with in the first block.
template <class P, int NT, int M, class Release>
__device__ __forceinline__ void row_step(const unsigned char* w, const unsigned char* s, Release release,
                                         const unsigned char* const (&x)[NT], const float* gs, float (&acc)[4 * NT * M]) {
    uint2 sc[2 * M];
    uint32_t w4[4][2 * M];
#pragma unroll
    for (int m = 0; m < 2 * M; ++m) sc[m] = *reinterpret_cast<const uint2*>(s + 8 * m * P::SROW);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < 2 * M; ++m) w4[i][m] = *reinterpret_cast<const uint32_t*>(w + 8 * m * P::WROW + 16 * i);
    release();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t(&v)[2 * M] = w4[i];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint4 xv = *reinterpret_cast<const uint4*>(x[nt] + 64 * i);
            const float2 c = *reinterpret_cast<const float2*>(gs + i * (8 * NT) + 8 * nt);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const uint32_t ua = i < 2 ? sc[2 * m].x : sc[2 * m].y, ub = i < 2 ? sc[2 * m + 1].x : sc[2 * m + 1].y;
                const float fa = i & 1 ? bf16hi(ua) : bf16lo(ua), fb = i & 1 ? bf16hi(ub) : bf16lo(ub);
                float cc[4];
                mma_word(cc, v[2 * m], v[2 * m + 1], xv, c.x, c.y, c.x, c.y);
                float* to = acc + 4 * (m * NT + nt);
                const float2 u = __ffma2_rn(make_float2(cc[0], cc[1]), make_float2(fa, fa), make_float2(to[0], to[1]));
                const float2 v2 = __ffma2_rn(make_float2(cc[2], cc[3]), make_float2(fb, fb), make_float2(to[2], to[3]));
                to[0] = u.x; to[1] = u.y; to[2] = v2.x; to[3] = v2.y;
            }
        }
    }
}

template <bool F32>
__device__ __forceinline__ void put(void* y, size_t i, float v) {
    if (F32) static_cast<float*>(y)[i] = v;
    else static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
}

// NT = 0: one token; otherwise NT blocks of eight. All of x in shared memory.
template <int NT, int M, bool F32, bool WHOLE>
__global__ void __launch_bounds__(32 * Plan<NT, M>::WARPS, 1) gemv_kernel(GemvParams p) {
    extern __shared__ __align__(16) unsigned char sm[];
    using P = Plan<NT, M>;
    constexpr bool ONE = P::ONE;
    constexpr int TOK = P::TOK, NA = P::NA, ROWS = P::ROWS, RING = P::SLOTS * P::SLOT;
    p.x += size_t(blockIdx.y) * p.share * p.K;
    p.y = static_cast<char*>(p.y) + size_t(blockIdx.y) * p.share * p.N * (F32 ? 4 : 2);
    p.T = min(p.share, p.T - int(blockIdx.y) * p.share);
    const int steps = (p.K + P::COLS - 1) / P::COLS, slices = (p.K + GV_COLS - 1) / GV_COLS, stride = row_stride(p.K);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int g = lane >> 2, q = lane & 3;
    unsigned char* xs = sm;
    unsigned char* zero = xs + size_t(p.T) * stride;
    int* exps = reinterpret_cast<int*>(zero + GV_ZERO);     // [TOK], in 128 bytes
    float* gsum = reinterpret_cast<float*>(exps + 32);      // [8 slices] or [8 slices][TOK]
    uint32_t* tops = reinterpret_cast<uint32_t*>(gsum + TOK * 8 * slices);  // 128 bytes
    float* red = reinterpret_cast<float*>(tops + 32);                      // [warps][NA][32]
    unsigned char* ring = reinterpret_cast<unsigned char*>(red + warps * NA * 32) + warp * RING;

    const int ntiles = (p.N + ROWS - 1) / ROWS;
    const int ta = int((long long)ntiles * blockIdx.x / gridDim.x), tb = int((long long)ntiles * (blockIdx.x + 1) / gridDim.x);
    // at most 2^24 tiles over 148 blocks or more, of 256 steps: total < 2^25
    const int total = (tb - ta) * steps, each = total / warps, more = total - each * warps;
    auto begin = [&](int w) { return w * each + min(w, more); };
    const int za = begin(warp), zb = begin(warp + 1);

    Cursor<P> in;
    in.at(p, ta + za / steps, za % steps, lane);
    int tile = in.tile, s = in.s, zin = za, sin = 0;
    static_assert(P::SLOTS == 2, "`later` is one step's");
    Scales later;
    auto ask = [&]() {  // one group per call, an empty one behind the last step
        if (zin < zb) {
            fetch<WHOLE, P>(p, in, lane, ring + sin, later);
            in.next(p, steps, lane);
            sin = sin + P::SLOT == RING ? 0 : sin + P::SLOT;
            ++zin;
        }
        cp_commit();
    };
    wait_for_previous();
    let_next_start();
    const RowShare share(p.T);
    fetch_x(p, share, stride, xs);
    cp_commit();
#pragma unroll
    for (int i = 0; i < P::SLOTS - 1; ++i) ask();
    if (threadIdx.x < GV_ZERO / 16) reinterpret_cast<uint4*>(zero)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
    cp_wait<P::SLOTS - 1>();
    shape_x<ONE, TOK>(p, share, stride, xs, zero, gsum, exps, tops);

    constexpr int NX = ONE ? 1 : NT;
    const unsigned char* x0[NX];
    int xstep[NX];  // bytes a step adds
#pragma unroll
    for (int i = 0; i < NX; ++i) {  // one token: zeros 32 bytes on, in other banks than x's (33.1 against 34.3 us, as above)
        const bool there = ONE ? (g & 3) == q : 8 * i + g < p.T;  // one token: this lane is its column's group
        x0[i] = there ? xs + (ONE ? 64 * g : (8 * i + g) * stride + 16 * q) : zero + (ONE ? 32 : 16 * q);
        xstep[i] = there ? 2 * P::COLS : 0;
    }
    const unsigned char* my_w = ring + (ONE ? (lane / 8) * P::WROW + 16 * (lane % 8) : g * P::WROW + 4 * q);
    const unsigned char* my_s = ring + ROWS * P::WROW + (ONE ? (lane / 8) * P::SROW + 4 * q : g * P::SROW);
    const float* my_g = gsum + 2 * q;

    float acc[NA] = {};
    auto put_tile = [&](int tl, const float (&v)[NA]) {
        if constexpr (ONE) {  // the sums are in all eight lanes of a row: lane m stores sum m
            const int m = lane % 8, n = tl * ROWS + lane / 8 + 4 * m;
            const float u = m == 0 ? v[0] : m == 1 ? v[1] : m == 2 ? v[2] : v[3];
            if (m < 4 && n < p.N) put<F32>(p.y, n, ldexpf(u, exps[0] + 133 - GV_TOP));
        } else {
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                const int t = 8 * (i / 4 % NT) + 2 * q + (i & 1), n = tl * ROWS + 16 * (i / (4 * NT)) + g + 8 * ((i >> 1) & 1);
                if (t < p.T && n < p.N) put<F32>(p.y, size_t(t) * p.N + n, ldexpf(v[i], exps[t] + 133 - GV_TOP));
            }
        }
    };
    bool whole = s == 0;  // the segment at hand starts at its tile's first step
    auto finish = [&](bool ended) {
        if constexpr (ONE) {  // add the four lanes that hold the row's groups; the other four hold none of it
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
        cp_wait<P::SLOTS - 2>();
        if (!WHOLE) settle<P>(lane, ring + slot, later);
        __syncwarp();
        const unsigned char *w = my_w + slot, *sc = my_s + slot;
        auto release = [&]() {
            __syncwarp();  // the slot has been read
            ask();
        };
        if constexpr (ONE) {
            const unsigned char* x = x0[0] + s * xstep[0];
            const float* gs = my_g + 16 * s;
            const bool two = (2 * s + 1) * GV_COLS < p.K;
            one_step<P>(w, sc, [&]() { if (!two) release(); }, x, gs, acc);
            if (two) one_step<P>(w + 128, sc + 16, release, x + xstep[0] / 2, gs + 8, acc);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const unsigned char* xp[NX];
#pragma unroll
                for (int i = 0; i < NX; ++i) xp[i] = x0[i] + s * xstep[i] + h * (xstep[i] / 2);
                row_step<P, NT, M>(w + 64 * h, sc + 8 * h, [&]() { if (h == 1) release(); }, xp, my_g + (8 * s + 4 * h) * TOK, acc);
            }
        }
        slot = slot + P::SLOT == RING ? 0 : slot + P::SLOT;
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

// Every p.share tokens a pass over W.
template <int NT, int M, bool F32, bool WHOLE>
bool launch_gemv(const GemvParams& p, const DevInfo& di, cudaStream_t stream) {
    using P = Plan<NT, M>;
    const int fixed = P::fixed_bytes(p.share, p.K), room = (di.max_smem_optin - fixed) / P::WARP_BYTES;
    const int warps = room < P::WARPS ? room : P::WARPS, smem = fixed + warps * P::WARP_BYTES;
    const auto kern = gemv_kernel<NT, M, F32, WHOLE>;
    if (!allow_smem(reinterpret_cast<const void*>(kern), smem)) return false;
    const int tiles = (p.N + P::ROWS - 1) / P::ROWS;
    const dim3 grid(tiles < di.sm_count ? tiles : di.sm_count, (p.T + p.share - 1) / p.share);
    return launch(kern, grid, 32 * warps, smem, stream, 1, p);
}

// Whether up to eight tokens take steps of two tiles: where all warps' rings fit beside x (24571 x
// 4096: 16.1, 16.3, 16.8 us at T = 2, 4, 5, one tile 16.5, 17.3, 17.9; but 18.5, 18.3, 19.6 against
// 18.1, 18.2, 18.3 at T = 6, 7, 8, which leave 15, 14, 13 warps), where blocks have more than one such
// step's rows (4736 x 4096: 8.1 against 7.7 us at T = 4) and where the coarser shares give none a tenth
// more rows (2048 x 4096, 32 instead of 16: 7.7 against 6.7 us at T = 4).
bool two_tiles(const GemvParams& p, const DevInfo& di) {
    using P = Plan<1, 2>;
    if (P::fixed_bytes(p.share, p.K) + P::WARPS * P::WARP_BYTES > di.max_smem_optin) return false;
    const int t1 = (p.N + 15) / 16, t2 = (p.N + 31) / 32, sms = di.sm_count;
    return t2 > sms && 20 * ((t2 + sms - 1) / sms) <= 11 * ((t1 + sms - 1) / sms);
}

// Whether T tokens of K columns leave room for eight warps' rings. Eight warps are slower than sixteen
// but faster than two passes (24571 x 5120 at T = 16: 39.1 us, as two passes of eight 41.9), six no
// longer (x 5376: 48.6 and 44.1).
bool fits(int T, int K, int smem) {
    const int need = T == 1    ? Plan<0>::fixed_bytes(T, K) + 8 * Plan<0>::WARP_BYTES
                     : T <= 8  ? Plan<1>::fixed_bytes(T, K) + 8 * Plan<1>::WARP_BYTES
                     : T <= 16 ? Plan<2>::fixed_bytes(T, K) + 8 * Plan<2>::WARP_BYTES
                               : Plan<4>::fixed_bytes(T, K) + 8 * Plan<4>::WARP_BYTES;
    return need <= smem;
}

template <bool F32, bool WHOLE>
bool launch_tokens(const GemvParams& p, const DevInfo& di, cudaStream_t s) {
    if (p.share == 1) return launch_gemv<0, 1, F32, WHOLE>(p, di, s);
    if (p.share <= 8) return two_tiles(p, di) ? launch_gemv<1, 2, F32, WHOLE>(p, di, s) : launch_gemv<1, 1, F32, WHOLE>(p, di, s);
    if (p.share <= 16) return launch_gemv<2, 1, F32, WHOLE>(p, di, s);
    return launch_gemv<4, 1, F32, WHOLE>(p, di, s);
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
    // Token rows at a time: all, or an equal share of them that leaves room for eight rings. A matrix of few
    // rows leaves multiprocessors free: as many shares as these can take at once (512 x 2048: 4.2 us at
    // T = 8, all in one share 4.5, at T = 32 4.6 and 10.6; 512 x 7040 at T = 32 10.5, in turn 48.9).
    p.T = T;
    p.x = static_cast<const uint16_t*>(x);
    p.y = y;
    const int tiles = (p.N + 15) / 16, free = di.sm_count / tiles;
    int n = free > 1 ? (free < T ? free : T) : 1;
    while (p.share = (T + n - 1) / n, p.share > 1 && !fits(p.share, p.K, di.max_smem_optin)) ++n;
    const bool f32 = y_dtype == DT_F32, whole = p.K % GV_COLS == 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool ok = f32 ? (whole ? launch_tokens<true, true>(p, di, st) : launch_tokens<true, false>(p, di, st))
                        : (whole ? launch_tokens<false, true>(p, di, st) : launch_tokens<false, false>(p, di, st));
    return ok ? REDMOE_OK : REDMOE_ERR_CUDA;
}
