// Per-expert counts, the balance loss and the z loss of a router's rows, and the gradient of
// both losses with respect to the logits.
//
// Of the T rows those count whose mask byte is not zero (no mask: all) and whose logits are
// not all -infinity; n is their number. Over them, with p = softmax(logits):
//   counts[e] = entries of topk_ids that name expert e (ids outside 0 .. E-1 name none)
//   P[e]      = (1/n) sum_t p[t, e]
//   loss[0]   = E sum_e counts[e] / (n k) P[e]         balance: 1 when both are uniform
//   loss[1]   = (1/n) sum_t logsumexp(logits[t])^2     z
// and with the counts held constant (a selection has no gradient), g = d / d loss:
//   d logits[t, e] = g0 E / (n^2 k) p[t, e] (counts[e] - sum_j p[t, j] counts[j])
//                  + g1 (2 / n) lse[t] p[t, e]
// The counts enter less floor(n k / E), the whole number below their mean: the difference in
// brackets is the same (p sums to 1) and even counts leave no rounding behind.
//
// Both directions are bound by memory: the logits are read once (forward) or read and written
// once (backward), rows that do not count are not read. A warp takes a row, or eight lanes of it where
// a row is short (up to 128 columns), a lane the same columns of every row, so the column sums of P
// stay in registers until the warp's rows are done. Rows are copied ahead into a ring of the warp's
// in shared memory as the flat byte range that they are, whole 16-byte pieces whatever E is (short
// and 16-bit rows need several in flight for full bandwidth). Forward, every block leaves its sums in
// the workspace and a second kernel, one cluster that waits where the first one ends, adds them: the
// last block of the first kernel doing that took 6 to 10 us behind fences and a counter, this takes
// 3. Measured on a B200: forward 65536 x 512 fp32 31.6 us (66% of the copy bandwidth, the exponentials and
// sums of 33 million values beside the launch of two kernels), 2048 x 512 9.6 us; backward 32768 x 512
// fp32 24 us (85%), in bf16 and a fifth masked 15.6 (59%: about six of them are launch, mask and first rows, the
// rows themselves run at 93%). Sums over rows are made in a fixed order (fp32 over a lane's rows, then warps and
// blocks: T / 9472 rows a lane up to 128 columns, T / 2368 at most beyond), counts are integers: results do not
// depend on timing.
#include "common.cuh"
#include "internal.h"
#include "launch.h"
#include "vec8.cuh"

namespace redmoe {
namespace {

constexpr int BAL_WARPS = 16;           // of a block, where no more are named
constexpr int BAL_WARPS_MID = 24;       // forward, rows of 129 .. 512 columns
constexpr int BAL_CLUSTER = 8;         // blocks of the second kernel
constexpr int BAL_MAX_BLOCKS = 160;    // of the first: one an SM
__host__ __device__ constexpr int padded(int E) { return (E + 3) & ~3; }  // a row of sums in the workspace

// A row lies over its LPR lanes in chunks of VEC consecutive values, chunk l + LPR i for lane l. VEC > 1
// needs E % VEC == 0 (whole 16-byte chunks in every row), VEC == 1 takes any E.

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}
__device__ __forceinline__ float2 all2(float a) { return make_float2(a, a); }

// v[] becomes exp(v - max) and z their sum over the row; returns the maximum. A row that holds a NaN
// comes out NaN whole; one of -infinity throughout (`any` false) comes out zero, with z = 0. Rounding
// the exponent makes exp(v - max) off by about |v - max| units, least where the probability is large.
template <int N2, int LPR>
__device__ __forceinline__ float row_exp(float2 (&v)[N2], float& z, bool& any) {
    float m = max_nan(v[0].x, v[0].y);
#pragma unroll
    for (int i = 1; i < N2; ++i) m = max_nan(m, max_nan(v[i].x, v[i].y));
    if constexpr (LPR == 32) {
        asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(m));
    } else {
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(FULL, m, o));
    }
    any = m != __uint_as_float(0xff800000u);
    if (!any) m = 0.0f;
    float2 s = all2(0.0f);
#pragma unroll
    for (int i = 0; i < N2; ++i) {
        const float2 d = __fmul2_rn(__fadd2_rn(v[i], all2(-m)), all2(LOG2E));
        v[i] = make_float2(ex2(d.x), ex2(d.y));
        s = __fadd2_rn(s, v[i]);
    }
    z = row_sum<LPR>(s.x + s.y);
    return m;
}

// A warp's ring of row groups (RPW rows each) in shared memory. Rows of whole 16-byte chunks: each
// lane copies, and later reads, its own chunks of its own row. Others: the group's flat byte range
// with the pieces of 16 that it shares with its neighbours.
__host__ __device__ constexpr int flat_bytes(int rows, int E, int size) { return (rows * E * size + 30) / 16 * 16 + 16; }

template <int DT, int VEC, int NCH, int LPR>
struct Ring {
    static constexpr int SIZE = DT == DT_F32 ? 4 : 2, RPW = 32 / LPR;
    static constexpr bool FLAT = VEC == 1;
    const uint8_t* mask;
    const char* src;        // this lane's row (FLAT: the group's first) of the next group
    int T, chunks, depth, slot, step;
    int row;                // the lane's row of the next group to ask for
    size_t step_bytes;
    uint32_t base;
    int in, use;            // bytes from base
    unsigned lives;         // whether the lane's row counts, in the groups asked for: newest in bit 0
    unsigned bits, bits2;   // whether the lane's row counts in the LPR groups from the next on, and in those behind
    int pos, row2;          // place in `bits`; the row that this lane looks up next

    // The mask bytes of LPR groups, a lane each: one load for as many rows of the lane's own.
    __device__ __forceinline__ unsigned look() {
        bool m = row2 < T;
        if (m && mask) m = mask[row2];
        row2 += LPR * step;
        const unsigned all = __ballot_sync(FULL, m);
        return LPR == 32 ? all : (all >> ((threadIdx.x & 31) / LPR * LPR)) & ((1u << (LPR & 31)) - 1u);
    }
    __device__ __forceinline__ void start(const void* logits, const uint8_t* m, int T_, int E, int depth_, unsigned char* b,
                                          int t0, int step_) {
        const int lane = threadIdx.x & 31;
        mask = m;
        T = T_; depth = depth_; step = step_;
        chunks = FLAT ? E * SIZE : E / VEC;  // FLAT: bytes of a row
        slot = FLAT ? flat_bytes(RPW, E, SIZE) : NCH * 512;
        base = smem_u32(b);
        row = t0 + lane / LPR;
        src = static_cast<const char*>(logits) + size_t(FLAT ? t0 : row) * (size_t(E) * SIZE);
        step_bytes = size_t(step) * (size_t(E) * SIZE);
        in = use = 0;
        lives = 0;
        row2 = row + lane % LPR * step;
        pos = 0;
        bits = look();
        bits2 = look();
        for (int i = 0; i + 1 < depth; ++i) ask();
    }
    // One group of copies (nothing of rows that do not count).
    __device__ __forceinline__ void ask() {
        const int lane = threadIdx.x & 31, l = lane % LPR;
        const bool live = (bits >> pos) & 1u;
        const uint32_t dst = base + in + 16 * lane;
        if constexpr (FLAT) {
            if (__any_sync(FULL, live)) {
                const int off = int(reinterpret_cast<uintptr_t>(src) & 15u), rows = min(RPW, T - (row - lane / LPR));
                const int bytes = off + rows * chunks;
                const char* from = src - off + 16 * lane;
                for (int i = 16 * lane, d = 0; i < bytes; i += 512, d += 512)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                                 :: "r"(dst + d), "l"(from + d), "r"(min(bytes - i, 16)) : "memory");
            }
        } else if (live) {
#pragma unroll
            for (int i = 0; i < NCH; ++i)
                if (l + LPR * i < chunks)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                 :: "r"(dst + 512 * i), "l"(src + 16 * (l + LPR * i)) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        in = in + slot == depth * slot ? 0 : in + slot;
        lives = (lives << 1) | (live ? 1u : 0u);
        src += step_bytes;
        row += step;
        if (++pos == LPR) {
            pos = 0;
            bits = bits2;
            bits2 = look();
        }
    }
    // Ask for one more group and wait for the oldest: its values, -infinity beyond the columns and in
    // rows that do not count. Returns whether any of the warp's rows does.
    __device__ __forceinline__ bool take(const void* logits, int t0, int E, float2 (&v)[NCH * VEC / 2], bool& now) {
        const int lane = threadIdx.x & 31, l = lane % LPR;
        ask();
        if (depth == 6) asm volatile("cp.async.wait_group 5;" ::: "memory");
        else if (depth == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
        else if (depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
        else asm volatile("cp.async.wait_group 1;" ::: "memory");
        now = (lives >> (depth - 1)) & 1u;
        const uint32_t at = base + use;
        use = use + slot == depth * slot ? 0 : use + slot;
        if (!__any_sync(FULL, now)) return false;
        const float none = __uint_as_float(0xff800000u);
        if constexpr (FLAT) {
            __syncwarp();
            const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(logits) + size_t(t0) * (size_t(E) * SIZE)) & 15u;
            const uint32_t r = at + off + (lane / LPR) * chunks;
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int c = l + LPR * i;
                float x = none;
                if (now && c < E) {
                    if constexpr (DT == DT_F32) {
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(r + 4 * c) : "memory");
                    } else {
                        uint16_t u;
                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(r + 2 * c) : "memory");
                        x = bf16f(u);
                    }
                }
                if (i & 1) v[i / 2].y = x;
                else v[i / 2].x = x;
            }
            __syncwarp();  // the slot has been read
        } else {
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                constexpr uint32_t NONE = DT == DT_F32 ? 0xff800000u : 0xff80ff80u;
                uint4 w = make_uint4(NONE, NONE, NONE, NONE);
                if (now && l + LPR * i < chunks)
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at + 16 * lane + 512 * i) : "memory");
                if constexpr (VEC == 4) {
                    v[2 * i] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
                    v[2 * i + 1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
                } else {
                    v[4 * i] = make_float2(bf16lo(w.x), bf16hi(w.x));
                    v[4 * i + 1] = make_float2(bf16lo(w.y), bf16hi(w.y));
                    v[4 * i + 2] = make_float2(bf16lo(w.z), bf16hi(w.z));
                    v[4 * i + 3] = make_float2(bf16lo(w.w), bf16hi(w.w));
                }
            }
        }
        return true;
    }
};

// Workspace: the control block (not used), then per block of the first kernel its column sums [E],
// its counts [E] and {sum of lse^2, rows}.
struct BalanceWs {
    size_t prob, counts, tail, total;
};
BalanceWs balance_layout(int blocks, int E) {
    BalanceWs w;
    size_t o = 256;
    w.prob = o; o = align256(o + 4ull * blocks * padded(E));
    w.counts = o; o = align256(o + 4ull * blocks * padded(E));
    w.tail = o; o = align256(o + 16ull * blocks);
    w.total = o;
    return w;
}
struct Tail {
    double z;
    int rows;
    int pad;
};

struct BalanceParams {
    const void* logits;
    const int32_t* ids;
    const uint8_t* mask;
    int T, E, k;
    float* loss;
    int32_t* counts;
    float* prob;
    int32_t* n_rows;
    float* ws_prob;
    int32_t* ws_counts;
    Tail* ws_tail;
    int blocks;             // of the first kernel
    int depth, ring_bytes;  // of a warp's ring
};

template <int DT, int VEC, int NCH, int LPR, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 1) balance_forward_kernel(const BalanceParams p) {
    constexpr int N2 = NCH * VEC / 2, RPW = 32 / LPR;  // pairs of a lane, rows of a warp
    const int threads = blockDim.x, warps = threads >> 5;  // up to WARPS
    // the warps' rings; behind the last row cols [warps][E], whose first row becomes the block's sums
    extern __shared__ __align__(16) float sm[];
    float* cols = sm;
    __shared__ int hist[MAX_EXPERTS];
    __shared__ double zsum[WARPS];
    __shared__ int nsum[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR;
    // T is at most 2^30, and row numbers go at most 100 steps of up to 20,480 rows beyond it
    const int step = gridDim.x * warps * RPW;
    int t0 = (blockIdx.x * warps + warp) * RPW, t = t0 + lane / LPR;  // the warp's first row, and this lane's
    Ring<DT, VEC, NCH, LPR> ring;
    wait_for_previous();
    ring.start(p.logits, p.mask, p.T, p.E, p.depth, reinterpret_cast<unsigned char*>(sm) + warp * p.ring_bytes, t0, step);
    for (int e = threadIdx.x; e < p.E; e += threads) hist[e] = 0;
    const int32_t* ids = p.ids + size_t(t) * p.k + l;
    const size_t ids_step = size_t(step) * p.k;
    int id_next = t < p.T && l < p.k ? *ids : -1;
    let_next_start();  // the second kernel
    __syncthreads();

    float2 acc[N2];
#pragma unroll
    for (int i = 0; i < N2; ++i) acc[i] = all2(0.0f);
    float z2 = 0.0f;
    int rows = 0;
    for (; t0 < p.T; t0 += step, t += step) {
        const int id = id_next;
        ids += ids_step;
        id_next = t + step < p.T && l < p.k ? *ids : -1;
        bool now;
        float2 v[N2];
        if (!ring.take(p.logits, t0, p.E, v, now)) continue;
        float z;
        bool any;
        const float m = row_exp<N2, LPR>(v, z, any);
        const float inv = any ? rcp(z) : 0.0f;
#pragma unroll
        for (int i = 0; i < N2; ++i) acc[i] = __ffma2_rn(v[i], all2(inv), acc[i]);
        if (any) {
            const float lse = fmaf(lg2(z), LN2, m);
            z2 = fmaf(lse, lse, z2);
            ++rows;
            if (id >= 0 && id < p.E) atomicAdd(&hist[id], 1);
            for (int j = l + LPR; j < p.k; j += LPR) {
                const int more = p.ids[size_t(t) * p.k + j];
                if (more >= 0 && more < p.E) atomicAdd(&hist[more], 1);
            }
        }
    }
    __syncthreads();  // the rings are done with
    // the warp's groups: columns, squares and rows (equal in all lanes of a group)
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
        for (int i = 0; i < N2; ++i) {
            acc[i].x += __shfl_xor_sync(FULL, acc[i].x, o);
            acc[i].y += __shfl_xor_sync(FULL, acc[i].y, o);
        }
        z2 += __shfl_xor_sync(FULL, z2, o);
        rows += __shfl_xor_sync(FULL, rows, o);
    }
    if (lane < LPR) {
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int e = (l + LPR * i) * VEC + j, k = i * VEC + j;
                if (e < p.E) cols[warp * p.E + e] = k & 1 ? acc[k / 2].y : acc[k / 2].x;
            }
    }
    if (lane == 0) {
        zsum[warp] = double(z2);
        nsum[warp] = rows;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += threads) {
        float s = 0.0f;
#pragma unroll 8
        for (int w = 0; w < warps; ++w) s += cols[w * p.E + e];
        p.ws_prob[size_t(blockIdx.x) * padded(p.E) + e] = s;
        p.ws_counts[size_t(blockIdx.x) * padded(p.E) + e] = hist[e];
    }
    if (warp == 0) {
        double z = lane < warps ? zsum[lane] : 0.0;
        int n = lane < warps ? nsum[lane] : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            z += __shfl_xor_sync(FULL, z, o);
            n += __shfl_xor_sync(FULL, n, o);
        }
        if (lane == 0) p.ws_tail[blockIdx.x] = Tail{z, n, 0};
    }
}

// The second kernel: rank r of the cluster adds the blocks' sums of its share of the columns, every
// thread four columns of every parts-th block, then the parts in order; rank 0 makes the losses.
constexpr int FIN_THREADS = 1024;
__global__ void __launch_bounds__(FIN_THREADS) balance_finish_kernel(const BalanceParams p) {
    __shared__ float4 fsum[FIN_THREADS];
    __shared__ int4 csum[FIN_THREADS];
    __shared__ double zsum[32];
    __shared__ int nsum[32];
    __shared__ double part_loss;
    __shared__ double wsum[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int quads = padded(p.E) / 4, share = (quads + BAL_CLUSTER - 1) / BAL_CLUSTER;  // 1 .. 32 column groups
    const int q0 = int(rank) * share, mine = max(0, min(share, quads - q0));
    const int parts = FIN_THREADS / share, quad = threadIdx.x % share, part = threadIdx.x / share;
    wait_for_previous();
    let_next_start();
    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    int4 c = make_int4(0, 0, 0, 0);
    if (part < parts && quad < mine) {
#pragma unroll 4
        for (int b = part; b < p.blocks; b += parts) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p.ws_prob) + size_t(b) * quads + q0 + quad);
            const int4 u = __ldcg(reinterpret_cast<const int4*>(p.ws_counts) + size_t(b) * quads + q0 + quad);
            f.x += v.x; f.y += v.y; f.z += v.z; f.w += v.w;
            c.x += u.x; c.y += u.y; c.z += u.z; c.w += u.w;
        }
    }
    fsum[threadIdx.x] = f;
    csum[threadIdx.x] = c;
    double z = 0.0;
    int n = 0;
    if (threadIdx.x < p.blocks) {  // at most BAL_MAX_BLOCKS < FIN_THREADS
        z = __ldcg(&p.ws_tail[threadIdx.x].z);
        n = __ldcg(&p.ws_tail[threadIdx.x].rows);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        z += __shfl_xor_sync(FULL, z, o);
        n += __shfl_xor_sync(FULL, n, o);
    }
    if (lane == 0) {
        zsum[warp] = z;
        nsum[warp] = n;
    }
    __syncthreads();
    z = zsum[lane];
    n = nsum[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        z += __shfl_xor_sync(FULL, z, o);
        n += __shfl_xor_sync(FULL, n, o);
    }
    const float inv_n = n ? 1.0f / float(n) : 0.0f;
    // eight threads a column: parts h, h + 8, ... each, then the eight
    double balance = 0.0;
    {
        const int col = threadIdx.x >> 3, h = threadIdx.x & 7;  // at most 128 columns a block
        float s = 0.0f;
        int m = 0;
        if (col < 4 * mine) {
            for (int i = h; i < parts; i += 8) {
                s += reinterpret_cast<const float*>(fsum + i * share)[col];
                m += reinterpret_cast<const int*>(csum + i * share)[col];
            }
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
            s += __shfl_xor_sync(FULL, s, o);
            m += __shfl_xor_sync(FULL, m, o);
        }
        const int e = 4 * q0 + col;
        if (h == 0 && col < 4 * mine && e < p.E) {
            p.prob[e] = s * inv_n;
            p.counts[e] = m;
            balance = double(m) * double(s * inv_n);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) balance += __shfl_xor_sync(FULL, balance, o);
    if (lane == 0) wsum[warp] = balance;
    __syncthreads();
    if (warp == 0) {
        balance = wsum[lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) balance += __shfl_xor_sync(FULL, balance, o);
        if (lane == 0) part_loss = balance;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank == 0 && threadIdx.x == 0) {
        double s = 0.0;
        for (int r = 0; r < BAL_CLUSTER; ++r) {
            uint32_t a;
            double v;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(&part_loss)), "r"(r));
            asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(a) : "memory");
            s += v;
        }
        p.loss[0] = n ? float(s * p.E / (double(n) * p.k)) : 0.0f;
        p.loss[1] = n ? float(z / n) : 0.0f;
        *p.n_rows = n;
    }
    // no block leaves while rank 0 reads its shared memory
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct BalanceGradParams {
    const void* logits;
    const uint8_t* mask;
    int T, E, k;
    const int32_t* counts;
    const int32_t* n_rows;
    const float* grad;
    void* dlogits;
    int depth, ring_bytes;
};

template <int DT, int VEC, int NCH, int LPR>
__device__ __forceinline__ void store_logits(void* out, size_t row, int E, int l, const float2 (&v)[NCH * VEC / 2]) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = l + LPR * i;
        if (c * VEC >= E) continue;
        if constexpr (VEC == 8) {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row + size_t(c) * 8) =
                make_uint4(pack_bf16(v[4 * i].x, v[4 * i].y), pack_bf16(v[4 * i + 1].x, v[4 * i + 1].y),
                           pack_bf16(v[4 * i + 2].x, v[4 * i + 2].y), pack_bf16(v[4 * i + 3].x, v[4 * i + 3].y));
        } else if constexpr (VEC == 4) {
            *reinterpret_cast<float4*>(static_cast<float*>(out) + row + size_t(c) * 4) =
                make_float4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
        } else {
            const float x = i & 1 ? v[i / 2].y : v[i / 2].x;
            if (DT == DT_F32) static_cast<float*>(out)[row + c] = x;
            else static_cast<uint16_t*>(out)[row + c] = uint16_t(pack_bf16(x, 0.0f));
        }
    }
}

template <int DT, int VEC, int NCH, int LPR, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 1) balance_backward_kernel(const BalanceGradParams p) {
    constexpr int N2 = NCH * VEC / 2, RPW = 32 / LPR;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR;
    const int step = gridDim.x * WARPS * RPW;
    int t0 = (blockIdx.x * WARPS + warp) * RPW, t = t0 + lane / LPR;
    extern __shared__ __align__(16) unsigned char rings[];
    Ring<DT, VEC, NCH, LPR> ring;
    wait_for_previous();
    ring.start(p.logits, p.mask, p.T, p.E, p.depth, rings + warp * p.ring_bytes, t0, step);
    let_next_start();
    const int n = max(*p.n_rows, 1);
    const int mean = int((long long)n * p.k / p.E);
    const float gb = p.grad[0] * (float(p.E) / (float(n) * float(p.k))) / float(n);
    const float gz = 2.0f * p.grad[1] / float(n);
    float2 f[N2];  // the centred counts
#pragma unroll
    for (int k = 0; k < 2 * N2; ++k) {
        const int e = (l + LPR * (k / VEC)) * VEC + k % VEC;
        const float c = e < p.E ? float(p.counts[e] - mean) : 0.0f;
        if (k & 1) f[k / 2].y = c;
        else f[k / 2].x = c;
    }
    for (; t0 < p.T; t0 += step, t += step) {
        float2 v[N2];
        bool now;
        if (ring.take(p.logits, t0, p.E, v, now)) {
            float z;
            bool any;
            const float m = row_exp<N2, LPR>(v, z, any);
            float2 q = all2(0.0f);
#pragma unroll
            for (int i = 0; i < N2; ++i) q = __ffma2_rn(v[i], f[i], q);
            // p (gb (f - s) + gz lse); nothing in rows that do not count, whose v is zero
            const float inv = any ? rcp(z) : 0.0f, s = row_sum<LPR>(q.x + q.y) * inv;
            const float zt = any ? gz * fmaf(lg2(z), LN2, m) * inv : 0.0f, a = gb * inv;
#pragma unroll
            for (int i = 0; i < N2; ++i)
                v[i] = __fmul2_rn(v[i], __ffma2_rn(__fadd2_rn(f[i], all2(-s)), all2(a), all2(zt)));
        } else {
#pragma unroll
            for (int i = 0; i < N2; ++i) v[i] = all2(0.0f);
        }
        if (t < p.T) store_logits<DT, VEC, NCH, LPR>(p.dlogits, size_t(t) * p.E, p.E, l, v);
    }
}

// ------------------------------------------------------------------------------ host side
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
    return a && b && x < y + bn && y < x + an;
}

redmoe_status check_balance(int dtype, int T, int E, int k) {
    if (dtype < 0 || dtype > DT_INT2 || T < 0 || E <= 0 || E > MAX_EXPERTS || k <= 0 || k > E || k > MAX_TOPK)
        return REDMOE_ERR_INVALID_ARG;
    if ((long long)T * k > (1ll << 30)) return REDMOE_ERR_INVALID_ARG;  // counts and their sum are int32
    return dtype == DT_F32 || dtype == DT_BF16 ? REDMOE_OK : REDMOE_ERR_UNSUPPORTED;
}

// Blocks of so many rows each that T rows need, at least one and at most `most`.
int balance_blocks(int T, int rows, int most) {
    const int need = int((T + (long long)rows - 1) / rows);
    return need < 1 ? 1 : (need < most ? need : most);
}

// Depth of the rings in `room` bytes of shared memory (2, 3, 4 or 6 slots), and a ring's bytes.
int ring_depth(int room, int warps, int E, int dtype, int* bytes) {
    const int size = dtype == DT_F32 ? 4 : 2, rows = E <= 128 ? 4 : 1;
    // rows of whole chunks: the lanes' places, at most 16 columns (E <= 128) or E / 32 rounded up to a
    // power of two each
    int slot = flat_bytes(rows, E, size);
    if (E * size % 16 == 0) {
        const int values = dtype == DT_F32 ? (E <= 32 ? 4 : E <= 128 ? 16 : E <= 256 ? 8 : E <= 512 ? 16 : 32)
                                           : (E <= 64 ? 8 : E <= 128 ? 16 : E <= 256 ? 8 : E <= 512 ? 16 : 32);
        slot = 32 * values * size;
    }
    const int fits = room / warps / slot;
    const int depth = fits >= 6 ? 6 : (fits >= 4 ? 4 : (fits == 3 ? 3 : 2));
    *bytes = depth * slot;
    return depth;
}

int rows_a_block(int E, int warps) { return E <= 128 ? 4 * warps : warps; }

// Warps of a block of the forward pass. Rows of 129 .. 512 columns take 24: 31.5 us for 65536 rows of 512
// (two blocks of 16 an SM 32.4), in bf16 27.8 (30.7), of 501 37.8 (48.1: 64 registers are too few); but
// 16 while that leaves a row to each (2048 rows: 9.5 us, 10.1 in fewer blocks).
int forward_warps(int T, int E, int sm_count) {
    return E > 128 && E <= 512 && T > BAL_WARPS * sm_count ? BAL_WARPS_MID : BAL_WARPS;
}

// 16-byte chunks where every row starts on one, else single values; eight lanes a row up to 128
// columns (65536 rows of 64 fp32 14.1 us, of 61 17.5; a whole warp a row 19.2 and 34.1); the smallest
// number of chunks a lane needs.
#define BALANCE_PICK(kernel, V)                                                                             \
    do {                                                                                                  \
        constexpr int F = DT_F32, B = DT_BF16, W = BAL_WARPS;                                             \
        if (dtype == B && E % 8 == 0)                                                                     \
            return E <= 64 ? kernel<B, 8, 1, 8, W> : E <= 128 ? kernel<B, 8, 2, 8, W> : E <= 256 ? kernel<B, 8, 1, 32, V> \
                 : E <= 512 ? kernel<B, 8, 2, 32, V> : kernel<B, 8, 4, 32, W>;                            \
        if (dtype == F && E % 4 == 0)                                                                     \
            return E <= 32 ? kernel<F, 4, 1, 8, W> : E <= 128 ? kernel<F, 4, 4, 8, W> : E <= 256 ? kernel<F, 4, 2, 32, V> \
                 : E <= 512 ? kernel<F, 4, 4, 32, V> : kernel<F, 4, 8, 32, W>;                            \
        if (dtype == F)                                                                                   \
            return E <= 32 ? kernel<F, 1, 4, 8, W> : E <= 128 ? kernel<F, 1, 16, 8, W> : E <= 512 ? kernel<F, 1, 16, 32, V> \
                 : kernel<F, 1, 32, 32, W>;                                                               \
        return E <= 32 ? kernel<B, 1, 4, 8, W> : E <= 128 ? kernel<B, 1, 16, 8, W> : E <= 512 ? kernel<B, 1, 16, 32, V> \
             : kernel<B, 1, 32, 32, W>;                                                                   \
    } while (0)

using ForwardKernel = void (*)(BalanceParams);
using BackwardKernel = void (*)(BalanceGradParams);
ForwardKernel pick_forward(int dtype, int E) { BALANCE_PICK(balance_forward_kernel, BAL_WARPS_MID); }
BackwardKernel pick_backward(int dtype, int E) { BALANCE_PICK(balance_backward_kernel, BAL_WARPS); }
#undef BALANCE_PICK

}  // namespace
}  // namespace redmoe

using namespace redmoe;

extern "C" {

size_t redmoe_balance_workspace_bytes(int32_t T, int32_t E) {
    if (T < 0 || E <= 0 || E > MAX_EXPERTS) return 0;
    return balance_layout(balance_blocks(T, rows_a_block(E, BAL_WARPS), BAL_MAX_BLOCKS), E).total;
}

redmoe_status redmoe_balance_forward(const void* logits, int32_t logits_dtype, const int32_t* topk_ids,
                                     const uint8_t* row_mask, int32_t T, int32_t E, int32_t k, float* loss,
                                     int32_t* counts, float* prob, int32_t* n_rows, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    redmoe_status st = check_balance(logits_dtype, T, E, k);
    if (st != REDMOE_OK) return st;
    if (!loss || !counts || !prob || !n_rows || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(prob, 4) ||
        !aligned(n_rows, 4))
        return REDMOE_ERR_INVALID_ARG;
    if (T > 0 && (!logits || !topk_ids)) return REDMOE_ERR_INVALID_ARG;
    if (!aligned(logits, 16) || !aligned(topk_ids, 4)) return REDMOE_ERR_INVALID_ARG;
    const size_t need = redmoe_balance_workspace_bytes(T, E);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return REDMOE_ERR_WORKSPACE;
    const size_t lb = size_t(T) * E * (logits_dtype == DT_F32 ? 4 : 2);
    const struct { const void* p; size_t n; } in[] = {{logits, lb}, {topk_ids, 4ull * T * k}, {row_mask, size_t(T)}},
        out[] = {{loss, 8}, {counts, 4ull * E}, {prob, 4ull * E}, {n_rows, 4}, {workspace, need}};
    for (int i = 0; i < 5; ++i) {
        for (const auto& r : in)
            if (overlap(r.p, r.n, out[i].p, out[i].n)) return REDMOE_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return REDMOE_ERR_INVALID_ARG;
    }
    DevInfo di;
    if (!get_dev_info(&di)) return REDMOE_ERR_CUDA;
    const int warps = forward_warps(T, E, di.sm_count), most = di.sm_count < BAL_MAX_BLOCKS ? di.sm_count : BAL_MAX_BLOCKS;
    const int blocks = balance_blocks(T, rows_a_block(E, warps), most);
    const BalanceWs w = balance_layout(blocks, E);
    char* base = static_cast<char*>(workspace);
    BalanceParams p;
    p.logits = logits;
    p.ids = topk_ids;
    p.mask = row_mask;
    p.T = T; p.E = E; p.k = k;
    p.loss = loss;
    p.counts = counts;
    p.prob = prob;
    p.n_rows = n_rows;
    p.blocks = blocks;
    p.ws_prob = reinterpret_cast<float*>(base + w.prob);
    p.ws_counts = reinterpret_cast<int32_t*>(base + w.counts);
    p.ws_tail = reinterpret_cast<Tail*>(base + w.tail);
    const ForwardKernel kern = pick_forward(logits_dtype, E);
    p.depth = ring_depth(di.max_smem_optin - 8 * 1024, warps, E, logits_dtype, &p.ring_bytes);  // less the static part
    int smem = p.ring_bytes * warps;
    const int sums = 4 * warps * E;
    smem = smem > sums ? smem : sums;
    if (!allow_smem(reinterpret_cast<const void*>(kern), smem)) return REDMOE_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!launch(kern, dim3(blocks), 32 * warps, smem, s, 1, p)) return REDMOE_ERR_CUDA;
    return launch(balance_finish_kernel, dim3(BAL_CLUSTER), FIN_THREADS, 0, s, BAL_CLUSTER, p) ? REDMOE_OK : REDMOE_ERR_CUDA;
}

redmoe_status redmoe_balance_backward(const void* logits, int32_t logits_dtype, const uint8_t* row_mask, int32_t T,
                                      int32_t E, int32_t k, const int32_t* counts, const int32_t* n_rows,
                                      const float* grad_loss, void* dlogits, void* stream) {
    redmoe_status st = check_balance(logits_dtype, T, E, k);
    if (st != REDMOE_OK) return st;
    if (T == 0) return REDMOE_OK;
    if (!logits || !counts || !n_rows || !grad_loss || !dlogits || !aligned(logits, 16) || !aligned(dlogits, 16) ||
        !aligned(counts, 4) || !aligned(n_rows, 4) || !aligned(grad_loss, 4))
        return REDMOE_ERR_INVALID_ARG;
    const size_t lb = size_t(T) * E * (logits_dtype == DT_F32 ? 4 : 2);
    if ((dlogits != logits && overlap(dlogits, lb, logits, lb)) || overlap(dlogits, lb, counts, 4ull * E) ||
        overlap(dlogits, lb, n_rows, 4) || overlap(dlogits, lb, grad_loss, 8) || overlap(dlogits, lb, row_mask, T))
        return REDMOE_ERR_INVALID_ARG;
    DevInfo di;
    if (!get_dev_info(&di)) return REDMOE_ERR_CUDA;
    BalanceGradParams p;
    p.logits = logits;
    p.mask = row_mask;
    p.T = T; p.E = E; p.k = k;
    p.counts = counts;
    p.n_rows = n_rows;
    p.grad = grad_loss;
    p.dlogits = dlogits;
    // one block an SM with the deepest ring: 32768 rows of 512 25.0 us (82% of the copy bandwidth; two
    // blocks 25.4), in bf16 and a fifth of them masked 16.5 (18.3). 16 warps: 24, as forward has, take 24.3
    // against 24.0 and 16.6 against 15.6 us
    p.depth = ring_depth(di.max_smem_optin - 2 * 1024, BAL_WARPS, E, logits_dtype, &p.ring_bytes);
    const int smem = p.ring_bytes * BAL_WARPS;
    const BackwardKernel kern = pick_backward(logits_dtype, E);
    if (!allow_smem(reinterpret_cast<const void*>(kern), smem)) return REDMOE_ERR_CUDA;
    const int blocks = balance_blocks(T, rows_a_block(E, BAL_WARPS), di.sm_count);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launch(kern, dim3(blocks), 32 * BAL_WARPS, smem, s, 1, p) ? REDMOE_OK : REDMOE_ERR_CUDA;
}

}  // extern "C"
