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
// once (backward), rows that do not count are not read. One warp takes a row, a lane the same
// columns of every row, so the column sums of P stay in registers until the warp's rows are done;
// the next row is asked for while one is worked on, its mask byte a row earlier. Forward, the
// blocks of a cluster add their sums through distributed shared memory, and the last block to
// finish adds the clusters': a single launch. Sums over rows are made in a fixed order (lane,
// warp, block, cluster), counts are integers: results do not depend on timing.
#include "common.cuh"
#include "internal.h"
#include "vec8.cuh"

namespace redmoe {
namespace {

constexpr int BAL_CLUSTER = 4;
constexpr int BAL_MAX_CLUSTERS = 80;  // two blocks an SM, 160 SMs
__host__ __device__ constexpr int padded(int E) { return (E + 3) & ~3; }  // a row of sums in the workspace

// How a lane's values map to columns: VEC consecutive values per chunk, chunk lane + 32 i.
// VEC > 1 needs E % VEC == 0 (whole 16-byte chunks in every row), VEC == 1 takes any E.
template <int DT, int VEC, int NCH>
struct RowOf {
    static constexpr int N = NCH * VEC, W = VEC == 1 ? 1 : 4;  // values, words a chunk
    uint32_t w[NCH][W];

    __device__ __forceinline__ void load(const void* logits, size_t row, int E, int lane) {
        constexpr uint32_t NONE = DT == DT_F32 ? 0xff800000u : 0xff80ff80u;  // -infinity
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = lane + 32 * i;
#pragma unroll
            for (int j = 0; j < W; ++j) w[i][j] = NONE;
            if (c * VEC >= E) continue;
            if constexpr (VEC == 1) {
                if (DT == DT_F32) w[i][0] = static_cast<const uint32_t*>(logits)[row + c];
                else w[i][0] = static_cast<const uint16_t*>(logits)[row + c] * 0x10001u;
            } else {
                const uint4 v = ld_row(static_cast<const char*>(logits) + (row * (DT == DT_F32 ? 4 : 2)) + size_t(c) * 16);
                w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[N]) const {
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (DT == DT_F32) v[i * VEC + j] = __uint_as_float(w[i][j % W]);
                else v[i * VEC + j] = j & 1 ? bf16hi(w[i][j / 2]) : bf16lo(w[i][j / 2]);
            }
    }
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
    return v;
}

// v[] becomes exp(v - max) and z their sum over the row; returns the maximum, or false in `any`
// where the row allows no expert. fmaxf drops a NaN, the sum does not: a row that holds one comes
// out NaN whole. The fast exponential is off by about 2 + 1.2 |v - max| units, which is least where
// the probability is large.
template <int N>
__device__ __forceinline__ float row_exp(float (&v)[N], float& z, bool& any) {
    const float none = __uint_as_float(0xff800000u);
    float m = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
    m = warp_max(m);
    any = true;
    if (m == none) {  // -infinity throughout, unless a NaN hides behind fmaxf
        bool other = false;
#pragma unroll
        for (int i = 0; i < N; ++i) other = other || v[i] != none;
        any = __any_sync(FULL, other);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = __expf(v[i] - m);
        s += v[i];
    }
    z = warp_sum(s);
    return m;
}

// Rows of one warp, two ahead: the mask byte of the row after the next, the next row's data.
template <int DT, int VEC, int NCH>
struct Walk {
    RowOf<DT, VEC, NCH> next;
    bool live, live2;  // of the next row and of the one behind it
    __device__ __forceinline__ static bool counts(const uint8_t* mask, long long t, int T) {
        return t < T && (!mask || __ldg(mask + t));
    }
    __device__ __forceinline__ void start(const void* logits, const uint8_t* mask, long long t, long long step, int T, int E,
                                          int lane) {
        live = counts(mask, t, T);
        live2 = counts(mask, t + step, T);
        if (live) next.load(logits, size_t(t) * E, E, lane);
    }
    // Row t's values into v (if it is to be read at all), and on.
    __device__ __forceinline__ bool take(const void* logits, const uint8_t* mask, long long t, long long step, int T, int E,
                                         int lane, float (&v)[NCH * VEC]) {
        const bool now = live;
        if (now) next.get(v);
        live = live2;
        live2 = counts(mask, t + 2 * step, T);
        if (live) next.load(logits, size_t(t + step) * E, E, lane);
        return now;
    }
};

// Workspace: the control block, whose word 8 counts the blocks that are done, then per cluster
// its column sums [E], its counts [E] and {sum of lse^2 (double), rows}.
struct BalanceWs {
    size_t prob, counts, tail, total;
};
constexpr int TICKET_WORD = 8;
BalanceWs balance_layout(int E) {
    BalanceWs w;
    size_t o = 256;
    w.prob = o; o = align256(o + 4ull * BAL_MAX_CLUSTERS * padded(E));
    w.counts = o; o = align256(o + 4ull * BAL_MAX_CLUSTERS * padded(E));
    w.tail = o; o = align256(o + 16ull * BAL_MAX_CLUSTERS);
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
    unsigned* ticket;
    float* ws_prob;
    int32_t* ws_counts;
    Tail* ws_tail;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(const void* p, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t peer_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

template <int DT, int VEC, int NCH, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, NCH * VEC <= 16 ? 2 : 1) balance_forward_kernel(const BalanceParams p) {
    constexpr int N = NCH * VEC, THREADS = 32 * WARPS;
    extern __shared__ __align__(16) float sm[];
    float* cols = sm;                                         // [WARPS][E]; then [E]: the block's
    int* hist = reinterpret_cast<int*>(cols + WARPS * p.E);   // [E]
    __shared__ double zsum[WARPS];
    __shared__ int nsum[WARPS];
    __shared__ Tail tail;
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long step = (long long)gridDim.x * WARPS;
    long long t = (long long)blockIdx.x * WARPS + warp;
    Walk<DT, VEC, NCH> walk;
    walk.start(p.logits, p.mask, t, step, p.T, p.E, lane);
    for (int e = threadIdx.x; e < p.E; e += THREADS) hist[e] = 0;
    __syncthreads();

    float acc[N] = {};
    double z2 = 0.0;
    int rows = 0;
    for (; t < p.T; t += step) {
        const bool live = walk.live;
        int id = -1;
        if (live && lane < p.k) id = p.ids[size_t(t) * p.k + lane];
        float v[N];
        if (!walk.take(p.logits, p.mask, t, step, p.T, p.E, lane, v)) continue;
        float z;
        bool any;
        const float m = row_exp<N>(v, z, any);
        if (!any) continue;
        const float inv = 1.0f / z;
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
        const float lse = m + logf(z);
        z2 += double(lse) * double(lse);
        ++rows;
        if (id >= 0 && id < p.E) atomicAdd(&hist[id], 1);
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int e = (lane + 32 * i) * VEC + j;
            if (e < p.E) cols[warp * p.E + e] = acc[i * VEC + j];
        }
    if (lane == 0) {
        zsum[warp] = z2;
        nsum[warp] = rows;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += THREADS) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += cols[w * p.E + e];
        cols[e] = s;  // this thread's column only
    }
    if (threadIdx.x == 0) {
        Tail u{0.0, 0, 0};
        for (int w = 0; w < WARPS; ++w) {
            u.z += zsum[w];
            u.rows += nsum[w];
        }
        tail = u;
    }
    // the cluster's sums, in block order: each of its blocks adds a share of the columns
    cluster_sync();
    const int rank = cluster_rank(), cluster = blockIdx.x / BAL_CLUSTER, clusters = gridDim.x / BAL_CLUSTER;
    for (int e = rank * THREADS + threadIdx.x; e < p.E; e += BAL_CLUSTER * THREADS) {
        float s = 0.0f;
        int c = 0;
#pragma unroll
        for (int r = 0; r < BAL_CLUSTER; ++r) {
            s += __uint_as_float(peer_u32(peer_addr(cols + e, r)));
            c += int(peer_u32(peer_addr(hist + e, r)));
        }
        p.ws_prob[size_t(cluster) * padded(p.E) + e] = s;
        p.ws_counts[size_t(cluster) * padded(p.E) + e] = c;
    }
    if (rank == 0 && threadIdx.x == 0) {
        Tail u{0.0, 0, 0};
        for (int r = 0; r < BAL_CLUSTER; ++r) {
            const uint32_t a = peer_addr(&tail, r);
            u.z += __hiloint2double(int(peer_u32(a + 4)), int(peer_u32(a)));
            u.rows += int(peer_u32(a + 8));
        }
        p.ws_tail[cluster] = u;
    }
    // the block that is last to finish adds the clusters' sums, in cluster order
    __threadfence();
    cluster_sync();  // no block leaves while another reads its shared memory
    if (threadIdx.x == 0) last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (threadIdx.x == 0) {
        *p.ticket = 0;
        double z = 0.0;
        long long n = 0;
        for (int b = 0; b < clusters; ++b) {
            z += __ldcg(&p.ws_tail[b].z);
            n += __ldcg(&p.ws_tail[b].rows);
        }
        zsum[0] = z;
        nsum[0] = int(n);
    }
    __syncthreads();
    const int n = nsum[0];
    const float inv_n = n ? 1.0f / float(n) : 0.0f;
    // four columns a thread, several threads a column group: each adds every parts-th cluster
    const int quads = padded(p.E) / 4, parts = THREADS / quads;
    const int quad = threadIdx.x % quads, part = threadIdx.x / quads;
    float4* fsum = reinterpret_cast<float4*>(cols);             // [parts][quads], at most THREADS
    int4* csum = reinterpret_cast<int4*>(fsum + THREADS);
    if (part < parts) {
        float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        int4 c = make_int4(0, 0, 0, 0);
#pragma unroll 8
        for (int b = part; b < clusters; b += parts) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p.ws_prob) + size_t(b) * quads + quad);
            const int4 u = __ldcg(reinterpret_cast<const int4*>(p.ws_counts) + size_t(b) * quads + quad);
            f.x += v.x; f.y += v.y; f.z += v.z; f.w += v.w;
            c.x += u.x; c.y += u.y; c.z += u.z; c.w += u.w;
        }
        fsum[threadIdx.x] = f;
        csum[threadIdx.x] = c;
    }
    __syncthreads();
    float balance = 0.0f;
    for (int e = threadIdx.x; e < p.E; e += THREADS) {
        float s = 0.0f;
        int c = 0;
        for (int i = 0; i < parts; ++i) {
            s += reinterpret_cast<const float*>(fsum + i * quads)[e];
            c += reinterpret_cast<const int*>(csum + i * quads)[e];
        }
        s *= inv_n;
        p.prob[e] = s;
        p.counts[e] = c;
        balance = fmaf(float(c), s, balance);
    }
    __syncthreads();  // the sums have been read
    balance = warp_sum(balance);
    if (lane == 0) cols[warp] = balance;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int w = 0; w < WARPS; ++w) s += cols[w];
        p.loss[0] = n ? float(s * p.E / (double(n) * p.k)) : 0.0f;
        p.loss[1] = n ? float(zsum[0] / n) : 0.0f;
        *p.n_rows = n;
    }
}

struct BalanceGradParams {
    const void* logits;
    const uint8_t* mask;
    int T, E, k;
    const int32_t* counts;
    const int32_t* n_rows;
    const float* grad;
    void* dlogits;
};

template <int DT, int VEC, int NCH>
__device__ __forceinline__ void store_logits(void* out, size_t row, int E, int lane, const float (&v)[NCH * VEC]) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = lane + 32 * i;
        if (c * VEC >= E) continue;
        if constexpr (VEC == 8) {
            uint32_t q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = pack_bf16(v[i * VEC + 2 * j], v[i * VEC + 2 * j + 1]);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row + size_t(c) * 8) = make_uint4(q[0], q[1], q[2], q[3]);
        } else if constexpr (VEC == 4) {
            *reinterpret_cast<float4*>(static_cast<float*>(out) + row + size_t(c) * 4) =
                make_float4(v[i * VEC], v[i * VEC + 1], v[i * VEC + 2], v[i * VEC + 3]);
        } else if (DT == DT_F32) {
            static_cast<float*>(out)[row + c] = v[i];
        } else {
            static_cast<uint16_t*>(out)[row + c] = uint16_t(pack_bf16(v[i], 0.0f));
        }
    }
}

template <int DT, int VEC, int NCH, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) balance_backward_kernel(const BalanceGradParams p) {
    constexpr int N = NCH * VEC;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long step = (long long)gridDim.x * WARPS;
    long long t = (long long)blockIdx.x * WARPS + warp;
    Walk<DT, VEC, NCH> walk;
    walk.start(p.logits, p.mask, t, step, p.T, p.E, lane);
    const int n = max(*p.n_rows, 1);
    const int mean = int((long long)n * p.k / p.E);
    const float gb = p.grad[0] * (float(p.E) / (float(n) * float(p.k))) / float(n);
    const float gz = 2.0f * p.grad[1] / float(n);
    float f[N];
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int e = (lane + 32 * i) * VEC + j;
            f[i * VEC + j] = e < p.E ? float(__ldg(p.counts + e) - mean) : 0.0f;
        }
    for (; t < p.T; t += step) {
        float v[N];
        bool any = walk.take(p.logits, p.mask, t, step, p.T, p.E, lane, v);
        float z, m;
        if (any) m = row_exp<N>(v, z, any);
        if (!any) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = 0.0f;
        } else {
            const float inv = 1.0f / z;
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) s = fmaf(v[i], f[i], s);
            s = warp_sum(s) * inv;
            const float zt = gz * (m + logf(z)) * inv, a = gb * inv;
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] *= fmaf(a, f[i] - s, zt);
        }
        store_logits<DT, VEC, NCH>(p.dlogits, size_t(t) * p.E, p.E, lane, v);
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

// Blocks that `warps` rows each keep busy, at most `most`.
int balance_blocks(int T, int warps, int most) {
    const int need = int((T + (long long)warps - 1) / warps);
    return need < 1 ? 1 : (need < most ? need : most);
}

// 16-byte chunks where every row starts on one, else single values; the smallest number of
// chunks a lane needs. W: warps of a block with up to 16 values a lane, and with more.
#define BALANCE_PICK(kernel, W, W32)                                                                          \
    do {                                                                                                      \
        if (dtype == DT_BF16 && E % 8 == 0)                                                                   \
            return E <= 256 ? kernel<DT_BF16, 8, 1, W> : (E <= 512 ? kernel<DT_BF16, 8, 2, W> : kernel<DT_BF16, 8, 4, W32>); \
        if (dtype == DT_F32 && E % 4 == 0)                                                                    \
            return E <= 128 ? kernel<DT_F32, 4, 1, W> : (E <= 512 ? kernel<DT_F32, 4, 4, W> : kernel<DT_F32, 4, 8, W32>); \
        if (dtype == DT_F32)                                                                                  \
            return E <= 128 ? kernel<DT_F32, 1, 4, W> : (E <= 512 ? kernel<DT_F32, 1, 16, W> : kernel<DT_F32, 1, 32, W32>); \
        return E <= 128 ? kernel<DT_BF16, 1, 4, W> : (E <= 512 ? kernel<DT_BF16, 1, 16, W> : kernel<DT_BF16, 1, 32, W32>); \
    } while (0)

using ForwardKernel = void (*)(BalanceParams);
using BackwardKernel = void (*)(BalanceGradParams);
constexpr int FORWARD_WARPS = 16, BACKWARD_WARPS = 16, WIDE_WARPS = 16;  // wide: over 512 columns
ForwardKernel pick_forward(int dtype, int E) { BALANCE_PICK(balance_forward_kernel, FORWARD_WARPS, WIDE_WARPS); }
BackwardKernel pick_backward(int dtype, int E) { BALANCE_PICK(balance_backward_kernel, BACKWARD_WARPS, WIDE_WARPS); }
#undef BALANCE_PICK

}  // namespace
}  // namespace redmoe

using namespace redmoe;

extern "C" {

size_t redmoe_balance_workspace_bytes(int32_t T, int32_t E) {
    if (T < 0 || E <= 0 || E > MAX_EXPERTS) return 0;
    return balance_layout(E).total;
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
    const BalanceWs w = balance_layout(E);
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
    p.ticket = reinterpret_cast<unsigned*>(base) + TICKET_WORD;
    p.ws_prob = reinterpret_cast<float*>(base + w.prob);
    p.ws_counts = reinterpret_cast<int32_t*>(base + w.counts);
    p.ws_tail = reinterpret_cast<Tail*>(base + w.tail);
    const ForwardKernel kern = pick_forward(logits_dtype, E);
    const int warps = E <= 512 ? FORWARD_WARPS : WIDE_WARPS;
    const int sums = 4 * (warps + 1) * E, ends = 32 * 32 * warps;  // columns and counts; the last block's
    const int smem = sums > ends ? sums : ends;                    // E = 1024: 69,632 bytes
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return REDMOE_ERR_CUDA;
    // whole clusters lie in one GPC each: about 24 of 25 places can be had
    const int places = di.sm_count * (E <= 512 ? 2 : 1) / BAL_CLUSTER * 24 / 25;
    const int most = places < 1 ? 1 : (places < BAL_MAX_CLUSTERS ? places : BAL_MAX_CLUSTERS);
    const int clusters = balance_blocks(T, warps * BAL_CLUSTER, most);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * BAL_CLUSTER);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = BAL_CLUSTER;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? REDMOE_OK : REDMOE_ERR_CUDA;
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
    const int warps = E <= 512 ? BACKWARD_WARPS : WIDE_WARPS;
    pick_backward(logits_dtype, E)<<<balance_blocks(T, warps, 2 * di.sm_count), 32 * warps, 0,
                                     static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? REDMOE_OK : REDMOE_ERR_CUDA;
}

}  // extern "C"
