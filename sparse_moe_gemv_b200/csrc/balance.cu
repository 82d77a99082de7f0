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
// once (backward). One warp takes a row, a lane the same columns of every row, so the column
// sums of P stay in registers until the warp's rows are done. Sums over rows are made in a
// fixed order (lane, warp, block), counts are integers: results do not depend on timing.
#include "common.cuh"
#include "internal.h"
#include "vec8.cuh"

namespace redmoe {
namespace {

constexpr int BAL_WARPS = 16;
constexpr int BAL_THREADS = 32 * BAL_WARPS;
constexpr int BAL_MAX_BLOCKS = 160;

// How a lane's values map to columns: VEC consecutive values per chunk, chunk lane + 32 i.
// VEC > 1 needs E % VEC == 0 (whole 16-byte chunks in every row), VEC == 1 takes any E.
template <int DT, int VEC, int NCH>
__device__ __forceinline__ void load_logits(const void* logits, size_t row, int E, int lane, float (&v)[NCH * VEC]) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = lane + 32 * i;
        const bool in = c * VEC < E;
        if (VEC == 8) {
            uint4 w = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);  // -infinity
            if (in) w = ld_row(static_cast<const uint16_t*>(logits) + row + size_t(c) * 8);
            const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i * VEC + 2 * j] = bf16lo(q[j]);
                v[i * VEC + (2 * j + 1) % VEC] = bf16hi(q[j]);
            }
        } else if (VEC == 4) {
            uint4 w = make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
            if (in) w = ld_row(static_cast<const float*>(logits) + row + size_t(c) * 4);
            v[i * VEC] = __uint_as_float(w.x);
            v[i * VEC + 1 % VEC] = __uint_as_float(w.y);
            v[i * VEC + 2 % VEC] = __uint_as_float(w.z);
            v[i * VEC + 3 % VEC] = __uint_as_float(w.w);
        } else {
            float x = __uint_as_float(0xff800000u);
            if (in) {
                if (DT == DT_F32) x = static_cast<const float*>(logits)[row + c];
                else x = bf16f(static_cast<const uint16_t*>(logits)[row + c]);
            }
            v[i] = x;
        }
    }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
    return v;
}

// v[] becomes exp(v - max), z their sum over the row; returns the row's maximum. fmaxf drops
// a NaN, the sum does not: a row that holds one comes out NaN whole.
template <int N>
__device__ __forceinline__ float row_exp(float (&v)[N], float& z) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
    m = warp_max(m);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = expf(v[i] - m);
        s += v[i];
    }
    z = warp_sum(s);
    return m;
}

// Workspace: the control block, whose word 8 counts the blocks that are done, then per block
// its column sums [E], its counts [E] and {sum of lse^2 (double), rows}.
struct BalanceWs {
    size_t prob, counts, tail, total;
};
constexpr int TICKET_WORD = 8;
BalanceWs balance_layout(int blocks, int E) {
    BalanceWs w;
    size_t o = 256;
    w.prob = o; o = align256(o + 4ull * blocks * E);
    w.counts = o; o = align256(o + 4ull * blocks * E);
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
    unsigned* ticket;
    float* ws_prob;
    int32_t* ws_counts;
    Tail* ws_tail;
};

template <int DT, int VEC, int NCH>
__global__ void __launch_bounds__(BAL_THREADS) balance_forward_kernel(const BalanceParams p) {
    constexpr int N = NCH * VEC;
    extern __shared__ __align__(16) float sm[];
    float* cols = sm;                                             // [BAL_WARPS][E]
    int* hist = reinterpret_cast<int*>(cols + BAL_WARPS * p.E);   // [E]
    __shared__ double zsum[BAL_WARPS];
    __shared__ int nsum[BAL_WARPS];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < p.E; e += BAL_THREADS) hist[e] = 0;
    __syncthreads();

    float acc[N] = {};
    double z2 = 0.0;
    int rows = 0;
    const long long step = (long long)gridDim.x * BAL_WARPS;
    for (long long t = (long long)blockIdx.x * BAL_WARPS + warp; t < p.T; t += step) {
        if (p.mask && !p.mask[t]) continue;
        int id = -1;
        if (lane < p.k) id = p.ids[size_t(t) * p.k + lane];
        float v[N];
        load_logits<DT, VEC, NCH>(p.logits, size_t(t) * p.E, p.E, lane, v);
        bool none = true;
#pragma unroll
        for (int i = 0; i < N; ++i) none = none && v[i] == __uint_as_float(0xff800000u);
        if (__all_sync(FULL, none)) continue;
        float z;
        const float m = row_exp<N>(v, z);
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
    for (int e = threadIdx.x; e < p.E; e += BAL_THREADS) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < BAL_WARPS; ++w) s += cols[w * p.E + e];
        p.ws_prob[size_t(blockIdx.x) * p.E + e] = s;
        p.ws_counts[size_t(blockIdx.x) * p.E + e] = hist[e];
    }
    if (threadIdx.x == 0) {
        Tail t{0.0, 0, 0};
        for (int w = 0; w < BAL_WARPS; ++w) {
            t.z += zsum[w];
            t.rows += nsum[w];
        }
        p.ws_tail[blockIdx.x] = t;
    }
    // the block that is last to finish adds the blocks' sums, in block order
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    if (threadIdx.x == 0) {
        *p.ticket = 0;
        double z = 0.0;
        long long n = 0;
        for (unsigned b = 0; b < gridDim.x; ++b) {
            z += __ldcg(&p.ws_tail[b].z);
            n += __ldcg(&p.ws_tail[b].rows);
        }
        zsum[0] = z;
        nsum[0] = int(n);
    }
    __syncthreads();
    const int n = nsum[0];
    const float inv_n = n ? 1.0f / float(n) : 0.0f;
    float balance = 0.0f;
    for (int e = threadIdx.x; e < p.E; e += BAL_THREADS) {
        float s = 0.0f;
        int c = 0;
        for (unsigned b = 0; b < gridDim.x; ++b) {
            s += __ldcg(p.ws_prob + size_t(b) * p.E + e);
            c += __ldcg(p.ws_counts + size_t(b) * p.E + e);
        }
        s *= inv_n;
        p.prob[e] = s;
        p.counts[e] = c;
        balance = fmaf(float(c), s, balance);
    }
    balance = warp_sum(balance);
    __syncthreads();  // cols is free again
    if (lane == 0) cols[warp] = balance;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int w = 0; w < BAL_WARPS; ++w) s += cols[w];
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
        if (VEC == 8) {
            uint32_t q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = pack_bf16(v[i * VEC + 2 * j], v[i * VEC + (2 * j + 1) % VEC]);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row + size_t(c) * 8) = make_uint4(q[0], q[1], q[2], q[3]);
        } else if (VEC == 4) {
            *reinterpret_cast<float4*>(static_cast<float*>(out) + row + size_t(c) * 4) =
                make_float4(v[i * VEC], v[i * VEC + 1 % VEC], v[i * VEC + 2 % VEC], v[i * VEC + 3 % VEC]);
        } else if (DT == DT_F32) {
            static_cast<float*>(out)[row + c] = v[i];
        } else {
            static_cast<uint16_t*>(out)[row + c] = uint16_t(pack_bf16(v[i], 0.0f));
        }
    }
}

template <int DT, int VEC, int NCH>
__global__ void __launch_bounds__(BAL_THREADS) balance_backward_kernel(const BalanceGradParams p) {
    constexpr int N = NCH * VEC;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
    const long long step = (long long)gridDim.x * BAL_WARPS;
    for (long long t = (long long)blockIdx.x * BAL_WARPS + warp; t < p.T; t += step) {
        const size_t row = size_t(t) * p.E;
        float v[N];
        bool none = p.mask && !p.mask[t];
        if (!none) {
            load_logits<DT, VEC, NCH>(p.logits, row, p.E, lane, v);
            none = true;
#pragma unroll
            for (int i = 0; i < N; ++i) none = none && v[i] == __uint_as_float(0xff800000u);
            none = __all_sync(FULL, none);
        }
        if (none) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = 0.0f;
        } else {
            float z;
            const float m = row_exp<N>(v, z);
            const float inv = 1.0f / z;
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v[i] *= inv;
                s = fmaf(v[i], f[i], s);
            }
            s = warp_sum(s);
            const float zt = gz * (m + logf(z));
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] *= fmaf(gb, f[i] - s, zt);
        }
        store_logits<DT, VEC, NCH>(p.dlogits, row, p.E, lane, v);
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

int balance_blocks(int T, int sm_count) {
    const int most = sm_count < BAL_MAX_BLOCKS ? sm_count : BAL_MAX_BLOCKS;
    const int need = (T + BAL_WARPS - 1) / BAL_WARPS;
    return need < 1 ? 1 : (need < most ? need : most);
}

// 16-byte chunks where every row starts on one, else single values; the smallest number of
// chunks a lane needs.
#define BALANCE_PICK(kernel)                                                                                     \
    do {                                                                                                         \
        if (dtype == DT_BF16 && E % 8 == 0)                                                                      \
            return E <= 256 ? kernel<DT_BF16, 8, 1> : (E <= 512 ? kernel<DT_BF16, 8, 2> : kernel<DT_BF16, 8, 4>); \
        if (dtype == DT_F32 && E % 4 == 0)                                                                       \
            return E <= 128 ? kernel<DT_F32, 4, 1> : (E <= 512 ? kernel<DT_F32, 4, 4> : kernel<DT_F32, 4, 8>);    \
        if (dtype == DT_F32)                                                                                     \
            return E <= 128 ? kernel<DT_F32, 1, 4> : (E <= 512 ? kernel<DT_F32, 1, 16> : kernel<DT_F32, 1, 32>);  \
        return E <= 128 ? kernel<DT_BF16, 1, 4> : (E <= 512 ? kernel<DT_BF16, 1, 16> : kernel<DT_BF16, 1, 32>);   \
    } while (0)

using ForwardKernel = void (*)(BalanceParams);
using BackwardKernel = void (*)(BalanceGradParams);
ForwardKernel pick_forward(int dtype, int E) { BALANCE_PICK(balance_forward_kernel); }
BackwardKernel pick_backward(int dtype, int E) { BALANCE_PICK(balance_backward_kernel); }
#undef BALANCE_PICK

}  // namespace
}  // namespace redmoe

using namespace redmoe;

extern "C" {

size_t redmoe_balance_workspace_bytes(int32_t T, int32_t E) {
    if (T < 0 || E <= 0 || E > MAX_EXPERTS) return 0;
    return balance_layout(balance_blocks(T, BAL_MAX_BLOCKS), E).total;
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
    const int blocks = balance_blocks(T, di.sm_count);
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
    p.ticket = reinterpret_cast<unsigned*>(base) + TICKET_WORD;
    p.ws_prob = reinterpret_cast<float*>(base + w.prob);
    p.ws_counts = reinterpret_cast<int32_t*>(base + w.counts);
    p.ws_tail = reinterpret_cast<Tail*>(base + w.tail);
    const ForwardKernel kern = pick_forward(logits_dtype, E);
    const int smem = 4 * (BAL_WARPS + 1) * E;  // E = 1024: 69,632 bytes
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return REDMOE_ERR_CUDA;
    kern<<<blocks, BAL_THREADS, smem, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? REDMOE_OK : REDMOE_ERR_CUDA;
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
    const int need = (T + BAL_WARPS - 1) / BAL_WARPS, most = 2 * di.sm_count;
    pick_backward(logits_dtype, E)<<<need < most ? need : most, BAL_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? REDMOE_OK : REDMOE_ERR_CUDA;
}

}  // extern "C"
