// The residual step between blocks: the norms before and after a block fused with the
// block's gate and scales, forward and backward.
//
// Forward, per token row (N(v; w) = v r(v) (w_offset + w), r(v) = 1 / sqrt(mean v^2 + eps)):
//   u     = N(y; post_w) or y
//   h_out = res_scale h + block_scale g u
//   x     = N(h_out; pre_w)
// x is normalised from the fp32 h_out, before that is rounded for storage: each output is
// rounded once.
//
// Backward, from the stored h_out (r2 = r(h_out), r1 = r(y) are recomputed: the row is in
// registers anyway, so saving them would only add bytes), a = dx (w_offset + pre_w):
//   G       = dh_out + r2 (a - h_out r2^2 mean(a h_out))
//   dpre_w  = sum_t dx h_out r2
//   dh      = res_scale G
//   b       = block_scale G;  dgate = sum (over what the gate broadcasts) b u act'(gate)
//   d       = b act(gate);    dpost_w = sum_t d y r1;  c = d (w_offset + post_w)
//   dy      = r1 (c - y r1^2 mean(c y))
//
// Both are bound by memory: forward reads y and h once and writes h_out and x once, backward
// reads h_out, y, dh_out and dx once and writes dh and dy once. A row belongs to a group of
// threads (whole warps, eight or sixteen columns a thread) that holds it on chip, so the
// statistics cost reductions over the group and nothing is read twice. All sums are fp32, in a
// fixed order. Measured on a B200, of the copy bandwidth: forward 8191 x 5120 fp32 with an element
// gate 106 us (84%), 8192 x 4096 47 us (86%), 2048 x 2048 11.8 us (54%: under two waves of blocks),
// one row of 2048 1.45 us; backward 8192 x 2048 42.4 us (72%: 95% in
// the steady state, ten us are launches, first rows and column sums), one row of 2048 4.2 us.
#include "common.cuh"
#include "internal.h"
#include "launch.h"
#include "norm.h"
#include "vec8.cuh"

namespace redmoe {
namespace {

constexpr int NORM_MAX_H = 8192;
// An upper bound on the blocks of the backward pass that needs no device: the workspace query
// works without one.
constexpr int MAX_SMS = 160, MAX_BLOCKS_SM = 2;
constexpr int NORM_THREADS = 256;  // threads of a block whose groups are smaller than that

enum : int { GATE_NONE = 0, GATE_TOKEN = 1, GATE_CHANNEL = 2, GATE_ELEMENT = 3 };

struct NormParams {
    int T, H, chunks;  // chunks of eight columns in a row
    int tpr;           // threads of a group (one row), a multiple of 32
    int post_norm, gate_kind, sigmoid;
    bool gate_f32, w_f32;
    float eps, w_offset, res_scale, block_scale, inv_h;
    const void *post_w, *pre_w, *gate;
    const void *h, *y;     // forward: h; backward: h_out
    void *h_out, *x;       // forward outputs
    const void *dh_out, *dx;
    void *dh, *dy, *dgate;
    float* part;  // backward: [blocks][2][H] column sums: dpre_w and A
    int units, ahead;  // walked rows: 16-byte units of a chunk, rows in flight (0 .. 2)
    bool want_pre, want_post, want_gate;
    float *dpre_w, *dpost_w;
    bool cluster;       // backward: the grid is one cluster, whose blocks add the column sums among themselves
};

// The sum over a group: warps by shuffles, then the warps' sums through shared memory, four to a lane
// of a quad (a loop over the warps takes registers that spill, 112 instead of 106 us for 8191 rows of
// 5120). Successive sums take their `buf` ([16], zeros behind the group's last warp) from two areas
// in turn, so one barrier a sum is enough: an area is written again only behind the barrier of the
// sum between, which every thread reaches after its reads.
constexpr int RED = 16;
__device__ __forceinline__ float group_sum(float v, float* buf, int tpr, int group, int wig) {
    v = warp_sum(v);
    if (tpr == 32) return v;
    if ((threadIdx.x & 31) == 0) buf[wig] = v;
    asm volatile("bar.sync %0, %1;" :: "r"(group + 1), "r"(tpr) : "memory");
    const float4 f = *reinterpret_cast<const float4*>(buf + ((threadIdx.x & 3) << 2));
    v = (f.x + f.y) + (f.z + f.w);
    v += __shfl_xor_sync(FULL, v, 1);
    return v + __shfl_xor_sync(FULL, v, 2);
}

// Six sums over the group at once: eight lanes' worth of values is halved three times while the warp
// is (nine shuffles for six sums), lane 4 v ends with value v; behind the barrier a quad of lanes adds
// one value's warps. buf: [6][16].
constexpr int RED6 = 6 * 16;
__device__ __forceinline__ void group_sum6(float (&v)[6], float* buf, int tpr, int group, int wig) {
    const int l = threadIdx.x & 31;
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // lanes 16 .. 31 keep values 4 .. 7 (6 and 7 are none), the others 0 .. 3
        const float hi = i < 2 ? v[4 + (i & 1)] : 0.0f;
        a[i] = (l & 16 ? hi : v[i]) + __shfl_xor_sync(FULL, l & 16 ? v[i] : hi, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) b[i] = (l & 8 ? a[2 + i] : a[i]) + __shfl_xor_sync(FULL, l & 8 ? a[i] : a[2 + i], 8);
    float c = (l & 4 ? b[1] : b[0]) + __shfl_xor_sync(FULL, l & 4 ? b[0] : b[1], 4);
    c += __shfl_xor_sync(FULL, c, 2);
    c += __shfl_xor_sync(FULL, c, 1);
    if (tpr > 32) {
        if ((l & 3) == 0 && l < 24) buf[(l >> 2) * 16 + wig] = c;
        asm volatile("bar.sync %0, %1;" :: "r"(group + 1), "r"(tpr) : "memory");
        float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (l < 24) f = *reinterpret_cast<const float4*>(buf + 4 * l);  // value l / 4, warps 4 (l % 4) ..
        c = (f.x + f.y) + (f.z + f.w);
        c += __shfl_xor_sync(FULL, c, 1);
        c += __shfl_xor_sync(FULL, c, 2);
    }
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(FULL, c, 4 * i);
}

// The places of warps that a group does not have, read as zeros by group_sum (whose barrier
// publishes them).
__device__ __forceinline__ void clear_unused(float* a, float* b, int n, int lane, int tpr) {
    for (int i = lane; i < n; i += tpr)
        if (i % 16 >= tpr / 32) a[i] = b[i] = 0.0f;
}

// 1 / (1 + e^-a) with e^-a = 2^(-a log2 e): rounding the exponent makes e^-a off by about |a| units,
// so the result only where e^-a decides (a < 0): 3 units in all at |a| = 1, 12 at a = -10. Four
// instructions an element, two of them of the unit for special functions; expf and an IEEE divide
// take some twenty more.
__device__ __forceinline__ float sigmoid(float a) { return rcp(1.0f + ex2(a * -LOG2E)); }
__device__ __forceinline__ F8 sigmoid(const F8& a) {
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = make_float2(sigmoid(a.v[i].x), sigmoid(a.v[i].y));
    return r;
}

// Its slope s(a) s(-a) = e / (1 + e)^2 with e = 2^(-|a| log2 e). From a rounded s the difference 1 - s
// would be off by some 2^-24 / e: 1e-3 of it at a = 10, all of it from 17 on.
__device__ __forceinline__ float sigmoid_slope(float a) {
    const float e = ex2(fabsf(a) * -LOG2E), r = rcp(1.0f + e);
    return e * r * r;
}
__device__ __forceinline__ F8 sigmoid_slope(const F8& a) {
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = make_float2(sigmoid_slope(a.v[i].x), sigmoid_slope(a.v[i].y));
    return r;
}

// One row per group of p.tpr threads; NC chunks a thread (chunk c = thread + i tpr). Everything a
// row needs is asked for before the first sum waits. 64 registers a thread,
// at which the two-chunk forms with a block output spill 8 to 28 bytes: 76 without a spill, and so fewer blocks
// on an SM, take 28.1 instead of 25.7 us for 8192 rows of 2048.
template <int HD, int YD, int XD, int NC, bool BRANCH>
__global__ void __launch_bounds__(512, 2) norm_forward_kernel(const NormParams p) {
    constexpr bool EARLY = NC == 1;  // the weights too, where registers allow
    __shared__ __align__(16) float red[2][8][RED];
    const int group = threadIdx.x / p.tpr, lane = threadIdx.x % p.tpr, wig = lane / 32;
    const int rows = blockDim.x / p.tpr;
    const long long t = (long long)blockIdx.x * rows + group;
    if (t >= p.T) return;  // whole groups only: the group barriers stay complete
    const size_t row = size_t(t) * p.chunks;
    clear_unused(red[0][group], red[1][group], RED, lane, p.tpr);
    wait_for_previous();
    let_next_start();

    Raw8<HD> hr[NC];
    Raw8<YD> yr[NC];
    RawAny w1[NC], w2[NC], gr[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = lane + i * p.tpr;
        hr[i].zero();
        if (BRANCH) yr[i].zero();
        if (c >= p.chunks) continue;
        if (BRANCH) yr[i].load(p.y, row + c);
        hr[i].load(p.h, row + c);
        if (BRANCH && p.gate_kind >= GATE_CHANNEL)
            gr[i].load(p.gate, p.gate_f32, p.gate_kind == GATE_ELEMENT ? row + c : size_t(c));
        if (EARLY && BRANCH && p.post_w) w1[i].load(p.post_w, p.w_f32, c);
        if (EARLY && p.x && p.pre_w) w2[i].load(p.pre_w, p.w_f32, c);
    }
    float token = 1.0f;
    if (BRANCH && p.gate_kind == GATE_TOKEN) {
        token = load1(p.gate, p.gate_f32, t);
        if (p.sigmoid) token = sigmoid(token);
    }
    F8 h[NC];
    if (BRANCH) {
        F8 y[NC];
        float scale = p.block_scale * token;
#pragma unroll
        for (int i = 0; i < NC; ++i) y[i] = yr[i].get();
        if (p.post_norm) {
            float2 q = both(0.0f);
#pragma unroll
            for (int i = 0; i < NC; ++i) dot(y[i], y[i], q);
            scale *= rsqrtf(fmaf(group_sum(q.x + q.y, red[0][group], p.tpr, group, wig), p.inv_h, p.eps));
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            h[i] = hr[i].get();
            if (c >= p.chunks) continue;
            if (p.post_w) {
                if (!EARLY) w1[i].load(p.post_w, p.w_f32, c);
                y[i] = mul(y[i], add(w1[i].get(p.w_f32), p.w_offset));
            }
            if (p.gate_kind >= GATE_CHANNEL) {
                const F8 g = gr[i].get(p.gate_f32);
                y[i] = mul(y[i], p.sigmoid ? sigmoid(g) : g);
            }
            h[i] = fma(y[i], scale, mul(h[i], p.res_scale));
            store8<HD>(p.h_out, row + c, h[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NC; ++i) h[i] = hr[i].get();
    }
    if (!p.x) return;
    float2 q = both(0.0f);
#pragma unroll
    for (int i = 0; i < NC; ++i) dot(h[i], h[i], q);  // zero beyond the row
    const float r2 = rsqrtf(fmaf(group_sum(q.x + q.y, red[1][group], p.tpr, group, wig), p.inv_h, p.eps));
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = lane + i * p.tpr;
        if (c >= p.chunks) continue;
        F8 x = mul(h[i], r2);
        if (p.pre_w) {
            if (!EARLY) w2[i].load(p.pre_w, p.w_f32, c);
            x = mul(x, add(w2[i].get(p.w_f32), p.w_offset));
        }
        store8<XD>(p.x, row + c, x);
    }
}

// ---- long batches: blocks that stay and walk rows, the next rows in flight ----
//
// A thread copies its own 16-byte units of the rows ahead into shared memory, asynchronously, and
// reads only those: a row's arrival needs no barrier, and what is in flight needs no registers.
// What all rows share is combined once per block into two fp32 vectors in shared memory:
//   pre[c]  = w_offset + pre_w                              (1 without weights)
//   post[c] = block_scale act(gate) (w_offset + post_w)     (no or channel gate)
//             w_offset + post_w                             (token or element gate)
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
template <int U>
__device__ __forceinline__ F8 lds8(uint32_t at, int stride) {  // one chunk of U units
    const uint4 a = lds16(at);
    if constexpr (U == 2) return f32x8(a, lds16(at + stride));
    else return bf16x8(a);
}
__device__ __forceinline__ F8 lds8f(uint32_t at) { return f32x8(lds16(at), lds16(at + 16)); }
// The shared vectors lie as the chunks' first four values, then their last four: lanes at 16-byte steps
// use every bank once, where 32-byte steps would use every second one twice.
__device__ __forceinline__ void put_shared(float* to, int chunks, int c, const F8& v) {
    float4* p = reinterpret_cast<float4*>(to);
    p[c] = make_float4(v.v[0].x, v.v[0].y, v.v[1].x, v.v[1].y);
    p[chunks + c] = make_float4(v.v[2].x, v.v[2].y, v.v[3].x, v.v[3].y);
}
__device__ __forceinline__ F8 get_shared(uint32_t from, int chunks, int c) {
    return f32x8(lds16(from + 16 * c), lds16(from + 16 * (chunks + c)));
}

template <int U>
__device__ __forceinline__ void copy_units(uint32_t dst, int stride, const void* p, size_t chunk) {
    const uint4* src = static_cast<const uint4*>(p) + U * chunk;
#pragma unroll
    for (int i = 0; i < U; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst + i * stride), "l"(src + i) : "memory");
}
__device__ __forceinline__ void copy_gate(const NormParams& p, uint32_t dst, int stride, size_t chunk) {
    if (p.gate_f32) copy_units<2>(dst, stride, p.gate, chunk);
    else copy_units<1>(dst, stride, p.gate, chunk);
}
__device__ __forceinline__ void rows_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void rows_wait(int ahead) {  // all but the `ahead` newest
    if (ahead == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (ahead == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ void shared_vectors(const NormParams& p, bool branch, float* post, float* pre) {
    for (int c = threadIdx.x; c < p.chunks; c += blockDim.x) {
        RawAny a, b, g;
        if (p.pre_w) a.load(p.pre_w, p.w_f32, c);
        if (p.post_w) b.load(p.post_w, p.w_f32, c);
        const bool channel = branch && p.gate_kind == GATE_CHANNEL;
        if (channel) g.load(p.gate, p.gate_f32, c);
        put_shared(pre, p.chunks, c, p.pre_w ? add(a.get(p.w_f32), p.w_offset) : fill8(1.0f));
        F8 v = p.post_w ? add(b.get(p.w_f32), p.w_offset) : fill8(1.0f);
        if (channel) {
            const F8 w = g.get(p.gate_f32);
            v = mul(v, p.sigmoid ? sigmoid(w) : w);
        }
        if (channel || (branch && p.gate_kind == GATE_NONE)) v = mul(v, p.block_scale);
        put_shared(post, p.chunks, c, v);
    }
}

// dpost_w and a channel gate's gradient in column c from that column's A (see below).
__device__ __forceinline__ void finish_post(const NormParams& p, int c, float a) {
    float v = p.block_scale;  // block_scale act(gate)
    if (p.gate_kind == GATE_CHANNEL) {
        const float g = load1(p.gate, p.gate_f32, c), w = p.post_w ? p.w_offset + load1(p.post_w, p.w_f32, c) : 1.0f;
        const float act = p.sigmoid ? sigmoid(g) : g, dact = p.sigmoid ? sigmoid_slope(g) : 1.0f;
        if (p.want_gate) static_cast<float*>(p.dgate)[c] = a * (p.block_scale * dact) * w;
        v *= act;
    }
    if (p.want_post) p.dpost_w[c] = p.gate_kind == GATE_TOKEN || p.gate_kind == GATE_ELEMENT ? a : a * v;
}

__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t at, unsigned rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(at), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// Backward. The sums that a row needs are six, all of what is read:
//   S = {h^2, dx pre h, y^2, dh_out e, dx pre e, h e},  e = y post (times an element gate)
// since sum G e = S3 + r2 (S4 - k2 S5) with k2 = r2^2 S1 / H: one reduction a row, where summing G e
// itself would wait for a first one. Without an element or token gate, the gradients of post_w and of
// a channel gate are per-column multiples of one sum, A = sum_t G y r1: norm_columns_kernel makes
// both from it. With them A takes each row's gate in and is dpost_w itself.
template <int HD, int YD, int XD, int NC, bool BRANCH, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 2 : 1) norm_backward_kernel(const NormParams p) {
    constexpr int UH = HD == DT_F32 ? 2 : 1, UX = XD == DT_F32 ? 2 : 1, UY = BRANCH ? (YD == DT_F32 ? 2 : 1) : 0;
    constexpr int AT_G = UH, AT_X = 2 * UH, AT_Y = AT_X + UX, AT_GATE = AT_Y + UY;  // units: h_out, dh_out, dx, y, gate
    extern __shared__ __align__(16) float dyn[];  // post, pre [H] each, then the rows' units; at the end
                                                  // the column sums [groups - 1][2][H]
    constexpr int GROUPS = THREADS == 512 ? 1 : NORM_THREADS / 32;  // over 256 threads are one row's
    __shared__ __align__(16) float red[2][GROUPS][RED6];
    const int group = threadIdx.x / p.tpr, lane = threadIdx.x % p.tpr, wig = lane / 32;
    const int rows = blockDim.x / p.tpr;
    clear_unused(red[0][group], red[1][group], RED6, lane, p.tpr);
    const int stride = blockDim.x * 16, chunk_bytes = p.units * stride, stage_bytes = NC * chunk_bytes;
    const uint32_t post = smem_u32(dyn), pre = post + 4 * p.H, mine = pre + 4 * p.H + 16 * threadIdx.x;
    const bool has_x = p.dx != nullptr, has_g = p.dh_out != nullptr, post_norm = BRANCH && p.post_norm,
               element = BRANCH && p.gate_kind == GATE_ELEMENT, tokens = BRANCH && p.gate_kind == GATE_TOKEN;
    const long long step = (long long)gridDim.x * rows;
    long long t = (long long)blockIdx.x * rows + group;
    int in = 0, use = 0;
    auto ask = [&](long long r) {
        if (r < p.T) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = lane + i * p.tpr;
                if (c >= p.chunks) continue;
                const size_t k = size_t(r) * p.chunks + c;
                const uint32_t d = mine + in * stage_bytes + i * chunk_bytes;
                copy_units<UH>(d, stride, p.h, k);
                if (has_g) copy_units<UH>(d + AT_G * stride, stride, p.dh_out, k);
                if (has_x) copy_units<UX>(d + AT_X * stride, stride, p.dx, k);
                if constexpr (BRANCH) copy_units<UY>(d + AT_Y * stride, stride, p.y, k);
                if (element) copy_gate(p, d + AT_GATE * stride, stride, k);
            }
        }
        in = in == p.ahead ? 0 : in + 1;
        rows_commit();
    };
    wait_for_previous();
    for (int i = 0; i < p.ahead; ++i) ask(t + i * step);
    shared_vectors(p, BRANCH, dyn, dyn + p.H);
    __syncthreads();

    int turn = 0;
    F8 acc_pre[NC], acc_post[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) acc_pre[i] = acc_post[i] = fill8(0.0f);
    for (; t < p.T; t += step) {
        const size_t row = size_t(t) * p.chunks;
        float kappa = tokens || element ? p.block_scale : 1.0f, dtoken = 1.0f;
        if (tokens) {
            float token = load1(p.gate, p.gate_f32, t);
            if (p.sigmoid) {
                dtoken = sigmoid_slope(token);
                token = sigmoid(token);
            }
            kappa *= token;
        }
        ask(t + p.ahead * step);
        rows_wait(p.ahead);
        const uint32_t at = mine + use * stage_bytes;
        use = use == p.ahead ? 0 : use + 1;

        // a thread's one chunk stays in registers across the sums; two would not fit beside the
        // column sums and are read again
        F8 h, a, y, dho, v;
        auto read_gate = [&](uint32_t u) {
            return p.gate_f32 ? lds8<2>(u + AT_GATE * stride, stride) : lds8<1>(u + AT_GATE * stride, stride);
        };
        auto read = [&](uint32_t u) {
            h = lds8<UH>(u, stride);
            if (has_g) dho = lds8<UH>(u + AT_G * stride, stride);
            else dho = fill8(0.0f);
            if (has_x) a = lds8<UX>(u + AT_X * stride, stride);
            if constexpr (BRANCH) {
                y = lds8<UY>(u + AT_Y * stride, stride);
                if (element) {
                    v = read_gate(u);
                    if (p.sigmoid) v = sigmoid(v);
                }
            }
        };
        float s[6];
        {
            float2 q[6];
#pragma unroll
            for (int i = 0; i < 6; ++i) q[i] = both(0.0f);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = lane + i * p.tpr;
                if (c >= p.chunks) continue;
                read(at + i * chunk_bytes);
                F8 e;
                if constexpr (BRANCH) {
                    e = mul(y, get_shared(post, p.chunks, c));
                    if (element) e = mul(e, v);
                    dot(y, y, q[2]);
                    dot(dho, e, q[3]);
                }
                if (has_x) {
                    const F8 ap = mul(a, get_shared(pre, p.chunks, c));
                    dot(h, h, q[0]);
                    dot(ap, h, q[1]);
                    if constexpr (BRANCH) {
                        dot(ap, e, q[4]);
                        dot(h, e, q[5]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 6; ++i) s[i] = q[i].x + q[i].y;
        }
        group_sum6(s, red[turn][group], p.tpr, group, wig);
        turn ^= 1;
        // a norm whose row passes the fp32 range of its squares (r = 0) is constant there: it sends nothing
        // back, and the other sums over that row may be infinite
        const float r2 = rsqrtf(fmaf(s[0], p.inv_h, p.eps)), k2 = r2 == 0.0f ? 0.0f : r2 * r2 * (s[1] * p.inv_h);
        const float r1 = post_norm ? rsqrtf(fmaf(s[2], p.inv_h, p.eps)) : 1.0f;
        float sum = has_x && r2 != 0.0f ? fmaf(r2, fmaf(-k2, s[5], s[4]), s[3]) : s[3];  // of G e
        if (r1 == 0.0f) sum = 0.0f;
        const float k1 = post_norm ? r1 * r1 * (sum * p.inv_h) : 0.0f, f1 = r1 * kappa;
        if (tokens && p.dgate && lane == 0)
            static_cast<float*>(p.dgate)[t] = p.block_scale * dtoken * r1 * sum;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            if (c >= p.chunks) continue;
            if (NC > 1) read(at + i * chunk_bytes);
            F8 G = dho;
            if (has_x) {
                acc_pre[i] = fma(a, mul(h, r2), acc_pre[i]);
                G = fma(fma(h, -k2, mul(a, get_shared(pre, p.chunks, c))), r2, G);
            }
            if constexpr (!BRANCH) {
                store8<HD>(p.dh, row + c, G);
            } else {
                store8<HD>(p.dh, row + c, mul(G, p.res_scale));
                F8 w = get_shared(post, p.chunks, c);
                if (element) {
                    if (p.dgate) {
                        F8 dg = mul(mul(G, mul(y, f1)), w);
                        if (p.sigmoid) dg = mul(dg, sigmoid_slope(read_gate(at + i * chunk_bytes)));
                        if (p.gate_f32) store8<DT_F32>(p.dgate, row + c, dg);
                        else store8<DT_BF16>(p.dgate, row + c, dg);
                    }
                    G = mul(G, v);
                }
                acc_post[i] = fma(G, mul(y, f1), acc_post[i]);
                store8<YD>(p.dy, row + c, mul(fma(y, -k1, mul(G, w)), f1));
            }
        }
    }
    let_next_start();  // norm_columns_kernel, if there is a part
    if (!p.part) return;
    // the groups' column sums, added in group order by group 0
    __syncthreads();
    if (group > 0) {
        float* m = dyn + size_t(group - 1) * 2 * p.H;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            if (c >= p.chunks) continue;
            store8<DT_F32>(m, c, acc_pre[i]);
            store8<DT_F32>(m + p.H, c, acc_post[i]);
        }
    }
    __syncthreads();
    if (group == 0) {
        float* out = p.cluster ? dyn : p.part + size_t(blockIdx.x) * 2 * p.H;  // dyn: over what this thread has read
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            if (c >= p.chunks) continue;
            for (int g = 0; g + 1 < rows; ++g) {
                const uint32_t m = post + 4 * (g * 2 * p.H + 8 * c);
                const F8 u = lds8f(m), v = lds8f(m + 4 * p.H);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc_pre[i].v[j] = __fadd2_rn(acc_pre[i].v[j], u.v[j]);
                    acc_post[i].v[j] = __fadd2_rn(acc_post[i].v[j], v.v[j]);
                }
            }
            if (p.cluster || p.want_pre) store8<DT_F32>(out, c, acc_pre[i]);
            if (p.cluster || p.want_post || p.want_gate) store8<DT_F32>(out + p.H, c, acc_post[i]);
        }
    }
    if (!p.cluster) return;
    // every block adds a share of the columns over the blocks, in block order
    cluster_sync();
    const int share = (p.H + gridDim.x - 1) / gridDim.x, c0 = int(blockIdx.x) * share, c1 = min(c0 + share, p.H);
    for (int c = c0 + threadIdx.x; c < c1; c += blockDim.x) {
        float a = 0.0f, b = 0.0f;
#pragma unroll 8
        for (unsigned r = 0; r < gridDim.x; ++r) {
            a += ld_cluster(post + 4 * c, r);
            b += ld_cluster(post + 4 * (p.H + c), r);
        }
        if (p.want_pre) p.dpre_w[c] = a;
        if (p.want_post || p.want_gate) finish_post(p, c, b);
    }
    cluster_sync();  // no block leaves while another reads its sums
}

// dpre_w[col] = sum over blocks of part[block][0][col]; A[col] likewise from part[block][1] gives
// dpost_w and a channel gate's gradient. 32 slices of the blocks, each in block order, then the
// slices in order; a thread has four columns.
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormParams p, int blocks) {
    __shared__ float4 sums[32][8];
    const int which = blockIdx.y, q = threadIdx.x & 7, slice = threadIdx.x >> 3;
    if (which == 0 ? !p.want_pre : !(p.want_post || p.want_gate)) return;
    const int col = blockIdx.x * 32 + 4 * q;
    wait_for_previous();
    let_next_start();
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (col < p.H) {
        const float* src = p.part + size_t(which) * p.H + col;
        constexpr int EACH = MAX_SMS * MAX_BLOCKS_SM / 32;  // all of a slice in flight at once
        float4 v[EACH];
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int b = slice + 32 * i;
            v[i] = b < blocks ? __ldcg(reinterpret_cast<const float4*>(src + size_t(b) * 2 * p.H)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            s.x += v[i].x; s.y += v[i].y; s.z += v[i].z; s.w += v[i].w;
        }
    }
    sums[slice][q] = s;
    __syncthreads();
    const int c = blockIdx.x * 32 + threadIdx.x;
    if (threadIdx.x >= 32 || c >= p.H) return;
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) a += reinterpret_cast<const float*>(&sums[i][threadIdx.x >> 2])[threadIdx.x & 3];
    if (which == 0) p.dpre_w[c] = a;
    else finish_post(p, c, a);
}

// ------------------------------------------------------------------------------ host side
struct NormShape {
    int nc, tpr, rows;  // chunks a thread, threads a row, rows a block
};
// A thread has one chunk of a row while the rows' warps find room on the device at once (the shortest
// way through a row: 512 rows of 2048 take 3.4 us, 3.7 with two), two where they do not (half the
// threads at a barrier, twice the loads in flight of each: 1024 rows 5.2 against 6.0, 4096 rows 16.1
// against 17.5) and where 512 threads would not do.
NormShape norm_shape(int H, long long T, int sm_count) {
    NormShape s;
    const int chunks = H / 8;
    s.nc = chunks > 512 || (chunks > 32 && T * ((chunks + 31) / 32) > 32ll * sm_count) ? 2 : 1;
    s.tpr = ((chunks + s.nc - 1) / s.nc + 31) / 32 * 32;
    s.rows = s.tpr >= NORM_THREADS ? 1 : NORM_THREADS / s.tpr;
    return s;
}

constexpr int MAX_CLUSTER = 8;  // blocks that add their column sums among themselves

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t dt_bytes(int dt) { return dt == DT_F32 ? 4 : 2; }
bool float_dt(int dt) { return dt == DT_F32 || dt == DT_BF16; }

struct Range {
    const char* p;
    size_t n;
};
bool overlap(Range a, Range b) { return a.p && b.p && a.p < b.p + b.n && b.p < a.p + a.n; }

size_t gate_elems(const redmoe_norm* N, int T) {
    switch (N->gate_kind) {
        case GATE_TOKEN: return T;
        case GATE_CHANNEL: return N->hidden;
        case GATE_ELEMENT: return size_t(T) * N->hidden;
        default: return 0;
    }
}

bool finite(float f) { return f - f == 0.0f; }

redmoe_status check_norm(const redmoe_norm* N) {
    if (!N) return REDMOE_ERR_INVALID_ARG;
    if (N->hidden < 8 || N->hidden % 8) return REDMOE_ERR_INVALID_ARG;
    const int dts[] = {N->h_dtype, N->y_dtype, N->x_dtype, N->w_dtype, N->gate_dtype};
    for (int d : dts) {
        if (d < 0 || d > DT_INT2) return REDMOE_ERR_INVALID_ARG;
        if (!float_dt(d)) return REDMOE_ERR_UNSUPPORTED;
    }
    if (N->gate_kind < GATE_NONE || N->gate_kind > GATE_ELEMENT) return REDMOE_ERR_INVALID_ARG;
    if (N->gate_act != 0 && N->gate_act != 1) return REDMOE_ERR_INVALID_ARG;
    if (N->post_norm != 0 && N->post_norm != 1) return REDMOE_ERR_INVALID_ARG;
    if (!(N->eps > 0.0f) || !finite(N->eps) || !finite(N->w_offset) || !finite(N->res_scale) || !finite(N->block_scale))
        return REDMOE_ERR_INVALID_ARG;
    if (!aligned(N->post_w, 16) || !aligned(N->pre_w, 16)) return REDMOE_ERR_INVALID_ARG;
    if (N->post_w && !N->post_norm) return REDMOE_ERR_INVALID_ARG;
    if (N->hidden > NORM_MAX_H) return REDMOE_ERR_UNSUPPORTED;
    return REDMOE_OK;
}

NormParams base_params(const redmoe_norm* N, int T, const void* gate, const NormShape& s) {
    NormParams p = {};
    p.T = T;
    p.H = N->hidden;
    p.chunks = N->hidden / 8;
    p.tpr = s.tpr;
    p.post_norm = N->post_norm;
    p.gate_kind = N->gate_kind;
    p.sigmoid = N->gate_act;
    p.gate_f32 = N->gate_dtype == DT_F32;
    p.w_f32 = N->w_dtype == DT_F32;
    p.eps = N->eps;
    p.w_offset = N->w_offset;
    p.res_scale = N->res_scale;
    p.block_scale = N->block_scale;
    p.inv_h = 1.0f / float(N->hidden);
    p.post_w = N->post_w;
    p.pre_w = N->pre_w;
    p.gate = gate;
    return p;
}

using NormKernel = void (*)(NormParams);

// Every combination of types; without y its type does not matter.
#define NORM_TYPES(kernel, ...)                                                                                        \
    (hd ? (yd ? (xd ? kernel<1, 1, 1, __VA_ARGS__> : kernel<1, 1, 0, __VA_ARGS__>)                                     \
              : (xd ? kernel<1, 0, 1, __VA_ARGS__> : kernel<1, 0, 0, __VA_ARGS__>))                                    \
        : (yd ? (xd ? kernel<0, 1, 1, __VA_ARGS__> : kernel<0, 1, 0, __VA_ARGS__>)                                     \
              : (xd ? kernel<0, 0, 1, __VA_ARGS__> : kernel<0, 0, 0, __VA_ARGS__>)))
#define NORM_ROWS(kernel, B)                                                                                           \
    (nc == 2 ? (threads <= 256 ? NORM_TYPES(kernel, 2, B, 256) : NORM_TYPES(kernel, 2, B, 512))                        \
             : (threads <= 256 ? NORM_TYPES(kernel, 1, B, 256) : NORM_TYPES(kernel, 1, B, 512)))

NormKernel pick_forward(const redmoe_norm* N, int nc, bool branch) {
    const bool hd = N->h_dtype == DT_BF16, xd = N->x_dtype == DT_BF16, yd = branch && N->y_dtype == DT_BF16;
    if (branch) return nc == 1 ? NORM_TYPES(norm_forward_kernel, 1, true) : NORM_TYPES(norm_forward_kernel, 2, true);
    return nc == 1 ? NORM_TYPES(norm_forward_kernel, 1, false) : NORM_TYPES(norm_forward_kernel, 2, false);
}
NormKernel pick_backward(const redmoe_norm* N, int nc, int threads, bool branch) {
    const bool hd = N->h_dtype == DT_BF16, xd = N->x_dtype == DT_BF16, yd = branch && N->y_dtype == DT_BF16;
    return branch ? NORM_ROWS(norm_backward_kernel, true) : NORM_ROWS(norm_backward_kernel, false);
}
#undef NORM_ROWS
#undef NORM_TYPES

int units(int dt) { return dt == DT_F32 ? 2 : 1; }

// Shared memory of a kernel that walks rows, and with it p.ahead: two rows in flight where `want` blocks
// of an SM can hold them, else one, else none. Where two blocks cannot even hold the row that each works
// on, `want` becomes one block, which then has rows in flight (4096 fp32 rows of 4096 with an fp32 element
// gate: 156 us, 194 as two waves of blocks). Two blocks without a row in flight stay: 8192 fp32 rows of 2048
// take 107 us, one block with rows ahead 116; 4096 x 4096 bf16 with an fp32 y 65 and 69 (but 300 such rows
// 15.6 and 14.3).
int rows_smem(NormParams& p, const NormShape& s, int& want, int max_smem) {
    const int stage = s.nc * p.units * s.tpr * s.rows * 16, fixed = 2 * p.H * 4;
    const int own = 2 * (s.tpr * s.rows > 256 ? 1 : 8) * RED6 * 4 + 64;  // static
    auto room = [&] { return max_smem / want - own - (want > 1 ? 1024 : 0); };  // 1 KiB of every block is the system's
    if (fixed + stage > room()) want = 1;
    p.ahead = 2;
    while (p.ahead > 0 && fixed + (p.ahead + 1) * stage > room()) --p.ahead;
    const int smem = fixed + (p.ahead + 1) * stage, ends = (s.rows - 1) * 2 * p.H * 4;
    return smem > ends ? smem : ends;
}

}  // namespace

redmoe_status norm_forward_check(const redmoe_norm* N, const void* h, const void* y, const void* gate, int T,
                                 const void* h_out, const void* x) {
    const redmoe_status st = check_norm(N);
    if (st != REDMOE_OK) return st;
    if (T < 0) return REDMOE_ERR_INVALID_ARG;
    if (T == 0) return REDMOE_OK;
    const bool branch = y != nullptr;
    if (!h || !aligned(h, 16) || !aligned(y, 16) || !aligned(h_out, 16) || !aligned(x, 16))
        return REDMOE_ERR_INVALID_ARG;
    if (branch ? !h_out : (h_out || !x || gate)) return REDMOE_ERR_INVALID_ARG;
    if (branch && (N->gate_kind != GATE_NONE) != (gate != nullptr)) return REDMOE_ERR_INVALID_ARG;
    if (gate && !aligned(gate, N->gate_kind == GATE_TOKEN ? dt_bytes(N->gate_dtype) : 16)) return REDMOE_ERR_INVALID_ARG;
    const size_t n = size_t(T) * N->hidden, wb = norm_weight_bytes(N);
    const Range rh{static_cast<const char*>(h), n * dt_bytes(N->h_dtype)};
    const Range ro{static_cast<const char*>(h_out), n * dt_bytes(N->h_dtype)};
    const Range rx{static_cast<const char*>(x), n * dt_bytes(N->x_dtype)};
    const Range in[] = {{static_cast<const char*>(y), n * dt_bytes(N->y_dtype)},
                        {static_cast<const char*>(gate), norm_gate_bytes(N, T)},
                        {static_cast<const char*>(N->pre_w), wb},
                        {static_cast<const char*>(N->post_w), wb}};
    for (const Range& r : in)
        if (overlap(r, ro) || overlap(r, rx)) return REDMOE_ERR_INVALID_ARG;
    if (overlap(rh, rx) || overlap(ro, rx) || (h_out != h && overlap(rh, ro))) return REDMOE_ERR_INVALID_ARG;
    return REDMOE_OK;
}

size_t norm_gate_bytes(const redmoe_norm* N, int T) { return gate_elems(N, T) * dt_bytes(N->gate_dtype); }
size_t norm_weight_bytes(const redmoe_norm* N) { return dt_bytes(N->w_dtype) * N->hidden; }

}  // namespace redmoe

using namespace redmoe;

extern "C" {

redmoe_status redmoe_norm_forward(const redmoe_norm* N, const void* h, const void* y, const void* gate, int32_t T,
                                  void* h_out, void* x, void* stream) {
    const redmoe_status st = norm_forward_check(N, h, y, gate, T, h_out, x);
    if (st != REDMOE_OK || T == 0) return st;
    const bool branch = y != nullptr;
    DevInfo di;
    if (!get_dev_info(&di)) return REDMOE_ERR_CUDA;
    const NormShape s = norm_shape(N->hidden, T, di.sm_count);
    NormParams p = base_params(N, T, gate, s);
    p.h = h;
    p.y = y;
    p.h_out = h_out;
    p.x = x;
    const long long need = (T + (long long)s.rows - 1) / s.rows;
    const int threads = s.tpr * s.rows;
    const NormKernel kern = pick_forward(N, s.nc, branch);
    return launch(kern, dim3(unsigned(need)), threads, 0, static_cast<cudaStream_t>(stream), 1, p) ? REDMOE_OK
                                                                                                       : REDMOE_ERR_CUDA;
}

size_t redmoe_norm_workspace_bytes(const redmoe_norm* N, int32_t T) {
    if (T < 0 || check_norm(N) != REDMOE_OK) return 0;
    const long long blocks = T < MAX_SMS * MAX_BLOCKS_SM ? T : MAX_SMS * MAX_BLOCKS_SM;  // a row each, at most
    return 256 + align256(size_t(blocks) * 2 * N->hidden * 4);
}

redmoe_status redmoe_norm_backward(const redmoe_norm* N, const void* h_out, const void* y, const void* gate,
                                   const void* dh_out, const void* dx, int32_t T, void* dh, void* dy, void* dgate,
                                   float* dpost_w, float* dpre_w, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    redmoe_status st = check_norm(N);
    if (st != REDMOE_OK) return st;
    if (T < 0) return REDMOE_ERR_INVALID_ARG;
    const bool branch = y != nullptr;
    const bool channel = N->gate_kind == GATE_CHANNEL;
    const void* ptrs[] = {h_out, y, dh_out, dx, dh, dy, dpost_w, dpre_w};
    for (const void* q : ptrs)
        if (!aligned(q, 16)) return REDMOE_ERR_INVALID_ARG;
    if (!aligned(gate, N->gate_kind == GATE_TOKEN ? dt_bytes(N->gate_dtype) : 16) ||
        !aligned(dgate, N->gate_kind == GATE_TOKEN ? 4 : 16))
        return REDMOE_ERR_INVALID_ARG;
    if (dpost_w && (!N->post_norm || !N->post_w)) return REDMOE_ERR_INVALID_ARG;
    if (dpre_w && !N->pre_w) return REDMOE_ERR_INVALID_ARG;
    if (dgate && N->gate_kind == GATE_NONE) return REDMOE_ERR_INVALID_ARG;
    cudaStream_t stm = static_cast<cudaStream_t>(stream);
    const size_t cb = 4ull * N->hidden;
    if (T == 0) {  // no rows: the gradients of what all rows share are zero
        float* zero[] = {dpost_w, dpre_w, channel ? static_cast<float*>(dgate) : nullptr};
        for (float* z : zero)
            if (z && cudaMemsetAsync(z, 0, cb, stm) != cudaSuccess) return REDMOE_ERR_CUDA;
        return REDMOE_OK;
    }
    if (!h_out || !dh || (!dh_out && !dx) || (dpre_w && !dx)) return REDMOE_ERR_INVALID_ARG;
    if (branch ? !dy : (dy || gate || dgate || dpost_w)) return REDMOE_ERR_INVALID_ARG;
    if (branch && (N->gate_kind != GATE_NONE) != (gate != nullptr)) return REDMOE_ERR_INVALID_ARG;
    const size_t n = size_t(T) * N->hidden, wb = dt_bytes(N->w_dtype) * N->hidden, ge = gate_elems(N, T);
    const size_t hb = n * dt_bytes(N->h_dtype), yb = n * dt_bytes(N->y_dtype);
    const Range in[] = {{static_cast<const char*>(h_out), hb},
                        {static_cast<const char*>(y), yb},
                        {static_cast<const char*>(gate), ge * dt_bytes(N->gate_dtype)},
                        {static_cast<const char*>(dh_out), hb},
                        {static_cast<const char*>(dx), n * dt_bytes(N->x_dtype)},
                        {static_cast<const char*>(N->pre_w), wb},
                        {static_cast<const char*>(N->post_w), wb}};
    const bool work = dpost_w || dpre_w || (dgate && channel);
    const size_t need = redmoe_norm_workspace_bytes(N, T);
    if (work && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return REDMOE_ERR_WORKSPACE;
    const Range out[] = {{static_cast<const char*>(dh), hb},
                         {static_cast<const char*>(dy), yb},
                         {static_cast<const char*>(dgate),
                          ge * (N->gate_kind == GATE_ELEMENT ? dt_bytes(N->gate_dtype) : 4)},
                         {reinterpret_cast<const char*>(dpost_w), cb},
                         {reinterpret_cast<const char*>(dpre_w), cb},
                         {static_cast<const char*>(work ? workspace : nullptr), need}};
    for (int i = 0; i < 6; ++i) {
        for (const Range& r : in)
            if (overlap(r, out[i]) && !(i == 0 && r.p == dh_out && dh == dh_out)) return REDMOE_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return REDMOE_ERR_INVALID_ARG;
    }
    DevInfo di;
    if (!get_dev_info(&di)) return REDMOE_ERR_CUDA;
    const NormShape s = norm_shape(N->hidden, T, di.sm_count);
    NormParams p = base_params(N, T, gate, s);
    p.h = h_out;
    p.y = y;
    p.dh_out = dh_out;
    p.dx = dx;
    p.dh = dh;
    p.dy = dy;
    p.dgate = dgate;
    p.part = work ? reinterpret_cast<float*>(static_cast<char*>(workspace) + 256) : nullptr;
    p.dpre_w = dpre_w;
    p.dpost_w = dpost_w;
    p.want_pre = dpre_w != nullptr;
    p.want_post = dpost_w != nullptr;
    p.want_gate = dgate != nullptr && channel;
    p.units = 2 * units(N->h_dtype) + units(N->x_dtype) + (branch ? units(N->y_dtype) : 0) +
              (branch && N->gate_kind == GATE_ELEMENT ? units(N->gate_dtype) : 0);
    const int threads = s.tpr * s.rows;
    int want = threads <= 256 ? MAX_BLOCKS_SM : 1;
    const int smem = rows_smem(p, s, want, di.max_smem_optin);
    const long long all = (T + (long long)s.rows - 1) / s.rows, most = want * (di.sm_count < MAX_SMS ? di.sm_count : MAX_SMS);
    // Where eight blocks have no more than two of their rows each, they are one cluster that adds its
    // column sums itself: 4.2 against 4.7 us for one row of 2048, and a launch less for the host (about
    // 2.5 us a call). 16 rows of 2048 take 5.3 instead of 4.9, as the host's 2.5 are worth.
    p.cluster = work && all <= 2 * MAX_CLUSTER;
    int blocks = int(all < most ? all : most);
    if (p.cluster) {
        blocks = 1;
        while (blocks < all && blocks < MAX_CLUSTER) blocks *= 2;  // those without rows add zeros
    }
    const NormKernel kern = pick_backward(N, s.nc, threads, branch);
    if (!allow_smem(reinterpret_cast<const void*>(kern), smem)) return REDMOE_ERR_CUDA;
    if (!launch(kern, dim3(blocks), threads, smem, stm, p.cluster ? blocks : 1, p)) return REDMOE_ERR_CUDA;
    if (!work || p.cluster) return REDMOE_OK;
    return launch(norm_columns_kernel, dim3((p.H + 31) / 32, 2), 256, 0, stm, 1, p, blocks) ? REDMOE_OK : REDMOE_ERR_CUDA;
}

}  // extern "C"
