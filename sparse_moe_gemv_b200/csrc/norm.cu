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
// reads h_out, y, dh_out and dx once and writes dh and dy once. A row lies in the registers of
// a group of threads (whole warps, eight columns a thread), so the statistics cost one
// reduction over the group each and nothing is read twice. All sums are fp32, in a fixed
// order.
#include "common.cuh"
#include "internal.h"
#include "norm.h"
#include "vec8.cuh"

namespace redmoe {
namespace {

constexpr int NORM_MAX_H = 8192;
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
    float* part;  // backward: [blocks][3][H] column sums (pre_w, post_w, channel gate)
    bool want_pre, want_post, want_gate;
};

// Sums of N values over the group: warps by shuffles, then the warps' sums through shared
// memory in warp order. `buf` alternates between two areas from call to call, so that one
// barrier a call is enough: an area is written again only behind the barrier of the call
// between, which every thread reaches after its reads.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* buf, int tpr, int group, int wig) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    if (tpr == 32) return;
    const int nw = tpr / 32;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) buf[wig * N + i] = v[i];
    }
    asm volatile("bar.sync %0, %1;" :: "r"(group + 1), "r"(tpr) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    for (int w = 0; w < nw; ++w) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += buf[w * N + i];
    }
}

__device__ __forceinline__ float sigmoid(float a) { return 1.0f / (1.0f + expf(-a)); }

__device__ __forceinline__ void gate8(const NormParams& p, int t, int c, float (&g)[8]) {
    if (p.gate_kind == GATE_ELEMENT) {
        load8_shared(p.gate, p.gate_f32, size_t(t) * p.chunks + c, g);
    } else if (p.gate_kind == GATE_CHANNEL) {
        load8_shared(p.gate, p.gate_f32, c, g);
    } else {
        const float v = load1(p.gate, p.gate_f32, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = v;
    }
}

// One row per group of p.tpr threads; NC chunks a thread (chunk c = thread + i tpr).
template <int HD, int YD, int XD, int NC, bool BRANCH>
__global__ void __launch_bounds__(512) norm_forward_kernel(const NormParams p) {
    __shared__ float red[2][32];
    const int group = threadIdx.x / p.tpr, lane = threadIdx.x % p.tpr, wig = lane / 32;
    const int rows = blockDim.x / p.tpr;
    const long long t = (long long)blockIdx.x * rows + group;
    if (t >= p.T) return;  // whole groups only: the group barriers stay complete
    const int wbase = group * (p.tpr / 32);
    const size_t row = size_t(t) * p.chunks;

    Raw8<HD> hr[NC];
    Raw8<YD> yr[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = lane + i * p.tpr;
        if (c < p.chunks) {
            if (BRANCH) yr[i].load(p.y, row + c);
            hr[i].load(p.h, row + c);
        } else {
            if (BRANCH) yr[i].zero();
            hr[i].zero();
        }
    }
    float h[NC][8];
    if (BRANCH) {
        float y[NC][8];
        float r1 = 1.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) yr[i].get(y[i]);
        if (p.post_norm) {
            float s[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) s[0] = fmaf(y[i][j], y[i][j], s[0]);
            group_sum<1>(s, red[0] + wbase, p.tpr, group, wig);
            r1 = rsqrtf(fmaf(s[0], p.inv_h, p.eps));
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            hr[i].get(h[i]);
            if (c >= p.chunks) continue;
            float u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = y[i][j] * r1;
            if (p.post_norm && p.post_w) {
                float w[8];
                load8_shared(p.post_w, p.w_f32, c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] *= p.w_offset + w[j];
            }
            if (p.gate_kind != GATE_NONE) {
                float g[8];
                gate8(p, int(t), c, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] *= p.sigmoid ? sigmoid(g[j]) : g[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = fmaf(p.res_scale, h[i][j], p.block_scale * u[j]);
            store8<HD>(p.h_out, row + c, h[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NC; ++i) hr[i].get(h[i]);
    }
    if (!p.x) return;
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] = fmaf(h[i][j], h[i][j], s[0]);  // zero beyond the row
    group_sum<1>(s, red[1] + wbase, p.tpr, group, wig);
    const float r2 = rsqrtf(fmaf(s[0], p.inv_h, p.eps));
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = lane + i * p.tpr;
        if (c >= p.chunks) continue;
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = h[i][j] * r2;
        if (p.pre_w) {
            float w[8];
            load8_shared(p.pre_w, p.w_f32, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= p.w_offset + w[j];
        }
        store8<XD>(p.x, row + c, x);
    }
}

// Backward: each group walks rows blockIdx * rows + group, + gridDim * rows, ... and keeps the
// column sums of its rows in registers; the block adds its groups' sums in order and stores
// one partial row per weight, which norm_columns_kernel adds over the blocks.
template <int HD, int YD, int XD, int NC, bool BRANCH>
__global__ void __launch_bounds__(512) norm_backward_kernel(const NormParams p) {
    extern __shared__ __align__(16) float cols[];  // [groups - 1][3][chunks * 8] where groups > 1
    __shared__ float red[2][3 * 32];
    const int group = threadIdx.x / p.tpr, lane = threadIdx.x % p.tpr, wig = lane / 32;
    const int rows = blockDim.x / p.tpr;
    const int wbase = group * (p.tpr / 32);
    int turn = 0;
    float acc_pre[NC][8] = {}, acc_post[NC][8] = {}, acc_gate[NC][8] = {};

    for (long long t = (long long)blockIdx.x * rows + group; t < p.T; t += (long long)gridDim.x * rows) {
        const size_t row = size_t(t) * p.chunks;
        Raw8<HD> hr[NC], gr[NC];
        Raw8<YD> yr[NC];
        Raw8<XD> xr[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            const bool in = c < p.chunks;
            hr[i].zero(); gr[i].zero(); xr[i].zero(); yr[i].zero();
            if (in) hr[i].load(p.h, row + c);
            if (in && p.dx) xr[i].load(p.dx, row + c);
            if (in && p.dh_out) gr[i].load(p.dh_out, row + c);
            if (BRANCH && in) yr[i].load(p.y, row + c);
        }
        float h[NC][8], G[NC][8], y[NC][8];
        float s[3] = {0.0f, 0.0f, 0.0f};  // h_out^2, dx w2 h_out, y^2
        float a[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            hr[i].get(h[i]);
            xr[i].get(a[i]);
            if (BRANCH) yr[i].get(y[i]);
            float w[8];
            if (p.dx && p.pre_w && c < p.chunks) {
                load8_shared(p.pre_w, p.w_f32, c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] += p.w_offset;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 1.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[0] = fmaf(h[i][j], h[i][j], s[0]);
                s[1] = fmaf(a[i][j] * w[j], h[i][j], s[1]);
                if (BRANCH) s[2] = fmaf(y[i][j], y[i][j], s[2]);
                G[i][j] = a[i][j] * w[j];
            }
        }
        group_sum<3>(s, red[turn] + 3 * wbase, p.tpr, group, wig);
        turn ^= 1;
        const float r2 = rsqrtf(fmaf(s[0], p.inv_h, p.eps));
        const float k2 = r2 * r2 * (s[1] * p.inv_h);
        const float r1 = BRANCH && p.post_norm ? rsqrtf(fmaf(s[2], p.inv_h, p.eps)) : 1.0f;
        float q[2] = {0.0f, 0.0f};  // d w1 y, and the token gate's b u
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            if (c >= p.chunks) continue;
            float dho[8], dh[8];
            gr[i].get(dho);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (p.dx) {
                    acc_pre[i][j] = fmaf(a[i][j] * r2, h[i][j], acc_pre[i][j]);
                    G[i][j] = fmaf(r2, G[i][j] - h[i][j] * k2, dho[j]);
                } else {
                    G[i][j] = dho[j];
                }
                dh[j] = BRANCH ? p.res_scale * G[i][j] : G[i][j];
            }
            store8<HD>(p.dh, row + c, dh);
            if (!BRANCH) continue;
            float w1[8];
            if (p.post_norm && p.post_w) {
                load8_shared(p.post_w, p.w_f32, c, w1);
#pragma unroll
                for (int j = 0; j < 8; ++j) w1[j] += p.w_offset;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) w1[j] = 1.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) G[i][j] *= p.block_scale;  // b
            if (p.gate_kind != GATE_NONE) {
                float g[8], dg[8];
                gate8(p, int(t), c, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float v = g[j], dv = 1.0f;
                    if (p.sigmoid) {
                        v = sigmoid(v);
                        dv = v * (1.0f - v);
                    }
                    dg[j] = G[i][j] * (y[i][j] * r1 * w1[j]) * dv;
                    G[i][j] *= v;  // d
                    q[1] += dg[j];
                    if (p.gate_kind == GATE_CHANNEL) acc_gate[i][j] += dg[j];
                }
                if (p.gate_kind == GATE_ELEMENT && p.dgate) {
                    if (p.gate_f32) store8<DT_F32>(p.dgate, row + c, dg);
                    else store8<DT_BF16>(p.dgate, row + c, dg);
                }
            }
            if (p.post_norm) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc_post[i][j] = fmaf(G[i][j] * r1, y[i][j], acc_post[i][j]);
                    G[i][j] *= w1[j];  // c
                    q[0] = fmaf(G[i][j], y[i][j], q[0]);
                }
            } else {
                store8<YD>(p.dy, row + c, G[i]);
            }
        }
        if (!BRANCH || !(p.post_norm || p.gate_kind == GATE_TOKEN)) continue;
        group_sum<2>(q, red[turn] + 3 * wbase, p.tpr, group, wig);
        turn ^= 1;
        if (p.gate_kind == GATE_TOKEN && p.dgate && lane == 0) static_cast<float*>(p.dgate)[t] = q[1];
        if (!p.post_norm) continue;
        const float k1 = r1 * r1 * (q[0] * p.inv_h);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            if (c >= p.chunks) continue;
            float dy[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) dy[j] = r1 * (G[i][j] - y[i][j] * k1);
            store8<YD>(p.dy, row + c, dy);
        }
    }
    if (!p.part) return;
    // the groups' column sums, added in group order by group 0
    if (group > 0) {
        float* m = cols + size_t(group - 1) * 3 * p.H;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            if (c >= p.chunks) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                m[c * 8 + j] = acc_pre[i][j];
                m[p.H + c * 8 + j] = acc_post[i][j];
                m[2 * p.H + c * 8 + j] = acc_gate[i][j];
            }
        }
    }
    __syncthreads();
    if (group > 0) return;
    float* out = p.part + size_t(blockIdx.x) * 3 * p.H;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = lane + i * p.tpr;
        if (c >= p.chunks) continue;
        for (int g = 0; g + 1 < rows; ++g) {
            const float* m = cols + size_t(g) * 3 * p.H;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                acc_pre[i][j] += m[c * 8 + j];
                acc_post[i][j] += m[p.H + c * 8 + j];
                acc_gate[i][j] += m[2 * p.H + c * 8 + j];
            }
        }
        if (p.want_pre) store8<DT_F32>(out, c, acc_pre[i]);
        if (p.want_post) store8<DT_F32>(out + p.H, c, acc_post[i]);
        if (p.want_gate) store8<DT_F32>(out + 2 * p.H, c, acc_gate[i]);
    }
}

// out[which][col] = sum over blocks of part[block][which][col], in block order within each of
// eight slices, then over the slices.
__global__ void __launch_bounds__(256) norm_columns_kernel(const float* part, int blocks, int H, float* dpre,
                                                           float* dpost, float* dgate) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    float* out = blockIdx.y == 0 ? dpre : (blockIdx.y == 1 ? dpost : dgate);
    if (!out) return;
    const int col = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (col < H) {
        const float* src = part + size_t(blockIdx.y) * H + col;
        for (int b = slice; b < blocks; b += 8) s += src[size_t(b) * 3 * H];
    }
    sums[slice][lane] = s;
    __syncthreads();
    if (slice == 0 && col < H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sums[i][lane];
        out[col] = s;
    }
}

// ------------------------------------------------------------------------------ host side
struct NormShape {
    int nc, tpr, rows;  // chunks a thread, threads a row, rows a block
};
NormShape norm_shape(int H) {
    NormShape s;
    const int chunks = H / 8;
    s.nc = chunks > 512 ? 2 : 1;
    s.tpr = ((chunks + s.nc - 1) / s.nc + 31) / 32 * 32;
    s.rows = s.tpr >= NORM_THREADS ? 1 : NORM_THREADS / s.tpr;
    return s;
}

int backward_blocks(int T, int rows, int sm_count) {
    const int need = (T + rows - 1) / rows;
    const int most = 2 * sm_count;
    return need < most ? need : most;
}
// An upper bound that needs no device: the workspace query works without one.
constexpr int MAX_BACKWARD_BLOCKS = 2 * 160;

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

#define NORM_PICK(kernel, NC, B)                                                                                       \
    (hd ? (yd ? (xd ? kernel<1, 1, 1, NC, B> : kernel<1, 1, 0, NC, B>) : (xd ? kernel<1, 0, 1, NC, B> : kernel<1, 0, 0, NC, B>)) \
        : (yd ? (xd ? kernel<0, 1, 1, NC, B> : kernel<0, 1, 0, NC, B>) : (xd ? kernel<0, 0, 1, NC, B> : kernel<0, 0, 0, NC, B>)))

NormKernel pick_forward(const redmoe_norm* N, int nc, bool branch) {
    const bool hd = N->h_dtype == DT_BF16, xd = N->x_dtype == DT_BF16;
    const bool yd = branch && N->y_dtype == DT_BF16;  // without y its type does not matter
    if (branch) return nc == 1 ? NORM_PICK(norm_forward_kernel, 1, true) : NORM_PICK(norm_forward_kernel, 2, true);
    return nc == 1 ? NORM_PICK(norm_forward_kernel, 1, false) : NORM_PICK(norm_forward_kernel, 2, false);
}
NormKernel pick_backward(const redmoe_norm* N, int nc, bool branch) {
    const bool hd = N->h_dtype == DT_BF16, xd = N->x_dtype == DT_BF16;
    const bool yd = branch && N->y_dtype == DT_BF16;
    if (branch) return nc == 1 ? NORM_PICK(norm_backward_kernel, 1, true) : NORM_PICK(norm_backward_kernel, 2, true);
    return nc == 1 ? NORM_PICK(norm_backward_kernel, 1, false) : NORM_PICK(norm_backward_kernel, 2, false);
}
#undef NORM_PICK

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
    const size_t n = size_t(T) * N->hidden, wb = dt_bytes(N->w_dtype) * N->hidden;
    const Range rh{static_cast<const char*>(h), n * dt_bytes(N->h_dtype)};
    const Range ro{static_cast<const char*>(h_out), n * dt_bytes(N->h_dtype)};
    const Range rx{static_cast<const char*>(x), n * dt_bytes(N->x_dtype)};
    const Range in[] = {{static_cast<const char*>(y), n * dt_bytes(N->y_dtype)},
                        {static_cast<const char*>(gate), gate_elems(N, T) * dt_bytes(N->gate_dtype)},
                        {static_cast<const char*>(N->pre_w), wb},
                        {static_cast<const char*>(N->post_w), wb}};
    for (const Range& r : in)
        if (overlap(r, ro) || overlap(r, rx)) return REDMOE_ERR_INVALID_ARG;
    if (overlap(rh, rx) || overlap(ro, rx) || (h_out != h && overlap(rh, ro))) return REDMOE_ERR_INVALID_ARG;
    return REDMOE_OK;
}

}  // namespace redmoe

using namespace redmoe;

extern "C" {

redmoe_status redmoe_norm_forward(const redmoe_norm* N, const void* h, const void* y, const void* gate, int32_t T,
                                  void* h_out, void* x, void* stream) {
    const redmoe_status st = norm_forward_check(N, h, y, gate, T, h_out, x);
    if (st != REDMOE_OK || T == 0) return st;
    const bool branch = y != nullptr;
    const NormShape s = norm_shape(N->hidden);
    NormParams p = base_params(N, T, gate, s);
    p.h = h;
    p.y = y;
    p.h_out = h_out;
    p.x = x;
    const NormKernel kern = pick_forward(N, s.nc, branch);
    const unsigned grid = unsigned((T + (long long)s.rows - 1) / s.rows);
    kern<<<grid, s.tpr * s.rows, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? REDMOE_OK : REDMOE_ERR_CUDA;
}

size_t redmoe_norm_workspace_bytes(const redmoe_norm* N, int32_t T) {
    if (T < 0 || check_norm(N) != REDMOE_OK) return 0;
    const NormShape s = norm_shape(N->hidden);
    const long long need = ((long long)T + s.rows - 1) / s.rows;
    const long long blocks = need < MAX_BACKWARD_BLOCKS ? need : MAX_BACKWARD_BLOCKS;
    return 256 + align256(size_t(blocks) * 3 * N->hidden * 4);
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
    const NormShape s = norm_shape(N->hidden);
    NormParams p = base_params(N, T, gate, s);
    p.h = h_out;
    p.y = y;
    p.dh_out = dh_out;
    p.dx = dx;
    p.dh = dh;
    p.dy = dy;
    p.dgate = dgate;
    p.part = work ? reinterpret_cast<float*>(static_cast<char*>(workspace) + 256) : nullptr;
    p.want_pre = dpre_w != nullptr;
    p.want_post = dpost_w != nullptr;
    p.want_gate = dgate != nullptr && channel;
    const int sms = di.sm_count < MAX_BACKWARD_BLOCKS / 2 ? di.sm_count : MAX_BACKWARD_BLOCKS / 2;
    const int blocks = backward_blocks(T, s.rows, sms);
    // at most 21,504 bytes (H = 256: eight groups): below what a launch gets without asking
    const size_t smem = work ? size_t(s.rows - 1) * 3 * p.H * 4 : 0;
    const NormKernel kern = pick_backward(N, s.nc, branch);
    kern<<<blocks, s.tpr * s.rows, smem, stm>>>(p);
    if (cudaGetLastError() != cudaSuccess) return REDMOE_ERR_CUDA;
    if (!work) return REDMOE_OK;
    norm_columns_kernel<<<dim3((p.H + 31) / 32, 3), 256, 0, stm>>>(p.part, blocks, p.H, dpre_w, dpost_w,
                                                                   p.want_gate ? static_cast<float*>(dgate) : nullptr);
    return cudaGetLastError() == cudaSuccess ? REDMOE_OK : REDMOE_ERR_CUDA;
}

}  // extern "C"
