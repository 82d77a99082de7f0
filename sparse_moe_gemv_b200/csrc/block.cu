// redmoe_forward_block: the residual block around the layer, on one stream: the norm before
// it, redmoe_forward, and the residual step behind it (norm.cu) with the next block's norm.
#include "common.cuh"
#include "internal.h"
#include "norm.h"

namespace redmoe {
namespace {

// The layer's own workspace, then its input [T, H] and its output [T, H] fp32.
struct BlockWs {
    size_t x, out, total;
};
bool block_layout(const redmoe_layer* L, int T, BlockWs* b) {
    size_t o = redmoe_workspace_bytes(L, T);
    if (o == 0) return false;
    b->x = o; o = align256(o + (L->x_dtype == DT_F32 ? 4ull : 2ull) * T * L->hidden);
    b->out = o; o = align256(o + 4ull * T * L->hidden);
    b->total = o;
    return true;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
    return a && b && x < y + bn && y < x + an;
}

}  // namespace
}  // namespace redmoe

using namespace redmoe;

extern "C" {

size_t redmoe_workspace_bytes_block(const redmoe_layer* L, int32_t T) {
    BlockWs b;
    return block_layout(L, T, &b) ? b.total : 0;
}

redmoe_status redmoe_forward_block(const redmoe_layer* L, const redmoe_norm* before, const redmoe_norm* after,
                                   const void* h, const void* gate, int32_t T, void* h_out, void* x_next,
                                   int32_t* topk_ids, float* topk_w, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    redmoe_status st = check_layer(L);
    if (st != REDMOE_OK) return st;
    if (!before || !after || T < 0) return REDMOE_ERR_INVALID_ARG;
    if (before->hidden != L->hidden || after->hidden != L->hidden || before->x_dtype != L->x_dtype ||
        after->h_dtype != before->h_dtype || after->y_dtype != DT_F32)
        return REDMOE_ERR_INVALID_ARG;
    if (T == 0) return REDMOE_OK;
    if (!h || !h_out || !topk_ids || !topk_w || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
        return REDMOE_ERR_INVALID_ARG;
    if (T > DECODE_MAX_T ? !batch_shape_ok(L) : (L->expert_dtype == DT_INT2 && (T != 1 || !decode1_shape_ok(L))))
        return REDMOE_ERR_UNSUPPORTED;
    if ((long long)T * L->top_k + T > (1ll << 30)) return REDMOE_ERR_INVALID_ARG;
    BlockWs b;
    if (!block_layout(L, T, &b)) return REDMOE_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < b.total) return REDMOE_ERR_WORKSPACE;
    char* base = static_cast<char*>(workspace);
    // every check is made before the first launch
    const size_t n = size_t(T) * L->hidden, hb = n * (before->h_dtype == DT_F32 ? 4 : 2),
                 xb = n * (after->x_dtype == DT_F32 ? 4 : 2), kb = 4ull * T * L->top_k;
    const struct { const void* p; size_t n; } out[] = {
        {h_out, hb}, {x_next, xb}, {topk_ids, kb}, {topk_w, kb}, {workspace, b.total}};
    for (int i = 0; i < 5; ++i) {
        if (overlap(out[i].p, out[i].n, h, hb) && !(i == 0 && h_out == h)) return REDMOE_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return REDMOE_ERR_INVALID_ARG;
    }
    if ((st = norm_forward_check(before, h, nullptr, nullptr, T, nullptr, base + b.x)) != REDMOE_OK) return st;
    if ((st = norm_forward_check(after, h, base + b.out, gate, T, h_out, x_next)) != REDMOE_OK) return st;
    // the second norm reads behind the layer, whose ids, weights and workspace must leave its inputs alone
    const struct { const void* p; size_t n; } in[] = {{gate, norm_gate_bytes(after, T)},
                                                      {before->pre_w, norm_weight_bytes(before)},
                                                      {after->pre_w, norm_weight_bytes(after)},
                                                      {after->post_w, norm_weight_bytes(after)}};
    for (const auto& o : out)
        for (const auto& r : in)
            if (overlap(o.p, o.n, r.p, r.n)) return REDMOE_ERR_INVALID_ARG;
    if ((st = redmoe_norm_forward(before, h, nullptr, nullptr, T, nullptr, base + b.x, stream)) != REDMOE_OK) return st;
    st = redmoe_forward(L, base + b.x, T, reinterpret_cast<float*>(base + b.out), topk_ids, topk_w, workspace,
                        workspace_bytes, nullptr, stream);
    if (st != REDMOE_OK) return st;
    return redmoe_norm_forward(after, h, base + b.out, gate, T, h_out, x_next, stream);
}

}  // extern "C"
