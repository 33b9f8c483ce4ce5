// C ABI of the calls around the expert layer (routing, norms, gradient norm): argument
// validation and dispatch.  See include/dg.h for the contract.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "train_internal.h"

using namespace dg;

namespace {

constexpr int64_t kMaxSlots = 1LL << 30;
constexpr int64_t kMaxWidth = 16384;             // of a normed row: four CTAs of 4096 columns
constexpr int64_t kMaxElements = 1LL << 42;      // of a gradient: its chunks are counted with 32 bits
constexpr int64_t kMaxTensors = 1LL << 24;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool bad_route_sizes(int64_t T, int G, int k) {
    return G < 1 || G > 1024 || k < 1 || k > 32 || k > G || T < 0 || T > kMaxSlots / k;
}

bool bad_options(const dg_route_options_t *o) {
    return !o || (o->score != DG_SCORE_SOFTMAX && o->score != DG_SCORE_SIGMOID) || !std::isfinite(o->scale);
}

bool bad_norm_sizes(int64_t T, int64_t H) { return T < 0 || T > 0x7FFFFFFFLL || H < 0 || H % 16 != 0 || H > kMaxWidth; }

dg_status_t b200(DeviceInfo *dev) { return current_device(dev, nullptr); }

dg_status_t check_norm(const void *X, const void *Y, const void *weight, const void *post, const void *gate,
                       const dg_norm_options_t *o, const void *R, const float *rstd, const float *rstd_y) {
    if (!o || !std::isfinite(o->alpha) || !(o->eps >= 0.0f) || !std::isfinite(o->eps) || !X || !weight) return DG_ERR_INVALID_ARG;
    if (Y ? !R : (R || post || gate || o->alpha != 1.0f)) return DG_ERR_INVALID_ARG;
    if (rstd_y && !post) return DG_ERR_INVALID_ARG;
    if (!aligned(X, 16) || !aligned(Y, 16) || !aligned(weight, 16) || !aligned(post, 16) || !aligned(gate, 16) ||
        !aligned(R, 16) || !aligned(rstd, 4) || !aligned(rstd_y, 4))
        return DG_ERR_ALIGNMENT;
    return DG_OK;
}

dg_status_t check_grads(const GradList &g) {
    if (g.count < 0 || g.count > kMaxTensors) return DG_ERR_SHAPE;
    if (g.count > 0 && (!g.in || !g.sizes || !g.bf16)) return DG_ERR_INVALID_ARG;
    for (int64_t i = 0; i < g.count; ++i) {
        if (g.sizes[i] < 0 || g.sizes[i] > kMaxElements) return DG_ERR_SHAPE;
        if (g.sizes[i] == 0) continue;
        if (!g.in[i] || (g.out && !g.out[i])) return DG_ERR_INVALID_ARG;
        const uintptr_t a = g.bf16[i] ? 2 : 4;
        if (!aligned(g.in[i], a) || (g.out && !aligned(g.out[i], a))) return DG_ERR_ALIGNMENT;
    }
    return DG_OK;
}

// A tensor that is written overlaps no other one, nor the norm: the kernel's CTAs run in no order.  What is
// written is put in order and drawn together into spans with gaps of less than 4 KB; a tensor
// that is only read seldom meets one, and only then is looked up among the written ones.
dg_status_t check_overlap(const GradList &g, const float *norm, bool norm_written) try {
    struct Range {
        uintptr_t begin, end;
    };
    std::vector<Range> written, spans;
    written.reserve(static_cast<size_t>(g.count));
    auto bytes = [&](int64_t i) { return static_cast<uintptr_t>(g.sizes[i]) * (g.bf16[i] ? 2 : 4); };
    auto target = [&](int64_t i) { return reinterpret_cast<uintptr_t>(g.out ? g.out[i] : g.in[i]); };
    const uintptr_t norm_at = reinterpret_cast<uintptr_t>(norm);
    const auto holds_norm = [&](uintptr_t begin, uintptr_t n) { return norm_at < begin + n && begin < norm_at + 4; };
    for (int64_t i = 0; i < g.count; ++i) {
        if (g.sizes[i] == 0) continue;
        written.push_back({target(i), target(i) + bytes(i)});
        if (holds_norm(target(i), bytes(i))) return DG_ERR_INVALID_ARG;
        if (norm_written && holds_norm(reinterpret_cast<uintptr_t>(g.in[i]), bytes(i))) return DG_ERR_INVALID_ARG;
    }
    const auto before = [](const Range &a, const Range &b) { return a.begin < b.begin; };
    if (!std::is_sorted(written.begin(), written.end(), before)) std::sort(written.begin(), written.end(), before);
    for (size_t i = 1; i < written.size(); ++i)
        if (written[i].begin < written[i - 1].end) return DG_ERR_INVALID_ARG;
    if (!g.out) return DG_OK;
    for (const Range &r : written) {
        if (spans.empty() || r.begin - spans.back().end >= 4096)
            spans.push_back(r);
        else
            spans.back().end = r.end;
    }
    for (int64_t i = 0; i < g.count; ++i) {
        const uintptr_t begin = reinterpret_cast<uintptr_t>(g.in[i]), end = begin + bytes(i);
        if (g.sizes[i] == 0 || begin == target(i)) continue;
        // the first range that ends past `begin`
        const auto past = [](uintptr_t at, const Range &r) { return at < r.end; };
        const auto span = std::upper_bound(spans.begin(), spans.end(), begin, past);
        if (span == spans.end() || span->begin >= end) continue;
        const auto one = std::upper_bound(written.begin(), written.end(), begin, past);
        if (one != written.end() && one->begin < end) return DG_ERR_INVALID_ARG;
    }
    return DG_OK;
} catch (...) {  // no host memory for the list: no exception may pass the C interface
    return DG_ERR_INVALID_ARG;
}

dg_status_t check_norm_workspace(int64_t count, const float *norm, const void *workspace, int64_t bytes) {
    if (!norm || !workspace || bytes < grad_norm_workspace(count)) return DG_ERR_INVALID_ARG;
    return aligned(norm, 4) && aligned(workspace, 16) ? DG_OK : DG_ERR_ALIGNMENT;
}

bool bad_limit(const float *max_norm) { return !max_norm || !(*max_norm >= 0.0f) || !std::isfinite(*max_norm); }

}  // namespace

extern "C" {

int64_t dg_moe_route_workspace(int64_t T, int G) { return bad_route_sizes(T, G, 1) ? 0 : route_workspace(T, G); }

dg_status_t dg_moe_route(const void *logits, int logits_bf16, const dg_route_options_t *options, const float *bias,
                         const uint8_t *mask, int64_t T, int G, int k, int32_t *topk_ids, float *weights, int32_t *counts,
                         float *loss, float *dprob, void *workspace, int64_t workspace_bytes,
                         cudaStream_t stream) {
    if (bad_route_sizes(T, G, k)) return DG_ERR_SHAPE;
    if (bad_options(options)) return DG_ERR_INVALID_ARG;
    const bool balance = counts != nullptr;
    if ((loss != nullptr) != balance || (dprob != nullptr) != balance) return DG_ERR_INVALID_ARG;
    if (T == 0 && !balance) return DG_OK;
    if (T > 0 && (!logits || !topk_ids || !weights)) return DG_ERR_INVALID_ARG;
    const int64_t need = balance ? route_workspace(T, G) : 0;
    if ((need > 0 && !workspace) || workspace_bytes < need) return DG_ERR_INVALID_ARG;
    if (!aligned(logits, logits_bf16 ? 2 : 4) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(weights, 4) ||
        !aligned(counts, 4) || !aligned(loss, 4) || !aligned(dprob, 4) || !aligned(workspace, 16))
        return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    const dg_status_t st = b200(&dev);
    if (st != DG_OK) return st;
    const RouteArgs a = {logits, logits_bf16 != 0, options->score == DG_SCORE_SIGMOID, options->renormalize != 0, options->scale, bias, mask,
                         T, G, k, topk_ids, weights, counts, loss, dprob, workspace};
    return launch_route(a, dev, stream);
}

dg_status_t dg_moe_route_backward(const void *logits, int logits_bf16, const dg_route_options_t *options,
                                  const int32_t *topk_ids, const float *dweights, const float *dprob, const float *dloss,
                                  int64_t T, int G, int k, void *dlogits, cudaStream_t stream) {
    if (bad_route_sizes(T, G, k)) return DG_ERR_SHAPE;
    if (bad_options(options) || (dprob != nullptr) != (dloss != nullptr)) return DG_ERR_INVALID_ARG;
    if (T == 0) return DG_OK;
    if (!logits || !topk_ids || !dlogits) return DG_ERR_INVALID_ARG;
    const uintptr_t element = logits_bf16 ? 2 : 4;
    if (!aligned(logits, element) || !aligned(dlogits, element) || !aligned(topk_ids, 4) || !aligned(dweights, 4) ||
        !aligned(dprob, 4) || !aligned(dloss, 4))
        return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    const dg_status_t st = b200(&dev);
    if (st != DG_OK) return st;
    const RouteBackwardArgs a = {logits, logits_bf16 != 0, options->score == DG_SCORE_SIGMOID, options->renormalize != 0, options->scale, topk_ids,
                                 dweights, dprob, dloss, T, G, k, dlogits};
    return launch_route_backward(a, dev, stream);
}

dg_status_t dg_rmsnorm_residual(const void *X_bf16, const void *Y_bf16, const void *weight, const void *post,
                                const void *gate, const dg_norm_options_t *options, int64_t T, int64_t H,
                                void *N_bf16, void *R_bf16, float *rstd, float *rstd_y, cudaStream_t stream) {
    if (bad_norm_sizes(T, H)) return DG_ERR_SHAPE;
    if (T == 0 || H == 0) return DG_OK;
    dg_status_t st = check_norm(X_bf16, Y_bf16, weight, post, gate, options, R_bf16, rstd, rstd_y);
    if (st != DG_OK) return st;
    if (!N_bf16) return DG_ERR_INVALID_ARG;
    if (!aligned(N_bf16, 16)) return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    st = b200(&dev);
    if (st != DG_OK) return st;
    const NormArgs a = {X_bf16, Y_bf16, weight, post, gate, options->vectors_bf16 != 0, options->alpha, options->eps, T, H,
                        N_bf16, R_bf16, nullptr, nullptr, rstd, rstd_y};
    return launch_rmsnorm(a, dev, stream);
}

dg_status_t dg_rmsnorm_residual_quantize(const void *X_bf16, const void *Y_bf16, const void *weight, const void *post,
                                         const void *gate, const dg_norm_options_t *options, int64_t T, int64_t H,
                                         uint8_t *Q, float *S_t, void *R_bf16, cudaStream_t stream) {
    if (bad_norm_sizes(T, H)) return DG_ERR_SHAPE;
    if (T == 0 || H == 0) return DG_OK;
    dg_status_t st = check_norm(X_bf16, Y_bf16, weight, post, gate, options, R_bf16, nullptr, nullptr);
    if (st != DG_OK) return st;
    if (!Q || !S_t) return DG_ERR_INVALID_ARG;
    if (!aligned(Q, 16) || !aligned(S_t, 4)) return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    st = b200(&dev);
    if (st != DG_OK) return st;
    const NormArgs a = {X_bf16, Y_bf16, weight, post, gate, options->vectors_bf16 != 0, options->alpha, options->eps, T, H,
                        nullptr, R_bf16, Q, S_t, nullptr, nullptr};
    return launch_rmsnorm(a, dev, stream);
}

int64_t dg_rmsnorm_residual_backward_workspace(int64_t T, int64_t H, int has_post, int has_gate) {
    return bad_norm_sizes(T, H) || H == 0 ? 0 : rmsnorm_backward_workspace(T, H, has_post != 0, has_gate != 0);
}

dg_status_t dg_rmsnorm_residual_backward(const void *dN_bf16, const void *dR_bf16, const void *R_bf16, const float *rstd,
                                         const void *Y_bf16, const float *rstd_y, const void *weight, const void *post,
                                         const void *gate, const dg_norm_options_t *options, int64_t T, int64_t H,
                                         void *dX_bf16, void *dY_bf16, float *dweight, float *dpost, float *dgate,
                                         void *workspace, int64_t workspace_bytes, cudaStream_t stream) {
    if (bad_norm_sizes(T, H)) return DG_ERR_SHAPE;
    if (H == 0) return DG_OK;
    if (!options || !std::isfinite(options->alpha) || !weight || !dweight) return DG_ERR_INVALID_ARG;
    if (T > 0 && (!dN_bf16 || !R_bf16 || !rstd || !dX_bf16)) return DG_ERR_INVALID_ARG;
    if ((post != nullptr) != (dpost != nullptr) || (gate != nullptr) != (dgate != nullptr)) return DG_ERR_INVALID_ARG;
    if (T > 0 && ((Y_bf16 != nullptr) != (dY_bf16 != nullptr) || (post != nullptr) != (rstd_y != nullptr) ||
                  (!Y_bf16 && (post || gate))))
        return DG_ERR_INVALID_ARG;
    const int64_t need = rmsnorm_backward_workspace(T, H, post != nullptr, gate != nullptr);
    if ((need > 0 && !workspace) || workspace_bytes < need) return DG_ERR_INVALID_ARG;
    if (!aligned(dN_bf16, 16) || !aligned(dR_bf16, 16) || !aligned(R_bf16, 16) || !aligned(Y_bf16, 16) ||
        !aligned(dX_bf16, 16) || !aligned(dY_bf16, 16) || !aligned(weight, 16) || !aligned(post, 16) ||
        !aligned(gate, 16) || !aligned(workspace, 16) || !aligned(rstd, 4) || !aligned(rstd_y, 4) ||
        !aligned(dweight, 4) || !aligned(dpost, 4) || !aligned(dgate, 4))
        return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    const dg_status_t st = b200(&dev);
    if (st != DG_OK) return st;
    const NormBackwardArgs a = {dN_bf16, dR_bf16, R_bf16, Y_bf16, weight, post, gate, rstd, rstd_y, options->vectors_bf16 != 0,
                                options->alpha, T, H, dX_bf16, dY_bf16, dweight, dpost, dgate, workspace};
    return launch_rmsnorm_backward(a, dev, stream);
}

int64_t dg_grad_norm_workspace(int64_t count) { return count < 0 || count > kMaxTensors ? 0 : grad_norm_workspace(count); }

dg_status_t dg_grad_norm(const void *const *grads, const int64_t *sizes, const uint8_t *bf16, int64_t count, float *norm,
                         void *workspace, int64_t workspace_bytes, cudaStream_t stream) {
    const GradList g = {grads, nullptr, sizes, bf16, count};
    dg_status_t st = check_grads(g);
    if (st == DG_OK) st = check_norm_workspace(count, norm, workspace, workspace_bytes);
    if (st != DG_OK) return st;
    DeviceInfo dev;
    st = b200(&dev);
    if (st != DG_OK) return st;
    return launch_grad_norm(g, norm, workspace, stream);
}

dg_status_t dg_grad_clip(const void *const *grads, const int64_t *sizes, const uint8_t *bf16, int64_t count,
                         const float *norm, const float *max_norm, void *const *out, cudaStream_t stream) {
    const GradList g = {grads, out, sizes, bf16, count};
    dg_status_t st = check_grads(g);
    if (st != DG_OK) return st;
    if (!norm || bad_limit(max_norm)) return DG_ERR_INVALID_ARG;
    if (!aligned(norm, 4)) return DG_ERR_ALIGNMENT;
    st = check_overlap(g, norm, false);
    if (st != DG_OK) return st;
    DeviceInfo dev;
    st = b200(&dev);
    if (st != DG_OK) return st;
    return launch_grad_clip(g, norm, *max_norm, stream);
}

dg_status_t dg_grad_norm_clip(const void *const *grads, const int64_t *sizes, const uint8_t *bf16, int64_t count,
                              const float *max_norm, void *const *out, float *norm, void *workspace, int64_t workspace_bytes,
                              cudaStream_t stream) {
    const GradList g = {grads, out, sizes, bf16, count};
    dg_status_t st = check_grads(g);
    if (st != DG_OK) return st;
    if (bad_limit(max_norm)) return DG_ERR_INVALID_ARG;
    st = check_norm_workspace(count, norm, workspace, workspace_bytes);
    if (st == DG_OK) st = check_overlap(g, norm, true);
    if (st != DG_OK) return st;
    DeviceInfo dev;
    st = b200(&dev);
    if (st != DG_OK) return st;
    return launch_grad_norm_clip(g, *max_norm, norm, workspace, stream);
}

}  // extern "C"
