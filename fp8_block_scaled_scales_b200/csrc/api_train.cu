// C ABI of the expert-layer calls and the gradient products: argument validation and
// dispatch.  See include/dg.h for the contract.
#include <cuda_runtime.h>
#include <stdint.h>

#include "train_internal.h"

using namespace dg;

namespace {

constexpr int64_t kInt32Max = 0x7FFFFFFFLL;
constexpr int64_t kMaxSlots = 1LL << 30;
constexpr int64_t kMaxWidth = 1LL << 24;  // SwiGLU: a block's rows are addressed with 32 bits

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool bad_slots(int64_t T, int k) { return T < 0 || k < 1 || T > kMaxSlots / k; }

bool bad_columns(int64_t H) { return H < 0 || H % 16 != 0 || H > kInt32Max; }

// the most rows the contiguous layout can need: every expert that has a slot pads by at most 127
int64_t most_rows(int64_t slots, int G) { return (slots + 127 * (slots < G ? slots : G)) / 128 * 128; }

}  // namespace

extern "C" {

int64_t dg_moe_sort_workspace(int64_t T, int k, int G) {
    return bad_slots(T, k) || G < 1 || G > 1024 ? 0 : moe_sort_workspace(T * k, G);
}

dg_status_t dg_moe_sort(const void *topk_ids, int ids_64bit, int64_t T, int k, int G, int32_t *group_offsets,
                        int32_t *row_of_slot, int32_t *slot_of_row, int64_t M_total_capacity, void *workspace,
                        int64_t workspace_bytes, cudaStream_t stream) {
    if (bad_slots(T, k) || G < 1 || G > 1024 || M_total_capacity < 0 || M_total_capacity % 128 != 0 ||
        M_total_capacity > kInt32Max || M_total_capacity < most_rows(T * k, G))
        return DG_ERR_SHAPE;
    const int64_t need = moe_sort_workspace(T * k, G);
    if (!group_offsets || (T > 0 && (!topk_ids || !row_of_slot)) || (M_total_capacity > 0 && !slot_of_row) ||
        (need > 0 && !workspace) || workspace_bytes < need)
        return DG_ERR_INVALID_ARG;
    if (!aligned(topk_ids, ids_64bit ? 8 : 4) || !aligned(group_offsets, 4) || !aligned(row_of_slot, 4) ||
        !aligned(slot_of_row, 4) || !aligned(workspace, 16))
        return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    const dg_status_t st = current_device(&dev, nullptr);
    if (st != DG_OK) return st;
    return launch_moe_sort(topk_ids, ids_64bit != 0, T * k, G, false, M_total_capacity, group_offsets, row_of_slot,
                           slot_of_row, static_cast<int32_t *>(workspace), stream);
}

dg_status_t dg_moe_sort_masked(const void *topk_ids, int ids_64bit, int64_t T, int k, int G, int32_t *masked_m,
                               int32_t *row_of_slot, int32_t *slot_of_row, int64_t M_max, void *workspace,
                               int64_t workspace_bytes, cudaStream_t stream) {
    if (bad_slots(T, k) || G < 1 || G > 1024 || M_max < 0 || M_max > kInt32Max / G) return DG_ERR_SHAPE;
    const int64_t need = moe_sort_workspace(T * k, G);
    if (!masked_m || (T > 0 && (!topk_ids || !row_of_slot)) || (M_max > 0 && !slot_of_row) ||
        (need > 0 && !workspace) || workspace_bytes < need)
        return DG_ERR_INVALID_ARG;
    if (!aligned(topk_ids, ids_64bit ? 8 : 4) || !aligned(masked_m, 4) || !aligned(row_of_slot, 4) ||
        !aligned(slot_of_row, 4) || !aligned(workspace, 16))
        return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    const dg_status_t st = current_device(&dev, nullptr);
    if (st != DG_OK) return st;
    return launch_moe_sort(topk_ids, ids_64bit != 0, T * k, G, true, M_max, masked_m, row_of_slot, slot_of_row,
                           static_cast<int32_t *>(workspace), stream);
}

int64_t dg_moe_dispatch_workspace(int64_t T, int k, int64_t H, int64_t M_total_capacity) {
    return bad_slots(T, k) || bad_columns(H) || M_total_capacity < 0 || M_total_capacity > kInt32Max
               ? 0
               : dispatch_workspace(T, k, H, M_total_capacity);
}

dg_status_t dg_moe_dispatch_quantize(const void *X_bf16, const float *weights, const int32_t *slot_of_row,
                                     const int32_t *group_offsets, int64_t T, int k, int64_t H,
                                     int64_t M_total_capacity, int G, uint8_t *Q, float *S, void *workspace,
                                     int64_t workspace_bytes, cudaStream_t stream) {
    if (bad_slots(T, k) || bad_columns(H) || M_total_capacity < 0 || M_total_capacity % 128 != 0 ||
        M_total_capacity > kInt32Max || G < 1 || G > 1024)
        return DG_ERR_SHAPE;
    if (M_total_capacity == 0 || H == 0) return DG_OK;
    const int64_t need = dispatch_workspace(T, k, H, M_total_capacity);
    if ((T > 0 && !X_bf16) || !slot_of_row || !group_offsets || !Q || !S || (need > 0 && !workspace) ||
        workspace_bytes < need)
        return DG_ERR_INVALID_ARG;
    if (!aligned(X_bf16, 16) || !aligned(Q, 16) || !aligned(S, 4) || !aligned(weights, 4) ||
        !aligned(slot_of_row, 4) || !aligned(group_offsets, 4) || !aligned(workspace, 16))
        return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    const dg_status_t st = current_device(&dev, nullptr);
    if (st != DG_OK) return st;
    return launch_dispatch_quantize(X_bf16, weights, slot_of_row, group_offsets, T * k, k, H, M_total_capacity, G, Q, S,
                                    workspace, dev, stream);
}

dg_status_t dg_moe_dispatch_quantize_masked(const void *X_bf16, const int32_t *slot_of_row, const int32_t *masked_m,
                                            int64_t T, int k, int64_t H, int G, int64_t M_max, uint8_t *Q, float *S,
                                            cudaStream_t stream) {
    if (bad_slots(T, k) || bad_columns(H) || G < 1 || G > 1024 || M_max < 0 || M_max > kInt32Max / G)
        return DG_ERR_SHAPE;
    if (M_max == 0 || H == 0) return DG_OK;
    if ((T > 0 && !X_bf16) || !slot_of_row || !masked_m || !Q || !S) return DG_ERR_INVALID_ARG;
    if (!aligned(X_bf16, 16) || !aligned(Q, 16) || !aligned(S, 4) || !aligned(slot_of_row, 4) || !aligned(masked_m, 4))
        return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    const dg_status_t st = current_device(&dev, nullptr);
    if (st != DG_OK) return st;
    return launch_dispatch_quantize_masked(X_bf16, slot_of_row, masked_m, T * k, k, H, G, M_max, Q, S, dev, stream);
}

dg_status_t dg_moe_combine(const void *Y_bf16, const float *weights, const int32_t *row_of_slot, int64_t T, int k,
                           int64_t H, int64_t rows, void *OUT_bf16, cudaStream_t stream) {
    if (bad_slots(T, k) || bad_columns(H) || rows < 0 || rows > kInt32Max) return DG_ERR_SHAPE;
    if (T == 0 || H == 0) return DG_OK;
    if ((rows > 0 && !Y_bf16) || !row_of_slot || !OUT_bf16) return DG_ERR_INVALID_ARG;
    if (!aligned(Y_bf16, 16) || !aligned(OUT_bf16, 16) || !aligned(weights, 4) || !aligned(row_of_slot, 4))
        return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    const dg_status_t st = current_device(&dev, nullptr);
    if (st != DG_OK) return st;
    return launch_combine(Y_bf16, weights, row_of_slot, T, k, H, rows, OUT_bf16, stream);
}

dg_status_t dg_moe_combine_backward(const void *dOUT_bf16, const void *Y_bf16, const int32_t *row_of_slot, int64_t T,
                                    int k, int64_t H, int64_t rows, float *dweights, cudaStream_t stream) {
    if (bad_slots(T, k) || bad_columns(H) || rows < 0 || rows > kInt32Max) return DG_ERR_SHAPE;
    if (T == 0) return DG_OK;
    if ((H > 0 && !dOUT_bf16) || (rows > 0 && H > 0 && !Y_bf16) || !row_of_slot || !dweights)
        return DG_ERR_INVALID_ARG;
    if (!aligned(dOUT_bf16, 16) || !aligned(Y_bf16, 16) || !aligned(row_of_slot, 4) || !aligned(dweights, 4))
        return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    const dg_status_t st = current_device(&dev, nullptr);
    if (st != DG_OK) return st;
    return launch_combine_backward(dOUT_bf16, Y_bf16, row_of_slot, T, k, H, rows, dweights, stream);
}

dg_status_t dg_swiglu_quantize(const void *H_bf16, const int32_t *group_offsets, int G, int64_t M, int64_t F,
                               uint8_t *Q, float *S, uint8_t *H8, float *sH_t, cudaStream_t stream) {
    if (M < 0 || M > kInt32Max || F < 0 || F > kMaxWidth || F % 128 != 0) return DG_ERR_SHAPE;
    if (group_offsets && (G < 1 || G > 1024 || M % 128 != 0)) return DG_ERR_SHAPE;
    if (M == 0 || F == 0) return DG_OK;
    if (!H_bf16 || !Q || !S || (H8 == nullptr) != (sH_t == nullptr)) return DG_ERR_INVALID_ARG;
    if (!aligned(H_bf16, 16) || !aligned(Q, 16) || !aligned(S, 4) || !aligned(H8, 16) || !aligned(sH_t, 4) ||
        !aligned(group_offsets, 4))
        return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    const dg_status_t st = current_device(&dev, nullptr);
    if (st != DG_OK) return st;
    return launch_swiglu(H_bf16, group_offsets, nullptr, G, M, F, Q, S, H8, sH_t, dev, stream);
}

dg_status_t dg_swiglu_quantize_masked(const void *H_bf16, const int32_t *masked_m, int G, int64_t M_max, int64_t F,
                                      uint8_t *Q, float *S, cudaStream_t stream) {
    if (G < 1 || G > 1024 || M_max < 0 || M_max > kInt32Max / G || F < 0 || F > kMaxWidth || F % 128 != 0) return DG_ERR_SHAPE;
    if (M_max == 0 || F == 0) return DG_OK;
    if (!H_bf16 || !masked_m || !Q || !S) return DG_ERR_INVALID_ARG;
    if (!aligned(H_bf16, 16) || !aligned(Q, 16) || !aligned(S, 4) || !aligned(masked_m, 4)) return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    const dg_status_t st = current_device(&dev, nullptr);
    if (st != DG_OK) return st;
    return launch_swiglu(H_bf16, nullptr, masked_m, G, M_max, F, Q, S, nullptr, nullptr, dev, stream);
}

dg_status_t dg_swiglu_quantize_backward(const uint8_t *H8, const float *sH_t, const void *dA_bf16,
                                        const int32_t *group_offsets, int G, int64_t M, int64_t F, uint8_t *Q,
                                        float *S, cudaStream_t stream) {
    if (M < 0 || M > kInt32Max || F < 0 || F > kMaxWidth || F % 128 != 0) return DG_ERR_SHAPE;
    if (group_offsets && (G < 1 || G > 1024 || M % 128 != 0)) return DG_ERR_SHAPE;
    if (M == 0 || F == 0) return DG_OK;
    if (!H8 || !sH_t || !dA_bf16 || !Q || !S) return DG_ERR_INVALID_ARG;
    if (!aligned(H8, 16) || !aligned(dA_bf16, 16) || !aligned(Q, 16) || !aligned(S, 4) || !aligned(sH_t, 4) ||
        !aligned(group_offsets, 4))
        return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    const dg_status_t st = current_device(&dev, nullptr);
    if (st != DG_OK) return st;
    return launch_swiglu_backward(H8, sH_t, dA_bf16, group_offsets, G, M, F, Q, S, dev, stream);
}

static dg_status_t check_grad(const void *dY, const float *sdY, const void *B, const float *sB, const void *C) {
    if (!dY || !sdY || !B || !sB || !C) return DG_ERR_INVALID_ARG;
    if (!aligned(dY, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(sdY, 4) || !aligned(sB, 4))
        return DG_ERR_ALIGNMENT;
    return DG_OK;
}

static bool bad_grad_sizes(int64_t M, int64_t N, int64_t K) {
    return M < 0 || N < 0 || K < 0 || N % 16 != 0 || K % 16 != 0 || M > kInt32Max || N > kInt32Max || K > kInt32Max;
}

int64_t dg_fp8_dgrad_workspace(int64_t M, int64_t N, int64_t K) {
    return bad_grad_sizes(M, N, K) || M == 0 || N == 0 || K == 0 ? 0 : grad_workspace(false, M, N, K);
}

int64_t dg_fp8_wgrad_workspace(int64_t M, int64_t N, int64_t K) {
    return bad_grad_sizes(M, N, K) || M == 0 || N == 0 || K == 0 ? 0 : grad_workspace(true, M, N, K);
}

static dg_status_t check_workspace(int64_t need, const void *workspace, int64_t bytes) {
    if ((need > 0 && !workspace) || bytes < need) return DG_ERR_INVALID_ARG;
    return aligned(workspace, 16) ? DG_OK : DG_ERR_ALIGNMENT;
}

dg_status_t dg_fp8_dgrad_blockscaled(const uint8_t *dY, const float *sdY, const uint8_t *W, const float *sW,
                                     void *dX_bf16, int64_t M, int64_t N, int64_t K, void *workspace,
                                     int64_t workspace_bytes, cudaStream_t stream) {
    if (bad_grad_sizes(M, N, K) || N == 0) return DG_ERR_SHAPE;
    if (M == 0 || K == 0) return DG_OK;
    dg_status_t st = check_grad(dY, sdY, W, sW, dX_bf16);
    if (st == DG_OK) st = check_workspace(dg_fp8_dgrad_workspace(M, N, K), workspace, workspace_bytes);
    if (st != DG_OK) return st;
    DeviceInfo dev;
    st = current_device(&dev, nullptr);
    if (st != DG_OK) return st;
    const GradArgs a = {dY, sdY, W, sW, dX_bf16, nullptr, M, N, K, 1, false, false, workspace};
    return launch_dgrad(a, dev, stream);
}

dg_status_t dg_fp8_grouped_dgrad_contiguous(const uint8_t *dY, const float *sdY, const uint8_t *W, const float *sW,
                                            void *dX_bf16, const int32_t *group_offsets, int64_t M_total_capacity,
                                            int G, int64_t N, int64_t K, cudaStream_t stream) {
    if (M_total_capacity < 0 || M_total_capacity % 128 != 0 || N <= 0 || N % 128 != 0 || K < 0 || K % 16 != 0 ||
        G < 1 || G > 1024)
        return DG_ERR_SHAPE;
    if (M_total_capacity > kInt32Max || N > kInt32Max / G || K > kInt32Max) return DG_ERR_SHAPE;
    if (M_total_capacity == 0 || K == 0) return DG_OK;
    if (!group_offsets) return DG_ERR_INVALID_ARG;
    dg_status_t st = check_grad(dY, sdY, W, sW, dX_bf16);
    if (st != DG_OK) return st;
    if (!aligned(group_offsets, 4)) return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    st = current_device(&dev, nullptr);
    if (st != DG_OK) return st;
    const GradArgs a = {dY, sdY, W, sW, dX_bf16, group_offsets, M_total_capacity, N, K, G, false, false, nullptr};
    return launch_dgrad(a, dev, stream);
}

// No rows at all: the gradient is zero (accumulated: nothing changes).
static dg_status_t wgrad_of_nothing(void *dW, int64_t elements, int out_fp32, int accumulate, cudaStream_t stream) {
    if (accumulate) return DG_OK;
    return cudaMemsetAsync(dW, 0, static_cast<size_t>(elements) * (out_fp32 ? 4 : 2), stream) == cudaSuccess
               ? DG_OK
               : DG_ERR_CUDA;
}

dg_status_t dg_fp8_wgrad_blockscaled(const uint8_t *dY, const float *sdY, const uint8_t *X, const float *sX, void *dW,
                                     int out_fp32, int accumulate, int64_t M, int64_t N, int64_t K, void *workspace,
                                     int64_t workspace_bytes, cudaStream_t stream) {
    if (bad_grad_sizes(M, N, K)) return DG_ERR_SHAPE;
    if (accumulate && !out_fp32) return DG_ERR_INVALID_ARG;
    if (N == 0 || K == 0) return DG_OK;
    dg_status_t st = M == 0 ? (dW ? (aligned(dW, 16) ? DG_OK : DG_ERR_ALIGNMENT) : DG_ERR_INVALID_ARG)
                            : check_grad(dY, sdY, X, sX, dW);
    if (st == DG_OK) st = check_workspace(dg_fp8_wgrad_workspace(M, N, K), workspace, workspace_bytes);
    if (st != DG_OK) return st;
    DeviceInfo dev;
    st = current_device(&dev, nullptr);
    if (st != DG_OK) return st;
    if (M == 0) return wgrad_of_nothing(dW, N * K, out_fp32, accumulate, stream);
    const GradArgs a = {dY, sdY, X, sX, dW, nullptr, M, N, K, 1, out_fp32 != 0, accumulate != 0, workspace};
    return launch_wgrad(a, dev, stream);
}

dg_status_t dg_fp8_grouped_wgrad_contiguous(const uint8_t *dY, const float *sdY, const uint8_t *X, const float *sX,
                                            void *dW, int out_fp32, int accumulate, const int32_t *group_offsets,
                                            int64_t M_total_capacity, int G, int64_t N, int64_t K,
                                            cudaStream_t stream) {
    if (M_total_capacity < 0 || M_total_capacity % 128 != 0 || N < 0 || N % 128 != 0 || K < 0 || K % 16 != 0 ||
        G < 1 || G > 1024)
        return DG_ERR_SHAPE;
    if (M_total_capacity > kInt32Max || N > kInt32Max / G || K > kInt32Max) return DG_ERR_SHAPE;
    if (accumulate && !out_fp32) return DG_ERR_INVALID_ARG;
    if (N == 0 || K == 0) return DG_OK;
    if (M_total_capacity > 0 && !group_offsets) return DG_ERR_INVALID_ARG;
    dg_status_t st = M_total_capacity == 0 ? (dW ? (aligned(dW, 16) ? DG_OK : DG_ERR_ALIGNMENT) : DG_ERR_INVALID_ARG)
                                           : check_grad(dY, sdY, X, sX, dW);
    if (st != DG_OK) return st;
    if (!aligned(group_offsets, 4)) return DG_ERR_ALIGNMENT;
    DeviceInfo dev;
    st = current_device(&dev, nullptr);
    if (st != DG_OK) return st;
    if (M_total_capacity == 0) return wgrad_of_nothing(dW, G * N * K, out_fp32, accumulate, stream);
    const GradArgs a = {dY, sdY, X, sX, dW, group_offsets, M_total_capacity, N, K, G, out_fp32 != 0, accumulate != 0, nullptr};
    return launch_wgrad(a, dev, stream);
}

}  // extern "C"
