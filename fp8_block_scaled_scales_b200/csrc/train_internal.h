// Host-side launchers of the expert-layer calls (sort, dispatch, combine, SwiGLU) and of
// the gradient products; validated arguments only.
#pragma once

#include "dg_internal.h"

namespace dg {

// Dynamic shared memory above the default needs the kernel's consent, once per device and
// thread.  configured_device: the caller's thread_local, -1 at first.
template <typename Kernel>
dg_status_t allow_smem(Kernel kernel, size_t bytes, int &configured_device) {
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return DG_ERR_CUDA;
    if (configured_device == device) return DG_OK;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) !=
        cudaSuccess)
        return DG_ERR_CUDA;
    configured_device = device;
    return DG_OK;
}

// moe_sort.cu.  masked: `offsets` receives the counts [G] and `rows` is M_max, else the
// group offsets [G+1] and the row capacity.  workspace: moe_sort_workspace bytes.
int64_t moe_sort_workspace(int64_t slots, int G);
dg_status_t launch_moe_sort(const void *ids, bool ids64, int64_t slots, int G, bool masked, int64_t rows,
                            int32_t *offsets, int32_t *row_of_slot, int32_t *slot_of_row, int32_t *workspace,
                            cudaStream_t stream);

// moe_rows.cu.  workspace: dispatch_workspace bytes.
int64_t dispatch_workspace(int64_t T, int k, int64_t H, int64_t rows);
dg_status_t launch_dispatch_quantize(const void *X, const float *weights, const int32_t *slot_of_row,
                                     const int32_t *offsets, int64_t slots, int k, int64_t H, int64_t rows, int G,
                                     uint8_t *Q, float *S, void *workspace, const DeviceInfo &dev,
                                     cudaStream_t stream);
dg_status_t launch_dispatch_quantize_masked(const void *X, const int32_t *slot_of_row, const int32_t *masked_m,
                                            int64_t slots, int k, int64_t H, int G, int64_t m_max, uint8_t *Q,
                                            float *S, const DeviceInfo &dev, cudaStream_t stream);
dg_status_t launch_combine(const void *Y, const float *weights, const int32_t *row_of_slot, int64_t T, int k,
                           int64_t H, int64_t rows, void *out, cudaStream_t stream);
dg_status_t launch_combine_backward(const void *dout, const void *Y, const int32_t *row_of_slot, int64_t T, int k,
                                    int64_t H, int64_t rows, float *dweights, cudaStream_t stream);

// swiglu.cu.  offsets may be null (all M rows); masked_m selects the masked layout (G slabs of M rows).
dg_status_t launch_swiglu(const void *H, const int32_t *offsets, const int32_t *masked_m, int G, int64_t M,
                          int64_t F, uint8_t *Q, float *S, uint8_t *H8, float *sH, const DeviceInfo &dev,
                          cudaStream_t stream);
dg_status_t launch_swiglu_backward(const uint8_t *H8, const float *sH, const void *dA, const int32_t *offsets,
                                   int G, int64_t M, int64_t F, uint8_t *Q, float *S, const DeviceInfo &dev,
                                   cudaStream_t stream);

// gemm_grad.cu
struct GradArgs {
    const uint8_t *dY;  // [M][N]
    const float *sdY;
    const uint8_t *B;   // dgrad: W [G][N][K]; wgrad: X [M][K]
    const float *sB;
    void *C;            // dgrad: BF16 [M][K]; wgrad: FP32 or BF16 [G][N][K]
    const int32_t *offsets;  // null: dense
    int64_t M, N, K;
    int G;
    bool fp32, accumulate;  // wgrad
    void *workspace;        // dense: grad_workspace bytes
};
int64_t grad_workspace(bool wgrad, int64_t M, int64_t N, int64_t K);
dg_status_t launch_dgrad(const GradArgs &a, const DeviceInfo &dev, cudaStream_t stream);
dg_status_t launch_wgrad(const GradArgs &a, const DeviceInfo &dev, cudaStream_t stream);

}  // namespace dg
