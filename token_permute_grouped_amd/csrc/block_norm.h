// Launchers of the norms around the block (block_norm.hip).
#pragma once
#include <type_traits>

#include "moe_internal.h"

namespace tpg {

struct NormArgs {
    const uint4 *weight;  // bf16 [H] or NULL: ones
    float eps, inv_h;
    bool on;              // false: no norm
};
struct ResidualArgs {
    const uint4 *x;  // bf16 [T][H] or NULL
    float scale;
    const float *gate;
    int gate_kind;
};

// workgroups (each with a partial row) of the backward kernels' sums over tokens: enough to fill
// the 256 CUs, each with up to 1024 threads
int norm_partials(const moe_problem &p);

// sets bytes (a multiple of 16) of dst, 16-byte aligned, to 0
hipError_t launch_zero(void *dst, size_t bytes, hipStream_t s);

hipError_t launch_prenorm(const void *x, const moe_norm *norm, const moe_problem &p, void *xn, void *xn8,
                          float *xn_scale, hipStream_t s);

// part: norm_partials(p) * H floats (unused without dweight)
hipError_t launch_prenorm_backward(const void *dx_perm, const int32_t *slot_row, const void *dxn, const void *dres,
                                   const void *x, const moe_norm *norm, const moe_problem &p, void *dx,
                                   float *dweight, float *part, hipStream_t s);

// slot_order as for launch_combine
hipError_t launch_combine_norm(const uint16_t *y, const int32_t *slot_row, const float *topk_w, const moe_norm *norm,
                               const moe_residual *residual, const moe_problem &p, bool slot_order, uint16_t *out,
                               hipStream_t s);

// part: norm_partials(p) * H floats (unused without dweight and a channel gate's dgate)
hipError_t launch_combine_norm_backward(const void *dout, const void *y, const int32_t *slot_row, const float *topk_w,
                                        const moe_norm *norm, const moe_residual *residual, const moe_problem &p,
                                        void *dy, float *dtopk_w, void *dresidual, float *dweight, float *dgate,
                                        float *part, hipStream_t s);

}  // namespace tpg
