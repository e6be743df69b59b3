// Router: one 16-lane row per token (the per-token body is route_token16, route_token.h), and its
// gradient.
#include "route_token.h"

namespace tpg {

// four tokens per wave (one per 16-lane row), 16 per workgroup
__global__ __launch_bounds__(256) void route_topk_kernel(const float *__restrict__ logits,
                                                         const uint8_t *__restrict__ slot_drop, int T, int E, int k,
                                                         int32_t *__restrict__ topk_idx,
                                                         float *__restrict__ topk_w) {
    const int lane = threadIdx.x & 63;
    const int64_t t0 = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 6) * 4;  // first token of this wave
    if (t0 >= T) return;  // whole wave leaves together
    const int64_t t = t0 + (lane >> 4);
    route_token16(logits, slot_drop, t < T ? t : T - 1, t < T, E, k, lane & 15, topk_idx, topk_w, nullptr);
}

// Gradient of the router.  With the chosen experts' weights w_j = exp(l_j) / sum_i exp(l_i) and the
// gradients d_j that reached them (0 for a dropped slot),
//     dlogits[chosen expert j] = w_j (d_j - sum_i w_i d_i),   0 for the other experts.
// The chosen experts are found again from the logits (route_row's k rounds: E floats are read either
// way, and a dropped slot's id is not in topk_idx), with sum_j exp(l_j - l_max) and sum_j exp(l_j -
// l_max) d_j formed on the way; the lane that holds a winner keeps its exp and d.  One pass: reads T E
// + T k, writes T E floats.
template <int V>
__device__ __forceinline__ void route_row_backward(const float *__restrict__ logits,
                                                   const uint8_t *__restrict__ slot_drop,
                                                   const float *__restrict__ dtopk_w, int64_t t, bool valid, int E,
                                                   int k, int i, float *__restrict__ dlogits) {
    using namespace route_detail;
    const float *l = logits + t * E;
    uint32_t key[V];
    float ex[V], d[V];
#pragma unroll
    for (int q = 0; q < V; ++q) {
        const int e = i + 16 * q;
        key[q] = e < E ? logit_key(l[e]) : 0u;
        ex[q] = 0.0f;
        d[q] = 0.0f;
    }
    float lmax = 0.0f, z = 0.0f, zd = 0.0f;
    for (int j = 0; j < k; ++j) {
        uint32_t bk = 0u;
        int bq = 0;
#pragma unroll
        for (int q = 0; q < V; ++q)
            if (key[q] > bk) {
                bk = key[q];
                bq = q;
            }
        const uint32_t m = row_max(bk);
        const int win = (int)row_min(bk == m ? (uint32_t)(i + 16 * bq) : ~0u);
        const float lj = key_logit(m);
        if (j == 0) lmax = lj;
        const float exj = expf(lj - lmax);
        const int64_t s = t * k + j;
        const float dj = slot_drop != nullptr && slot_drop[s] != 0 ? 0.0f : dtopk_w[s];
        z += exj;
        zd = fmaf(exj, dj, zd);
        if ((win & 15) == i) {
#pragma unroll
            for (int q = 0; q < V; ++q)
                if (q == (win >> 4)) {
                    key[q] = 0u;
                    ex[q] = exj;
                    d[q] = dj;
                }
        }
    }
    if (!valid) return;
    const float mean = zd / z;
#pragma unroll
    for (int q = 0; q < V; ++q) {
        const int e = i + 16 * q;
        // a taken expert's key is 0, every other's is not
        if (e < E) dlogits[t * E + e] = key[q] == 0u ? ex[q] / z * (d[q] - mean) : 0.0f;
    }
}

constexpr int64_t kRouteGridX = 1 << 20;  // a grid dimension holds fewer than 2^32 threads

template <int V>
__global__ __launch_bounds__(256) void route_topk_backward_kernel(const float *__restrict__ logits,
                                                                  const uint8_t *__restrict__ slot_drop,
                                                                  const float *__restrict__ dtopk_w, int T, int E,
                                                                  int k, float *__restrict__ dlogits) {
    const int lane = threadIdx.x & 63;
    const int64_t t0 = ((int64_t)blockIdx.y * kRouteGridX + blockIdx.x) * 16 + (threadIdx.x >> 6) * 4;
    if (t0 >= T) return;
    const int64_t t = t0 + (lane >> 4);
    route_row_backward<V>(logits, slot_drop, dtopk_w, t < T ? t : T - 1, t < T, E, k, lane & 15, dlogits);
}

hipError_t launch_route_topk_backward(const float *logits, const uint8_t *slot_drop, const float *dtopk_w, int T,
                                      int E, int k, float *dlogits, hipStream_t s) {
    const int64_t blocks = ((int64_t)T + 15) / 16;
    const dim3 grid(std::min(blocks, kRouteGridX), (blocks + kRouteGridX - 1) / kRouteGridX);
    // experts per lane: the smallest power of two that holds E (route_token16's choice)
    const auto kernel = E <= 16    ? route_topk_backward_kernel<1>
                        : E <= 32  ? route_topk_backward_kernel<2>
                        : E <= 64  ? route_topk_backward_kernel<4>
                        : E <= 128 ? route_topk_backward_kernel<8>
                                   : route_topk_backward_kernel<16>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, logits, slot_drop, dtopk_w, T, E, k, dlogits);
    return hipGetLastError();
}

hipError_t launch_route_topk(const float *logits, const uint8_t *slot_drop, int T, int E, int k, int32_t *topk_idx,
                             float *topk_w, hipStream_t s) {
    const int blocks = (T + 15) / 16;
    hipLaunchKernelGGL(route_topk_kernel, dim3(blocks), dim3(256), 0, s, logits, slot_drop, T, E, k, topk_idx,
                       topk_w);
    return hipGetLastError();
}
}  // namespace tpg
