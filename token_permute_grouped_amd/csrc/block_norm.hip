// The norms in front of and behind the MoE block, and their gradients.
//
//   prenorm            n = v r w,  r = rsqrt(mean(v^2) + eps),  v = x[t]           (bf16 and / or fp8 + scales)
//   prenorm backward   dn = sum_j dx_perm[slot_row[j]] + dxn,  b = dn w
//                      dx = dres + r b - v r^3 mean(b v),  dweight = sum_t dn v r
//   combine norm       c = sum_j w_j y[slot_row[j]],  out = scale res + gate c r w
//   combine backward   b = dout gate w,  dc = r b - c r^3 mean(b c),  dy_j = w_j dc,  dw_j = dc . y_j,
//                      dweight = sum_t dout gate c r,  dgate = (sum over the gate's other index) dout c r w
//
// All of them are bound by HBM: a row is read once, kept in registers in fp32 (8 columns, one
// 16-byte chunk, per thread and pass), reduced once over the workgroup, and written once.  One
// workgroup works on one token at a time, with as many threads as the row has chunks (64 to 1024;
// NC = 1, 2, 4 or 8 chunks per thread, so that H = 65536 fits).  The combine's rows and the
// experts' gradient rows are read through slot_row in ascending j, as the combine kernel does.
//
// Both reductions of a backward pass are merged into one: mean(v^2) and mean(b v) do not depend
// on r, so one trip through the LDS gives r and the projection onto v at once.
//
// The sums over tokens (dweight, dgate of a channel gate) are kept in registers by workgroups that
// each walk over every G-th token; their G partial rows go to the workspace and a second launch adds
// them in a fixed order.
#include "block_norm.h"
#include "wave_ops.h"

namespace tpg {

namespace {
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxWaves = 16;

// One workgroup per token, the grid in two dimensions: a dimension holds fewer than 2^32 threads.
constexpr int kGridX = 1 << 20;
dim3 token_grid(int T) { return dim3(std::min(T, kGridX), ((int64_t)T + kGridX - 1) / kGridX); }
__device__ __forceinline__ int64_t token_of_block() { return (int64_t)blockIdx.y * kGridX + blockIdx.x; }

__device__ __forceinline__ uint4 load_once(const uint4 *p) {
    const u32x4 v = __builtin_nontemporal_load((const u32x4 *)p);
    return make_uint4(v.x, v.y, v.z, v.w);
}

__device__ __forceinline__ void unpack8(const uint4 &v, float *f) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        f[2 * q] = __uint_as_float(u[q] << 16);
        f[2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
    }
}

__device__ __forceinline__ float wave_sum(float x) {
    using namespace wave;
    x += __uint_as_float(dpp<kQuadSwap1, 0xf>(__float_as_uint(x), 0u));
    x += __uint_as_float(dpp<kQuadSwap2, 0xf>(__float_as_uint(x), 0u));
    x += __uint_as_float(dpp<kRowHalfMirror, 0xf>(__float_as_uint(x), 0u));
    x += __uint_as_float(dpp<kRowMirror, 0xf>(__float_as_uint(x), 0u));  // every lane: the sum of its row of 16
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// Sums of N values over the workgroup, in every thread, in an order that depends on its size
// alone.  `red` is kMaxWaves * N floats of LDS, which the workgroup may write again after its next
// barrier.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float *red) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, nw = blockDim.x >> 6;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if (nw == 1) return;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[wv * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = red[i];
        for (int w = 1; w < nw; ++w) s += red[w * N + i];
        v[i] = s;
    }
}

// acc = fp32 fma chain over a token's live slots in ascending j of (w ? w[j] : 1) * row slot_row[j]
// (or row j of the slot order); eight rows' loads are issued before any arithmetic
__device__ __forceinline__ void slot_sum(const uint4 *rows, const int32_t *slots, const float *w, int64_t t, int k,
                                         int row_vec, bool slot_order, int c, float *acc) {
    for (int j0 = 0; j0 < k; j0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int j = j0 + q;
            const int32_t r = j < k ? slots[j] : -1;
            v[q] = r >= 0 ? load_once(rows + (slot_order ? t * k + j : (int64_t)r) * row_vec + c)
                          : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int j = j0 + q;
            if (j < k && slots[j] >= 0) combine_fma8(acc, w ? w[j] : 1.0f, v[q]);
        }
    }
}

__device__ __forceinline__ void weight8(const uint4 *w, int c, float *f) {
    if (w) {
        unpack8(w[c], f);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = 1.0f;
    }
}

__device__ __forceinline__ void gate8(const float *gate, int kind, int64_t t, int c, float *f) {
    if (kind == MOE_GATE_CHANNEL) {
        const float4 a = ((const float4 *)gate)[2 * c], b = ((const float4 *)gate)[2 * c + 1];
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
        const float g = kind == MOE_GATE_TOKEN ? gate[t] : 1.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = g;
    }
}

__device__ __forceinline__ uint32_t fp8x4(const float *v) {
    int o = 0;
    float c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) c[q] = __builtin_amdgcn_fmed3f(v[q], -448.0f, 448.0f);
    o = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], o, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], o, true);
}

__device__ __forceinline__ void store_partial8(float *dst, int c, const float *f) {
    ((float4 *)dst)[2 * c] = make_float4(f[0], f[1], f[2], f[3]);
    ((float4 *)dst)[2 * c + 1] = make_float4(f[4], f[5], f[6], f[7]);
}
}  // namespace

template <int NC>
__global__ __launch_bounds__(1024) void prenorm_kernel(const uint4 *x, NormArgs n, int T, int row_vec, uint4 *xn,
                                                       uint2 *__restrict__ xn8, float *__restrict__ xn_scale) {
    __shared__ float red[kMaxWaves];
    const int64_t t = token_of_block();
    if (t >= T) return;
    const int nt = blockDim.x;
    float v[NC][8];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = threadIdx.x + i * nt;
        if (c < row_vec) {
            unpack8(x[t * row_vec + c], v[i]);
#pragma unroll
            for (int q = 0; q < 8; ++q) s[0] = fmaf(v[i][q], v[i][q], s[0]);
        }
    }
    float r = 1.0f;
    if (n.on) {
        block_sum<1>(s, red);
        r = rsqrtf(s[0] * n.inv_h + n.eps);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = threadIdx.x + i * nt;
        if (c >= row_vec) break;
        if (n.on) {
            float w[8];
            weight8(n.weight, c, w);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[i][q] = v[i][q] * r * w[q];
        }
        if (xn) xn[t * row_vec + c] = combine_pack8(v[i]);
        if (xn8) {
            // 128 columns are the chunks of 16 neighbouring lanes (row_vec and blockDim are multiples of 16)
            uint32_t m = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(v[i][q]) & 0x7fffffffu);
            using namespace wave;
            m = max(m, dpp<kQuadSwap1, 0xf>(m, 0u));
            m = max(m, dpp<kQuadSwap2, 0xf>(m, 0u));
            m = max(m, dpp<kRowHalfMirror, 0xf>(m, 0u));
            m = max(m, dpp<kRowMirror, 0xf>(m, 0u));
            float sc = __uint_as_float(m) / 448.0f;
            if (sc == 0.0f) sc = 1.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q) v[i][q] = v[i][q] / sc;
            xn8[t * row_vec + c] = make_uint2(fp8x4(v[i]), fp8x4(v[i] + 4));
            if ((c & 15) == 0) xn_scale[t * (row_vec >> 4) + (c >> 4)] = sc;
        }
    }
}

template <int NC>
__global__ __launch_bounds__(1024) void prenorm_backward_kernel(const uint4 *dx_perm, const int32_t *slot_row,
                                                                const uint4 *dxn, const uint4 *dres, const uint4 *x,
                                                                NormArgs n, int T, int k, int row_vec, uint4 *dx,
                                                                float *__restrict__ part) {
    __shared__ float red[2][kMaxWaves * 2];
    const int nt = blockDim.x;
    float dw[NC][8] = {};
    int flip = 0;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x, flip ^= 1) {
        float dn[NC][8], v[NC][8];
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = threadIdx.x + i * nt;
            if (c >= row_vec) break;
#pragma unroll
            for (int q = 0; q < 8; ++q) dn[i][q] = 0.f;
            if (dx_perm) slot_sum(dx_perm, slot_row + t * k, nullptr, t, k, row_vec, false, c, dn[i]);
            if (dxn) combine_fma8(dn[i], 1.0f, dxn[t * row_vec + c]);
            if (n.on) {
                float w[8];
                unpack8(x[t * row_vec + c], v[i]);
                weight8(n.weight, c, w);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    s[0] = fmaf(v[i][q], v[i][q], s[0]);
                    s[1] = fmaf(dn[i][q] * w[q], v[i][q], s[1]);
                }
            }
        }
        float r = 1.0f, coef = 0.0f;
        if (n.on) {
            block_sum<2>(s, red[flip]);
            r = rsqrtf(s[0] * n.inv_h + n.eps);
            coef = s[1] * n.inv_h * r * r * r;
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = threadIdx.x + i * nt;
            if (c >= row_vec) break;
            float o[8] = {};
            if (dres) unpack8(dres[t * row_vec + c], o);
            if (n.on) {
                float w[8];
                weight8(n.weight, c, w);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    dw[i][q] = fmaf(dn[i][q], v[i][q] * r, dw[i][q]);
                    o[q] += r * (dn[i][q] * w[q]) - v[i][q] * coef;
                }
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) o[q] += dn[i][q];
            }
            dx[t * row_vec + c] = combine_pack8(o);
        }
    }
    if (part) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = threadIdx.x + i * nt;
            if (c < row_vec) store_partial8(part + (int64_t)blockIdx.x * row_vec * 8, c, dw[i]);
        }
    }
}

template <int NC>
__global__ __launch_bounds__(1024) void combine_norm_kernel(const uint4 *__restrict__ y,
                                                            const int32_t *__restrict__ slot_row,
                                                            const float *__restrict__ topk_w, NormArgs n,
                                                            ResidualArgs res, int T, int k, int row_vec,
                                                            bool slot_order,
                                                            uint4 *out) {
    __shared__ float red[kMaxWaves];
    const int64_t t = token_of_block();
    if (t >= T) return;
    const int nt = blockDim.x;
    float v[NC][8];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = threadIdx.x + i * nt;
        if (c >= row_vec) break;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[i][q] = 0.f;
        slot_sum(y, slot_row + t * k, topk_w + t * k, t, k, row_vec, slot_order, c, v[i]);
#pragma unroll
        for (int q = 0; q < 8; ++q) s[0] = fmaf(v[i][q], v[i][q], s[0]);
    }
    float r = 1.0f;
    if (n.on) {
        block_sum<1>(s, red);
        r = rsqrtf(s[0] * n.inv_h + n.eps);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = threadIdx.x + i * nt;
        if (c >= row_vec) break;
        float g[8], w[8];
        gate8(res.gate, res.gate_kind, t, c, g);
        if (n.on) {
            weight8(n.weight, c, w);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[i][q] = v[i][q] * r * w[q];
        }
        float o[8];
        if (res.x) {
            unpack8(res.x[t * row_vec + c], o);
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = fmaf(res.scale, o[q], g[q] * v[i][q]);
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = g[q] * v[i][q];
        }
        out[t * row_vec + c] = combine_pack8(o);
    }
}

template <int NC>
__global__ __launch_bounds__(1024) void combine_norm_backward_kernel(
    const uint4 *dout, const uint4 *y, const int32_t *__restrict__ slot_row, const float *__restrict__ topk_w,
    NormArgs n, ResidualArgs res, int T, int k, int row_vec, uint4 *dy, float *__restrict__ dtopk_w, uint4 *dresidual,
    float *__restrict__ dgate_token, float *__restrict__ part_w, float *__restrict__ part_g) {
    __shared__ float red[kMaxWaves * 3], dots[2][kMaxWaves * 8];
    const int nt = blockDim.x, lane = threadIdx.x & 63, wv = threadIdx.x >> 6, nw = nt >> 6;
    float dw[NC][8] = {}, dg[NC][8] = {};
    int flip = 0;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const int32_t *slots = slot_row + t * k;
        const float *tw = topk_w + t * k;
        float c_[NC][8], d_[NC][8];  // the combined row, and dout
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = threadIdx.x + i * nt;
            if (c >= row_vec) break;
#pragma unroll
            for (int q = 0; q < 8; ++q) c_[i][q] = 0.f;
            slot_sum(y, slots, tw, t, k, row_vec, false, c, c_[i]);
            unpack8(dout[t * row_vec + c], d_[i]);
            float w[8], g[8];
            weight8(n.weight, c, w);
            gate8(res.gate, res.gate_kind, t, c, g);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float dwc = d_[i][q] * w[q] * c_[i][q];
                s[0] = fmaf(c_[i][q], c_[i][q], s[0]);
                s[1] = fmaf(g[q], dwc, s[1]);
                s[2] += dwc;
            }
        }
        block_sum<3>(s, red);
        float r = 1.0f, coef = 0.0f;
        if (n.on) {
            r = rsqrtf(s[0] * n.inv_h + n.eps);
            coef = s[1] * n.inv_h * r * r * r;
        }
        if (dgate_token && threadIdx.x == 0) dgate_token[t] = s[2] * r;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = threadIdx.x + i * nt;
            if (c >= row_vec) break;
            float w[8], g[8], o[8];
            weight8(n.weight, c, w);
            gate8(res.gate, res.gate_kind, t, c, g);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float ch = c_[i][q] * r;
                dw[i][q] = fmaf(d_[i][q] * g[q], ch, dw[i][q]);
                dg[i][q] = fmaf(d_[i][q] * w[q], ch, dg[i][q]);
                o[q] = d_[i][q] * res.scale;
                d_[i][q] = r * (d_[i][q] * g[q] * w[q]) - c_[i][q] * coef;  // dc
            }
            if (dresidual) dresidual[t * row_vec + c] = combine_pack8(o);
        }
        for (int j0 = 0; j0 < k; j0 += 8, flip ^= 1) {
            float dot[8] = {};
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = threadIdx.x + i * nt;
                if (c >= row_vec) break;
                uint4 v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int32_t row = j0 + q < k ? slots[j0 + q] : -1;
                    v[q] = row >= 0 && dtopk_w ? y[(int64_t)row * row_vec + c] : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    if (j0 + q >= k || slots[j0 + q] < 0) continue;
                    float f[8], o[8];
                    unpack8(v[q], f);
#pragma unroll
                    for (int z = 0; z < 8; ++z) {
                        dot[q] = fmaf(d_[i][z], f[z], dot[q]);
                        o[z] = tw[j0 + q] * d_[i][z];
                    }
                    dy[(int64_t)slots[j0 + q] * row_vec + c] = combine_pack8(o);
                }
            }
            if (dtopk_w) {
#pragma unroll
                for (int q = 0; q < 8; ++q) dot[q] = wave_sum(dot[q]);
                if (lane == 0)
#pragma unroll
                    for (int q = 0; q < 8; ++q) dots[flip][wv * 8 + q] = dot[q];
                __syncthreads();
                const int j = j0 + threadIdx.x;
                if (threadIdx.x < 8 && j < k) {
                    float sum = 0.f;
                    for (int w = 0; w < nw; ++w) sum += dots[flip][w * 8 + threadIdx.x];
                    dtopk_w[t * k + j] = slots[j] >= 0 ? sum : 0.f;
                }
            }
        }
        if (!dtopk_w) __syncthreads();  // red is written again
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = threadIdx.x + i * nt;
        if (c >= row_vec) break;
        if (part_w) store_partial8(part_w + (int64_t)blockIdx.x * row_vec * 8, c, dw[i]);
        if (part_g) store_partial8(part_g + (int64_t)blockIdx.x * row_vec * 8, c, dg[i]);
    }
}

// out[h] = sum over the G partial rows, in a fixed order: 32 columns and 32 row groups per workgroup
__global__ __launch_bounds__(1024) void column_sum_kernel(const float *__restrict__ part, int G, int H,
                                                          float *__restrict__ out) {
    __shared__ float red[32][33];
    const int col = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int h = blockIdx.x * 32 + col;  // H is a multiple of 128
    float s = 0.f;
    for (int g = grp; g < G; g += 32) s += part[(int64_t)g * H + h];
    red[grp][col] = s;
    __syncthreads();
    if (grp == 0) {
        float a = 0.f;
#pragma unroll
        for (int g = 0; g < 32; ++g) a += red[g][col];
        out[h] = a;
    }
}

// bytes of dst set to 0 (a kernel and not a memset, so that a captured call replays as one)
__global__ __launch_bounds__(256) void zero_kernel(uint4 *__restrict__ dst, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        dst[i] = make_uint4(0, 0, 0, 0);
}

namespace {
struct RowShape {
    int threads, chunks;  // threads of a workgroup, chunks per thread (1, 2, 4 or 8)
};
RowShape row_shape(int H) {
    const int row_vec = H / 8;
    int nc = 1;
    while (row_vec > 1024 * nc) nc *= 2;
    return {((row_vec + nc - 1) / nc + 63) / 64 * 64, nc};
}

template <typename F>
void with_chunks(int nc, F f) {
    switch (nc) {
        case 1: f(std::integral_constant<int, 1>{}); break;
        case 2: f(std::integral_constant<int, 2>{}); break;
        case 4: f(std::integral_constant<int, 4>{}); break;
        default: f(std::integral_constant<int, 8>{}); break;
    }
}

NormArgs norm_args(const moe_norm *n, int H) {
    return {n ? (const uint4 *)n->weight : nullptr, n ? n->eps : 0.f, 1.0f / (float)H, n != nullptr};
}
ResidualArgs residual_args(const moe_residual *r) {
    if (!r) return {nullptr, 0.f, nullptr, MOE_GATE_NONE};
    return {(const uint4 *)r->x, r->scale, r->gate, r->gate_kind};
}
}  // namespace

int norm_partials(const moe_problem &p) {
    const int per_cu = std::max(1, std::min(8, 1024 / row_shape(p.H).threads));
    return std::min(p.T, 256 * per_cu);
}

hipError_t launch_zero(void *dst, size_t bytes, hipStream_t s) {
    const int64_t n = (int64_t)(bytes / 16);
    hipLaunchKernelGGL(zero_kernel, dim3(std::min<int64_t>((n + 255) / 256, 4096)), dim3(256), 0, s, (uint4 *)dst, n);
    return hipGetLastError();
}

hipError_t launch_prenorm(const void *x, const moe_norm *norm, const moe_problem &p, void *xn, void *xn8,
                          float *xn_scale, hipStream_t s) {
    const RowShape rs = row_shape(p.H);
    with_chunks(rs.chunks, [&](auto nc) {
        hipLaunchKernelGGL(prenorm_kernel<decltype(nc)::value>, token_grid(p.T), dim3(rs.threads), 0, s,
                           (const uint4 *)x, norm_args(norm, p.H), p.T, p.H / 8, (uint4 *)xn, (uint2 *)xn8, xn_scale);
    });
    return hipGetLastError();
}

hipError_t launch_prenorm_backward(const void *dx_perm, const int32_t *slot_row, const void *dxn, const void *dres,
                                   const void *x, const moe_norm *norm, const moe_problem &p, void *dx,
                                   float *dweight, float *part, hipStream_t s) {
    const RowShape rs = row_shape(p.H);
    const int G = norm_partials(p);
    with_chunks(rs.chunks, [&](auto nc) {
        hipLaunchKernelGGL(prenorm_backward_kernel<decltype(nc)::value>, dim3(G), dim3(rs.threads), 0, s,
                           (const uint4 *)dx_perm, slot_row, (const uint4 *)dxn, (const uint4 *)dres, (const uint4 *)x,
                           norm_args(norm, p.H), p.T, p.k, p.H / 8, (uint4 *)dx, dweight ? part : nullptr);
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !dweight) return e;
    hipLaunchKernelGGL(column_sum_kernel, dim3(p.H / 32), dim3(1024), 0, s, part, G, p.H, dweight);
    return hipGetLastError();
}

hipError_t launch_combine_norm(const uint16_t *y, const int32_t *slot_row, const float *topk_w, const moe_norm *norm,
                               const moe_residual *residual, const moe_problem &p, bool slot_order, uint16_t *out,
                               hipStream_t s) {
    const RowShape rs = row_shape(p.H);
    with_chunks(rs.chunks, [&](auto nc) {
        hipLaunchKernelGGL(combine_norm_kernel<decltype(nc)::value>, token_grid(p.T), dim3(rs.threads), 0, s,
                           (const uint4 *)y, slot_row, topk_w, norm_args(norm, p.H), residual_args(residual), p.T, p.k,
                           p.H / 8, slot_order, (uint4 *)out);
    });
    return hipGetLastError();
}

hipError_t launch_combine_norm_backward(const void *dout, const void *y, const int32_t *slot_row, const float *topk_w,
                                        const moe_norm *norm, const moe_residual *residual, const moe_problem &p,
                                        void *dy, float *dtopk_w, void *dresidual, float *dweight, float *dgate,
                                        float *part, hipStream_t s) {
    const RowShape rs = row_shape(p.H);
    const int G = norm_partials(p);
    const bool channel = dgate && residual->gate_kind == MOE_GATE_CHANNEL;
    float *part_w = dweight ? part : nullptr, *part_g = channel ? part + (size_t)G * p.H : nullptr;
    with_chunks(rs.chunks, [&](auto nc) {
        hipLaunchKernelGGL(combine_norm_backward_kernel<decltype(nc)::value>, dim3(G), dim3(rs.threads), 0, s,
                           (const uint4 *)dout, (const uint4 *)y, slot_row, topk_w, norm_args(norm, p.H),
                           residual_args(residual), p.T, p.k, p.H / 8, (uint4 *)dy, dtopk_w, (uint4 *)dresidual,
                           channel ? nullptr : dgate, part_w, part_g);
    });
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && dweight) {
        hipLaunchKernelGGL(column_sum_kernel, dim3(p.H / 32), dim3(1024), 0, s, part_w, G, p.H, dweight);
        e = hipGetLastError();
    }
    if (e == hipSuccess && channel) {
        hipLaunchKernelGGL(column_sum_kernel, dim3(p.H / 32), dim3(1024), 0, s, part_g, G, p.H, dgate);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace tpg
