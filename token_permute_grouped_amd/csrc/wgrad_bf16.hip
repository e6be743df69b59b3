// Weight gradients of the grouped FFN in bf16 on CDNA4 matrix cores (v_mfma_f32_32x32x16_bf16):
//
//     dW_e[m][n] = sum over the rows r of expert e of P[r][m] Q[r][n]
//
// dW1: P = dgu, Q = x_perm; dW2: P = dy_perm, Q = h.  The sum runs over the expert's ragged row
// count (0 to T k); M x N outputs per expert.  4 R H I (dW1) and 2 R H I (dW2) flops; with many rows the
// matrix cores bound it, with few the M N outputs' stores.
//
// Both operands have the sum's index on their rows, so a stage is 32 rows of 256 columns of each,
// brought straight into LDS by 16-byte-per-lane DMAs (512 bytes contiguous per row), and the MFMA
// fragments come through the LDS's transposing reads (load_trans).  A workgroup of 8 waves owns a 256 x 256
// output tile (128 x 64 per wave).  LDS is a ring of five 32 KB stages.  A stage's one barrier stands
// before its last 16-row step: by then every wave has read the stage's fragments, so its slot takes the
// DMAs of the stage five ahead, and the next stage's first fragments load under the step's MFMAs.
//
// Rows past the expert's last read as zero (buffer bounds, set for every stage, so that 64-bit row
// offsets stay in the base address); columns past M or N are computed from whatever the row holds and not
// stored.  The DMAs of stages past the end are issued too, so that one wait count fits every stage.
//
// Work order.  Experts go largest first.  32 (or fewer) neighbouring tiles of one expert form a rectangle that
// one XCD (block index mod 8) works on at once, sharing the rectangle's row and column slabs in its L2.
#include "gemm_trans.h"

namespace tpg {

namespace {
constexpr int kBM = 256, kBN = 256, kBK = 32;
constexpr int kWaves = 8, kThreads = 64 * kWaves, kWaveN = 4;
constexpr int kHalf = kBK * 512;      // 16 KB: one operand of a stage
constexpr int kStage = 2 * kHalf;     // 32 KB
constexpr int kStages = 5;
constexpr int kOps = kHalf / 1024 / kWaves;  // DMAs per wave, stage and operand (2)

struct Rects {
    int rm, rn, cols, per_expert;  // tiles of a rectangle, rectangles along n, rectangles of an expert
};
__host__ __device__ inline Rects rects(int M, int N) {
    const int nb_m = (M + kBM - 1) / kBM, nb_n = (N + kBN - 1) / kBN;
    const int rn = nb_n < 8 ? nb_n : 8, rm = nb_m < 32 / rn ? nb_m : 32 / rn;
    const int cols = (nb_n + rn - 1) / rn;
    return {rm, rn, cols, cols * ((nb_m + rm - 1) / rm)};
}
}  // namespace

// order[rank] = expert, by descending row count (ties: lower expert first); one workgroup of 256
__global__ __launch_bounds__(256) void expert_order_kernel(const int32_t *__restrict__ offsets, int E,
                                                           int32_t *__restrict__ order) {
    __shared__ int cnt[256];
    const int e = threadIdx.x;
    cnt[e] = e < E ? offsets[e + 1] - offsets[e] : -1;
    __syncthreads();
    if (e >= E) return;
    int rank = 0;
    for (int i = 0; i < E; ++i) rank += cnt[i] > cnt[e] || (cnt[i] == cnt[e] && i < e);
    order[rank] = e;
}

__global__ __launch_bounds__(kThreads, 1) void wgrad_bf16_kernel(const uint16_t *__restrict__ P, int M,
                                                                 const uint16_t *__restrict__ Q, int N,
                                                                 const int32_t *__restrict__ offsets,
                                                                 const int32_t *__restrict__ order, int E,
                                                                 uint16_t *__restrict__ dW) {
    __shared__ __attribute__((aligned(1024))) unsigned char lds[kStages * kStage];
    const Rects rc = rects(M, N);
    const int area = rc.rm * rc.rn;
    const int q = blockIdx.x >> 3, rect = q / area * 8 + (blockIdx.x & 7), in = q % area;
    if (rect >= E * rc.per_expert) return;
    const int e = order[rect / rc.per_expert], re = rect % rc.per_expert;
    const int m0 = ((re / rc.cols) * rc.rm + in / rc.rn) * kBM, n0 = ((re % rc.cols) * rc.rn + in % rc.rn) * kBN;
    if (m0 >= M || n0 >= N) return;
    const int64_t row0 = offsets[e];
    const int rows = offsets[e + 1] - (int)row0;
    const int nk = (rows + kBK - 1) / kBK;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / kWaveN, wn = wave % kWaveN;

    // byte offsets of this lane's DMAs within a stage's rows
    uint32_t offP[kOps], offQ[kOps];
#pragma unroll
    for (int i = 0; i < kOps; ++i) {
        const int r = wave * (kBK / kWaves) + i * 2 + (lane >> 5), c = tchunk(r, lane & 31) * 8;
        offP[i] = (uint32_t)(r * M + m0 + c) * 2u;
        offQ[i] = (uint32_t)(r * N + n0 + c) * 2u;
    }
    auto dma = [&](int kt, int slot) {
        const int left = max(0, min(kBK, rows - kt * kBK));  // 0: every lane is out of bounds
        const int64_t r = row0 + (left > 0 ? (int64_t)kt * kBK : 0);
        const __amdgpu_buffer_rsrc_t rp =
            __builtin_amdgcn_make_buffer_rsrc((void *)(P + r * M), (short)0, left * M * 2, 0x00020000);
        const __amdgpu_buffer_rsrc_t rq =
            __builtin_amdgcn_make_buffer_rsrc((void *)(Q + r * N), (short)0, left * N * 2, 0x00020000);
        unsigned char *dst = lds + slot * kStage + wave * (kBK / kWaves) * 512;
#pragma unroll
        for (int i = 0; i < kOps; ++i) {
            dma16(rp, offP[i], 0, dst + i * 1024);
            dma16(rq, offQ[i], 0, dst + kHalf + i * 1024);
        }
    };

    f32x16 acc[2][4];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.f;

    if (nk > 0) {
        bf16x8 fq[2][2], fp[2][4];
        auto load = [&](int buf, int slot, int ks) {
            const unsigned char *s = lds + slot * kStage;
#pragma unroll
            for (int a = 0; a < 2; ++a) fq[buf][a] = load_trans(s + kHalf, wn * 64 + a * 32, ks, lane);
#pragma unroll
            for (int b = 0; b < 4; ++b) fp[buf][b] = load_trans(s, wm * 128 + b * 32, ks, lane);
        };
        auto mfmas = [&](int buf) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int a = 0; a < 2; ++a)
                    acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fq[buf][a], fp[buf][b], acc[a][b], 0, 0, 0);
        };
        constexpr int G = 2 * kOps;  // DMAs of one stage
#pragma unroll
        for (int s = 0; s < kStages; ++s) {
            dma(s, s);
            asm volatile("" ::: "memory");
        }
        wait_vmcnt<(kStages - 1) * G>();
        lds_barrier();
        load(0, 0, 0);
        int slot = 0;
        for (int kt = 0; kt < nk; ++kt) {
            load(1, slot, 1);
            mfmas(0);
            interleave_ds_mfma<12, 8>();
            // stages kt+2 .. kt+4 may be in flight
            wait_vmcnt<(kStages - 2) * G>();
            lds_barrier();
            dma(kt + kStages, slot);
            __builtin_amdgcn_sched_group_barrier(0x020, G, 0);
            slot = slot + 1 == kStages ? 0 : slot + 1;
            load(0, slot, 0);
            mfmas(1);
            interleave_ds_mfma<12, 8>();
        }
        wait_vmcnt<0>();  // the LDS is written again below
    }

    // lane holds row m = wm 128 + b 32 + (lane & 31) and columns wn 64 + a 32 + 8 (v >> 2) + 4 (lane >> 5) +
    // (v & 3); the tile goes through LDS so that whole rows are stored
    auto cofs = [](int r, int c) { return r * (kBN * 2) + ((c ^ (r & 15)) << 4); };
    const int half = lane >> 5;
    lds_barrier();
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int tr = wm * 128 + b * 32 + (lane & 31);
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int g4 = 0; g4 < 4; ++g4) {
                u32x2 o;
                o.x = pack_bf16x2(acc[a][b][g4 * 4 + 0], acc[a][b][g4 * 4 + 1]);
                o.y = pack_bf16x2(acc[a][b][g4 * 4 + 2], acc[a][b][g4 * 4 + 3]);
                *(u32x2 *)(lds + cofs(tr, wn * 8 + a * 4 + g4) + half * 8) = o;
            }
    }
    lds_barrier();
    const int c = n0 + (lane & 31) * 8;
    if (c < N) {
        uint16_t *out = dW + (int64_t)e * M * N;
#pragma unroll 4
        for (int tr = wave * 2 + half; tr < kBM; tr += kWaves * 2)
            if (m0 + tr < M)
                *(u32x4 *)(out + (int64_t)(m0 + tr) * N + c) = *(const u32x4 *)(lds + cofs(tr, lane & 31));
    }
}

hipError_t launch_expert_order(const int32_t *offsets, int E, int32_t *order, hipStream_t s) {
    hipLaunchKernelGGL(expert_order_kernel, dim3(1), dim3(256), 0, s, offsets, E, order);
    return hipGetLastError();
}

hipError_t launch_wgrad_bf16(const uint16_t *p, int M, const uint16_t *q, int N, const int32_t *offsets,
                             const int32_t *order, int E, uint16_t *dw, hipStream_t s) {
    const Rects rc = rects(M, N);
    const int64_t blocks = ((int64_t)E * rc.per_expert + 7) / 8 * 8 * rc.rm * rc.rn;
    hipLaunchKernelGGL(wgrad_bf16_kernel, dim3(blocks), dim3(kThreads), 0, s, p, M, q, N, offsets, order, E, dw);
    return hipGetLastError();
}

}  // namespace tpg
