// Building blocks shared by the bf16 GEMM kernels: buffer DMAs into LDS, their waits, the scheduling
// patterns, and MFMA fragments read from K-major stages through the LDS's transposing reads.
#pragma once
#include "moe_internal.h"

namespace tpg {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// A K-major stage (rows of 256 columns of one k): a row is sixteen 32-byte segments, segment s of row
// r at s ^ 2 (r & 3).  The logical 16-byte chunk that chunk position p of row r holds:
__device__ __forceinline__ int tchunk(int r, int p) { return p ^ ((r & 3) << 2); }

// MFMA fragment of 32 columns n0.. and the 16 k of step ks from a K-major stage: lane l gets column
// n0 + (l & 31), k = 16 ks + 8 (l >> 5) + 0..7, by two transposing reads of 4 k each.  In one, lane i
// of a group of 16 names 4 columns (i & 3) of row i >> 2 and gets column i of the 4 rows; the 32
// lanes that go together then read 8 distinct 32-byte segments, one per bank group.
__device__ __forceinline__ bf16x8 load_trans(const unsigned char *stage, int n0, int ks, int lane) {
    const int r = (lane & 15) >> 2, seg = (n0 >> 4) + ((lane >> 4) & 1);
    const unsigned char *p =
        stage + (ks * 16 + (lane >> 5) * 8 + r) * 512 + ((seg ^ (2 * r)) << 5) + (lane & 3) * 8;
    typedef __attribute__((address_space(3))) bf16x4 *lds_ptr;
    const bf16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_ptr)p);
    const bf16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_ptr)(p + 4 * 512));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// one 16-byte-per-lane DMA from a raw buffer straight into LDS (1 KB per wave, lane-linear)
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff, uint32_t soff, void *dst) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void *)dst, 16, voff, soff, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// LDS barrier without a global-memory fence: register loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// scheduling pattern: NR fragment reads (DS) spread evenly over M MFMAs
template <int NR, int M, int I = 0>
__device__ __forceinline__ void interleave_ds_mfma() {
    if constexpr (I < NR) {
        constexpr int m = (M * (I + 1)) / NR - (M * I) / NR;
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                       // DS read
        if constexpr (m > 0) __builtin_amdgcn_sched_group_barrier(0x008, m, 0);  // MFMA
        interleave_ds_mfma<NR, M, I + 1>();
    }
}

}  // namespace

}  // namespace tpg
