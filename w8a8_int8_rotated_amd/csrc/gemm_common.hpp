// Pieces shared by the GEMM kernels (gemm_i8.hip, gemm_fp8.hip): explicit waits,
// the barrier, and the interleaving of LDS reads and copies with the matrix
// instructions.
#pragma once

#include "common.hpp"

#include <utility>

namespace convrot {
namespace {

// buffer resource word 3: raw (untyped) 32-bit data format, no swizzle
constexpr int kRsrcWord3 = 0x00020000;

__device__ __forceinline__ int swz(int r) { return (r >> 2) & 3; }

// s_waitcnt vmcnt(n) with expcnt/lgkmcnt left unconstrained (gfx9 encoding).
template <int N>
__device__ __forceinline__ void wait_vmcnt()
{
    static_assert(N >= 0 && N < 64, "");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// s_waitcnt lgkmcnt(0) with vmcnt/expcnt left unconstrained.
__device__ __forceinline__ void wait_lds_reads()
{
    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));
}

__device__ __forceinline__ void block_barrier() { asm volatile("s_barrier" ::: "memory"); }

// Scheduling-group masks (LLVM AMDGPU sched_group_barrier).
constexpr int kSgMfma = 0x008, kSgVmemRead = 0x020, kSgDsRead = 0x100;

// Order the current scheduling region so that LDS reads and global->LDS
// copies trickle out between matrix instructions instead of blocking issue in
// bursts: the reads take every other MFMA slot from the first, the copies are
// spread evenly from the first slot on, so neither the LDS nor the
// texture-address queue sees the whole wave's requests at once.  (Copies
// spread from the first slot rather than ending at the last gave 0.5-0.9%
// at K = 512, 5376 and 21504: each copy gets a little longer to land.)
template <int MFMAS, int VMEMS, int DSREADS, int K>
__device__ __forceinline__ void interleave_slot()
{
    // reads [RD_LO, RD_HI) and copies [VM_LO, VM_HI) follow MFMA slot K
    constexpr int RD_LO = (K * DSREADS + MFMAS - 1) / MFMAS;
    constexpr int RD_HI = ((K + 1) * DSREADS + MFMAS - 1) / MFMAS;
    constexpr int VM_LO = (K * VMEMS + MFMAS - 1) / MFMAS;
    constexpr int VM_HI = ((K + 1) * VMEMS + MFMAS - 1) / MFMAS;
    __builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0);
    if constexpr (RD_HI > RD_LO) __builtin_amdgcn_sched_group_barrier(kSgDsRead, RD_HI - RD_LO, 0);
    if constexpr (VM_HI > VM_LO) __builtin_amdgcn_sched_group_barrier(kSgVmemRead, VM_HI - VM_LO, 0);
}

template <int MFMAS, int VMEMS, int DSREADS, int... K>
__device__ __forceinline__ void interleave_all(std::integer_sequence<int, K...>)
{
    (interleave_slot<MFMAS, VMEMS, DSREADS, K>(), ...);
}

template <int MFMAS, int VMEMS, int DSREADS>
__device__ __forceinline__ void interleave()
{
    interleave_all<MFMAS, VMEMS, DSREADS>(std::make_integer_sequence<int, MFMAS>{});
}

} // namespace
} // namespace convrot
