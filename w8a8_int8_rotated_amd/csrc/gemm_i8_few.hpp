// The INT8 product for few rows (gfx950): y[m, n] = ((float)(qx[m] . qw[n]) sx[m]) sw[n]
// (+ bias[n]), the bits of the tiled kernel (integer sums have no order).
//
// Bound: the weight's codes, read once.  A workgroup owns 16 RT outputs n; its 8 waves
// share out the tiles of 64 inputs and join their integer sums in LDS.  One K-tile of
// 16 rows is one contiguous 1 KiB and exactly one operand of v_mfma_i32_16x16x64_i8
// (weight rows as rows, tokens as columns).  Each wave keeps a ring of D tiles in
// registers: the next is requested as soon as one is used.
#pragma once

#include "common.hpp"

namespace convrot {

constexpr int64_t kFewRows = 16;

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
constexpr int kWaves = 8;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t range_of(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes,
                                             0x00020000);
}

template <int RT, int D>
__global__ __launch_bounds__(64 * kWaves, 4) void few_kernel(
    const int8_t *__restrict__ qx, const int8_t *__restrict__ qw, const float *__restrict__ sx,
    const float *__restrict__ sw, const float *__restrict__ bias, void *__restrict__ Y, bool f32,
    int M, int N, int K)
{
    __shared__ int red[kWaves * RT * 256];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = K / 64, nb0 = blockIdx.x * RT, blocks = N / 16;
    const int in_tile = r * 64 + ((q ^ ((r >> 2) & 3)) << 4);
    const __amdgpu_buffer_rsrc_t xs = range_of(qx, 16 * K);
    // blocks past the last have an empty range
    __amdgpu_buffer_rsrc_t ws[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const bool in = nb0 + i < blocks;
        ws[i] = range_of(qw + (int64_t)(in ? nb0 + i : 0) * 16 * K, in ? 16 * K : 0);
    }
    v4i acc[RT], a[D][RT], b[D];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = (v4i)(0);
    int next = wave;
    auto request = [&](int d) {
        if (next >= tiles) return;
        const int at = next * 1024 + in_tile;
#pragma unroll
        for (int i = 0; i < RT; ++i)
            a[d][i] = __builtin_amdgcn_raw_buffer_load_b128(ws[i], at, 0, 0);
        b[d] = __builtin_amdgcn_raw_buffer_load_b128(xs, at, 0, 0);
        next += kWaves;
        __builtin_amdgcn_sched_barrier(0);     // not all D uses first, then all requests
    };
#pragma unroll
    for (int d = 0; d < D; ++d) request(d);
    for (int t = wave; t < tiles; t += kWaves * D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (t + d * kWaves >= tiles) break;
#pragma unroll
            for (int i = 0; i < RT; ++i)
                acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[d][i], b[d], acc[i], 0, 0, 0);
            request(d);
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
        *reinterpret_cast<v4i *>(red + (wave * RT + i) * 256 + lane * 4) = acc[i];
    __syncthreads();
    // lane (r, q) of block i: outputs 16 (nb0 + i) + 4 q .. + 3 of row r
    if (wave >= RT || nb0 + wave >= blocks || r >= M) return;
    v4i v = (v4i)(0);
#pragma unroll
    for (int k = 0; k < kWaves; ++k)
        v += *reinterpret_cast<const v4i *>(red + (k * RT + wave) * 256 + lane * 4);
    const int n = (nb0 + wave) * 16 + q * 4;
    const v4f s = *reinterpret_cast<const v4f *>(sw + n);
    const float sxm = sx[r];
    v4f y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = __fmul_rn(__fmul_rn((float)v[e], sxm), s[e]);
    if (bias) {
        const v4f c = *reinterpret_cast<const v4f *>(bias + n);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __fadd_rn(y[e], c[e]);
    }
    const int64_t o = (int64_t)r * N + n;
    if (f32)
        *reinterpret_cast<v4f *>(static_cast<float *>(Y) + o) = y;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(Y) + o) =
            make_uint2(cvt_pk_bf16(y[0], y[1]), cvt_pk_bf16(y[2], y[3]));
}

// With the results of launch_gemm_i8 for OutKind::BF16 and F32.
hipError_t launch_gemm_i8_few(const int8_t *qx, const int8_t *qw, const float *sx,
                              const float *sw, const float *bias, void *Y, bool f32, int64_t M,
                              int64_t N, int64_t K, hipStream_t stream)
{
    const int64_t blocks = N / 16;
    const int64_t cus = device_cu_count();
    auto rounds = [&](int64_t t) { return ((blocks + t - 1) / t + cus - 1) / cus; };
    const int rt = rounds(1) == 1 ? 1 : rounds(2) >= 2 * rounds(4) ? 4 : 2;
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)((blocks + rt - 1) / rt)), dim3(64 * kWaves), 0,
                           stream, qx, qw, sx, sw, bias, Y, f32, (int)M, (int)N, (int)K);
    };
    if (rt == 1) launch(few_kernel<1, 4>);
    else if (rt == 2) launch(few_kernel<2, 4>);
    else launch(few_kernel<4, 2>);
    return hipGetLastError();
}

} // namespace
} // namespace convrot
