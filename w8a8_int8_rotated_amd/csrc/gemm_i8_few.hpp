// The INT8 product for few rows (gfx950): y[m, n] = ((float)(qx[m] . qw[n]) sx[m]) sw[n]
// (+ bias[n]), the bits of the tiled kernel (integer sums have no order).
//
// Bound: the weight's codes, read once (5 rows, K = 5376, N = 16128: 14 us, 6.2 TB/s).  A
// workgroup owns 16 RT outputs n of up to 16 CT rows; its 8 waves share out the tiles of 64
// inputs and join their integer sums in LDS.  One K-tile of 16 rows is one contiguous 1 KiB
// and exactly one operand of v_mfma_i32_16x16x64_i8 (weight rows as rows, tokens as columns).
// Each wave keeps a ring of D tiles in registers: the next is requested as soon as one is
// used.  RT: 1 where that gives every CU at most one workgroup, 4 where it halves the rounds
// of workgroups over the CUs that 2 makes (and its accumulators fit), else 2.
#pragma once

#include "common.hpp"

namespace convrot {

// Whether this kernel takes M rows of N outputs.  Up to 16 rows it always leads: N = 2^22, K = 128
// and 256: 173 us a call here, 254 in tiles, and 234, 324.  Up to 32 it does to about 2^20 outputs,
// where both write more than they read (K = 128, bf16, 32 rows: N = 2^19 37.1, 38.0; 2^20 74.4,
// 74.2; 2^21 156, 147; K = 512: 65.5, 68.8; 131, 133; 265, 255; K = 1024, 2^20: 215, 226), and up to
// 64 while a CU has at most 96 outputs: us here and in tiles for 32 and 64 rows, K = 5376: N = 5376:
// 10.4, 18.6 and 10.4, 19.7; 16128: 17.5, 33.4 and 24.3, 35.6; 32256: 32.2, 39.8 and 45.9, 42.7;
// 43008: 45.0, 49.5 and 64.8, 51.8 (four row tiles of X come from L2 for every two of the weight,
// and a tile's 256 rows cost the tiled kernel nothing once all CUs have one); 64 rows of
// N = 24576: K = 1024 9.8, 11.8; 5376 35.3, 40.0; 16384 99, 111; K = 21504, N = 5376: 30.9, 109 for
// 32 and 40.9, 117 for 64.
bool few_rows(int64_t M, int64_t N, int64_t cus)
{
    return M <= 16 || (M <= 32 && N <= 4096 * cus) || (M <= 64 && N <= 96 * cus);
}

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
constexpr int kWaves = 8;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t range_of(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes,
                                             0x00020000);
}

template <int RT, int CT, int D>
__global__ __launch_bounds__(64 * kWaves, 4) void few_kernel(
    const int8_t *__restrict__ qx, const int8_t *__restrict__ qw, const float *__restrict__ sx,
    const float *__restrict__ sw, const float *__restrict__ bias, void *__restrict__ Y, bool f32,
    int M, int N, int K)
{
    static_assert(RT * CT <= 8, "64 KiB of LDS");
    __shared__ int red[kWaves * RT * CT * 256];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = K / 64, nb0 = blockIdx.x * RT, blocks = N / 16;
    const int in_tile = r * 64 + ((q ^ ((r >> 2) & 3)) << 4);
    // row tiles past the last, and blocks, have an empty range
    __amdgpu_buffer_rsrc_t xs[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c)
        xs[c] = range_of(qx + (c * 16 < M ? c : 0) * 16 * (int64_t)K, c * 16 < M ? 16 * K : 0);
    __amdgpu_buffer_rsrc_t ws[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const bool in = nb0 + i < blocks;
        ws[i] = range_of(qw + (int64_t)(in ? nb0 + i : 0) * 16 * K, in ? 16 * K : 0);
    }
    v4i acc[RT][CT], a[D][RT], b[D][CT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[i][c] = (v4i)(0);
    int next = wave;
    auto request = [&](int d) {
        if (next >= tiles) return;
        const int at = next * 1024 + in_tile;
#pragma unroll
        for (int i = 0; i < RT; ++i)
            a[d][i] = __builtin_amdgcn_raw_buffer_load_b128(ws[i], at, 0, 0);
#pragma unroll
        for (int c = 0; c < CT; ++c)
            b[d][c] = __builtin_amdgcn_raw_buffer_load_b128(xs[c], at, 0, 0);
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
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    acc[i][c] =
                        __builtin_amdgcn_mfma_i32_16x16x64_i8(a[d][i], b[d][c], acc[i][c], 0, 0, 0);
            request(d);
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < CT; ++c)
            *reinterpret_cast<v4i *>(red + ((wave * RT + i) * CT + c) * 256 + lane * 4) = acc[i][c];
    __syncthreads();
    // a wave a tile; lane (r, q) of block i, row tile c: outputs 16 (nb0 + i) + 4 q .. + 3 of
    // row 16 c + r
    const int i = wave / CT, row = wave % CT * 16 + r;
    if (i >= RT || nb0 + i >= blocks || row >= M) return;
    v4i v = (v4i)(0);
#pragma unroll
    for (int k = 0; k < kWaves; ++k)
        v += *reinterpret_cast<const v4i *>(red + (k * RT * CT + wave) * 256 + lane * 4);
    const int n = (nb0 + i) * 16 + q * 4;
    const v4f s = *reinterpret_cast<const v4f *>(sw + n);
    const float sxm = sx[row];
    v4f y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = __fmul_rn(__fmul_rn((float)v[e], sxm), s[e]);
    if (bias) {
        const v4f c = *reinterpret_cast<const v4f *>(bias + n);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __fadd_rn(y[e], c[e]);
    }
    const int64_t o = (int64_t)row * N + n;
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
    const int rt = rounds(1) == 1 ? 1 : rounds(2) >= 2 * rounds(4) && M <= 32 ? 4 : 2;
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)((blocks + rt - 1) / rt)), dim3(64 * kWaves), 0,
                           stream, qx, qw, sx, sw, bias, Y, f32, (int)M, (int)N, (int)K);
    };
    if (M <= 16) {
        if (rt == 1) launch(few_kernel<1, 1, 4>);
        else if (rt == 2) launch(few_kernel<2, 1, 4>);
        else launch(few_kernel<4, 1, 2>);
    } else if (M <= 32) {
        if (rt == 1) launch(few_kernel<1, 2, 4>);
        else if (rt == 2) launch(few_kernel<2, 2, 3>);
        else launch(few_kernel<4, 2, 2>);
    } else {
        if (rt == 1) launch(few_kernel<1, 4, 3>);
        else launch(few_kernel<2, 4, 2>);
    }
    return hipGetLastError();
}

} // namespace
} // namespace convrot
