// Norms of queries and keys for each head and the rotation by positions with
// several axes, in one pass over the rows (gfx950).
//
//   rope:      y = R(pos) x
//   norm:      y = R(pos) (x r w),  r = rsqrt(mean(x^2) + eps) over a head's D
//   backward:  g' = R(pos)^T g;  dw = sum g' x r;  t = g' w;
//              dx = r (t - x r^2 mean(t x))
//
// Each row is read and written once, so the bound is memory: 4 bytes per bf16
// element forward, 6 backward.
//
// A workgroup takes one token at a time: its threads evaluate the token's R/2
// cosines and sines once, into LDS, and its waves share out the token's heads
// (84 heads of 128 channels use 64 sincos).  A lane holds 16 channels of a head,
// two runs of 8: adjacent ones when pairs are interleaved, 8 channels and their
// 8 partners for the half-split pairs, so that a rotation never leaves the
// lane.  A head is LPH lanes (a power of two), a wave 64 / LPH heads, and the
// norm's sum runs over the LPH lanes with DPP.
//
// Angles: positions times frequencies in fp64, reduced to revolutions in
// [-1/2, 1/2] there (an fp32 angle at position 10^6 is off by 0.06 radians),
// then sin and cos of the reduced angle in fp32.
#include "common.hpp"

#include <algorithm>

namespace convrot {
namespace {

enum Pairing { kInterleaved = 0, kHalf8 = 1, kHalf4 = 2 };

// Sum over aligned groups of 1 << lg lanes (lg uniform).
__device__ __forceinline__ float group_sum(float v, int lg)
{
#define CR_DPP_ADD(CTRL)                                                                          \
    v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true))
    if (lg >= 1) CR_DPP_ADD(0xB1);    // lane ^ 1
    if (lg >= 2) CR_DPP_ADD(0x4E);    // lane ^ 2
    if (lg >= 3) CR_DPP_ADD(0x141);   // the other four lanes of eight
    if (lg >= 4) CR_DPP_ADD(0x140);   // the other eight of sixteen
#undef CR_DPP_ADD
    if (lg >= 5) v += __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401F));
    if (lg >= 6) v += __shfl_xor(v, 32, 64);
    return v;
}

// The channels of one lane: two runs of up to 8, starting at a and b, and its
// first pair.  n[0], n[1]: channels in each run (0, 4 or 8); nrot: how many of
// its 8 pairs are rotated.
struct LaneMap {
    int off[2], n[2], p0, nrot;
};

template <int PAIR>
__device__ __forceinline__ LaneMap lane_map(int c, int D, int R)
{
    LaneMap m;
    const int half = R >> 1;
    m.p0 = 8 * c;
    m.nrot = min(max(half - 8 * c, 0), 8);
    if (PAIR == kInterleaved) {
        m.off[0] = 16 * c;
        m.off[1] = 16 * c + 8;
        m.n[0] = m.off[0] < D ? 8 : 0;
        m.n[1] = m.off[1] < D ? 8 : 0;
    } else {
        const int lanes = (half + 7) >> 3;     // lanes that rotate
        if (c < lanes) {
            m.off[0] = 8 * c;
            m.off[1] = half + 8 * c;
            m.n[0] = m.n[1] = m.nrot;
        } else {
            m.off[0] = R + 16 * (c - lanes);
            m.off[1] = m.off[0] + 8;
            m.n[0] = m.off[0] < D ? 8 : 0;
            m.n[1] = m.off[1] < D ? 8 : 0;
        }
    }
    return m;
}

// A run of n (0, 4 or 8) channels at p; zeros beyond n.  Half-split pairs with
// R/2 an odd multiple of 4 (kHalf4) start runs 8 bytes off, so bf16 runs move as two
// 8-byte halves there.
template <bool F32, int PAIR>
__device__ __forceinline__ void load_run(const void *base, int64_t off, int n, float (&v)[8])
{
    if constexpr (F32) {
        const float *p = static_cast<const float *>(base) + off;
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 a = n > 0 ? *reinterpret_cast<const float4 *>(p) : z;
        const float4 b = n > 4 ? *reinterpret_cast<const float4 *>(p + 4) : z;
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(base) + off;
        uint4 u = make_uint4(0, 0, 0, 0);
        if constexpr (PAIR == kHalf4) {
            if (n > 0) {
                const uint2 a = *reinterpret_cast<const uint2 *>(p);
                u.x = a.x; u.y = a.y;
            }
            if (n > 4) {
                const uint2 b = *reinterpret_cast<const uint2 *>(p + 4);
                u.z = b.x; u.w = b.y;
            }
        } else {
            if (n > 0) u = *reinterpret_cast<const uint4 *>(p);
        }
        v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
    }
}

template <bool F32, int PAIR>
__device__ __forceinline__ void store_run(void *base, int64_t off, int n, const float (&v)[8])
{
    if constexpr (F32) {
        float *p = static_cast<float *>(base) + off;
        if (n > 0) *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        if (n > 4) *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint16_t *p = static_cast<uint16_t *>(base) + off;
        const uint4 u = make_uint4(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]),
                                   cvt_pk_bf16(v[4], v[5]), cvt_pk_bf16(v[6], v[7]));
        if constexpr (PAIR == kHalf4) {
            if (n > 0) *reinterpret_cast<uint2 *>(p) = make_uint2(u.x, u.y);
            if (n > 4) *reinterpret_cast<uint2 *>(p + 4) = make_uint2(u.z, u.w);
        } else {
            if (n > 0) *reinterpret_cast<uint4 *>(p) = u;
        }
    }
}

// The lane's pairs turned by (cs, sn); pairs from nrot on pass unchanged.
template <int PAIR>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float (&cs)[8],
                                       const float (&sn)[8], int nrot)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float &u = PAIR == kInterleaved ? (i < 4 ? a[2 * i] : b[2 * i - 8]) : a[i];
        float &v = PAIR == kInterleaved ? (i < 4 ? a[2 * i + 1] : b[2 * i - 7]) : b[i];
        const float x = __builtin_fmaf(u, cs[i], -(v * sn[i]));
        const float y = __builtin_fmaf(v, cs[i], u * sn[i]);
        u = i < nrot ? x : u;
        v = i < nrot ? y : v;
    }
}

// cos and sin of the token's pairs into tab; entries from R/2 up to npad are
// never used in a rotation but are read.
__device__ __forceinline__ void fill_table(const NormRope &a, int64_t pos_at, float2 *tab,
                                           int npad)
{
    const int half = a.R >> 1;
    for (int p = threadIdx.x; p < npad; p += blockDim.x) {
        float s = 0.0f, c = 1.0f;
        if (p < half) {
            const int ax = min(max(a.axis[p], 0), a.axes - 1);
            const double pos = a.pos_f32
                                   ? (double)static_cast<const float *>(a.pos)[pos_at + ax]
                                   : (double)static_cast<const int32_t *>(a.pos)[pos_at + ax];
            double rev = pos * a.freq[p] * 0.15915494309189535;
            rev -= rint(rev);
            sincospif((float)(2.0 * rev), &s, &c);
            if (a.inverse) s = -s;
        }
        tab[p] = make_float2(c, s);
    }
}

// Token loop of a workgroup of W waves; wave w takes units w, w + W, ..., a
// unit being up to 64 / LPH heads of the queries or of the keys.  The table is
// double-buffered, so one barrier per token separates its writers from its
// readers (a wave can be at most one token ahead of another).
template <bool F32, NormRopeMode MODE, int PAIR>
__global__ void norm_rope_kernel(NormRope a, int lg)
{
    constexpr bool NORM = MODE != NormRopeMode::ROPE;
    constexpr bool BWD = MODE == NormRopeMode::BACKWARD;
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const int lph = 1 << lg, hpw = 64 >> lg, npad = 8 * lph;
    float2 *const tab = reinterpret_cast<float2 *>(lds);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const LaneMap m = lane_map<PAIR>(lane & (lph - 1), a.D, a.R);
    const int hg = lane >> lg;
    const int units0 = (a.heads[0] + hpw - 1) >> (6 - lg);
    const int units = units0 + ((a.heads[1] + hpw - 1) >> (6 - lg));
    const int tokens = a.B * a.T;
    const float invD = 1.0f / (float)a.D;

    float dw[2][2][8] = {};   // backward: [side][run] sums of g' x r
    int buf = 0;
    for (int tok = blockIdx.x; tok < tokens; tok += gridDim.x, buf ^= 1) {
        const int b = tok / a.T, t = tok - b * a.T;
        float2 *const tb = tab + buf * npad;
        fill_table(a, b * a.pos_sb + (int64_t)t * a.axes, tb, npad);
        __syncthreads();
        float cs[8], sn[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = tb[m.p0 + i];
            cs[i] = v.x;
            sn[i] = v.y;
        }
        for (int u = wave; u < units; u += waves) {
            const int side = u >= units0 ? 1 : 0;
            const int head = (u - (side ? units0 : 0)) * hpw + hg;
            const bool live = head < a.heads[side];
            const HeadRows &xr = a.x[side], &yr = a.out[side];
            const int na = live ? m.n[0] : 0, nb = live ? m.n[1] : 0;
            float va[8], vb[8], w[2][8];
            const int64_t xo = b * xr.sb + t * xr.st + head * xr.sh;
            load_run<F32, PAIR>(xr.p, xo + m.off[0], na, va);
            load_run<F32, PAIR>(xr.p, xo + m.off[1], nb, vb);
            if constexpr (NORM) {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[0][i] = w[1][i] = 1.0f;
                if (a.w[side]) {
                    load_run<true, PAIR>(a.w[side], m.off[0], m.n[0], w[0]);
                    load_run<true, PAIR>(a.w[side], m.off[1], m.n[1], w[1]);
                }
            }
            float r = 1.0f;
            if constexpr (NORM) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    ss = __builtin_fmaf(va[i], va[i], __builtin_fmaf(vb[i], vb[i], ss));
                r = rsqrtf(__builtin_fmaf(group_sum(ss, lg), invD, a.eps));
            }
            if constexpr (!BWD) {
                if constexpr (NORM) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        va[i] = va[i] * r * w[0][i];
                        vb[i] = vb[i] * r * w[1][i];
                    }
                }
                rotate<PAIR>(va, vb, cs, sn, m.nrot);
            } else {
                const HeadRows &gr = a.g[side];
                const int64_t go = b * gr.sb + t * gr.st + head * gr.sh;
                float ga[8], gb[8];
                load_run<F32, PAIR>(gr.p, go + m.off[0], na, ga);
                load_run<F32, PAIR>(gr.p, go + m.off[1], nb, gb);
                rotate<PAIR>(ga, gb, cs, sn, m.nrot);
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    va[i] *= r;
                    vb[i] *= r;
                    if (side) {
                        dw[1][0][i] = __builtin_fmaf(ga[i], va[i], dw[1][0][i]);
                        dw[1][1][i] = __builtin_fmaf(gb[i], vb[i], dw[1][1][i]);
                    } else {
                        dw[0][0][i] = __builtin_fmaf(ga[i], va[i], dw[0][0][i]);
                        dw[0][1][i] = __builtin_fmaf(gb[i], vb[i], dw[0][1][i]);
                    }
                    ga[i] *= w[0][i];
                    gb[i] *= w[1][i];
                    dot = __builtin_fmaf(ga[i], va[i], __builtin_fmaf(gb[i], vb[i], dot));
                }
                const float mean = group_sum(dot, lg) * invD;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    va[i] = r * __builtin_fmaf(-va[i], mean, ga[i]);
                    vb[i] = r * __builtin_fmaf(-vb[i], mean, gb[i]);
                }
            }
            const int64_t yo = b * yr.sb + t * yr.st + head * yr.sh;
            store_run<F32, PAIR>(yr.p, yo + m.off[0], na, va);
            store_run<F32, PAIR>(yr.p, yo + m.off[1], nb, vb);
        }
    }
    if constexpr (BWD) {
        // the workgroup's sums: over a wave's head groups, then over its waves
        __syncthreads();
        float *const red = lds;   // [wave][side][D]
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int run = 0; run < 2; ++run)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float v = dw[s][run][i];
                    for (int k = lph; k < 64; k <<= 1) v += __shfl_xor(v, k, 64);
                    if (hg == 0 && i < m.n[run]) red[(wave * 2 + s) * a.D + m.off[run] + i] = v;
                }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * a.D; i += blockDim.x) {
            float v = 0.0f;
            for (int k = 0; k < waves; ++k) v += red[k * 2 * a.D + i];
            a.partial[(int64_t)blockIdx.x * 2 * a.D + i] = v;
        }
    }
}

// dw[side][d] = the sum of `rows` partial rows, in fp64 and in a fixed order:
// a workgroup takes 16 columns, its 16 thread rows every 16th partial row.
__global__ __launch_bounds__(256) void weight_grad_kernel(const float *__restrict__ partial,
                                                          int rows, int D, float *dw0, float *dw1)
{
    __shared__ double sum[16][16];
    const int c = threadIdx.x & 15, k = threadIdx.x >> 4;
    const int col = blockIdx.x * 16 + c;      // 2 D is a multiple of 16
    double v = 0.0;
    for (int i = k; i < rows; i += 16) v += (double)partial[(int64_t)i * 2 * D + col];
    sum[k][c] = v;
    __syncthreads();
    if (k != 0) return;
    for (int i = 1; i < 16; ++i) v += sum[i][c];
    float *const dst = col < D ? dw0 : dw1;
    if (dst) dst[col < D ? col : col - D] = (float)v;
}

__global__ __launch_bounds__(256) void rope_tables_kernel(RopeDims dims, int axes, double theta,
                                                          bool whole, int half, double *freq,
                                                          int32_t *axis)
{
    const int p = blockIdx.x * 256 + threadIdx.x;
    if (p >= half) return;
    int ax = 0, j = p;
    while (ax + 1 < axes && j >= dims.d[ax] / 2) j -= dims.d[ax++] / 2;
    const double e = whole ? (double)p / half : 2.0 * j / dims.d[ax];
    freq[p] = pow(theta, -e);
    axis[p] = ax;
}

template <bool F32, NormRopeMode MODE>
void launch_pairing(const NormRope &a, int lg, unsigned grid, unsigned threads, size_t lds,
                    hipStream_t stream)
{
    if (!a.half)
        hipLaunchKernelGGL((norm_rope_kernel<F32, MODE, kInterleaved>), dim3(grid), dim3(threads),
                           lds, stream, a, lg);
    else if (a.R % 16 == 0)
        hipLaunchKernelGGL((norm_rope_kernel<F32, MODE, kHalf8>), dim3(grid), dim3(threads), lds,
                           stream, a, lg);
    else
        hipLaunchKernelGGL((norm_rope_kernel<F32, MODE, kHalf4>), dim3(grid), dim3(threads), lds,
                           stream, a, lg);
}

} // namespace

int64_t norm_rope_partial_rows(int64_t tokens) { return std::min<int64_t>(tokens, 1024); }

hipError_t launch_norm_rope(NormRopeMode mode, const NormRope &a, hipStream_t stream)
{
    const int64_t tokens = (int64_t)a.B * a.T;
    const bool bwd = mode == NormRopeMode::BACKWARD;
    const int64_t grid = bwd ? norm_rope_partial_rows(tokens) : std::min<int64_t>(tokens, 8192);
    // the sum of the partial rows (none without tokens: zeros)
    auto weight_grads = [&] {
        hipLaunchKernelGGL(weight_grad_kernel, dim3(2 * a.D / 16), dim3(256), 0, stream, a.partial,
                           (int)grid, a.D, a.dw[0], a.heads[1] ? a.dw[1] : nullptr);
    };
    if (tokens == 0) {
        if (bwd) weight_grads();
        return bwd ? hipGetLastError() : hipSuccess;
    }
    // lanes of a head: 16 channels each, half-split pairs and the channels
    // that pass unchanged in lanes of their own
    const int half = a.R / 2;
    const int lanes = a.half ? (half + 7) / 8 + (a.D - a.R + 15) / 16 : (a.D + 15) / 16;
    int lg = 0;
    while ((1 << lg) < lanes) ++lg;
    const int hpw = 64 >> lg;
    const int units = (a.heads[0] + hpw - 1) / hpw + (a.heads[1] + hpw - 1) / hpw;
    const int waves = std::min(units, bwd && a.D > 256 ? 8 : 16);
    size_t lds = (size_t)2 * 8 * (1 << lg) * sizeof(float2);
    if (bwd) lds = std::max(lds, (size_t)waves * 2 * a.D * sizeof(float));
    const unsigned threads = 64 * waves;
    switch (mode) {
    case NormRopeMode::ROPE:
        a.f32 ? launch_pairing<true, NormRopeMode::ROPE>(a, lg, grid, threads, lds, stream)
              : launch_pairing<false, NormRopeMode::ROPE>(a, lg, grid, threads, lds, stream);
        break;
    case NormRopeMode::NORM:
        a.f32 ? launch_pairing<true, NormRopeMode::NORM>(a, lg, grid, threads, lds, stream)
              : launch_pairing<false, NormRopeMode::NORM>(a, lg, grid, threads, lds, stream);
        break;
    case NormRopeMode::BACKWARD:
        a.f32 ? launch_pairing<true, NormRopeMode::BACKWARD>(a, lg, grid, threads, lds, stream)
              : launch_pairing<false, NormRopeMode::BACKWARD>(a, lg, grid, threads, lds, stream);
        weight_grads();
        break;
    }
    return hipGetLastError();
}

hipError_t launch_rope_tables(RopeDims dims, int axes, double theta, bool whole, double *freq,
                              int32_t *axis, hipStream_t stream)
{
    int half = 0;
    for (int i = 0; i < axes; ++i) half += dims.d[i] / 2;
    hipLaunchKernelGGL(rope_tables_kernel, dim3((half + 255) / 256), dim3(256), 0, stream, dims,
                       axes, theta, whole, half, freq, axis);
    return hipGetLastError();
}

} // namespace convrot
