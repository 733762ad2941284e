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
// A lane holds 16 channels of a head, two runs of 8: adjacent ones when pairs
// are interleaved, 8 channels and their 8 partners for the half-split pairs, so
// that a rotation never leaves the lane.  A head is LPH lanes (a power of two), a
// wave 64 / LPH heads ("unit"), and the norm's sum runs over the LPH lanes with DPP.
//
// A wave takes units of the queries or of the keys of one token (all of them
// when tokens are many).  It evaluates the token's R/2 cosines and sines once,
// one pair per lane, and hands them round through its own piece of LDS, so waves
// never wait for each other; the first rows are on their way meanwhile and each
// unit's rows are requested before the unit before is finished.  (One workgroup
// per token, sharing one table behind a barrier, left the loads of a token in
// line behind its table: 595 us for 84 heads of 38656 tokens.)
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

// A run of n (0, 4 or 8) channels as it was loaded; zeros beyond n.  Half-split
// pairs with R/2 an odd multiple of 4 (kHalf4) start runs 8 bytes off, so bf16 runs
// move as two 8-byte halves there.
template <bool F32> struct Raw {
    uint4 u[F32 ? 2 : 1];
};

template <bool F32, int PAIR>
__device__ __forceinline__ Raw<F32> load_raw(const void *base, int64_t off, int n)
{
    Raw<F32> r;
    r.u[0] = make_uint4(0, 0, 0, 0);
    if constexpr (F32) {
        r.u[1] = r.u[0];
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + off);
        if (n > 0) r.u[0] = p[0];
        if (n > 4) r.u[1] = p[1];
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(base) + off;
        if constexpr (PAIR == kHalf4) {
            if (n > 0) {
                const uint2 a = *reinterpret_cast<const uint2 *>(p);
                r.u[0].x = a.x; r.u[0].y = a.y;
            }
            if (n > 4) {
                const uint2 b = *reinterpret_cast<const uint2 *>(p + 4);
                r.u[0].z = b.x; r.u[0].w = b.y;
            }
        } else {
            if (n > 0) r.u[0] = *reinterpret_cast<const uint4 *>(p);
        }
    }
    return r;
}

template <bool F32>
__device__ __forceinline__ void widen(const Raw<F32> &r, float (&v)[8])
{
    const uint4 &u = r.u[0];
    if constexpr (F32) {
        const uint4 &w = r.u[1];
        v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
        v[4] = __uint_as_float(w.x); v[5] = __uint_as_float(w.y);
        v[6] = __uint_as_float(w.z); v[7] = __uint_as_float(w.w);
    } else {
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

// cos and sin of the token's pairs into this wave's table; entries from R/2 up
// to npad are never used in a rotation but are read.
__device__ __forceinline__ void fill_table(const NormRope &a, int64_t pos_at, float2 *tab,
                                           int npad, int lane)
{
    const int half = a.R >> 1;
    double pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t at = pos_at + min(i, a.axes - 1);
        pos[i] = a.pos_f32 ? (double)static_cast<const float *>(a.pos)[at]
                           : (double)static_cast<const int32_t *>(a.pos)[at];
    }
    for (int p = lane; p < npad; p += 64) {
        float s = 0.0f, c = 1.0f;
        if (p < half) {
            const int ax = min(max(a.axis[p], 0), a.axes - 1);
            const double x = ax == 0 ? pos[0] : ax == 1 ? pos[1] : ax == 2 ? pos[2] : pos[3];
            double rev = x * a.freq[p] * 0.15915494309189535;
            rev -= rint(rev);
            sincospif((float)(2.0 * rev), &s, &c);
            if (a.inverse) s = -s;
        }
        tab[p] = make_float2(c, s);
    }
    // the table is written and read by this wave only: LDS serves it in order,
    // the compiler must keep that order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A launch's shape: W = wq + wk waves per token, wave w < wq on the queries'
// units w, w + wq, ..., the others on the keys'; `slots` tokens at a time.
struct Shape {
    int lg, wq, wk, slots;
};

template <bool F32, NormRopeMode MODE, int PAIR>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormRope a, Shape sh)
{
    constexpr bool NORM = MODE != NormRopeMode::ROPE;
    constexpr bool BWD = MODE == NormRopeMode::BACKWARD;
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const int lg = sh.lg, lph = 1 << lg, hpw = 64 >> lg, npad = 8 * lph;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float2 *const tab = reinterpret_cast<float2 *>(lds) + wave * npad;
    const LaneMap m = lane_map<PAIR>(lane & (lph - 1), a.D, a.R);
    const int hg = lane >> lg;
    const uint32_t tokens = (uint32_t)(a.B * a.T);
    const float invD = 1.0f / (float)a.D;

    const int W = sh.wq + sh.wk;
    const int gw = blockIdx.x * 4 + wave;
    const int slot = gw / W, w = gw - slot * W;
    const int side = w >= sh.wq ? 1 : 0;
    const int first = side ? w - sh.wq : w, step = side ? sh.wk : sh.wq;
    const int heads = side ? a.heads[1] : a.heads[0];
    const HeadRows xr = side ? a.x[1] : a.x[0], yr = side ? a.out[1] : a.out[0];
    const HeadRows gr = side ? a.g[1] : a.g[0];
    const float *const wp = side ? a.w[1] : a.w[0];
    const int units = (heads + hpw - 1) >> (6 - lg);

    float wa[8], wb[8];
    if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < 8; ++i) wa[i] = wb[i] = 1.0f;
        if (wp) {
            widen<true>(load_raw<true, PAIR>(wp, m.off[0], m.n[0]), wa);
            widen<true>(load_raw<true, PAIR>(wp, m.off[1], m.n[1]), wb);
        }
    }
    float dwa[8] = {}, dwb[8] = {};      // backward: sums of g' x r

    for (uint32_t tok = slot < sh.slots ? slot : tokens; tok < tokens; tok += sh.slots) {
        const int b = (int)(tok / (uint32_t)a.T), t = (int)tok - b * a.T;
        const int64_t x0 = b * xr.sb + t * xr.st, y0 = b * yr.sb + t * yr.st;
        const int64_t g0 = b * gr.sb + t * gr.st;
        Raw<F32> xa, xb, ga, gb;
        auto load = [&](int u, Raw<F32> &pa, Raw<F32> &pb, const HeadRows &v, int64_t at) {
            const int head = u * hpw + hg;
            const bool live = head < heads;
            at += head * v.sh;
            pa = load_raw<F32, PAIR>(v.p, at + m.off[0], live ? m.n[0] : 0);
            pb = load_raw<F32, PAIR>(v.p, at + m.off[1], live ? m.n[1] : 0);
        };
        load(first, xa, xb, xr, x0);
        if constexpr (BWD) load(first, ga, gb, gr, g0);
        fill_table(a, b * a.pos_sb + (int64_t)t * a.axes, tab, npad, lane);
        float cs[8], sn[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = tab[m.p0 + i];
            cs[i] = v.x;
            sn[i] = v.y;
        }
        for (int u = first; u < units; u += step) {
            const int head = u * hpw + hg;
            const bool live = head < heads;
            float va[8], vb[8], da[8], db[8];
            widen(xa, va);
            widen(xb, vb);
            if constexpr (BWD) {
                widen(ga, da);
                widen(gb, db);
            }
            if (u + step < units) {
                load(u + step, xa, xb, xr, x0);
                if constexpr (BWD) load(u + step, ga, gb, gr, g0);
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
                        va[i] = va[i] * r * wa[i];
                        vb[i] = vb[i] * r * wb[i];
                    }
                }
                rotate<PAIR>(va, vb, cs, sn, m.nrot);
            } else {
                rotate<PAIR>(da, db, cs, sn, m.nrot);
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    va[i] *= r;
                    vb[i] *= r;
                    dwa[i] = __builtin_fmaf(da[i], va[i], dwa[i]);
                    dwb[i] = __builtin_fmaf(db[i], vb[i], dwb[i]);
                    da[i] *= wa[i];
                    db[i] *= wb[i];
                    dot = __builtin_fmaf(da[i], va[i], __builtin_fmaf(db[i], vb[i], dot));
                }
                const float mean = group_sum(dot, lg) * invD;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    va[i] = r * __builtin_fmaf(-va[i], mean, da[i]);
                    vb[i] = r * __builtin_fmaf(-vb[i], mean, db[i]);
                }
            }
            const int64_t at = y0 + head * yr.sh;
            store_run<F32, PAIR>(yr.p, at + m.off[0], live ? m.n[0] : 0, va);
            store_run<F32, PAIR>(yr.p, at + m.off[1], live ? m.n[1] : 0, vb);
        }
    }
    if constexpr (BWD) {
        // the workgroup's sums: over a wave's head groups, then over its waves
        // of either side (a wave without a token adds zeros)
        __syncthreads();
        float *const red = lds;   // [wave][side][D]
        for (int i = lane; i < a.D; i += 64) red[(wave * 2 + (side ^ 1)) * a.D + i] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float va = dwa[i], vb = dwb[i];
            for (int k = lph; k < 64; k <<= 1) {
                va += __shfl_xor(va, k, 64);
                vb += __shfl_xor(vb, k, 64);
            }
            float *const dst = red + (wave * 2 + side) * a.D;
            if (hg == 0 && i < m.n[0]) dst[m.off[0] + i] = va;
            if (hg == 0 && i < m.n[1]) dst[m.off[1] + i] = vb;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * a.D; i += 256) {
            float v = 0.0f;
            for (int k = 0; k < 4; ++k) v += red[k * 2 * a.D + i];
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
void launch_pairing(const NormRope &a, const Shape &sh, unsigned grid, size_t lds,
                    hipStream_t stream)
{
    if (!a.half)
        hipLaunchKernelGGL((norm_rope_kernel<F32, MODE, kInterleaved>), dim3(grid), dim3(256), lds,
                           stream, a, sh);
    else if (a.R % 16 == 0)
        hipLaunchKernelGGL((norm_rope_kernel<F32, MODE, kHalf8>), dim3(grid), dim3(256), lds,
                           stream, a, sh);
    else
        hipLaunchKernelGGL((norm_rope_kernel<F32, MODE, kHalf4>), dim3(grid), dim3(256), lds,
                           stream, a, sh);
}

} // namespace

// Waves of a launch when tokens are few (each then takes fewer units), and at
// most of a backward launch, whose workgroups each write a row of partial sums.
constexpr int64_t kWaves = 8192, kBackwardWaves = 4096;
constexpr int kMaxSideWaves = 32;
constexpr int64_t kMaxSlots = 1 << 22;

int64_t norm_rope_partial_rows(int64_t tokens)
{
    return std::min<int64_t>((tokens * 2 * kMaxSideWaves + 3) / 4, kBackwardWaves / 4);
}

hipError_t launch_norm_rope(NormRopeMode mode, const NormRope &a, hipStream_t stream)
{
    const int64_t tokens = (int64_t)a.B * a.T;
    const bool bwd = mode == NormRopeMode::BACKWARD;
    // lanes of a head: 16 channels each, half-split pairs and the channels
    // that pass unchanged in lanes of their own
    const int half = a.R / 2;
    const int lanes = a.half ? (half + 7) / 8 + (a.D - a.R + 15) / 16 : (a.D + 15) / 16;
    Shape sh = {};
    while ((1 << sh.lg) < lanes) ++sh.lg;
    const int hpw = 64 >> sh.lg;
    int64_t grid = 0;
    if (tokens > 0) {
        const int units0 = (a.heads[0] + hpw - 1) / hpw, units1 = (a.heads[1] + hpw - 1) / hpw;
        // waves per side: its share of kWaves, at least one unit each
        auto waves = [&](int units) {
            const int64_t w = (kWaves * units / (units0 + units1) + tokens - 1) / tokens;
            return (int)std::max<int64_t>(std::min<int64_t>({w, units, kMaxSideWaves}),
                                          units > 0 ? 1 : 0);
        };
        sh.wq = waves(units0);
        sh.wk = waves(units1);
        const int W = sh.wq + sh.wk;
        sh.slots = (int)(bwd ? std::min<int64_t>(tokens, kBackwardWaves / W)
                              : std::min<int64_t>(tokens, kMaxSlots));
        grid = ((int64_t)sh.slots * W + 3) / 4;
        size_t lds = (size_t)4 * 8 * (1 << sh.lg) * sizeof(float2);
        if (bwd) lds = std::max(lds, (size_t)4 * 2 * a.D * sizeof(float));
        switch (mode) {
        case NormRopeMode::ROPE:
            a.f32 ? launch_pairing<true, NormRopeMode::ROPE>(a, sh, grid, lds, stream)
                  : launch_pairing<false, NormRopeMode::ROPE>(a, sh, grid, lds, stream);
            break;
        case NormRopeMode::NORM:
            a.f32 ? launch_pairing<true, NormRopeMode::NORM>(a, sh, grid, lds, stream)
                  : launch_pairing<false, NormRopeMode::NORM>(a, sh, grid, lds, stream);
            break;
        case NormRopeMode::BACKWARD:
            a.f32 ? launch_pairing<true, NormRopeMode::BACKWARD>(a, sh, grid, lds, stream)
                  : launch_pairing<false, NormRopeMode::BACKWARD>(a, sh, grid, lds, stream);
            break;
        }
    }
    // the sum of the partial rows (none without tokens: zeros)
    if (bwd)
        hipLaunchKernelGGL(weight_grad_kernel, dim3(2 * a.D / 16), dim3(256), 0, stream, a.partial,
                           (int)grid, a.D, a.dw[0], a.heads[1] ? a.dw[1] : nullptr);
    return bwd || tokens > 0 ? hipGetLastError() : hipSuccess;
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
