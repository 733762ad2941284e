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
// A lane holds 8 channels of a head, two runs of 4, so that a rotation never
// leaves the lane: for half-split pairs the second run holds the first's partners.
// Neighbouring lanes hold neighbouring runs, so loads and stores cover whole cache
// lines.  A head is LPH lanes (a power of two), a wave 64 / LPH heads ("unit"), and
// the norm's sum runs over the LPH lanes with DPP.  (16 channels a lane left the
// backward pass three waves per SIMD, 576 us for 84 heads of 38656 tokens, or
// spilled registers.)
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

enum Pairing { kInterleaved = 0, kHalf = 1 };

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

// The channels of one lane: two runs of 4, starting at off[0] and off[1], present
// if on[0], on[1]; the pairs of either run start at p[0], p[1] (2 each when
// interleaved; half-split, the 4 pairs between the runs), and the first rot[0], rot[1]
// of them are rotated.
struct LaneMap {
    int off[2], p[2], rot[2];
    bool on[2];
};

template <bool F32, int PAIR>
__device__ __forceinline__ LaneMap lane_map(int c, int D, int R)
{
    LaneMap m;
    const int half = R >> 1;
    if (PAIR == kInterleaved) {
        // bf16: one run of 8 (16 bytes); fp32: one run of 4 in either half of the head
        m.off[0] = F32 ? 4 * c : 8 * c;
        m.off[1] = F32 ? D / 2 + 4 * c : 8 * c + 4;
        m.on[0] = m.on[1] = 8 * c < D;
        m.p[0] = m.off[0] >> 1;
        m.p[1] = m.on[0] ? m.off[1] >> 1 : m.p[0];
        m.rot[0] = min(max(half - m.p[0], 0), 2);
        m.rot[1] = min(max(half - m.p[1], 0), 2);
    } else {
        const int lanes = half >> 2;           // lanes that rotate
        const bool turns = c < lanes;
        m.off[0] = turns ? 4 * c : R + 8 * (c - lanes);
        m.off[1] = turns ? half + 4 * c : m.off[0] + 4;
        m.on[0] = m.on[1] = m.off[0] < D;
        m.p[0] = m.p[1] = 4 * c;
        m.rot[0] = m.rot[1] = turns ? 4 : 0;
    }
    return m;
}

// A lane's 8 channels as loaded, zeros where it has none.
template <bool F32> struct Raw {
    uint4 u[F32 ? 2 : 1];
};

template <bool F32, int PAIR>
__device__ __forceinline__ Raw<F32> load_raw(const void *base, int64_t at, const LaneMap &m,
                                             bool live)
{
    Raw<F32> r;
    r.u[0] = make_uint4(0, 0, 0, 0);
    if constexpr (F32) r.u[1] = r.u[0];
    if (!live || !m.on[0]) return r;
    if constexpr (F32) {
        const float *p = static_cast<const float *>(base) + at;
        r.u[0] = *reinterpret_cast<const uint4 *>(p + m.off[0]);
        r.u[1] = *reinterpret_cast<const uint4 *>(p + m.off[1]);
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(base) + at;
        if constexpr (PAIR == kInterleaved) {
            r.u[0] = *reinterpret_cast<const uint4 *>(p + m.off[0]);
        } else {
            const uint2 a = *reinterpret_cast<const uint2 *>(p + m.off[0]);
            const uint2 b = *reinterpret_cast<const uint2 *>(p + m.off[1]);
            r.u[0] = make_uint4(a.x, a.y, b.x, b.y);
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

// Outputs are written past the caches that hold the inputs still to come (nt
// stores): 300 against 309 us for 84 heads of 38656 tokens, 20.2 against 21.7 us for
// 2381 tokens.  (nt loads too: 295 us, but 24.9 us.)
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <bool F32, int PAIR>
__device__ __forceinline__ void store(void *base, int64_t at, const LaneMap &m, bool live,
                                      const float (&v)[8])
{
    if (!live || !m.on[0]) return;
    if constexpr (F32) {
        float *p = static_cast<float *>(base) + at;
        __builtin_nontemporal_store((f32x4){v[0], v[1], v[2], v[3]},
                                    reinterpret_cast<f32x4 *>(p + m.off[0]));
        __builtin_nontemporal_store((f32x4){v[4], v[5], v[6], v[7]},
                                    reinterpret_cast<f32x4 *>(p + m.off[1]));
    } else {
        uint16_t *p = static_cast<uint16_t *>(base) + at;
        const u32x2 a = {cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
        const u32x2 b = {cvt_pk_bf16(v[4], v[5]), cvt_pk_bf16(v[6], v[7])};
        if constexpr (PAIR == kInterleaved) {
            __builtin_nontemporal_store((u32x4){a.x, a.y, b.x, b.y},
                                        reinterpret_cast<u32x4 *>(p + m.off[0]));
        } else {
            __builtin_nontemporal_store(a, reinterpret_cast<u32x2 *>(p + m.off[0]));
            __builtin_nontemporal_store(b, reinterpret_cast<u32x2 *>(p + m.off[1]));
        }
    }
}

// The lane's four pairs turned by (cs, sn); those not rotated pass unchanged.
template <int PAIR>
__device__ __forceinline__ void rotate(float (&v)[8], const float (&cs)[4], const float (&sn)[4],
                                       const LaneMap &m)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float &a = v[PAIR == kInterleaved ? 2 * i : i];
        float &b = v[PAIR == kInterleaved ? 2 * i + 1 : i + 4];
        const bool turn = PAIR == kInterleaved ? i % 2 < m.rot[i / 2] : i < m.rot[0];
        const float x = __builtin_fmaf(a, cs[i], -(b * sn[i]));
        const float y = __builtin_fmaf(b, cs[i], a * sn[i]);
        a = turn ? x : a;
        b = turn ? y : b;
    }
}

// A token's positions as loaded (int32 or fp32), `axes` of them.
struct Positions {
    uint32_t v[4];
};

__device__ __forceinline__ Positions load_positions(const NormRope &a, int64_t at)
{
    Positions p = {};
    const uint32_t *const src = static_cast<const uint32_t *>(a.pos) + at;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < a.axes) p.v[i] = src[i];
    return p;
}

// The frequency (in revolutions per position unit) and axis of pair p.
__device__ __forceinline__ void load_pair(const NormRope &a, int p, double &f, int &ax)
{
    f = a.freq[p] * 0.15915494309189535;
    ax = min(max(a.axis[p], 0), a.axes - 1);
}

// cos and sin of the token's pairs into this wave's table; entries from R/2 up
// to npad are never used in a rotation but are read.  (f, ax): pair `lane`.
__device__ __forceinline__ void fill_table(const NormRope &a, const Positions &ps, double f, int ax,
                                           float2 *tab, int npad, int lane)
{
    const int half = a.R >> 1;
    double pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        pos[i] = a.pos_f32 ? (double)__uint_as_float(ps.v[i]) : (double)(int)ps.v[i];
    for (int p = lane; p < npad; p += 64) {
        float s = 0.0f, c = 1.0f;
        if (p < half) {
            if (p >= 64) load_pair(a, p, f, ax);
            const double x = ax == 0 ? pos[0] : ax == 1 ? pos[1] : ax == 2 ? pos[2] : pos[3];
            double rev = x * f;
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
// units w, w + wq, ..., the others on the keys'; `slots` tokens at a time, which
// are db batches and dt tokens.
struct Shape {
    int lg, wq, wk, slots, db, dt;
};

template <bool F32, NormRopeMode MODE, int PAIR>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormRope a, Shape sh)
{
    constexpr bool NORM = MODE != NormRopeMode::ROPE;
    constexpr bool BWD = MODE == NormRopeMode::BACKWARD;
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const int lg = sh.lg, lph = 1 << lg, hpw = 64 >> lg, npad = 4 * lph;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float2 *const tab = reinterpret_cast<float2 *>(lds) + wave * npad;
    const LaneMap m = lane_map<F32, PAIR>(lane & (lph - 1), a.D, a.R);
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

    float wt[8];
    if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < 8; ++i) wt[i] = 1.0f;
        if (wp) {
            Raw<true> r = {};
            if (m.on[0]) {
                r.u[0] = *reinterpret_cast<const uint4 *>(wp + m.off[0]);
                r.u[1] = *reinterpret_cast<const uint4 *>(wp + m.off[1]);
            }
            widen<true>(r, wt);
        }
    }
    float dw[8] = {};                    // backward: sums of g' x r

    uint32_t tok = slot < sh.slots ? slot : tokens;
    int b = (int)(tok / (uint32_t)a.T), t = (int)tok - b * a.T;
    int64_t x0 = 0, y0 = 0, g0 = 0;
    Raw<F32> rx, rg;
    auto load = [&](int u) {
        const int head = u * hpw + hg;
        rx = load_raw<F32, PAIR>(xr.p, x0 + head * xr.sh, m, head < heads);
        if constexpr (BWD) rg = load_raw<F32, PAIR>(gr.p, g0 + head * gr.sh, m, head < heads);
    };
    auto load_first = [&] {
        x0 = b * xr.sb + t * xr.st;
        y0 = b * yr.sb + t * yr.st;
        g0 = b * gr.sb + t * gr.st;
        load(first);
    };
    // Loads return in order, so a token's positions are requested before its rows and
    // the frequency of a lane's pair once a wave: the table is then evaluated while
    // the rows are on their way (8 + 4 heads of 36135 tokens, backward: 76 us, 105 us
    // with rows, positions and frequencies requested in this order for every token).
    // Only a forward wave's first token has its rows first: with many heads it is its
    // only one (84 heads of 38656 tokens: 313 us, 316 us).
    double f = 0.0;
    int ax = 0;
    Positions ps = {};
    auto load_token = [&] {
        ps = load_positions(a, b * a.pos_sb + (int64_t)t * a.axes);
        __builtin_amdgcn_sched_barrier(0);
        load_first();
    };
    if (tok < tokens) {
        if constexpr (!BWD) {
            load_first();
            __builtin_amdgcn_sched_barrier(0);
            ps = load_positions(a, b * a.pos_sb + (int64_t)t * a.axes);
        }
        if (lane < a.R >> 1) load_pair(a, lane, f, ax);
    }
    while (tok < tokens) {
        if constexpr (BWD) load_token();
        fill_table(a, ps, f, ax, tab, npad, lane);
        float cs[4], sn[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = tab[PAIR == kInterleaved ? m.p[i / 2] + i % 2 : m.p[0] + i];
            cs[i] = v.x;
            sn[i] = v.y;
        }
        for (int u = first; u < units; u += step) {
            const int head = u * hpw + hg;
            float v[8], d[8];
            widen(rx, v);
            if constexpr (BWD) widen(rg, d);
            if (u + step < units) load(u + step);
            float r = 1.0f;
            if constexpr (NORM) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(v[i], v[i], ss);
                r = rsqrtf(__builtin_fmaf(group_sum(ss, lg), invD, a.eps));
            }
            if constexpr (!BWD) {
                if constexpr (NORM) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = v[i] * r * wt[i];
                }
                rotate<PAIR>(v, cs, sn, m);
            } else {
                rotate<PAIR>(d, cs, sn, m);
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] *= r;
                    dw[i] = __builtin_fmaf(d[i], v[i], dw[i]);
                    d[i] *= wt[i];
                    dot = __builtin_fmaf(d[i], v[i], dot);
                }
                const float mean = group_sum(dot, lg) * invD;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = r * __builtin_fmaf(-v[i], mean, d[i]);
            }
            store<F32, PAIR>(yr.p, y0 + head * yr.sh, m, head < heads, v);
        }
        tok += sh.slots;
        b += sh.db;
        t += sh.dt;
        if (t >= a.T) t -= a.T, ++b;
        if constexpr (!BWD) {
            if (tok < tokens) load_token();
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
            float s = dw[i];
            for (int k = lph; k < 64; k <<= 1) s += __shfl_xor(s, k, 64);
            if (hg == 0 && m.on[0]) red[(wave * 2 + side) * a.D + m.off[i / 4] + i % 4] = s;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * a.D; i += 256) {
            float s = 0.0f;
            for (int k = 0; k < 4; ++k) s += red[k * 2 * a.D + i];
            a.partial[(int64_t)blockIdx.x * 2 * a.D + i] = s;
        }
    }
}

// dw[side][d] = the sum of `rows` partial rows, in fp64 and in a fixed order:
// a workgroup takes 16 columns, its 64 thread rows every 64th partial row, four
// loads at a time; then halves are joined in LDS.
__global__ __launch_bounds__(1024) void weight_grad_kernel(const float *__restrict__ partial,
                                                           int rows, int D, float *dw0,
                                                           float *dw1)
{
    __shared__ double sum[64][16];
    const int c = threadIdx.x & 15, k = threadIdx.x >> 4;
    const int col = blockIdx.x * 16 + c;      // 2 D is a multiple of 16
    const float *const p = partial + col;
    double v = 0.0;
    for (int i = k; i < rows; i += 256) {
        float x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            x[u] = i + 64 * u < rows ? p[(int64_t)(i + 64 * u) * 2 * D] : 0.0f;
        v += ((double)x[0] + (double)x[1]) + ((double)x[2] + (double)x[3]);
    }
    sum[k][c] = v;
    for (int h = 32; h > 0; h >>= 1) {
        __syncthreads();
        if (k < h) sum[k][c] += sum[k + h][c];
    }
    float *const dst = col < D ? dw0 : dw1;
    if (k == 0 && dst) dst[col < D ? col : col - D] = (float)sum[0][c];
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
    else
        hipLaunchKernelGGL((norm_rope_kernel<F32, MODE, kHalf>), dim3(grid), dim3(256), lds,
                           stream, a, sh);
}

} // namespace

// Waves of a launch when tokens are few (each then takes fewer units), and at
// most of a backward launch, whose workgroups each write a row of partial sums.
constexpr int64_t kWaves = 8192, kBackwardWaves = 4096;
constexpr int kMaxSideWaves = 32;
constexpr int64_t kMaxSlots = 1 << 22;
constexpr int kFewUnits = 8;
constexpr int64_t kFewUnitWaves = 16384;

int64_t norm_rope_partial_rows(int64_t tokens)
{
    return std::min<int64_t>((tokens * 2 * kMaxSideWaves + 3) / 4, kBackwardWaves / 4);
}

hipError_t launch_norm_rope(NormRopeMode mode, const NormRope &a, hipStream_t stream)
{
    const int64_t tokens = (int64_t)a.B * a.T;
    const bool bwd = mode == NormRopeMode::BACKWARD;
    Shape sh = {};
    while ((8 << sh.lg) < a.D) ++sh.lg;      // 8 channels a lane
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
        // A wave of few units spends more on its frequencies than on its rows, so it
        // takes several tokens (2 + 2 units, 38274 tokens: 61.7 us, 70 us with a token a
        // wave); one of many is better off with one (11 + 11 units, 38656 tokens:
        // 317 us, 328 us with 16384 waves).
        const int64_t most = bwd ? kBackwardWaves / W
                             : units0 + units1 <= kFewUnits ? kFewUnitWaves / W : kMaxSlots;
        sh.slots = (int)std::min<int64_t>(tokens, most);
        sh.db = sh.slots / a.T;
        sh.dt = sh.slots % a.T;
        grid = ((int64_t)sh.slots * W + 3) / 4;
        size_t lds = (size_t)4 * 4 * (1 << sh.lg) * sizeof(float2);
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
        hipLaunchKernelGGL(weight_grad_kernel, dim3(2 * a.D / 16), dim3(1024), 0, stream, a.partial,
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
