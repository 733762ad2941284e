// A mixture-of-experts layer for a few tokens (gfx950).
//
//   logits = x router^T;  the top_k experts of each token by logit (with a bias: by
//   score + bias), ties to the lowest index;  weights = scores (softmax or sigmoid),
//   divided by their sum or not, times a factor
//   g_e = silu(G_e x) * (U_e x);   y = sum_e weight_e D_e g_e  (+ the shared experts')
//
// Bound: the codes of the experts that some token chose, read once: few tokens leave
// the matrix cores idle, so activations stay bf16 (8 bits would only cost precision)
// and the e4m3 codes are widened to bf16, which holds them exactly, in registers:
// v_mfma_f32_16x16x32_bf16 with 16 outputs as rows and 16 tokens as columns.  A block
// of 128 inputs is summed from zero and joined by an fp32 multiply-add with its scale.
//
// Precision.  The logits are summed in fp64 (v_mfma_f64_16x16x4_f64): the choice of
// experts then does not depend on the order of the sums, a batch or a shape.  g is
// carried as two bf16 parts for bf16 outputs and as three, which hold an fp32 value
// exactly, for F32 outputs.
//
// Kernels: router (partial logits over pieces of K), select (one workgroup: choices,
// and for each chosen expert, a "unit", its tokens), gate_up, down.  For one token
// every wave of gate_up makes the choice itself.
#include "moe.hpp"

#include "fp8_common.hpp"

#include <algorithm>
#include <type_traits>

namespace convrot {
namespace {

typedef double v4d __attribute__((ext_vector_type(4)));
typedef unsigned long long u64;

constexpr int kMaxUnits = kMoeMaxExperts + kMoeMaxShared;

// What select leaves for the experts' kernels.  Rows of g: those of the first unit, in
// the order of its tokens, then those of the second, ...
struct Row {
    int token;
    float weight;
};
struct Units {
    int count, pad;
    int expert[kMaxUnits];
    int base[kMaxUnits];                   // first of the unit's rows
    u64 tokens[kMaxUnits];
};

constexpr int kRouterPieces = 8, kRouterWaves = 8;

struct Layout {
    size_t logits, units, rows, g, partial, bytes;
};

// ------------------------------------------------------------- router ----
// logits[piece][t][e]: a workgroup takes 16 experts, 16 tokens and a piece of K, whose
// runs of 32 inputs its waves share out; they join in LDS in order.  Lane (r, q) holds
// inputs 8 q .. 8 q + 7 of a run of expert r and of token r, one of them per product.
template <bool RF32>
__global__ __launch_bounds__(64 * kRouterWaves) void router_kernel(Moe m,
                                                                   double *__restrict__ logits)
{
    __shared__ double red[kRouterWaves][256];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4, wave = threadIdx.x >> 6;
    const int e0 = blockIdx.x * 16, t0 = blockIdx.z * 16, runs = m.K >> 5;
    const int64_t er = (int64_t)min(e0 + r, m.E - 1) * m.K;
    const uint16_t *const xr = m.x + (int64_t)min(t0 + r, m.T - 1) * m.K;
    v4d acc = (v4d)(0.0);
    for (int i = blockIdx.y * kRouterWaves + wave; i < runs; i += kRouterWaves * gridDim.y) {
        const int k = i * 32 + q * 8;
        const uint4 u = *reinterpret_cast<const uint4 *>(xr + k);
        float wv[8];
        if constexpr (RF32) {
            const float *p = static_cast<const float *>(m.router) + er + k;
            const v4f a = *reinterpret_cast<const v4f *>(p), b = *reinterpret_cast<const v4f *>(p + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) wv[j] = a[j], wv[4 + j] = b[j];
        } else {
            const uint4 w = *reinterpret_cast<const uint4 *>(
                static_cast<const uint16_t *>(m.router) + er + k);
            wv[0] = bf16_lo(w.x); wv[1] = bf16_hi(w.x); wv[2] = bf16_lo(w.y);
            wv[3] = bf16_hi(w.y); wv[4] = bf16_lo(w.z); wv[5] = bf16_hi(w.z);
            wv[6] = bf16_lo(w.w); wv[7] = bf16_hi(w.w);
        }
        const float xv[8] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y),
                             bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w)};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)wv[j], (double)xv[j], acc, 0, 0, 0);
    }
    // register i of lane (r, q): expert 4 i + q, token r
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][(4 * i + q) * 16 + r] = acc[i];
    __syncthreads();
    const int e = threadIdx.x & 15, t = threadIdx.x >> 4;
    if (t < 16 && e0 + e < m.E && t0 + t < m.T) {
        double v = 0.0;
#pragma unroll
        for (int k = 0; k < kRouterWaves; ++k) v += red[k][e * 16 + t];
        logits[((int64_t)blockIdx.y * m.T + t0 + t) * m.E + e0 + e] = v;
    }
}

// ------------------------------------------------------------- choice ----

// Every lane gets the sum of its 16, then the wave's.
#define CR_DPP_I(v, CTRL) __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, true)
__device__ __forceinline__ double wave_sum(double v)
{
    auto add = [&](auto ctrl) {
        constexpr int C = decltype(ctrl)::value;
        const int2 u = __builtin_bit_cast(int2, v);
        v += __builtin_bit_cast(double, make_int2(CR_DPP_I(u.x, C), CR_DPP_I(u.y, C)));
    };
    add(std::integral_constant<int, 0xB1>{});
    add(std::integral_constant<int, 0x4E>{});
    add(std::integral_constant<int, 0x141>{});
    add(std::integral_constant<int, 0x140>{});
    double s = 0.0;
#pragma unroll
    for (int l = 0; l < 64; l += 16) {
        const int2 u = __builtin_bit_cast(int2, v);
        s += __builtin_bit_cast(double, make_int2(__builtin_amdgcn_readlane(u.x, l),
                                                  __builtin_amdgcn_readlane(u.y, l)));
    }
    return s;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = max(v, (uint32_t)CR_DPP_I((int)v, 0xB1));
    v = max(v, (uint32_t)CR_DPP_I((int)v, 0x4E));
    v = max(v, (uint32_t)CR_DPP_I((int)v, 0x141));
    v = max(v, (uint32_t)CR_DPP_I((int)v, 0x140));
    return max(max((uint32_t)__builtin_amdgcn_readlane((int)v, 0),
                   (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
               max((uint32_t)__builtin_amdgcn_readlane((int)v, 32),
                   (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
}
__device__ __forceinline__ u64 wave_max(u64 v)
{
    const uint32_t hi = wave_max((uint32_t)(v >> 32));
    const uint32_t lo = wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (u64)hi << 32 | lo;
}

// Doubles in the order of unsigned numbers; above 0 for every value, NaN as -infinity,
// -0 as +0; and back.
__device__ __forceinline__ u64 order_of(double v)
{
    if (!(v == v)) v = -__builtin_inf();
    const u64 b = __builtin_bit_cast(u64, v + 0.0);
    return b >> 63 ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ double value_of(u64 k)
{
    return __builtin_bit_cast(double, k >> 63 ? k & ~(1ull << 63) : ~k);
}

// The choice of token t by one wave: lane j gets the j-th expert and its weight.  EP
// experts a lane (expert lane + 64 i).  A round takes the wave's largest key and the
// lowest expert that has it.
template <int EP>
__device__ __forceinline__ void choose(const Moe &m, const double *__restrict__ logits, int pieces,
                                       int t, int &id, float &weight)
{
    const int lane = threadIdx.x & 63;
    double p[EP];
    u64 key[EP];
#pragma unroll
    for (int i = 0; i < EP; ++i) p[i] = 0.0;
    for (int c0 = 0; c0 < pieces; c0 += 4) {
        double v[4][EP];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < EP; ++i) {
                const int e = lane + 64 * i;
                v[c][i] = e < m.E && c0 + c < pieces
                              ? logits[((int64_t)(c0 + c) * m.T + t) * m.E + e] : 0.0;
            }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < EP; ++i) p[i] += v[c][i];
    }
    u64 best = 0;
#pragma unroll
    for (int i = 0; i < EP; ++i) {
        key[i] = lane + 64 * i < m.E ? order_of(p[i]) : 0;
        best = key[i] > best ? key[i] : best;
    }
    if (m.sigmoid) {
#pragma unroll
        for (int i = 0; i < EP; ++i) p[i] = 1.0 / (1.0 + exp(-p[i]));
    } else {
        const double top = value_of(wave_max(best));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            p[i] = exp(p[i] - top);
            if (lane + 64 * i < m.E) sum += p[i];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int i = 0; i < EP; ++i) p[i] /= sum;
    }
    if (m.bias) {
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            const int e = lane + 64 * i;
            if (e < m.E) key[i] = order_of(p[i] + (double)m.bias[e]);
        }
    }
    double w = 0.0, total = 0.0;
    id = 0;
    for (int j = 0; j < m.top_k; ++j) {
        best = 0;
#pragma unroll
        for (int i = 0; i < EP; ++i) best = key[i] > best ? key[i] : best;
        best = wave_max(best);
        int e = -1;
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            const u64 hit = __ballot(key[i] == best);
            if (e >= 0 || hit == 0) continue;
            const int l = __builtin_ctzll(hit);
            e = 64 * i + l;
            const int2 u = __builtin_bit_cast(int2, p[i]);
            s = __builtin_bit_cast(double, make_int2(__builtin_amdgcn_readlane(u.x, l),
                                                     __builtin_amdgcn_readlane(u.y, l)));
            if (lane == l) key[i] = 0;
        }
        total += s;
        if (lane == j) id = e, w = s;
    }
    if (m.renormalize) w = total == 0.0 ? 0.0 : w / total;
    weight = (float)(w * m.factor);
}

// The choices of several tokens, a wave for one after another, and the units.
template <int EP>
__global__ __launch_bounds__(1024) void select_kernel(Moe m, const double *__restrict__ logits,
                                                      int pieces, Units *__restrict__ units,
                                                      Row *__restrict__ rows)
{
    __shared__ u64 tokens[kMoeMaxExperts];
    __shared__ int unit_base[kMoeMaxExperts], wave_units[16], wave_rows[16];
    __shared__ int ids[kMoeTokens * kMoeMaxTopK];
    __shared__ float wts[kMoeTokens * kMoeMaxTopK];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int i = threadIdx.x; i < kMoeMaxExperts; i += 1024) tokens[i] = 0;
    __syncthreads();

    for (int t = wave; t < m.T; t += 16) {
        int id;
        float w;
        choose<EP>(m, logits, pieces, t, id, w);
        if (lane < m.top_k) {
            const int i = t * m.top_k + lane;
            ids[i] = id;
            wts[i] = w;
            m.ids[i] = id;
            m.weights[i] = w;
            atomicOr(&tokens[id], 1ull << t);
        }
    }
    __syncthreads();

    // units: the chosen experts in order, their rows one after another
    const int e = threadIdx.x;
    const u64 mine = e < m.E ? tokens[e] : 0;
    const u64 active = __ballot(mine != 0);
    const int before = __popcll(active & ((1ull << lane) - 1));
    int n = __popcll(mine);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(n, o, 64);
        if (lane >= o) n += up;
    }
    if (lane == 63) {
        wave_units[wave] = __popcll(active);
        wave_rows[wave] = n;
    }
    __syncthreads();
    int u = before, base = n - __popcll(mine), count = 0;
    for (int k = 0; k < 16; ++k) {
        if (k < wave) u += wave_units[k], base += wave_rows[k];
        count += wave_units[k];
    }
    if (mine != 0) {
        units->expert[u] = e;
        units->base[u] = base;
        units->tokens[u] = mine;
        unit_base[e] = base;
    }
    const u64 all = m.T == 64 ? ~0ull : (1ull << m.T) - 1;
    const int chosen = m.T * m.top_k;
    if (e < m.S) {
        units->expert[count + e] = m.E + e;
        units->base[count + e] = chosen + e * m.T;
        units->tokens[count + e] = all;
    }
    if (e == 0) units->count = count + m.S;
    __syncthreads();
    for (int i = threadIdx.x; i < chosen; i += 1024) {
        const int t = i / m.top_k, x = ids[i];
        rows[unit_base[x] + __popcll(tokens[x] & ((1ull << t) - 1))] = {t, wts[i]};
    }
    for (int i = threadIdx.x; i < m.S * m.T; i += 1024) rows[chosen + i] = {i % m.T, 1.0f};
}

// ------------------------------------------------------------ experts ----

// One 16 x 128 block of codes as two 16-byte pieces a lane.
struct Block {
    v4i lo, hi;
};
__device__ __forceinline__ Block load_block(const uint8_t *p)
{
    return {*reinterpret_cast<const v4i *>(p), *reinterpret_cast<const v4i *>(p + 1024)};
}

// 16 tokens' inputs of a block of 128: four pieces of 8 a lane.
struct Cols {
    uint4 u[4];
};
__device__ __forceinline__ Cols load_cols(const uint16_t *p, bool on)
{
    Cols c;
#pragma unroll
    for (int i = 0; i < 4; ++i) c.u[i] = make_uint4(0, 0, 0, 0);
    if (on) {
        c.u[0] = *reinterpret_cast<const uint4 *>(p);
        c.u[1] = *reinterpret_cast<const uint4 *>(p + 8);
        c.u[2] = *reinterpret_cast<const uint4 *>(p + 64);
        c.u[3] = *reinterpret_cast<const uint4 *>(p + 72);
    }
    return c;
}

__device__ __forceinline__ v4f block_sum(const Block &a, const Cols &b, v4f s)
{
    s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16_of_codes(a.lo[0], a.lo[1]),
                                                __builtin_bit_cast(v8bf, b.u[0]), s, 0, 0, 0);
    s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16_of_codes(a.lo[2], a.lo[3]),
                                                __builtin_bit_cast(v8bf, b.u[1]), s, 0, 0, 0);
    s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16_of_codes(a.hi[0], a.hi[1]),
                                                __builtin_bit_cast(v8bf, b.u[2]), s, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16_of_codes(a.hi[2], a.hi[3]),
                                                   __builtin_bit_cast(v8bf, b.u[3]), s, 0, 0, 0);
}

// g of one unit: a workgroup takes 16 gate and the same 16 up channels, its waves the
// blocks of K in turn, D at a time.  Columns are the unit's rows, in up to CT tiles of
// 16.  EP > 0: one token, whose choice every wave makes; the first workgroup leaves it
// for the down projection.
template <int CT, int D, int EP>
__global__ __launch_bounds__(256) void gate_up_kernel(Moe m, Units *__restrict__ units,
                                                      Row *__restrict__ rows,
                                                      uint16_t *__restrict__ g, int64_t plane,
                                                      const double *__restrict__ logits,
                                                      int pieces)
{
    extern __shared__ float red[];                 // [wave][2][CT][256]
    const int u = blockIdx.y;
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    int expert, base, n;
    if constexpr (EP > 0) {
        int id;
        float w;
        choose<EP>(m, logits, pieces, 0, id, w);
        if (lane >= m.top_k) id = m.E + lane - m.top_k, w = 1.0f;
        expert = __builtin_amdgcn_readlane(id, u);
        base = u;
        n = 1;
        if (blockIdx.x == 0 && u == 0 && wave == 0 && lane < m.top_k + m.S) {
            units->expert[lane] = id;
            units->base[lane] = lane;
            units->tokens[lane] = 1;
            rows[lane] = {0, w};
            if (lane == 0) units->count = m.top_k + m.S;
            if (lane < m.top_k) m.ids[lane] = id, m.weights[lane] = w;
        }
    } else {
        if (u >= units->count) return;
        expert = units->expert[u];
        base = units->base[u];
        n = __popcll(units->tokens[u]);
    }
    const int nkb = m.K >> 7, fb = blockIdx.x;
    const int in_tile = r * 64 + ((q ^ ((r >> 2) & 3)) << 4);
    const int64_t row_bytes = (int64_t)16 * m.K;
    const uint8_t *const codes = m.gate_up + (int64_t)expert * 2 * m.F * m.K + in_tile;
    const uint8_t *const gate = codes + fb * row_bytes, *const up = gate + (int64_t)m.F * m.K;
    const float *const sg = m.gate_up_scale +
                            ((int64_t)expert * (m.F >> 6) + (fb >> 3)) * nkb;
    const float *const su = sg + (int64_t)(m.F >> 7) * nkb;

    const uint16_t *col[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const bool on = c * 16 + r < n;
        const int t = EP > 0 || !on ? 0 : rows[base + c * 16 + r].token;
        col[c] = m.x + (int64_t)t * m.K + q * 16;
    }
    v4f ag[CT], au[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) ag[c] = au[c] = (v4f)(0.0f);
    for (int k0 = wave; k0 < nkb; k0 += waves * D) {
        Block a[D], b[D];
        Cols x[D];
        float fg[D], fu[D];
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int kb = k0 + d * waves;
            if (kb >= nkb) continue;
            a[d] = load_block(gate + kb * 2048);
            b[d] = load_block(up + kb * 2048);
            x[d] = load_cols(col[0] + kb * 128, r < n);
            fg[d] = sg[kb];
            fu[d] = su[kb];
        }
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int kb = k0 + d * waves;
            if (kb >= nkb) continue;
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                if (c > 0 && c * 16 >= n) continue;
                if (c > 0) x[d] = load_cols(col[c] + kb * 128, c * 16 + r < n);
                const v4f pg = block_sum(a[d], x[d], (v4f)(0.0f));
                const v4f pu = block_sum(b[d], x[d], (v4f)(0.0f));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ag[c][i] = __builtin_fmaf(pg[i], fg[d], ag[c][i]);
                    au[c][i] = __builtin_fmaf(pu[i], fu[d], au[c][i]);
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        if (c > 0 && c * 16 >= n) continue;
        *reinterpret_cast<v4f *>(red + ((wave * 2 + 0) * CT + c) * 256 + lane * 4) = ag[c];
        *reinterpret_cast<v4f *>(red + ((wave * 2 + 1) * CT + c) * 256 + lane * 4) = au[c];
    }
    __syncthreads();
    for (int c = wave; c * 16 < n; c += waves) {
        v4f a = (v4f)(0.0f), b = (v4f)(0.0f);
        for (int k = 0; k < waves; ++k) {
            a += *reinterpret_cast<const v4f *>(red + ((k * 2 + 0) * CT + c) * 256 + lane * 4);
            b += *reinterpret_cast<const v4f *>(red + ((k * 2 + 1) * CT + c) * 256 + lane * 4);
        }
        if (c * 16 + r >= n) continue;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i] / (1.0f + expf(-a[i])) * b[i];
        uint16_t *p = g + (int64_t)(base + c * 16 + r) * m.F + fb * 16 + q * 4;
        // the part that bf16 holds, then what it leaves
        for (int part = 1;; ++part) {
            const uint2 o = make_uint2(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]));
            *reinterpret_cast<uint2 *>(p) = o;
            if (part == (m.y_f32 ? 3 : 2)) break;
            v[0] -= bf16_lo(o.x);
            v[1] -= bf16_hi(o.x);
            v[2] -= bf16_lo(o.y);
            v[3] -= bf16_hi(o.y);
            p += plane;
        }
    }
}

__device__ __forceinline__ void store_y(const Moe &m, float *partial, int64_t o, v4f v)
{
    if (partial)
        *reinterpret_cast<v4f *>(partial + (int64_t)blockIdx.y * m.T * m.K + o) = v;
    else if (m.y_f32)
        *reinterpret_cast<v4f *>(static_cast<float *>(m.y) + o) = v;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(m.y) + o) =
            make_uint2(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]));
}

// y of 16 outputs for up to 16 tokens: a workgroup's waves take (unit, block of F) pairs
// in turn, D at a time, of the units of its part (gridDim.y parts).  Columns are tokens,
// zero where a token did not choose the unit, so that a token's sums over its experts
// stay in one accumulator.  partial (or null): [part][T][K].
template <int WAVES, int D, int PLANES>
__global__ __launch_bounds__(64 * WAVES) void down_kernel(Moe m, const Units *__restrict__ units,
                                                    const Row *__restrict__ rows,
                                                    const uint16_t *__restrict__ g, int64_t plane,
                                                    float *__restrict__ partial)
{
    constexpr int waves = WAVES;
    __shared__ float red[WAVES * 256];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nkb = m.F >> 7, nb = blockIdx.x;
    const int count = units->count;
    const int u0 = count * blockIdx.y / gridDim.y, u1 = count * (blockIdx.y + 1) / gridDim.y;
    const int in_tile = r * 64 + ((q ^ ((r >> 2) & 3)) << 4);

    v4f acc = (v4f)(0.0f);
    const int items = (u1 - u0) * nkb;
    for (int i0 = wave; i0 < items; i0 += waves * D) {
        Block a[D];
        Cols x[D][PLANES];
        float w[D];
        bool on[D];
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int i = i0 + d * waves;
            if (i >= items) continue;
            const int u = u0 + i / nkb, kb = i % nkb;
            const int64_t e = units->expert[u];
            a[d] = load_block(m.down + e * m.K * m.F + (int64_t)nb * 16 * m.F + kb * 2048 +
                              in_tile);
            const float f = m.down_scale[(e * (m.K >> 7) + (nb >> 3)) * nkb + kb];
            const u64 tokens = units->tokens[u];
            on[d] = (tokens >> r) & 1;
            const int row = units->base[u] + __popcll(tokens & ((1ull << r) - 1));
            w[d] = 0.0f;
            if (on[d]) w[d] = rows[row].weight * f;
#pragma unroll
            for (int k = 0; k < PLANES; ++k)
                x[d][k] = load_cols(g + k * plane + (int64_t)row * m.F + kb * 128 + q * 16, on[d]);
        }
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (i0 + d * waves >= items) continue;
            v4f s = (v4f)(0.0f);
#pragma unroll
            for (int k = 0; k < PLANES; ++k) s = block_sum(a[d], x[d][k], s);
            // a token that did not choose the expert takes nothing of it, codes of NaN
            // included
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[k] = on[d] ? __builtin_fmaf(s[k], w[d], acc[k]) : acc[k];
        }
    }
    *reinterpret_cast<v4f *>(red + wave * 256 + lane * 4) = acc;
    __syncthreads();
    if (wave > 0) return;
    v4f v = (v4f)(0.0f);
    for (int k = 0; k < waves; ++k) v += *reinterpret_cast<const v4f *>(red + k * 256 + lane * 4);
    if (r < m.T) store_y(m, partial, (int64_t)r * m.K + nb * 16 + q * 4, v);
}

// The same for more tokens: a wave takes whole units, whose rows are its columns (up to 4
// tiles of 16), and adds each unit's sums, weighted, to its own [T][16] sums in LDS.
template <int PLANES>
__global__ __launch_bounds__(512) void down_many_kernel(Moe m, const Units *__restrict__ units,
                                                        const Row *__restrict__ rows,
                                                        const uint16_t *__restrict__ g,
                                                        int64_t plane,
                                                        float *__restrict__ partial)
{
    constexpr int CT = kMoeTokens / 16, D = 2;
    extern __shared__ float red[];                 // [wave][T][16]
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int nkb = m.F >> 7, nb = blockIdx.x;
    const int count = units->count;
    const int u0 = count * blockIdx.y / gridDim.y, u1 = count * (blockIdx.y + 1) / gridDim.y;
    const int in_tile = r * 64 + ((q ^ ((r >> 2) & 3)) << 4);
    float *const mine = red + wave * m.T * 16;
    for (int i = lane; i < m.T * 4; i += 64)
        *reinterpret_cast<v4f *>(mine + i * 4) = (v4f)(0.0f);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();

    for (int u = u0 + wave; u < u1; u += waves) {
        const int64_t e = units->expert[u];
        const int base = units->base[u], n = __popcll(units->tokens[u]);
        const uint8_t *const codes = m.down + e * m.K * m.F + (int64_t)nb * 16 * m.F + in_tile;
        const float *const sc = m.down_scale + (e * (m.K >> 7) + (nb >> 3)) * nkb;
        v4f acc[CT];
        Row row[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            acc[c] = (v4f)(0.0f);
            row[c] = {0, 0.0f};
            if (c * 16 + r < n) row[c] = rows[base + c * 16 + r];
        }
        const uint16_t *const x0 = g + (int64_t)(base + r) * m.F + q * 16;
        for (int k0 = 0; k0 < nkb; k0 += D) {
            Block a[D];
            Cols x[D][PLANES];
            float f[D];
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int kb = k0 + d;
                if (kb >= nkb) continue;
                a[d] = load_block(codes + kb * 2048);
                f[d] = sc[kb];
#pragma unroll
                for (int k = 0; k < PLANES; ++k)
                    x[d][k] = load_cols(x0 + k * plane + kb * 128, r < n);
            }
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const int kb = k0 + d;
                if (kb >= nkb) continue;
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    if (c > 0 && c * 16 >= n) continue;
                    v4f s = (v4f)(0.0f);
#pragma unroll
                    for (int k = 0; k < PLANES; ++k) {
                        if (c > 0)
                            x[d][k] = load_cols(x0 + k * plane + (int64_t)c * 16 * m.F + kb * 128,
                                                c * 16 + r < n);
                        s = block_sum(a[d], x[d][k], s);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[c][k] = __builtin_fmaf(s[k], f[d], acc[c][k]);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            if (c * 16 + r >= n) continue;
            v4f *const p = reinterpret_cast<v4f *>(mine + row[c].token * 16 + q * 4);
            v4f v = *p;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = __builtin_fmaf(acc[c][k], row[c].weight, v[k]);
            *p = v;
        }
        // LDS serves a wave in order; the next unit's sums may be another lane's
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    for (int i = threadIdx.x; i < m.T * 4; i += blockDim.x) {
        v4f v = (v4f)(0.0f);
        for (int k = 0; k < waves; ++k)
            v += *reinterpret_cast<const v4f *>(red + k * m.T * 16 + i * 4);
        store_y(m, partial, (int64_t)(i >> 2) * m.K + nb * 16 + (i & 3) * 4, v);
    }
}

// y = the sum of the parts, in order.
__global__ __launch_bounds__(256) void join_parts_kernel(const float *__restrict__ partial,
                                                         int parts, int64_t n, void *y, bool f32)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    v4f v = *reinterpret_cast<const v4f *>(partial + i);
    for (int k = 1; k < parts; ++k) v += *reinterpret_cast<const v4f *>(partial + k * n + i);
    if (f32)
        *reinterpret_cast<v4f *>(static_cast<float *>(y) + i) = v;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(y) + i) =
            make_uint2(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]));
}

constexpr int kMaxParts = 8;

Layout moe_layout(int T, int E, int S, int top_k, int K, int F)
{
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t rows = (size_t)T * (top_k + S);
    Layout l;
    l.logits = 0;
    l.units = l.logits + up((size_t)kRouterPieces * T * E * 8);
    l.rows = l.units + up(sizeof(Units));
    l.g = l.rows + up(rows * sizeof(Row));
    l.partial = l.g + up(3 * rows * F * 2);
    l.bytes = l.partial + up((size_t)kMaxParts * T * K * 4);
    return l;
}

} // namespace

size_t moe_workspace_bytes(int T, int E, int S, int top_k, int K, int F)
{
    return moe_layout(std::min(T, kMoeTokens), E, S, top_k, K, F).bytes;
}

hipError_t launch_moe(const Moe &m, hipStream_t stream)
{
    if (m.T == 0) return hipSuccess;
    const Layout l = moe_layout(m.T, m.E, m.S, m.top_k, m.K, m.F);
    char *const ws = static_cast<char *>(m.ws);
    double *const logits = reinterpret_cast<double *>(ws + l.logits);
    Units *const units = reinterpret_cast<Units *>(ws + l.units);
    Row *const rows = reinterpret_cast<Row *>(ws + l.rows);
    uint16_t *const g = reinterpret_cast<uint16_t *>(ws + l.g);
    const int64_t plane = (int64_t)m.T * (m.top_k + m.S) * m.F;
    const int most = std::min(m.T * m.top_k, m.E) + m.S;      // units

    // at most two runs of 32 inputs a wave up to K = 4096
    const int pieces = std::min(kRouterPieces, (m.K / 32 + 2 * kRouterWaves - 1) / (2 * kRouterWaves));
    hipLaunchKernelGGL(m.router_f32 ? router_kernel<true> : router_kernel<false>,
                       dim3((m.E + 15) / 16, pieces, (m.T + 15) / 16), dim3(64 * kRouterWaves), 0,
                       stream, m, logits);
    auto by_experts = [&](auto launch) {
        if (m.E <= 128) launch(std::integral_constant<int, 2>{});
        else if (m.E <= 256) launch(std::integral_constant<int, 4>{});
        else launch(std::integral_constant<int, 8>{});
    };
    constexpr int GW = 4;
    auto gate_up = [&](auto kernel, int tiles) {
        hipLaunchKernelGGL(kernel, dim3(m.F / 16, most), dim3(64 * GW), GW * 2 * tiles * 1024,
                           stream, m, units, rows, g, plane, logits, pieces);
    };
    if (m.T == 1) {
        by_experts([&](auto ep) { gate_up(gate_up_kernel<1, 4, decltype(ep)::value>, 1); });
    } else {
        by_experts([&](auto ep) {
            hipLaunchKernelGGL((select_kernel<decltype(ep)::value>), dim3(1), dim3(1024), 0, stream,
                               m, logits, pieces, units, rows);
        });
        if (m.T <= 16) gate_up(gate_up_kernel<1, 4, 0>, 1);
        else gate_up(gate_up_kernel<4, 2, 0>, 4);
    }

    const int blocks = m.K / 16;
    const int parts = m.T == 1 ? 1 : std::max(1, std::min({kMaxParts, most, 1024 / blocks}));
    float *const partial = parts > 1 ? reinterpret_cast<float *>(ws + l.partial) : nullptr;
    if (m.T <= 16) {
        auto down = [&](auto kernel, int waves) {
            hipLaunchKernelGGL(kernel, dim3(blocks, parts), dim3(64 * waves), 0, stream, m, units,
                               rows, g, plane, partial);
        };
        if (m.T == 1) m.y_f32 ? down(down_kernel<16, 1, 3>, 16) : down(down_kernel<16, 2, 2>, 16);
        else m.y_f32 ? down(down_kernel<8, 2, 3>, 8) : down(down_kernel<8, 2, 2>, 8);
    } else {
        constexpr int DW = 8;
        auto down = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3(blocks, parts), dim3(64 * DW), DW * m.T * 64, stream, m,
                               units, rows, g, plane, partial);
        };
        if (m.y_f32) down(down_many_kernel<3>);
        else down(down_many_kernel<2>);
    }
    if (parts > 1) {
        const int64_t n = (int64_t)m.T * m.K;
        hipLaunchKernelGGL(join_parts_kernel, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0,
                           stream, partial, parts, n, m.y, m.y_f32);
    }
    return hipGetLastError();
}

} // namespace convrot
