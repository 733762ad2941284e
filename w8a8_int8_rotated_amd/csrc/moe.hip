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
// rounded to bf16 for bf16 outputs, whose own rounding is as large (together 2.4e-3 of the
// outputs' rms, 1.7e-3 with g exact); for F32 outputs it is carried as three bf16 parts,
// which hold an fp32 value of 2^-110 or more exactly, and a smaller one to 2^-133.
//
// Loads.  A wave keeps a ring of D blocks of codes with their columns in registers: the
// next block is requested as soon as one is used.  Idle columns read past the end of a
// buffer resource, which gives zeros without a branch; blocks past the wave's share are not
// requested at all (a request past the end takes its turn all the same: 5 tokens, 4 of 32
// experts of 5376 x 1408 and a shared one, 89 us a call with those, 83 without).
//
// Kernels: router (partial logits over pieces of K), choose (a wave a token; for a few
// tokens gate_up's workgroups choose for themselves), gate_up, down, and where down was
// split a join.  Measured, us a call and in brackets the chosen experts' codes at the
// 5.1 TB/s of a large copy (reading alone is faster: gate_up reaches 6.0): 64 tokens, 6 of 64
// experts of 5376 x 1408 each: 262 to 267 [283]; 5 tokens, 4 of 32 of them and a shared one: 78
// to 85 [74]; one token, 8 of 128 experts of 2048 x 768: 21 [7.5], three launches whose shortest
// takes 4.4.
#include "moe.hpp"

#include "fp8_common.hpp"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace convrot {
namespace {

typedef double v4d __attribute__((ext_vector_type(4)));
typedef unsigned long long u64;

constexpr int kMaxUnits = kMoeMaxExperts + kMoeMaxShared;
constexpr float kMaxBf16 = 0x1.fep127f;

// A unit is an expert and the tokens that chose it: choose leaves a set of tokens for every
// expert, gate_up finds its unit from them and leaves it here for down.  Rows of g: an expert's
// lie behind those of the experts before it, in the order of its tokens; the shared experts'
// behind all of them.  In memory a unit's n rows, in `planes` parts of bf16 each (one, or three for F32 outputs), are
// [F / 8][planes][n][8]: a block of 128 inputs is one run of memory, and 8 inputs of all rows
// are neighbours in it.  (A load takes its time for the cache lines that it touches; row by
// row each of 16 lanes touches one of its own.  down of 64 tokens so 94.5 us, 102 by rows.)
struct Row {
    int token;
    float weight;
};
struct Units {
    int expert[kMaxUnits];
    int base[kMaxUnits];                   // first of the unit's rows
    u64 tokens[kMaxUnits];                 // none: not a unit
};

constexpr int kRouterPieces = 8, kRouterWaves = 8;
constexpr int kGateWaves = 4, kOwnChoice = kGateWaves;     // tokens that gate_up chooses for itself

struct Layout {
    size_t logits, sets, units, rows, g, partial, bytes;
};

// ------------------------------------------------------------- router ----
// logits[piece][t][e]: a workgroup takes 16 experts, 16 tokens and a piece of K, whose
// runs of 32 inputs its waves share out; they join in LDS in order.  Lane (r, q) holds
// inputs 8 q .. 8 q + 7 of a run of expert r and of token r, one of them per product.
template <bool RF32>
__global__ __launch_bounds__(64 * kRouterWaves) void router_kernel(Moe m,
                                                                   double *__restrict__ logits,
                                                                   u64 *__restrict__ sets)
{
    if (blockIdx.x + blockIdx.y + blockIdx.z == 0)        // choose sets bits in them
        for (int e = threadIdx.x; e < m.E; e += 64 * kRouterWaves) sets[e] = 0;
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
__device__ __forceinline__ int wave_sum(int v)
{
    v += CR_DPP_I(v, 0xB1);
    v += CR_DPP_I(v, 0x4E);
    v += CR_DPP_I(v, 0x141);
    v += CR_DPP_I(v, 0x140);
    return (__builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16)) +
           (__builtin_amdgcn_readlane(v, 32) + __builtin_amdgcn_readlane(v, 48));
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
    const u64 have = __ballot((uint32_t)(v >> 32) == hi);
    // mostly one lane has the largest upper half
    if (__popcll(have) == 1)
        return (u64)hi << 32 |
               (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, __builtin_ctzll(have));
    return (u64)hi << 32 | wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
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
// lowest expert that has it.  Without a bias the order is the logits', and scores are
// formed of the chosen ones alone, where their sum does not need the others.
template <int EP>
__device__ __forceinline__ void choose(const Moe &m, const double *__restrict__ logits, int pieces,
                                       int t, int &id, float &weight)
{
    const int lane = threadIdx.x & 63;
    double p[EP];                        // logits, or with a bias the scores
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
    double top = 0.0, sum = 1.0;
    if (!m.sigmoid) {
        top = value_of(wave_max(best));
        if (m.bias || !m.renormalize) {
            sum = 0.0;
#pragma unroll
            for (int i = 0; i < EP; ++i)
                if (lane + 64 * i < m.E) sum += exp(p[i] - top);
            sum = wave_sum(sum);
        }
    }
    auto score = [&](double x) {
        return m.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - top) / sum;
    };
    if (m.bias) {
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            const int e = lane + 64 * i;
            p[i] = score(p[i]);
            if (e < m.E) key[i] = order_of(p[i] + (double)m.bias[e]);
        }
    }
    double w = 0.0;
    id = 0;
    for (int j = 0; j < m.top_k; ++j) {
        best = 0;
#pragma unroll
        for (int i = 0; i < EP; ++i) best = key[i] > best ? key[i] : best;
        best = wave_max(best);
        int e = -1;
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            const u64 hit = __ballot(key[i] == best);
            if (e >= 0 || hit == 0) continue;
            const int l = __builtin_ctzll(hit);
            e = 64 * i + l;
            const int2 u = __builtin_bit_cast(int2, p[i]);
            const double s = __builtin_bit_cast(
                double, make_int2(__builtin_amdgcn_readlane(u.x, l),
                                  __builtin_amdgcn_readlane(u.y, l)));
            if (lane == l) key[i] = 0;
            if (lane == j) id = e, w = s;
        }
    }
    if (!m.bias) w = score(w);
    if (m.renormalize) {
        const double total = wave_sum(lane < m.top_k ? w : 0.0);
        w = total == 0.0 ? 0.0 : w / total;
    }
    weight = (float)(w * m.factor);
}

template <int EP>
__global__ __launch_bounds__(64) void choose_kernel(Moe m, const double *__restrict__ logits,
                                                    int pieces, u64 *__restrict__ sets)
{
    int id;
    float w;
    choose<EP>(m, logits, pieces, blockIdx.x, id, w);
    const int lane = threadIdx.x;
    if (lane >= m.top_k) return;
    m.ids[(int64_t)blockIdx.x * m.top_k + lane] = id;
    m.weights[(int64_t)blockIdx.x * m.top_k + lane] = w;
    atomicOr(sets + id, 1ull << blockIdx.x);               // bits: no order
}

// ------------------------------------------------------------ experts ----

constexpr uint32_t kOut = 0x7f000000u;     // an offset beyond every range used here

__device__ __forceinline__ __amdgpu_buffer_rsrc_t range_of(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes,
                                             0x00020000);
}
__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t p, uint32_t off)
{
    return __builtin_amdgcn_raw_buffer_load_b128(p, (int)off, 0, 0);
}
__device__ __forceinline__ float load4(__amdgpu_buffer_rsrc_t p, uint32_t off)
{
    return __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(p, (int)off, 0, 0));
}

// One 16 x 128 block of codes as two 16-byte pieces a lane.
struct Block {
    v4i lo, hi;
};
__device__ __forceinline__ Block load_block(__amdgpu_buffer_rsrc_t p, uint32_t off)
{
    return {load16(p, off), load16(p, off + 1024)};
}

// 16 columns' inputs of a block of 128: four pieces of 8 a lane, step bytes apart.
struct Cols {
    v4i u[4];
};
__device__ __forceinline__ Cols load_cols(__amdgpu_buffer_rsrc_t p, uint32_t off, uint32_t step)
{
    return {{load16(p, off), load16(p, off + step), load16(p, off + 8 * step),
             load16(p, off + 9 * step)}};
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ u64 uniform(u64 v)
{
    return (u64)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
           (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}

// The codes of a block as bf16, and its products with 16 columns added to s.
struct Wide {
    v8bf k[4];
};
__device__ __forceinline__ Wide widen(const Block &a)
{
    return {{bf16_of_codes(a.lo[0], a.lo[1]), bf16_of_codes(a.lo[2], a.lo[3]),
             bf16_of_codes(a.hi[0], a.hi[1]), bf16_of_codes(a.hi[2], a.hi[3])}};
}
__device__ __forceinline__ v4f block_sum(const Wide &a, const Cols &b)
{
    v4f s = (v4f)(0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.k[i], __builtin_bit_cast(v8bf, b.u[i]), s, 0,
                                                    0, 0);
    return s;
}

// g of one unit: a workgroup takes 16 gate and the same 16 up channels, its waves the
// groups of P blocks of K in turn.  Columns are the unit's n rows, from row `base` of g on,
// in up to CT tiles of 16; with P > 1 (up to 16 / P rows) column j * (16 / P) + i is row i's
// part of the group's block j, so that one set of columns serves P blocks.  token: of row
// `lane`.
template <int CT, int D, int P>
__device__ __forceinline__ void gate_up(const Moe &m, int expert, int base, int n,
                                        int token, float *red,
                                        uint16_t *__restrict__ g)
{
    static_assert(CT == 1 || P == 1, "");
    constexpr int CP = 16 / P;                     // columns of one block
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int waves = kGateWaves;
    const int ri = r % CP, rj = r / CP;            // the lane's row (of a tile) and block
    const int nkb = m.K >> 7, fb = blockIdx.x;
    const uint32_t in_tile = r * 64 + ((q ^ ((r >> 2) & 3)) << 4);
    const uint8_t *const codes = m.gate_up + ((int64_t)expert * 2 * m.F + fb * 16) * m.K;
    const __amdgpu_buffer_rsrc_t gate = range_of(codes, 16 * m.K);
    const __amdgpu_buffer_rsrc_t up = range_of(codes + (int64_t)m.F * m.K, 16 * m.K);
    const float *const sg = m.gate_up_scale +
                            ((int64_t)expert * (m.F >> 6) + (fb >> 3)) * nkb;
    const __amdgpu_buffer_rsrc_t gate_scale = range_of(sg, nkb * 4);
    const __amdgpu_buffer_rsrc_t up_scale = range_of(sg + (int64_t)(m.F >> 7) * nkb, nkb * 4);
    const __amdgpu_buffer_rsrc_t xs = range_of(m.x, (uint32_t)(m.T * m.K * 2));

    uint32_t col[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int from = __shfl(token, c * 16 + ri, 64);
        col[c] = c * 16 + ri < n ? (uint32_t)(from * m.K + q * 16) * 2 : kOut;
    }
    v4f ag[CT], au[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) ag[c] = au[c] = (v4f)(0.0f);
    Block a[D][P], b[D][P];
    Cols x[D][CT];
    float fg[D], fu[D];
    const int step = waves * P;
    int next = wave * P;                           // the group to request
    auto request = [&](int d) {
        if (next >= nkb) return;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const uint32_t at = next + j < nkb ? (next + j) * 2048 + in_tile : kOut;
            a[d][j] = load_block(gate, at);
            b[d][j] = load_block(up, at);
        }
        const int kb = next + rj;
#pragma unroll
        for (int c = 0; c < CT; ++c)
            if (c == 0 || c * 16 < n)
                x[d][c] = load_cols(xs, kb < nkb && c * 16 + ri < n ? col[c] + kb * 256 : kOut, 16);
        fg[d] = load4(gate_scale, kb < nkb ? kb * 4 : kOut);
        fu[d] = load4(up_scale, kb < nkb ? kb * 4 : kOut);
        next += step;
        __builtin_amdgcn_sched_barrier(0);         // not all D uses first, then all requests
    };
#pragma unroll
    for (int d = 0; d < D; ++d) request(d);
    for (int k0 = wave * P; k0 < nkb; k0 += step * D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (k0 + d * step >= nkb) break;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const bool on = rj == j;
                // gate, then up: one of them widened at a time
                auto add = [&](const Block &codes, float f, v4f (&acc)[CT]) {
                    const Wide w = widen(codes);
#pragma unroll
                    for (int c = 0; c < CT; ++c) {
                        if (c > 0 && c * 16 >= n) continue;
                        const v4f s = block_sum(w, x[d][c]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[c][i] = on ? __builtin_fmaf(s[i], f, acc[c][i]) : acc[c][i];
                    }
                };
                add(a[d][j], fg[d], ag);
                if constexpr (CT > 1) __builtin_amdgcn_sched_barrier(0);
                add(b[d][j], fu[d], au);
            }
            request(d);
        }
    }
    // tile by tile, in two buffers in turn: a tile's sums are read before the next but one's
    // are written
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        if (c > 0 && c * 16 >= n) break;
        float *const buf = red + (c & 1) * waves * 512;
        *reinterpret_cast<v4f *>(buf + (wave * 2 + 0) * 256 + lane * 4) = ag[c];
        *reinterpret_cast<v4f *>(buf + (wave * 2 + 1) * 256 + lane * 4) = au[c];
        __syncthreads();
        if (wave != c || rj > 0 || c * 16 + ri >= n) continue;
        v4f a = (v4f)(0.0f), b = (v4f)(0.0f);
        for (int k = 0; k < waves; ++k)
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float *const p = buf + k * 512 + (lane + j * CP) * 4;
                a += *reinterpret_cast<const v4f *>(p);
                b += *reinterpret_cast<const v4f *>(p + 256);
            }
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i] / (1.0f + expf(-a[i])) * b[i];
        const int planes = m.y_f32 ? 3 : 1;
        uint16_t *p = g + (int64_t)base * planes * m.F +
                      ((fb * 2 + (q >> 1)) * planes * n + c * 16 + r) * 8 + (q & 1) * 4;
        // the part that bf16 holds; for F32 outputs what it leaves, twice more.  A part that others
        // follow stays within bf16's largest value: rounded past it, it would be infinite and
        // what it leaves minus infinity
        for (int part = 1;; ++part) {
            const float most = part < planes ? kMaxBf16 : __builtin_inff();
            float c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = fabsf(v[i]) > most ? copysignf(most, v[i]) : v[i];
            const uint2 o = make_uint2(cvt_pk_bf16(c[0], c[1]), cvt_pk_bf16(c[2], c[3]));
            *reinterpret_cast<uint2 *>(p) = o;
            if (part == planes) break;
            v[0] -= bf16_lo(o.x);
            v[1] -= bf16_hi(o.x);
            v[2] -= bf16_lo(o.y);
            v[3] -= bf16_hi(o.y);
            p += n * 8;
        }
    }
}

// blockIdx.y: with fewer choices than experts a choice, whose expert is taken up where it
// comes first, else an expert; then the shared ones.  ROWS: the most rows of a unit.
// EP > 0: up to kOwnChoice tokens, whose choices the workgroup makes itself, a wave a token
// (of a single token every wave, and no wave waits for another).
template <int ROWS, int EP>
__global__ __launch_bounds__(64 * kGateWaves, 3) void gate_up_kernel(
    Moe m, Units *__restrict__ units, Row *__restrict__ rows, uint16_t *__restrict__ g,
    const double *__restrict__ logits, int pieces, const u64 *__restrict__ sets)
{
    extern __shared__ float red[];                 // [1 or 2 tiles of 16 rows][wave][2][256]
    __shared__ int s_ids[EP > 0 ? kOwnChoice * kMoeMaxTopK : 1];
    __shared__ float s_weights[EP > 0 ? kOwnChoice * kMoeMaxTopK : 1];
    const int u = blockIdx.y, chosen = m.T * m.top_k, routed = min(chosen, m.E);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool shared = u >= routed, single = EP > 0 && m.T == 1;
    int expert = m.E + u - routed, base = chosen + (u - routed) * m.T;
    u64 tokens = m.T == 64 ? ~0ull : (1ull << m.T) - 1;
    int id = 0;
    float weight = 1.0f;
    if constexpr (EP > 0) {
        if (!shared) {
            if (single || wave < m.T) choose<EP>(m, logits, pieces, single ? 0 : wave, id, weight);
            if (single) {
                expert = __builtin_amdgcn_readlane(id, u);
                weight = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), u));
                base = u;
            } else {
                if (wave < m.T && lane < m.top_k) {
                    const int i = wave * m.top_k + lane;
                    s_ids[i] = id;
                    s_weights[i] = weight;
                    if (blockIdx.x == 0 && u == 0) m.ids[i] = id, m.weights[i] = weight;
                }
                __syncthreads();
                expert = uniform(chosen < m.E ? s_ids[u] : u);
                tokens = 0;
                base = 0;
                for (int i0 = 0; i0 < chosen; i0 += 64) {
                    const int i = i0 + lane, e = i < chosen ? s_ids[i] : kMaxUnits;
                    base += __popcll(__ballot(e < expert));
                    for (u64 hit = __ballot(e == expert); hit; hit &= hit - 1)
                        tokens |= 1ull << ((i0 + __builtin_ctzll(hit)) / m.top_k);
                }
            }
        }
    } else if (!shared) {
        if (chosen < m.E) expert = uniform(m.ids[u]);
        else expert = u;
        tokens = uniform(sets[expert]);
        int before = 0;
        for (int e = lane; e < expert; e += 64) before += __popcll(sets[e]);
        base = wave_sum(before);
    }
    // a choice whose expert an earlier token chose too is not a unit of its own
    if (!shared && !single && chosen < m.E && tokens != 0 && __builtin_ctzll(tokens) != u / m.top_k)
        tokens = 0;
    const int n = uniform((int)__popcll(tokens));
    const int rank = __popcll(tokens & ((1ull << lane) - 1));
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        units->expert[u] = expert;
        units->base[u] = base;
        units->tokens[u] = tokens;
    }
    if (tokens == 0) return;
    // lane i gets the token of row i (the lanes of no row go behind them)
    const int to = (tokens >> lane) & 1 ? rank : n + lane - rank;
    const int token = __builtin_amdgcn_ds_permute(to * 4, lane);
    // the deepest rings that 168 registers hold (three waves a SIMD): 64 tokens, 2 of 8 experts
    // of 4096 x 2048, us with two tiles in the ring and with the further tiles loaded where they
    // are used: 32.7, 40
    if (ROWS == 8 || n <= 8) gate_up<1, 2, 2>(m, expert, base, n, token, red, g);
    if constexpr (ROWS == 16) {
        if (n > 8) gate_up<1, 3, 1>(m, expert, base, n, token, red, g);
    } else if constexpr (ROWS == 64) {
        if (n > 32) gate_up<4, 1, 1>(m, expert, base, n, token, red, g);
        else if (n > 16) gate_up<2, 2, 1>(m, expert, base, n, token, red, g);
        else if (n > 8) gate_up<1, 3, 1>(m, expert, base, n, token, red, g);
    }
    // the unit's rows for down
    if (blockIdx.x > 0 || wave > 0 || lane >= m.T || !((tokens >> lane) & 1)) return;
    if (!shared && !single)
        for (int j = lane * m.top_k; j < (lane + 1) * m.top_k; ++j) {
            const int e = EP > 0 ? s_ids[j] : m.ids[j];
            const float w = EP > 0 ? s_weights[j] : m.weights[j];
            if (e == expert) weight = w;
        }
    else if (single && !shared)
        m.ids[u] = expert, m.weights[u] = weight;
    rows[base + rank] = {lane, weight};
}

// This wave's share of n things: of all waves of the workgroups that sum the same outputs.
__device__ __forceinline__ int share(int n, int waves, int wave)
{
    return (int)((int64_t)n * ((int)blockIdx.y * waves + wave) / ((int)gridDim.y * waves));
}

// The units, compacted into LDS by the whole workgroup in three classes by their rows: up to
// few, up to some, more; class c is order[first[c]] .. order[first[c + 1]].
struct UnitList {
    u64 tokens[kMaxUnits];
    short expert[kMaxUnits], base[kMaxUnits], order[kMaxUnits];
    int first[4];
};
static_assert(kMoeTokens * (kMoeMaxTopK + kMoeMaxShared) < 32768, "rows fit short");
__device__ __forceinline__ void list_units(const Units *__restrict__ units, int most, int few,
                                           int some, UnitList &l)
{
    const int lane = threadIdx.x & 63;
    for (int u = threadIdx.x; u < most; u += blockDim.x) {
        l.tokens[u] = units->tokens[u];
        l.expert[u] = (short)units->expert[u];
        l.base[u] = (short)units->base[u];
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        int at = 0;
        for (int c = 0; c < 3; ++c) {
            if (lane == 0) l.first[c] = at;
            for (int i = 0; i < most; i += 64) {
                const int u = i + lane;
                const int n = u < most ? __popcll(l.tokens[u]) : 0;
                const bool in = c == 0 ? n > 0 && n <= few : c == 1 ? n > few && n <= some : n > some;
                const u64 have = __ballot(in);
                if (in) l.order[at + __popcll(have & ((1ull << lane) - 1))] = (short)u;
                at += __popcll(have);
            }
        }
        if (lane == 0) l.first[3] = at;
    }
    __syncthreads();
}

// 4 outputs of y, or of this workgroup's part of the units (partial: [part][T][K]).
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

// One expert's codes and scales of a workgroup's 16 outputs.
struct DownRows {
    __amdgpu_buffer_rsrc_t codes, scale;
};
__device__ __forceinline__ DownRows down_rows(const Moe &m, int64_t e, int nb)
{
    const int nkb = m.F >> 7;
    return {range_of(m.down + (e * m.K + nb * 16) * m.F, 16 * m.F),
            range_of(m.down_scale + (e * (m.K >> 7) + (nb >> 3)) * nkb, nkb * 4)};
}

// y of 16 outputs for up to CP = 16 / (P PLANES) tokens: the units' blocks of F, in groups
// of P, are one sequence, of which each wave takes an even share.  Column
// (j PLANES + p) CP + t is, for the group's block j, part p of token t's g, zero where the
// token did not choose the unit: a token's sums over its experts stay in one place, and
// its parts and the group's further blocks need no further columns.
template <int D, int P, int PLANES>
__global__ __launch_bounds__(512, 4) void down_kernel(Moe m, const Units *__restrict__ units,
                                                      int most, const Row *__restrict__ rows,
                                                      const uint16_t *__restrict__ g,
                                                      float *__restrict__ partial)
{
    constexpr int WAVES = 8, CP = 16 / (P * PLANES);
    __shared__ float red[WAVES * 256];
    __shared__ float weight[CP * (kMoeMaxTopK + kMoeMaxShared)];
    __shared__ UnitList list;
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = r % CP, part = r / CP % PLANES, rj = r / CP / PLANES;
    const int nkb = m.F >> 7, nb = blockIdx.x, groups = (nkb + P - 1) / P;
    const uint32_t in_tile = r * 64 + ((q ^ ((r >> 2) & 3)) << 4);
    const __amdgpu_buffer_rsrc_t gs = range_of(g, m.T * (m.top_k + m.S) * m.F * 2 * PLANES);
    for (int i = threadIdx.x; i < m.T * (m.top_k + m.S); i += 64 * WAVES)
        weight[i] = rows[i].weight;
    list_units(units, most, kMoeTokens, kMoeTokens, list);
    const int count = uniform(list.first[1]);

    v4f acc = (v4f)(0.0f);
    const int total = count * groups;
    const int i0 = share(total, WAVES, wave), i1 = share(total, WAVES, wave + 1);
    if (i0 < i1) {
        int u = i0 / groups, kb = (i0 - u * groups) * P, left = i1 - i0;
        DownRows rw;
        uint32_t col = 0, piece = 0;
        float wu = 0.0f;
        bool has = false;
        auto enter = [&] {
            const int at = uniform(list.order[min(u, count - 1)]);
            rw = down_rows(m, uniform(list.expert[at]), nb);
            const u64 tokens = uniform(list.tokens[at]);
            has = rj < P && ((tokens >> t) & 1);
            const int base = uniform(list.base[at]);
            const int row = __popcll(tokens & ((1ull << t) - 1));
            wu = has ? weight[base + row] : 0.0f;
            const int n = __popcll(tokens);
            piece = PLANES * n * 16;
            col = base * m.F * 2 * PLANES + 2 * q * piece + (part * n + row) * 16;
        };
        enter();
        Block a[D][P];
        Cols x[D];
        float w[D], f[D];
        bool on[D];
        auto request = [&](int d) {
            if (left <= 0) return;
#pragma unroll
            for (int j = 0; j < P; ++j)
                a[d][j] = load_block(rw.codes, kb + j < nkb ? (kb + j) * 2048 + in_tile : kOut);
            on[d] = has && kb + rj < nkb;
            x[d] = load_cols(gs, on[d] ? col + (kb + rj) * 16 * piece : kOut, piece);
            f[d] = load4(rw.scale, on[d] ? (kb + rj) * 4 : kOut);
            w[d] = wu;
            --left;
            kb += P;
            if (kb >= nkb) {
                kb = 0;
                ++u;
                enter();
            }
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int d = 0; d < D; ++d) request(d);
        for (int i = i0; i < i1; i += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (i + d >= i1) break;
                const float c = w[d] * f[d];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const v4f s = block_sum(widen(a[d][j]), x[d]);
                    // a token that did not choose the expert takes nothing of it, codes of
                    // NaN included
                    const bool take = on[d] && rj == j;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        acc[k] = take ? __builtin_fmaf(s[k], c, acc[k]) : acc[k];
                }
                request(d);
            }
        }
    }
    *reinterpret_cast<v4f *>(red + wave * 256 + lane * 4) = acc;
    __syncthreads();
    if (wave > 0 || r >= CP || t >= m.T) return;
    v4f v = (v4f)(0.0f);
    for (int k = 0; k < WAVES; ++k)
#pragma unroll
        for (int p = 0; p < P * PLANES; ++p)
            v += *reinterpret_cast<const v4f *>(red + k * 256 + (lane + p * CP) * 4);
    store_y(m, partial, (int64_t)t * m.K + nb * 16 + q * 4, v);
}

// The same for more tokens.  Columns are the parts of a unit's rows one after another:
// column p * n + i is part p of row i.  A unit's sums, weighted, are added to the wave's own
// [T][16] sums in LDS, part by part (two columns of one token are never added at once).
// Units whose columns fit 8 (one part) make one sequence of groups of two blocks (columns
// 8 .. 15 belong to the group's second block), those whose columns fit two tiles of 16 one of
// single blocks; of a sequence each wave takes an even share and its ring runs on from unit
// to unit.  The others follow, up to CT tiles in one pass over their codes.  Bound: memory
// and what a wave can keep in flight beside the columns: 64 tokens, 6 of 64 experts of
// 5376 x 1408: bf16 95 us (5.1 TB/s of codes), F32 outputs 143.  (Units of two tiles outside
// the ring, a block at a time: F32 205, with g by rows then; 175 in the ring.)
template <int PLANES>
__global__ __launch_bounds__(512, 4) void down_many_kernel(Moe m, const Units *__restrict__ units,
                                                           int most, const Row *__restrict__ rows,
                                                           const uint16_t *__restrict__ g,
                                                           float *__restrict__ partial)
{
    constexpr int CT = 4, WAVES = 8;
    extern __shared__ float red[];                 // [wave][T][16], rows
    __shared__ UnitList list;
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nkb = m.F >> 7, nb = blockIdx.x;
    const uint32_t in_tile = r * 64 + ((q ^ ((r >> 2) & 3)) << 4);
    const __amdgpu_buffer_rsrc_t gs = range_of(g, m.T * (m.top_k + m.S) * m.F * 2 * PLANES);
    float *const mine = red + wave * m.T * 16;
    Row *const lrows = reinterpret_cast<Row *>(red + WAVES * m.T * 16);
    for (int i = threadIdx.x; i < m.T * (m.top_k + m.S); i += 64 * WAVES) lrows[i] = rows[i];
    for (int i = lane; i < m.T * 4; i += 64)
        *reinterpret_cast<v4f *>(mine + i * 4) = (v4f)(0.0f);
    list_units(units, most, PLANES == 1 ? 8 : 0, 32 / PLANES, list);

    // the part that column v of a unit of n rows belongs to (PLANES or more: none)
    auto part_of = [](int v, int n) {
        int part = 0;
#pragma unroll
        for (int p = 1; p <= PLANES; ++p) part += v >= p * n;
        return part;
    };
    // adds to the sums of column v of a unit of n rows from `base` on (v past its columns: none)
    auto flush = [&](const v4f &acc, int v, int base, int n) {
        const int part = part_of(v, n);
        const Row row = lrows[base + (part < PLANES ? v - part * n : 0)];
#pragma unroll
        for (int p = 0; p < PLANES; ++p) {
            if (part == p) {
                v4f *const to = reinterpret_cast<v4f *>(mine + row.token * 16 + q * 4);
                v4f s = *to;
#pragma unroll
                for (int k = 0; k < 4; ++k) s[k] = __builtin_fmaf(acc[k], row.weight, s[k]);
                *to = s;
            }
            // LDS serves a wave in order; the compiler must keep that order
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    };
    // byte offset of column v of such a unit, at its first block
    auto column = [&](int v, int base, int n) -> uint32_t {
        return v < PLANES * n
                   ? (uint32_t)(base * m.F * 2 * PLANES + (2 * q * PLANES * n + v) * 16)
                   : kOut;
    };

    // the units of class c, whose columns fit 16 / P, with P = 1 also two tiles of 16
    auto run = [&](auto p, int c) {
        constexpr int P = decltype(p)::value, D = 2, CP = 16 / P, TILES = P == 1 ? 2 : 1;
        const int from = uniform(list.first[c]), count = uniform(list.first[c + 1]) - from;
        const int groups = (nkb + P - 1) / P, rj = r / CP, total = count * groups;
        const int i0 = share(total, WAVES, wave), i1 = share(total, WAVES, wave + 1);
        if (i0 >= i1) return;
        Block a[D][P];
        Cols x[D][TILES];
        float f[D];
        bool two[D];                                   // the block's unit takes two tiles
        int u = i0 / groups, kb = (i0 - u * groups) * P, left = i1 - i0;   // to request
        DownRows rw;
        uint32_t col[TILES], piece = 0;
        bool wide = false;
        auto enter = [&] {
            const int at = uniform(list.order[from + min(u, count - 1)]);
            rw = down_rows(m, uniform(list.expert[at]), nb);
            const int base = uniform(list.base[at]), n = __popcll(uniform(list.tokens[at]));
            piece = PLANES * n * 16;
            wide = TILES > 1 && PLANES * n > 16;
#pragma unroll
            for (int c = 0; c < TILES; ++c) col[c] = column(c * 16 + r % CP, base, n);
        };
        enter();
        int cu = u, ckb = kb;                                              // in use
        auto request = [&](int d) {
            if (left <= 0) return;
#pragma unroll
            for (int j = 0; j < P; ++j)
                a[d][j] = load_block(rw.codes, kb + j < nkb ? (kb + j) * 2048 + in_tile : kOut);
            const bool on = kb + rj < nkb;
            two[d] = wide;
#pragma unroll
            for (int c = 0; c < TILES; ++c)
                if (c == 0 || wide)
                    x[d][c] = load_cols(
                        gs, on && col[c] != kOut ? col[c] + (kb + rj) * 16 * piece : kOut, piece);
            f[d] = load4(rw.scale, on ? (kb + rj) * 4 : kOut);
            --left;
            kb += P;
            if (kb >= nkb) {
                kb = 0;
                ++u;
                enter();
            }
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int d = 0; d < D; ++d) request(d);
        v4f acc[TILES];
#pragma unroll
        for (int c = 0; c < TILES; ++c) acc[c] = (v4f)(0.0f);
        for (int i = i0; i < i1; i += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (i + d >= i1) break;
                const bool both = two[d];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const Wide w = widen(a[d][j]);
#pragma unroll
                    for (int c = 0; c < TILES; ++c) {
                        if (c > 0 && !both) continue;
                        const v4f s = block_sum(w, x[d][c]);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            acc[c][k] = rj == j ? __builtin_fmaf(s[k], f[d], acc[c][k]) : acc[c][k];
                    }
                }
                request(d);
                ckb += P;
                if (ckb >= nkb || i + d + 1 == i1) {
                    const int at = uniform(list.order[from + cu]);
                    const int base = uniform(list.base[at]);
                    const int n = __popcll(uniform(list.tokens[at]));
                    if constexpr (P == 2) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)            // columns 8 apart: row_ror:8
                            acc[0][k] += __int_as_float(CR_DPP_I(__float_as_int(acc[0][k]), 0x128));
                    }
#pragma unroll
                    for (int c = 0; c < TILES; ++c) {
                        if (c > 0 && !both) continue;
                        flush(acc[c], rj == 0 ? c * 16 + r : PLANES * n, base, n);
                        acc[c] = (v4f)(0.0f);
                    }
                    ckb = 0;
                    ++cu;
                }
            }
        }
    };
    // (three parts of a row in two groups of columns leave room for two rows only)
    if constexpr (PLANES == 1) run(std::integral_constant<int, 2>{}, 0);
    run(std::integral_constant<int, 1>{}, 1);

    const int from = uniform(list.first[2]), total = (uniform(list.first[3]) - from) * nkb;
    for (int i = share(total, WAVES, wave), end = share(total, WAVES, wave + 1); i < end;) {
        const int u = i / nkb, kb0 = i - u * nkb, kb1 = min(nkb, kb0 + end - i);
        i += kb1 - kb0;
        const int at = uniform(list.order[from + u]);
        const DownRows rw = down_rows(m, uniform(list.expert[at]), nb);
        const int base = uniform(list.base[at]), n = __popcll(uniform(list.tokens[at]));
        const uint32_t piece = PLANES * n * 16;
        for (int c0 = 0; c0 < PLANES * n; c0 += 16 * CT) {
            v4f acc[CT];
            uint32_t col[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                acc[c] = (v4f)(0.0f);
                col[c] = column(c0 + c * 16 + r, base, n);
            }
            Block a = load_block(rw.codes, kb0 * 2048 + in_tile);
            float f = load4(rw.scale, kb0 * 4);
            for (int kb = kb0; kb < kb1; ++kb) {
                Cols x[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    x[c] = load_cols(gs, col[c] != kOut ? col[c] + kb * 16 * piece : kOut, piece);
                const Wide w = widen(a);
                const float fk = f;
                const bool more = kb + 1 < kb1;
                a = load_block(rw.codes, more ? (kb + 1) * 2048 + in_tile : kOut);
                f = load4(rw.scale, more ? (kb + 1) * 4 : kOut);
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    if (c0 + c * 16 >= PLANES * n) continue;
                    const v4f s = block_sum(w, x[c]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[c][k] = __builtin_fmaf(s[k], fk, acc[c][k]);
                }
            }
#pragma unroll
            for (int c = 0; c < CT; ++c)
                if (c0 + c * 16 < PLANES * n) flush(acc[c], c0 + c * 16 + r, base, n);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < m.T * 4; i += 64 * WAVES) {
        v4f v = (v4f)(0.0f);
        for (int k = 0; k < WAVES; ++k)
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
    l.sets = l.logits + up((size_t)kRouterPieces * T * E * 8);
    l.units = l.sets + up((size_t)E * 8);
    l.rows = l.units + up(sizeof(Units));
    l.g = l.rows + up(rows * sizeof(Row));
    l.partial = l.g + up(3 * rows * F * 2);
    l.bytes = l.partial + up((size_t)kMaxParts * T * K * 4);
    return l;
}

// Parts of the units whose sums a second kernel joins: the CUs hold two workgroups each,
// and a round that they do not fill reads more slowly.  64 tokens, 64 experts of
// K = 5376, F = 1408 (336 workgroups a part), us with 1, 2, 3, 4, 6 parts and without the
// join (5 us): 120, 101, 95, 103, 101; 23 tokens, 40 experts of K = 2560, F = 640, F32 (160
// workgroups a part): 25.5, 25.9, 20.8, 23.2, 23.1.  The bytes are those of the experts that
// the tokens are expected to choose.  More than one part is charged 8 us, the join and the
// parts' way through memory: with the join's 5 alone, the calls whose estimates lie between are
// mostly slower, us with 5 and with 8: 1 token, 4 of 16 experts of 4096 x 2048, 2 parts and 1: 30.1,
// 28.1; 23 tokens, 4 of 32 of 5376 x 384 and a shared one, 3 and 1: 58.0, 55.2; 64 tokens, 4 of 16
// of 5376 x 640, 3 and 1: bf16 59.9, 57.9, F32 71.9, 74.9; 4 tokens, 6 of 64 of 5376 x 640: 55.6, 57.0.
int down_parts(const Moe &m)
{
    const double units = m.E * (1.0 - std::pow(1.0 - (double)m.top_k / m.E, m.T)) + m.S;
    const double us = units * m.K * m.F / 5.1e6;
    const int blocks = m.K / 16, round = 2 * device_cu_count();
    int best = 1;
    double least = 0.0;
    for (int p = 1; p <= kMaxParts; ++p) {
        const int rounds = (blocks * p + round - 1) / round;
        const double t = us * rounds * round / (blocks * p) + (p > 1 ? 8.0 : 0.0);
        if (p == 1 || t < least) best = p, least = t;
    }
    return best;
}

} // namespace

// Up to kOwnChoice tokens the workgroups of gate_up choose for themselves while they are one
// round of the CUs (three a CU), since each pays for it.  us a call with that and with the
// kernel of its own, 256 CUs:
//   1 token: 8 of 128 experts of 2048 x 768 (384 workgroups) 20.6, 23.4; of 2048 x 1536 (768)
//     27.4, 29.9; of 2048 x 2048 (1024) 34.0, 34.1; 16 of 256 of 2048 x 1024 (1024) 40.9, 37.7;
//     32 of 512 of 1024 x 512 (1024) 55.8, 42.3; of 512 x 2048 (4096) 135, 58.5
//   2 tokens: 45 experts, 8 each, of 2944 x 1792 (1792) 62.2, 57.8;  3 tokens: 5 experts of
//     256 x 896 21.7, 25.2
bool moe_own_choice(int T, int64_t workgroups, int64_t cus)
{
    return T <= kOwnChoice && workgroups <= 3 * cus;
}

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
    u64 *const sets = reinterpret_cast<u64 *>(ws + l.sets);
    Units *const units = reinterpret_cast<Units *>(ws + l.units);
    Row *const rows = reinterpret_cast<Row *>(ws + l.rows);
    uint16_t *const g = reinterpret_cast<uint16_t *>(ws + l.g);
    const int most = std::min(m.T * m.top_k, m.E) + m.S;      // units

    // at most two runs of 32 inputs a wave up to K = 4096
    const int pieces = std::min(kRouterPieces, (m.K / 32 + 2 * kRouterWaves - 1) / (2 * kRouterWaves));
    hipLaunchKernelGGL(m.router_f32 ? router_kernel<true> : router_kernel<false>,
                       dim3((m.E + 15) / 16, pieces, (m.T + 15) / 16), dim3(64 * kRouterWaves), 0,
                       stream, m, logits, sets);
    auto by_experts = [&](auto launch) {
        if (m.E <= 128) launch(std::integral_constant<int, 2>{});
        else if (m.E <= 256) launch(std::integral_constant<int, 4>{});
        else launch(std::integral_constant<int, 8>{});
    };
    const int tiles = m.F / 16;
    auto gate_up = [&](auto kernel, int buffers) {
        hipLaunchKernelGGL(kernel, dim3(tiles, most), dim3(64 * kGateWaves),
                           buffers * kGateWaves * 2 * 1024, stream, m, units, rows, g,
                           logits, pieces, sets);
    };
    if (moe_own_choice(m.T, tiles * most, device_cu_count())) {
        by_experts([&](auto ep) { gate_up(gate_up_kernel<8, decltype(ep)::value>, 1); });
    } else {
        by_experts([&](auto ep) {
            hipLaunchKernelGGL((choose_kernel<decltype(ep)::value>), dim3(m.T), dim3(64), 0,
                               stream, m, logits, pieces, sets);
        });
        if (m.T <= 8) gate_up(gate_up_kernel<8, 0>, 1);
        else if (m.T <= 16) gate_up(gate_up_kernel<16, 0>, 1);
        else gate_up(gate_up_kernel<64, 0>, 2);
    }

    const int parts = down_parts(m);
    float *const partial = parts > 1 ? reinterpret_cast<float *>(ws + l.partial) : nullptr;
    auto down = [&](auto kernel, size_t lds) {
        hipLaunchKernelGGL(kernel, dim3(m.K / 16, parts), dim3(512), lds, stream, m, units, most,
                           rows, g, partial);
    };
    const size_t many = m.T * (8 * 64 + (m.top_k + m.S) * sizeof(Row));
    static_assert(kMoeTokens * (8 * 64 + (kMoeMaxTopK + kMoeMaxShared) * sizeof(Row)) +
                          sizeof(UnitList) <= 65536, "LDS of down_many_kernel");
    if (m.y_f32) m.T <= 5 ? down(down_kernel<3, 1, 3>, 0) : down(down_many_kernel<3>, many);
    else if (m.T <= 8) down(down_kernel<1, 2, 1>, 0);
    else if (m.T <= 16) down(down_kernel<3, 1, 1>, 0);
    else down(down_many_kernel<1>, many);
    if (parts > 1) {
        const int64_t n = (int64_t)m.T * m.K;
        hipLaunchKernelGGL(join_parts_kernel, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0,
                           stream, partial, parts, n, m.y, m.y_f32);
    }
    return hipGetLastError();
}

} // namespace convrot
