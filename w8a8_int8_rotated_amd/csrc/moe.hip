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
// Columns are tokens, not slots: column t of every expert's tile is token t, zero where
// t did not choose it.  So the sums of a token's experts stay in one accumulator of the
// down projection, and nothing is scattered.
//
// Precision.  The logits are summed in fp64 (v_mfma_f64_16x16x4_f64): the choice of
// experts then does not depend on the order of the sums, a batch or a shape.  g is
// rounded to bf16 for bf16 outputs (their own rounding is as large); for F32 outputs it
// is carried as three bf16 parts, which hold an fp32 value exactly.
//
// Kernels: router (partial logits over pieces of K), select (one workgroup: choices,
// and for each chosen expert, a "unit", the set of its tokens), gate_up, down.
#include "moe.hpp"

#include "fp8_common.hpp"

#include <algorithm>

namespace convrot {
namespace {

typedef double v4d __attribute__((ext_vector_type(4)));
typedef unsigned long long u64;

constexpr int kMaxUnits = kMoeMaxExperts + kMoeMaxShared;

// What select leaves for the experts' kernels.
struct Units {
    int count, pad;
    int expert[kMaxUnits];
    int base[kMaxUnits];                   // first of the unit's rows of g, in token order
    u64 tokens[kMaxUnits];
};

constexpr int kRouterPieces = 16;

struct Layout {
    size_t logits, units, row_weight, g, partial, bytes;
};

// ------------------------------------------------------------- router ----
// logits[piece][t][e]: a workgroup takes 16 experts, 16 tokens and a piece of K, whose
// runs of 32 inputs its 4 waves share out; they join in LDS in order.  Lane (r, q) holds
// inputs 8 q .. 8 q + 7 of a run of expert r and of token r, one of them per product.
template <bool RF32>
__global__ __launch_bounds__(256) void router_kernel(Moe m, double *__restrict__ logits)
{
    __shared__ double red[4][256];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4, wave = threadIdx.x >> 6;
    const int e0 = blockIdx.x * 16, t0 = blockIdx.z * 16, runs = m.K >> 5;
    const int64_t er = (int64_t)min(e0 + r, m.E - 1) * m.K;
    const uint16_t *const xr = m.x + (int64_t)min(t0 + r, m.T - 1) * m.K;
    v4d acc = (v4d)(0.0);
    for (int i = blockIdx.y * 4 + wave; i < runs; i += 4 * gridDim.y) {
        const int k = i * 32 + q * 8;
        const uint4 u = *reinterpret_cast<const uint4 *>(xr + k);
        float xv[8] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y),
                       bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w)};
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
#pragma unroll
        for (int j = 0; j < 8; ++j)
            acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)wv[j], (double)xv[j], acc, 0, 0, 0);
    }
    // register i of lane (r, q): expert 4 i + q, token r
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][(4 * i + q) * 16 + r] = acc[i];
    __syncthreads();
    const int e = threadIdx.x & 15, t = threadIdx.x >> 4;
    if (e0 + e < m.E && t0 + t < m.T)
        logits[((int64_t)blockIdx.y * m.T + t0 + t) * m.E + e0 + e] =
            ((red[0][e * 16 + t] + red[1][e * 16 + t]) + red[2][e * 16 + t]) + red[3][e * 16 + t];
}

// ------------------------------------------------------------- select ----

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}
__device__ __forceinline__ double wave_max(double v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmax(v, __shfl_xor(v, o, 64));
    return v;
}
__device__ __forceinline__ u64 wave_max(u64 v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const u64 w = __shfl_xor(v, o, 64);
        v = w > v ? w : v;
    }
    return v;
}

// Doubles in the order of unsigned numbers; above 0 for every value, NaN as -infinity,
// -0 as +0.
__device__ __forceinline__ u64 order_of(double v)
{
    if (!(v == v)) v = -__builtin_inf();
    const u64 b = __builtin_bit_cast(u64, v + 0.0);
    return b >> 63 ? ~b : b | (1ull << 63);
}

// A wave takes one token after another, EP experts a lane (expert lane + 64 i).
template <int EP>
__global__ __launch_bounds__(1024) void select_kernel(Moe m, const double *__restrict__ logits,
                                                      int pieces, Units *__restrict__ units,
                                                      float *__restrict__ row_weight)
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
        double p[EP];
        u64 key[EP];
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            const int e = lane + 64 * i;
            p[i] = 0.0;
            if (e < m.E)
                for (int c = 0; c < pieces; ++c) p[i] += logits[((int64_t)c * m.T + t) * m.E + e];
        }
        double top = -__builtin_inf(), sum = 0.0;
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            const bool in = lane + 64 * i < m.E;
            key[i] = in ? order_of(p[i]) : 0;
            if (in) top = fmax(top, p[i]);
        }
        if (m.sigmoid) {
#pragma unroll
            for (int i = 0; i < EP; ++i) p[i] = 1.0 / (1.0 + exp(-p[i]));
        } else {
            top = wave_max(top);
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
        int id = 0;                              // lane j: the j-th choice
        double w = 0.0, total = 0.0;
        for (int j = 0; j < m.top_k; ++j) {
            u64 best = 0;
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
                s = __shfl(p[i], l, 64);
                if (lane == l) key[i] = 0;
            }
            total += s;
            if (lane == j) id = e, w = s;
        }
        if (lane < m.top_k) {
            if (m.renormalize) w = total == 0.0 ? 0.0 : w / total;
            const float f = (float)(w * m.factor);
            ids[t * m.top_k + lane] = id;
            wts[t * m.top_k + lane] = f;
            m.ids[t * m.top_k + lane] = id;
            m.weights[t * m.top_k + lane] = f;
            atomicOr(&tokens[id], 1ull << t);
        }
    }
    __syncthreads();

    // units: the chosen experts in order, their rows one after another
    const int e = threadIdx.x;
    const u64 mine = e < m.E ? tokens[e] : 0;
    const u64 active = __ballot(mine != 0);
    const int before = __popcll(active & ((1ull << lane) - 1));
    int rows = __popcll(mine);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(rows, o, 64);
        if (lane >= o) rows += up;
    }
    if (lane == 63) {
        wave_units[wave] = __popcll(active);
        wave_rows[wave] = rows;
    }
    __syncthreads();
    int u = before, base = rows - __popcll(mine), count = 0;
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
        row_weight[unit_base[x] + __popcll(tokens[x] & ((1ull << t) - 1))] = wts[i];
    }
    for (int i = threadIdx.x; i < m.S * m.T; i += 1024) row_weight[chosen + i] = 1.0f;
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
// blocks of K in turn, D at a time.  CT: tiles of 16 tokens.
template <int CT, int D>
__global__ __launch_bounds__(256) void gate_up_kernel(Moe m, const Units *__restrict__ units,
                                                      uint16_t *__restrict__ g, int64_t plane)
{
    extern __shared__ float red[];                 // [wave][2][CT][256]
    const int u = blockIdx.y;
    if (u >= units->count) return;
    const u64 tokens = units->tokens[u];
    const int expert = units->expert[u], base = units->base[u];
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int nkb = m.K >> 7, fb = blockIdx.x;
    const int in_tile = r * 64 + ((q ^ ((r >> 2) & 3)) << 4);
    const int64_t row_bytes = (int64_t)16 * m.K;
    const uint8_t *const codes = m.gate_up + (int64_t)expert * 2 * m.F * m.K + in_tile;
    const uint8_t *const gate = codes + fb * row_bytes, *const up = gate + (int64_t)m.F * m.K;
    const float *const sg = m.gate_up_scale +
                            ((int64_t)expert * (m.F >> 6) + (fb >> 3)) * nkb;
    const float *const su = sg + (int64_t)(m.F >> 7) * nkb;

    const uint16_t *col[CT];
    bool on[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int t = c * 16 + r;
        on[c] = (tokens >> t) & 1;
        col[c] = m.x + (int64_t)(on[c] ? t : 0) * m.K + q * 16;
    }
    v4f ag[CT], au[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) ag[c] = au[c] = (v4f)(0.0f);
    for (int k0 = wave; k0 < nkb; k0 += waves * D) {
        Block a[D], b[D];
        float fg[D], fu[D];
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int kb = k0 + d * waves;
            if (kb >= nkb) continue;
            a[d] = load_block(gate + kb * 2048);
            b[d] = load_block(up + kb * 2048);
            fg[d] = sg[kb];
            fu[d] = su[kb];
        }
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int kb = k0 + d * waves;
            if (kb >= nkb) continue;
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                if (CT > 1 && ((tokens >> (16 * c)) & 0xffff) == 0) continue;
                const Cols x = load_cols(col[c] + kb * 128, on[c]);
                const v4f pg = block_sum(a[d], x, (v4f)(0.0f));
                const v4f pu = block_sum(b[d], x, (v4f)(0.0f));
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
        *reinterpret_cast<v4f *>(red + ((wave * 2 + 0) * CT + c) * 256 + lane * 4) = ag[c];
        *reinterpret_cast<v4f *>(red + ((wave * 2 + 1) * CT + c) * 256 + lane * 4) = au[c];
    }
    __syncthreads();
    for (int c = wave; c < CT; c += waves) {
        v4f a = (v4f)(0.0f), b = (v4f)(0.0f);
        for (int k = 0; k < waves; ++k) {
            a += *reinterpret_cast<const v4f *>(red + ((k * 2 + 0) * CT + c) * 256 + lane * 4);
            b += *reinterpret_cast<const v4f *>(red + ((k * 2 + 1) * CT + c) * 256 + lane * 4);
        }
        const int t = c * 16 + r;
        if (!((tokens >> t) & 1)) continue;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i] / (1.0f + expf(-a[i])) * b[i];
        const int64_t row = base + __popcll(tokens & ((1ull << t) - 1));
        uint16_t *p = g + row * m.F + fb * 16 + q * 4;
        // the part that bf16 holds; with planes, what it leaves, twice more
        for (int part = 0;; ++part) {
            const uint2 o = make_uint2(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]));
            *reinterpret_cast<uint2 *>(p) = o;
            if (plane == 0 || part == 2) break;
            v[0] -= bf16_lo(o.x);
            v[1] -= bf16_hi(o.x);
            v[2] -= bf16_lo(o.y);
            v[3] -= bf16_hi(o.y);
            p += plane;
        }
    }
}

// y of 16 outputs: a workgroup's waves take (unit, block of F) pairs in turn, D at a
// time, of the units of its part (gridDim.y parts).  partial (or null): [part][T][K].
template <int CT, int D, int PLANES>
__global__ __launch_bounds__(1024) void down_kernel(Moe m, const Units *__restrict__ units,
                                                    const float *__restrict__ row_weight,
                                                    const uint16_t *__restrict__ g, int64_t plane,
                                                    float *__restrict__ partial)
{
    extern __shared__ float red[];                 // [wave][CT][256]
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int nkb = m.F >> 7, nb = blockIdx.x;
    const int count = units->count;
    const int u0 = count * blockIdx.y / gridDim.y, u1 = count * (blockIdx.y + 1) / gridDim.y;
    const int in_tile = r * 64 + ((q ^ ((r >> 2) & 3)) << 4);

    v4f acc[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c] = (v4f)(0.0f);
    const int items = (u1 - u0) * nkb;
    for (int i0 = wave; i0 < items; i0 += waves * D) {
        Block a[D];
        float f[D];
        int un[D], kbs[D];
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int i = i0 + d * waves;
            if (i >= items) continue;
            const int u = i / nkb;
            un[d] = u0 + u;
            kbs[d] = i - u * nkb;
            const int64_t e = units->expert[un[d]];
            a[d] = load_block(m.down + e * m.K * m.F + (int64_t)nb * 16 * m.F + kbs[d] * 2048 +
                              in_tile);
            f[d] = m.down_scale[(e * (m.K >> 7) + (nb >> 3)) * nkb + kbs[d]];
        }
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (i0 + d * waves >= items) continue;
            const u64 tokens = units->tokens[un[d]];
            const int base = units->base[un[d]];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                if (CT > 1 && ((tokens >> (16 * c)) & 0xffff) == 0) continue;
                const int t = c * 16 + r;
                const bool on = (tokens >> t) & 1;
                const int64_t row = on ? base + __popcll(tokens & ((1ull << t) - 1)) : 0;
                const uint16_t *p = g + row * m.F + kbs[d] * 128 + q * 16;
                const float w = on ? row_weight[row] * f[d] : 0.0f;
                v4f s = (v4f)(0.0f);
#pragma unroll
                for (int k = 0; k < PLANES; ++k) s = block_sum(a[d], load_cols(p + k * plane, on), s);
                // a token that did not choose the expert takes nothing of it, codes of NaN
                // included
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    acc[c][k] = on ? __builtin_fmaf(s[k], w, acc[c][k]) : acc[c][k];
            }
        }
    }
#pragma unroll
    for (int c = 0; c < CT; ++c)
        *reinterpret_cast<v4f *>(red + (wave * CT + c) * 256 + lane * 4) = acc[c];
    __syncthreads();
    for (int c = wave; c < CT; c += waves) {
        v4f v = (v4f)(0.0f);
        for (int k = 0; k < waves; ++k)
            v += *reinterpret_cast<const v4f *>(red + (k * CT + c) * 256 + lane * 4);
        const int t = c * 16 + r;
        if (t >= m.T) continue;
        const int64_t o = (int64_t)t * m.K + nb * 16 + q * 4;
        if (partial)
            *reinterpret_cast<v4f *>(partial + (int64_t)blockIdx.y * m.T * m.K + o) = v;
        else if (m.y_f32)
            *reinterpret_cast<v4f *>(static_cast<float *>(m.y) + o) = v;
        else
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(m.y) + o) =
                make_uint2(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]));
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
    l.row_weight = l.units + up(sizeof(Units));
    l.g = l.row_weight + up(rows * 4);
    l.partial = l.g + up(3 * rows * F * 2);
    l.bytes = l.partial + up((size_t)kMaxParts * T * K * 4);
    return l;
}

template <int CT> hipError_t launch_experts(const Moe &m, const Layout &l, hipStream_t stream)
{
    char *const ws = static_cast<char *>(m.ws);
    const Units *units = reinterpret_cast<const Units *>(ws + l.units);
    const float *row_weight = reinterpret_cast<const float *>(ws + l.row_weight);
    uint16_t *g = reinterpret_cast<uint16_t *>(ws + l.g);
    const int most = std::min(m.T * m.top_k, m.E) + m.S;
    const int64_t plane = m.y_f32 ? (int64_t)m.T * (m.top_k + m.S) * m.F : 0;
    constexpr int GW = 4, DW = 8, D = CT == 1 ? 4 : 2;
    hipLaunchKernelGGL((gate_up_kernel<CT, D>), dim3(m.F / 16, most), dim3(64 * GW),
                       GW * 2 * CT * 1024, stream, m, units, g, plane);
    const int blocks = m.K / 16;
    const int parts = std::max(1, std::min({kMaxParts, most, 1024 / blocks}));
    float *const partial = parts > 1 ? reinterpret_cast<float *>(ws + l.partial) : nullptr;
    auto down = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(blocks, parts), dim3(64 * DW), DW * CT * 1024, stream, m,
                           units, row_weight, g, plane, partial);
    };
    if (m.y_f32) down(down_kernel<CT, 2, 3>);
    else down(down_kernel<CT, D, 1>);
    if (parts > 1) {
        const int64_t n = (int64_t)m.T * m.K;
        hipLaunchKernelGGL(join_parts_kernel, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0,
                           stream, partial, parts, n, m.y, m.y_f32);
    }
    return hipGetLastError();
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
    float *const row_weight = reinterpret_cast<float *>(ws + l.row_weight);
    const int pieces = std::min(kRouterPieces, (m.K / 32 + 3) / 4);
    const dim3 grid((m.E + 15) / 16, pieces, (m.T + 15) / 16);
    if (m.router_f32)
        hipLaunchKernelGGL(router_kernel<true>, grid, dim3(256), 0, stream, m, logits);
    else
        hipLaunchKernelGGL(router_kernel<false>, grid, dim3(256), 0, stream, m, logits);
    auto select = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(1), dim3(1024), 0, stream, m, logits, pieces, units,
                           row_weight);
    };
    if (m.E <= 128) select(select_kernel<2>);
    else if (m.E <= 256) select(select_kernel<4>);
    else select(select_kernel<8>);
    if (m.T <= 16) return launch_experts<1>(m, l, stream);
    if (m.T <= 32) return launch_experts<2>(m, l, stream);
    return launch_experts<4>(m, l, stream);
}

} // namespace convrot
