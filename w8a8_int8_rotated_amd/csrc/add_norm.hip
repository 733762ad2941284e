// The residual's addition and the RMS norm in front of a projection, and their
// backward pass, in one pass over the rows (gfx950).
//
//   forward:   h = x + r;  q = rsqrt(mean(h^2) + eps);  n = (h q) w
//              out: n (bf16 or fp32), or the codes that the INT8 or the FP8 linear
//              multiplies: v = H_b n, amax, rint(v 127 / amax); or per 128 channels
//              e4m3(n / s)
//   backward:  t = g w;  dh = gh + q (t - h q mean(t h q));  dw = sum_m g h q
//
// Bound: memory.  Every row is read once and every result written once; h is held
// in registers between its sum of squares and its use.  All arithmetic is fp32; h is
// rounded to its own type first and everything after uses the rounded value, so the
// norm of a stored h gives the same bits.  8-bit outputs are quantised from the fp32
// n, without a rounding to bf16 in between.
//
// Measured (us; K = 5376, bf16 rows beside an fp32 residual stream): 38656 rows forward 414
// (6.0 TB/s of 12 bytes a channel), to INT8 codes 411 (5.6 TB/s), backward with bf16
// gradients and dx 582 (5.7 TB/s of 16 bytes); 5 rows 3.5, a launch's length.  Rows of more
// than 16384 channels take 8 (forward) or 4 (backward) steps a wave in the 128 registers that
// 1024 threads leave a lane; fp32 rows forward and every backward keep 40 to 68 bytes of them in
// scratch (8192 rows of 32768, fp32: forward 863, 5.0 TB/s of 16 bytes, backward 833, 5.2; of 16384,
// without: 367 and 375, 5.8).
#include "add_norm.hpp"

#include "fp8_common.hpp"
#include "rotate.hpp"

#include <algorithm>
#include <type_traits>

namespace convrot {
namespace {

// an element offset beyond every range used here, whose byte offset still fits 32 bits
constexpr uint32_t kPast = 0x1fc00000u;
constexpr uint32_t kOut = 4 * kPast;

// 8 channels as loaded, bf16 or fp32: 4 from element e0 and 4 from e1 of a range.  RUNS: e1
// is anywhere (neighbouring lanes then hold neighbouring runs, so that loads of fp32 rows
// cover whole cache lines); otherwise e1 = e0 + 4.  AUX: the cache policy (2: past the caches).
template <bool F32> struct Raw {
    v4i u[F32 ? 2 : 1];
};

template <bool F32, bool RUNS, int AUX>
__device__ __forceinline__ Raw<F32> load8(__amdgpu_buffer_rsrc_t rows, uint32_t e0, uint32_t e1)
{
    Raw<F32> r;
    if constexpr (F32) {
        r.u[0] = __builtin_amdgcn_raw_buffer_load_b128(rows, (int)(e0 * 4), 0, AUX);
        r.u[1] = __builtin_amdgcn_raw_buffer_load_b128(rows, (int)(e1 * 4), 0, AUX);
    } else if constexpr (RUNS) {
        const v2i a = __builtin_amdgcn_raw_buffer_load_b64(rows, (int)(e0 * 2), 0, AUX);
        const v2i b = __builtin_amdgcn_raw_buffer_load_b64(rows, (int)(e1 * 2), 0, AUX);
        r.u[0] = (v4i){a[0], a[1], b[0], b[1]};
    } else {
        r.u[0] = __builtin_amdgcn_raw_buffer_load_b128(rows, (int)(e0 * 2), 0, AUX);
    }
    return r;
}

template <bool RUNS, int AUX, bool F32>
__device__ __forceinline__ void store8(const Raw<F32> &r, __amdgpu_buffer_rsrc_t rows, uint32_t e0,
                                       uint32_t e1)
{
    if constexpr (F32) {
        __builtin_amdgcn_raw_buffer_store_b128(r.u[0], rows, (int)(e0 * 4), 0, AUX);
        __builtin_amdgcn_raw_buffer_store_b128(r.u[1], rows, (int)(e1 * 4), 0, AUX);
    } else if constexpr (RUNS) {
        const v4i u = r.u[0];
        __builtin_amdgcn_raw_buffer_store_b64((v2i){u[0], u[1]}, rows, (int)(e0 * 2), 0, AUX);
        __builtin_amdgcn_raw_buffer_store_b64((v2i){u[2], u[3]}, rows, (int)(e1 * 2), 0, AUX);
    } else {
        __builtin_amdgcn_raw_buffer_store_b128(r.u[0], rows, (int)(e0 * 2), 0, AUX);
    }
}

template <bool F32> __device__ __forceinline__ void widen(const Raw<F32> &r, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (F32) {
            v[j] = __int_as_float(r.u[0][j]);
            v[4 + j] = __int_as_float(r.u[1][j]);
        } else {
            v[2 * j] = bf16_lo((uint32_t)r.u[0][j]);
            v[2 * j + 1] = bf16_hi((uint32_t)r.u[0][j]);
        }
    }
}

template <bool F32> __device__ __forceinline__ Raw<F32> narrow(const float (&v)[8])
{
    Raw<F32> r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (F32) {
            r.u[0][j] = __float_as_int(v[j]);
            r.u[1][j] = __float_as_int(v[4 + j]);
        } else {
            r.u[0][j] = (int)cvt_pk_bf16(v[2 * j], v[2 * j + 1]);
        }
    }
    return r;
}

// Sum and maximum over a half-wave.  The maximum keeps a NaN (v_maximum3_f32): a weight of NaN
// makes a NaN of its whole block, and a maximum that dropped it would leave the row a finite
// scale and codes of 0.
#define CR_DPP(v, CTRL)                                                                           \
    __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true))
__device__ __forceinline__ float half_sum(float v)
{
    v += CR_DPP(v, 0xB1);
    v += CR_DPP(v, 0x4E);
    v += CR_DPP(v, 0x141);
    v += CR_DPP(v, 0x140);
    return v + __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401F));
}
__device__ __forceinline__ float max_or_nan(float a, float b)
{
    return __builtin_elementwise_maximum(a, b);
}
__device__ __forceinline__ float half_max(float v)
{
    v = max_or_nan(v, CR_DPP(v, 0xB1));
    v = max_or_nan(v, CR_DPP(v, 0x4E));
    v = max_or_nan(v, CR_DPP(v, 0x141));
    v = max_or_nan(v, CR_DPP(v, 0x140));
    return max_or_nan(v, __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401F)));
}

// Outputs of the forward kernel: rows, e4m3 codes, or INT8 codes of blocks of b
// channels (b, or b + 1 for the regular rotation).
constexpr int kRows = 0, kFp8 = 2;

// Two rows a wave, one per half-wave: a wave step is 256 channels of both, 8 a lane,
// so that a store of codes covers whole cache lines of the K-tiled layout (two rows
// of a 16-row block are neighbours in it).  A pair of rows is split over W waves of
// at most SPR steps; a workgroup holds blockDim / 64 / W pairs.
template <bool XF, bool RF, int MODE, int SPR, int AUX>
__global__ __launch_bounds__(1024) void add_norm_kernel(AddNorm a, int W)
{
    constexpr bool RUNS = MODE == kRows && RF;
    constexpr bool I8 = MODE != kRows && MODE != kFp8;
    constexpr int B = I8 ? MODE & ~1 : 64, ROT = I8 ? MODE & 1 : 0, LPB = B / 8;
    constexpr int NSTAGE = B == 64 ? 3 : B == 128 ? 4 : 5;
    constexpr int XS = XF ? 4 : 2, RS = RF ? 4 : 2;
    __shared__ float red[2][16][2];

    const int lane = threadIdx.x & 63, half = lane >> 5, hl = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int grp = wave / W, part = wave - grp * W, pairs = waves / W;
    const int K = a.K, steps = (K + 255) >> 8;
    const int mine = (steps - part + W - 1) / W;     // steps of this wave
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t row0 = 2 * (block * pairs + grp), row = row0 + half;
    const int64_t first = row0 < a.M ? row0 : 0;
    const int rows = row0 < a.M ? (int)min(a.M - row0, (int64_t)2) : 0;
    const bool in = row < a.M;
    const int chunk = I8 ? chunk_of_lane(hl % LPB) : 0;
    const int lane_off = I8 ? (hl / LPB) * B + chunk * 8 : hl * (RUNS ? 4 : 8);
    const int run = RUNS ? 128 : 4;                  // from the lane's first run to the second
    // this lane's element in step t, of a pair of rows and of one row (kPast past the end)
    auto element = [&](int t) { return ((part + W * t) << 8) + lane_off; };
    auto at = [&](int t, int o) -> uint32_t {
        const int e = element(t) + o;
        return in && e < K ? (uint32_t)(half * K + e) : kPast;
    };
    auto range = [&](const void *p, int es) {
        return row_rsrc(static_cast<const char *>(p) + first * K * es, rows * K * es);
    };

    const bool add = a.r != nullptr;
    Raw<XF> xr[SPR];
    Raw<RF> rr[SPR];
    {
        const __amdgpu_buffer_rsrc_t xs = range(a.x, XS);
#pragma unroll
        for (int t = 0; t < SPR; ++t)
            if (t < mine) xr[t] = load8<XF, RUNS, AUX>(xs, at(t, 0), at(t, run));
    }
    if (add) {
        const __amdgpu_buffer_rsrc_t rs = range(a.r, RS);
#pragma unroll
        for (int t = 0; t < SPR; ++t)
            if (t < mine) rr[t] = load8<RF, RUNS, AUX>(rs, at(t, 0), at(t, run));
    }
    // the weights of this lane's channels, requested with the rows
    const __amdgpu_buffer_rsrc_t ws = row_rsrc(a.w ? a.w : a.x, a.w ? K * 4 : 0);
    auto load_w = [&](int t) {
        const int e = element(t);
        return load8<true, RUNS, 0>(ws, e < K ? (uint32_t)e : kPast,
                                    e + run < K ? (uint32_t)(e + run) : kPast);
    };
    constexpr bool EARLY = SPR <= 4;
    Raw<true> wr[EARLY ? SPR : 1];
    if constexpr (EARLY) {
#pragma unroll
        for (int t = 0; t < SPR; ++t)
            if (t < mine) wr[t] = load_w(t);
    }

    float v[SPR][8], part_sum[2] = {};
    const __amdgpu_buffer_rsrc_t hs = range(add ? a.h : a.x, add ? RS : 0);
#pragma unroll
    for (int t = 0; t < SPR; ++t) {
        if (t >= mine) continue;
        widen<XF>(xr[t], v[t]);
        if (add) {
            float r[8];
            widen<RF>(rr[t], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[t][j] += r[j];
            const Raw<RF> h = narrow<RF>(v[t]);
            store8<RUNS, AUX>(h, hs, at(t, 0), at(t, run));
            widen<RF>(h, v[t]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            part_sum[j / 4] = __builtin_fmaf(v[t][j], v[t][j], part_sum[j / 4]);
    }
    // one tree over the runs of 4 channels, whichever lane holds which: every output form
    // of the same rows has the same bits
    float sum = RUNS ? half_sum(part_sum[0]) + half_sum(part_sum[1])
                     : half_sum(part_sum[0] + part_sum[1]);
    if (W > 1) {
        if (hl == 0) red[0][wave][half] = sum;
        __syncthreads();
        sum = 0.0f;
        for (int k = 0; k < W; ++k) sum += red[0][grp * W + k][half];
    }
    const float q = rsqrtf(sum / (float)K + a.eps);
#pragma unroll
    for (int t = 0; t < SPR; ++t) {
        if (t >= mine) continue;
        float w[8];
        widen<true>(EARLY ? wr[EARLY ? t : 0] : load_w(t), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[t][j] = (v[t][j] * q) * (a.w ? w[j] : 1.0f);
    }

    if constexpr (MODE == kRows) {
        if (a.y_f32) {
            const __amdgpu_buffer_rsrc_t ys = range(a.y, 4);
#pragma unroll
            for (int t = 0; t < SPR; ++t)
                if (t < mine) store8<RUNS, AUX>(narrow<true>(v[t]), ys, at(t, 0), at(t, run));
        } else {
            const __amdgpu_buffer_rsrc_t ys = range(a.y, 2);
#pragma unroll
            for (int t = 0; t < SPR; ++t)
                if (t < mine) store8<RUNS, AUX>(narrow<false>(v[t]), ys, at(t, 0), at(t, run));
        }
        return;
    }
    // codes: the pair's 16-row block of the K-tiled layout; a step is 4 KiB of it
    const __amdgpu_buffer_rsrc_t qs =
        row_rsrc(a.q + (first & ~int64_t(15)) * K, rows ? 16 * K : 0);
    const uint32_t q_off = (uint32_t)tiled_offset(row & 15, lane_off, K);
    auto store_codes = [&](int t, int lo, int hi) {
        __builtin_amdgcn_raw_buffer_store_b64(
            (v2i){lo, hi}, qs, in && element(t) < K ? (int)((part + W * t) * 4096 + q_off) : (int)kOut, 0,
            0);
    };
    if constexpr (MODE == kFp8) {
        const int64_t Mp = padded_rows(a.M);
#pragma unroll
        for (int t = 0; t < SPR; ++t) {
            if (t >= mine) continue;
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[t][j]));
            float s, inv;
            block_scale(max16(m), a.pow2, s, inv);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[t][j] *= inv;
            store_codes(t, cvt_e4m3x4(v[t][0], v[t][1], v[t][2], v[t][3]),
                        cvt_e4m3x4(v[t][4], v[t][5], v[t][6], v[t][7]));
            const int kb = (part + W * t) * 2 + (hl >> 4);
            if ((hl & 15) == 0 && in && kb * 128 < K) a.s[kb * Mp + row] = s;
        }
    }
    if constexpr (I8) {
        float csign[NSTAGE], m = 0.0f;
#pragma unroll
        for (int k = 0; k < NSTAGE; ++k) csign[k] = ((chunk >> k) & 1) ? -1.0f : 1.0f;
#pragma unroll
        for (int t = 0; t < SPR; ++t) {
            if (t >= mine) continue;
            rotate_chunk<B, ROT>(v[t], csign);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max_or_nan(m, fabsf(v[t][j]));
        }
        m = half_max(m);
        if (W > 1) {
            if (hl == 0) red[1][wave][half] = m;
            __syncthreads();
            m = 0.0f;
            for (int k = 0; k < W; ++k) m = max_or_nan(m, red[1][grp * W + k][half]);
        }
        const float inv = m > 0.0f ? __fdiv_rn(127.0f, m) : 0.0f;
        // the Sylvester sign trick leaves the upper lanes' values negated
        const float invs = ROT == 0 && (__builtin_popcount(chunk) & 1) ? -inv : inv;
        // a row that is not finite gets a scale of NaN (infinities of n alone an infinite one:
        // infinity times the codes' 0), and so NaN outputs
        if (part == 0 && hl == 0 && in)
            a.s[row] = sum < __builtin_inff() ? __fmul_rn(__fdiv_rn(m, 127.0f), a.inv_sqrt_b)
                                              : __builtin_nanf("");
#pragma unroll
        for (int t = 0; t < SPR; ++t) {
            if (t >= mine) continue;
            const uint2 c = quantise_chunk(v[t], invs);
            store_codes(t, (int)c.x, (int)c.y);
        }
    }
}

// Rows out and backward: a call that moves more than the last-level cache holds reads and
// writes past the caches (AUX = 2).  us without and with that, K = 5376, bf16 rows and
// residual, bf16 rows and fp32 residual:
//   forward   3121 rows  23.9  26.6   36.2  37.0;   6242  49.4  49.1    76.8  69.8;
//            24966       195   183    285   268
//   backward  3121       31.1  36.2   47.9  50.9;   6242  60.6  61.8   105    94;
//            24966       222   218    408   376
// Codes gain nothing (38656 rows to INT8: 411, 436): an fp32 residual is read there in
// pieces of 16 of every 32 bytes, the other half from the caches.
constexpr int64_t kPastCaches = (int64_t)1 << 28;

template <bool XF, bool RF, int MODE>
void launch_steps(const AddNorm &a, hipStream_t stream)
{
    const int steps = (a.K + 255) / 256;
    const int spr = steps <= 32 ? 2 : steps <= 64 ? 4 : 8;
    const int W = (steps + spr - 1) / spr, pairs = std::max(1, 4 / W);
    // a grid dimension holds less than 2^32 threads
    const int64_t blocks = (a.M + 2 * pairs - 1) / (2 * pairs), kWide = 1 << 21;
    const dim3 grid((unsigned)std::min(blocks, kWide), (unsigned)((blocks + kWide - 1) / kWide));
    const dim3 block(64 * W * pairs);
    auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, W); };
    if (spr == 2) {
        const int bytes = (XF ? 4 : 2) + (a.r ? RF ? 8 : 4 : 0) + (a.y_f32 ? 4 : 2);
        if (MODE == kRows && a.M * a.K * bytes >= kPastCaches)
            launch(add_norm_kernel<XF, RF, MODE, 2, MODE == kRows ? 2 : 0>);
        else
            launch(add_norm_kernel<XF, RF, MODE, 2, 0>);
    } else if (spr == 4) launch(add_norm_kernel<XF, RF, MODE, 4, 0>);
    else launch(add_norm_kernel<XF, RF, MODE, 8, 0>);
}

template <int MODE> void launch_types(const AddNorm &a, hipStream_t stream)
{
    if (a.x_f32) launch_steps<true, true, MODE>(a, stream);
    else if (a.r_f32) launch_steps<false, true, MODE>(a, stream);
    else launch_steps<false, false, MODE>(a, stream);
}

// Backward.  A wave step is 512 channels of one row, 8 a lane in two runs of 4.  A row is
// split over W waves of at most SPR steps; a workgroup holds `pairs` rows at a time and
// walks the rows, the next one's loads on their way while it finishes the last, and keeps
// its sums of dw in registers.
constexpr int kGradStep = 512;

// LEAN (rows of many steps a wave): no loads ahead, gh and w read where they are
// needed; the registers hold g, h and dw (with four steps 10 to 16 of them are spilled).
template <bool GF, bool HF, int SPR, int AUX>
__global__ __launch_bounds__(1024) void add_norm_grad_kernel(AddNormGrad a, int W)
{
    constexpr int GS = GF ? 4 : 2, HS = HF ? 4 : 2;
    constexpr bool LEAN = SPR > 1;
    __shared__ float red[2][2][16];
    extern __shared__ float sums[];                  // [pairs][K] (pairs > 1)

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int grp = wave / W, part = wave - grp * W, pairs = waves / W;
    const int K = a.K, steps = (K + kGradStep - 1) / kGradStep;
    const int mine = (steps - part + W - 1) / W;
    const float invK = 1.0f / (float)K;

    uint32_t e0[SPR], e1[SPR];
    float dw[SPR][8], wk[LEAN ? 1 : SPR][8];
    const __amdgpu_buffer_rsrc_t ws = row_rsrc(a.w ? a.w : a.h, a.w ? K * 4 : 0);
    auto load_w = [&](int t, float (&w)[8]) {
        widen<true>(load8<true, true, 0>(ws, e0[t], e1[t]), w);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (!a.w) w[j] = 1.0f;
    };
#pragma unroll
    for (int t = 0; t < SPR; ++t) {
        const uint32_t e = (uint32_t)((part + W * t) * kGradStep + lane * 4);
        e0[t] = e < (uint32_t)K ? e : kPast;
        e1[t] = e + 256 < (uint32_t)K ? e + 256 : kPast;
        if constexpr (!LEAN) load_w(t, wk[t]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[t][j] = 0.0f;
    }

    Raw<GF> g[SPR];
    Raw<HF> h[SPR], gh[LEAN ? 1 : SPR];
    const bool more = a.gh != nullptr;
    auto row_of = [&](const void *p, int64_t row, int es) {
        const bool in = row < a.M;
        return row_rsrc(static_cast<const char *>(p) + (in ? row : 0) * K * es, in ? K * es : 0);
    };
    auto issue = [&](int64_t row) {
        const __amdgpu_buffer_rsrc_t gs = row_of(a.g, row, GS), hs = row_of(a.h, row, HS);
#pragma unroll
        for (int t = 0; t < SPR; ++t)
            if (t < mine) h[t] = load8<HF, true, AUX>(hs, e0[t], e1[t]);
#pragma unroll
        for (int t = 0; t < SPR; ++t)
            if (t < mine) g[t] = load8<GF, true, AUX>(gs, e0[t], e1[t]);
        if constexpr (!LEAN) {
            if (!more) return;
            const __amdgpu_buffer_rsrc_t ms = row_of(a.gh, row, HS);
#pragma unroll
            for (int t = 0; t < SPR; ++t)
                if (t < mine) gh[t] = load8<HF, true, AUX>(ms, e0[t], e1[t]);
        }
    };

    const int64_t stride = (int64_t)gridDim.x * pairs;
    int64_t row = (int64_t)blockIdx.x * pairs + grp;
    if constexpr (!LEAN) issue(row);
    int par = 0;
    // every group of the workgroup makes the same number of passes (rows past M are empty)
    for (int64_t base = (int64_t)blockIdx.x * pairs; base < a.M;
         base += stride, row += stride, par ^= 1) {
        if constexpr (LEAN) issue(row);
        Raw<GF> gc[SPR];
        Raw<HF> hc[SPR], mc[LEAN ? 1 : SPR];
#pragma unroll
        for (int t = 0; t < SPR; ++t) {
            gc[t] = g[t];
            hc[t] = h[t];
            if constexpr (!LEAN) mc[t] = gh[t];
        }
        if constexpr (!LEAN) issue(row + stride);
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int t = 0; t < SPR; ++t) {
            if (t >= mine) continue;
            float hv[8], gv[8], w[8];
            widen<HF>(hc[t], hv);
            widen<GF>(gc[t], gv);
            if constexpr (LEAN) load_w(t, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s1 = __builtin_fmaf(hv[j], hv[j], s1);
                s2 = __builtin_fmaf(gv[j] * (LEAN ? w[j] : wk[LEAN ? 0 : t][j]), hv[j], s2);
            }
        }
        s1 = half_sum(s1);
        s2 = half_sum(s2);
        s1 += __shfl_xor(s1, 32, 64);
        s2 += __shfl_xor(s2, 32, 64);
        if (W > 1) {
            if (lane == 0) {
                red[par][0][wave] = s1;
                red[par][1][wave] = s2;
            }
            __syncthreads();
            s1 = s2 = 0.0f;
            for (int k = 0; k < W; ++k) {
                s1 += red[par][0][grp * W + k];
                s2 += red[par][1][grp * W + k];
            }
        }
        const float q = rsqrtf(s1 * invK + a.eps);
        // (through h q, which is bounded: q^3 need not be finite)
        const float c = (s2 * invK) * q;
        const __amdgpu_buffer_rsrc_t ds = row_of(a.dh, row, HS);
        const __amdgpu_buffer_rsrc_t xs = a.dx ? row_of(a.dx, row, 2) : row_rsrc(a.dh, 0);
        const __amdgpu_buffer_rsrc_t ms = row_of(more ? a.gh : a.h, row, HS);
#pragma unroll
        for (int t = 0; t < SPR; ++t) {
            if (t >= mine) continue;
            float hv[8], gv[8], m[8], w[8], d[8];
            widen<HF>(hc[t], hv);
            widen<GF>(gc[t], gv);
            if constexpr (LEAN) {
                load_w(t, w);
                if (more) widen<HF>(load8<HF, true, AUX>(ms, e0[t], e1[t]), m);
            } else if (more) {
                widen<HF>(mc[t], m);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float hq = hv[j] * q;
                dw[t][j] = __builtin_fmaf(gv[j], hq, dw[t][j]);
                d[j] = q * __builtin_fmaf(-hq, c, gv[j] * (LEAN ? w[j] : wk[LEAN ? 0 : t][j]));
                if (more) d[j] += m[j];
            }
            store8<true, AUX>(narrow<HF>(d), ds, e0[t], e1[t]);
            if (HF && a.dx) store8<true, AUX>(narrow<false>(d), xs, e0[t], e1[t]);
        }
    }
    if (!a.dw) return;
    // this workgroup's sums: its groups joined in order
    const __amdgpu_buffer_rsrc_t out =
        row_rsrc(a.partial + (int64_t)blockIdx.x * K, K * 4);
    if (pairs == 1) {
#pragma unroll
        for (int t = 0; t < SPR; ++t)
            if (t < mine) store8<true, 0>(narrow<true>(dw[t]), out, e0[t], e1[t]);
        return;
    }
#pragma unroll
    for (int t = 0; t < SPR; ++t) {
        if (t >= mine) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t e = (j < 4 ? e0[t] : e1[t]) + (j & 3);
            if (e < (uint32_t)K) sums[grp * K + e] = dw[t][j];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < K; i += blockDim.x) {
        float s = 0.0f;
        for (int k = 0; k < pairs; ++k) s += sums[k * K + i];
        a.partial[(int64_t)blockIdx.x * K + i] = s;
    }
}

// dw = the sum of `rows` partial rows, in fp64 and in a fixed order: a workgroup takes
// 16 columns, its 64 thread rows every 64th partial row, four loads at a time; then
// halves are joined in LDS.
__global__ __launch_bounds__(1024) void join_kernel(const float *__restrict__ partial, int rows,
                                                    int K, float *__restrict__ dw)
{
    __shared__ double sum[64][16];
    const int c = threadIdx.x & 15, k = threadIdx.x >> 4;
    const int col = blockIdx.x * 16 + c;
    double v = 0.0;
    for (int i = k; i < rows; i += 256) {
        float x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            x[u] = i + 64 * u < rows && col < K ? partial[(int64_t)(i + 64 * u) * K + col] : 0.0f;
        v += ((double)x[0] + (double)x[1]) + ((double)x[2] + (double)x[3]);
    }
    sum[k][c] = v;
    for (int h = 32; h > 0; h >>= 1) {
        __syncthreads();
        if (k < h) sum[k][c] += sum[k + h][c];
    }
    if (k == 0 && col < K) dw[col] = (float)sum[0][c];
}

struct GradShape {
    int spr, W, pairs;
    int64_t grid;
};

GradShape grad_shape(int64_t M, int64_t K)
{
    GradShape g;
    const int steps = (int)((K + kGradStep - 1) / kGradStep);
    g.spr = steps <= 16 ? 1 : steps <= 32 ? 2 : 4;
    g.W = (steps + g.spr - 1) / g.spr;
    g.pairs = std::max(1, 4 / g.W);
    // workgroups: what the CUs hold at once, and few enough that the partial sums stay
    // small beside the rows
    const int64_t rows = (M + g.pairs - 1) / g.pairs;
    const int64_t held = 256 * std::max(1, 16 / (g.W * g.pairs));
    g.grid = std::min(held, std::max<int64_t>((rows + 5) / 6, std::min<int64_t>(rows, 64)));
    return g;
}

} // namespace

hipError_t launch_add_norm(NormOut out, const AddNorm &a, hipStream_t stream)
{
    if (a.M == 0) return hipSuccess;
    if (out == NormOut::ROWS) launch_types<kRows>(a, stream);
    else if (out == NormOut::FP8) launch_types<kFp8>(a, stream);
    else if (a.block == 64)
        a.regular ? launch_types<65>(a, stream) : launch_types<64>(a, stream);
    else if (a.block == 128) launch_types<128>(a, stream);
    else a.regular ? launch_types<257>(a, stream) : launch_types<256>(a, stream);
    return hipGetLastError();
}

int64_t add_norm_partial_rows(int64_t M, int64_t K) { return grad_shape(M, K).grid; }

hipError_t launch_add_norm_grad(const AddNormGrad &a, hipStream_t stream)
{
    const GradShape g = grad_shape(a.M, a.K);
    if (g.grid > 0) {
        const dim3 grid((unsigned)g.grid), block(64 * g.W * g.pairs);
        const size_t lds = g.pairs > 1 ? (size_t)g.pairs * a.K * 4 : 0;
        auto launch = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, grid, block, lds, stream, a, g.W);
        };
        auto types = [&](auto spr) {
            constexpr int S = decltype(spr)::value;
            auto past = [&](auto aux) {
                constexpr int A = decltype(aux)::value;
                if (a.g_f32) a.h_f32 ? launch(add_norm_grad_kernel<true, true, S, A>)
                                     : launch(add_norm_grad_kernel<true, false, S, A>);
                else a.h_f32 ? launch(add_norm_grad_kernel<false, true, S, A>)
                             : launch(add_norm_grad_kernel<false, false, S, A>);
            };
            const int bytes = (a.g_f32 ? 4 : 2) + (a.h_f32 ? 4 : 2) * (a.gh ? 3 : 2) + (a.dx ? 2 : 0);
            if (a.M * a.K * bytes >= kPastCaches) past(std::integral_constant<int, 2>{});
            else past(std::integral_constant<int, 0>{});
        };
        if (g.spr == 1) types(std::integral_constant<int, 1>{});
        else if (g.spr == 2) types(std::integral_constant<int, 2>{});
        else types(std::integral_constant<int, 4>{});
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.dw)
        hipLaunchKernelGGL(join_kernel, dim3((unsigned)((a.K + 15) / 16)), dim3(1024), 0, stream,
                           a.partial, (int)g.grid, a.K, a.dw);
    return hipGetLastError();
}

} // namespace convrot
