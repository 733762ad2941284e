// FP8 (e4m3) block-scaled linear for gfx950: quantisation of weights and rows,
// and the product for few rows.  (The large product is in gemm_fp8.hip.)
//
//   s = max(amax / 448, 2^-126) over a block, 0 if amax is 0 (POW2: rounded up
//   to a power of two);  q = e4m3(x * (1 / s)).
//   y[m, n] = sum_b (sum_{k in b} qx[m, k] qw[n, k]) (sx[b, m] sw[n / 128, b])
//
// Codes are K-tiled like the INT8 ones (common.hpp), so one 128-input block of
// 16 rows is two consecutive 1 KiB tiles: exactly the operand of one
// v_mfma_f32_16x16x128_f8f6f4, 32 bytes per lane.  Which 32 of the 128 inputs a
// lane holds does not matter as long as both operands agree; lane (r, g) takes
// chunk g of either tile, so each of its two loads is part of a contiguous 1 KiB.
//
// Precision of the sums.  The FP8 matrix instructions of gfx950 (those with
// K = 32 give the same results) add the products of 8 consecutive inputs at a
// common exponent: each is cut to a multiple of 2^-13 of the power of two of the
// largest one, and only the groups' sums are added in fp32 (measured with single
// products: 2^16 + 2^3 is exact inside a group, 2^16 + 2^2 gives 2^16; across
// groups 2^16 + 2^-7 is exact).  On Gaussian codes that is 2e-6 of the sum of
// magnitudes (rms).  bf16 outputs use them, at twice the rate of the bf16
// instructions: beside their own rounding (1.66e-3 of the outputs' rms) the cut does
// not show in the total error, which stays 1.66e-3.  It does show in single outputs
// whose terms cancel: at K = 5376, 1.2% of the outputs are not the bf16 value nearest
// to the exact sum (2.6%, and 3.3% with power-of-two scales, where 1% of the channels
// are 30 times larger; fp32 sums 0.01%), 0.2% (0.5%, 0.6%) are off by more than one
// unit and 0.1% (0.2%, 0.3%) by more than 1% of their small value.  F32 outputs
// convert the codes to bf16, which holds every e4m3 value, and use
// v_mfma_f32_16x16x32_bf16, whose sums keep 24 bits throughout (1e-7 of the outputs'
// rms).
#include "fp8_common.hpp"

#include <algorithm>

namespace convrot {
namespace {

// One 128 x 128 block of the weight per workgroup (load time only): thread t
// holds 64 consecutive inputs of row t / 2.
template <typename T>
__global__ __launch_bounds__(256) void block_weights_kernel(const T *__restrict__ W, int N, int K,
                                                            bool pow2,
                                                            uint8_t *__restrict__ codes,
                                                            float *__restrict__ scale)
{
    __shared__ float red[4];
    const int n = blockIdx.x * 128 + (threadIdx.x >> 1);
    const int k0 = blockIdx.y * 128 + (threadIdx.x & 1) * 64;
    const bool live = n < N;
    auto at = [&](int i) -> float {
        if constexpr (sizeof(T) == 4) return W[(int64_t)n * K + k0 + i];
        else return __uint_as_float((uint32_t)W[(int64_t)n * K + k0 + i] << 16);
    };
    float amax = 0.0f;
    for (int i = 0; live && i < 64; ++i) amax = fmaxf(amax, fabsf(at(i)));
    amax = max16(amax);
    amax = fmaxf(amax, __shfl_xor(amax, 16, 64));
    amax = fmaxf(amax, __shfl_xor(amax, 32, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    float s, inv;
    block_scale(amax, pow2, s, inv);
    if (threadIdx.x == 0) scale[(int64_t)blockIdx.x * gridDim.y + blockIdx.y] = s;
    if (!live) return;
    for (int i = 0; i < 64; i += 4)
        *reinterpret_cast<int *>(codes + tiled_offset(n, k0 + i, K)) =
            cvt_e4m3x4(__fmul_rn(at(i), inv), __fmul_rn(at(i + 1), inv),
                       __fmul_rn(at(i + 2), inv), __fmul_rn(at(i + 3), inv));
}

// Rows: a wave takes 4 rows x one 128-input block per step, 16 lanes x 8 inputs
// per row, so a step writes two contiguous 256-byte pieces (4 rows of a K-tile).
// A workgroup is the 16 rows of a row block and KBS of its k-blocks, whose loads all
// go out first.  Neighbouring workgroups take the row block's next k-blocks, so that
// the rows are read as they lie: 108 us for 38656 x 5376 (627 MB, 5.8 TB/s), 127 us
// with the row blocks next to each other; KBS 1, 3, 4: 123, 108, 111 us (333 rows:
// 3.4 us with 2, 3.8 us with 3).
template <int KBS>
__global__ __launch_bounds__(256) void quantize_kernel(const uint16_t *__restrict__ X, int M,
                                                       int K, bool pow2,
                                                       uint8_t *__restrict__ q,
                                                       float *__restrict__ s)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int nkb = K / 128, parts = (nkb + KBS - 1) / KBS;
    const int m = blockIdx.x / parts * 16 + wave * 4 + (lane >> 4), c = (lane & 15) * 8;
    const int kb0 = blockIdx.x % parts * KBS;
    const int64_t Mp = padded_rows(M);
    const bool live = m < M;
    uint4 u[KBS];
#pragma unroll
    for (int i = 0; i < KBS; ++i) {
        u[i] = make_uint4(0, 0, 0, 0);
        if (live && kb0 + i < nkb)
            u[i] = *reinterpret_cast<const uint4 *>(X + (int64_t)m * K + (kb0 + i) * 128 + c);
    }
#pragma unroll
    for (int i = 0; i < KBS; ++i) {
        const int kb = kb0 + i;
        const float amax = max16(max8(u[i]));
        float sc, inv;
        block_scale(amax, pow2, sc, inv);
        if (!live || kb >= nkb) continue;
        *reinterpret_cast<int2 *>(q + tiled_offset(m, kb * 128 + c, K)) = codes8(u[i], inv);
        if ((lane & 15) == 0) s[kb * Mp + m] = sc;
    }
}

// The product for few rows.  A workgroup owns 16 RT outputs n and 16 MT tokens;
// its waves split the k-blocks and join their sums in LDS, in wave order.  Per
// k-block a wave runs one MFMA for each of its RT x MT tiles (the weight rows
// are the A operand, tokens the columns), from zero, and adds the result times
// s_x s_w to its fp32 sums.
// FUSE: tokens come as bf16 rows X and are quantised in registers (a lane's 32
// inputs and those of the three other lanes of its token are one block); the
// same arithmetic as quantize_kernel.
// F32: fp32 outputs, summed with the bf16 matrix instructions (see above).
template <int RT, int MT, bool FUSE, bool F32>
__global__ __launch_bounds__(512) void skinny_kernel(const void *__restrict__ X,
                                                      const float *__restrict__ sx,
                                                      const uint8_t *__restrict__ qw,
                                                      const float *__restrict__ sw,
                                                      const float *__restrict__ bias,
                                                      void *__restrict__ Y, bool pow2, int M,
                                                      int N, int K)
{
    extern __shared__ float red[];     // [wave][RT * MT * 256]
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int nkb = K / 128, tiles_k = K / 64;
    const int nb0 = blockIdx.x * RT, nblocks = N / 16;
    const int mb0 = blockIdx.y * MT, mblocks = (M + 15) / 16;
    const int64_t Mp = padded_rows(M);
    const int in_tile = r * 64 + ((g ^ ((r >> 2) & 3)) << 4);

    v4f acc[RT][MT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = (v4f)(0.0f);

    for (int kb = wave; kb < nkb; kb += waves) {
        v8i a[RT], b[MT];
        float sc[MT];
        auto tile_frag = [&](const uint8_t *base, int blk) {
            const uint8_t *p = base + ((int64_t)blk * tiles_k + 2 * kb) * 1024 + in_tile;
            const v4i lo = *reinterpret_cast<const v4i *>(p);
            const v4i hi = *reinterpret_cast<const v4i *>(p + 1024);
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        };
        // blocks past the end repeat the last one; their sums are not stored
#pragma unroll
        for (int i = 0; i < RT; ++i) a[i] = tile_frag(qw, min(nb0 + i, nblocks - 1));
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int blk = min(mb0 + j, mblocks - 1);
            if constexpr (FUSE) {
                const uint16_t *p = static_cast<const uint16_t *>(X) +
                                    (int64_t)min(blk * 16 + r, M - 1) * K + kb * 128 + g * 16;
                const uint4 u0 = *reinterpret_cast<const uint4 *>(p);
                const uint4 u1 = *reinterpret_cast<const uint4 *>(p + 8);
                const uint4 u2 = *reinterpret_cast<const uint4 *>(p + 64);
                const uint4 u3 = *reinterpret_cast<const uint4 *>(p + 72);
                float amax = fmaxf(fmaxf(max8(u0), max8(u1)), fmaxf(max8(u2), max8(u3)));
                amax = fmaxf(amax, __shfl_xor(amax, 16, 64));
                amax = fmaxf(amax, __shfl_xor(amax, 32, 64));
                float inv;
                block_scale(amax, pow2, sc[j], inv);
                const int2 c0 = codes8(u0, inv), c1 = codes8(u1, inv);
                const int2 c2 = codes8(u2, inv), c3 = codes8(u3, inv);
                b[j] = (v8i){c0.x, c0.y, c1.x, c1.y, c2.x, c2.y, c3.x, c3.y};
            } else {
                b[j] = tile_frag(static_cast<const uint8_t *>(X), blk);
                sc[j] = sx[kb * Mp + min(blk * 16 + r, M - 1)];
            }
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const float swb = sw[(int64_t)(min(nb0 + i, nblocks - 1) >> 3) * nkb + kb];
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                v4f p = (v4f)(0.0f);
                if constexpr (F32) {
#pragma unroll
                    for (int h = 0; h < 8; h += 2)
                        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            bf16_of_codes(a[i][h], a[i][h + 1]),
                            bf16_of_codes(b[j][h], b[j][h + 1]), p, 0, 0, 0);
                } else {
                    p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[i], b[j], p, 0, 0, 0, 0,
                                                                         0, 0);
                }
                const float f = sc[j] * swb;
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(p[e], f, acc[i][j][e]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
            *reinterpret_cast<v4f *>(red + (wave * RT * MT + i * MT + j) * 256 + lane * 4) =
                acc[i][j];
    __syncthreads();
    // lane (r, g) of tile (i, j): outputs 16 (nb0 + i) + 4 g .. + 3 of token r
    for (int t = wave; t < RT * MT; t += waves) {
        const int nb = nb0 + t / MT, m = (mb0 + t % MT) * 16 + r;
        v4f v = (v4f)(0.0f);
        for (int k = 0; k < waves; ++k)
            v += *reinterpret_cast<const v4f *>(red + (k * RT * MT + t) * 256 + lane * 4);
        if (nb >= nblocks || m >= M) continue;
        const int n = nb * 16 + g * 4;
        if (bias) v += *reinterpret_cast<const v4f *>(bias + n);
        const int64_t o = (int64_t)m * N + n;
        if constexpr (F32)
            *reinterpret_cast<v4f *>(static_cast<float *>(Y) + o) = v;
        else
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(Y) + o) =
                make_uint2(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]));
    }
}

template <int RT, int MT, bool FUSE>
hipError_t launch_skinny(const Fp8Gemm &g, int waves, hipStream_t stream)
{
    const dim3 grid((unsigned)((g.N / 16 + RT - 1) / RT),
                    (unsigned)(((g.M + 15) / 16 + MT - 1) / MT));
    const size_t lds = (size_t)waves * RT * MT * 256 * sizeof(float);
    const void *const X = FUSE ? g.X : g.qx;
    if (g.f32_out)
        hipLaunchKernelGGL((skinny_kernel<RT, MT, FUSE, true>), grid, dim3(64 * waves), lds, stream,
                           X, g.sx, g.qw, g.sw, g.bias, g.Y, g.pow2, (int)g.M, (int)g.N,
                           (int)g.K);
    else
        hipLaunchKernelGGL((skinny_kernel<RT, MT, FUSE, false>), grid, dim3(64 * waves), lds,
                           stream, X, g.sx, g.qw, g.sw, g.bias, g.Y, g.pow2, (int)g.M, (int)g.N,
                           (int)g.K);
    return hipGetLastError();
}

// The shapes of the few-rows kernel on quantised rows and the time of one k-block
// per wave, in us: each workgroup's 8 waves take nkb / 8 k-blocks in turn, whose
// loads nothing covers but a CU's other workgroups.  Measured from N = 32, K = 15360
// (a few workgroups) to N = 16128 (several a CU): within a fifth of
//   3 us + rounds of workgroups over the CUs * ceil(nkb / 8) * us.
// The tiles read each code less often but take nkb k-blocks in turn, so they win
// where N and M give the CUs a tile each (128 rows, K = 5376, N = 16128: 20.4 us,
// here 35.0 us), and lose far below that (96 rows, N = 5376: 18.2 us, here 13.1 us; 64
// rows, N = 1008, K = 18944: 54.4 us, here 31.5 us with 2 x 4, 14.0 us with 1 x 1).
struct SkinnyShape {
    int rt, mt;
    double us;
};
constexpr SkinnyShape kSkinnyShapes[] = {{1, 1, 0.40}, {2, 1, 0.62}, {2, 2, 0.90}, {2, 4, 1.45}};
constexpr double kSkinnyF32Us = 1.65;       // 2 x 4 with F32 outputs: the conversions
constexpr int64_t kMaxGridY = 65535;

} // namespace

hipError_t launch_fp8_block_weights(const void *W, InType in, int64_t N, int64_t K, bool pow2,
                                    uint8_t *codes, float *scale, hipStream_t stream)
{
    // (the second extent is at most 65535 in a launch: N / 128 can be more)
    const dim3 grid((unsigned)((N + 127) / 128), (unsigned)(K / 128));
    if (in == InType::F32)
        hipLaunchKernelGGL((block_weights_kernel<float>), grid, dim3(256), 0, stream,
                           static_cast<const float *>(W), (int)N, (int)K, pow2, codes, scale);
    else
        hipLaunchKernelGGL((block_weights_kernel<uint16_t>), grid, dim3(256), 0, stream,
                           static_cast<const uint16_t *>(W), (int)N, (int)K, pow2, codes, scale);
    return hipGetLastError();
}

hipError_t launch_fp8_quantize(const void *X, int64_t M, int64_t K, bool pow2, uint8_t *q,
                               float *s, hipStream_t stream)
{
    if (M == 0) return hipSuccess;
    constexpr int kbs = 2;
    const dim3 grid((unsigned)((M + 15) / 16 * ((K / 128 + kbs - 1) / kbs)));
    hipLaunchKernelGGL(quantize_kernel<kbs>, grid, dim3(256), 0, stream,
                       static_cast<const uint16_t *>(X), (int)M, (int)K, pow2, q, s);
    return hipGetLastError();
}

bool fp8_fuses_quantize(int64_t M) { return M <= 16; }

Fp8Plan fp8_plan(int64_t M, int64_t N, int64_t K, bool f32_out, bool fused, int64_t cus)
{
    const int64_t nb = N / 16, mb = (M + 15) / 16;
    // Row tiles per workgroup, which shares one quantised k-block of the rows
    // among them, by the rounds of workgroups over the CUs: 1 while that is one
    // round, and of 2 and 4 the larger where it takes half the rounds.  Either
    // side of each border at K = 5376, us with (1, 2 or 2, 4):
    //   N = 4096:  one row 9.0, 9.3;   16 rows, F32 outputs  9.5, 11.4
    //   N = 4608:         11.2, 10.2;                       16.3, 11.4
    //   N = 8064:  one row 11.1, 13.9; 16 rows 12.0, 15.2
    //   N = 10240:        15.9, 13.9;         20.2, 18.4
    //   N = 16384: one row 18.5, 18.8; 16 rows 21.0, 18.5
    //   N = 17408:        23.0, 25.4;         29.5, 29.2
    //   N = 24576: one row 26.6, 28.6; 16 rows 33.0, 32.3
    //   N = 32256:        34.0, 33.8;         42.3, 35.5
    if (fused) {
        auto rounds = [&](int64_t rt) { return ((nb + rt - 1) / rt + cus - 1) / cus; };
        const int rt = rounds(1) == 1 ? 1 : rounds(2) >= 2 * rounds(4) ? 4 : 2;
        return {rt, 1, 0, 0, 0};
    }
    const int64_t steps = (K / 128 + 7) / 8;
    double best_us = fp8_tiles_us(M, N, K, f32_out, cus);
    int best = -1;
    for (int i = 0; i < 4; ++i) {
        const SkinnyShape &s = kSkinnyShapes[i];
        const int64_t gx = (nb + s.rt - 1) / s.rt, gy = (mb + s.mt - 1) / s.mt;
        const double step = i == 3 && f32_out ? kSkinnyF32Us : s.us;
        const double us = 3.0 + (double)((gx * gy + cus - 1) / cus * steps) * step;
        if (gy <= kMaxGridY && us < best_us) best = i, best_us = us;
    }
    if (best < 0) return fp8_tiles_plan(M, N, f32_out, cus);
    return {kSkinnyShapes[best].rt, kSkinnyShapes[best].mt, 0, 0, 0};
}

hipError_t launch_fp8_gemm(const Fp8Gemm &g, hipStream_t stream)
{
    const Fp8Plan p = fp8_plan(g.M, g.N, g.K, g.f32_out, !g.qx, device_cu_count());
    if (!g.qx)
        return p.rt == 1   ? launch_skinny<1, 1, true>(g, 8, stream)
               : p.rt == 2 ? launch_skinny<2, 1, true>(g, 8, stream)
                           : launch_skinny<4, 1, true>(g, 8, stream);
    switch (p.rt * p.mt) {
    case 1: return launch_skinny<1, 1, false>(g, 8, stream);
    case 2: return launch_skinny<2, 1, false>(g, 8, stream);
    case 4: return launch_skinny<2, 2, false>(g, 8, stream);
    case 8: return launch_skinny<2, 4, false>(g, 8, stream);
    default: return launch_fp8_tiles(g, p, stream);
    }
}

} // namespace convrot
