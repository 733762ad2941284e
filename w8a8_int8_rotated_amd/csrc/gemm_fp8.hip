// FP8 (e4m3) x FP8 GEMM on gfx950 matrix cores with a scale per 128 inputs:
//   Y[m, n] = sum_b (sum_{k in b} qx[m, k] qw[n, k]) (sx[b, m] sw[n / 128, b])
//             (+ bias[n])
// Both code matrices are K-tiled (common.hpp); a k-block of 128 inputs is two
// consecutive 1 KiB tiles of each 16-row block.
//
// Any scales.  The scale changes with every k-block, so each block's sum is formed
// from zero by one v_mfma_f32_16x16x128_f8f6f4 and joined by four fp32 fused
// multiply-adds per lane: 16 VALU cycles for 32 matrix cycles, on the same SIMD.  A
// VALU instruction cannot name an accumulator register, so the 128 sums of a lane
// have to sit in ordinary registers: 8 waves (two per SIMD, 256 registers each) own
// 128 x 64 of a 256 (n) x 256 (m) tile, and one wave's matrix instructions run under
// the other's additions.  The sums of row tile i are joined while row tile i + 1
// multiplies.
//
// Powers of two.  v_mfma_scale_f32_16x16x128_f8f6f4 applies both scales (their
// exponent fields are its e8m0 operands) and keeps the sums: no additions.
//
// F32 outputs convert the codes to bf16 and use v_mfma_f32_16x16x32_bf16 (see
// fp8.hip on the precision of the FP8 sums): half the matrix rate, the conversions
// of the activations kept for a k-block.
//
// Copies go straight to LDS (buffer_load ... lds), one k-block (64 KiB) per stage,
// two stages; see CONVROT_FP8_K_BLOCK for the turns at which halves of a stage
// are freed and refilled.  The stream of k-blocks runs on across the tiles of a
// persistent workgroup.  With an odd number of k-blocks a tile takes one more, of
// zeros.
//
// At M = 38656, K = 5376, N = 16128 (6.70 TFLOP; the GEMM alone, bf16 outputs, by
// step, any scales / powers of two):
//   one wait and barrier per k-block, operands read after it       3.04 ms
//   conflict-free LDS slots                                        3.00 ms
//   next k-block's operands requested under the last row tile,
//   weight scales through LDS (a scalar load made every LDS wait
//   a full one)                                                    2.76 / 2.58 ms
//   halves of a stage refilled 1.5 k-blocks ahead                  2.75 / 2.46 ms
//   row tiles requested two ahead                                  2.69 / 2.40 ms
// 2.5 and 2.8 PFLOP/s; the matrix cores are busy 0.65 and 0.72 of the time at
// 1.75 GHz.  LDS is the next bound: a k-block costs 192 reads of 1 KiB and 64 KiB
// of copies, 2048 cycles at 128 bytes a cycle, as many as its matrix instructions;
// a wave tile larger than 128 x 64 would not fit its registers.
#include "fp8_common.hpp"
#include "gemm_common.hpp"

#include <algorithm>
#include <climits>

namespace convrot {
namespace {

constexpr int kKB = 128;        // inputs per k-block
constexpr int kGroup = 4;       // tile-rows per L2 group (2: 1% slower, 8: 1%, 16: 6%)

// The slot of chunk c of row r in an LDS tile is c ^ lds_swz(r).  A 16 x 16 operand
// read takes lane (r, g) to chunk g of row r; LDS serves ds_read_b128 in four
// turns, the first of lanes 0-3, 12-15, 20-23 and 24-27, the second of the other
// lanes below 32.  With (r >> 2) & 3, as in memory, two lanes of a turn share their
// banks (half of all LDS cycles were conflicts, SQ_LDS_BANK_CONFLICT); with 0, 2,
// 3, 1 for the four row quads none do.  A copy's lane fetches the chunk that
// belongs in its place, from the same contiguous 1 KiB.
__device__ __forceinline__ int lds_swz(int r)
{
    const int q = (r >> 2) & 3;
    return ((q << 1) & 3) ^ ((q >> 1) * 3);
}

// One tile's operands: rows past the end are out of range and read as zero.
struct Src {
    const uint8_t *w, *x;
    const float *s;
    int wn, xn, sn;             // bytes in range
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *p, int n)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, n, kRsrcWord3);
}

__device__ __forceinline__ v8i frag(const uint8_t *__restrict__ tile)
{
    const v4i lo = *reinterpret_cast<const v4i *>(tile);
    const v4i hi = *reinterpret_cast<const v4i *>(tile + 1024);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// How a kernel multiplies: FP8 products joined by fp32 additions (any scales),
// FP8 products scaled by the matrix instruction itself (powers of two), or
// bf16 products (fp32 outputs, any scales).
enum Math { kAnyScale, kPow2Scale, kBf16 };

// An operand tile as the matrix instructions take it.
template <bool F32> struct Operand;
template <> struct Operand<false> {
    v8i q;
    __device__ __forceinline__ void set(const v8i &v) { q = v; }
};
template <> struct Operand<true> {
    v8bf h[4];
    __device__ __forceinline__ void set(const v8i &v)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = bf16_of_codes(v[2 * i], v[2 * i + 1]);
    }
};

__device__ __forceinline__ v4f product(const Operand<false> &a, const Operand<false> &b)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.q, b.q, (v4f)(0.0f), 0, 0, 0, 0, 0,
                                                            0);
}
__device__ __forceinline__ v4f product(const Operand<true> &a, const Operand<true> &b)
{
    v4f p = (v4f)(0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.h[i], b.h[i], p, 0, 0, 0);
    return p;
}

// Registers that live from one k-block to the next.
template <int NI, int NJ>
struct State {
    v4f acc[NI][NJ];
    v4f t[NJ];                  // products of the row tile not joined yet
    float f[NJ];                // ... and their scales
    int ex[NJ], ew;             // kPow2Scale: the k-block's scale exponents
    float sx[NJ], sw;           // the scales of the k-block that begins
    v8i a[2], b[NJ];            // its first two row tiles and its column tiles
};

// Row tile i of a k-block against the column tiles in registers, while the
// products of the row tile before it are joined: four additions (16 cycles) beside
// each matrix instruction.
template <Math MATH, int NI, int NJ>
__device__ __forceinline__ void row_tile(State<NI, NJ> &st, const Operand<MATH == kBf16> &a,
                                         const Operand<MATH == kBf16> (&b)[NJ], int i)
{
    if constexpr (MATH == kPow2Scale) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            st.acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                a.q, b[j].q, st.acc[i][j], 0, 0, 0, st.ew, 0, st.ex[j]);
    } else {
        v4f t[NJ];
        v4f(&prev)[NJ] = st.acc[i == 0 ? NI - 1 : i - 1];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            t[j] = product(a, b[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                prev[j][e] = __builtin_fmaf(st.t[j][e], st.f[j], prev[j][e]);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) st.t[j] = t[j];
    }
}

// The scales of the k-block that begins.  A power of two's exponent field is
// its e8m0 scale (0 stands for 2^-127, where all codes are 0; 255 for NaN).
template <Math MATH, int NI, int NJ>
__device__ __forceinline__ void take_scales(State<NI, NJ> &st)
{
    if constexpr (MATH == kPow2Scale) {
        st.ew = __float_as_uint(st.sw) >> 23;
#pragma unroll
        for (int j = 0; j < NJ; ++j) st.ex[j] = __float_as_uint(st.sx[j]) >> 23;
    } else {
#pragma unroll
        for (int j = 0; j < NJ; ++j) st.f[j] = st.sx[j] * st.sw;
    }
}

// Order of one row tile: the next row tile's LDS reads, then its matrix
// instructions with the additions (and, in the last row tile, copies) between.
constexpr int kSgValu = 0x002;
template <Math MATH, int NJ, int READS, int VMEMS>
__device__ __forceinline__ void order_row_tile()
{
    if constexpr (MATH != kBf16) __builtin_amdgcn_sched_group_barrier(kSgDsRead, READS, 0);
#pragma unroll
    for (int j = 0; j < NJ && MATH != kBf16; ++j) {
        __builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0);
        if (MATH == kAnyScale) __builtin_amdgcn_sched_group_barrier(kSgValu, 4, 0);
        if (VMEMS) __builtin_amdgcn_sched_group_barrier(kSgVmemRead, VMEMS, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// One k-block, in two halves.  Row tiles are requested two ahead (one ahead
// leaves a wave that has its SIMD to itself waiting for LDS), so before the last
// two row tiles of a half this wave has read all that the half needs; then it
// waits for its copies but the last VM, and the barrier says that every wave has
// done both:
//  - at the first half's end the second half's weight rows have landed, and the
//    first half's and the activations (in registers since the k-block's start)
//    are free: COPY_A refills them for the k-block after next;
//  - at the second half's end the next k-block's activations and first half have
//    landed in (na, nx, ns), and the second half is free (COPY_B).
// The two halves (ca, cb) are separate LDS objects: a read of one need not wait
// for copies into the other.
// Every copy so has one and a half k-blocks to land.  The next k-block's column
// tiles are requested ahead of the last row tile, which still uses the current
// ones: two to registers of their own, the others after it.
#define CONVROT_FP8_TURN(VM)                                                                  \
    wait_lds_reads();                                                                         \
    wait_vmcnt<VM>();                                                                         \
    block_barrier();                                                                          \
    __builtin_amdgcn_sched_barrier(0)

#define CONVROT_FP8_K_BLOCK(st, ca, cb, na, nx, ns, VM, COPY_A, COPY_B)                       \
    do {                                                                                      \
        Operand<MATH == kBf16> b_[NJ];                                                        \
        _Pragma("unroll") for (int j = 0; j < NJ; ++j) b_[j].set(st.b[j]);                    \
        v8i n0_, n1_;                                                                         \
        _Pragma("unroll") for (int i = 0; i < NI; ++i) {                                      \
            if (i == NI / 2 - 2 || i == NI - 2) {                                             \
                CONVROT_FP8_TURN(VM);                                                         \
            }                                                                                 \
            Operand<MATH == kBf16> a_;                                                        \
            a_.set(st.a[0]);                                                                  \
            st.a[0] = st.a[1];                                                                \
            st.a[1] = frag((i + 2 >= NI ? na : i + 2 < NI / 2 ? ca : cb) + off_w +            \
                           (i + 2) % (NI / 2) * 2048);                                        \
            if (i == NI / 2 - 2) COPY_A;                                                      \
            if (i == NI - 2) COPY_B;                                                          \
            if (i == NI - 1) {                                                                \
                n0_ = frag(nx + off_x);                                                       \
                if constexpr (NJ > 1) n1_ = frag(nx + off_x + 2048);                          \
                _Pragma("unroll") for (int j = 0; j < NJ; ++j)                                \
                    st.sx[j] = ns[off_s + 16 * j];                                            \
                st.sw = ns[256 + wn_s];                                                       \
            }                                                                                 \
            if (i == 0 && MATH == kPow2Scale) take_scales<MATH>(st);                          \
            row_tile<MATH>(st, a_, b_, i);                                                    \
            if (i == 0 && MATH != kPow2Scale) take_scales<MATH>(st);                          \
            if (i == NI - 1) order_row_tile<MATH, NJ, 5 + NJ + 2 * (NJ > 1), 0>();            \
            else if (i == NI / 2 - 2) order_row_tile<MATH, NJ, 2, (CA + NJ - 1) / NJ>();      \
            else if (i == NI - 2) order_row_tile<MATH, NJ, 2, 1>();                           \
            else order_row_tile<MATH, NJ, 2, 0>();                                            \
        }                                                                                     \
        st.b[0] = n0_;                                                                        \
        if constexpr (NJ > 1) st.b[NJ > 1] = n1_;                                             \
        _Pragma("unroll") for (int j = 2; j < NJ; ++j) st.b[j] = frag(nx + off_x + j * 2048); \
        __builtin_amdgcn_sched_barrier(0);                                                    \
    } while (0)

// This wave's copies of (half of) the weight rows of a k-block into a stage:
// CH copies of 1 KiB, of the half whose lane offset is vw.  Zeros if `none`.
template <int CH>
__device__ __forceinline__ void copy_weights(const Src &s, int kb, bool none, uint32_t vw,
                                             uint8_t *dst)
{
    const __amdgpu_buffer_rsrc_t rw = rsrc(s.w, none ? 0 : s.wn);
#pragma unroll
    for (int j = 0; j < CH; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rw, (__attribute__((address_space(3))) void *)(dst + j * 1024), 16, vw,
            kb * 2048 + j * 1024, 0, 0);
}

// ... and of its activations and scales.
template <int CX>
__device__ __forceinline__ void copy_tokens(const Src &s, int kb, bool none, const uint32_t *vx,
                                            int odd, uint32_t vs, uint8_t *dst, float *dst_s)
{
    const __amdgpu_buffer_rsrc_t rx = rsrc(s.x, none ? 0 : s.xn), rs = rsrc(s.s, none ? 0 : s.sn);
#pragma unroll
    for (int j = 0; j < CX; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rx, (__attribute__((address_space(3))) void *)(dst + j * 1024), 16, vx[j >> 1],
            kb * 2048 + (j & 1) * 1024 + odd, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void *)dst_s, 4,
                                             vs, 0, 0, 0);
}

template <int NI, int NJ, Math MATH, bool HAS_BIAS>
__global__ __launch_bounds__(512, 2) void fp8_gemm_kernel(
    const uint8_t *__restrict__ qx, const float *__restrict__ sx, const uint8_t *__restrict__ qw,
    const float *__restrict__ sw, const float *__restrict__ bias, void *__restrict__ Y, int M,
    int N, int K, int m_base, int tiles_m, int tiles_n, int tiles_per_xcd, int wgs_per_xcd)
{
    constexpr int TN = 32 * NI, TM = 64 * NJ;
    constexpr bool F32 = MATH == kBf16;                          // ... outputs
    // copies per wave and k-block: CX of activations and one of scales, twice CH
    // of weights; CA: those of its first half
    constexpr int CX = TM / 64, CH = NI / 4, CA = CX + 1 + CH;
    // copies issued after the ones a turn waits for: half a k-block's of either
    // kind (a tile's first turn waits for part of the last tile's stores as well)
    constexpr int VM = CA + CH;
    __shared__ __attribute__((aligned(1024))) uint8_t wa0[TN * kKB / 2], wb0[TN * kKB / 2],
        wa1[TN * kKB / 2], wb1[TN * kKB / 2];
    __shared__ __attribute__((aligned(1024))) uint8_t sx0[TM * kKB], sx1[TM * kKB];
    __shared__ __attribute__((aligned(1024))) float ss0[320], ss1[320];
    __shared__ __attribute__((aligned(16))) float sbias[TN];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave & 1, wm = wave >> 1;
    const int r = lane & 15, g = lane >> 4;
    const int nkb = K / kKB, nkp = (nkb + 1) & ~1;
    const int Mp = (int)padded_rows(M);
    const int tiles = tiles_m * tiles_n;
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;

    // i-th tile of this workgroup (XCD-contiguous ranges, grouped along m)
    auto tile_at = [&](int i, int &m0, int &n0) -> bool {
        const int tl = slot + i * wgs_per_xcd;
        const int t = xcd * tiles_per_xcd + tl;
        if (tl >= tiles_per_xcd || t >= tiles) return false;
        const int width = kGroup * tiles_n;
        const int first_m = (t / width) * kGroup;
        const int gsz = min(tiles_m - first_m, kGroup);
        m0 = m_base + (first_m + (t % width) % gsz) * TM;
        n0 = ((t % width) / gsz) * TN;
        return true;
    };
    // scales: waves 0-3 copy the tokens' (TM of them, 64 per wave; with fewer
    // tokens some waves repeat others), waves 4-7 those of the tile's one or two
    // blocks of 128 weight rows
    const bool tok = wave < 4;
    auto src_of = [&](int m0, int n0) {
        const int row = n0 >> 7, rows = (N + 127) >> 7;
        return Src{qw + (int64_t)n0 * K, qx + (int64_t)m0 * K,
                   tok ? sx + m0 : sw + (int64_t)row * nkb, (N - n0) * K, (Mp - m0) * K,
                   tok ? (Mp - m0) * 4 : row + 1 < rows ? (nkb + 1) * 4 : 4};
    };
    const int s_step = tok ? Mp : 1;

    int m0, n0;
    if (!tile_at(0, m0, n0)) return;
    int nm0 = m0, nn0 = n0;
    bool more = tile_at(1, nm0, nn0);
    Src nxt = src_of(nm0, nn0);

    // Copy c of a stage moves 1 KiB: tile c & 1 of row block c >> 1.  The row's
    // offset is in the lane's offset (the one that is checked against the range),
    // the k-block's in the scalar one.  Weight halves: row tiles 0 .. NI/2 - 1 of
    // both waves wn, then the others.
    constexpr int VX = (CX + 1) / 2;
    const int cr = lane >> 2, cell = cr * 64 + (((lane & 3) ^ swz(cr) ^ lds_swz(cr)) << 4);
    const int cw = wave * CH, rb = (cw >> 1) / (NI / 2) * NI + (cw >> 1) % (NI / 2);
    const uint32_t vw0 = rb * 16 * K + (CH == 1 ? (wave & 1) * 1024 : 0) + cell;
    const uint32_t vw1 = vw0 + NI / 2 * 16 * K;
    uint32_t vx[VX];
#pragma unroll
    for (int j = 0; j < VX; ++j) vx[j] = ((wave * CX) / 2 + j) * 16 * K + cell;
    const int odd = CX == 1 ? (wave & 1) * 1024 : 0;
    const int sgrp = tok ? wave & (CX - 1) : 4;
    const uint32_t vs = tok ? sgrp * 256 + lane * 4 : (lane & 1) * nkb * 4;

    // The stream of k-blocks: the next one to copy is k-block ikb of `is` (of
    // nothing, zeros, beyond a tile's k-blocks and after the last tile).  It turns
    // to the next tile when it needs it, not at the end of the one before: with
    // two k-blocks a tile, that tile is known only by then.
    Src is = src_of(m0, n0);
    int ikb = 0;
    auto copy_a = [&](uint8_t *dw, uint8_t *dx, float *ds) {
        // (selects, not branches: a branch here would split the k-block into
        // regions the additions get moved across)
        const bool wrap = ikb == nkp;
        is.w = wrap ? nxt.w : is.w;
        is.x = wrap ? nxt.x : is.x;
        is.s = wrap ? nxt.s : is.s;
        is.wn = wrap ? nxt.wn : is.wn;
        is.xn = wrap ? nxt.xn : is.xn;
        is.sn = wrap ? nxt.sn : is.sn;
        ikb = wrap ? (more ? 0 : INT_MAX / 2) : ikb;         // no more: past every k-block
        const bool none = ikb >= nkb;
        copy_tokens<CX>(is, none ? 0 : ikb, none, vx, odd, vs, dx + wave * CX * 1024,
                        ds + sgrp * 64);
        copy_weights<CH>(is, none ? 0 : ikb, none, vw0, dw + wave * CH * 1024);
    };
    auto copy_b = [&](uint8_t *dw) {
        const bool none = ikb >= nkb;
        copy_weights<CH>(is, none ? 0 : ikb, none, vw1, dw + wave * CH * 1024);
        is.s += none ? 0 : s_step;
        ++ikb;
    };

    const int in_tile = r * 64 + ((g ^ lds_swz(r)) << 4);
    const int off_w = wn * (NI / 2) * 2048 + in_tile, off_x = wm * NJ * 2048 + in_tile;
    const int off_s = wm * NJ * 16 + r, wn_s = (wn * 16 * NI) >> 7;

    float b_reg = 0.0f;
    auto load_bias = [&](int n0_) {
        if constexpr (HAS_BIAS) b_reg = bias[min(n0_ + (tid & (TN - 1)), N - 1)];
    };
    load_bias(n0);

    State<NI, NJ> st;
    copy_a(wa0, sx0, ss0);
    copy_b(wb0);
    copy_a(wa1, sx1, ss1);
    copy_b(wb1);
    wait_vmcnt<0>();
    block_barrier();
    st.a[0] = frag(wa0 + off_w);
    st.a[1] = frag(wa0 + off_w + 2048);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        st.b[j] = frag(sx0 + off_x + j * 2048);
        st.sx[j] = ss0[off_s + 16 * j];
    }
    st.sw = ss0[256 + wn_s];

    for (int it = 0;; ++it) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) st.acc[i][j] = (v4f)(0.0f);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            st.t[j] = (v4f)(0.0f);
            st.f[j] = 0.0f;
        }
        // two k-blocks per round, so that every access names its stage
        for (int k = 0; k < nkp; k += 2) {
            CONVROT_FP8_K_BLOCK(st, wa0, wb0, wa1, sx1, ss1, VM, copy_a(wa0, sx0, ss0), copy_b(wb0));
            CONVROT_FP8_K_BLOCK(st, wa1, wb1, wa0, sx0, ss0, VM, copy_a(wa1, sx1, ss1), copy_b(wb1));
        }
#pragma unroll
        for (int j = 0; j < NJ && MATH != kPow2Scale; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                st.acc[NI - 1][j][e] = __builtin_fmaf(st.t[j][e], st.f[j], st.acc[NI - 1][j][e]);

        if constexpr (HAS_BIAS) {
            sbias[tid & (TN - 1)] = b_reg;
            wait_lds_reads();
            block_barrier();
        }
        // lane (r, g) holds outputs 16 i + 4 g + 0..3 of token r of its tiles
        const bool full = m0 + TM <= M && n0 + TN <= N;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int m = m0 + (wm * NJ + j) * 16 + r;
#pragma unroll
            for (int i = 0; i < NI; i += 2) {
                const int nl = wn * 16 * NI + 16 * i;
                v4f v0 = st.acc[i][j], v1 = st.acc[i + 1][j];
                if constexpr (HAS_BIAS) {
                    v0 += *reinterpret_cast<const v4f *>(&sbias[nl + 4 * g]);
                    v1 += *reinterpret_cast<const v4f *>(&sbias[nl + 16 + 4 * g]);
                }
                if constexpr (F32) {
                    float *const o = static_cast<float *>(Y) + (int64_t)m * N + n0 + nl + 4 * g;
                    if (full || (m < M && n0 + nl < N)) *reinterpret_cast<v4f *>(o) = v0;
                    if (full || (m < M && n0 + nl + 16 < N)) *reinterpret_cast<v4f *>(o + 16) = v1;
                } else {
                    // neighbouring lane rows trade halves: even g then hold 8
                    // consecutive outputs of tile i, odd g of tile i + 1
                    const auto s0 = __builtin_amdgcn_permlane16_swap(
                        cvt_pk_bf16(v0[0], v0[1]), cvt_pk_bf16(v1[0], v1[1]), false, false);
                    const auto s1 = __builtin_amdgcn_permlane16_swap(
                        cvt_pk_bf16(v0[2], v0[3]), cvt_pk_bf16(v1[2], v1[3]), false, false);
                    const int n = n0 + nl + (g & 1) * 16 + (g >> 1) * 8;
                    if (full || (m < M && n < N))
                        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(Y) + (int64_t)m * N + n) =
                            make_uint4(s0[0], s1[0], s0[1], s1[1]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (!more) break;
        m0 = nm0;
        n0 = nn0;
        load_bias(n0);
        more = tile_at(it + 2, nm0, nn0);
        nxt = src_of(nm0, nn0);
        // sbias is rewritten only after the next tile's barriers
    }
    // no copy may still be writing LDS when the workgroup ends
    wait_vmcnt<0>();
}

// Rows m_base .. m_base + rows - 1 of the product, in 32 NI (n) x 64 NJ (m) tiles.
template <int NI, int NJ, Math MATH>
hipError_t launch_tile(const Fp8Gemm &g, int64_t m_base, int64_t rows, hipStream_t stream)
{
    constexpr int TN = 32 * NI, TM = 64 * NJ;
    const int tiles_m = (int)((rows + TM - 1) / TM), tiles_n = (int)((g.N + TN - 1) / TN);
    const int per_xcd = (tiles_m * tiles_n + 7) / 8;
    const int wgs = std::max(1, std::min(device_cu_count() / 8, per_xcd));
    const dim3 grid(8 * wgs), block(512);
    if (g.bias)
        hipLaunchKernelGGL((fp8_gemm_kernel<NI, NJ, MATH, true>), grid, block, 0, stream, g.qx,
                           g.sx, g.qw, g.sw, g.bias, g.Y, (int)g.M, (int)g.N, (int)g.K,
                           (int)m_base, tiles_m, tiles_n, per_xcd, wgs);
    else
        hipLaunchKernelGGL((fp8_gemm_kernel<NI, NJ, MATH, false>), grid, block, 0, stream, g.qx,
                           g.sx, g.qw, g.sw, g.bias, g.Y, (int)g.M, (int)g.N, (int)g.K,
                           (int)m_base, tiles_m, tiles_n, per_xcd, wgs);
    return hipGetLastError();
}

template <Math MATH>
hipError_t launch_shape(int tn, int tm, const Fp8Gemm &g, int64_t m_base, int64_t rows,
                        hipStream_t stream)
{
    if constexpr (MATH != kBf16) {
        if (tn == 256)
            return tm == 256   ? launch_tile<8, 4, MATH>(g, m_base, rows, stream)
                   : tm == 128 ? launch_tile<8, 2, MATH>(g, m_base, rows, stream)
                               : launch_tile<8, 1, MATH>(g, m_base, rows, stream);
    }
    return tm == 256   ? launch_tile<4, 4, MATH>(g, m_base, rows, stream)
           : tm == 128 ? launch_tile<4, 2, MATH>(g, m_base, rows, stream)
                       : launch_tile<4, 1, MATH>(g, m_base, rows, stream);
}

// Tile shapes and the time of one tile per CU, in units of the largest shape's;
// measured at K = 5376: bf16 outputs 56 us for 256 x 256 (any scales), F32 outputs
// 70 us for 128 x 256.  A 128 x 64 tile's k-block (18 us) is bound by the latency of
// its copies and by LDS: four stages of it, or waves that split the k-blocks and
// read half as much from LDS, took 17 to 20 us.
struct TileShape {
    int tn, tm;
    double cost;
};
constexpr TileShape kFp8Shapes[] = {{256, 256, 1.0}, {256, 128, 0.64}, {128, 256, 0.64},
                                    {256, 64, 0.46}, {128, 128, 0.42}, {128, 64, 0.32}};
constexpr TileShape kBf16Shapes[] = {{128, 256, 1.0}, {128, 128, 0.61}, {128, 64, 0.49}};
constexpr double kSecondLaunch = 0.06;

// Rounds of one shape's tiles over the CUs, in units of the largest shape's tile.
double shape_cost(const TileShape &s, int64_t rows, int64_t N, int64_t cus)
{
    const int64_t tiles = (rows + s.tm - 1) / s.tm * ((N + s.tn - 1) / s.tn);
    return (double)((tiles + cus - 1) / cus) * s.cost;
}

} // namespace

// Where the tiles compete with the few-rows kernel (one shape, a round or a few):
// k-blocks in turn, 0.35 us each in a 128 x 64 tile (F32 outputs 0.69 us).  At
// N = 1024 .. 5376: 9.2, 18.1, 36.1 and 61 us for 16, 42, 96 and 168 of them, F32
// outputs 15.5, 33, 70.7 and 122 us; within a tenth of this.
double fp8_tiles_us(int64_t M, int64_t N, int64_t K, bool f32_out, int64_t cus)
{
    double best = 1e30;
    if (f32_out)
        for (const TileShape &s : kBf16Shapes) best = std::min(best, shape_cost(s, M, N, cus));
    else
        for (const TileShape &s : kFp8Shapes) best = std::min(best, shape_cost(s, M, N, cus));
    return 4.0 + best * (double)(K / kKB) * (f32_out ? 1.41 : 1.08);
}

// The plan with the least estimated time: one shape throughout, or whole rounds
// of the largest shape and another one for the last rows (M = 4096 at
// N = K = 5376: 252 tiles of 256 x 256, then 1024 rows in 168 of 256 x 128).
Fp8Plan fp8_tiles_plan(int64_t M, int64_t N, bool f32_out, int64_t cus)
{
    const TileShape *const shapes = f32_out ? kBf16Shapes : kFp8Shapes;
    const int n_shapes = f32_out ? 3 : 6;
    auto cost = [&](int i, int64_t rows) { return shape_cost(shapes[i], rows, N, cus); };
    int best = 0;
    int64_t m1 = 0;                  // rows of the first launch (shape 0)
    double best_cost = 1e30;
    for (int i = 0; i < n_shapes; ++i) {
        const double c = cost(i, M);
        if (c < best_cost) best = i, best_cost = c;
    }
    const int64_t rows0 = (M - 1) / shapes[0].tm;        // whole tile-rows before the last
    for (int64_t a = rows0; a > 0 && a > rows0 - 16; --a)
        for (int i = 1; i < n_shapes; ++i) {
            const double c = cost(0, a * shapes[0].tm) + cost(i, M - a * shapes[0].tm) +
                             kSecondLaunch;
            if (c < best_cost - 0.1) best = i, best_cost = c, m1 = a * shapes[0].tm;
        }
    return {0, 0, shapes[best].tn, shapes[best].tm, m1};
}

hipError_t launch_fp8_tiles(const Fp8Gemm &g, const Fp8Plan &p, hipStream_t stream)
{
    auto launch = [&](int tn, int tm, int64_t base, int64_t rows) {
        return g.f32_out ? launch_shape<kBf16>(tn, tm, g, base, rows, stream)
               : g.pow2  ? launch_shape<kPow2Scale>(tn, tm, g, base, rows, stream)
                         : launch_shape<kAnyScale>(tn, tm, g, base, rows, stream);
    };
    if (p.first > 0) {
        const TileShape &s = g.f32_out ? kBf16Shapes[0] : kFp8Shapes[0];
        const hipError_t e = launch(s.tn, s.tm, 0, p.first);
        if (e != hipSuccess) return e;
    }
    return launch(p.tn, p.tm, p.first, g.M - p.first);
}

} // namespace convrot
