// fp8.hip -- matrices held in 8-bit floating point (e4m3) with a scale for
// each block of 128, and the product of two of them: an 8-bit output head.
//
// Quantiser: a block (128 columns of one row, or 128 x 128) gets
//   s = amax * (1 / 448), both factors and the product in fp32 (448 is e4m3's
//   largest value), at least 2^-126;
//   code = the e4m3 value nearest to the exact quotient x / s, ties to even.
// Product: out[m, n] = sum_b sA[b, m] sB[n / 128, b] P_b[m, n],
//   P_b[m, n] = sum over the 128 columns of block b of A8[m, k] B8[n, k].
// The codes' products are exact in the matrix cores and summed in fp32; each
// block's sum is scaled and added in fp32, and the result is rounded once, to
// the output's type.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "api_internal.hpp"
#include "archead.h"
#include "device.hpp"
#include "e4m3.hpp"
#include "entry.hpp"
#include "lds_copy.hpp"

namespace archead {
namespace {

typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x8u __attribute__((ext_vector_type(8), aligned(2)));

constexpr int kBlk = 128; // columns (and weight rows) that share a scale
constexpr int64_t kMaxStride = int64_t(1) << 23; // of A and B: a tile's offsets fit 32 bits

// ---------------------------------------------------------------------------
// quantiser
// ---------------------------------------------------------------------------
__device__ __forceinline__ void load8(const float *p, float v[8])
{
    const f32x4u a = *(const f32x4u *)p, b = *(const f32x4u *)(p + 4);
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
}
__device__ __forceinline__ void load8(const uint16_t *p, float v[8])
{
    const u16x8u a = *(const u16x8u *)p;
    for (int i = 0; i < 8; ++i)
        v[i] = __uint_as_float((uint32_t)a[i] << 16);
}

// Whether codes are taken the exact way at once.  The quotients of bf16 values are true
// ties often enough for some third of the waves to need it, and where a launch is short
// enough for the longest wave's time to count, the quick way before it is time lost (bf16,
// exact at once, quick first, in us: 1 row of 4096 4.3, 5.6; 512 rows 7.2, 7.6; 2048 16.6,
// 16.7; 4096 28.5, 27.4; 8192 50.0, 46.8; 128 x 4096 by 128 x 128 blocks 23, 36; 1024 x
// 4096 25, 33; 4096 x 4096 66.6, 62.5).  fp32 values have few such ties (1 row 4.3, 2.4;
// 8192 rows 54.7, 27.3).
constexpr int64_t kExactRows = 4096, kExactTiles = 512; // workgroups

// One row's blocks: 16 lanes a block, 8 columns a lane, so that a block's
// largest magnitude takes four exchanges and a lane one load and one store
// (2048 x 4096 bf16: 16.6 us against 5 of its bytes, the vector units busy
// throughout: finding a thread's row divides 64-bit numbers, and exact quotients are
// a division, its remainder and the last bit of every element; one row 4.3 us, a launch).
template <typename T, bool kExact>
__global__ __launch_bounds__(256) void quant_rows_kernel(const T *x, int64_t ldx, int64_t rows, int64_t cols,
                                                         uint8_t *q, int64_t ldq, float *s, int64_t lds)
{
    const int64_t nb = (cols + kBlk - 1) / kBlk;
    const int64_t g = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); // (row, block)
    const int64_t row = g / nb, b = g % nb;
    if (row >= rows) // whole groups of 16 lanes leave together
        return;
    const int64_t c = b * kBlk + 8 * (threadIdx.x & 15);
    const bool in = c < cols; // cols is a multiple of 16
    float v[8] = {};
    if (in)
        load8(x + row * ldx + c, v);
    float m = 0.f;
    for (int i = 0; i < 8; ++i)
        m = fmaxf(m, fabsf(v[i]));
    for (int off = 8; off >= 1; off >>= 1)
        m = fmaxf(m, __shfl_xor(m, off));
    const float sc = block_scale(m);
    if (in)
        *(u32x2 *)(q + row * ldq + c) = kExact ? codes8_exact(v, sc) : codes8(v, sc);
    if ((threadIdx.x & 15) == 0)
        s[b * lds + row] = sc;
}

// 128 x 128 blocks, one per workgroup: two threads a row, 64 columns each, read
// once for the scale and again for the codes.  151936 x 4096 bf16, once per
// head: 3.4 ms against 0.4 of its bytes, since a thread's 16-byte loads come to a
// 128-byte line eight times in each pass, and 18 GB are fetched for 1.2.
template <typename T, bool kExact>
__global__ __launch_bounds__(256) void quant_tiles_kernel(const T *x, int64_t ldx, int64_t rows, int64_t cols,
                                                          uint8_t *q, int64_t ldq, float *s, int64_t lds)
{
    __shared__ float red[4];
    const int64_t nb = (cols + kBlk - 1) / kBlk;
    const int64_t rb = blockIdx.x / nb, b = blockIdx.x % nb;
    const int64_t row = rb * kBlk + (threadIdx.x >> 1), c0 = b * kBlk + 64 * (threadIdx.x & 1);
    const T *xr = x + row * ldx;
    float m = 0.f, v[8];
    for (int j = 0; j < 8; ++j)
        if (row < rows && c0 + 8 * j < cols) {
            load8(xr + c0 + 8 * j, v);
            for (int i = 0; i < 8; ++i)
                m = fmaxf(m, fabsf(v[i]));
        }
    for (int off = 32; off >= 1; off >>= 1)
        m = fmaxf(m, __shfl_xor(m, off));
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = m;
    __syncthreads();
    const float sc = block_scale(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    for (int j = 0; j < 8; ++j)
        if (row < rows && c0 + 8 * j < cols) {
            load8(xr + c0 + 8 * j, v);
            *(u32x2 *)(q + row * ldq + c0 + 8 * j) = kExact ? codes8_exact(v, sc) : codes8(v, sc);
        }
    if (threadIdx.x == 0)
        s[rb * lds + b] = sc;
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
struct ProdArgs {
    int64_t M, N, K, lda, ldb, ldo, ldsa, ldsb;
    const uint8_t *A, *B;
    const float *sA, *sB; // sA[block][row], sB[row / 128][block]
    void *out;
};

// e4m3 codes of one dword pair as eight fp16 values (exact), in order
__device__ __forceinline__ f16x8 halves(uint32_t lo, uint32_t hi)
{
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true);
    return f16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// c + the product of 16 rows' 128 columns with 16 others', 32 bytes a lane.
// The products are taken in fp16 matrix instructions, which add them in full
// fp32.  The fp8 forms align each group of eight products to its largest and
// cut off what lies 2^13 below it (measured: 2e-5 of the terms' magnitudes,
// 1e-4 of a typical result), which would show in an fp32 result; a bf16
// result, rounded at 2^-8, hides it, and there the tiles for many rows use
// them (2048 x 151936 x 4096: 1.62 ms against 2.19 in fp16).
__device__ __forceinline__ f32x4 block_product(i32x8 a, i32x8 b, f32x4 c)
{
    for (int i = 0; i < 8; i += 2)
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(halves(a[i], a[i + 1]), halves(b[i], b[i + 1]), c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ void put4(float *p, f32x4 v, int64_t left)
{
    if (left >= 4)
        *(f32x4u *)p = v;
    else
        for (int i = 0; i < left; ++i)
            p[i] = v[i];
}
__device__ __forceinline__ void put4(uint16_t *p, f32x4 v, int64_t left)
{
    for (int i = 0; i < 4; ++i)
        if (i < left)
            p[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
}

// 16 bytes of a row at column c, zeros past K (a multiple of 16)
__device__ __forceinline__ i32x4 piece(const uint8_t *row, int64_t c, int64_t K)
{
    const i32x4 z = {0, 0, 0, 0};
    return c < K ? *(const i32x4 *)(row + c) : z;
}
__device__ __forceinline__ i32x8 join(i32x4 a, i32x4 b)
{
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// ---------------------------------------------------------------------------
// Few rows (M <= 16): the weights are streamed once, which bounds it (1 x 151936
// x 4096: 105 us, 5.9 TB/s; a large copy runs at 4.9).  The workgroups of 4
// waves stay and take every gridDim-th block of 16 weight rows; each wave takes
// a quarter of the row block's column blocks, and the waves' sums meet in LDS.
// Each wave keeps kDepth column blocks (2 KiB of weights each) in flight, across
// the row blocks' ends; half or twice as many run alike.  The weights are the A
// operand, so that a lane's four results are consecutive columns of one output
// row.  Lane l takes bytes 16 (l / 16) .. +15 of both halves of a block's 128
// columns: any order of the columns serves as long as both operands share it.
// The hidden states' codes lie in LDS where they fit, M K <= 64 KiB: read
// through the caches they pass at the weights' own rate (M = 16, N = 151936,
// K = 4096: 163 us against 141).
// ---------------------------------------------------------------------------
constexpr int kSkinnyM = 16, kSkinnyWaves = 4, kDepth = 4;
constexpr int64_t kSkinnyX = 64 << 10;   // LDS for the hidden states' codes, two workgroups a compute unit
constexpr int64_t kCu = 256;
constexpr int64_t kSkinnyGrid = kCu * 4; // workgroups: four a compute unit

template <bool XL, typename O> __global__ __launch_bounds__(kSkinnyWaves * 64) void product_skinny_kernel(ProdArgs a)
{
    __shared__ f32x4 part[2][kSkinnyWaves][64];
    extern __shared__ i32x4 xs[]; // XL: A's pieces [block][half][quarter][row], zeros past K
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, q = lane >> 4, r = lane & 15;
    const int64_t nb = (a.K + kBlk - 1) / kBlk, per = (nb + kSkinnyWaves - 1) / kSkinnyWaves;
    const int64_t nrb = (a.N + 15) / 16;
    const int64_t m = min((int64_t)r, a.M - 1);
    const uint8_t *x = a.A + m * a.lda;
    if (XL) {
        for (int64_t i = threadIdx.x; i < nb * 8 * a.M; i += kSkinnyWaves * 64)
            xs[i] = piece(a.A + i % a.M * a.lda, i / a.M * 16, a.K);
        __syncthreads();
    }
    struct Unit {
        i32x4 w0, w1, x0, x1;
        float s, sx;
        int xb;
    } u[kDepth];
    // the next column block to load: number j of this wave's in row block rb
    int64_t rb = blockIdx.x, j = 0;
    const uint8_t *w = a.B + min(rb * 16 + r, a.N - 1) * a.ldb;
    const float *sw = a.sB + rb / (kBlk / 16) * a.ldsb;
    auto load = [&](Unit &v) {
        if (rb < nrb) {
            const int64_t b = wv * per + j, c = b * kBlk + 16 * q, bc = min(b, nb - 1);
            v.w0 = piece(w, c, a.K);
            v.w1 = piece(w, c + 64, a.K);
            if (XL) {
                v.xb = (int)bc;
            } else {
                v.x0 = piece(x, c, a.K);
                v.x1 = piece(x, c + 64, a.K);
            }
            v.sx = a.sA[bc * a.ldsa + m];
            v.s = b < nb ? sw[bc] : 0.f;
            if (b >= nb)
                v.sx = 0.f;
            if (++j == per) {
                j = 0;
                rb += gridDim.x;
                w = a.B + min(rb * 16 + r, a.N - 1) * a.ldb;
                sw = a.sB + min(rb, nrb - 1) / (kBlk / 16) * a.ldsb;
            }
        }
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        load(u[d]);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    int64_t done = 0, at = blockIdx.x;
    int par = 0;
    const int64_t mine = ((nrb - blockIdx.x + gridDim.x - 1) / gridDim.x) * per; // column blocks of this wave
    for (int64_t i = 0; i < mine; i += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            if (i + d < mine) {
                if (XL) {
                    const int at_x = (u[d].xb * 8 + q) * (int)a.M + (int)m;
                    u[d].x0 = xs[at_x];
                    u[d].x1 = xs[at_x + 4 * (int)a.M];
                }
                const f32x4 p = block_product(join(u[d].w0, u[d].w1), join(u[d].x0, u[d].x1),
                                              f32x4{0.f, 0.f, 0.f, 0.f});
                const float f = u[d].s * u[d].sx;
                for (int e = 0; e < 4; ++e)
                    acc[e] = __builtin_fmaf(p[e], f, acc[e]);
                load(u[d]);
                if (++done == per) { // the row block's end: the four sums in wave order
                    part[par][wv][lane] = acc;
                    // LDS alone has to be waited for: the loads stay in flight
                    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
                    __builtin_amdgcn_s_barrier();
                    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
                    // wave 0 writes; the other buffer's readers are two barriers behind
                    if (wv == 0) {
                        for (int v = 1; v < kSkinnyWaves; ++v)
                            acc += part[par][v][lane];
                        const int64_t c = at * 16 + 4 * q;
                        if (r < a.M)
                            put4((O *)a.out + r * a.ldo + c, acc, a.N - c);
                    }
                    acc = f32x4{0.f, 0.f, 0.f, 0.f};
                    done = 0;
                    at += gridDim.x;
                    par ^= 1;
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Many rows: tiles of BM output rows x BN columns, each wave [BM / 2 x 64].  A
// stage is one block of 128 columns of both operands, copied straight into LDS
// as codes (16-byte pieces, a row's pieces exchanged by the row's low bits so
// that the reads of eight neighbouring rows fall on different banks: no
// conflicts counted) while the other buffer is worked on; the block's sums are
// scaled into the accumulator in fp32.  2048 x 151936 x 4096: fp32 2.19 ms, 1166
// TFLOP/s of the 1219 that a large bf16 library product reaches here; bf16 1.62
// ms, 1570 TFLOP/s of the 2940 of an fp8 one: matrix cores 35 % busy, all copies
// of a stage waited for before each of its barriers.
// ---------------------------------------------------------------------------
__device__ const u32x4 kNothing = {0u, 0u, 0u, 0u}; // what a piece past K is copied from

template <int BM, int BN> struct Tile {
    static constexpr int waves = BN / 32;                           // two along the rows, each 64 columns
    static constexpr int rows = BM + BN, codes = rows * kBlk / 4;
    static constexpr int words = codes + BM;                        // LDS of a stage: the codes, the rows' scales
    static constexpr int copies = rows / 8 / waves;                 // 1 KiB copies per wave and stage
    static constexpr int mt = BM / 32;                              // 16 x 16 tiles per wave: mt x 4
    static constexpr int wgs = 160 * 1024 / (words * 8);            // workgroups a compute unit holds
};

template <int BM, int BN, bool F8, typename O>
__global__ __launch_bounds__((BN * 2), (Tile<BM, BN>::wgs * BN / 128)) void product_tile_kernel(ProdArgs a)
{
    using T = Tile<BM, BN>;
    // two stage buffers, each the codes and then the rows' scales
    __shared__ __attribute__((aligned(16))) uint32_t smem[2 * T::words];
    const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Workgroup b runs on XCD b mod 8: an XCD takes every eighth column tile
    // and all row tiles of it in turn, so that the weights pass through one L2.
    const int64_t n_mt = (a.M + BM - 1) / BM, n_nt = (a.N + BN - 1) / BN;
    const int64_t id = blockIdx.x >> 3, ni = (id / n_mt) * 8 + (blockIdx.x & 7), mi = id % n_mt;
    if (ni >= n_nt)
        return;
    const int64_t m0 = mi * BM, n0 = ni * BN;
    const int64_t nb = (a.K + kBlk - 1) / kBlk;

    // copy c of this wave: LDS rows 8 (waves c + wv) .. +7 (rows 0 .. BM-1 from
    // A, the rest from B), lane l piece l % 8 of row l / 8
    const int wm = wv / (BN / 64) * (BM / 2), wn = wv % (BN / 64) * 64;
    const int col = 16 * ((lane & 7) ^ (lane >> 3)); // row & 7 = lane / 8
    const uint8_t *baseA = a.A + m0 * a.lda, *baseB = a.B + n0 * a.ldb;
    uint32_t off[T::copies]; // byte offsets from them: row strides are below 2^23
#pragma unroll
    for (int c = 0; c < T::copies; ++c) {
        const int row = 8 * (T::waves * c + wv) + (lane >> 3);
        off[c] = (8 * T::waves * c < BM ? (uint32_t)min((int64_t)row, a.M - 1 - m0) * (uint32_t)a.lda
                                        : (uint32_t)min((int64_t)row - BM, a.N - 1 - n0) * (uint32_t)a.ldb) + col;
    }
    const uint32_t lds0 = lds_address(smem);
    auto fill = [&](int at, int64_t b) { // at: the buffer's first word
        const int64_t k0 = b * kBlk;
        if (k0 + kBlk <= a.K) {
#pragma unroll
            for (int c = 0; c < T::copies; ++c)
                lds_dma16_from((8 * T::waves * c < BM ? baseA : baseB) + k0, off[c],
                               lds0 + 4 * (at + (T::waves * c + wv) * 256));
        } else { // the last, shorter block: zeros past K
#pragma unroll
            for (int c = 0; c < T::copies; ++c) {
                const uint8_t *p = (8 * T::waves * c < BM ? baseA : baseB) + k0 + off[c];
                lds_dma16<false>(k0 + col < a.K ? p : (const uint8_t *)&kNothing, &smem[at + (T::waves * c + wv) * 256]);
            }
        }
        if (wv < BM / 64)
            lds_dma4(a.sA + b * a.ldsa + min(m0 + 64 * wv + lane, a.M - 1), &smem[at + T::codes + 64 * wv]);
    };
    const float *sw = a.sB + min((n0 + wn) / kBlk, (a.N - 1) / kBlk) * a.ldsb;
    // the two pieces of a lane's 32 bytes of one row
    const int p0 = 4 * (q ^ (r & 7)), p1 = 4 * ((q + 4) ^ (r & 7));
    const int f0 = r * 32 + p0, f1 = r * 32 + p1;
    auto frag = [&](int at, int row) {
        return join(*(const i32x4 *)&smem[at + f0 + row * 32], *(const i32x4 *)&smem[at + f1 + row * 32]);
    };
    auto row_scale = [&](int at, int t) {
        return __uint_as_float(smem[at + T::codes + wm + 16 * t + r]);
    };
    f32x4 acc[T::mt][4];
    for (int t = 0; t < T::mt; ++t)
        for (int n = 0; n < 4; ++n)
            acc[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};

    // The scheduler is held to one row tile at a time: left alone it loads all
    // tiles' operands first and spills the accumulator.
    auto work = [&](int at, float f) {
        float s = row_scale(at, 0) * f;
        if constexpr (F8) {
            i32x8 x = frag(at, wm);
            i32x8 w[4];
            for (int n = 0; n < 4; ++n)
                w[n] = frag(at, BM + wn + 16 * n);
            f32x4 pp[2][4];
            float s1 = 0.f;
            auto add = [&](int t, int n, float st) {
                for (int i = 0; i < 4; ++i)
                    acc[t][n][i] = __builtin_fmaf(pp[t & 1][n][i], st, acc[t][n][i]);
            };
#pragma unroll
            for (int t = 0; t < T::mt; ++t) {
                const i32x8 xt = x;
                const float st = s;
                if (t + 1 < T::mt) {
                    x = frag(at, wm + 16 * (t + 1));
                    s = row_scale(at, t + 1) * f;
                }
                for (int n = 0; n < 4; ++n) {
                    pp[t & 1][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[n], xt, f32x4{0.f, 0.f, 0.f, 0.f},
                                                                                    0, 0, 0, 0, 0, 0);
                    if (t > 0)
                        add(t - 1, n, s1);
                    __builtin_amdgcn_sched_barrier(0);
                }
                s1 = st;
            }
            for (int n = 0; n < 4; ++n)
                add(T::mt - 1, n, s1);
        } else {
            // the operand with fewer tiles stays in registers as fp16, the
            // other's tiles pass (all fit only that way beside the accumulator)
            constexpr bool hold_x = T::mt < 4;
            constexpr int nh = hold_x ? T::mt : 4, np = hold_x ? 4 : T::mt;
            const int h0 = hold_x ? wm : BM + wn, s0 = hold_x ? BM + wn : wm;
            f16x8 held[nh][4];
            i32x8 next = frag(at, s0);
            float sh[nh];
            for (int n = 0; n < nh; ++n) {
                const i32x8 c = frag(at, h0 + 16 * n);
                for (int h = 0; h < 4; ++h)
                    held[n][h] = halves(c[2 * h], c[2 * h + 1]);
                if (hold_x)
                    sh[n] = row_scale(at, n) * f;
            }
            // sums scaled while the next tile's are formed, but with 256 rows,
            // where registers for one tile's sums are left alone
            constexpr int depth = BM == 256 ? 1 : 2;
            f32x4 pp[depth][nh];
            float s1 = 0.f;
            auto add = [&](int t, float st) {
                for (int n = 0; n < nh; ++n)
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (hold_x)
                            acc[n][t][i] = __builtin_fmaf(pp[t % depth][n][i], sh[n], acc[n][t][i]);
                        else
                            acc[t][n][i] = __builtin_fmaf(pp[t % depth][n][i], st, acc[t][n][i]);
                    }
            };
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < np; ++t) {
                const i32x8 c = next;
                const float st = s;
                if (t + 1 < np) {
                    next = frag(at, s0 + 16 * (t + 1));
                    if (!hold_x)
                        s = row_scale(at, t + 1) * f;
                }
                f32x4 (&p)[nh] = pp[t % depth];
                for (int n = 0; n < nh; ++n)
                    p[n] = f32x4{0.f, 0.f, 0.f, 0.f};
                for (int h = 0; h < 4; ++h) {
                    const f16x8 y = halves(c[2 * h], c[2 * h + 1]);
                    for (int n = 0; n < nh; ++n)
                        p[n] = hold_x ? __builtin_amdgcn_mfma_f32_16x16x32_f16(y, held[n][h], p[n], 0, 0, 0)
                                      : __builtin_amdgcn_mfma_f32_16x16x32_f16(held[n][h], y, p[n], 0, 0, 0);
                }
                if (depth == 1)
                    add(t, st);
                else if (t > 0)
                    add(t - 1, s1);
                s1 = st;
                __builtin_amdgcn_sched_barrier(0);
            }
            if (depth == 2)
                add(np - 1, s1);
        }
    };
    fill(0, 0);
    for (int64_t b = 0; b < nb; ++b) {
        const int cur = (b & 1) * T::words;
        const float f = sw[b];
        wait_vm_all();
        __syncthreads(); // this stage is filled, and everyone is done with the other buffer
        if (b + 1 < nb)
            fill(T::words - cur, b + 1);
        work(cur, f);
    }
    for (int t = 0; t < T::mt; ++t) {
        const int64_t m = m0 + wm + 16 * t + r;
        for (int n = 0; n < 4; ++n) {
            const int64_t c = n0 + wn + 16 * n + 4 * q;
            if (m < a.M)
                put4((O *)a.out + m * a.ldo + c, acc[t][n], a.N - c);
        }
    }
}

bool bad_rows(const void *p, int64_t ld, int64_t cols) { return (uintptr_t)p % 16 || ld % 16 || ld < cols; }

template <typename O> void run_skinny(const ProdArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)std::min<int64_t>((a.N + 15) / 16, kSkinnyGrid));
    const int64_t lds = (a.K + kBlk - 1) / kBlk * kBlk * a.M;
    if (lds <= kSkinnyX)
        hipLaunchKernelGGL((product_skinny_kernel<true, O>), grid, dim3(kSkinnyWaves * 64), (size_t)lds, st, a);
    else
        hipLaunchKernelGGL((product_skinny_kernel<false, O>), grid, dim3(kSkinnyWaves * 64), 0, st, a);
}

template <int BM, int BN, typename O> void run_tile(const ProdArgs &a, hipStream_t st)
{
    const int64_t n_mt = (a.M + BM - 1) / BM, n_nt = (a.N + BN - 1) / BN;
    const dim3 grid((unsigned)((n_nt + 7) / 8 * 8 * n_mt));
    hipLaunchKernelGGL((product_tile_kernel<BM, BN, sizeof(O) == 2 && (BM > 64), O>), grid, dim3(BN * 2), 0, st, a);
}

template <typename O> archead_status run_product(const ProdArgs &a, hipStream_t st)
{
    if (a.M <= kSkinnyM)
        run_skinny<O>(a, st);
    // 64 x 128, three of which run beside each other on a compute unit, for few
    // rows (64 x 151936 x 4096, fp32: 166 us; 128 x 128: 188) and, in fp32,
    // where 128 x 128 would leave compute units idle or alone with one (512 x 4096
    // x 4096: 29 us against 42; 1000 x 4096 x 4096: 42 against 43).
    else if (a.M <= 64 || (sizeof(O) == 4 && (a.M + 127) / 128 * ((a.N + 127) / 128) <= kCu))
        run_tile<64, 128, O>(a, st);
    else {
        // 128 x 128, two of which run beside each other on a compute unit, or 256
        // x 256, which move and convert less per product (2048 x 151936 x 4096:
        // fp32 2.19 ms against 2.42, bf16 1.62 against 1.99) but fill a chip in
        // coarser steps (333 x 50021 x 2576, bf16: 115 us against 90; 2048 x
        // 50021 x 2576, fp32: 620 against 596): by the rounds each takes, a round
        // of the large ones being 1.64 (bf16, in fp8) or 1.88 times (fp32, in
        // fp16) as long.
        auto rounds = [&](int64_t b, int64_t places) {
            return double(((a.M + b - 1) / b * ((a.N + b - 1) / b) + places - 1) / places);
        };
        if ((sizeof(O) == 2 ? 1.64 : 1.88) * rounds(256, kCu) < rounds(128, 2 * kCu))
            run_tile<256, 256, O>(a, st);
        else
            run_tile<128, 128, O>(a, st);
    }
    return launched("archead_fp8_matmul");
}

} // namespace
} // namespace archead

using namespace archead;

extern "C" archead_status archead_fp8_quantize(int64_t rows, int64_t cols, const void *x, int type, int64_t ldx,
                                               int block_rows, uint8_t *q, int64_t ldq, float *s, int64_t lds,
                                               void *hip_stream)
{
    if (rows < 0)
        return api_fail(ARCHEAD_EINVAL, "rows < 0");
    if (rows >= (int64_t(1) << 31) || cols < 16 || cols % 16 || cols > (int64_t(1) << 20) ||
        rows * ((cols + kBlk - 1) / kBlk) >= (int64_t(1) << 28))
        return api_fail(ARCHEAD_ESHAPE, "rows < 2^31, cols a multiple of 16 in [16, 2^20], fewer than 2^28 row blocks");
    if (type != ARCHEAD_F32 && type != ARCHEAD_BF16)
        return api_fail(ARCHEAD_EINVAL, "x must be ARCHEAD_F32 or ARCHEAD_BF16");
    if (block_rows != 1 && block_rows != kBlk)
        return api_fail(ARCHEAD_EINVAL, "block_rows must be 1 or 128");
    const int64_t nb = (cols + kBlk - 1) / kBlk;
    // a launch holds fewer than 2^32 threads: 2^24 - 1 workgroups of 256, 16 row blocks each
    if (block_rows == 1 && rows * nb > (int64_t(1) << 28) - 16)
        return api_fail(ARCHEAD_ESHAPE, "with a scale per row at most 2^28 - 16 row blocks");
    if (ldx < cols || lds < (block_rows == 1 ? rows : nb))
        return api_fail(ARCHEAD_EINVAL, "a row stride is shorter than a row");
    if (rows == 0)
        return ARCHEAD_OK;
    if (!x || !q || !s)
        return api_fail(ARCHEAD_EINVAL, "x, q and s are required");
    if ((uintptr_t)x % (type == ARCHEAD_F32 ? 4 : 2) || bad_rows(q, ldq, cols))
        return api_fail(ARCHEAD_EINVAL, "x aligned to its element; q and its row stride to 16 bytes");
    hipStream_t st = (hipStream_t)hip_stream;
    const bool by_rows = block_rows == 1;
    const int64_t groups = by_rows ? (rows * nb + 15) / 16 : (rows + kBlk - 1) / kBlk * nb;
    const bool exact = type == ARCHEAD_BF16 && groups <= (by_rows ? kExactRows : kExactTiles);
    const dim3 grid((unsigned)groups);
    const float *x4 = (const float *)x;
    const uint16_t *x2 = (const uint16_t *)x;
    if (by_rows && type == ARCHEAD_F32)
        hipLaunchKernelGGL((quant_rows_kernel<float, false>), grid, dim3(256), 0, st, x4, ldx, rows, cols, q, ldq, s, lds);
    else if (by_rows && exact)
        hipLaunchKernelGGL((quant_rows_kernel<uint16_t, true>), grid, dim3(256), 0, st, x2, ldx, rows, cols, q, ldq, s, lds);
    else if (by_rows)
        hipLaunchKernelGGL((quant_rows_kernel<uint16_t, false>), grid, dim3(256), 0, st, x2, ldx, rows, cols, q, ldq, s, lds);
    else if (type == ARCHEAD_F32)
        hipLaunchKernelGGL((quant_tiles_kernel<float, false>), grid, dim3(256), 0, st, x4, ldx, rows, cols, q, ldq, s, lds);
    else if (exact)
        hipLaunchKernelGGL((quant_tiles_kernel<uint16_t, true>), grid, dim3(256), 0, st, x2, ldx, rows, cols, q, ldq, s, lds);
    else
        hipLaunchKernelGGL((quant_tiles_kernel<uint16_t, false>), grid, dim3(256), 0, st, x2, ldx, rows, cols, q, ldq, s, lds);
    return launched("archead_fp8_quantize");
}

extern "C" archead_status archead_fp8_matmul(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda,
                                             const float *sA, int64_t ldsa, const uint8_t *B, int64_t ldb,
                                             const float *sB, int64_t ldsb, void *out, int out_type, int64_t ldo,
                                             void *hip_stream)
{
    if (M < 0 || N < 0)
        return api_fail(ARCHEAD_EINVAL, "M < 0 or N < 0");
    // a launch holds fewer than 2^32 threads: the tiles have one for 32 elements or more
    if (M > (int64_t(1) << 20) || N > (int64_t(1) << 30) || M * N > (int64_t(1) << 36) || K < 16 || K % 16 ||
        K > (int64_t(1) << 20))
        return api_fail(ARCHEAD_ESHAPE, "M <= 2^20, N <= 2^30, M N <= 2^36 and K a multiple of 16 in [16, 2^20]");
    if (out_type != ARCHEAD_F32 && out_type != ARCHEAD_BF16)
        return api_fail(ARCHEAD_EINVAL, "out must be ARCHEAD_F32 or ARCHEAD_BF16");
    const int64_t nb = (K + kBlk - 1) / kBlk;
    if (ldsa < M || ldsb < nb || ldo < N)
        return api_fail(ARCHEAD_EINVAL, "a row stride is shorter than a row");
    if (M == 0 || N == 0)
        return ARCHEAD_OK;
    if (!A || !sA || !B || !sB || !out)
        return api_fail(ARCHEAD_EINVAL, "A, sA, B, sB and out are required");
    if (lda >= kMaxStride || ldb >= kMaxStride)
        return api_fail(ARCHEAD_ESHAPE, "row strides of A and B must lie below 2^23 bytes");
    if (bad_rows(A, lda, K) || bad_rows(B, ldb, K))
        return api_fail(ARCHEAD_EINVAL, "A, B and their row strides must be multiples of 16 bytes, strides at least K");
    if ((uintptr_t)out % (out_type == ARCHEAD_F32 ? 4 : 2))
        return api_fail(ARCHEAD_EINVAL, "out must be aligned to its element");
    hipStream_t st = (hipStream_t)hip_stream;
    const ProdArgs a{M, N, K, lda, ldb, ldo, ldsa, ldsb, A, B, sA, sB, out};
    if (out_type == ARCHEAD_F32)
        return run_product<float>(a, st);
    return run_product<uint16_t>(a, st);
}
