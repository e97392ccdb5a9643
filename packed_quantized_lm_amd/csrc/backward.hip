// backward.hip -- the packed head's gradient by its hidden states,
//   dX[m, j] = sum_v G[m, v] W_hat[v, j],   G = dlogits,
// with W_hat in its stored fields (eq 6 and the text after eq 7 of the
// ARCHead paper; the head itself is frozen), again without a dense W_hat:
//   dX = G (sR o R4) + (T sB) B8 + sum_grp (U sD_grp) D8_grp,
//   T = G (sA o A5),  U = G (sC o C8).
//
// Everything that sums over the vocabulary is one kind of product: rows of G
// against integer codes with a scale per (v, 32 columns): R4's 4-bit codes, and
// A5's and C8's as bytes.  The codes are laid out a second time, eight
// vocabulary rows of one column beside each other (the forward's layout holds
// eight columns of one row), so that a dword of nibbles, or two of bytes, is one
// lane's matrix operand.
//
//   amax, convert  G 2^f_m as fp16 rows, f_m putting row m's largest entry
//                  into [2^14, 2^15): exact for bf16 G within 2^28 of it
//   tile kernel    [BM rows x 256 columns of dX, 128 of T and U] over a range
//                  of the vocabulary
//   sums           T sB and U from their ranges, fp32
//   finish         dX's ranges + the products with B8 and D8, one rounding
// Few rows are bound by the codes' bytes, many by the matrix cores.  In us:
//                    16 x 151936 x 4096     2048 x 151936 x 4096
//   amax, convert         10                    240  (6.1 TB/s fetched and written)
//   tiles                 86 (5.1 TB/s)         322 + 1919 (1330 TFLOP/s in dX's,
//                                               matrix cores 65 % busy)
//   sums, finish          16                     73
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <string>
#include <type_traits>

#include "api_internal.hpp"
#include "archead.h"
#include "device.hpp"
#include "lds_copy.hpp"

namespace archead {
namespace {

constexpr int kVC = 128;    // vocabulary rows per stage ("chunk")
constexpr int kJT = 256;    // columns per tile of dX
constexpr int kLT = 128;    // columns per tile of T and U
constexpr int kUnit = 32;   // columns that share a scale
constexpr int64_t kChunkM = 2048; // most rows of G held at a time
constexpr int64_t kMaxV = int64_t(1) << 22; // a tile's offsets into G fit 32 bits

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x8u __attribute__((ext_vector_type(8), aligned(2)));
typedef uint16_t u16x4u __attribute__((ext_vector_type(4), aligned(2)));

// Columns of the second layout: dX's d columns, and the columns of T and U by
// units of 32: kst units of the core, then rst of the correction.
struct Cols {
    int64_t d, kst, rst;
    __host__ __device__ int64_t main_tiles() const { return (d + kJT - 1) / kJT; }
    __host__ __device__ int64_t low_units() const { return kst + rst; }
    __host__ __device__ int64_t low_tiles() const { return (low_units() * kUnit + kLT - 1) / kLT; }
};
Cols cols_of(const Shape &s) { return Cols{s.d, s.kst(), s.rst()}; }

// ---------------------------------------------------------------------------
// The second layout (once per head)
//   codes uint32 [chunk][16-column block][64 lanes][4]: lane l holds column
//         l % 16 of the block, dword s the chunk's rows 32 s + 8 (l / 16) + e,
//         e = 0 .. 7, offset binary, in the nibble order of the first layout
//   low   uint32 [chunk][block][2][64 lanes][4]: the same rows of a core or
//         correction column as bytes a + 16 or c + 128, dwords 2 s and 2 s + 1 of
//         a lane in half s / 2
//   sc, lsc  fp16 [chunk][unit][128 rows], scale 2^E, the exponents E (ex:
//         residual, core, correction) keeping every code times scale below 2^15
//   b8t, d8t  int8 [d][kpad], [d][rpad]: B8 and D8 by columns
// ---------------------------------------------------------------------------
struct Layout {
    DevHead h;
    Cols c;
    int64_t nvc;
    uint32_t *codes, *low;
    uint16_t *sc, *lsc;
    int8_t *b8t, *d8t;
    uint32_t *peak; // largest |sR|, |sA|, |sC| as fp32 bits
    int32_t *ex;
};

__global__ __launch_bounds__(256) void peak_kernel(Layout a)
{
    const int which = blockIdx.y;
    const uint16_t *p = which == 0 ? a.h.sr : which == 1 ? a.h.sa : a.h.sc;
    const int64_t n = which == 0 ? (int64_t)a.h.s.n_sr() : (int64_t)a.h.s.n_rows();
    float m = 0.f;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const float f = fabsf(h2f(p[i]));
        m = f <= 65504.f ? fmaxf(m, f) : m; // NaN and Inf scales only propagate
    }
    for (int off = 32; off >= 1; off >>= 1)
        m = fmaxf(m, __shfl_xor(m, off));
    if ((threadIdx.x & 63) == 0)
        atomicMax(a.peak + which, __float_as_uint(m)); // any order gives the same maximum
}

__global__ void exponent_kernel(Layout a)
{
    const int w = threadIdx.x;
    if (w >= 3)
        return;
    const float m = __uint_as_float(a.peak[w]) * (w == 0 ? 1.f : w == 1 ? 2.f : 16.f);
    a.ex[w] = m > 0.f ? 11 - ilogbf(m) : 0; // codes reach 8, 16 and 128
}

// residual code (offset binary) of row v, column j in the first layout
__device__ __forceinline__ uint32_t r4_code(const DevHead &h, int64_t v, int64_t j)
{
    const int64_t lane = (v & 15) + 16 * ((j >> 3) & 3);
    const uint32_t w = h.r4[(((j >> 7) * h.s.nvb() + (v >> 4)) * 64 + lane) * 4 + ((j >> 5) & 3)];
    const int e = (int)(j & 7);
    return w >> (4 * ((e >> 1) + 4 * (e & 1))) & 15u;
}
// core code + 16, correction code + 128
__device__ __forceinline__ uint32_t a5_code(const DevHead &h, int64_t v, int64_t i)
{
    const int64_t ks = i >> 5, q = ks % 3, lane = (v & 15) + 16 * ((i >> 3) & 3);
    const uint32_t *c = h.lr + (((ks / 3) * h.s.nvb() + (v >> 4)) * 64 + lane) * 4;
    const int e = (int)(i & 7);
    const uint32_t nib = c[q] >> (4 * ((e >> 1) + 4 * (e & 1))) & 15u;
    return nib | (c[3] >> ((4 + 4 * q + (e >> 1) + 16 * (e & 1)) & 31) & 1u) << 4;
}
__device__ __forceinline__ uint32_t c8_code(const DevHead &h, int64_t v, int64_t i)
{
    const int64_t ks = i >> 5, lane = (v & 15) + 16 * ((i >> 3) & 3);
    const uint32_t *c = h.lr + (((h.s.lr_na() + ks / 2) * h.s.nvb() + (v >> 4)) * 64 + lane) * 4;
    return c[2 * (ks & 1) + ((i >> 2) & 1)] >> (8 * (i & 3)) & 255u;
}

// one dword of nibbles per thread; workgroup (block, chunk), at most 2^15 chunks
__global__ __launch_bounds__(256) void codes_kernel(Layout a, int64_t nblk)
{
    const int64_t vc = blockIdx.y, blk = blockIdx.x; // chunk, 16-column block
    const int lane = threadIdx.x >> 2, s = threadIdx.x & 3;
    const int64_t j = blk * 16 + (lane & 15);
    uint32_t w = 0;
    for (int e = 0; e < 8; ++e) {
        const int64_t v = vc * kVC + 32 * s + 8 * (lane >> 4) + e;
        // the first layout's padding rows hold codes of zero
        const uint32_t u = v < a.h.s.nvb() * kVB && j < a.h.s.d ? r4_code(a.h, v, j) : 8u;
        w |= u << (4 * ((e >> 1) + 4 * (e & 1)));
    }
    a.codes[((vc * nblk + blk) * 64 + lane) * 4 + s] = w;
}

// one dword of bytes per thread
__global__ __launch_bounds__(512) void low_codes_kernel(Layout a, int64_t nblk)
{
    const int64_t vc = blockIdx.y, blk = blockIdx.x;
    const int half = threadIdx.x >> 8, lane = threadIdx.x >> 2 & 63, dw = threadIdx.x & 3;
    const int64_t unit = blk / 2, i = (blk & 1) * 16 + (lane & 15);
    uint32_t w = 0;
    for (int e = 0; e < 4; ++e) {
        const int64_t v = vc * kVC + 32 * (2 * half + (dw >> 1)) + 8 * (lane >> 4) + 4 * (dw & 1) + e;
        const bool in = v < a.h.s.nvb() * kVB;
        uint32_t u = unit < a.c.kst ? 16u : 128u;
        if (in && unit < a.c.kst)
            u = a5_code(a.h, v, unit * kUnit + i);
        else if (in && unit < a.c.low_units())
            u = c8_code(a.h, v, (unit - a.c.kst) * kUnit + i);
        w |= u << (8 * e);
    }
    a.low[(((vc * nblk + blk) * 2 + half) * 64 + lane) * 4 + dw] = w;
}

__global__ __launch_bounds__(128) void scales_kernel(Layout a, int64_t nunit)
{
    const int64_t vc = blockIdx.y, unit = blockIdx.x, v = vc * kVC + threadIdx.x;
    float f = 0.f;
    if (v < a.h.s.V && unit * kUnit < a.h.s.d)
        f = ldexpf(h2f(a.h.sr[((v >> 4) * a.h.s.G() + unit * kUnit / a.h.s.g) * kVB + (v & 15)]), a.ex[0]);
    a.sc[(vc * nunit + unit) * kVC + threadIdx.x] = __builtin_bit_cast(uint16_t, (_Float16)f);
}

__global__ __launch_bounds__(128) void low_scales_kernel(Layout a, int64_t nunit)
{
    const int64_t vc = blockIdx.y, unit = blockIdx.x, v = vc * kVC + threadIdx.x;
    float f = 0.f;
    if (v < a.h.s.V && unit < a.c.kst)
        f = ldexpf(h2f(a.h.sa[v]), a.ex[1]);
    else if (v < a.h.s.V && unit < a.c.low_units())
        f = ldexpf(h2f(a.h.sc[v]), a.ex[2]);
    a.lsc[(vc * nunit + unit) * kVC + threadIdx.x] = __builtin_bit_cast(uint16_t, (_Float16)f);
}

__global__ __launch_bounds__(256) void columns_kernel(const int8_t *x, int64_t rows, int64_t d, int64_t pad, int8_t *out)
{
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < d * pad; t += (int64_t)gridDim.x * 256) {
        const int64_t j = t / pad, i = t % pad;
        out[t] = i < rows ? x[i * d + j] : (int8_t)0;
    }
}

// ---------------------------------------------------------------------------
// G 2^f_m as fp16
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
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }

struct GArgs {
    const void *g;
    int64_t M, V, ld, Vp;  // Vp: V rounded up to chunks
    int64_t S, slice;      // slices of a row
    float *amax;           // [M][S]
    uint16_t *g16;         // [M][Vp]
    float *unscale;        // [M] 2^-f_m
};

// f_m: mx 2^f in [2^14, 2^15) (0 for a row of zeros or with an infinity)
__device__ __forceinline__ int row_exponent(float mx)
{
    return mx > 0.f && mx <= 3.4028235e38f ? min(14 - ilogbf(mx), 126) : 0;
}

template <typename T> __device__ __forceinline__ void load8_edge(const T *row, int64_t v, int64_t V, float x[8])
{
    if (v + 8 <= V) {
        load8(row + v, x);
        return;
    }
    for (int i = 0; i < 8; ++i)
        x[i] = v + i < V ? load1(row + v + i) : 0.f;
}

template <typename T> __global__ __launch_bounds__(256) void amax_kernel(GArgs a)
{
    __shared__ float red[4];
    const int64_t m = blockIdx.x / a.S, sl = blockIdx.x % a.S;
    const T *row = (const T *)a.g + m * a.ld;
    float mx = 0.f;
    const int64_t end = min((sl + 1) * a.slice, a.V);
    for (int64_t v = sl * a.slice + 8 * threadIdx.x; v < end; v += 256 * 8) {
        float x[8];
        load8_edge(row, v, a.V, x);
        for (int i = 0; i < 8; ++i)
            mx = fmaxf(mx, fabsf(x[i]));
    }
    for (int off = 32; off >= 1; off >>= 1)
        mx = fmaxf(mx, __shfl_xor(mx, off));
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = mx;
    __syncthreads();
    if (threadIdx.x == 0)
        a.amax[blockIdx.x] = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

template <typename T> __global__ __launch_bounds__(256) void convert_kernel(GArgs a)
{
    const int64_t m = blockIdx.x / a.S, sl = blockIdx.x % a.S;
    const T *row = (const T *)a.g + m * a.ld;
    float mx = 0.f;
    for (int64_t i = 0; i < a.S; ++i)
        mx = fmaxf(mx, a.amax[m * a.S + i]);
    const int f = row_exponent(mx);
    if (sl == 0 && threadIdx.x == 0)
        a.unscale[m] = ldexpf(1.f, -f);
    const float up = ldexpf(1.f, f);
    uint16_t *out = a.g16 + m * a.Vp;
    const int64_t end = min((sl + 1) * a.slice, a.Vp);
    for (int64_t v = sl * a.slice + 8 * threadIdx.x; v < end; v += 256 * 8) {
        float x[8];
        load8_edge(row, v, a.V, x);
        f16x8 o;
        for (int i = 0; i < 8; ++i)
            o[i] = (_Float16)(x[i] * up);
        *(f16x8 *)(out + v) = o;
    }
}

// Both in one pass over a row, a workgroup each: the second half finds the
// row's first H vectors of each thread in registers, the rest in the caches.
constexpr int kWide = 1024;
template <int H, typename T> __global__ __launch_bounds__(kWide) void convert_row_kernel(GArgs a)
{
    __shared__ float red[kWide / 64];
    const int64_t m = blockIdx.x;
    const T *row = (const T *)a.g + m * a.ld;
    typedef T Raw __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    Raw held[H];
    const int64_t nv = a.V / 8; // whole vectors; the rest of the row is one step of the loop below
#pragma unroll
    for (int h = 0; h < H; ++h)
        held[h] = nv ? *(const Raw *)(row + min((int64_t)threadIdx.x + h * kWide, nv - 1) * 8) : Raw{};
    auto value = [](T x) { return load1(&x); };
    float mx = 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h) // past the end the last vector again: the maximum stays
        for (int i = 0; i < 8; ++i)
            mx = fmaxf(mx, fabsf(value(held[h][i])));
    for (int64_t v = 8 * ((int64_t)threadIdx.x + H * kWide); v < a.V; v += 8 * kWide) {
        float x[8];
        load8_edge(row, v, a.V, x);
        for (int i = 0; i < 8; ++i)
            mx = fmaxf(mx, fabsf(x[i]));
    }
    if (nv < H * kWide && threadIdx.x < a.V - nv * 8)
        mx = fmaxf(mx, fabsf(load1(row + nv * 8 + threadIdx.x)));
    for (int off = 32; off >= 1; off >>= 1)
        mx = fmaxf(mx, __shfl_xor(mx, off));
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = mx;
    __syncthreads();
    for (int w = 0; w < kWide / 64; ++w)
        mx = fmaxf(mx, red[w]);
    const int f = row_exponent(mx);
    if (threadIdx.x == 0)
        a.unscale[m] = ldexpf(1.f, -f);
    const float up = ldexpf(1.f, f);
    uint16_t *out = a.g16 + m * a.Vp;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const int64_t v = threadIdx.x + h * kWide;
        if (v < nv) {
            f16x8 o;
            for (int i = 0; i < 8; ++i)
                o[i] = (_Float16)(value(held[h][i]) * up);
            *(f16x8 *)(out + 8 * v) = o;
        }
    }
    for (int64_t v = 8 * (threadIdx.x + min((int64_t)H * kWide, nv)); v < a.Vp; v += 8 * kWide) {
        float x[8];
        load8_edge(row, v, a.V, x);
        f16x8 o;
        for (int i = 0; i < 8; ++i)
            o[i] = (_Float16)(x[i] * up);
        *(f16x8 *)(out + v) = o;
    }
}

// ---------------------------------------------------------------------------
// tile kernel
// ---------------------------------------------------------------------------
struct TileArgs {
    const uint16_t *g16;
    const float *unscale;
    const uint32_t *codes;
    const uint16_t *sc;
    const int32_t *ex;
    int64_t M, Vp, nvc;
    int64_t n_jt, n_mt, S; // column tiles, row tiles, vocabulary ranges
    int64_t kst, units;    // core units and all units of the low-rank columns
    float *part;           // [S][M][columns of the tiles]
};

__device__ __forceinline__ f16x2 as_h2(uint32_t x) { return __builtin_bit_cast(f16x2, x); }

// Eight nibbles of a lane as fp16 q S: the codes spliced into 1024 + u (and
// 1024 + 16 u), exact integers after one add (one fma), one rounding in the
// product with the scales.
__device__ __forceinline__ f16x8 dequant4(uint32_t w, u32x4 s, uint32_t magic)
{
    const f16x2 off0 = {(_Float16)-1032.f, (_Float16)-1032.f}, off1 = {(_Float16)-72.f, (_Float16)-72.f};
    const f16x2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
    const uint32_t w8 = w >> 8;
    const f16x2 a = (as_h2((w & 0x000F000Fu) | magic) + off0) * as_h2(s.x);
    const f16x2 b = __builtin_elementwise_fma(as_h2((w & 0x00F000F0u) | magic), sixteenth, off1) * as_h2(s.y);
    const f16x2 c = (as_h2((w8 & 0x000F000Fu) | magic) + off0) * as_h2(s.z);
    const f16x2 d = __builtin_elementwise_fma(as_h2((w8 & 0x00F000F0u) | magic), sixteenth, off1) * as_h2(s.w);
    return f16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// eight bytes likewise; off = -(1024 + the codes' offset)
__device__ __forceinline__ f16x8 dequant8(uint32_t w0, uint32_t w1, u32x4 s, uint32_t magic, f16x2 off)
{
    // bytes 2 p, 2 p + 1 of a dword into the low bytes of two halves, the high
    // ones from magic (1024 in fp16)
    const f16x2 a = (as_h2(__builtin_amdgcn_perm(magic, w0, 0x05010500u)) + off) * as_h2(s.x);
    const f16x2 b = (as_h2(__builtin_amdgcn_perm(magic, w0, 0x05030502u)) + off) * as_h2(s.y);
    const f16x2 c = (as_h2(__builtin_amdgcn_perm(magic, w1, 0x05010500u)) + off) * as_h2(s.z);
    const f16x2 d = (as_h2(__builtin_amdgcn_perm(magic, w1, 0x05030502u)) + off) * as_h2(s.w);
    return f16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

template <int BM, bool LOW> struct BTile {
    // waves along rows and columns: each 64 columns of dX, at least 32 of T and U
    static constexpr int wm = BM == 256 ? LOW ? 4 : 2 : 1, wj = 8 / wm;
    // vocabulary rows of G per stage: half a chunk where a whole one of 256
    // rows would not fit twice; codes and scales come by whole chunks
    static constexpr int gv = BM == 256 ? kVC / 2 : kVC, parts = kVC / gv;
    static constexpr int jt = LOW ? kLT : kJT;
    static constexpr int mt = BM / wm / 16, jb = jt / wj / 16;     // 16 x 16 tiles per wave
    static constexpr int un = jb > 1 ? jb / 2 : 1;                 // units of 32 columns per wave
    static constexpr int bw = LOW ? 512 : 256;                     // words of a 16-column block's codes
    static constexpr int su = jt / kUnit;                          // units of a tile
    static constexpr int gw = BM * gv / 2, cw = jt / 16 * bw, sw = su * kVC / 2; // words of a buffer: G, codes, scales
    static constexpr int kw = cw + sw, words = 2 * (gw + kw);      // G twice, codes with scales twice
};

// workgroup wg of a's tiles
template <int BM, bool LOW, int N>
__device__ __forceinline__ void tile_of(const TileArgs &a, uint32_t (&smem)[N], int64_t wg)
{
    using T = BTile<BM, LOW>;
    static_assert(T::words <= N, "LDS");
    const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Workgroup wg runs on XCD wg mod 8; an XCD takes a contiguous run of
    // (range, row tile, column tile), column tiles fastest, so that the rows
    // of G pass through one L2 for all column tiles.
    const int64_t total = a.S * a.n_mt * a.n_jt, per = (total + 7) / 8;
    const int64_t id = (wg & 7) * per + (wg >> 3);
    if (id >= total)
        return;
    const int64_t jt = id % a.n_jt, mi = id / a.n_jt % a.n_mt, sp = id / a.n_jt / a.n_mt;
    const int64_t m0 = mi * BM;
    const int64_t c0 = a.nvc * sp / a.S, c1 = a.nvc * (sp + 1) / a.S;
    const int wm0 = wv / T::wj * (BM / T::wm), wj0 = wv % T::wj * T::jb; // first row, first 16-column block

    // Stage i of this range: G's vocabulary rows T::gv i .., and with every
    // T::parts-th stage a chunk's codes.  G comes in 1 KiB copies of rows of
    // 2 T::gv bytes, 16-byte pieces exchanged by the row's low bits so that
    // eight rows' reads fall on different banks.
    constexpr int pieces = T::gv / 8, rows = 64 / pieces, copies = T::gw / 2048; // of a row; of a copy; per wave
    const uint16_t *gbase = a.g16 + m0 * a.Vp + c0 * kVC;
    uint32_t goff[copies]; // byte offsets from it: rows are shorter than 2^24 bytes
#pragma unroll
    for (int c = 0; c < copies; ++c) {
        const int row = rows * (8 * c + wv) + lane / pieces;
        goff[c] = (uint32_t)min((int64_t)row, a.M - 1 - m0) * (uint32_t)(2 * a.Vp) +
                  16 * ((lane % pieces) ^ (row & 7));
    }
    const uint32_t lds0 = lds_address(smem), lane16 = 16 * lane;
    auto fill = [&](int64_t i) {
        const uint32_t g = lds0 + 4 * (uint32_t)((int)(i & 1) * T::gw);
#pragma unroll
        for (int c = 0; c < copies; ++c)
            lds_dma16_from(gbase + i * T::gv, goff[c], g + 1024 * (8 * c + wv));
        if (i % T::parts == 0) {
            const int64_t at = (c0 + i / T::parts) * a.n_jt + jt;
            const uint32_t k = lds0 + 4 * (uint32_t)(2 * T::gw + (int)(i / T::parts & 1) * T::kw);
#pragma unroll
            for (int c = 0; c < T::cw / 2048; ++c)
                lds_dma16_from(a.codes + at * T::cw + (8 * c + wv) * 256, lane16, k + 1024 * (8 * c + wv));
            if (wv < T::sw / 256)
                lds_dma16_from(a.sc + (at * T::su + 4 * wv) * kVC, lane16, k + 4 * T::cw + 1024 * wv);
        }
    };
    const uint32_t magic = vgpr_const(kF16Magic);
    f16x2 off[T::un]; // LOW: a core's or a correction's byte offset
    bool idle = LOW;  // and whether this wave's columns are padding only
    for (int u = 0; u < T::un; ++u) {
        const int64_t unit = jt * T::su + (wj0 >> 1) + u;
        const _Float16 o = (_Float16)(LOW && unit < a.kst ? -1040.f : -1152.f);
        off[u] = f16x2{o, o};
        idle = idle && unit >= a.units;
    }
    f32x4 acc[T::mt][T::jb];
    for (int t = 0; t < T::mt; ++t)
        for (int n = 0; n < T::jb; ++n)
            acc[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};

    u32x4 c[T::jb];
    // the 32-row steps of part h of a chunk
    auto work = [&](int g, int k, auto part) {
        constexpr int h = decltype(part)::value;
        if constexpr (!LOW && h == 0)
            for (int n = 0; n < T::jb; ++n)
                c[n] = *(const u32x4 *)&smem[k + (wj0 + n) * 256 + lane * 4];
#pragma unroll
        for (int s = h * 4 / T::parts; s < (h + 1) * 4 / T::parts; ++s) {
            if constexpr (LOW)
                if ((s & 1) == 0)
                    for (int n = 0; n < T::jb; ++n)
                        c[n] = *(const u32x4 *)&smem[k + (wj0 + n) * 512 + (s >> 1) * 256 + lane * 4];
            f16x8 w[T::jb];
            for (int u = 0; u < T::un; ++u) {
                const u32x4 sc = *(const u32x4 *)&smem[k + T::cw + ((wj0 >> 1) + u) * (kVC / 2) + 16 * s + 4 * q];
                for (int n = 2 * u; n < 2 * u + 2 && n < T::jb; ++n) {
                    if constexpr (LOW)
                        w[n] = dequant8(c[n][2 * (s & 1)], c[n][2 * (s & 1) + 1], sc, magic, off[u]);
                    else
                        w[n] = dequant4(c[n][s], sc, magic);
                }
            }
            for (int t = 0; t < T::mt; ++t) {
                const int row = wm0 + 16 * t + r; // row & 7 = r & 7
                const f16x8 x = *(const f16x8 *)&smem[g + row * (T::gv / 2) + 4 * ((4 * (s % (4 / T::parts)) + q) ^ (r & 7))];
                for (int n = 0; n < T::jb; ++n)
                    acc[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[n], x, acc[t][n], 0, 0, 0);
            }
        }
    };
    const int64_t stages = (c1 - c0) * T::parts;
    if (stages > 0)
        fill(0);
    for (int64_t i = 0; i < stages; i += T::parts) {
        const int k = 2 * T::gw + (int)(i / T::parts & 1) * T::kw;
        auto stage = [&](auto part) {
            const int64_t j = i + decltype(part)::value;
            wait_vm_all();
            __syncthreads(); // this stage is filled, and everyone is done with the other buffers
            if (j + 1 < stages)
                fill(j + 1);
            if (!LOW || !idle)
                work((int)(j & 1) * T::gw, k, part);
        };
        stage(std::integral_constant<int, 0>{});
        if constexpr (T::parts == 2)
            stage(std::integral_constant<int, 1>{});
    }
    if (idle)
        return;
    // lane: row m = r of each row tile, four consecutive columns
    for (int n = 0; n < T::jb; ++n) {
        const float down = ldexpf(1.f, -a.ex[!LOW ? 0 : jt * T::su + ((wj0 + n) >> 1) < a.kst ? 1 : 2]);
        for (int t = 0; t < T::mt; ++t) {
            const int64_t m = m0 + wm0 + 16 * t + r;
            if (m < a.M) {
                f32x4 o = acc[t][n];
                const float un = a.unscale[m];
                for (int i = 0; i < 4; ++i)
                    o[i] = o[i] * down * un;
                *(f32x4 *)(a.part + ((sp * a.M + m) * a.n_jt + jt) * T::jt + (wj0 + n) * 16 + 4 * q) = o;
            }
        }
    }
}

// T's and U's tiles, the first low_groups workgroups (a multiple of 8), and dX's
// behind them
template <int BM> __global__ __launch_bounds__(512) void tile_kernel(TileArgs low, TileArgs main, uint32_t low_groups)
{
    constexpr int words = std::max(BTile<BM, true>::words, BTile<BM, false>::words);
    __shared__ __attribute__((aligned(16))) uint32_t smem[words];
    if (blockIdx.x < low_groups)
        tile_of<BM, true>(low, smem, blockIdx.x);
    else
        tile_of<BM, false>(main, smem, blockIdx.x - low_groups);
}

// ---------------------------------------------------------------------------
// T sB and U: the ranges' sums.  T sB is left in two bf16 parts (16
// significant bits), as the finish multiplies it.
// ---------------------------------------------------------------------------
struct LowArgs {
    int64_t M, S, k, r;
    Cols c;
    const float *part, *sb;
    uint16_t *thi, *tlo; // [M][kp]
    float *u;            // [M][rp]
};

constexpr int kLowLanes = 8; // threads that share a column's ranges

__global__ __launch_bounds__(256) void low_sum_kernel(LowArgs a)
{
    const int64_t kp = a.c.kst * kUnit, rp = a.c.rst * kUnit, w = kp + rp, pitch = a.c.low_tiles() * kLT;
    // thread (column, share): 32 columns of one row per workgroup (w is a multiple of 32)
    const int64_t t = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const int sh = threadIdx.x >> 5;
    const int64_t m = t / w, i = t % w;
    __shared__ float red[kLowLanes][32];
    const bool core = i < kp;
    float s = 0.f;
#pragma unroll 4
    for (int64_t p = sh; p < a.S; p += kLowLanes)
        s += a.part[(p * a.M + m) * pitch + i];
    red[sh][threadIdx.x & 31] = s;
    __syncthreads();
    if (sh)
        return;
    s = 0.f;
    for (int p = 0; p < kLowLanes; ++p)
        s += red[p][threadIdx.x];
    if (core) {
        const float x = i < a.k ? s * a.sb[i] : 0.f;
        const __bf16 h = (__bf16)x;
        a.thi[m * kp + i] = __builtin_bit_cast(uint16_t, h);
        a.tlo[m * kp + i] = __builtin_bit_cast(uint16_t, (__bf16)(x - (float)h));
    } else {
        a.u[m * rp + i - kp] = i - kp < a.r ? s : 0.f;
    }
}

// ---------------------------------------------------------------------------
// finish: one wave per [16 NT rows x 16 NJ columns], or with few rows (SPLIT)
// a workgroup's four waves, each with every fourth range and 32 columns of the
// factors: the loads' latency is what such a call waits for
// ---------------------------------------------------------------------------
struct FinishArgs {
    int64_t M, d, k, r, G, g, S, pitch; // pitch: columns of a range's rows
    Cols c;
    const float *part, *u, *sd;
    const uint16_t *thi, *tlo;
    const int8_t *b8t, *d8t;
    uint16_t *dx;
};

// eight int8 in order as exact bf16
__device__ __forceinline__ bf16x8 codes_bf16(const int8_t *p)
{
    const u32x2 w = *(const u32x2 *)p;
    return as_bf16x8(c8_bf16(u32x2{w.x ^ 0x80808080u, w.y ^ 0x80808080u}));
}

template <int NT, int NJ, bool SPLIT> __global__ __launch_bounds__(256) void finish_kernel(FinishArgs a)
{
    __shared__ f32x4 red[SPLIT ? 3 : 1][64];
    const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
    const int wv = threadIdx.x >> 6;
    constexpr int step = SPLIT ? 4 : 1;
    const int first = SPLIT ? wv : 0;
    const int64_t blocks = a.d / (16 * NJ), id = SPLIT ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + wv;
    const int64_t j0 = id % blocks * 16 * NJ, m0 = id / blocks * 16 * NT;
    if (m0 >= a.M)
        return;
    const int64_t kp = a.c.kst * kUnit, rp = a.c.rst * kUnit;
    f32x4 acc[NT][NJ];
    int64_t m[NT];
    for (int t = 0; t < NT; ++t) {
        m[t] = min(m0 + 16 * t + r, a.M - 1);
        for (int n = 0; n < NJ; ++n) {
            acc[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
            const float *p = a.part + m[t] * a.pitch + j0 + 16 * n + 4 * q;
#pragma unroll(NJ > 1 ? 1 : 8)
            for (int64_t i = first; i < a.S; i += step) // the ranges in order
                acc[t][n] += *(const f32x4 *)(p + i * a.M * a.pitch);
        }
    }
#pragma unroll(NJ > 1 ? 1 : 2)
    for (int64_t i = first * kUnit; i < kp; i += step * kUnit) {
        bf16x8 code[NJ];
        for (int n = 0; n < NJ; ++n)
            code[n] = codes_bf16(a.b8t + (j0 + 16 * n + r) * kp + i + 8 * q);
        for (int t = 0; t < NT; ++t) {
            const int64_t at = m[t] * kp + i + 8 * q;
            const bf16x8 hi = *(const bf16x8 *)(a.thi + at), lo = *(const bf16x8 *)(a.tlo + at);
            for (int n = 0; n < NJ; ++n) {
                acc[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(code[n], hi, acc[t][n], 0, 0, 0);
                acc[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(code[n], lo, acc[t][n], 0, 0, 0);
            }
        }
    }
    // U sD in two bf16 parts against the exact codes; NJ pairs of 16 columns
    // share a group by twos (groups are multiples of 32 columns)
    constexpr int NP = NJ > 1 ? 2 : 1;
    for (int64_t i = first * kUnit; i < rp; i += step * kUnit)
        for (int p = 0; p < NJ; p += NP) {
            bf16x8 code[NP];
            for (int n = 0; n < NP; ++n)
                code[n] = codes_bf16(a.d8t + (j0 + 16 * (p + n) + r) * rp + i + 8 * q);
            float sd[8];
            for (int e = 0; e < 8; ++e)
                sd[e] = i + 8 * q + e < a.r ? a.sd[(i + 8 * q + e) * a.G + (j0 + 16 * p) / a.g] : 0.f;
            for (int t = 0; t < NT; ++t) {
                float x[8];
                load8(a.u + m[t] * rp + i + 8 * q, x);
                bf16x8 hi, lo;
                for (int e = 0; e < 8; ++e) {
                    x[e] *= sd[e];
                    hi[e] = (__bf16)x[e];
                    lo[e] = (__bf16)(x[e] - (float)hi[e]);
                }
                for (int n = 0; n < NP; ++n) {
                    acc[t][p + n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(code[n], hi, acc[t][p + n], 0, 0, 0);
                    acc[t][p + n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(code[n], lo, acc[t][p + n], 0, 0, 0);
                }
            }
        }
    if constexpr (SPLIT) {
        static_assert(NT == 1 && NJ == 1, "one tile per workgroup");
        if (wv)
            red[wv - 1][lane] = acc[0][0];
        __syncthreads();
        if (wv)
            return;
        for (int w = 0; w < 3; ++w)
            acc[0][0] += red[w][lane];
    }
    for (int t = 0; t < NT; ++t)
        if (m0 + 16 * t + r < a.M)
            for (int n = 0; n < NJ; ++n) {
                u16x4u o;
                for (int i = 0; i < 4; ++i)
                    o[i] = __builtin_bit_cast(uint16_t, (__bf16)acc[t][n][i]);
                *(u16x4u *)(a.dx + m[t] * a.d + j0 + 16 * n + 4 * q) = o;
            }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
size_t up(size_t x) { return (x + 255) / 256 * 256; }

struct Plan {
    int bm;            // rows of a tile
    int64_t low, main; // vocabulary ranges of T's and U's tiles, and of dX's
};

// Row tiles and ranges by the time a launch is expected to take.  Ranges: the
// vocabulary is cut so that the workgroups fill the compute units' places (by
// LDS: one of 256 rows, two of 64, three of 32) in whole rounds, each with two
// stages of latency, against the ranges' sums written and read.  Tiles: 32 rows
// as far as they go; beyond, 256 rows take 3.5 us a chunk on a full chip and 64
// rows 2.2, so that 64 win where 256 would be mostly empty (260 rows of 151936 x
// 4096: 509 us against 613; 512 rows: 790 against 695) or need more ranges
// (1000 rows of 30011 x 640: 156 against 198).
constexpr int64_t kCu = 256, kMaxWg = 1024, kMinChunks = 2;
struct TileKind {
    int rows, places; // places on a compute unit
    double us;        // a chunk's time with all places taken
};
constexpr TileKind kTiles[] = {{32, 3, 2.6}, {64, 2, 2.2}, {256, 1, 3.5}};
constexpr double kSumRate = 4e6; // bytes a us

// the best ranges for tiles of one kind, and their time
double ranges_of(const TileKind &k, int64_t M, int64_t tiles, int64_t tile_cols, int64_t nvc, int64_t *ranges)
{
    const int64_t t = std::max<int64_t>(tiles * ((M + k.rows - 1) / k.rows), 1);
    const int64_t places = kCu * k.places, most = std::max<int64_t>(1, nvc / kMinChunks);
    const double sums = double(M) * double(tiles * tile_cols) * 8 / kSumRate;
    double least = 1e300;
    for (int64_t S = 1; S <= most && (S == 1 || S * t <= kMaxWg);) {
        const int64_t chunks = (nvc + S - 1) / S;
        const double cost = double((S * t + places - 1) / places) * (double(chunks) + 2.0) * k.us + double(S) * sums;
        if (cost < least * 0.995) {
            least = cost;
            *ranges = S;
        }
        if (chunks == 1)
            break;
        S = (nvc + chunks - 2) / (chunks - 1); // the fewest ranges that shorten the longest
    }
    return least;
}

Plan plan_of(const Cols &c, int64_t M, int64_t nvc)
{
    Plan best{};
    double least = 1e300;
    for (const TileKind &k : kTiles) {
        if ((k.rows == 32) != (M <= 32))
            continue;
        Plan p{k.rows, 1, 1};
        const double cost = ranges_of(k, M, c.main_tiles(), kJT, nvc, &p.main) +
                            (c.low_tiles() ? ranges_of(k, M, c.low_tiles(), kLT, nvc, &p.low) : 0.);
        if (cost < least) {
            least = cost;
            best = p;
        }
    }
    return best;
}

constexpr int64_t kAmaxSlices = 64;

} // namespace

// byte offsets into the workspace
struct BackwardWs {
    size_t g16, amax, unscale, low, thi, tlo, u, part, total;
};

namespace {

// Fits every call of up to rows rows: the ranges' sums by the plans of all of them
// (151936 x 4096, k = 256, r = 64, 2048 rows: 623 MB for G, 264 MB for dX's sums,
// 33 MB for T's and U's: 923 MB).
BackwardWs backward_ws(const Shape &s, int64_t rows)
{
    const Cols c = cols_of(s);
    const int64_t nvc = (s.V + kVC - 1) / kVC;
    int64_t low = 0, part = 0;
    for (int64_t M = 1; M <= rows; ++M) {
        const Plan p = plan_of(c, M, nvc);
        low = std::max(low, p.low * M * c.low_tiles() * kLT);
        part = std::max(part, p.main * M * c.main_tiles() * kJT);
    }
    BackwardWs w;
    size_t off = 0;
    auto place = [&](size_t bytes) {
        const size_t o = off;
        off += up(std::max<size_t>(bytes, 16));
        return o;
    };
    w.g16 = place(size_t(rows) * nvc * kVC * 2);
    w.amax = place(size_t(rows) * kAmaxSlices * 4);
    w.unscale = place(size_t(rows) * 4);
    w.low = place(size_t(low) * 4);
    w.thi = place(size_t(rows) * c.kst * kUnit * 2);
    w.tlo = place(size_t(rows) * c.kst * kUnit * 2);
    w.u = place(size_t(rows) * c.rst * kUnit * 4);
    w.part = place(size_t(part) * 4);
    w.total = off;
    return w;
}

} // namespace

struct BackwardState {
    void *block; // the second layout
    size_t block_bytes;
    uint32_t *codes, *low;
    uint16_t *sc, *lsc;
    int8_t *b8t, *d8t;
    int32_t *ex;
    void *ws;
    size_t ws_bytes;
    BackwardWs at; // in the workspace
    int64_t rows;  // rows it holds
};

void backward_release(BackwardState *b)
{
    if (!b)
        return;
    if (b->ws)
        (void)hipFree(b->ws);
    if (b->block)
        (void)hipFree(b->block);
    delete b;
}

size_t backward_bytes(const BackwardState *b) { return b ? b->block_bytes + b->ws_bytes : 0; }

namespace {

#define BW_TRY(expr)                                                                               \
    do {                                                                                           \
        hipError_t e_ = (expr);                                                                    \
        if (e_ != hipSuccess)                                                                      \
            return api_fail(ARCHEAD_EHIP, std::string(#expr) + ": " + hipGetErrorString(e_));      \
    } while (0)

archead_status device_alloc(void **p, size_t bytes, const char *what)
{
    *p = nullptr;
    if (alloc_refused(bytes))
        return api_fail(ARCHEAD_ENOMEM, std::string(what) + " of " + std::to_string(bytes) +
                                            " bytes refused (ARCHEAD_TEST_ALLOC_LIMIT)");
    const hipError_t e = hipMalloc(p, bytes);
    if (e != hipSuccess) {
        *p = nullptr;
        return api_fail(ARCHEAD_ENOMEM, std::string("hipMalloc of the ") + what + ": " + hipGetErrorString(e));
    }
    return ARCHEAD_OK;
}

// lays the codes out a second time into a fresh block
archead_status lay_out(const DevHead &h, BackwardState *b, hipStream_t st)
{
    Layout a{};
    a.h = h;
    a.c = cols_of(h.s);
    a.nvc = (h.s.V + kVC - 1) / kVC;
    const int64_t nblk = a.c.main_tiles() * 16, nunit = a.c.main_tiles() * (kJT / kUnit);
    const int64_t lblk = a.c.low_tiles() * (kLT / 16), lunit = a.c.low_tiles() * (kLT / kUnit);
    if (a.nvc * std::max(nblk, lblk) >= int64_t(1) << 31)
        return api_fail(ARCHEAD_ESHAPE, "head too large for the backward's layout");
    size_t off = 0;
    auto place = [&](size_t bytes) {
        const size_t o = off;
        off += up(std::max<size_t>(bytes, 16));
        return o;
    };
    const size_t kp = a.c.kst * kUnit, rp = a.c.rst * kUnit;
    const size_t o_codes = place(size_t(a.nvc) * nblk * 1024), o_sc = place(size_t(a.nvc) * nunit * kVC * 2);
    const size_t o_low = place(size_t(a.nvc) * lblk * 2048), o_lsc = place(size_t(a.nvc) * lunit * kVC * 2);
    const size_t o_b8 = place(h.s.d * kp), o_d8 = place(h.s.d * rp), o_ex = place(64);
    archead_status s = device_alloc(&b->block, off, "backward layout");
    if (s != ARCHEAD_OK)
        return s;
    b->block_bytes = off;
    char *p = (char *)b->block;
    a.codes = b->codes = (uint32_t *)(p + o_codes);
    a.sc = b->sc = (uint16_t *)(p + o_sc);
    a.low = b->low = (uint32_t *)(p + o_low);
    a.lsc = b->lsc = (uint16_t *)(p + o_lsc);
    a.b8t = b->b8t = (int8_t *)(p + o_b8);
    a.d8t = b->d8t = (int8_t *)(p + o_d8);
    a.ex = b->ex = (int32_t *)(p + o_ex);
    a.peak = (uint32_t *)(p + o_ex + 32);
    BW_TRY(hipMemsetAsync(p + o_ex, 0, 64, st)); // never under capture (checked by the caller)
    hipLaunchKernelGGL(peak_kernel, dim3(256, 3), dim3(256), 0, st, a);
    hipLaunchKernelGGL(exponent_kernel, dim3(1), dim3(64), 0, st, a);
    hipLaunchKernelGGL(codes_kernel, dim3((unsigned)nblk, (unsigned)a.nvc), dim3(256), 0, st, a, nblk);
    hipLaunchKernelGGL(scales_kernel, dim3((unsigned)nunit, (unsigned)a.nvc), dim3(kVC), 0, st, a, nunit);
    if (lblk) {
        hipLaunchKernelGGL(low_codes_kernel, dim3((unsigned)lblk, (unsigned)a.nvc), dim3(512), 0, st, a, lblk);
        hipLaunchKernelGGL(low_scales_kernel, dim3((unsigned)lunit, (unsigned)a.nvc), dim3(kVC), 0, st, a, lunit);
    }
    if (kp)
        hipLaunchKernelGGL(columns_kernel, dim3(1024), dim3(256), 0, st, h.b8, h.s.k, h.s.d, (int64_t)kp, a.b8t);
    if (rp)
        hipLaunchKernelGGL(columns_kernel, dim3(1024), dim3(256), 0, st, h.d8, h.s.r, h.s.d, (int64_t)rp, a.d8t);
    BW_TRY(hipGetLastError());
    return ARCHEAD_OK;
}

// Neither kind of tile waits for the other, and a launch of both saves the end
// of one: 1 row of 151936 x 4096 98 us against 106, 133 rows of 30011 x 640 44
// against 47.  Where both would come in several rounds they get in each other's
// way (2048 rows of 151936 x 4096: 2.61 ms together, 2.55 apart; 300 rows of
// 50257 x 1280: 100 us, 94).
void run_tiles(int bm, const TileArgs &low, const TileArgs &main, hipStream_t st)
{
    auto groups = [](const TileArgs &a) { return (uint32_t)((a.S * a.n_mt * a.n_jt + 7) / 8 * 8); };
    auto launch = [&](uint32_t n, uint32_t grid) {
        if (bm == 32)
            hipLaunchKernelGGL(tile_kernel<32>, dim3(grid), dim3(512), 0, st, low, main, n);
        else if (bm == 64)
            hipLaunchKernelGGL(tile_kernel<64>, dim3(grid), dim3(512), 0, st, low, main, n);
        else
            hipLaunchKernelGGL(tile_kernel<256>, dim3(grid), dim3(512), 0, st, low, main, n);
    };
    const uint32_t n = groups(low), all = n + groups(main), places = (uint32_t)kCu * (bm == 64 ? 2 : 1);
    if (n == 0 || bm == 32 || all <= places + places / 2)
        launch(n, all);
    else {
        launch(n, n);
        launch(0, all - n);
    }
}

// up to b.rows rows of G
void backward_rows(const DevHead &h, const BackwardState &b, int64_t M, const void *g, int type, int64_t ld,
                   uint16_t *dx, hipStream_t st)
{
    const Shape &s = h.s;
    const Cols c = cols_of(s);
    const BackwardWs &L = b.at;
    char *ws = (char *)b.ws;
    const int64_t nvc = (s.V + kVC - 1) / kVC;
    GArgs ga{};
    ga.g = g;
    ga.M = M;
    ga.V = s.V;
    ga.ld = ld;
    ga.Vp = nvc * kVC;
    const int64_t step = 256 * 8; // a workgroup's elements per step
    ga.S = std::max<int64_t>(1, std::min<int64_t>({kAmaxSlices, 2048 / std::max<int64_t>(M, 1), ga.Vp / step}));
    ga.slice = (ga.Vp + ga.S * step - 1) / (ga.S * step) * step;
    ga.S = (ga.Vp + ga.slice - 1) / ga.slice;
    ga.amax = (float *)(ws + L.amax);
    ga.g16 = (uint16_t *)(ws + L.g16);
    ga.unscale = (float *)(ws + L.unscale);
    const dim3 grid((unsigned)(M * ga.S));
    // long rows enough to fill most of a round of compute units: one pass each
    const bool whole = s.V >= kWide * 8 && 10 * M >= 7 * ((M + kCu - 1) / kCu * kCu);
    if (whole && type == ARCHEAD_F32)
        hipLaunchKernelGGL((convert_row_kernel<8, float>), dim3((unsigned)M), dim3(kWide), 0, st, ga);
    else if (whole)
        hipLaunchKernelGGL((convert_row_kernel<12, uint16_t>), dim3((unsigned)M), dim3(kWide), 0, st, ga);
    else if (type == ARCHEAD_F32) {
        hipLaunchKernelGGL(amax_kernel<float>, grid, dim3(256), 0, st, ga);
        hipLaunchKernelGGL(convert_kernel<float>, grid, dim3(256), 0, st, ga);
    } else {
        hipLaunchKernelGGL(amax_kernel<uint16_t>, grid, dim3(256), 0, st, ga);
        hipLaunchKernelGGL(convert_kernel<uint16_t>, grid, dim3(256), 0, st, ga);
    }
    const Plan p = plan_of(c, M, nvc);
    float *low = (float *)(ws + L.low), *u = (float *)(ws + L.u), *part = (float *)(ws + L.part);
    uint16_t *thi = (uint16_t *)(ws + L.thi), *tlo = (uint16_t *)(ws + L.tlo);
    TileArgs tl{};
    tl.g16 = ga.g16;
    tl.unscale = ga.unscale;
    tl.ex = b.ex;
    tl.M = M;
    tl.Vp = ga.Vp;
    tl.nvc = nvc;
    tl.kst = c.kst;
    tl.units = c.low_units();
    tl.n_mt = (M + p.bm - 1) / p.bm;
    TileArgs tm = tl;
    tl.codes = b.low;
    tl.sc = b.lsc;
    tl.n_jt = c.low_tiles();
    tl.S = p.low;
    tl.part = low;
    tm.codes = b.codes;
    tm.sc = b.sc;
    tm.n_jt = c.main_tiles();
    tm.S = p.main;
    tm.part = part;
    run_tiles(p.bm, tl, tm, st);
    if (c.low_tiles() > 0) {
        const LowArgs l{M, p.low, s.k, s.r, c, low, h.sb, thi, tlo, u};
        hipLaunchKernelGGL(low_sum_kernel, dim3((unsigned)(M * (c.kst + c.rst))), dim3(256), 0, st, l);
    }
    const FinishArgs f{M, s.d, s.k, s.r, s.G(), s.g, p.main, c.main_tiles() * kJT, c, part, u, h.sd, thi, tlo,
                       b.b8t, b.d8t, dx};
    // Measured, us of whole calls, split / 16 x 16 / 64 x 64:
    //   d      V       16 rows         64 rows         256 rows        512 rows        768 rows
    //   4096   20011   34/38/116       48/47/134       97/92/122       158/154/162     208/203/203
    //   1280   50257   36/49/312       47/48/288       88/84/175       134/130/175     182/184/207
    //   640    30011   29/34/194       35/42/323       53/51/178       81/79/154       104/100/154
    // The first border holds throughout; the second is that of d >= 4096, and for
    // shorter rows of more than 512 gradients 16 x 16 would be ahead.
    const int64_t tiles = (M + 15) / 16 * (s.d / 16), waves = (M + 63) / 64 * (s.d / 64);
    if (tiles <= 512)
        hipLaunchKernelGGL((finish_kernel<1, 1, true>), dim3((unsigned)tiles), dim3(256), 0, st, f);
    else if (M <= 512)
        hipLaunchKernelGGL((finish_kernel<1, 1, false>), dim3((unsigned)((tiles + 3) / 4)), dim3(256), 0, st, f);
    else
        hipLaunchKernelGGL((finish_kernel<4, 4, false>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, st, f);
}

} // namespace
} // namespace archead

using namespace archead;

extern "C" archead_status archead_reserve_backward(archead_t h, int64_t M_max, void *hip_stream)
{
    const DevHead *dev = nullptr;
    BackwardState **slot = nullptr;
    int device = 0;
    archead_status s = backward_slot(h, &dev, &slot, &device);
    if (s != ARCHEAD_OK)
        return s;
    if (M_max < 1)
        return api_fail(ARCHEAD_EINVAL, "M_max must be at least 1");
    if (M_max > int64_t(1) << 20)
        return api_fail(ARCHEAD_ESHAPE, "M_max above 2^20");
    if (dev->s.V > kMaxV)
        return api_fail(ARCHEAD_ESHAPE, "the backward takes V up to 2^22");
    const int64_t rows = std::min(M_max, kChunkM);
    if (*slot && (*slot)->rows >= rows)
        return ARCHEAD_OK;
    hipStream_t st = (hipStream_t)hip_stream;
    BW_TRY(hipSetDevice(device));
    hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
    BW_TRY(hipStreamIsCapturing(st, &cap));
    if (cap != hipStreamCaptureStatusNone)
        return api_fail(ARCHEAD_EINVAL, "archead_reserve_backward allocates: call it before the capture");
    // a state of its own until all of it is there
    BackwardState *b = *slot ? *slot : new (std::nothrow) BackwardState();
    if (!b)
        return api_fail(ARCHEAD_ENOMEM, "host allocation failed");
    void *ws = nullptr;
    const BackwardWs at = backward_ws(dev->s, rows);
    const size_t bytes = at.total;
    s = device_alloc(&ws, bytes, "backward workspace");
    if (s == ARCHEAD_OK && !b->block)
        s = lay_out(*dev, b, st);
    if (s == ARCHEAD_OK && hipStreamSynchronize(st) != hipSuccess)
        s = api_fail(ARCHEAD_EHIP, "the backward's layout did not complete");
    if (s != ARCHEAD_OK) {
        if (ws)
            (void)hipFree(ws);
        if (!*slot)
            backward_release(b);
        return s;
    }
    if (b->ws)
        (void)hipFree(b->ws); // waits for the device
    b->ws = ws;
    b->ws_bytes = bytes;
    b->at = at;
    b->rows = rows;
    *slot = b;
    return ARCHEAD_OK;
}

extern "C" archead_status archead_backward(archead_t h, int64_t M, const void *dlogits, int type, int64_t ld, void *dX,
                                           void *hip_stream)
{
    const DevHead *dev = nullptr;
    BackwardState **slot = nullptr;
    int device = 0;
    archead_status s = backward_slot(h, &dev, &slot, &device);
    if (s != ARCHEAD_OK)
        return s;
    if (M < 0)
        return api_fail(ARCHEAD_EINVAL, "M < 0");
    if (M > int64_t(1) << 20)
        return api_fail(ARCHEAD_ESHAPE, "M above 2^20");
    if (type != ARCHEAD_F32 && type != ARCHEAD_BF16)
        return api_fail(ARCHEAD_EINVAL, "dlogits must be ARCHEAD_F32 or ARCHEAD_BF16");
    if (ld < dev->s.V || ld > int64_t(1) << 40)
        return api_fail(ARCHEAD_EINVAL, "the row stride must lie in [V, 2^40]");
    if (M == 0)
        return ARCHEAD_OK;
    if (!dlogits || !dX)
        return api_fail(ARCHEAD_EINVAL, "dlogits and dX are required");
    if ((uintptr_t)dlogits % (type == ARCHEAD_F32 ? 4 : 2) || (uintptr_t)dX % 2)
        return api_fail(ARCHEAD_EINVAL, "dlogits and dX must be aligned to their elements");
    if (!*slot)
        return api_fail(ARCHEAD_EINVAL, "call archead_reserve_backward first");
    BW_TRY(hipSetDevice(device));
    const BackwardState &b = **slot;
    const size_t esz = type == ARCHEAD_F32 ? 4 : 2;
    for (int64_t m = 0; m < M; m += b.rows)
        backward_rows(*dev, b, std::min(b.rows, M - m), (const char *)dlogits + size_t(m) * ld * esz, type, ld,
                      (uint16_t *)dX + m * dev->s.d, (hipStream_t)hip_stream);
    BW_TRY(hipGetLastError());
    return ARCHEAD_OK;
}
