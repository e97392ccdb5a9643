// fp8.hip -- matrices held in 8-bit floating point (e4m3) with a scale for
// each block of 128, and the product of two of them: an 8-bit output head.
//
// Quantiser: a block (128 columns of one row, or 128 x 128) gets
//   s = amax / 448 in fp32 (448 is e4m3's largest value), at least 2^-126;
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

namespace archead {
namespace {

typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x8u __attribute__((ext_vector_type(8), aligned(2)));

constexpr int kBlk = 128; // columns (and weight rows) that share a scale
constexpr float kE4m3Max = 448.f;

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

__device__ __forceinline__ float block_scale(float amax)
{
    return amax > 0.f ? fmaxf(amax / kE4m3Max, 1.17549435e-38f) : 0.f;
}

// x / s with the last bit set where the quotient is not exact, so that the
// rounding to e4m3 that follows never sees a tie that is not one: the
// division's remainder x - q s is exact in one fma and says on which side of
// q the quotient lies.
__device__ __forceinline__ float sticky_quotient(float x, float s)
{
    float q, rem;
    if (s < 7.9e-31f) { // 2^-100: the remainder could fall below fp32's range
        const double d = (double)x / (double)s;
        q = (float)d;
        rem = (float)(d - (double)q);
    } else {
        q = x / s;
        rem = __builtin_fmaf(-q, s, x);
    }
    uint32_t b = __float_as_uint(q);
    if (rem != 0.f && (b & 1u) == 0u && fabsf(q) < 3.0e38f) {
        const bool outward = (rem > 0.f) == (q > 0.f);
        b = outward ? b + 1 : b - 1;
    }
    return q == 0.f ? q : __uint_as_float(b);
}

// eight codes in order
__device__ __forceinline__ u32x2 codes8(const float v[8], float s)
{
    float q[8];
    uint32_t nan = 0;
    for (int i = 0; i < 8; ++i) {
        const float t = s > 0.f ? sticky_quotient(v[i], s) : 0.f;
        const bool is_nan = v[i] != v[i] || t != t;
        nan |= (uint32_t)is_nan << i;
        q[i] = is_nan ? 0.f : fminf(fmaxf(t, -kE4m3Max), kE4m3Max);
    }
    u32x2 o;
    for (int h = 0; h < 2; ++h) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
        o[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], w, true);
        for (int i = 0; i < 4; ++i)
            if (nan >> (4 * h + i) & 1)
                o[h] |= 0x7Fu << (8 * i);
    }
    return o;
}

// one row's blocks: 16 lanes a block, 8 columns a lane
template <typename T>
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
        *(u32x2 *)(q + row * ldq + c) = codes8(v, sc);
    if ((threadIdx.x & 15) == 0)
        s[b * lds + row] = sc;
}

// 128 x 128 blocks, one per workgroup: two threads a row, 64 columns each
template <typename T>
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
            *(u32x2 *)(q + row * ldq + c0 + 8 * j) = codes8(v, sc);
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
// fp32: the fp8 forms align each group of eight products to its largest and
// drop what lies 2^14 below (measured: 2e-5 of the terms' magnitudes, which
// shows in an fp32 result).
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

// One wave per 16 x 16 tile of the output.  The weights are the A operand, so
// that a lane's four results are consecutive columns of one output row.  Lane
// l takes bytes 16 (l / 16) .. +15 of both halves of a block's 128 columns:
// any order of the columns serves as long as both operands share it.
template <typename O> __global__ __launch_bounds__(64) void product_simple_kernel(ProdArgs a)
{
    const int lane = threadIdx.x, q = lane >> 4;
    const int64_t nt = (a.N + 15) / 16;
    const int64_t n0 = (blockIdx.x % nt) * 16, m0 = (blockIdx.x / nt) * 16;
    const uint8_t *w = a.B + min(n0 + (lane & 15), a.N - 1) * a.ldb;
    const int64_t m = m0 + (lane & 15), mc = min(m, a.M - 1);
    const uint8_t *x = a.A + mc * a.lda;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    const int64_t nb = (a.K + kBlk - 1) / kBlk;
    for (int64_t b = 0; b < nb; ++b) {
        const int64_t c = b * kBlk + 16 * q;
        const f32x4 p = block_product(join(piece(w, c, a.K), piece(w, c + 64, a.K)),
                                      join(piece(x, c, a.K), piece(x, c + 64, a.K)), f32x4{0.f, 0.f, 0.f, 0.f});
        const float sc = a.sA[b * a.ldsa + mc] * a.sB[n0 / kBlk * a.ldsb + b];
        for (int i = 0; i < 4; ++i)
            acc[i] = __builtin_fmaf(p[i], sc, acc[i]);
    }
    if (m < a.M)
        put4((O *)a.out + m * a.ldo + n0 + 4 * q, acc, a.N - n0 - 4 * q);
}

archead_status launched(const char *what)
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return api_fail(ARCHEAD_EHIP, std::string(what) + ": " + hipGetErrorString(e));
    return ARCHEAD_OK;
}

bool bad_rows(const void *p, int64_t ld, int64_t cols) { return (uintptr_t)p % 16 || ld % 16 || ld < cols; }

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
        rows * ((cols + kBlk - 1) / kBlk) > (int64_t(1) << 34))
        return api_fail(ARCHEAD_ESHAPE, "rows < 2^31, cols a multiple of 16 in [16, 2^20], at most 2^34 row blocks");
    if (type != ARCHEAD_F32 && type != ARCHEAD_BF16)
        return api_fail(ARCHEAD_EINVAL, "x must be ARCHEAD_F32 or ARCHEAD_BF16");
    if (block_rows != 1 && block_rows != kBlk)
        return api_fail(ARCHEAD_EINVAL, "block_rows must be 1 or 128");
    const int64_t nb = (cols + kBlk - 1) / kBlk;
    if (ldx < cols || lds < (block_rows == 1 ? rows : nb))
        return api_fail(ARCHEAD_EINVAL, "a row stride is shorter than a row");
    if (rows == 0)
        return ARCHEAD_OK;
    if (!x || !q || !s)
        return api_fail(ARCHEAD_EINVAL, "x, q and s are required");
    if ((uintptr_t)x % (type == ARCHEAD_F32 ? 4 : 2) || bad_rows(q, ldq, cols))
        return api_fail(ARCHEAD_EINVAL, "x aligned to its element; q and its row stride to 16 bytes");
    hipStream_t st = (hipStream_t)hip_stream;
    if (block_rows == 1) {
        const dim3 grid((unsigned)((rows * nb + 15) / 16));
        if (type == ARCHEAD_F32)
            hipLaunchKernelGGL(quant_rows_kernel<float>, grid, dim3(256), 0, st, (const float *)x, ldx, rows, cols, q,
                               ldq, s, lds);
        else
            hipLaunchKernelGGL(quant_rows_kernel<uint16_t>, grid, dim3(256), 0, st, (const uint16_t *)x, ldx, rows,
                               cols, q, ldq, s, lds);
    } else {
        const dim3 grid((unsigned)((rows + kBlk - 1) / kBlk * nb));
        if (type == ARCHEAD_F32)
            hipLaunchKernelGGL(quant_tiles_kernel<float>, grid, dim3(256), 0, st, (const float *)x, ldx, rows, cols, q,
                               ldq, s, lds);
        else
            hipLaunchKernelGGL(quant_tiles_kernel<uint16_t>, grid, dim3(256), 0, st, (const uint16_t *)x, ldx, rows,
                               cols, q, ldq, s, lds);
    }
    return launched("archead_fp8_quantize");
}

extern "C" archead_status archead_fp8_matmul(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda,
                                             const float *sA, int64_t ldsa, const uint8_t *B, int64_t ldb,
                                             const float *sB, int64_t ldsb, void *out, int out_type, int64_t ldo,
                                             void *hip_stream)
{
    if (M < 0 || N < 0)
        return api_fail(ARCHEAD_EINVAL, "M < 0 or N < 0");
    if (M > (int64_t(1) << 20) || N >= (int64_t(1) << 31) || K < 16 || K % 16 || K > (int64_t(1) << 20))
        return api_fail(ARCHEAD_ESHAPE, "M <= 2^20, N < 2^31 and K a multiple of 16 in [16, 2^20]");
    if (out_type != ARCHEAD_F32 && out_type != ARCHEAD_BF16)
        return api_fail(ARCHEAD_EINVAL, "out must be ARCHEAD_F32 or ARCHEAD_BF16");
    const int64_t nb = (K + kBlk - 1) / kBlk;
    if (ldsa < M || ldsb < nb || ldo < N)
        return api_fail(ARCHEAD_EINVAL, "a row stride is shorter than a row");
    if (M == 0 || N == 0)
        return ARCHEAD_OK;
    if (!A || !sA || !B || !sB || !out)
        return api_fail(ARCHEAD_EINVAL, "A, sA, B, sB and out are required");
    if (bad_rows(A, lda, K) || bad_rows(B, ldb, K))
        return api_fail(ARCHEAD_EINVAL, "A, B and their row strides must be multiples of 16 bytes, strides at least K");
    if ((uintptr_t)out % (out_type == ARCHEAD_F32 ? 4 : 2))
        return api_fail(ARCHEAD_EINVAL, "out must be aligned to its element");
    hipStream_t st = (hipStream_t)hip_stream;
    const ProdArgs a{M, N, K, lda, ldb, ldo, ldsa, ldsb, A, B, sA, sB, out};
    const int64_t tiles = (M + 15) / 16 * ((N + 15) / 16);
    if (tiles >= (int64_t(1) << 31))
        return api_fail(ARCHEAD_ESHAPE, "product too large");
    if (out_type == ARCHEAD_F32)
        hipLaunchKernelGGL(product_simple_kernel<float>, dim3((unsigned)tiles), dim3(64), 0, st, a);
    else
        hipLaunchKernelGGL(product_simple_kernel<uint16_t>, dim3((unsigned)tiles), dim3(64), 0, st, a);
    return launched("archead_fp8_matmul");
}
