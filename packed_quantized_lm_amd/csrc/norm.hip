// norm.hip -- the root-mean-square norm with the residual's addition, written in
// fp32 or bf16 and as the 8-bit head's codes and scales, and its backward.
//
// Row m, d wide:
//   h = x + residual, rounded to the residual's type (h = x without one)
//   r = 1 / sqrt(mean_j h_j^2 + eps),  n_j = h_j r (w_j + offset)
//   y = n rounded once; codes of n in blocks of 128 columns as the row quantiser's.
// Backward, for u = dy:
//   g_j = u_j (w_j + offset),  c = mean_j g_j h_j,
//   dh_j = r (g_j - h_j r^2 c) + dres_j,   dw_j = sum_m u_mj h_mj r_m.
// Both are bound by their rows' bytes: a row is read once and stays in registers
// between its sums and its results (8192 x 4096 bf16 with the residual: codes out 50
// us, 4.7 TB/s, backward 51 + 5 of dw's last sum, 5.0 TB/s; a large copy runs at
// 4.9).  One row is a launch and the loads' and the sum's latency: 3.7 us.
// A row's sums are fp64 (its squares pass fp32's range from 2^64 on), dw's parts fp32
// over at most 64 rows a team, then fp64.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "api_internal.hpp"
#include "archead.h"
#include "e4m3.hpp"
#include "elements.hpp"
#include "entry.hpp"
#include "overlap.hpp"

namespace archead {
namespace {

constexpr int kBlk = 128;                       // columns that share a scale
constexpr int64_t kMaxRows = int64_t(1) << 22;  // a launch holds fewer than 2^32 threads
constexpr int64_t kMaxWidth = int64_t(1) << 20;
constexpr int64_t kMaxStride = int64_t(1) << 40;

// sum over T threads that share a row (T a power of two; above 64 whole
// workgroups of T), in every one of them, in a fixed order
template <int T> __device__ __forceinline__ double team_sum(double v, double *red)
{
    for (int off = (T < 64 ? T : 64) / 2; off >= 1; off >>= 1)
        v += __shfl_xor(v, off);
    if (T > 64) {
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
        for (int w = 1; w < T / 64; ++w)
            v += red[w];
    }
    return v;
}

// 1 / sqrt(v): the instruction's estimate and one step of Newton's.  Rows at the ends of
// fp32's range have one, from 2^-128 to 2^149, that fp32 does not hold.
__device__ __forceinline__ double inverse_root(double v)
{
    const double r = __builtin_amdgcn_rsq(v);
    const double better = r * __builtin_fma(-0.5 * v * r, r, 1.5);
    return v > 0. && v < INFINITY ? better : r; // 0 and infinity have theirs; NaN stays NaN
}

// the same of two sums at once, one wait: red holds two sets, taken in turn, so
// that a wave may be a row ahead of one that still reads
template <int T>
__device__ __forceinline__ void team_sums(double &v, double &w, double (*red)[T > 64 ? T / 64 : 1])
{
    for (int off = (T < 64 ? T : 64) / 2; off >= 1; off >>= 1) {
        v += __shfl_xor(v, off);
        w += __shfl_xor(w, off);
    }
    if (T > 64) {
        if ((threadIdx.x & 63) == 0) {
            red[0][threadIdx.x >> 6] = v;
            red[1][threadIdx.x >> 6] = w;
        }
        __syncthreads();
        v = red[0][0];
        w = red[1][0];
        for (int k = 1; k < T / 64; ++k) {
            v += red[0][k];
            w += red[1][k];
        }
    }
}

struct NormArgs {
    int64_t M;
    int d;
    int64_t ldx, ldr, ldh, ldy, ldq, lds;
    const void *x, *residual, *weight;
    void *h, *y;
    uint8_t *q;
    float *s;
    double inv_d;
    float eps, offset;
    int weight_type, y_type;
};

// (weight + offset) times, a power of two
__device__ __forceinline__ void weights_of(const NormArgs &a, int q, float times, float w[8])
{
    if (a.weight_type == ARCHEAD_F32)
        vector_values(q, a.d, load_vector((const float *)a.weight, q, a.d), w);
    else
        vector_values(q, a.d, load_vector((const uint16_t *)a.weight, q, a.d), w);
    for (int i = 0; i < 8; ++i)
        w[i] = __builtin_fmaf(w[i], times, a.offset * times);
}

// r as by * times: times, a power of two, goes to the weights, where it costs nothing, and
// by stays far enough inside fp32's range for its full precision
struct Root {
    float by, times;
};
__device__ __forceinline__ Root split(double r)
{
    Root s{(float)r, 1.f};
    if (__builtin_expect(s.by > 0x1p125f || s.by < 0x1p-125f, 0)) {
        s.times = s.by > 1.f ? 0x1p24f : 0x1p-4f;
        s.by = (float)(r / (double)s.times);
    }
    return s;
}

// results of one vector n; sixteen neighbouring threads hold a block of columns
__device__ __forceinline__ void put(const NormArgs &a, int64_t m, int q, bool in, const float n[8])
{
    if (a.y && in) {
        if (a.y_type == ARCHEAD_F32)
            store_vector((float *)a.y + m * a.ldy, q, a.d, n);
        else
            store_vector((uint16_t *)a.y + m * a.ldy, q, a.d, n);
    }
    if (a.q) {
        float top = 0.f;
        for (int i = 0; i < 8; ++i)
            top = fmaxf(top, fabsf(n[i]));
        for (int off = 8; off >= 1; off >>= 1)
            top = fmaxf(top, __shfl_xor(top, off));
        const float sc = block_scale(top);
        if (in) {
            *(u32x2 *)(a.q + m * a.ldq + 8 * q) = codes8(n, sc);
            if ((q & 15) == 0)
                a.s[(q >> 4) * a.lds + m] = sc;
        }
    }
}

// T threads a row, H vectors of eight a thread; XT, RT as they lie in memory
// (RT = void: no residual)
template <int T, int H, typename XT, typename RT>
__global__ __launch_bounds__(T > 256 ? T : 256) void norm_kernel(NormArgs a)
{
    constexpr bool kRes = !std::is_same_v<RT, void>;
    using RM = std::conditional_t<kRes, RT, XT>;
    constexpr int kTeams = (T > 256 ? T : 256) / T;
    __shared__ double red[T > 64 ? T / 64 : 1];
    const int t = threadIdx.x % T;
    const int64_t m = (int64_t)blockIdx.x * kTeams + threadIdx.x / T;
    if (m >= a.M) // whole teams; a team of a workgroup's size always has its row
        return;
    const XT *x = (const XT *)a.x + m * a.ldx;
    const RM *res = (const RM *)a.residual + m * a.ldr;
    const int nv = (a.d + 7) / 8;
    float v[H][8];
    {
        Eight<XT> xr[H];
        Eight<RM> rr[H];
#pragma unroll
        for (int j = 0; j < H; ++j) {
            xr[j] = load_vector(x, t + j * T, a.d);
            if constexpr (kRes)
                rr[j] = load_vector(res, t + j * T, a.d);
        }
#pragma unroll
        for (int j = 0; j < H; ++j) {
            const int q = t + j * T;
            vector_values(q, a.d, xr[j], v[j]);
            if constexpr (kRes) {
                float o[8];
                vector_values(q, a.d, rr[j], o);
                for (int i = 0; i < 8; ++i)
                    o[i] += v[j][i];
                Eight<RM> sum;
                narrow(o, sum);
                widen(sum, v[j]); // the norm is the stored sum's
                if (q < nv)
                    store_vector((RM *)a.h + m * a.ldh, q, a.d, v[j]);
            }
        }
    }
    double ss = 0.;
#pragma unroll
    for (int j = 0; j < H; ++j)
        if (t + j * T < nv)
            for (int i = 0; i < 8; ++i)
                ss = __builtin_fma((double)v[j][i], (double)v[j][i], ss);
    ss = team_sum<T>(ss, red);
    const Root r = split(inverse_root(__builtin_fma(ss, a.inv_d, (double)a.eps)));
#pragma unroll
    for (int j = 0; j < H; ++j) {
        const int q = t + j * T;
        if (j * T < nv) { // not uniform in a team only past the row's end
            float w[8], n[8];
            weights_of(a, q, r.times, w);
            for (int i = 0; i < 8; ++i)
                n[i] = q < nv ? v[j][i] * r.by * w[i] : 0.f;
            put(a, m, q, q < nv, n);
        }
    }
}

// rows that registers do not hold: the sum is written (or x is read) a second time
constexpr int kLongT = 1024;
template <typename XT, typename RT> __global__ __launch_bounds__(kLongT) void norm_long_kernel(NormArgs a)
{
    constexpr bool kRes = !std::is_same_v<RT, void>;
    using RM = std::conditional_t<kRes, RT, XT>;
    __shared__ double red[kLongT / 64];
    const int64_t m = blockIdx.x;
    const int nv = (a.d + 7) / 8;
    const XT *x = (const XT *)a.x + m * a.ldx;
    const RM *res = (const RM *)a.residual + m * a.ldr;
    const RM *sum = kRes ? (const RM *)a.h + m * a.ldh : (const RM *)x;
    double ss = 0.;
    for (int q = threadIdx.x; q < nv; q += kLongT) {
        float v[8];
        vector_values(q, a.d, load_vector(x, q, a.d), v);
        if constexpr (kRes) {
            float o[8];
            vector_values(q, a.d, load_vector(res, q, a.d), o);
            for (int i = 0; i < 8; ++i)
                o[i] += v[i];
            Eight<RM> kept;
            narrow(o, kept);
            widen(kept, v);
            store_vector((RM *)a.h + m * a.ldh, q, a.d, v);
        }
        for (int i = 0; i < 8; ++i)
            ss = __builtin_fma((double)v[i], (double)v[i], ss);
    }
    ss = team_sum<kLongT>(ss, red);
    const Root r = split(inverse_root(__builtin_fma(ss, a.inv_d, (double)a.eps)));
    for (int q0 = 0; q0 < nv; q0 += kLongT) { // each thread reads back what it wrote
        const int q = q0 + threadIdx.x;
        float v[8] = {}, w[8] = {};
        if (q < nv) {
            vector_values(q, a.d, load_vector(sum, q, a.d), v);
            weights_of(a, q, r.times, w);
        }
        for (int i = 0; i < 8; ++i)
            v[i] = q < nv ? v[i] * r.by * w[i] : 0.f;
        put(a, m, q, q < nv, v);
    }
}

template <int T, int H, typename XT, typename RT> void launch_norm(const NormArgs &a, hipStream_t st)
{
    constexpr int kWg = T > 256 ? T : 256;
    hipLaunchKernelGGL((norm_kernel<T, H, XT, RT>), dim3((unsigned)((a.M + kWg / T - 1) / (kWg / T))), dim3(kWg), 0, st,
                       a);
}

// Threads a row: enough for its vectors to stay in registers, and few where that
// leaves lanes idle or waves waiting for each other (bf16 with a residual, in us: 128
// wide, 65535 rows, 16 threads 13, 64 31; 512 wide, 65535, 64 threads 49, 256 109;
// 2048 wide, 16384, 256 threads 48.6, 64 50.6; 8192 wide, 4096, 256 threads 51, 1024
// 60; 2571 wide, 8192, 256 threads 45.6, 512 52).  With a row to a compute unit or
// fewer the loads' latency is what counts, and one vector a thread is fastest (one row of
// 4096 3.7 against 4.2, 256 rows 4.4, 4.9; one of 8192 4.2, 5.5, 256 rows 6.0, 7.4; 1024
// rows of 8192 16.6, 14.1).
constexpr int64_t kFewRows = 256;
template <typename XT, typename RT> void run_norm(const NormArgs &a, hipStream_t st)
{
    if (a.d <= 128)
        launch_norm<16, 1, XT, RT>(a, st);
    else if (a.d <= 512)
        launch_norm<64, 1, XT, RT>(a, st);
    else if (a.d <= 2048)
        launch_norm<256, 1, XT, RT>(a, st);
    else if (a.d <= 4096 && a.M <= kFewRows)
        launch_norm<512, 1, XT, RT>(a, st);
    else if (a.d <= 4096)
        launch_norm<256, 2, XT, RT>(a, st);
    else if (a.d <= 8192 && a.M <= kFewRows)
        launch_norm<1024, 1, XT, RT>(a, st);
    else if (a.d <= 8192)
        launch_norm<256, 4, XT, RT>(a, st);
    else if (a.d <= 16384)
        launch_norm<1024, 2, XT, RT>(a, st);
    else
        hipLaunchKernelGGL((norm_long_kernel<XT, RT>), dim3((unsigned)a.M), dim3(kLongT), 0, st, a);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
struct BackArgs {
    int64_t M;
    int d;
    int64_t ldu, ldh, ldr, ldd;
    const void *u, *h, *weight, *dres; // dres may be null
    void *dh;
    float *part; // [groups][d]
    float4 *inv; // [M], the long rows' us, hs and rw
    double inv_d;
    float eps, offset;
    int weight_type;
    int64_t groups, slice; // long rows: rows a part sums
};

__device__ __forceinline__ void weights_of(const BackArgs &a, int q, float w[8])
{
    NormArgs n{};
    n.weight = a.weight;
    n.weight_type = a.weight_type;
    n.d = a.d;
    n.offset = a.offset;
    weights_of(n, q, 1.f, w);
}

// Rows near the ends of fp32's range have an r, or an r^2 c beside it, that fp32 does not
// hold.  Their u and h are multiplied by powers of two, us and hs, first, and
//   dh = r / us (g us - (h hs) (r^2 c us / hs)),   dw's term = (u us) (h hs) (r / us / hs).
// All others' are taken as they are.
struct FarRow {
    float us, hs, r, rw, k;
};
template <int T> __device__ __forceinline__ bool is_far(float r) // the same for a wave that shares a row
{
    const bool far = r < 0x1p-60f || r > 0x1p60f;
    return T < 64 ? far : __ballot(far) != 0;
}
__device__ __forceinline__ FarRow far_row(double r, double c)
{
    const double us = r > 1. ? 0x1p24 : 0x1p-4, hs = r > 1. ? 0x1p64 : 0x1p-64;
    return {(float)us, (float)hs, (float)(r / us), (float)(r / us / hs), (float)(r * r * c * (us / hs))};
}

// A workgroup's teams of T threads take every (groups x teams)-th row; the weights
// and dw's sums stay in registers (8192 x 4096: 55 us, weights from cache twice a row 79).
// kAhead: the next row is on its way while one is summed, where registers allow that (two
// vectors a thread: 8192 x 4096 55 us against 57; four: 8192 x 2048 104 against 59).  The
// teams' sums meet in LDS.
template <int T, int H, bool kAhead, typename UT, typename HT>
__global__ __launch_bounds__(T > 256 ? T : 256) void norm_back_kernel(BackArgs a)
{
    constexpr int kWg = T > 256 ? T : 256, kTeams = kWg / T;
    __shared__ double red[2][2][T > 64 ? T / 64 : 1];
    __shared__ float meet[kTeams > 1 ? kTeams * T * H * 8 : 1];
    const int t = threadIdx.x % T, team = threadIdx.x / T;
    const int nv = (a.d + 7) / 8;
    const int64_t step = a.groups * kTeams;
    constexpr bool kShared = T >= 512 && H == 4; // a thread's weights in LDS: 256 registers do not hold them too
    __shared__ f32x4 own[kShared ? H * 2 * T : 1];
    float held[kShared ? 1 : H][8], dw[H][8] = {};
#pragma unroll
    for (int j = 0; j < H; ++j) {
        float *w = held[kShared ? 0 : j];
        weights_of(a, t + j * T, w);
        if constexpr (kShared) { // read by this thread alone
            own[2 * j * T + t] = f32x4{w[0], w[1], w[2], w[3]};
            own[(2 * j + 1) * T + t] = f32x4{w[4], w[5], w[6], w[7]};
        }
    }
    auto weight = [&](int j, float w[8]) __attribute__((always_inline)) {
        if constexpr (kShared) {
            const f32x4 lo = own[2 * j * T + t], hi = own[(2 * j + 1) * T + t];
            for (int i = 0; i < 4; ++i) {
                w[i] = lo[i];
                w[4 + i] = hi[i];
            }
        } else
            for (int i = 0; i < 8; ++i)
                w[i] = held[j][i];
    };
    Eight<UT> ur[H];
    Eight<HT> hr[H], rr[H];
    auto fetch = [&](int64_t m) __attribute__((always_inline)) {
        const UT *u = (const UT *)a.u + m * a.ldu;
        const HT *h = (const HT *)a.h + m * a.ldh;
#pragma unroll
        for (int j = 0; j < H; ++j) {
            ur[j] = load_vector(u, t + j * T, a.d);
            hr[j] = load_vector(h, t + j * T, a.d);
        }
    };
    auto fetch_res = [&](int64_t m) __attribute__((always_inline)) {
        if (a.dres)
#pragma unroll
            for (int j = 0; j < H; ++j)
                rr[j] = load_vector((const HT *)a.dres + m * a.ldr, t + j * T, a.d);
    };
    int turn = 0;
    int64_t m = (int64_t)blockIdx.x * kTeams + team;
    if (kAhead && m < a.M)
        fetch(m);
    for (; m < a.M; m += step, turn ^= 1) {
        if (!kAhead)
            fetch(m);
        fetch_res(m);
        float uv[H][8], hv[H][8], g[H][8];
        double ss = 0., c = 0.;
#pragma unroll
        for (int j = 0; j < H; ++j) {
            vector_values(t + j * T, a.d, ur[j], uv[j]);
            vector_values(t + j * T, a.d, hr[j], hv[j]);
        }
        if (kAhead && m + step < a.M)
            fetch(m + step); // the next row is on its way while this one is summed
#pragma unroll
        for (int j = 0; j < H; ++j) {
            weight(j, g[j]);
            for (int i = 0; i < 8; ++i) {
                const double hd = hv[j][i];
                g[j][i] *= uv[j][i];
                ss = __builtin_fma(hd, hd, ss);
                c = __builtin_fma((double)g[j][i], hd, c);
            }
        }
        team_sums<T>(ss, c, red[turn]);
        const double root = inverse_root(__builtin_fma(ss, a.inv_d, (double)a.eps));
        float r = (float)root, rw = r, k = (float)((double)r * (double)r * (c * a.inv_d));
        if (__builtin_expect(is_far<T>(r), 0)) {
            const FarRow f = far_row(root, c * a.inv_d);
            r = f.r, rw = f.rw, k = f.k;
#pragma unroll
            for (int j = 0; j < H; ++j)
                for (int i = 0; i < 8; ++i) {
                    uv[j][i] *= f.us;
                    g[j][i] *= f.us;
                    hv[j][i] *= f.hs;
                }
        }
#pragma unroll
        for (int j = 0; j < H; ++j) {
            const int q = t + j * T;
            float o[8] = {};
            if (a.dres)
                vector_values(q, a.d, rr[j], o);
            for (int i = 0; i < 8; ++i) {
                o[i] = __builtin_fmaf(r, __builtin_fmaf(-hv[j][i], k, g[j][i]), o[i]);
                dw[j][i] = __builtin_fmaf(uv[j][i], hv[j][i] * rw, dw[j][i]);
            }
            if (q < nv)
                store_vector((HT *)a.dh + m * a.ldd, q, a.d, o);
        }
    }
    float *part = a.part + (int64_t)blockIdx.x * a.d;
    if constexpr (kTeams > 1) {
#pragma unroll
        for (int j = 0; j < H; ++j)
            for (int i = 0; i < 8; ++i)
                meet[(team * T * H + j * T + t) * 8 + i] = dw[j][i];
        __syncthreads();
        for (int e = threadIdx.x; e < a.d; e += kWg) {
            float s = 0.f;
            for (int k = 0; k < kTeams; ++k)
                s += meet[k * T * H * 8 + e];
            part[e] = s;
        }
    } else {
#pragma unroll
        for (int j = 0; j < H; ++j)
            if (t + j * T < nv)
                store_vector(part, t + j * T, a.d, dw[j]);
    }
}

// rows that registers do not hold: sums, then the results in a second reading;
// dw from r and a third
template <typename UT, typename HT> __global__ __launch_bounds__(kLongT) void norm_back_long_kernel(BackArgs a)
{
    __shared__ double red[2][kLongT / 64];
    const int64_t m = blockIdx.x;
    const int nv = (a.d + 7) / 8;
    const UT *u = (const UT *)a.u + m * a.ldu;
    const HT *h = (const HT *)a.h + m * a.ldh;
    const HT *res = (const HT *)a.dres + m * a.ldr;
    double ss = 0., c = 0.;
    for (int q = threadIdx.x; q < nv; q += kLongT) {
        float uv[8], hv[8], w[8];
        vector_values(q, a.d, load_vector(u, q, a.d), uv);
        vector_values(q, a.d, load_vector(h, q, a.d), hv);
        weights_of(a, q, w);
        for (int i = 0; i < 8; ++i) {
            ss = __builtin_fma((double)hv[i], (double)hv[i], ss);
            c = __builtin_fma((double)(uv[i] * w[i]), (double)hv[i], c);
        }
    }
    team_sums<kLongT>(ss, c, red);
    const double root = inverse_root(__builtin_fma(ss, a.inv_d, (double)a.eps));
    const float r0 = (float)root;
    FarRow f{1.f, 1.f, r0, r0, (float)((double)r0 * (double)r0 * (c * a.inv_d))};
    if (is_far<kLongT>(r0))
        f = far_row(root, c * a.inv_d);
    if (threadIdx.x == 0)
        a.inv[m] = make_float4(f.us, f.hs, f.rw, 0.f);
    for (int q = threadIdx.x; q < nv; q += kLongT) {
        float uv[8], hv[8], w[8], o[8] = {};
        vector_values(q, a.d, load_vector(u, q, a.d), uv);
        vector_values(q, a.d, load_vector(h, q, a.d), hv);
        weights_of(a, q, w);
        if (a.dres)
            vector_values(q, a.d, load_vector(res, q, a.d), o);
        for (int i = 0; i < 8; ++i)
            o[i] = __builtin_fmaf(f.r, __builtin_fmaf(-(hv[i] * f.hs), f.k, uv[i] * f.us * w[i]), o[i]);
        store_vector((HT *)a.dh + m * a.ldd, q, a.d, o);
    }
}
template <typename UT, typename HT> __global__ __launch_bounds__(256) void weight_long_kernel(BackArgs a)
{
    const int q = (int)blockIdx.y * 256 + (int)threadIdx.x, nv = (a.d + 7) / 8;
    const int64_t g = blockIdx.x;
    if (q >= nv)
        return;
    float dw[8] = {};
    for (int64_t m = g * a.slice; m < min((g + 1) * a.slice, a.M); ++m) {
        float uv[8], hv[8];
        const UT *u = (const UT *)a.u + m * a.ldu;
        const HT *h = (const HT *)a.h + m * a.ldh;
        vector_values(q, a.d, load_vector(u, q, a.d), uv);
        vector_values(q, a.d, load_vector(h, q, a.d), hv);
        const float4 r = a.inv[m];
        for (int i = 0; i < 8; ++i)
            dw[i] = __builtin_fmaf(uv[i] * r.x, hv[i] * r.y * r.z, dw[i]);
    }
    store_vector(a.part + g * a.d, q, a.d, dw);
}

// dw = the sum of the workgroups' parts: 32 columns a workgroup, 32 threads a column
__global__ __launch_bounds__(1024) void weight_sum_kernel(const float *part, int64_t groups, int64_t d, float *dw)
{
    constexpr int kFly = 16;
    __shared__ double meet[32][33];
    const int col = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + col;
    double s = 0.;
    if (c < d)
        for (int64_t g0 = row; g0 < groups; g0 += 32 * kFly) { // loads in flight together, past the end not added
            float v[kFly];
#pragma unroll
            for (int k = 0; k < kFly; ++k)
                v[k] = part[min(g0 + 32 * k, groups - 1) * d + c];
#pragma unroll
            for (int k = 0; k < kFly; ++k)
                s += g0 + 32 * k < groups ? (double)v[k] : 0.;
        }
    meet[row][col] = s;
    __syncthreads();
    if (row == 0 && c < d) {
        for (int k = 1; k < 32; ++k)
            s += meet[k][col];
        dw[c] = (float)s;
    }
}

// how a backward is cut: threads a row (0: long rows), and parts of dw
struct BackPlan {
    int T, H;
    int64_t groups, slice;
    size_t inv, total; // byte offsets in the workspace
};
// workgroups that share the rows: more leave dw's last sum more parts, fewer leave
// compute units waiting (256, 512, 1024: 8192 x 4096 80, 55, 66 us; 777 x 2571 fp32 18,
// 16, 19; 16384 x 2048 -, 59, 64)
constexpr int64_t kGroups = 512;
constexpr int64_t kPartRows = 64; // rows whose terms of dw are added in fp32

// Threads a row and vectors a thread.  Narrow rows stay within a wave, whose sums wait
// for no other (bf16, 2^25 elements, in us: 512 wide, 16 threads of four vectors 58, 64 of
// one 75; 1024 wide, 64 of two 55, 256 of one 112; 2048 wide, 64 of four 59, 256 of one
// 65); wide ones take as many threads as hold them in two vectors each (8192 wide, 512 60,
// 256 of four 64), up to where 1024 have too few registers (16384 wide, 512 of four 82,
// 1024 of two 232).
BackPlan plan_back(int64_t M, int64_t d)
{
    BackPlan p{};
    if (d <= 128)
        p = {16, 1};
    else if (d <= 512)
        p = {16, 4};
    else if (d <= 1024)
        p = {64, 2};
    else if (d <= 2048)
        p = {64, 4};
    else if (d <= 4096)
        p = {256, 2};
    else if (d <= 8192)
        p = {512, 2};
    else if (d <= 16384)
        p = {512, 4};
    if (p.T) {
        const int64_t teams = std::max(256, p.T) / p.T;
        p.groups = std::max(std::min((M + teams - 1) / teams, kGroups), (M + teams * kPartRows - 1) / (teams * kPartRows));
    } else {
        p.slice = kPartRows;
        p.groups = (M + kPartRows - 1) / kPartRows;
    }
    p.inv = (size_t)((p.groups * d * 4 + 15) / 16 * 16);
    p.total = std::max<size_t>(16, p.inv + (p.T ? 0 : (size_t)M * sizeof(float4)));
    return p;
}

template <int T, int H, bool kAhead, typename UT, typename HT> void launch_back(const BackArgs &a, hipStream_t st)
{
    hipLaunchKernelGGL((norm_back_kernel<T, H, kAhead, UT, HT>), dim3((unsigned)a.groups), dim3(T > 256 ? T : 256), 0, st, a);
}

template <typename UT, typename HT> void run_back(const BackArgs &a, const BackPlan &p, float *dw, hipStream_t st)
{
    if (p.T == 16 && p.H == 1)
        launch_back<16, 1, true, UT, HT>(a, st);
    else if (p.T == 16)
        launch_back<16, 4, false, UT, HT>(a, st);
    else if (p.T == 64 && p.H == 2)
        launch_back<64, 2, false, UT, HT>(a, st);
    else if (p.T == 64)
        launch_back<64, 4, false, UT, HT>(a, st);
    else if (p.T == 256)
        launch_back<256, 2, true, UT, HT>(a, st);
    else if (p.T == 512 && p.H == 2)
        launch_back<512, 2, true, UT, HT>(a, st);
    else if (p.T == 512)
        launch_back<512, 4, false, UT, HT>(a, st);
    else {
        hipLaunchKernelGGL((norm_back_long_kernel<UT, HT>), dim3((unsigned)a.M), dim3(kLongT), 0, st, a);
        hipLaunchKernelGGL((weight_long_kernel<UT, HT>),
                           dim3((unsigned)a.groups, (unsigned)(((a.d + 7) / 8 + 255) / 256)), dim3(256), 0, st, a);
    }
    if (dw)
        hipLaunchKernelGGL(weight_sum_kernel, dim3((unsigned)((a.d + 31) / 32)), dim3(1024), 0, st, a.part, a.groups,
                           a.d, dw);
}

archead_status check_sizes(int64_t M, int64_t d, float eps, float offset)
{
    if (M < 0)
        return api_fail(ARCHEAD_EINVAL, "M < 0");
    if (M >= kMaxRows || d < 1 || d > kMaxWidth)
        return api_fail(ARCHEAD_ESHAPE, "M < 2^22 and 1 <= d <= 2^20");
    if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(offset))
        return api_fail(ARCHEAD_EINVAL, "eps must be finite and not negative, offset finite");
    return ARCHEAD_OK;
}

} // namespace
} // namespace archead

using namespace archead;

extern "C" archead_status archead_rms_norm(int64_t M, int64_t d, const void *x, int x_type, int64_t ldx,
                                           const void *residual, int res_type, int64_t ldr, void *h, int64_t ldh,
                                           const void *weight, int weight_type, float eps, float offset, void *y,
                                           int y_type, int64_t ldy, uint8_t *q, int64_t ldq, float *s, int64_t lds,
                                           void *hip_stream)
{
    archead_status st = check_sizes(M, d, eps, offset);
    if (st != ARCHEAD_OK)
        return st;
    if (bad_type(x_type) || bad_type(weight_type) || (residual && bad_type(res_type)) || (y && bad_type(y_type)))
        return api_fail(ARCHEAD_EINVAL, "types are ARCHEAD_F32 or ARCHEAD_BF16");
    if (!y && !q)
        return api_fail(ARCHEAD_EINVAL, "y and q are both NULL");
    if (!residual != !h || !q != !s)
        return api_fail(ARCHEAD_EINVAL, "residual and h, q and s come together");
    if (q && d % 16 != 0)
        return api_fail(ARCHEAD_ESHAPE, "codes need d to be a multiple of 16");
    for (int64_t ld : {ldx, residual ? ldr : d, residual ? ldh : d, y ? ldy : d, q ? ldq : d})
        if (ld < d || ld > kMaxStride)
            return api_fail(ARCHEAD_EINVAL, "row strides must lie in [d, 2^40]");
    if (q && (lds < M || lds > kMaxStride))
        return api_fail(ARCHEAD_EINVAL, "the scales' stride must lie in [M, 2^40]");
    if (M == 0)
        return ARCHEAD_OK;
    if (!x || !weight)
        return api_fail(ARCHEAD_EINVAL, "x and weight are required");
    if (misaligned(x, size_of(x_type)) || misaligned(weight, size_of(weight_type)) || misaligned(y, size_of(y_type)) ||
        (residual && (misaligned(residual, size_of(res_type)) || misaligned(h, size_of(res_type)))) || misaligned(s, 4) ||
        (uintptr_t)q % 16 || (q && ldq % 16))
        return api_fail(ARCHEAD_EINVAL, "buffers aligned to their element; q and its row stride to 16 bytes");
    if (residual && ((h == residual && ldh != ldr) || (h == x && (res_type != x_type || ldh != ldx))))
        return api_fail(ARCHEAD_EINVAL, "in place, h needs the type and row stride of what it replaces");
    if (y && ((y == x && (y_type != x_type || ldy != ldx)) || y == h || y == residual))
        return api_fail(ARCHEAD_EINVAL, "y may be x, with its type and row stride, not h or residual");
    const Span sx = matrix_span(x, M, d, ldx, size_of(x_type)), sr = matrix_span(residual, M, d, ldr, size_of(res_type)),
               sh = matrix_span(h, M, d, ldh, size_of(res_type)), sy = matrix_span(y, M, d, ldy, size_of(y_type)),
               sq = matrix_span(q, M, d, ldq, 1), ss = matrix_span(s, (d + kBlk - 1) / kBlk, M, lds, 4);
    if (overlap_but_itself(sh, sx) || overlap_but_itself(sh, sr) || overlap_but_itself(sy, sx) || overlap(sy, sr) ||
        overlap({sq, ss}, {sx, sr}) || overlap({sh, sy, sq, ss}, {vector_span(weight, d * size_of(weight_type))}) ||
        overlap({sh, sy, sq, ss}))
        return api_fail(ARCHEAD_EINVAL, "a result overlaps what is read, or another result");
    const NormArgs a{M, (int)d, ldx, ldr, ldh, ldy, ldq, lds, x, residual, weight, h, y, q, s, 1. / (double)d, eps, offset,
                     weight_type, y_type};
    hipStream_t stream = (hipStream_t)hip_stream;
    const bool xf = x_type == ARCHEAD_F32, rf = res_type == ARCHEAD_F32;
    if (!residual)
        xf ? run_norm<float, void>(a, stream) : run_norm<uint16_t, void>(a, stream);
    else if (xf)
        rf ? run_norm<float, float>(a, stream) : run_norm<float, uint16_t>(a, stream);
    else
        rf ? run_norm<uint16_t, float>(a, stream) : run_norm<uint16_t, uint16_t>(a, stream);
    return launched("archead_rms_norm");
}

extern "C" archead_status archead_rms_norm_workspace(int64_t M, int64_t d, uint64_t *bytes)
{
    if (!bytes)
        return api_fail(ARCHEAD_EINVAL, "bytes is NULL");
    archead_status st = check_sizes(M, d, 0.f, 0.f);
    if (st == ARCHEAD_OK)
        *bytes = plan_back(M, d).total;
    return st;
}

extern "C" archead_status archead_rms_norm_backward(int64_t M, int64_t d, const void *dy, int dy_type, int64_t ldy,
                                                    const void *h, int h_type, int64_t ldh, const void *weight,
                                                    int weight_type, float eps, float offset, const void *dres,
                                                    int64_t ldr, void *dh, int64_t ldd, float *dweight, void *ws,
                                                    uint64_t ws_bytes, void *hip_stream)
{
    archead_status st = check_sizes(M, d, eps, offset);
    if (st != ARCHEAD_OK)
        return st;
    if (bad_type(dy_type) || bad_type(h_type) || bad_type(weight_type))
        return api_fail(ARCHEAD_EINVAL, "types are ARCHEAD_F32 or ARCHEAD_BF16");
    for (int64_t ld : {ldy, ldh, ldd, dres ? ldr : d})
        if (ld < d || ld > kMaxStride)
            return api_fail(ARCHEAD_EINVAL, "row strides must lie in [d, 2^40]");
    if (M > 0 && (!dy || !h || !weight || !dh))
        return api_fail(ARCHEAD_EINVAL, "dy, h, weight and dh are required");
    if (dh && (dh == dy || dh == h))
        return api_fail(ARCHEAD_EINVAL, "dh may be dres, not dy or h");
    if (dres && dres == dh && ldr != ldd)
        return api_fail(ARCHEAD_EINVAL, "in place of dres, dh needs its row stride");
    if (misaligned(dy, size_of(dy_type)) || misaligned(h, size_of(h_type)) || misaligned(weight, size_of(weight_type)) ||
        misaligned(dres, size_of(h_type)) || misaligned(dh, size_of(h_type)) || misaligned(dweight, 4))
        return api_fail(ARCHEAD_EINVAL, "buffers must be aligned to their element");
    if (!ws || (uintptr_t)ws % 16)
        return api_fail(ARCHEAD_EINVAL, "a 16-byte aligned workspace is required");
    const BackPlan p = plan_back(M, d);
    if (ws_bytes < p.total)
        return api_fail(ARCHEAD_EINVAL, "the workspace is smaller than archead_rms_norm_workspace asks for");
    const Span su = matrix_span(dy, M, d, ldy, size_of(dy_type)), sh = matrix_span(h, M, d, ldh, size_of(h_type)),
               sr = matrix_span(dres, M, d, ldr, size_of(h_type)), sd = matrix_span(dh, M, d, ldd, size_of(h_type)),
               sg = vector_span(dweight, 4 * d), sw = vector_span(weight, d * size_of(weight_type)),
               work = vector_span(ws, (int64_t)p.total);
    if (overlap({sd, sg, work}, {su, sh, sw}) || overlap_but_itself(sd, sr) || overlap({sg, work}, {sr}) ||
        overlap({sd, sg, work}))
        return api_fail(ARCHEAD_EINVAL, "a result or the workspace overlaps what is read, or another result");
    if (M == 0 && !dweight)
        return ARCHEAD_OK;
    const BackArgs a{M, (int)d, ldy, ldh, ldr, ldd, dy, h, weight, dres, dh, (float *)ws, (float4 *)((char *)ws + p.inv),
                     1. / (double)d, eps, offset, weight_type, p.groups, p.slice};
    hipStream_t stream = (hipStream_t)hip_stream;
    const bool uf = dy_type == ARCHEAD_F32, hf = h_type == ARCHEAD_F32;
    if (M == 0) // no parts: zeros
        hipLaunchKernelGGL(weight_sum_kernel, dim3((unsigned)((d + 31) / 32)), dim3(1024), 0, stream, a.part, 0, d,
                           dweight);
    else if (uf)
        hf ? run_back<float, float>(a, p, dweight, stream) : run_back<float, uint16_t>(a, p, dweight, stream);
    else
        hf ? run_back<uint16_t, float>(a, p, dweight, stream) : run_back<uint16_t, uint16_t>(a, p, dweight, stream);
    return launched("archead_rms_norm_backward");
}
