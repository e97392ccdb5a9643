// loss.hip -- token log probabilities and the two post-training losses over
// logits, with the logits' gradient: the clipped policy loss with a KL term
// and the preference loss over paired answers.
//
// Row m of the logits y (V wide, target t) has
//   top = max_v y[v],  Z = sum_v exp(y[v] - top),  lse = top + log Z,
//   logp = (y[t] - top) - log Z,  p[v] = exp(y[v] - top) / Z,
// and both losses reach the logits through logp alone:
//   dlogits[v] = c (1[v = t] - p[v]),   c = d loss / d logp[m],
// with 1 - p[t] taken from what is beside the target.
// Policy:     rho = exp(logp - old), kl = exp(ref - logp) - (ref - logp) - 1,
//   loss = sum_m w (-min(rho A, clip(rho, 1 - el, 1 + eh) A) + beta kl),
//   c = w (-A rho [the unclipped branch] + beta (1 - exp(ref - logp))).
// Preference: with s_i = sum w (logp - ref) over answer i and, per pair,
//   h = beta (s_chosen - s_rejected),
//   loss = mean over pairs of -(1 - e) log sigma(h) - e log sigma(-h),
//   c = +-beta/P (sigma(h) - (1 - e)) w  (+ for the chosen answer).
//
// Everything is bound by the logits' bytes: one read for the statistics (a
// running maximum and sum; 2047 x 151936 fp32 205 us, 6.0 TB/s), one more
// read with a write for the gradient.  Where a row's loss needs that row alone
// (policy), a workgroup may keep much of it for the gradient; the preference
// loss sums over answers first and reads twice (1800 x 151936 fp32, bf16
// gradient: 173 + 11 + 294 us).  Every sum has a fixed order: repeated calls
// agree bit for bit.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "api_internal.hpp"
#include "archead.h"
#include "device.hpp"

namespace archead {
namespace {

constexpr int kNT = 256;            // threads of a slice's workgroup
constexpr int kWide = 1024;         // threads of a long row's workgroup
constexpr int kVec = 8;             // elements per thread and step
constexpr int64_t kSliceMin = 4096; // smallest slice of a row
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLog2eLow = (float)(1.44269504088896340736 - (double)kLog2e);

// rows need not be aligned beyond one element (odd V): these vectors are
// loaded and stored as 16 bytes from any element boundary
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x8u __attribute__((ext_vector_type(8), aligned(2)));
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;

// eight elements as they lie in memory, and their values
template <typename T> struct Raw;
template <> struct Raw<float> {
    f32x4u a, b;
};
template <> struct Raw<uint16_t> {
    u16x8u a;
};
__device__ __forceinline__ Raw<float> load_raw(const float *p) { return {*(const f32x4u *)p, *(const f32x4u *)(p + 4)}; }
__device__ __forceinline__ Raw<uint16_t> load_raw(const uint16_t *p) { return {*(const u16x8u *)p}; }
__device__ __forceinline__ void values(const Raw<float> &r, float v[kVec])
{
    for (int i = 0; i < 4; ++i) {
        v[i] = r.a[i];
        v[4 + i] = r.b[i];
    }
}
__device__ __forceinline__ void values(const Raw<uint16_t> &r, float v[kVec])
{
    for (int i = 0; i < 8; ++i)
        v[i] = __uint_as_float((uint32_t)r.a[i] << 16);
}
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }

// the gradient is rounded once, to the type the caller asked for
__device__ __forceinline__ uint16_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
__device__ __forceinline__ void store8(float *p, const float v[kVec])
{
    __builtin_nontemporal_store(f32x4u{v[0], v[1], v[2], v[3]}, (f32x4u *)p);
    __builtin_nontemporal_store(f32x4u{v[4], v[5], v[6], v[7]}, (f32x4u *)(p + 4));
}
__device__ __forceinline__ void store8(uint16_t *p, const float v[kVec])
{
    u16x8u o;
    for (int i = 0; i < 8; i += 2) {
        const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[i], v[i + 1]}, bf16x2));
        o[i] = (uint16_t)w;
        o[i + 1] = (uint16_t)(w >> 16);
    }
    __builtin_nontemporal_store(o, (u16x8u *)p);
}
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = to_bf16(v); }

// exp(x) for x <= 0 as exp2(x log2(e)).  log2(e) is taken in two parts: fp32's
// alone is off by 1.3e-8 relative, which bends every term of a sum the same
// way (measured: margins over 190 tokens five times further from their fp64
// values).
__device__ __forceinline__ float exp_neg(float x)
{
    return __builtin_amdgcn_exp2f(__builtin_fmaf(x, kLog2e, x * kLog2eLow));
}

// Running maximum m and rest = Z - 1, Z = sum of exp(y - m): what there is beside
// the 1 of the maximum itself; m = -inf when empty.  Next to a term of 1 a sum
// rounds off what a token of probability near 1 has for its log probability,
// -log(1 + rest), so the maximum is kept out of the sum (of two logits 18 apart
// in one vector, fp32 keeps nothing of the smaller beside the 1).  rest is fp64
// between vectors of eight.  Against a sum with the maximum in it: 2047 x 151936
// fp32 206 us (206), bf16 113 (110); 2048 x 50021 bf16 policy step 107 (101).
struct Stat {
    double rest;
    float m;
};

// what exp is taken against: the maximum, or 0 while it is -inf (a row or
// part of one whose entries are all -inf adds nothing, and -inf - -inf is
// never formed)
__device__ __forceinline__ float anchor(float m) { return m == -INFINITY ? 0.f : m; }

// Eight logits: of the maximum so far and the next two, the largest goes on and
// the other two are terms of the sum.  A NaN is the least of its three and makes
// rest NaN; an infinite maximum does so in the block's merge.
__device__ __forceinline__ void add8(Stat &st, const float v[kVec])
{
    float m = st.m, e[kVec];
    for (int i = 0; i < kVec; i += 2) {
        const float a = v[i], b = v[i + 1];
        e[i] = __builtin_elementwise_minimum(__builtin_elementwise_minimum(m, a), b);
        e[i + 1] = __builtin_amdgcn_fmed3f(m, a, b);
        m = fmaxf(fmaxf(m, a), b);
    }
    const float r = anchor(m);
    for (int i = 0; i < kVec; ++i)
        e[i] = exp_neg(e[i] - r);
    // pairwise: a thread's chain of additions is an eighth as long
    const float add = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    st = Stat{__builtin_fma(st.rest, (double)exp_neg(st.m - r), (double)add), m};
}
__device__ __forceinline__ void add1(Stat &st, float v)
{
    const float m = fmaxf(st.m, v), r = anchor(m), e = exp_neg(__builtin_elementwise_minimum(st.m, v) - r);
    st = Stat{__builtin_fma(st.rest, (double)exp_neg(st.m - r), (double)e), m};
}

__device__ __forceinline__ Stat merge(Stat a, Stat b)
{
    const bool up = b.m > a.m;
    const Stat hi = up ? b : a, lo = up ? a : b;
    const double x = exp_neg(lo.m - anchor(hi.m));
    return Stat{hi.rest + __builtin_fma(lo.rest, x, x), hi.m};
}

// many parts at once, at their maximum r: exp(p.m - r) is 1 for the parts at the
// maximum, which are counted, and below 1 for the others
struct Fold {
    double rest = 0.;
    float ones = -1.f;
    __device__ __forceinline__ void add(Stat p, float r)
    {
        const float x = exp_neg(p.m - r), f = __builtin_amdgcn_fractf(x);
        rest += __builtin_fma(p.rest, (double)x, (double)f);
        ones += x - f;
    }
    __device__ __forceinline__ double total() const { return rest + (double)ones; }
};

// Statistics of y[0 .. n), one part per thread.  The thread's first H vectors
// stay in held and its next L in its places of more (LDS), for the gradient that
// follows them.
template <int NT, int H, int L, typename T>
__device__ __forceinline__ Stat scan_part(const T *y, int64_t n, Raw<T> (&held)[H > 0 ? H : 1], Raw<T> *more)
{
    Stat st{0., -INFINITY};
    const int64_t nv = n / kVec;
    int64_t q = threadIdx.x;
    if (H > 0 && nv > 0) {
#pragma unroll
        for (int j = 0; j < H; ++j) // all in flight; past the end the last vector again, not counted
            held[j] = load_raw(y + min(q + j * NT, nv - 1) * kVec);
#pragma unroll
        for (int j = 0; j < H; ++j)
            if (q + j * NT < nv) {
                float v[kVec];
                values(held[j], v);
                add8(st, v);
            }
        q += H * NT;
    }
    if (L > 0 && nv > 0) {
        Raw<T> w[L > 0 ? L : 1];
#pragma unroll
        for (int j = 0; j < L; ++j)
            w[j] = load_raw(y + min(q + j * NT, nv - 1) * kVec);
#pragma unroll
        for (int j = 0; j < L; ++j)
            if (q + j * NT < nv) {
                float v[kVec];
                values(w[j], v);
                add8(st, v);
                more[j * NT + threadIdx.x] = w[j]; // read back by this thread alone
            }
        q += L * NT;
    }
    for (; q + NT < nv; q += 4 * NT) { // four loads in flight, past the end as above
        Raw<T> w[4];
        for (int u = 0; u < 4; ++u)
            w[u] = load_raw(y + min(q + u * NT, nv - 1) * kVec);
        for (int u = 0; u < 4; ++u)
            if (q + u * NT < nv) {
                float v[kVec];
                values(w[u], v);
                add8(st, v);
            }
    }
    if (q < nv) {
        float v[kVec];
        values(load_raw(y + q * kVec), v);
        add8(st, v);
    }
    const int64_t i = nv * kVec + threadIdx.x;
    if (i < n)
        add1(st, load1(y + i));
    return st;
}

// merge over the workgroup, the result in every thread
template <int NT> __device__ __forceinline__ Stat block_merge(Stat st, Stat *red)
{
    for (int off = 32; off >= 1; off >>= 1)
        st = merge(st, Stat{__shfl_xor(st.rest, off), __shfl_xor(st.m, off)});
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = st;
    __syncthreads();
    float m = red[0].m;
    for (int w = 1; w < NT / 64; ++w)
        m = fmaxf(m, red[w].m);
    const float r = anchor(m);
    Fold f;
    for (int w = 0; w < NT / 64; ++w)
        f.add(red[w], r);
    return Stat{f.total(), m};
}

struct Rows {
    int64_t M, V, ld;
    const void *y;
    const int32_t *targets;
    const float *weights;   // null: every row counts
    const int32_t *offsets; // preference: answer bounds, else null
    int64_t n_off;
    int64_t S, slice; // slices per row and their length
};

// a row that carries no loss is not read: its logits may hold anything
__device__ __forceinline__ bool row_counts(const Rows &a, int64_t m)
{
    if (a.weights && a.weights[m] == 0.f)
        return false;
    if (a.offsets && (m < a.offsets[0] || m >= a.offsets[a.n_off - 1]))
        return false;
    return true;
}

template <typename T> __device__ __forceinline__ const T *row_ptr(const Rows &a, int64_t m)
{
    return (const T *)a.y + m * a.ld;
}

// log(1 + rest) to rest's own precision: log of the rounded sum and what the
// rounding left out
__device__ __forceinline__ double log_z(double rest)
{
    const double z = 1. + rest;
    return log(z) + (rest - (z - 1.)) * (double)__builtin_amdgcn_rcpf((float)fmax(z, 1.));
}

// Log probability of a row's target and 1 - p, both NaN for a logit yt that is.  A
// row's few scalars are taken in fp64: log Z in fp32 alone is off by up to 5e-7,
// which the losses' differences of log probabilities would keep.  1 - p from
// what is beside the target, (rest + 1 - exp(yt - m)) / Z: with p of fp32 the
// difference would keep nothing for tokens of probability near 1.
struct Token {
    double logp;
    float other;
};
__device__ __forceinline__ Token token_of(Stat st, float yt)
{
    const double beside = st.rest + (1. - (double)exp_neg(yt - anchor(st.m)));
    return Token{((double)yt - (double)st.m) - log_z(st.rest), (float)beside / (float)(1. + st.rest)};
}
// row m's target's logit, NaN for a target outside [0, V)
template <typename T> __device__ __forceinline__ float target_logit(const Rows &a, int64_t m)
{
    const int32_t t = a.targets[m];
    return t >= 0 && t < a.V ? load1(row_ptr<T>(a, m) + t) : __builtin_nanf("");
}
template <typename T> __device__ __forceinline__ Token row_token(const Rows &a, int64_t m, Stat st)
{
    return token_of(st, target_logit<T>(a, m));
}
__device__ __forceinline__ float stat_lse(Stat st) { return (float)((double)st.m + log_z(st.rest)); }

// the slices' parts of one row, eight loads in flight
__device__ __forceinline__ Stat merge_slices(const Stat *part, int64_t S)
{
    Stat st{0., -INFINITY};
    for (int64_t i = 0; i < S; i += 8) {
        Stat p[8];
        for (int u = 0; u < 8; ++u)
            p[u] = part[min(i + u, S - 1)];
        float m = st.m;
        for (int u = 0; u < 8; ++u)
            m = fmaxf(m, p[u].m);
        const float r = anchor(m);
        Fold f;
        f.add(st, r);
        for (int u = 0; u < 8; ++u)
            if (i + u < S)
                f.add(p[u], r);
        st = Stat{f.total(), m};
    }
    return st;
}

// a row's derivative of the loss by its log probability, c, and the target's
// gradient c (1 - p)
struct Coef {
    float c, own;
};

// --- statistics: workgroup (row, slice) -> part[row][slice]; with one slice
// per row logp and lse (if not null) as well ---------------------------------------
template <int NT, typename T>
__global__ __launch_bounds__(NT) void stats_kernel(Rows a, Stat *part, float *logp, float *lse, Coef *coef)
{
    __shared__ Stat red[NT / 64];
    const int64_t m = blockIdx.x / a.S, sl = blockIdx.x % a.S;
    if (!row_counts(a, m)) {
        if (sl == 0 && threadIdx.x == 0) { // no later kernel looks at a row outside every answer
            if (logp)
                logp[m] = 0.f;
            if (coef)
                coef[m] = Coef{0.f, 0.f};
        }
        return;
    }
    const int64_t v0 = sl * a.slice, n = min(a.slice, a.V - v0);
    Raw<T> none[1];
    const Stat st = block_merge<NT>(scan_part<NT, 0, 0, T>(row_ptr<T>(a, m) + v0, n, none, nullptr), red);
    if (threadIdx.x == 0) {
        part[blockIdx.x] = st;
        if (logp && a.S == 1)
            logp[m] = (float)row_token<T>(a, m, st).logp;
        if (lse)
            lse[m] = stat_lse(st);
    }
}

template <typename T>
__global__ __launch_bounds__(kNT) void logp_kernel(Rows a, const Stat *part, float *logp, float *lse)
{
    const int64_t m = (int64_t)blockIdx.x * kNT + threadIdx.x;
    if (m >= a.M)
        return;
    const Stat st = merge_slices(part + m * a.S, a.S);
    if (logp)
        logp[m] = (float)row_token<T>(a, m, st).logp;
    if (lse)
        lse[m] = stat_lse(st);
}

// --- sums in a fixed order ----------------------------------------------------
struct Sum {
    const float *x;
    int64_t n;
    double scale;
    float *out;
};

template <int NT> __device__ __forceinline__ double block_sum(double x, double *red)
{
    for (int off = 32; off >= 1; off >>= 1)
        x += __shfl_xor(x, off);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.;
    for (int w = 0; w < NT / 64; ++w)
        x += red[w];
    return x;
}

template <int NT> __device__ __forceinline__ void sum_all(const Sum &a)
{
    __shared__ double red[NT / 64];
    double s = 0.;
    for (int64_t i = threadIdx.x; i < a.n; i += NT)
        s += a.x[i];
    s = block_sum<NT>(s, red);
    if (threadIdx.x == 0)
        *a.out = (float)(s * a.scale);
}

__global__ __launch_bounds__(kWide) void sum_kernel(Sum a) { sum_all<kWide>(a); }

// --- gradient of a slice -----------------------------------------------------
template <typename G> __device__ __forceinline__ void zero_part(G *g, int64_t n)
{
    const float z[kVec] = {};
    for (int64_t q = threadIdx.x; q < n / kVec; q += blockDim.x)
        store8(g + q * kVec, z);
    const int64_t i = n / kVec * kVec + threadIdx.x;
    if (i < n)
        store1(g + i, 0.f);
}

// g[i] = -c exp(y[i] - m) / (1 + rest) for i in [0, n), own at i = t (relative to y)
template <int NT, int H, int L, typename T, typename G>
__device__ __forceinline__ void grad_part(const T *y, G *g, int64_t n, int64_t t, Coef c, Stat st,
                                          const Raw<T> (&held)[H > 0 ? H : 1], const Raw<T> *more)
{
    const float r = anchor(st.m), k = -c.c / (float)(1. + st.rest);
    auto put = [&](const Raw<T> &w, int64_t q) {
        float v[kVec];
        values(w, v);
        for (int i = 0; i < kVec; ++i)
            v[i] = k * exp_neg(v[i] - r);
        if (t >> 3 == q)
            for (int i = 0; i < kVec; ++i)
                v[i] = (t & 7) == i ? c.own : v[i];
        store8(g + q * kVec, v);
    };
    static_assert(kVec == 8, "t >> 3");
    const int64_t nv = n / kVec;
    int64_t q = threadIdx.x;
    if (H > 0 && nv > 0) {
#pragma unroll
        for (int j = 0; j < H; ++j)
            if (q + j * NT < nv)
                put(held[j], q + j * NT);
        q += H * NT;
    }
    if (L > 0 && nv > 0) {
        for (int j = 0; j < L; ++j)
            if (q + j * NT < nv)
                put(more[j * NT + threadIdx.x], q + j * NT);
        q += L * NT;
    }
    for (; q + NT < nv; q += 4 * NT) {
        Raw<T> w[4];
        for (int u = 0; u < 4; ++u)
            w[u] = load_raw(y + min(q + u * NT, nv - 1) * kVec);
        for (int u = 0; u < 4; ++u)
            if (q + u * NT < nv)
                put(w[u], q + u * NT);
    }
    if (q < nv)
        put(load_raw(y + q * kVec), q);
    const int64_t i = nv * kVec + threadIdx.x;
    if (i < n) {
        const float x = k * exp_neg(load1(y + i) - r);
        store1(g + i, i == t ? c.own : x);
    }
}

// dlogits of slice (row, sl): the row's statistics merged from part, its
// coefficient from coef.  No logit outside the slice is read, so that the
// gradient may be written over the logits.  The first workgroup also sums
// the loss, which saves a launch.
template <typename T, typename G>
__global__ __launch_bounds__(kNT) void grad_kernel(Rows a, const Stat *part, const Coef *coef, const float *gscale,
                                                   G *dy, int64_t ldg, Sum total)
{
    if (blockIdx.x == 0)
        sum_all<kNT>(total);
    // last rows first: the statistics read them last, and what the memory-side
    // cache (256 MB) still holds of them is not fetched again
    const int64_t b = gridDim.x - 1 - (int64_t)blockIdx.x, m = b / a.S, sl = b % a.S;
    const int64_t v0 = sl * a.slice, n = min(a.slice, a.V - v0);
    G *g = dy + m * ldg + v0;
    Coef c = coef[m];
    if (c.c == 0.f) { // a masked or clipped token: its logits are not read
        zero_part(g, n);
        return;
    }
    if (gscale)
        c = Coef{c.c * *gscale, c.own * *gscale};
    const Stat st = merge_slices(part + m * a.S, a.S);
    const Raw<T> none[1] = {};
    grad_part<kNT, 0, 0, T>(row_ptr<T>(a, m) + v0, g, n, (int64_t)a.targets[m] - v0, c, st, none, nullptr);
}

struct Policy {
    const float *old_logp, *ref_logp, *adv;
    float eps_low, eps_high, beta;
};

// one token's loss and its derivative
__device__ __forceinline__ float policy_token(const Policy &p, int64_t m, float w, const Token &tok, Coef *c)
{
    const double logp = tok.logp;
    const double A = p.adv[m], rho = exp(logp - (double)p.old_logp[m]);
    const double cl = fmin(fmax(rho, 1. - (double)p.eps_low), 1. + (double)p.eps_high);
    const double gain = A == 0. ? 0. : rho * A; // no advantage, no gain: also at an infinite ratio
    double loss = -fmin(gain, cl * A);
    double d = gain <= cl * A ? -gain : 0.;
    if (rho != rho || gain != gain) // fmin, fmax and the comparison drop a NaN
        loss = d = __builtin_nan("");
    if (p.beta != 0.f) { // without a KL term an infinite one is never formed
        const double gap = (double)p.ref_logp[m] - logp, e = expm1(gap);
        loss += (double)p.beta * (gap == INFINITY ? e : e - gap); // a masked token's: infinite, not inf - inf
        d -= (double)p.beta * e;
    }
    c->c = (float)(w * d);
    c->own = c->c * tok.other;
    return (float)(w * loss);
}

// The policy loss of a whole row in one workgroup: statistics, loss,
// coefficient and gradient.  The gradient's second pass finds the row in
// registers (the first H vectors of each thread), in LDS (the next L) and in the
// caches.
template <int NT, int H, int L, typename T, typename G>
__global__ __launch_bounds__(NT) void policy_row_kernel(Rows a, Policy pol, const float *gscale, float *logp,
                                                        float *token, G *dy, int64_t ldg)
{
    __shared__ Stat red[NT / 64];
    const int64_t m = blockIdx.x;
    __shared__ Coef coef;
    Stat st{0., 0.f};
    Raw<T> held[H > 0 ? H : 1];
    __shared__ Raw<T> more[L > 0 ? L * NT : 1];
    const T *y = row_ptr<T>(a, m);
    int64_t t = -1;
    float lp = 0.f, loss = 0.f;
    Coef c{0.f, 0.f};
    const bool counts = row_counts(a, m);
    if (counts) {
        t = a.targets[m];
        // read before the barriers: the gradient may be written over it
        const float yt = target_logit<T>(a, m);
        st = block_merge<NT>(scan_part<NT, H, L, T>(y, a.V, held, more), red);
        if (threadIdx.x < 64) { // one wave: fp64 is slow
            const Token tok = token_of(st, yt);
            lp = (float)tok.logp;
            loss = policy_token(pol, m, a.weights[m], tok, &c);
        }
    }
    if (threadIdx.x == 0) {
        token[m] = loss;
        coef = c;
        if (logp)
            logp[m] = lp;
    }
    __syncthreads();
    c = coef;
    if (!dy)
        return;
    G *g = dy + m * ldg;
    if (c.c == 0.f) {
        zero_part(g, a.V);
        return;
    }
    if (gscale)
        c = Coef{c.c * *gscale, c.own * *gscale};
    grad_part<NT, H, L, T>(y, g, a.V, t, c, st, held, more);
}

// --- policy rows: logp, token loss and coefficient of every row -----------------
template <typename T>
__global__ __launch_bounds__(kNT) void policy_rows_kernel(Rows a, const Stat *part, Policy pol, float *logp,
                                                          float *token, Coef *coef)
{
    const int64_t m = (int64_t)blockIdx.x * kNT + threadIdx.x;
    if (m >= a.M)
        return;
    float lp = 0.f, loss = 0.f;
    Coef c{0.f, 0.f};
    if (row_counts(a, m)) {
        const Token tok = row_token<T>(a, m, merge_slices(part + m * a.S, a.S));
        lp = (float)tok.logp;
        loss = policy_token(pol, m, a.weights[m], tok, &c);
    }
    token[m] = loss;
    coef[m] = c;
    if (logp)
        logp[m] = lp;
}

// --- preference pairs: workgroup p -> margin, pair loss, row coefficients ------
template <typename T>
__global__ __launch_bounds__(kNT) void pair_kernel(Rows a, const Stat *part, const float *ref, int64_t P, float beta,
                                                   float smooth, float *logp, float *margins, float *pair,
                                                   Coef *coef)
{
    __shared__ double red[kNT / 64];
    const int64_t p = blockIdx.x;
    // bounds are kept inside [0, M] and in order, whatever the offsets hold
    int64_t b[3];
    for (int i = 0; i < 3; ++i) {
        b[i] = min(max((int64_t)a.offsets[2 * p + i], (int64_t)0), a.M);
        if (i > 0)
            b[i] = max(b[i], b[i - 1]);
    }
    // both answers in one pass, the rejected one's rows with a minus
    double s = 0.;
    for (int64_t m = b[0] + threadIdx.x; m < b[2]; m += kNT) {
        double lp = 0.;
        if (row_counts(a, m)) {
            const Token tok = row_token<T>(a, m, merge_slices(part + m * a.S, a.S));
            lp = tok.logp;
            coef[m].own = tok.other; // this thread's again below
            const double term = (double)a.weights[m] * (lp - (double)(ref ? ref[m] : 0.f));
            s += m < b[1] ? term : -term;
        }
        if (logp)
            logp[m] = (float)lp;
    }
    const double h = (double)beta * block_sum<kNT>(s, red), sm = smooth;
    const double e = exp(-fabs(h)), sp = log1p(e);             // log(1 + exp(-|h|))
    const double up = 1. / (1. + e), down = e / (1. + e);      // sigma(|h|), sigma(-|h|)
    // sigma(h) - (1 - smooth) = smooth sigma(h) - (1 - smooth) sigma(-h)
    const double slope = (double)beta / (double)P * (sm * (h >= 0. ? up : down) - (1. - sm) * (h >= 0. ? down : up));
    for (int64_t m = b[0] + threadIdx.x; m < b[2]; m += kNT) {
        if (row_counts(a, m)) {
            const float c = (float)((m < b[1] ? slope : -slope) * a.weights[m]);
            coef[m] = Coef{c, c * coef[m].own};
        } else {
            coef[m] = Coef{0.f, 0.f};
        }
    }
    if (threadIdx.x == 0) {
        const double over = h != h ? h : fmax(h, 0.), under = h != h ? h : fmax(-h, 0.); // a NaN stays
        // without smoothing the second term's infinity at h = inf is never formed
        pair[p] = (float)((1. - sm) * (sp + under) + (sm != 0. ? sm * (sp + over) : 0.));
        if (margins)
            margins[p] = (float)h;
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr int64_t kMaxRows = int64_t(1) << 20;
constexpr int64_t kTargetWg = 4096; // workgroups that fill the chip with slices
constexpr int64_t kHoldMin = 4096;  // row length from which a row's workgroup keeps logits in registers
constexpr int64_t kCu = 256;        // compute units

// Slices of a row: enough workgroups to fill the chip evenly, each with at
// least kSliceMin logits, in whole steps of a workgroup.
void choose_slices(int64_t M, int64_t V, int64_t *S, int64_t *slice)
{
    int64_t s = std::max<int64_t>(1, kTargetWg / std::max<int64_t>(M, 1));
    s = std::min(s, std::max<int64_t>(1, V / kSliceMin));
    int64_t len = (V + s - 1) / s;
    len = (len + kNT * kVec - 1) / (kNT * kVec) * (kNT * kVec);
    *slice = len;
    *S = (V + len - 1) / len;
}

// Whether the policy loss runs as one workgroup per row (the logits read from
// HBM once) rather than in slices (read twice).  A long row's workgroup fills
// a compute unit, so the rows go in rounds of kCu, and a round that is mostly
// empty can cost more than the second read; the rule asks for 0.7 of a round.
// Measured, fp32 logits, bf16 gradient, us in slices against whole rows:
//   rows               16       64      160      256      300      512
//   V = 151936      17/27    33/28    55/36    70/50    79/72   134/94
//   V = 50257       13/15    16/15    26/17    34/21    36/31    50/36
//   V = 32000       12/12    12/12    19/13    25/13    27/22    37/26
//   V = 12000        11/9    11/10    12/10    13/10    15/15    22/16
// so whole rows are ahead from some 50 rows on, earlier than the rule takes
// them.  Without a gradient the slices lead by up to 11 us at V = 151936 below
// 200 rows (64 rows: 18/30) and the two are within 3 us elsewhere.
bool whole_rows(int64_t M, int64_t V)
{
    if (V <= 4 * kNT * kVec)
        return true; // several rows fit a compute unit
    const int64_t rounds = (M + kCu - 1) / kCu;
    return 10 * M >= 7 * rounds * kCu;
}

struct LossWs {
    size_t part, token, coef, pair, total;
};

LossWs loss_ws(int64_t M, int64_t V, int64_t P)
{
    int64_t S, slice;
    choose_slices(M, V, &S, &slice);
    LossWs w;
    size_t off = 0;
    auto place = [&](size_t bytes) {
        const size_t o = off;
        off += (bytes + 255) / 256 * 256;
        return o;
    };
    w.part = place(sizeof(Stat) * (size_t)(M * S));
    w.token = place(4 * (size_t)M);
    w.coef = place(sizeof(Coef) * (size_t)M);
    w.pair = place(4 * (size_t)P);
    w.total = std::max<size_t>(off, 256);
    return w;
}

archead_status check_common(int64_t M, int64_t V, const void *logits, int type, int64_t ld, const int32_t *targets,
                            void *ws, size_t ws_bytes, int64_t P)
{
    if (M < 0)
        return api_fail(ARCHEAD_EINVAL, "M < 0");
    if (M > kMaxRows)
        return api_fail(ARCHEAD_ESHAPE, "M above 2^20");
    if (V < 1 || V >= (int64_t(1) << 31))
        return api_fail(ARCHEAD_ESHAPE, "V must satisfy 1 <= V < 2^31");
    if (type != ARCHEAD_F32 && type != ARCHEAD_BF16)
        return api_fail(ARCHEAD_EINVAL, "logits must be ARCHEAD_F32 or ARCHEAD_BF16");
    if (ld < V || ld > (int64_t(1) << 40))
        return api_fail(ARCHEAD_EINVAL, "the row stride must lie in [V, 2^40]");
    if (M > 0 && (!logits || !targets))
        return api_fail(ARCHEAD_EINVAL, "logits and targets are required");
    if (!ws || (uintptr_t)ws % 16)
        return api_fail(ARCHEAD_EINVAL, "a 16-byte aligned workspace is required");
    if (ws_bytes < loss_ws(M, V, P).total)
        return api_fail(ARCHEAD_EINVAL, "the workspace is smaller than archead_loss_workspace asks for");
    if ((uintptr_t)logits % (type == ARCHEAD_F32 ? 4 : 2))
        return api_fail(ARCHEAD_EINVAL, "logits must be aligned to their element");
    return ARCHEAD_OK;
}

archead_status check_grad(int64_t V, const void *logits, int type, int64_t ld, const void *dlogits, int grad_type,
                          int64_t ldg)
{
    if (!dlogits)
        return ARCHEAD_OK;
    if (grad_type != ARCHEAD_F32 && grad_type != ARCHEAD_BF16)
        return api_fail(ARCHEAD_EINVAL, "dlogits must be ARCHEAD_F32 or ARCHEAD_BF16");
    if (ldg < V || ldg > (int64_t(1) << 40))
        return api_fail(ARCHEAD_EINVAL, "the gradient's row stride must lie in [V, 2^40]");
    if ((uintptr_t)dlogits % (grad_type == ARCHEAD_F32 ? 4 : 2))
        return api_fail(ARCHEAD_EINVAL, "dlogits must be aligned to its element");
    if (dlogits == logits && (grad_type != type || ldg != ld))
        return api_fail(ARCHEAD_EINVAL, "a gradient in place needs the logits' type and row stride");
    return ARCHEAD_OK;
}

archead_status launched(const char *what)
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return api_fail(ARCHEAD_EHIP, std::string(what) + ": " + hipGetErrorString(e));
    return ARCHEAD_OK;
}

Rows make_rows(int64_t M, int64_t V, const void *logits, int64_t ld, const int32_t *targets, const float *weights)
{
    Rows a{};
    a.M = M;
    a.V = V;
    a.ld = ld;
    a.y = logits;
    a.targets = targets;
    a.weights = weights;
    choose_slices(M, V, &a.S, &a.slice);
    return a;
}

template <typename T>
void run_stats(const Rows &a, Stat *part, float *logp, float *lse, Coef *coef, hipStream_t st)
{
    hipLaunchKernelGGL((stats_kernel<kNT, T>), dim3((unsigned)(a.M * a.S)), dim3(kNT), 0, st, a, part, logp, lse, coef);
}

// Whether the log probabilities take one workgroup of 1024 threads a row, and
// one launch, rather than slices of rows and a second launch that merges them:
// for rows of moderate length unless they are very many (16 x 8200 fp32: 5.9 us
// against 7.1; 1500 x 16000: 23.8 against 21.8), for long ones where they fill
// whole rounds of compute units (256 x 151936: fp32 27.7 us against 32.1, bf16
// 18.6 against 25.0; one row: 14.2 against 9.2).
bool whole_logp(int64_t M, int64_t V)
{
    if (V <= 32768)
        return M <= 2 * kCu;
    return 10 * M >= 9 * ((M + kCu - 1) / kCu * kCu);
}

template <typename T> void run_logp(Rows a, Stat *part, float *logp, float *lse, hipStream_t st)
{
    if (a.S > 1 && whole_logp(a.M, a.V)) {
        a.S = 1;
        a.slice = a.V;
        hipLaunchKernelGGL((stats_kernel<kWide, T>), dim3((unsigned)a.M), dim3(kWide), 0, st, a, part, logp, lse,
                           (Coef *)nullptr);
        return;
    }
    const bool whole = a.S == 1;
    run_stats<T>(a, part, whole ? logp : nullptr, whole ? lse : nullptr, nullptr, st);
    if (!whole)
        hipLaunchKernelGGL(logp_kernel<T>, dim3((unsigned)((a.M + kNT - 1) / kNT)), dim3(kNT), 0, st, a, part, logp,
                           lse);
}

void run_sum(const float *x, int64_t n, double scale, float *out, hipStream_t st)
{
    hipLaunchKernelGGL(sum_kernel, dim3(1), dim3(kWide), 0, st, Sum{x, n, scale, out});
}

struct Grad {
    const float *scale;
    void *dy;
    int type;
    int64_t ld;
};

template <typename T>
void run_grad(const Rows &a, const Stat *part, const Coef *coef, const Grad &g, const Sum &total, hipStream_t st)
{
    const dim3 grid((unsigned)(a.M * a.S));
    if (g.type == ARCHEAD_F32)
        hipLaunchKernelGGL((grad_kernel<T, float>), grid, dim3(kNT), 0, st, a, part, coef, g.scale, (float *)g.dy, g.ld,
                           total);
    else
        hipLaunchKernelGGL((grad_kernel<T, uint16_t>), grid, dim3(kNT), 0, st, a, part, coef, g.scale,
                           (uint16_t *)g.dy, g.ld, total);
}

template <int NT, int H, int L, typename T>
void run_policy_rows(const Rows &a, const Policy &pol, float *logp, float *token, const Grad &g, hipStream_t st)
{
    if (g.type == ARCHEAD_F32)
        hipLaunchKernelGGL((policy_row_kernel<NT, H, 0, T, float>), dim3((unsigned)a.M), dim3(NT), 0, st, a, pol, g.scale,
                           logp, token, (float *)g.dy, g.ld);
    else
        hipLaunchKernelGGL((policy_row_kernel<NT, H, L, T, uint16_t>), dim3((unsigned)a.M), dim3(NT), 0, st, a, pol,
                           g.scale, logp, token, (uint16_t *)g.dy, g.ld);
}

// Threads and held vectors by the row's length: as many vectors held as the
// row fills (a vector past its end is a wasted load: 2048 rows of 50021 bf16
// logits take 130 us with 16 held of which 6 are filled, 113 us with none) and
// the registers of 1024 threads allow.  2048 rows of 151936 fp32 logits with a
// bf16 gradient: 411 us with eight held, 508 us with none.  LDS holds four more
// of fp32 logits where the gradient is in bf16 (393 us; 2048 x 128256: 318
// against 343); with an fp32 gradient they cost more than they save (687 us
// against 661).  bf16 logits do without them (274 us; with them 262).
template <typename T>
void run_policy_whole(const Rows &a, const Policy &pol, float *logp, float *token, const Grad &g, hipStream_t st)
{
    const int64_t narrow = (a.V + kNT * kVec - 1) / (kNT * kVec), wide = (a.V + kWide * kVec - 1) / (kWide * kVec);
    if (!g.dy || a.V < kHoldMin)
        run_policy_rows<kNT, 0, 0, T>(a, pol, logp, token, g, st);
    else if (narrow <= 4)
        run_policy_rows<kNT, 4, 0, T>(a, pol, logp, token, g, st);
    else if (wide < 4)
        run_policy_rows<kWide, 2, 0, T>(a, pol, logp, token, g, st);
    else if (wide < 8)
        run_policy_rows<kWide, 4, 0, T>(a, pol, logp, token, g, st);
    else if constexpr (sizeof(T) == 2) {
        if (wide < 16)
            run_policy_rows<kWide, 8, 0, T>(a, pol, logp, token, g, st);
        else
            run_policy_rows<kWide, 16, 0, T>(a, pol, logp, token, g, st);
    } else if (wide < 12)
        run_policy_rows<kWide, 8, 0, T>(a, pol, logp, token, g, st);
    else
        run_policy_rows<kWide, 8, 4, T>(a, pol, logp, token, g, st);
}

template <typename T>
void run_policy(const Rows &a, void *ws, const LossWs &L, const Policy &pol, float *loss, float *logp, const Grad &g,
                hipStream_t st)
{
    Stat *part = (Stat *)((char *)ws + L.part);
    float *token = (float *)((char *)ws + L.token);
    Coef *coef = (Coef *)((char *)ws + L.coef);
    if (whole_rows(a.M, a.V)) {
        run_policy_whole<T>(a, pol, logp, token, g, st);
        run_sum(token, a.M, 1.0, loss, st);
        return;
    }
    run_stats<T>(a, part, nullptr, nullptr, nullptr, st);
    hipLaunchKernelGGL(policy_rows_kernel<T>, dim3((unsigned)((a.M + kNT - 1) / kNT)), dim3(kNT), 0, st, a, part, pol,
                       logp, token, coef);
    if (g.dy)
        run_grad<T>(a, part, coef, g, Sum{token, a.M, 1.0, loss}, st);
    else
        run_sum(token, a.M, 1.0, loss, st);
}

template <typename T>
void run_preference(const Rows &a, void *ws, const LossWs &L, const float *ref, int64_t P, float beta, float smoothing,
                    float *loss, float *logp, float *margins, const Grad &g, hipStream_t st)
{
    Stat *part = (Stat *)((char *)ws + L.part);
    Coef *coef = (Coef *)((char *)ws + L.coef);
    float *pair = (float *)((char *)ws + L.pair);
    if (a.M > 0)
        run_stats<T>(a, part, logp, nullptr, coef, st);
    hipLaunchKernelGGL(pair_kernel<T>, dim3((unsigned)P), dim3(kNT), 0, st, a, part, ref, P, beta, smoothing, logp,
                       margins, pair, coef);
    if (a.M > 0 && g.dy)
        run_grad<T>(a, part, coef, g, Sum{pair, P, 1.0 / (double)P, loss}, st);
    else
        run_sum(pair, P, 1.0 / (double)P, loss, st);
}

} // namespace
} // namespace archead

using namespace archead;

extern "C" archead_status archead_loss_workspace(int64_t M, int64_t V, int64_t P, uint64_t *bytes)
{
    if (!bytes)
        return api_fail(ARCHEAD_EINVAL, "bytes is NULL");
    if (M < 0 || P < 0)
        return api_fail(ARCHEAD_EINVAL, "M < 0 or P < 0");
    if (M > kMaxRows || P > kMaxRows || V < 1 || V >= (int64_t(1) << 31))
        return api_fail(ARCHEAD_ESHAPE, "M, P <= 2^20 and 1 <= V < 2^31");
    *bytes = loss_ws(M, V, P).total;
    return ARCHEAD_OK;
}

extern "C" archead_status archead_token_logp(int64_t M, int64_t V, const void *logits, int type, int64_t ld,
                                             const int32_t *targets, float *logp, float *lse, void *ws,
                                             uint64_t ws_bytes, void *hip_stream)
{
    archead_status s = check_common(M, V, logits, type, ld, targets, ws, ws_bytes, 0);
    if (s != ARCHEAD_OK)
        return s;
    if (M > 0 && !logp && !lse)
        return api_fail(ARCHEAD_EINVAL, "logp and lse are both NULL");
    if (M == 0)
        return ARCHEAD_OK;
    hipStream_t st = (hipStream_t)hip_stream;
    const Rows a = make_rows(M, V, logits, ld, targets, nullptr);
    Stat *part = (Stat *)((char *)ws + loss_ws(M, V, 0).part);
    if (type == ARCHEAD_F32)
        run_logp<float>(a, part, logp, lse, st);
    else
        run_logp<uint16_t>(a, part, logp, lse, st);
    return launched("archead_token_logp");
}

extern "C" archead_status archead_policy_loss(int64_t M, int64_t V, const void *logits, int type, int64_t ld,
                                              const int32_t *targets, const float *old_logp, const float *ref_logp,
                                              const float *advantages, const float *weights, float eps_low,
                                              float eps_high, float beta, const float *grad_scale, float *loss,
                                              float *logp, void *dlogits, int grad_type, int64_t ldg, void *ws,
                                              uint64_t ws_bytes, void *hip_stream)
{
    archead_status s = check_common(M, V, logits, type, ld, targets, ws, ws_bytes, 0);
    if (s == ARCHEAD_OK)
        s = check_grad(V, logits, type, ld, dlogits, grad_type, ldg);
    if (s != ARCHEAD_OK)
        return s;
    if (!(eps_low >= 0.f && eps_low <= 1.f) || !(eps_high >= 0.f) || !std::isfinite(eps_high))
        return api_fail(ARCHEAD_EINVAL, "0 <= eps_low <= 1 and a finite eps_high >= 0");
    if (!(beta >= 0.f) || !std::isfinite(beta))
        return api_fail(ARCHEAD_EINVAL, "beta must be finite and not negative");
    if (!loss)
        return api_fail(ARCHEAD_EINVAL, "loss is NULL");
    if (M > 0 && (!old_logp || !advantages || !weights || (beta != 0.f && !ref_logp)))
        return api_fail(ARCHEAD_EINVAL, "old_logp, advantages, weights and, with beta, ref_logp are required");
    hipStream_t st = (hipStream_t)hip_stream;
    const LossWs L = loss_ws(M, V, 0);
    const Policy pol{old_logp, ref_logp, advantages, eps_low, eps_high, beta};
    const Grad g{grad_scale, dlogits, grad_type, ldg};
    const Rows a = make_rows(M, V, logits, ld, targets, weights);
    if (M > 0 && type == ARCHEAD_F32)
        run_policy<float>(a, ws, L, pol, loss, logp, g, st);
    else if (M > 0)
        run_policy<uint16_t>(a, ws, L, pol, loss, logp, g, st);
    else
        run_sum(nullptr, 0, 1.0, loss, st);
    return launched("archead_policy_loss");
}

extern "C" archead_status archead_preference_loss(int64_t M, int64_t V, const void *logits, int type, int64_t ld,
                                                  const int32_t *targets, const float *weights, int64_t P,
                                                  const int32_t *offsets, const float *ref_logp, float beta,
                                                  float smoothing, const float *grad_scale, float *loss,
                                                  float *margins, float *logp, void *dlogits, int grad_type,
                                                  int64_t ldg, void *ws, uint64_t ws_bytes, void *hip_stream)
{
    if (P < 1)
        return api_fail(ARCHEAD_EINVAL, "P must be at least 1");
    if (P > kMaxRows)
        return api_fail(ARCHEAD_ESHAPE, "P above 2^20");
    archead_status s = check_common(M, V, logits, type, ld, targets, ws, ws_bytes, P);
    if (s == ARCHEAD_OK)
        s = check_grad(V, logits, type, ld, dlogits, grad_type, ldg);
    if (s != ARCHEAD_OK)
        return s;
    if (!(beta > 0.f) || !std::isfinite(beta))
        return api_fail(ARCHEAD_EINVAL, "beta must be finite and positive");
    if (!(smoothing >= 0.f && smoothing < 0.5f))
        return api_fail(ARCHEAD_EINVAL, "0 <= smoothing < 1/2");
    if (!loss || !offsets || (M > 0 && !weights))
        return api_fail(ARCHEAD_EINVAL, "loss, offsets and weights are required");
    hipStream_t st = (hipStream_t)hip_stream;
    const LossWs L = loss_ws(M, V, P);
    Rows a = make_rows(M, V, logits, ld, targets, weights);
    a.offsets = offsets;
    a.n_off = 2 * P + 1;
    const Grad g{grad_scale, dlogits, grad_type, ldg};
    if (type == ARCHEAD_F32)
        run_preference<float>(a, ws, L, ref_logp, P, beta, smoothing, loss, logp, margins, g, st);
    else
        run_preference<uint16_t>(a, ws, L, ref_logp, P, beta, smoothing, loss, logp, margins, g, st);
    return launched("archead_preference_loss");
}
