// rules.hip -- what a request asks of its logits before a token is drawn from
// them: penalties for tokens that have occurred, biases and a grammar's mask; the
// adjusted logits themselves, or their K largest and a draw from those.
//
// Column v of row m, with the row's rho, beta, alpha:
//   y1 = y / rho for y > 0, y rho otherwise, where v occurs in the row's history
//   y2 = (y1 - beta count) - alpha where v occurs count > 0 times behind the prompt
//   y3 = y2 + bias of the row's last list entry for v (-inf bans)
//   y4 = -inf where the mask's bit is clear
// Every step is rounded to fp32 by itself.  Draw: as topk.hip's, in fp64.
//
// Bound by the logits' bytes, read once.  A workgroup takes a slice of a row: the
// slice's logits are on their way into registers while the row's history and
// biases are gathered into one word of LDS a column, so that no count is kept
// in memory between calls and a long history costs its own length only (each
// slice reads the row's list, from cache).  The K largest of a slice are found
// among the few that reach a bound: the K-th largest of a wave's 64 lane maxima is
// reached by K of the wave's columns at least, so no column of the slice below the
// best of the four waves' bounds is among the slice's K largest.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "api_internal.hpp"
#include "archead.h"
#include "elements.hpp"
#include "kernels.hpp"

namespace archead {
namespace {

constexpr int kNT = 256;
constexpr int64_t kMaxRows = int64_t(1) << 20;
constexpr int64_t kMaxHistory = int64_t(1) << 20;
constexpr int64_t kMaxBias = 1023;
constexpr int64_t kMaxStride = int64_t(1) << 40;
// a column's word in LDS: how often it was generated, whether the prompt has it,
// and its last bias entry (from 1)
constexpr uint32_t kCount = (1u << 21) - 1, kPrompt = 1u << 21;
constexpr int kBiasAt = 22;

struct RuleArgs {
    int64_t M, V, ld, ldo, L, ldh, B, ldb, R, ldm, S;
    const void *y;
    void *out;
    const int32_t *history, *lengths, *prompts;
    const float *repetition, *frequency, *presence;
    const int32_t *bias_ids;
    const float *bias_values;
    const uint32_t *mask;
    const int32_t *mask_rows;
    int K;
    uint64_t *part; // [M][S][K] keys, 0 = none
};

struct Row {
    float rho, beta, alpha;
    const float *bias;
    const uint32_t *mask; // null: none
};

// one column; every operation rounded by itself, so that equal logits stay equal
__device__ __forceinline__ float adjust(const Row &r, float x, uint32_t w)
{
#pragma clang fp contract(off)
    if (w & (kCount | kPrompt))
        x = x > 0.f ? x / r.rho : x * r.rho;
    if (w & kCount) {
        const float taken = r.beta * (float)(w & kCount);
        x = x - taken;
        x = x - r.alpha;
    }
    if (w >> kBiasAt) {
        const float b = r.bias[(w >> kBiasAt) - 1];
        x = b == -INFINITY ? b : x + b;
    }
    return x;
}

// order of the draw: larger value first, NaN before all; -0 as +0
__device__ __forceinline__ uint32_t order_of(float x) { return x != x ? 0xFFFFFFFFu : orderable(x); }
__device__ __forceinline__ float value_of(uint64_t key)
{
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

__device__ __forceinline__ uint64_t shfl_xor_key(uint64_t k, int off)
{
    return (uint64_t)(uint32_t)__shfl_xor((int)(k >> 32), off) << 32 | (uint32_t)__shfl_xor((int)(uint32_t)k, off);
}

// the wave's keys in descending order over its lanes
__device__ __forceinline__ uint64_t wave_sort(uint64_t k)
{
    const int lane = threadIdx.x & 63;
    for (int size = 2; size <= 64; size <<= 1)
        for (int off = size >> 1; off >= 1; off >>= 1) {
            const uint64_t o = shfl_xor_key(k, off);
            const bool keep_max = ((lane & off) == 0) == ((lane & size) == 0);
            k = (k > o) == keep_max ? k : o;
        }
    return k;
}

// The K largest of the workgroup's keys (key(e), e < E, of each thread; 0 for
// none), in order, written by best(rank, key); list holds 64 E keys.
template <int E, typename Key, typename Best>
__device__ __forceinline__ void block_top(int K, Key key, Best best, uint64_t *list)
{
    __shared__ uint64_t bounds[kNT / 64];
    __shared__ uint32_t n_list;
    uint64_t top = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
        top = umax64(top, key(e));
    const uint64_t sorted = wave_sort(top);
    if ((int)(threadIdx.x & 63) == K - 1)
        bounds[threadIdx.x >> 6] = sorted;
    if (threadIdx.x == 0)
        n_list = 0;
    __syncthreads(); // also: what list overlays has been read
    const uint64_t bound = umax64(umax64(bounds[0], bounds[1]), umax64(bounds[2], bounds[3]));
    if (top >= bound)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint64_t k = key(e);
            if (k >= bound && k != 0)
                list[atomicAdd(&n_list, 1u)] = k; // in any order: keys are distinct and ranked below
        }
    __syncthreads();
    const int n = (int)n_list;
    for (int c = threadIdx.x; c < n; c += kNT) {
        const uint64_t k = list[c];
        int rank = 0;
        for (int j = 0; j < n; ++j)
            rank += list[j] > k;
        if (rank < K)
            best(rank, k);
    }
    for (int c = n + (int)threadIdx.x; c < K; c += kNT)
        best(c, (uint64_t)0);
}

// E columns a thread, in vectors of eight
template <int E, typename T, bool kWrite, bool kSelect> __global__ __launch_bounds__(kNT) void rules_kernel(RuleArgs a)
{
    constexpr int kCols = kNT * E, kVecs = E / 8;
    __shared__ alignas(16) uint32_t word[kCols];
    const int64_t m = blockIdx.x / a.S, sl = blockIdx.x % a.S, base = sl * kCols, q0 = base / 8 + threadIdx.x;
    const int cols = (int)min((int64_t)kCols, a.V - base);
    const T *y = (const T *)a.y + m * a.ld;
    Row r{a.repetition ? a.repetition[m] : 1.f, a.frequency ? a.frequency[m] : 0.f, a.presence ? a.presence[m] : 0.f,
          a.bias_values ? a.bias_values + m * a.ldb : nullptr, nullptr};
    if (a.mask) {
        const int64_t at = a.mask_rows ? a.mask_rows[m] : m;
        r.mask = at >= 0 && at < a.R ? a.mask + at * a.ldm : nullptr;
    }
    Eight<T> raw[kVecs];
    uint32_t bits[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        raw[j] = load_vector(y, q0 + j * kNT, a.V);
        bits[j] = r.mask ? r.mask[min((q0 + j * kNT) >> 2, (a.V - 1) >> 5)] : 0xFFFFFFFFu;
    }
    const bool lists = a.history || a.bias_ids;
    if (lists) {
        for (int c = threadIdx.x * 4; c < kCols; c += kNT * 4)
            *(u32x4 *)&word[c] = u32x4{0, 0, 0, 0};
        __syncthreads();
        if (a.bias_ids) {
            const int32_t *ids = a.bias_ids + m * a.ldb;
            for (int64_t j = threadIdx.x; j < a.B; j += kNT) {
                const int64_t c = (int64_t)ids[j] - base;
                if (c >= 0 && c < cols)
                    atomicMax(&word[c], (uint32_t)(j + 1) << kBiasAt); // the last entry of an id
            }
            __syncthreads();
        }
        if (a.history) {
            const int32_t *h = a.history + m * a.ldh;
            const int64_t len = a.lengths ? max((int64_t)0, min((int64_t)a.lengths[m], a.L)) : a.L;
            const int64_t prompt = a.prompts ? (int64_t)a.prompts[m] : 0;
            for (int64_t i = threadIdx.x; i < len; i += kNT) {
                const int64_t c = (int64_t)h[i] - base;
                if (c >= 0 && c < cols) {
                    if (i < prompt)
                        atomicOr(&word[c], kPrompt);
                    else
                        atomicAdd(&word[c], 1u);
                }
            }
        }
        __syncthreads();
    }
    uint32_t ord[kSelect ? E : 1];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int64_t q = q0 + j * kNT;
        float v[8];
        vector_values(q, a.V, raw[j], v);
        bool changed = false;
        if (lists) {
            const u32x4 lo = *(const u32x4 *)&word[8 * (j * kNT + threadIdx.x)];
            const u32x4 hi = *(const u32x4 *)&word[8 * (j * kNT + threadIdx.x) + 4];
            if ((lo.x | lo.y | lo.z | lo.w | hi.x | hi.y | hi.z | hi.w) != 0) {
                changed = true;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = adjust(r, v[i], lo[i]);
                    v[4 + i] = adjust(r, v[4 + i], hi[i]);
                }
            }
        }
        const uint32_t byte = bits[j] >> (8 * (q & 3)) & 0xFFu;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = byte >> i & 1 ? v[i] : -INFINITY;
        if (kWrite && 8 * q < a.V && (changed || r.mask || a.out != a.y))
            store_vector((T *)a.out + m * a.ldo, q, a.V, v);
        if constexpr (kSelect)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ord[8 * j + i] = 8 * q + i < a.V ? order_of(v[i]) : 0;
    }
    if constexpr (kSelect) {
        uint64_t *part = a.part + (m * a.S + sl) * a.K;
        block_top<E>(
            a.K,
            [&](int e) {
                const uint32_t c = (uint32_t)(base + 8 * ((e >> 3) * kNT + threadIdx.x) + (e & 7));
                return ord[e] ? (uint64_t)ord[e] << 32 | (0xFFFFFFFFu - c) : 0;
            },
            [&](int rank, uint64_t k) { part[rank] = k; }, (uint64_t *)word);
    }
}

struct DrawArgs {
    int64_t M, n; // keys a row
    const uint64_t *part;
    int K;
    float temperature;
    const float *temperatures, *u;
    float *values;
    int32_t *indices, *samples;
};

// one row a workgroup: the K largest of its slices' keys, kPer a thread at a time,
// and the draw
constexpr int kPer = 8;
__global__ __launch_bounds__(kNT) void draw_kernel(DrawArgs a)
{
    __shared__ uint64_t list[64 * (kPer + 1)];
    __shared__ uint64_t win[kTopKMax];
    const int64_t m = blockIdx.x;
    const uint64_t *part = a.part + m * a.n;
    for (int64_t at = 0; at < a.n; at += kNT * kPer) {
        uint64_t k[kPer + 1];
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int64_t i = at + e * kNT + threadIdx.x;
            k[e] = part[min(i, a.n - 1)];
            k[e] = i < a.n ? k[e] : 0;
        }
        k[kPer] = at > 0 && (int)threadIdx.x < a.K ? win[threadIdx.x] : 0; // the best so far
        block_top<kPer + 1>(a.K, [&](int e) { return k[e]; }, [&](int rank, uint64_t key) { win[rank] = key; }, list);
        __syncthreads();
    }
    if (threadIdx.x >= 64)
        return;
    const int j = threadIdx.x;
    const uint64_t key = win[j < a.K ? j : a.K - 1];
    const float v = value_of(key), v0 = value_of(win[0]);
    const int32_t id = (int32_t)(0xFFFFFFFFu - (uint32_t)key);
    if (j < a.K) {
        if (a.values)
            a.values[m * a.K + j] = v;
        if (a.indices)
            a.indices[m * a.K + j] = id;
    }
    if (!a.samples)
        return;
    const float tau = a.temperatures ? a.temperatures[m] : a.temperature;
    const bool none = !(v0 > -INFINITY), first = v0 == INFINITY || !(tau > 0.f);
    double w = 0.;
    if (j < a.K && !none && !first)
        w = exp(((double)v - (double)v0) / (double)tau);
    double run = w; // sums of the weights so far, in a fixed order
    for (int off = 1; off < 16; off <<= 1) {
        const double o = __shfl_up(run, off);
        run += j >= off ? o : 0.;
    }
    const double total = __shfl(run, a.K - 1), t = (double)a.u[m] * total;
    const uint64_t over = __ballot(j < a.K && run > t), has = __ballot(w > 0.);
    int pick = over ? __builtin_ctzll(over) : has ? 63 - __builtin_clzll(has) : 0;
    pick = first ? 0 : pick;
    const int32_t drawn = __shfl(id, pick);
    if (j == 0)
        a.samples[m] = none ? -1 : drawn;
}

// columns a thread: the more, the fewer slices read a row's lists; fewer where
// that leaves compute units without a workgroup
int columns_of(int64_t M, int64_t V)
{
    for (int e : {32, 16})
        if (M * ((V + kNT * e - 1) / (kNT * e)) >= 1024)
            return e;
    return 8;
}
int64_t slices_of(int64_t M, int64_t V)
{
    const int64_t c = (int64_t)kNT * columns_of(M, V);
    return (V + c - 1) / c;
}

template <int E, typename T> void launch_rules(const RuleArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)(a.M * a.S));
    if (a.part)
        hipLaunchKernelGGL((rules_kernel<E, T, false, true>), grid, dim3(kNT), 0, st, a);
    else
        hipLaunchKernelGGL((rules_kernel<E, T, true, false>), grid, dim3(kNT), 0, st, a);
}
template <typename T> void run_rules(const RuleArgs &a, hipStream_t st)
{
    switch (columns_of(a.M, a.V)) {
    case 32: return launch_rules<32, T>(a, st);
    case 16: return launch_rules<16, T>(a, st);
    default: return launch_rules<8, T>(a, st);
    }
}

bool misaligned(const void *p, size_t to) { return (uintptr_t)p % to != 0; }

archead_status check_rules(const RuleArgs &a, int type)
{
    if (a.M < 0)
        return api_fail(ARCHEAD_EINVAL, "M < 0");
    if (a.M > kMaxRows || a.V < 1 || a.V >= (int64_t(1) << 31) || a.L > kMaxHistory || a.B > kMaxBias)
        return api_fail(ARCHEAD_ESHAPE, "M <= 2^20, 1 <= V < 2^31, histories up to 2^20 tokens, up to 1023 biases a row");
    // a launch holds fewer than 2^32 threads
    if (a.M * ((a.V + kNT * 32 - 1) / (kNT * 32)) >= (int64_t(1) << 24))
        return api_fail(ARCHEAD_ESHAPE, "M ceil(V / 8192) must lie below 2^24");
    if (type != ARCHEAD_F32 && type != ARCHEAD_BF16)
        return api_fail(ARCHEAD_EINVAL, "logits must be ARCHEAD_F32 or ARCHEAD_BF16");
    if (a.ld < a.V || a.ld > kMaxStride)
        return api_fail(ARCHEAD_EINVAL, "the row stride must lie in [V, 2^40]");
    if (a.L < 0 || a.B < 0 || a.R < 0)
        return api_fail(ARCHEAD_EINVAL, "a list's length is negative");
    if (a.history ? a.ldh < a.L || a.ldh > kMaxStride : a.lengths || a.prompts)
        return api_fail(ARCHEAD_EINVAL, "a history has a row stride in [its length, 2^40]; lengths belong to one");
    if (!a.bias_ids != !a.bias_values || (a.bias_ids && a.ldb != 0 && (a.ldb < a.B || a.ldb > kMaxStride)))
        return api_fail(ARCHEAD_EINVAL, "bias ids and values come together, with a row stride of 0 or in [entries, 2^40]");
    if (a.mask ? a.ldm < (a.V + 31) / 32 || a.ldm > kMaxStride : a.mask_rows != nullptr)
        return api_fail(ARCHEAD_EINVAL, "a mask has a row stride in [ceil(V / 32), 2^40]; mask rows belong to one");
    if (a.mask && !a.mask_rows && a.R < a.M)
        return api_fail(ARCHEAD_EINVAL, "without mask rows a mask has a row for each row of logits");
    if (a.M > 0 && !a.y)
        return api_fail(ARCHEAD_EINVAL, "logits are required");
    if (misaligned(a.y, type == ARCHEAD_F32 ? 4 : 2))
        return api_fail(ARCHEAD_EINVAL, "logits must be aligned to their element");
    for (const void *p : {(const void *)a.history, (const void *)a.lengths, (const void *)a.prompts,
                          (const void *)a.repetition, (const void *)a.frequency, (const void *)a.presence,
                          (const void *)a.bias_ids, (const void *)a.bias_values, (const void *)a.mask,
                          (const void *)a.mask_rows})
        if (misaligned(p, 4))
            return api_fail(ARCHEAD_EINVAL, "buffers must be aligned to their element");
    return ARCHEAD_OK;
}

archead_status launched(const char *what)
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return api_fail(ARCHEAD_EHIP, std::string(what) + ": " + hipGetErrorString(e));
    return ARCHEAD_OK;
}

RuleArgs rule_args(int64_t M, int64_t V, const void *logits, int64_t ld, const int32_t *history, int64_t L, int64_t ldh,
                   const int32_t *lengths, const int32_t *prompts, const float *repetition, const float *frequency,
                   const float *presence, const int32_t *bias_ids, const float *bias_values, int64_t B, int64_t ldb,
                   const uint32_t *mask, int64_t R, int64_t ldm, const int32_t *mask_rows)
{
    RuleArgs a{};
    a.M = M;
    a.V = V;
    a.y = logits;
    a.ld = ld;
    a.history = history;
    a.L = L;
    a.ldh = ldh;
    a.lengths = lengths;
    a.prompts = prompts;
    a.repetition = repetition;
    a.frequency = frequency;
    a.presence = presence;
    a.bias_ids = bias_ids;
    a.bias_values = bias_values;
    a.B = B;
    a.ldb = ldb;
    a.mask = mask;
    a.R = R;
    a.ldm = ldm;
    a.mask_rows = mask_rows;
    return a;
}

} // namespace
} // namespace archead

using namespace archead;

extern "C" archead_status archead_adjust_logits(int64_t M, int64_t V, const void *logits, int type, int64_t ld,
                                                const int32_t *history, int64_t L, int64_t ldh, const int32_t *lengths,
                                                const int32_t *prompt_lengths, const float *repetition,
                                                const float *frequency, const float *presence, const int32_t *bias_ids,
                                                const float *bias_values, int64_t B, int64_t ldb, const uint32_t *mask,
                                                int64_t R, int64_t ldm, const int32_t *mask_rows, void *out, int64_t ldo,
                                                void *hip_stream)
{
    RuleArgs a = rule_args(M, V, logits, ld, history, L, ldh, lengths, prompt_lengths, repetition, frequency, presence,
                           bias_ids, bias_values, B, ldb, mask, R, ldm, mask_rows);
    archead_status s = check_rules(a, type);
    if (s != ARCHEAD_OK)
        return s;
    if (ldo < V || ldo > kMaxStride)
        return api_fail(ARCHEAD_EINVAL, "out's row stride must lie in [V, 2^40]");
    if (M > 0 && !out)
        return api_fail(ARCHEAD_EINVAL, "out is required");
    if (out == logits && M > 0 && ldo != ld)
        return api_fail(ARCHEAD_EINVAL, "in place, out needs the logits' row stride");
    if (misaligned(out, type == ARCHEAD_F32 ? 4 : 2))
        return api_fail(ARCHEAD_EINVAL, "out must be aligned to its element");
    if (M == 0)
        return ARCHEAD_OK;
    a.out = out;
    a.ldo = ldo;
    a.S = slices_of(M, V);
    if (type == ARCHEAD_F32)
        run_rules<float>(a, (hipStream_t)hip_stream);
    else
        run_rules<uint16_t>(a, (hipStream_t)hip_stream);
    return launched("archead_adjust_logits");
}

extern "C" archead_status archead_sample_workspace(int64_t M, int64_t V, int32_t K, uint64_t *bytes)
{
    if (!bytes)
        return api_fail(ARCHEAD_EINVAL, "bytes is NULL");
    if (M < 0)
        return api_fail(ARCHEAD_EINVAL, "M < 0");
    if (M > kMaxRows || V < 1 || V >= (int64_t(1) << 31) || K < 1 || K > kTopKMax || K > V)
        return api_fail(ARCHEAD_ESHAPE, "M <= 2^20, 1 <= V < 2^31 and 1 <= K <= min(16, V)");
    *bytes = std::max<uint64_t>(16, (uint64_t)M * slices_of(M, V) * K * 8);
    return ARCHEAD_OK;
}

extern "C" archead_status archead_sample_logits(int64_t M, int64_t V, const void *logits, int type, int64_t ld,
                                                const int32_t *history, int64_t L, int64_t ldh, const int32_t *lengths,
                                                const int32_t *prompt_lengths, const float *repetition,
                                                const float *frequency, const float *presence, const int32_t *bias_ids,
                                                const float *bias_values, int64_t B, int64_t ldb, const uint32_t *mask,
                                                int64_t R, int64_t ldm, const int32_t *mask_rows, int32_t K,
                                                float temperature, const float *temperatures, const float *u,
                                                float *values, int32_t *indices, int32_t *samples, void *ws,
                                                uint64_t ws_bytes, void *hip_stream)
{
    RuleArgs a = rule_args(M, V, logits, ld, history, L, ldh, lengths, prompt_lengths, repetition, frequency, presence,
                           bias_ids, bias_values, B, ldb, mask, R, ldm, mask_rows);
    archead_status s = check_rules(a, type);
    if (s != ARCHEAD_OK)
        return s;
    if (K < 1 || K > kTopKMax || K > V)
        return api_fail(ARCHEAD_ESHAPE, "1 <= K <= min(16, V)");
    if (samples && !temperatures && !(temperature > 0.f && std::isfinite(temperature)))
        return api_fail(ARCHEAD_EINVAL, "the temperature must be finite and positive");
    if (M > 0 && !values && !indices && !samples)
        return api_fail(ARCHEAD_EINVAL, "values, indices and samples are all NULL");
    if (M > 0 && samples && !u)
        return api_fail(ARCHEAD_EINVAL, "samples need u");
    for (const void *p : {(const void *)temperatures, (const void *)u, (const void *)values, (const void *)indices,
                          (const void *)samples})
        if (misaligned(p, 4))
            return api_fail(ARCHEAD_EINVAL, "buffers must be aligned to their element");
    if (!ws || misaligned(ws, 16))
        return api_fail(ARCHEAD_EINVAL, "a 16-byte aligned workspace is required");
    a.S = slices_of(M, V);
    if (ws_bytes < (uint64_t)M * a.S * K * 8)
        return api_fail(ARCHEAD_EINVAL, "the workspace is smaller than archead_sample_workspace asks for");
    if (M == 0)
        return ARCHEAD_OK;
    a.K = K;
    a.part = (uint64_t *)ws;
    hipStream_t st = (hipStream_t)hip_stream;
    if (type == ARCHEAD_F32)
        run_rules<float>(a, st);
    else
        run_rules<uint16_t>(a, st);
    const DrawArgs d{M, a.S * K, a.part, K, temperature, temperatures, u, values, indices, samples};
    hipLaunchKernelGGL(draw_kernel, dim3((unsigned)M), dim3(kNT), 0, st, d);
    return launched("archead_sample_logits");
}
