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
// among the few that reach a bound that sixteen of its columns reach.
// 256 x 151936 fp32 with grammars: 1024 tokens of history, adjusted logits out 61 us,
// 5.1 TB/s, a copy's rate; 8192 tokens and 64 biases, a draw 67 us: routing the
// histories 10, this kernel 53 (2.9 TB/s: of it 37 without any rule, each slice a chain
// of waits with eight workgroups a compute unit to hide them), the draw 7.  One row
// 12 us, of it two launches' work and waits.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "api_internal.hpp"
#include "archead.h"
#include "elements.hpp"
#include "entry.hpp"
#include "kernels.hpp"
#include "overlap.hpp"

namespace archead {
namespace {

typedef int32_t i32x4u __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kNT = 256;
constexpr int64_t kMaxRows = int64_t(1) << 20;
constexpr int64_t kMaxColumns = int64_t(1) << 30; // offsets within a row fit 32 bits
constexpr int64_t kMaxHistory = int64_t(1) << 20;
constexpr int64_t kMaxBias = 1023;
constexpr int64_t kMaxStride = int64_t(1) << 40;
// a column's word in LDS: how often it was generated, whether the prompt has it,
// and its last bias entry (from 1)
constexpr uint32_t kCount = (1u << 21) - 1, kPrompt = 1u << 21;
constexpr int kBiasAt = 22;

struct RuleArgs {
    int64_t M;
    int V, L, B; // columns, tokens and biases of a row
    int64_t ld, ldo, ldh, ldb, R, ldm, S;
    const void *y;
    void *out;
    const int32_t *history, *lengths, *prompts;
    const float *repetition, *frequency, *presence;
    const int32_t *bias_ids;
    const float *bias_values;
    const uint32_t *mask;
    const int32_t *mask_rows;
    int K;
    uint64_t *part;       // [M][K][S] keys, 0 = none
    uint16_t *routed;     // [M][L]: the history by slices (column within one, kRoutedPrompt), or null
    uint32_t *ends;       // [M][S]: where each slice's tokens end
};
constexpr uint32_t kRoutedPrompt = 1u << 15;

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

// A bound that K of the wave's 64 values reach and no more, or, where values are
// equal, the K-th largest of them (0 counts as none): by bits from the top, one
// comparison a bit and scalar arithmetic, where sorting would take 21 exchanges
// through LDS.
__device__ __forceinline__ uint32_t wave_kth(uint32_t v, int K)
{
    uint32_t t = 0;
#pragma unroll 1
    for (uint32_t bit = 1u << 31; bit; bit >>= 1) {
        const int reach = __builtin_popcountll(__ballot(v >= (t | bit)));
        t = reach >= K ? t | bit : t;
        if (reach == K)
            break;
    }
    return t;
}

// the largest, and the smallest, of the values of lanes that are equal in their last
// four bits, and of a row of sixteen
__device__ __forceinline__ uint32_t max_of_rows(uint32_t v)
{
    const auto half = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max((uint32_t)half[0], (uint32_t)half[1]);
    const auto row = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return max((uint32_t)row[0], (uint32_t)row[1]);
}
template <int kCtrl> __device__ __forceinline__ uint32_t min_moved(uint32_t v)
{
    return min(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t min_of_row(uint32_t v)
{
    v = min_moved<kDppQuadXor1>(v);
    v = min_moved<kDppQuadXor2>(v);
    v = min_moved<kDppHalfMirror>(v);
    return min_moved<kDppRowMirror>(v);
}

// The K largest of a workgroup's keys, in order, written by best(rank, key).  A key
// is order << 32 | place, 0 for none; key(thread, e), e < E, reads them from LDS, and
// top is the largest order of the thread's own.  The keys are in sixteen groups (threads
// equal in their last four bits), so sixteen of them, at least K, reach the least of
// the groups' largest, and few others do (of 4096 random ones some 45); the lanes whose
// largest does are looked through by all threads (256 x 151936 without rules 46 us, by
// the waves' bounds alone 53).  Where many do (equal values, a group without any), by a
// bound of a wave's own: at most K of its lanes reach that.
template <int NT, int E, typename Key, typename Best>
__device__ __forceinline__ void block_top(int K, uint32_t top, Key key, Best best)
{
    // at least NT / 64 K, which a wave's own bounds leave (more only where one lane holds
    // many of the slice's largest), and no more than leaves rules_kernel's eight
    // workgroups a compute unit their LDS (seven: 256 x 151936 with rules 77 us, eight 73)
    constexpr int kList = 192;
    constexpr int kGroups = 16, kFewLanes = NT / 2;
    static_assert(kGroups >= kTopKMax);
    __shared__ uint32_t tops[NT / 64][kGroups];
    __shared__ uint64_t bounds[NT / 64];
    __shared__ uint64_t list[kList];
    __shared__ uint32_t n_list, n_lanes;
    __shared__ uint32_t ranks[64];
    __shared__ uint16_t lanes[NT];
    const int tid = threadIdx.x;
    const uint32_t largest = max_of_rows(top);
    if ((tid & 63) < kGroups)
        tops[tid >> 6][tid & 63] = largest;
    if (tid < 64)
        ranks[tid] = 0;
    if (tid == 0)
        n_list = n_lanes = 0;
    __syncthreads();
    uint32_t least = tops[0][tid & (kGroups - 1)];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w)
        least = max(least, tops[w][tid & (kGroups - 1)]);
    least = __builtin_amdgcn_readfirstlane(min_of_row(least));
    uint64_t bound = (uint64_t)least << 32;
    if (top != 0 && top >= least)
        lanes[atomicAdd(&n_lanes, 1u)] = (uint16_t)tid;
    __syncthreads();
    auto gather = [&]() __attribute__((always_inline)) {
#pragma unroll 1
        for (int i = tid; i < (int)n_lanes * E; i += NT) {
            const uint64_t k = key(lanes[i / E], i % E);
            if (k >= bound && k != 0) {
                const uint32_t to = atomicAdd(&n_list, 1u); // in any order: keys are distinct and ranked below
                if (to < kList)
                    list[to] = k;
            }
        }
        __syncthreads();
    };
    const bool few = n_lanes <= (uint32_t)kFewLanes; // of all threads
    if (few)
        gather();
    if (!few || n_list > (uint32_t)kList) {
        auto first = [&](uint32_t t) { // the largest place of the thread's keys of order t
            uint32_t place = 0;
#pragma unroll 1
            for (int e = 0; e < E; ++e) {
                const uint64_t k = key(tid, e);
                place = (uint32_t)(k >> 32) == t ? max(place, (uint32_t)k) : place;
            }
            return place;
        };
        const uint32_t t = wave_kth(top, K);
        uint32_t low = 0;
        if (t != 0 && __builtin_popcountll(__ballot(top >= t)) > K) // several lanes at the bound's value: by place
            low = wave_kth(top == t ? first(t) : 0, K - __builtin_popcountll(__ballot(top > t)));
        if ((tid & 63) == 0)
            bounds[tid >> 6] = (uint64_t)t << 32 | low;
        __syncthreads(); // the counts have been read
        if (tid == 0)
            n_list = n_lanes = 0;
        __syncthreads();
        bound = bounds[0];
#pragma unroll
        for (int w = 1; w < NT / 64; ++w)
            bound = umax64(bound, bounds[w]);
        least = (uint32_t)(bound >> 32);
        if (top != 0 && top >= least && (top > least || (uint32_t)bound == 0 || first(least) >= (uint32_t)bound))
            lanes[atomicAdd(&n_lanes, 1u)] = (uint16_t)tid;
        __syncthreads();
        gather();
    }
    const int n = (int)n_list;
    if (n <= 64) { // a key's rank, counted by a thread of each wave
        const int c = tid & 63, part = tid >> 6;
        const uint64_t k = c < n ? list[c] : 0;
        uint32_t rank = 0;
        for (int j = part; j < n; j += NT / 64)
            rank += list[j] > k;
        if (c < n && rank)
            atomicAdd(&ranks[c], rank);
        __syncthreads();
        if (part == 0 && c < n && ranks[c] < (uint32_t)K)
            best((int)ranks[c], k);
    } else if (n <= kList) {
        const uint64_t k = tid < n ? list[tid] : 0;
        int rank = 0;
        for (int j = 0; j < n; ++j)
            rank += list[j] > k;
        if (tid < n && rank < K)
            best(rank, k);
    } else { // the largest below the last, K times
        uint64_t last = ~(uint64_t)0;
#pragma unroll 1
        for (int rank = 0; rank < K; ++rank) {
            uint64_t most = 0;
#pragma unroll 1
            for (int i = tid; i < (int)n_lanes * E; i += NT) {
                const uint64_t k = key(lanes[i / E], i % E);
                most = k < last ? umax64(most, k) : most;
            }
            for (int off = 32; off >= 1; off >>= 1)
                most = umax64(most, shfl_xor_u64(most, off));
            __syncthreads(); // bounds have been read
            if ((tid & 63) == 0)
                bounds[tid >> 6] = most;
            __syncthreads();
            last = bounds[0];
            for (int w = 1; w < NT / 64; ++w)
                last = umax64(last, bounds[w]);
            if (tid == 0)
                best(rank, last);
        }
    }
    if (tid >= n && tid < K)
        best(tid, (uint64_t)0);
}

// a column that rules name, once its logit is adjusted: its bits + 1, never 0
__device__ __forceinline__ uint32_t settled(float x) { return (x != x ? 0x7FC00000u : __float_as_uint(x)) + 1u; }

// One slice of a row, and what is on its way into registers for it: the first of
// the row's history, then the logits and the mask's words, so that the history's
// arrival does not wait for theirs.
constexpr int kAhead = 4; // loads of four tokens in flight
template <int NT, int E, typename T> struct Slice {
    static constexpr int kCols = NT * E, kVecs = E / 8;
    int64_t m;
    int sl, base, cols, n, prompt; // columns; tokens of the history and of its prompt
    uint32_t from, to;   // or the slice's own of a routed one
    Row r;
    const int32_t *h;
    i32x4u tok[kAhead];
    int routed, bias; // the first of a routed history's words and of the row's bias columns
    Eight<T> raw[kVecs];
    uint32_t bits[kVecs];

    // tokens [i0, i0 + 16 NT) of the history's first `most`, four a thread and load;
    // their last four where there are fewer
    __device__ __forceinline__ void tokens(int i0, int most)
    {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + (k * NT + (int)threadIdx.x) * 4;
            tok[k] = most >= 4 ? *(const i32x4u *)(h + min(i, most - 4))
                               : i32x4u{h[0], h[min(1, most - 1)], h[most - 1], -1};
        }
    }
    static __device__ __forceinline__ int same(int v) { return __builtin_amdgcn_readfirstlane(v); }
    static __device__ __forceinline__ float same(float v) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v))); }
    __device__ __forceinline__ void fetch(const RuleArgs &a, uint32_t at)
    {
        m = at / (uint32_t)a.S;
        sl = (int)(at % (uint32_t)a.S);
        base = sl * kCols;
        cols = min(kCols, a.V - base);
        const T *y = (const T *)a.y + m * a.ld;
        const float rho = a.repetition ? a.repetition[m] : 1.f, beta = a.frequency ? a.frequency[m] : 0.f;
        const float alpha = a.presence ? a.presence[m] : 0.f;
        const int row = a.mask_rows ? a.mask_rows[m] : (int)m, len = a.lengths ? a.lengths[m] : a.L;
        const int head = a.prompts ? a.prompts[m] : 0;
        n = 0;
        if (a.routed) {
            const uint32_t *e = a.ends + m * a.S + sl;
            to = e[0];
            from = sl ? e[-1] : 0;
        } else if (a.history) {
            h = a.history + m * a.ldh;
            if (a.L > 0)
                tokens(0, a.L);
        }
        if (a.bias_ids && a.B > 0)
            bias = a.bias_ids[m * a.ldb + min((int)threadIdx.x, a.B - 1)];
        const int q0 = base / 8 + (int)threadIdx.x;
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
            raw[j] = load_vector<E == 8>(y, q0 + j * NT, a.V);
        if (a.routed && to > from)
            routed = a.routed[m * a.L + min(from + threadIdx.x, to - 1)];
        if (a.history && !a.routed) {
            n = max(0, min(same(len), a.L));
            prompt = same(head);
        }
        r = Row{same(rho), same(beta), same(alpha), a.bias_values ? a.bias_values + m * a.ldb : nullptr,
                nullptr};
        if (a.mask) {
            const int64_t at_row = same(row);
            r.mask = at_row >= 0 && at_row < a.R ? a.mask + at_row * a.ldm : nullptr;
        }
        if (r.mask)
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
                bits[j] = r.mask[min((q0 + j * NT) >> 2, (a.V - 1) >> 5)];
    }
};

// E columns a thread, in vectors of eight
template <int NT, int E, typename T, bool kSelect> __global__ __launch_bounds__(NT) void rules_kernel(RuleArgs a)
{
    constexpr int kCols = NT * E, kVecs = E / 8;
    // Columns that rules name are listed as they are found and adjusted by a thread
    // each: in place, every vector with such a column among its wave's 512 would pay
    // for eight divisions.  A slice with more of them than the list holds does.
    constexpr int kListed = kCols / 8;
    __shared__ alignas(16) uint32_t word[kCols];
    __shared__ uint16_t listed[kListed];
    __shared__ uint32_t n_listed;
    const bool lists = a.history || a.bias_ids;
    Slice<NT, E, T> s;
    s.fetch(a, blockIdx.x);
    const int64_t m = s.m;
    const int sl = s.sl, base = s.base, q0 = base / 8 + (int)threadIdx.x, cols = s.cols;
    const T *y = (const T *)a.y + m * a.ld;
    if (lists) {
        for (int c = threadIdx.x * 4; c < kCols; c += NT * 4)
            *(u32x4 *)&word[c] = u32x4{0, 0, 0, 0};
        if (threadIdx.x == 0)
            n_listed = 0;
        __syncthreads();
        if (a.bias_ids) {
            const int32_t *ids = a.bias_ids + m * a.ldb;
            for (int j = threadIdx.x; j < a.B; j += NT) {
                const uint32_t c = (uint32_t)(j < NT ? s.bias : ids[j]) - (uint32_t)base;
                if (c < (uint32_t)cols && atomicMax(&word[c], (uint32_t)(j + 1) << kBiasAt) == 0) {
                    const uint32_t i = atomicAdd(&n_listed, 1u); // the first to name the column
                    if (i < (uint32_t)kListed)
                        listed[i] = (uint16_t)c;
                }
            }
            __syncthreads();
        }
        if (a.routed) {
            const uint16_t *mine = a.routed + m * a.L;
            for (uint32_t i = s.from + threadIdx.x; i < s.to; i += NT) {
                const uint32_t t = i - s.from < NT ? s.routed : mine[i], c = t & (kRoutedPrompt - 1);
                if ((t & kRoutedPrompt ? atomicOr(&word[c], kPrompt) : atomicAdd(&word[c], 1u)) == 0) {
                    const uint32_t at = atomicAdd(&n_listed, 1u);
                    if (at < (uint32_t)kListed)
                        listed[at] = (uint16_t)c;
                }
            }
        }
        for (int i0 = 0; i0 < s.n; i0 += NT * 4 * kAhead) {
            if (i0 > 0)
                s.tokens(i0, a.L);
            if (i0 + NT * 4 * kAhead > s.n) { // every token once
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int i = i0 + (k * NT + (int)threadIdx.x) * 4, first = max(0, min(i, a.L - 4));
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s.tok[k][e] = first + e >= i && first + e < s.n ? s.tok[k][e] : -1;
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = max(0, min(i0 + (k * NT + (int)threadIdx.x) * 4, a.L - 4));
                uint32_t before[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t c = (uint32_t)s.tok[k][e] - (uint32_t)base; // negative tokens stay above cols
                    before[e] = 1;
                    if (c < (uint32_t)cols)
                        before[e] = i + e < s.prompt ? atomicOr(&word[c], kPrompt) : atomicAdd(&word[c], 1u);
                }
                uint32_t fresh = 0; // columns this thread is the first to name
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    fresh += before[e] == 0;
                if (fresh) {
                    uint32_t to = atomicAdd(&n_listed, fresh);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (before[e] == 0) {
                            if (to < (uint32_t)kListed)
                                listed[to] = (uint16_t)((uint32_t)s.tok[k][e] - (uint32_t)base);
                            ++to;
                        }
                }
            }
        }
        __syncthreads();
        if (n_listed <= (uint32_t)kListed) {
            for (int i = threadIdx.x; i < (int)n_listed; i += NT) {
                const int c = listed[i];
                word[c] = settled(adjust(s.r, load_one(y + base + c), word[c]));
            }
            __syncthreads();
        }
    }
    const bool crowded = lists && n_listed > (uint32_t)kListed;
    float most = -INFINITY; // NaN if any is
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int q = q0 + j * NT;
        uint32_t *mine = &word[8 * (j * NT + threadIdx.x)];
        float v[8];
        widen(s.raw[j], v);
        if (cols < kCols) // the row's last slice
            keep_values(q, a.V, v);
        bool changed = false;
        if (lists) {
            const u32x4 lo = *(const u32x4 *)mine, hi = *(const u32x4 *)(mine + 4);
            changed = (lo.x | lo.y | lo.z | lo.w | hi.x | hi.y | hi.z | hi.w) != 0;
            if (crowded) {
                if (changed)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] = adjust(s.r, v[i], lo[i]);
                        v[4 + i] = adjust(s.r, v[4 + i], hi[i]);
                    }
            } else
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = lo[i] ? __uint_as_float(lo[i] - 1u) : v[i];
                    v[4 + i] = hi[i] ? __uint_as_float(hi[i] - 1u) : v[4 + i];
                }
        }
        if (s.r.mask) {
            const uint32_t byte = s.bits[j] >> (8 * (q & 3));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t let = (uint32_t)__builtin_amdgcn_sbfe((int)byte, i, 1); // all ones or none
                v[i] = __uint_as_float((__float_as_uint(v[i]) & let) | (0xFF800000u & ~let));
            }
        }
        if constexpr (kSelect) {
            if (cols < kCols)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = 8 * q + i < a.V ? v[i] : -INFINITY; // and no key
#pragma unroll
            for (int i = 0; i < 8; ++i)
                most = __builtin_elementwise_maximum(most, v[i]);
            *(f32x4 *)mine = f32x4{v[0], v[1], v[2], v[3]}; // the adjusted logits in the words' place
            *(f32x4 *)(mine + 4) = f32x4{v[4], v[5], v[6], v[7]};
        } else if (8 * q < a.V && (changed || s.r.mask || a.out != a.y))
            store_vector((T *)a.out + m * a.ldo, q, a.V, v);
    }
    if constexpr (kSelect) {
        uint64_t *part = a.part + m * a.S * a.K + sl; // the slices' best first: draw_kernel's groups have each a few
        block_top<NT, E>(
            a.K, 8 * (int)threadIdx.x < cols ? order_of(most) : 0u,
            [&](int thread, int e) {
                const int c = 8 * ((e >> 3) * NT + thread) + (e & 7);
                return c < cols ? (uint64_t)order_of(__uint_as_float(word[c])) << 32 | ~((uint32_t)base + (uint32_t)c)
                                : 0;
            },
            [&](int rank, uint64_t k) { part[rank * a.S] = k; });
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
    __shared__ uint64_t keys[kPer + 1][kNT];
    __shared__ uint64_t win[kTopKMax];
    const int64_t m = blockIdx.x;
    const uint64_t *part = a.part + m * a.n;
    for (int64_t at = 0; at < a.n; at += kNT * kPer) {
        uint64_t k[kPer + 1];
        k[0] = at > 0 && (int)threadIdx.x < a.K ? win[threadIdx.x] : 0; // the best so far
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int64_t i = at + e * kNT + threadIdx.x;
            k[1 + e] = part[min(i, a.n - 1)];
            k[1 + e] = i < a.n ? k[1 + e] : 0;
        }
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e <= kPer; ++e) {
            top = max(top, (uint32_t)(k[e] >> 32));
            keys[e][threadIdx.x] = k[e];
        }
        block_top<kNT, kPer + 1>(
            a.K, top, [&](int thread, int e) { return keys[e][thread]; },
            [&](int rank, uint64_t key) { win[rank] = key; });
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
    if (j < a.K && !none && !first && v > -INFINITY) // -inf / inf, at an infinite temperature, is no number
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

// Long histories of many rows are first sorted by the slices they fall into: a slice's
// workgroup then takes its own tokens in place of the whole list.  One row a
// workgroup; the order within a slice is any, since its tokens are counted.
constexpr int kRouteT = 1024;
constexpr int64_t kRouteSlices = 1024;
constexpr int64_t kRouteRows = 128, kRouteMin = 65536;
__global__ __launch_bounds__(kRouteT) void route_kernel(RuleArgs a, int shift)
{
    __shared__ uint32_t count[kRouteSlices], wave_sums[kRouteT / 64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t m = blockIdx.x;
    const int32_t *h = a.history + m * a.ldh;
    const int n = a.lengths ? max(0, min(a.lengths[m], a.L)) : a.L, prompt = a.prompts ? a.prompts[m] : 0;
    constexpr int kHeld = 8; // a thread's tokens in flight, and kept for the second pass where these are all
    uint32_t t[kHeld];
    auto load = [&](int i0) __attribute__((always_inline)) { // past the end none, negative ones above V
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
            t[k] = (uint32_t)h[min(i0 + k * kRouteT + tid, n - 1)];
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
            t[k] = i0 + k * kRouteT + tid < n ? t[k] : ~0u;
    };
    count[tid] = 0;
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += kHeld * kRouteT) {
        load(i0);
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
            if (t[k] < (uint32_t)a.V)
                atomicAdd(&count[t[k] >> shift], 1u);
    }
    __syncthreads();
    const uint32_t mine = count[tid];
    uint32_t run = mine;
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t o = __shfl_up(run, off);
        run += lane >= off ? o : 0;
    }
    if (lane == 63)
        wave_sums[tid >> 6] = run;
    __syncthreads();
    for (int w = 0; w < tid >> 6; ++w)
        run += wave_sums[w];
    count[tid] = run - mine; // where the slice's next token goes
    if (tid < a.S)
        a.ends[m * a.S + tid] = run;
    __syncthreads();
    uint16_t *to = a.routed + m * a.L;
    for (int i0 = 0; i0 < n; i0 += kHeld * kRouteT) {
        if (n > kHeld * kRouteT)
            load(i0);
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
            if (t[k] < (uint32_t)a.V)
                to[atomicAdd(&count[t[k] >> shift], 1u)] =
                    (uint16_t)((t[k] & ((1u << shift) - 1)) | (i0 + k * kRouteT + tid < prompt ? kRoutedPrompt : 0));
    }
}

// columns a thread: the more, the fewer slices go through a row's lists; fewer where
// that leaves compute units without a workgroup (rows of 151936 with 1024 tokens, a
// draw, in us: 16 columns, 8 columns: one row 15.0, 14.4; 16 rows 22.5, 21.3; 32 rows
// 26.1, 26.9; 128 rows 41, 49), and for rows shorter than a vector, which only that form
// reads element by element
int columns_of(int64_t M, int64_t V) { return V >= 8 && M * ((V + kNT * 16 - 1) / (kNT * 16)) >= 1024 ? 16 : 8; }
int64_t slices_of(int64_t M, int64_t V)
{
    const int64_t c = (int64_t)kNT * columns_of(M, V);
    return (V + c - 1) / c;
}

// where things lie in a workspace: the draw's keys, the routed history
struct RuleWs {
    int64_t S;
    bool route;
    size_t ends, routed, total;
};
RuleWs rule_ws(int64_t M, int64_t V, int64_t L, int K)
{
    RuleWs w{};
    w.S = slices_of(M, V);
    w.ends = (size_t)M * w.S * K * 8;
    w.total = w.ends;
    // a launch of a workgroup a row against every slice's own pass over the row's list: 256
    // rows of 151936 with 2048 tokens 61 us routed, 64 not; 1024 tokens 59, 60; 8192
    // 76, 91; 16 rows with 32768 tokens 53, 46
    w.route = M >= kRouteRows && w.S <= kRouteSlices && w.S * L >= kRouteMin;
    if (w.route) {
        w.routed = w.ends + (size_t)M * w.S * 4;
        w.total = w.routed + (size_t)M * L * 2;
    }
    return w;
}

template <int E, typename T> void launch_rules(const RuleArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)(a.M * a.S));
    if (a.part)
        hipLaunchKernelGGL((rules_kernel<kNT, E, T, true>), grid, dim3(kNT), 0, st, a);
    else
        hipLaunchKernelGGL((rules_kernel<kNT, E, T, false>), grid, dim3(kNT), 0, st, a);
}
template <typename T> void run_rules(const RuleArgs &a, hipStream_t st)
{
    const int e = columns_of(a.M, a.V);
    if (a.routed)
        hipLaunchKernelGGL(route_kernel, dim3((unsigned)a.M), dim3(kRouteT), 0, st, a, e == 16 ? 12 : 11);
    e == 16 ? launch_rules<16, T>(a, st) : launch_rules<8, T>(a, st);
}
// the slices and the workspace's parts
void lay_out(RuleArgs &a, const RuleWs &w, void *ws)
{
    a.S = w.S;
    if (w.route && a.history) {
        a.ends = (uint32_t *)((char *)ws + w.ends);
        a.routed = (uint16_t *)((char *)ws + w.routed);
    }
}

archead_status check_rules(const RuleArgs &a, int64_t V, int64_t L, int64_t B, int type)
{
    if (a.M < 0)
        return api_fail(ARCHEAD_EINVAL, "M < 0");
    if (a.M > kMaxRows || V < 1 || V > kMaxColumns || L > kMaxHistory || B > kMaxBias)
        return api_fail(ARCHEAD_ESHAPE, "M <= 2^20, 1 <= V <= 2^30, histories up to 2^20 tokens, up to 1023 biases a row");
    // a launch holds fewer than 2^32 threads
    if (a.M * slices_of(a.M, V) >= (int64_t(1) << 24))
        return api_fail(ARCHEAD_ESHAPE, "M ceil(V / 4096) must lie below 2^24");
    if (type != ARCHEAD_F32 && type != ARCHEAD_BF16)
        return api_fail(ARCHEAD_EINVAL, "logits must be ARCHEAD_F32 or ARCHEAD_BF16");
    if (a.ld < a.V || a.ld > kMaxStride)
        return api_fail(ARCHEAD_EINVAL, "the row stride must lie in [V, 2^40]");
    if (L < 0 || B < 0 || a.R < 0)
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
    if (misaligned(a.y, size_of(type)))
        return api_fail(ARCHEAD_EINVAL, "logits must be aligned to their element");
    for (const void *p : {(const void *)a.history, (const void *)a.lengths, (const void *)a.prompts,
                          (const void *)a.repetition, (const void *)a.frequency, (const void *)a.presence,
                          (const void *)a.bias_ids, (const void *)a.bias_values, (const void *)a.mask,
                          (const void *)a.mask_rows})
        if (misaligned(p, 4))
            return api_fail(ARCHEAD_EINVAL, "buffers must be aligned to their element");
    return ARCHEAD_OK;
}

// whether a result lies in what the rules are read from, beside the logits
bool in_the_rules(const RuleArgs &a, std::initializer_list<Span> results)
{
    const int64_t lists = a.ldb == 0 ? 1 : a.M;
    return overlap(results, {matrix_span(a.history, a.M, a.L, a.ldh, 4), vector_span(a.lengths, 4 * a.M),
                             vector_span(a.prompts, 4 * a.M), vector_span(a.repetition, 4 * a.M),
                             vector_span(a.frequency, 4 * a.M), vector_span(a.presence, 4 * a.M),
                             matrix_span(a.bias_ids, lists, a.B, a.ldb, 4), matrix_span(a.bias_values, lists, a.B, a.ldb, 4),
                             matrix_span(a.mask, a.R, (a.V + 31) / 32, a.ldm, 4), vector_span(a.mask_rows, 4 * a.M)});
}

archead_status check_ws(const RuleWs &w, const void *ws, uint64_t bytes)
{
    if (w.total && (!ws || misaligned(ws, 16)))
        return api_fail(ARCHEAD_EINVAL, "a 16-byte aligned workspace is required");
    if (bytes < w.total)
        return api_fail(ARCHEAD_EINVAL, "the workspace is smaller than archead_rules_workspace asks for");
    return ARCHEAD_OK;
}

RuleArgs rule_args(int64_t M, int64_t V, const void *logits, int64_t ld, const int32_t *history, int64_t L, int64_t ldh,
                   const int32_t *lengths, const int32_t *prompts, const float *repetition, const float *frequency,
                   const float *presence, const int32_t *bias_ids, const float *bias_values, int64_t B, int64_t ldb,
                   const uint32_t *mask, int64_t R, int64_t ldm, const int32_t *mask_rows)
{
    RuleArgs a{};
    a.M = M;
    a.V = (int)V;
    a.y = logits;
    a.ld = ld;
    a.history = history;
    a.L = (int)L;
    a.ldh = ldh;
    a.lengths = lengths;
    a.prompts = prompts;
    a.repetition = repetition;
    a.frequency = frequency;
    a.presence = presence;
    a.bias_ids = bias_ids;
    a.bias_values = bias_values;
    a.B = (int)B;
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
                                                void *ws, uint64_t ws_bytes, void *hip_stream)
{
    RuleArgs a = rule_args(M, V, logits, ld, history, L, ldh, lengths, prompt_lengths, repetition, frequency, presence,
                           bias_ids, bias_values, B, ldb, mask, R, ldm, mask_rows);
    archead_status s = check_rules(a, V, L, B, type);
    if (s != ARCHEAD_OK)
        return s;
    if (ldo < V || ldo > kMaxStride)
        return api_fail(ARCHEAD_EINVAL, "out's row stride must lie in [V, 2^40]");
    if (M > 0 && !out)
        return api_fail(ARCHEAD_EINVAL, "out is required");
    if (out == logits && M > 0 && ldo != ld)
        return api_fail(ARCHEAD_EINVAL, "in place, out needs the logits' row stride");
    if (misaligned(out, size_of(type)))
        return api_fail(ARCHEAD_EINVAL, "out must be aligned to its element");
    const RuleWs w = rule_ws(M, V, L, 0);
    s = check_ws(w, ws, ws_bytes);
    if (s != ARCHEAD_OK || M == 0)
        return s;
    const int64_t element = size_of(type);
    const Span read = matrix_span(logits, M, V, ld, element), result = matrix_span(out, M, V, ldo, element),
               work = vector_span(w.total ? ws : nullptr, (int64_t)w.total);
    if (overlap_but_itself(result, read) || overlap(work, read) || overlap(result, work) || in_the_rules(a, {result, work}))
        return api_fail(ARCHEAD_EINVAL, "out or the workspace overlaps what is read, or each other");
    a.out = out;
    a.ldo = ldo;
    lay_out(a, w, ws);
    if (type == ARCHEAD_F32)
        run_rules<float>(a, (hipStream_t)hip_stream);
    else
        run_rules<uint16_t>(a, (hipStream_t)hip_stream);
    return launched("archead_adjust_logits");
}

extern "C" archead_status archead_rules_workspace(int64_t M, int64_t V, int64_t L, int32_t K, uint64_t *bytes)
{
    if (!bytes)
        return api_fail(ARCHEAD_EINVAL, "bytes is NULL");
    if (M < 0 || L < 0)
        return api_fail(ARCHEAD_EINVAL, "M < 0 or L < 0");
    if (M > kMaxRows || V < 1 || V > kMaxColumns || L > kMaxHistory || K < 0 || K > kTopKMax || K > V)
        return api_fail(ARCHEAD_ESHAPE, "M, L <= 2^20, 1 <= V <= 2^30 and 0 <= K <= min(16, V)");
    *bytes = rule_ws(M, V, L, K).total;
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
    archead_status s = check_rules(a, V, L, B, type);
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
    const RuleWs w = rule_ws(M, V, L, K);
    s = check_ws(w, ws, ws_bytes);
    if (s != ARCHEAD_OK || M == 0)
        return s;
    const std::initializer_list<Span> results = {vector_span(values, 4 * M * K), vector_span(indices, 4 * M * K),
                                                 vector_span(samples, 4 * M), vector_span(ws, (int64_t)w.total)};
    if (overlap(results, {matrix_span(logits, M, V, ld, size_of(type)), vector_span(temperatures, 4 * M),
                          vector_span(u, 4 * M)}) ||
        overlap(results) || in_the_rules(a, results))
        return api_fail(ARCHEAD_EINVAL, "a result or the workspace overlaps what is read, or another result");
    a.K = K;
    a.part = (uint64_t *)ws;
    lay_out(a, w, ws);
    hipStream_t st = (hipStream_t)hip_stream;
    if (type == ARCHEAD_F32)
        run_rules<float>(a, st);
    else
        run_rules<uint16_t>(a, st);
    const DrawArgs d{M, a.S * K, a.part, K, temperature, temperatures, u, values, indices, samples};
    hipLaunchKernelGGL(draw_kernel, dim3((unsigned)M), dim3(kNT), 0, st, d);
    return launched("archead_sample_logits");
}
