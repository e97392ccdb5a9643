// embed.hip -- rows of an embedding table by token, and the table's gradient.
//
//   out_i = scale * table[token_i]          (8-bit tables: code * its block's scale)
//   dtable[v] = scale * sum over i with token_i = v of dout_i
// Lookup: bound by the rows' bytes (8192 x 2560 bf16: 84 MB in 14 us).  Gradient: bound
// by the table's, where all of it is written, and then by dout's (8192 x 4096 into
// 151936: 1.25 GB written in 205 us, 6.1 TB/s, then 50 us for the rows that occur).  The tokens are sorted (stable, so that a row's
// terms are always added in their order); what a row sums is then one run of the
// sorted list.  Runs are of very different lengths (a few tokens hold much of a
// text): each level of parts sums 32 neighbouring entries of the list where one
// token holds them all, so that a run of any length ends in at most 62 entries of
// each level.  Equal calls give equal bits.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "api_internal.hpp"
#include "archead.h"
#include "elements.hpp"
#include "entry.hpp"
#include "overlap.hpp"

namespace archead {
namespace {

constexpr int kBlk = 128;                        // columns and rows that share a scale of an 8-bit table
constexpr int64_t kMaxTokens = int64_t(1) << 20;
constexpr int64_t kMaxWidth = int64_t(1) << 20;
constexpr int64_t kMaxStride = int64_t(1) << 40;

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
struct LookArgs {
    int64_t n, V;
    int d;
    int64_t ldt, lds, ldo;
    const void *table;
    const float *scales;
    const int32_t *tokens;
    void *out;
    float scale;
    int32_t pad;
};

struct E4m3 {
    uint8_t b;
};
template <typename T> struct Piece {
    Eight<T> raw;
    __device__ __forceinline__ void load(const LookArgs &a, int64_t row, int q)
    {
        raw = load_vector((const T *)a.table + row * a.ldt, q, a.d);
    }
    __device__ __forceinline__ void get(const LookArgs &a, int64_t row, int q, float v[8]) const
    {
        vector_values(q, a.d, raw, v);
    }
};
template <> struct Piece<E4m3> { // d is a multiple of 16, rows 8-byte aligned
    u32x2 raw;
    float s;
    __device__ __forceinline__ void load(const LookArgs &a, int64_t row, int q)
    {
        q = min(q, a.d / 8 - 1);
        raw = *(const u32x2 *)((const uint8_t *)a.table + row * a.ldt + 8 * q);
        s = a.scales[row / kBlk * a.lds + q / (kBlk / 8)];
    }
    __device__ __forceinline__ void get(const LookArgs &, int64_t, int, float v[8]) const
    {
        for (int i = 0; i < 2; ++i) {
            const f32x2e lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)raw[i], false);
            const f32x2e hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)raw[i], true);
            v[4 * i] = lo[0] * s;
            v[4 * i + 1] = lo[1] * s;
            v[4 * i + 2] = hi[0] * s;
            v[4 * i + 3] = hi[1] * s;
        }
    }
};

// T threads a token, U vectors of eight a thread; blockIdx.y walks a long row.  Many wide
// rows: four loads in flight a thread; fewer than fill the card so: one; narrow rows: the
// threads that have a vector (bf16, in us: 8192 x 2560 64 threads of four 14.8, of one
// 15.5; 64 x 4096 32 of one 3.1, 64 of four 3.6; 256 x 4096 3.2, 3.7; 65536 x 64 8 threads
// 4.6, 32 7.9; 65536 x 256 32 of one 11.0, 64 of four 17.2).
template <int T, int U, typename TT, typename OT> __global__ __launch_bounds__(256) void look_kernel(LookArgs a)
{
    const int64_t i = (int64_t)blockIdx.x * (256 / T) + threadIdx.x / T;
    if (i >= a.n)
        return;
    const int nv = (a.d + 7) / 8, q0 = (int)blockIdx.y * (T * U) + (int)threadIdx.x % T;
    const int32_t tok = a.tokens[i];
    const bool held = tok >= 0 && tok < a.V && tok != a.pad;
    const int64_t row = held ? tok : 0;
    OT *out = (OT *)a.out + i * a.ldo;
    Piece<TT> p[U];
    if (held)
#pragma unroll
        for (int j = 0; j < U; ++j)
            p[j].load(a, row, q0 + j * T);
    const float none = tok == a.pad ? 0.f : __builtin_nanf("");
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const int q = q0 + j * T;
        if (q >= nv)
            break;
        float v[8];
        for (int e = 0; e < 8; ++e)
            v[e] = none;
        if (held) {
            p[j].get(a, row, q, v);
            for (int e = 0; e < 8; ++e)
                v[e] *= a.scale;
        }
        store_vector(out, q, a.d, v);
    }
}

template <int T, int U, typename TT, typename OT> void launch_look(const LookArgs &a, hipStream_t st)
{
    const int64_t nv = (a.d + 7) / 8;
    hipLaunchKernelGGL((look_kernel<T, U, TT, OT>),
                       dim3((unsigned)((a.n + 256 / T - 1) / (256 / T)), (unsigned)((nv + T * U - 1) / (T * U))),
                       dim3(256), 0, st, a);
}
template <typename TT, typename OT> void run_look(const LookArgs &a, hipStream_t st)
{
    if (a.d <= 64)
        launch_look<8, 1, TT, OT>(a, st);
    else if (a.d <= 256 || a.n * (int64_t)a.d <= (int64_t(1) << 20))
        launch_look<32, 1, TT, OT>(a, st);
    else
        launch_look<64, 4, TT, OT>(a, st);
}
template <typename TT> void run_look(const LookArgs &a, int out_type, hipStream_t st)
{
    if (out_type == ARCHEAD_F32)
        run_look<TT, float>(a, st);
    else
        run_look<TT, uint16_t>(a, st);
}

// ---------------------------------------------------------------------------
// sorting the tokens
// ---------------------------------------------------------------------------
struct Pair {
    uint32_t key; // the token; the table's length for one that has no row
    uint32_t at;  // its place among the tokens
};

// The table is cleared, where it is written whole, by workgroups of the first launch
// that come after its own `after` ones: all of it, while the tokens are sorted; what
// occurs is written over it (8192 tokens into 151936 x 4096 bf16: clearing alone 190 us,
// 6.5 TB/s, beside 15 of sorting).  Rows as 16-bit words.
struct Clear {
    uint32_t after;
    int64_t rows, ld;
    int words;
    uint16_t *table; // null: nothing to clear
};
__device__ __forceinline__ void clear_rows(const Clear &c)
{
    const int64_t v = (int64_t)(blockIdx.x - c.after) * (blockDim.x / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (v >= c.rows)
        return;
    const float none[8] = {};
    for (int q = threadIdx.x & 63; 8 * q < c.words; q += 64)
        store_vector(c.table + v * c.ld, q, c.words, none);
}
// workgroups of `threads` that clear it
int64_t clear_groups(const Clear &c, int threads) { return c.table ? (c.rows + threads / 64 - 1) / (threads / 64) : 0; }

__device__ __forceinline__ uint32_t key_of(int32_t tok, int64_t V, int32_t pad)
{
    return tok >= 0 && tok < V && tok != pad ? (uint32_t)tok : (uint32_t)V;
}

// Few tokens: each one's place is the number of tokens before it in (key, place)
// order, counted outright: n^2 / 64 comparisons of a wave.  A workgroup places kRank
// tokens; its waves hold 64 kHold tokens of the list at a time in their lanes, and
// compare them with one of the kRank after the other (in a scalar register): one vector
// instruction for 64 pairs, the counting is scalar.  Against the passes below, a whole
// gradient into 32000 x 512: 2048 tokens 23 us, 33; 8192 37, 41; 10240 51, 45 (from 256
// workgroups on a compute unit has two); 16384 70, 50.
constexpr int kRank = 32, kHold = 4, kRankT = 1024;
__global__ __launch_bounds__(kRankT) void rank_kernel(const int32_t *tokens, int64_t n64, int64_t V, int32_t pad,
                                                      Pair *sorted, Clear c)
{
    __shared__ uint32_t meet[kRankT / 64][kRank];
    if (blockIdx.x >= c.after) {
        clear_rows(c);
        return;
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = (int)n64;
    const int first = (int)blockIdx.x * kRank, i = first + (lane & (kRank - 1));
    const int own = i < n ? (int)key_of(tokens[i], V, pad) : 0; // keys fit 31 bits
    uint32_t before = 0; // lane k's: of token first + k
    for (int j0 = wave * 64 * kHold; j0 < n; j0 += kRankT * kHold) {
        int key[kHold];
#pragma unroll
        for (int h = 0; h < kHold; ++h) { // tokens before the workgroup's own count also where keys are equal
            const int j = j0 + 64 * h + lane;
            const int k = (int)key_of(tokens[min(j, n - 1)], V, pad) - (j < first ? 1 : 0);
            key[h] = j < n ? k : 0x7FFFFFFF;
        }
#pragma unroll 4
        for (int k = 0; k < kRank; ++k) {
            const int one = __builtin_amdgcn_readlane(own, k);
            uint32_t c = 0;
#pragma unroll
            for (int h = 0; h < kHold; ++h)
                c += __builtin_popcountll(__ballot(key[h] < one));
            before = lane == k ? before + c : before;
        }
    }
    if (lane < kRank)
        meet[wave][lane] = before;
    __syncthreads();
    if (wave == 0) {
        uint32_t place = 0, ties = 0; // and equal ones before it among the own
        for (int w = 0; w < kRankT / 64; ++w)
            place += meet[w][lane & (kRank - 1)];
        for (int k = 0; k < kRank; ++k) {
            const int one = __builtin_amdgcn_readlane(own, k);
            ties += one == own && k < lane;
        }
        if (lane < kRank && i < n)
            sorted[place + ties] = Pair{(uint32_t)own, (uint32_t)i};
    }
}

// Many tokens: stable passes over kDigit bits of the key, tiles of kTile pairs.
// Each workgroup counts its tile's digits, then every workgroup forms its own
// places from all tiles' counts.
constexpr int kDigit = 9, kDigits = 1 << kDigit, kTile = 2048, kSortT = 512, kPer = kTile / kSortT;

struct SortArgs {
    const int32_t *tokens; // first pass: the keys are theirs
    const Pair *from;
    Pair *to;
    uint32_t *count; // [tiles][kDigits]
    int64_t n, V;
    int32_t pad;
    int shift;
    Clear c;
};
__device__ __forceinline__ Pair sort_pair(const SortArgs &a, int64_t i)
{
    return a.from ? a.from[i] : Pair{key_of(a.tokens[i], a.V, a.pad), (uint32_t)i};
}
__device__ __forceinline__ int digit_of(const SortArgs &a, Pair p) { return (p.key >> a.shift) & (kDigits - 1); }

__global__ __launch_bounds__(kSortT) void digit_count_kernel(SortArgs a)
{
    __shared__ uint32_t count[kDigits];
    if (blockIdx.x >= a.c.after) {
        clear_rows(a.c);
        return;
    }
    count[threadIdx.x] = 0;
    __syncthreads();
    for (int k = 0; k < kPer; ++k) {
        const int64_t i = (int64_t)blockIdx.x * kTile + k * kSortT + threadIdx.x;
        if (i < a.n)
            atomicAdd(&count[digit_of(a, sort_pair(a, i))], 1u); // whole numbers: any order
    }
    __syncthreads();
    a.count[(int64_t)blockIdx.x * kDigits + threadIdx.x] = count[threadIdx.x];
}

__global__ __launch_bounds__(kSortT) void digit_place_kernel(SortArgs a)
{
    constexpr int kWaves = kSortT / 64;
    __shared__ uint32_t mine[kWaves][kDigits]; // a wave's counts, then where its next pair of a digit goes
    __shared__ uint32_t sums[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, d = threadIdx.x; // one digit a thread
    for (int w = 0; w < kWaves; ++w)
        mine[w][d] = 0;
    // all pairs of smaller digits, and the digit's in earlier tiles
    uint32_t all = 0, earlier = 0;
    for (int64_t t = 0; t < gridDim.x; ++t) {
        const uint32_t c = a.count[t * kDigits + d];
        all += c;
        earlier += t < blockIdx.x ? c : 0;
    }
    uint32_t run = all;
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t o = __shfl_up(run, off);
        run += lane >= off ? o : 0;
    }
    if (lane == 63)
        sums[wave] = run;
    __syncthreads();
    uint32_t base = run - all + earlier;
    for (int w = 0; w < wave; ++w)
        base += sums[w];
    // each wave takes kPer rounds of 64 consecutive pairs; a pair's rank in its
    // wave is the count so far and the lanes before it with the same digit
    Pair p[kPer];
    uint32_t rank[kPer];
    int dig[kPer];
    for (int k = 0; k < kPer; ++k) {
        const int64_t i = (int64_t)blockIdx.x * kTile + (wave * kPer + k) * 64 + lane;
        const bool in = i < a.n;
        p[k] = in ? sort_pair(a, i) : Pair{0, 0};
        dig[k] = in ? digit_of(a, p[k]) : -1;
        uint64_t same = __ballot(in);
        for (int b = 0; b < kDigit; ++b) {
            const uint64_t set = __ballot(dig[k] >> b & 1);
            same &= dig[k] >> b & 1 ? set : ~set;
        }
        const uint32_t lower = (uint32_t)__popcll(same & ((uint64_t(1) << lane) - 1));
        rank[k] = in ? mine[wave][dig[k]] + lower : 0;
        __builtin_amdgcn_wave_barrier();
        if (in && lower == 0)
            mine[wave][dig[k]] += (uint32_t)__popcll(same);
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) {
        const uint32_t c = mine[w][d];
        mine[w][d] = base;
        base += c;
    }
    __syncthreads();
    for (int k = 0; k < kPer; ++k)
        if (dig[k] >= 0)
            a.to[mine[wave][dig[k]] + rank[k]] = p[k];
}

// ---------------------------------------------------------------------------
// the rows' sums
// ---------------------------------------------------------------------------
// 32: a wave of a part sums eight rows, all of them soon in flight, and a run is left
// with at most 62 rows of each level
constexpr int kGroup = 32;     // entries of the sorted list (or of a level) a part sums
constexpr int kMaxLevels = 3;  // 32^3 tokens to a part of the last
constexpr int kCols = 512;     // columns a wave takes: eight a lane

struct GradArgs {
    int64_t n, V;
    int d;
    int64_t ldo, ldt;
    const void *dout;
    const Pair *sorted;
    float *part[kMaxLevels]; // [n / 32^(l+1)][d]
    int levels;
    void *dtable;
    float scale;
    int add;
    int64_t tiles; // of kCols columns
};

// rows row(i) .. row(i + left - 1) at vector q onto s, kFly in flight; past the end the
// last again, not added
template <int kFly, bool kShort, typename T, typename Row>
__device__ __forceinline__ void add_some(Row row, int64_t i, int64_t left, int q, int d, float s[8])
{
    Eight<T> r[kFly];
#pragma unroll
    for (int k = 0; k < kFly; ++k)
        r[k] = load_vector<kShort>(row(i + min((int64_t)k, left - 1)), q, d);
#pragma unroll
    for (int k = 0; k < kFly; ++k)
        if (k < left) {
            float v[8];
            vector_values(q, d, r[k], v);
            for (int e = 0; e < 8; ++e)
                s[e] += v[e];
        }
}
// The sum of rows row(from) .. row(to - 1) onto s; most runs are one row.  kDeep: eight
// of a long run in flight in place of four.
template <bool kShort, bool kDeep, typename T, typename Row>
__device__ __forceinline__ void add_rows(Row row, int64_t from, int64_t to, int q, int d, float s[8])
{
    constexpr int kFly = 4;
    int64_t i = from;
    if (kDeep)
        for (; to - i >= 8; i += 8)
            add_some<8, kShort, T>(row, i, 8, q, d, s);
    for (; to - i > 2; i += kFly)
        add_some<kFly, kShort, T>(row, i, to - i, q, d, s);
    for (; i < to; ++i)
        add_some<1, kShort, T>(row, i, 1, q, d, s);
}
// Entries [from, to) of the sorted list (level 0), or of the parts of a level below.
// All 64 lanes come along, whatever their columns: they hold the entries' places.
template <bool kShort, bool kDeep, typename T>
__device__ __forceinline__ void add_entries(const GradArgs &a, int level, int64_t from, int64_t to, int q, float s[8])
{
    if (level == 0) {
        for (int64_t b = from; b < to; b += 64) {
            const uint32_t at = a.sorted[min(b + (int64_t)(threadIdx.x & 63), to - 1)].at;
            add_rows<kShort, kDeep, T>(
                [&](int64_t i) {
                    return (const T *)a.dout + (int64_t)(uint32_t)__builtin_amdgcn_readlane(at, (int)i) * a.ldo;
                },
                0, min(to - b, (int64_t)64), q, a.d, s);
        }
    } else
        add_rows<kShort, kDeep, float>([&](int64_t i) { return a.part[level - 1] + i * a.d; }, from, to, q, a.d, s);
}

// A workgroup per part and kCols columns, for parts whose entries are one token's: its
// four waves sum a quarter each, all of it in flight, and meet in LDS.
template <bool kShort, typename T> __global__ __launch_bounds__(256) void part_kernel(GradArgs a, int level, int64_t parts)
{
    __shared__ float meet[4][64][9]; // nine: neighbouring lanes in different banks
    const int64_t g = blockIdx.x / a.tiles;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (g >= parts)
        return;
    int64_t size = kGroup;
    for (int l = 0; l < level; ++l)
        size *= kGroup;
    const uint32_t key = a.sorted[g * size].key;
    if (key >= a.V || a.sorted[(g + 1) * size - 1].key != key)
        return; // the whole workgroup
    const int q = (int)(blockIdx.x % a.tiles) * (kCols / 8) + lane;
    const int64_t from = g * kGroup + wave * (kGroup / 4);
    float s[8] = {};
    add_entries<kShort, true, T>(a, level, from, from + kGroup / 4, q, s);
    for (int e = 0; e < 8; ++e)
        meet[wave][lane][e] = s[e];
    __syncthreads();
    if (wave == 0 && 8 * q < a.d) {
        for (int e = 0; e < 8; ++e)
            s[e] = (meet[0][lane][e] + meet[1][lane][e]) + (meet[2][lane][e] + meet[3][lane][e]);
        store_vector(a.part[level] + g * a.d, q, a.d, s);
    }
}

template <bool kShort, typename GT> __device__ __forceinline__ void put_row(const GradArgs &a, int64_t v, int q, const float s[8])
{
    GT *row = (GT *)a.dtable + v * a.ldt;
    float o[8] = {};
    if (a.add)
        vector_values(q, a.d, load_vector<kShort>(row, q, a.d), o);
    for (int e = 0; e < 8; ++e)
        o[e] = __builtin_fmaf(a.scale, s[e], o[e]);
    store_vector(row, q, a.d, o);
}

// A wave per entry of the sorted list that begins a run, and kCols columns.
template <bool kShort, bool kDeep, typename T, typename GT> __global__ __launch_bounds__(256) void grad_kernel(GradArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t i = w / a.tiles;
    const int q = (int)(w % a.tiles) * (kCols / 8) + lane;
    if (i >= a.n)
        return;
    // lane l holds entry i - 1 + l: the one before, the run's first and what follows
    const Pair p = a.sorted[max((int64_t)0, min(i - 1 + lane, a.n - 1))];
    const uint32_t key = __builtin_amdgcn_readlane(p.key, 1);
    if (key >= a.V || (i > 0 && __builtin_amdgcn_readlane(p.key, 0) == key))
        return;
    // the run's end: within the lanes', or by halves
    int64_t end = a.n;
    const uint64_t other = __ballot(lane >= 2 && (i - 1 + lane >= a.n || p.key != key));
    if (other)
        end = i - 1 + __builtin_ctzll(other);
    else {
        int64_t lo = i + 63, hi = a.n; // entries below lo are the run's
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if (a.sorted[mid].key == key)
                lo = mid + 1;
            else
                hi = mid;
        }
        end = lo;
    }
    // entries up to the first whole part, parts up to the first whole part of the
    // next level, and so on; then back down
    float s[8] = {};
    auto add_held = [&](int64_t first, int64_t last) __attribute__((always_inline)) { // at most 62 entries from i on
        add_rows<kShort, kDeep, T>(
            [&](int64_t e) {
                return (const T *)a.dout + (int64_t)(uint32_t)__builtin_amdgcn_readlane(p.at, (int)(e - i) + 1) * a.ldo;
            },
            first, last, q, a.d, s);
    };
    int64_t from = i, to = end;
    int64_t tail_from[kMaxLevels + 1], tail_to[kMaxLevels + 1];
    int top = 0;
    for (int l = 0; l <= a.levels; ++l) {
        const int64_t lo = (from + kGroup - 1) / kGroup, hi = to / kGroup;
        top = l;
        if (l == a.levels || lo >= hi) {
            tail_from[l] = from;
            tail_to[l] = to;
            break;
        }
        if (l == 0)
            add_held(from, lo * kGroup);
        else
            add_entries<kShort, kDeep, T>(a, l, from, lo * kGroup, q, s);
        tail_from[l] = hi * kGroup;
        tail_to[l] = to;
        from = lo;
        to = hi;
    }
    for (int l = top; l >= 0; --l) {
        if (l == 0 && top == 0) // no whole part: all of a run of 62 at most
            add_held(tail_from[0], tail_to[0]);
        else
            add_entries<kShort, kDeep, T>(a, l, tail_from[l], tail_to[l], q, s);
    }
    if (8 * q < a.d)
        put_row<kShort, GT>(a, key, q, s);
}

// ---------------------------------------------------------------------------
// Few tokens and a small table: one launch.  A workgroup takes R rows of the table
// (and kCols columns), goes through all tokens for those of its rows, in order, and
// sums each row by a wave, or, where it has many terms, by all of them.
// ---------------------------------------------------------------------------
constexpr int kScanT = 512, kScanWaves = kScanT / 64, kScanMax = 1024, kScanRows = 64, kScanLong = 32;
constexpr int kAtBits = 10; // of a token's place

// the terms of row r among entries [from, to) of the list of matches, added in order
template <bool kShort, typename T>
__device__ __forceinline__ void add_matches(const GradArgs &a, const uint32_t *match, int from, int to, uint32_t r, int q,
                                            float s[8])
{
    constexpr int kFly = 8;
    const int lane = threadIdx.x & 63;
    for (int b = from; b < to; b += 64) {
        const uint32_t e = b + lane < to ? match[b + lane] : ~0u;
        uint64_t bits = __ballot(e >> kAtBits == r);
        while (bits) { // uniform
            const int n = min(__builtin_popcountll(bits), kFly);
            Eight<T> v[kFly];
            int at = 0;
#pragma unroll
            for (int k = 0; k < kFly; ++k) { // past the last the last again, not added
                if (k < n) {
                    at = (int)(__builtin_amdgcn_readlane(e, __builtin_ctzll(bits)) & ((1u << kAtBits) - 1));
                    bits &= bits - 1;
                }
                v[k] = load_vector<kShort>((const T *)a.dout + (int64_t)at * a.ldo, q, a.d);
            }
#pragma unroll
            for (int k = 0; k < kFly; ++k)
                if (k < n) {
                    float f[8];
                    vector_values(q, a.d, v[k], f);
                    for (int i = 0; i < 8; ++i)
                        s[i] += f[i];
                }
        }
    }
}

template <bool kShort, typename T, typename GT>
__global__ __launch_bounds__(kScanT) void scan_grad_kernel(GradArgs a, const int32_t *tokens, int32_t pad, int rows)
{
    __shared__ uint32_t match[kScanMax];
    __shared__ float meet[kScanWaves][64 * 8];
    __shared__ uint32_t count[kScanRows], found[kScanWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = (int)a.n;
    const int64_t v0 = (int64_t)blockIdx.x * rows;
    const uint32_t here = (uint32_t)min((int64_t)rows, a.V - v0);
    const int q = (int)blockIdx.y * (kCols / 8) + lane;
    if (threadIdx.x < kScanRows)
        count[threadIdx.x] = 0;
    // the tokens of a wave's part of the list, and where its matches go
    constexpr int kRounds = kScanMax / kScanT;
    const int part = (n + kScanT - 1) / kScanT * 64, first = wave * part;
    uint32_t row[kRounds];
    uint32_t mine = 0;
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const int i = first + 64 * k + lane;
        const bool in = 64 * k < part && i < n;
        const int32_t t = in ? tokens[i] : -1;
        row[k] = t >= 0 && t != pad ? (uint32_t)t - (uint32_t)v0 : ~0u; // tokens of other rows wrap past `here`
        mine += __builtin_popcountll(__ballot(row[k] < here));
    }
    if (lane == 0)
        found[wave] = mine;
    __syncthreads();
    int to = 0, total = 0;
    for (int w = 0; w < kScanWaves; ++w) {
        to += w < wave ? (int)found[w] : 0;
        total += (int)found[w];
    }
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const bool in = row[k] < here;
        const uint64_t all = __ballot(in);
        if (in) {
            match[to + __builtin_popcountll(all & ((uint64_t(1) << lane) - 1))] =
                row[k] << kAtBits | (uint32_t)(first + 64 * k + lane);
            atomicAdd(&count[row[k]], 1u);
        }
        to += __builtin_popcountll(all);
    }
    __syncthreads();
    for (uint32_t r = wave; r < here; r += kScanWaves) { // a wave a row
        const uint32_t c = count[r];
        if (c > kScanLong || (c == 0 && a.add)) // the same for the wave: all lanes look for matches
            continue;
        float s[8] = {};
        if (c)
            add_matches<kShort, T>(a, match, 0, total, r, q, s);
        if (8 * q < a.d)
            put_row<kShort, GT>(a, v0 + r, q, s);
    }
    for (uint32_t r = 0; r < here; ++r) { // all waves a row
        if (count[r] <= kScanLong)
            continue;
        const int share = (total + kScanWaves - 1) / kScanWaves;
        float s[8] = {};
        add_matches<kShort, T>(a, match, min(wave * share, total), min((wave + 1) * share, total), r, q, s);
        *(f32x4 *)&meet[wave][8 * lane] = f32x4{s[0], s[1], s[2], s[3]};
        *(f32x4 *)&meet[wave][8 * lane + 4] = f32x4{s[4], s[5], s[6], s[7]};
        __syncthreads();
        if (wave == 0 && 8 * q < a.d) {
            for (int w = 1; w < kScanWaves; ++w)
                for (int i = 0; i < 8; ++i)
                    s[i] += meet[w][8 * lane + i];
            put_row<kShort, GT>(a, v0 + r, q, s);
        }
        __syncthreads();
    }
}

// where things lie in a gradient's workspace
struct GradWs {
    size_t sorted, other, count, part[kMaxLevels], total;
    int64_t parts[kMaxLevels], tiles;
    int levels;
};
constexpr int64_t kFewParts = 256;  // of a level, that a run sums without another
constexpr int64_t kRankMax = 8192; // tokens up to which places are counted outright

size_t up16(size_t b) { return (b + 15) / 16 * 16; }
GradWs grad_ws(int64_t n, int64_t V, int64_t d)
{
    GradWs w{};
    w.tiles = (n + kTile - 1) / kTile;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += up16(bytes);
        return here;
    };
    w.sorted = take((size_t)n * sizeof(Pair));
    if (n > kRankMax) {
        w.other = take((size_t)n * sizeof(Pair));
        w.count = take((size_t)w.tiles * kDigits * 4);
    }
    for (int64_t m = n / kGroup; m > 0 && w.levels < kMaxLevels && (w.levels == 0 || w.parts[w.levels - 1] > kFewParts);
         m /= kGroup) {
        w.parts[w.levels] = m;
        w.part[w.levels++] = take((size_t)m * d * 4);
    }
    w.total = std::max<size_t>(16, at);
    return w;
}

template <bool kShort, bool kDeep, typename T> void run_heads(const GradArgs &a, int grad_type, hipStream_t st)
{
    const dim3 grid((unsigned)((a.n * a.tiles + 3) / 4));
    if (grad_type == ARCHEAD_F32)
        hipLaunchKernelGGL((grad_kernel<kShort, kDeep, T, float>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((grad_kernel<kShort, kDeep, T, uint16_t>), grid, dim3(256), 0, st, a);
}
// waves of the last launch up to which the longest run's chain of waits counts, not how
// many waves the registers leave (a whole gradient, deep, not, in us: 4099 x 257 fp32 26.0,
// 28.0; 4096 x 2048 bf16 40.7, 44.0; 8192 x 1000 fp32 61, 66; 8192 x 4096 bf16 265, 260;
// 65536 x 2048 bf16 182, 167)
constexpr int64_t kDeepWaves = 16384;
template <bool kShort, typename T> void run_grad(const GradArgs &a, const GradWs &w, int grad_type, hipStream_t st)
{
    for (int l = 0; l < w.levels; ++l)
        hipLaunchKernelGGL((part_kernel<kShort, T>), dim3((unsigned)(w.parts[l] * a.tiles)), dim3(256), 0, st, a, l,
                           w.parts[l]);
    const int64_t waves = a.n * a.tiles;
    if (waves == 0)
        return;
    waves <= kDeepWaves ? run_heads<kShort, true, T>(a, grad_type, st) : run_heads<kShort, false, T>(a, grad_type, st);
}
// Whether the gradient is taken in one launch: few tokens, and a table small enough that
// the workgroups' passes over the tokens cost less than sorting them (64 tokens into
// 2048 x 256: 6.5 us against 14; 1000 into 32000 x 512: 22, 26; 1000 into 32000 x 2048:
// 67, 38; 4099 into 2048 x 257: 39, 26).
bool scans(int64_t n, int64_t V, int64_t d)
{
    return n <= kScanMax && V * ((d + kCols - 1) / kCols) <= (1 << 15);
}
template <bool kShort, typename T>
void run_scan(const GradArgs &a, const int32_t *tokens, int32_t pad, int grad_type, hipStream_t st)
{
    int rows = 1; // a workgroup's: as many as leave 512 workgroups
    while (rows < kScanRows && a.V * a.tiles >= 1024 * rows)
        rows *= 2;
    const dim3 grid((unsigned)((a.V + rows - 1) / rows), (unsigned)a.tiles);
    if (grad_type == ARCHEAD_F32)
        hipLaunchKernelGGL((scan_grad_kernel<kShort, T, float>), grid, dim3(kScanT), 0, st, a, tokens, pad, rows);
    else
        hipLaunchKernelGGL((scan_grad_kernel<kShort, T, uint16_t>), grid, dim3(kScanT), 0, st, a, tokens, pad, rows);
}
template <typename T>
void run_scan(const GradArgs &a, const int32_t *tokens, int32_t pad, int grad_type, hipStream_t st)
{
    a.d < 8 ? run_scan<true, T>(a, tokens, pad, grad_type, st) : run_scan<false, T>(a, tokens, pad, grad_type, st);
}
template <typename T> void run_grad(const GradArgs &a, const GradWs &w, int grad_type, hipStream_t st)
{
    a.d < 8 ? run_grad<true, T>(a, w, grad_type, st) : run_grad<false, T>(a, w, grad_type, st);
}

archead_status check_sizes(int64_t n, int64_t V, int64_t d)
{
    if (n < 0)
        return api_fail(ARCHEAD_EINVAL, "n < 0");
    if (n > kMaxTokens || V < 1 || V >= (int64_t(1) << 31) || d < 1 || d > kMaxWidth)
        return api_fail(ARCHEAD_ESHAPE, "n <= 2^20, 1 <= V < 2^31 and 1 <= d <= 2^20");
    return ARCHEAD_OK;
}

} // namespace
} // namespace archead

using namespace archead;

extern "C" archead_status archead_embed(int64_t n, int64_t V, int64_t d, const void *table, int table_type, int64_t ldt,
                                        const float *scales, int64_t lds, const int32_t *tokens, int32_t pad,
                                        float scale, void *out, int out_type, int64_t ldo, void *hip_stream)
{
    archead_status st = check_sizes(n, V, d);
    if (st != ARCHEAD_OK)
        return st;
    const bool f8 = table_type == ARCHEAD_E4M3;
    if ((!f8 && bad_type(table_type)) || bad_type(out_type))
        return api_fail(ARCHEAD_EINVAL, "table: ARCHEAD_F32, ARCHEAD_BF16 or ARCHEAD_E4M3; out: the former two");
    if (f8 && d % 16 != 0)
        return api_fail(ARCHEAD_ESHAPE, "an 8-bit table's d is a multiple of 16");
    if (!std::isfinite(scale))
        return api_fail(ARCHEAD_EINVAL, "scale must be finite");
    if (ldt < d || ldt > kMaxStride || ldo < d || ldo > kMaxStride || (f8 && (lds < (d + kBlk - 1) / kBlk || lds > kMaxStride)))
        return api_fail(ARCHEAD_EINVAL, "row strides must lie in [row length, 2^40]");
    if (n == 0)
        return ARCHEAD_OK;
    if (!table || !tokens || !out || (f8 && !scales))
        return api_fail(ARCHEAD_EINVAL, "table, tokens, out and an 8-bit table's scales are required");
    if (f8 ? (uintptr_t)table % 16 || ldt % 16 || misaligned(scales, 4) : misaligned(table, size_of(table_type)))
        return api_fail(ARCHEAD_EINVAL, "table aligned to its element; 8-bit tables and their row strides to 16 bytes");
    if (misaligned(out, size_of(out_type)) || misaligned(tokens, 4))
        return api_fail(ARCHEAD_EINVAL, "buffers must be aligned to their element");
    if (overlap({matrix_span(out, n, d, ldo, size_of(out_type))},
                {matrix_span(table, V, d, ldt, size_of(table_type)), vector_span(tokens, 4 * n),
                 matrix_span(f8 ? scales : nullptr, (V + kBlk - 1) / kBlk, (d + kBlk - 1) / kBlk, lds, 4)}))
        return api_fail(ARCHEAD_EINVAL, "out overlaps what is read");
    const LookArgs a{n, V, (int)d, ldt, lds, ldo, table, scales, tokens, out, scale, pad};
    hipStream_t stream = (hipStream_t)hip_stream;
    if (f8)
        run_look<E4m3>(a, out_type, stream);
    else if (table_type == ARCHEAD_F32)
        run_look<float>(a, out_type, stream);
    else
        run_look<uint16_t>(a, out_type, stream);
    return launched("archead_embed");
}

extern "C" archead_status archead_embed_workspace(int64_t n, int64_t V, int64_t d, uint64_t *bytes)
{
    if (!bytes)
        return api_fail(ARCHEAD_EINVAL, "bytes is NULL");
    archead_status st = check_sizes(n, V, d);
    if (st == ARCHEAD_OK)
        *bytes = grad_ws(n, V, d).total;
    return st;
}

extern "C" archead_status archead_embed_backward(int64_t n, int64_t V, int64_t d, const void *dout, int dout_type,
                                                 int64_t ldo, const int32_t *tokens, int32_t pad, float scale,
                                                 int accumulate, void *dtable, int grad_type, int64_t ldt, void *ws,
                                                 uint64_t ws_bytes, void *hip_stream)
{
    archead_status st = check_sizes(n, V, d);
    if (st != ARCHEAD_OK)
        return st;
    if (bad_type(dout_type) || bad_type(grad_type))
        return api_fail(ARCHEAD_EINVAL, "types are ARCHEAD_F32 or ARCHEAD_BF16");
    if (!std::isfinite(scale))
        return api_fail(ARCHEAD_EINVAL, "scale must be finite");
    if (ldo < d || ldo > kMaxStride || ldt < d || ldt > kMaxStride)
        return api_fail(ARCHEAD_EINVAL, "row strides must lie in [d, 2^40]");
    const GradWs w = grad_ws(n, V, d);
    const int64_t tiles = (d + kCols - 1) / kCols;
    // a launch holds fewer than 2^32 threads
    if (n * tiles > (int64_t(1) << 26) - 4 || V >= (int64_t(1) << 26) - (int64_t(1) << 24))
        return api_fail(ARCHEAD_ESHAPE, "n ceil(d / 512) must be 2^26 - 4 at most, V below 2^26 - 2^24");
    if (!dtable || (n > 0 && (!dout || !tokens)))
        return api_fail(ARCHEAD_EINVAL, "dout, tokens and dtable are required");
    if (misaligned(dout, size_of(dout_type)) || misaligned(dtable, size_of(grad_type)) || misaligned(tokens, 4))
        return api_fail(ARCHEAD_EINVAL, "buffers must be aligned to their element");
    if (!ws || (uintptr_t)ws % 16)
        return api_fail(ARCHEAD_EINVAL, "a 16-byte aligned workspace is required");
    if (ws_bytes < w.total)
        return api_fail(ARCHEAD_EINVAL, "the workspace is smaller than archead_embed_workspace asks for");
    const Span grad = matrix_span(dtable, V, d, ldt, size_of(grad_type)), work = vector_span(ws, (int64_t)w.total);
    if (overlap({grad, work}, {matrix_span(dout, n, d, ldo, size_of(dout_type)), vector_span(tokens, 4 * n)}) ||
        overlap(grad, work))
        return api_fail(ARCHEAD_EINVAL, "dtable or the workspace overlaps what is read, or each other");
    if (n == 0 && accumulate)
        return ARCHEAD_OK;
    char *base = (char *)ws;
    hipStream_t stream = (hipStream_t)hip_stream;
    GradArgs a{};
    a.n = n;
    a.V = V;
    a.d = (int)d;
    a.ldo = ldo;
    a.ldt = ldt;
    a.dout = dout;
    a.sorted = (const Pair *)(base + w.sorted);
    for (int l = 0; l < w.levels; ++l)
        a.part[l] = (float *)(base + w.part[l]);
    a.levels = w.levels;
    a.dtable = dtable;
    a.scale = scale;
    a.add = accumulate != 0;
    a.tiles = tiles;
    if (scans(n, V, d)) {
        dout_type == ARCHEAD_F32 ? run_scan<float>(a, tokens, pad, grad_type, stream)
                                 : run_scan<uint16_t>(a, tokens, pad, grad_type, stream);
        return launched("archead_embed_backward");
    }
    const int words = grad_type == ARCHEAD_F32 ? 2 : 1;
    Clear c{0, V, ldt * words, (int)d * words, accumulate ? nullptr : (uint16_t *)dtable};
    if (n <= kRankMax) {
        c.after = (uint32_t)((n + kRank - 1) / kRank);
        const int64_t groups = c.after + clear_groups(c, kRankT);
        hipLaunchKernelGGL(rank_kernel, dim3((unsigned)groups), dim3(kRankT), 0, stream, tokens, n, V, pad,
                           (Pair *)(base + w.sorted), c);
    } else {
        int bits = 1;
        while (bits < 32 && V >> bits)
            ++bits;
        const int passes = (bits + kDigit - 1) / kDigit;
        c.after = (uint32_t)w.tiles;
        SortArgs s{tokens, nullptr, nullptr, (uint32_t *)(base + w.count), n, V, pad, 0, c};
        for (int p = 0; p < passes; ++p) {
            s.to = (Pair *)(base + ((passes - 1 - p) % 2 ? w.other : w.sorted));
            s.shift = p * kDigit;
            const int64_t groups = w.tiles + (p == 0 ? clear_groups(c, kSortT) : 0);
            hipLaunchKernelGGL(digit_count_kernel, dim3((unsigned)groups), dim3(kSortT), 0, stream, s);
            hipLaunchKernelGGL(digit_place_kernel, dim3((unsigned)w.tiles), dim3(kSortT), 0, stream, s);
            s.from = s.to;
        }
    }
    if (dout_type == ARCHEAD_F32)
        run_grad<float>(a, w, grad_type, stream);
    else
        run_grad<uint16_t>(a, w, grad_type, stream);
    return launched("archead_embed_backward");
}
