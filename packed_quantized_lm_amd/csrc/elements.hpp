// elements.hpp -- rows of fp32 or bf16 (uint16_t) elements as vectors of eight,
// from any element boundary: a row's last vector may be partial, and rows of odd
// length start anywhere.
#pragma once

#include "device.hpp"

namespace archead {

typedef float f32x4e __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x8e __attribute__((ext_vector_type(8), aligned(2)));
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2e;
typedef __attribute__((ext_vector_type(2))) float f32x2e;

// eight elements as they lie in memory
template <typename T> struct Eight;
template <> struct Eight<float> {
    f32x4e a, b;
};
template <> struct Eight<uint16_t> {
    u16x8e a;
};

__device__ __forceinline__ Eight<float> load_eight(const float *p) { return {*(const f32x4e *)p, *(const f32x4e *)(p + 4)}; }
__device__ __forceinline__ Eight<uint16_t> load_eight(const uint16_t *p) { return {*(const u16x8e *)p}; }
__device__ __forceinline__ float load_one(const float *p) { return *p; }
__device__ __forceinline__ float load_one(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }

__device__ __forceinline__ void widen(const Eight<float> &r, float v[8])
{
    for (int i = 0; i < 4; ++i) {
        v[i] = r.a[i];
        v[4 + i] = r.b[i];
    }
}
__device__ __forceinline__ void widen(const Eight<uint16_t> &r, float v[8])
{
    for (int i = 0; i < 8; ++i)
        v[i] = __uint_as_float((uint32_t)r.a[i] << 16);
}

// values as they lie in memory, rounded once to nearest even
__device__ __forceinline__ void narrow(const float v[8], Eight<float> &o)
{
    for (int i = 0; i < 4; ++i) {
        o.a[i] = v[i];
        o.b[i] = v[4 + i];
    }
}
__device__ __forceinline__ void narrow(const float v[8], Eight<uint16_t> &o)
{
    for (int i = 0; i < 8; i += 2) {
        const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2e{v[i], v[i + 1]}, bf16x2e));
        o.a[i] = (uint16_t)w;
        o.a[i + 1] = (uint16_t)(w >> 16);
    }
}
__device__ __forceinline__ void store_eight(float *p, const Eight<float> &o)
{
    *(f32x4e *)p = o.a;
    *(f32x4e *)(p + 4) = o.b;
}
__device__ __forceinline__ void store_eight(uint16_t *p, const Eight<uint16_t> &o) { *(u16x8e *)p = o.a; }
__device__ __forceinline__ void store_one(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_one(uint16_t *p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

__device__ __forceinline__ void set_element(Eight<float> &r, int i, float e) { (i < 4 ? r.a : r.b)[i & 3] = e; }
__device__ __forceinline__ void set_element(Eight<uint16_t> &r, int i, uint16_t e) { r.a[i] = e; }

// What vector q of a row of d elements is made from: its eight elements, or the
// row's last eight where it has fewer or lies past the end.  No load is under a
// branch of a lane's own, so that all of a thread's stay in flight together.  Int is
// int where rows are short enough (an offset of 32 bits from a uniform base).
template <bool kShort = true, typename T, typename Int>
__device__ __forceinline__ Eight<T> load_vector(const T *row, Int q, Int d)
{
    if (!kShort || d >= 8) // kShort: rows may be shorter than a vector
        return load_eight(row + min((Int)(8 * q), (Int)(d - 8)));
    Eight<T> r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // held in a vector register: of a uniform row the compiler makes scalar loads
        // whose base and offset it splits into halves that need not be multiples of
        // 4 (seen where one kernel reads both element types), and the hardware
        // rounds each down
        int at = (int)min((Int)i, (Int)(d - 1));
        asm volatile("" : "+v"(at));
        set_element(r, i, row[at]);
    }
    return r;
}
// the values of vector q from what load_vector read, zeros past the row's end
template <typename Int> __device__ __forceinline__ void keep_values(Int q, Int d, float v[8])
{
    if (d < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = 8 * q + i < d ? v[i] : 0.f;
    } else {
        const Int past = 8 * q - (d - 8); // elements read before the vector's first
        if (d & 7) {
#pragma unroll
            for (int step = 4; step >= 1; step >>= 1)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = past > 0 && (past & step) ? (i + step < 8 ? v[i + step] : 0.f) : v[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = past >= 8 ? 0.f : v[i];
    }
}
template <typename T, typename Int>
__device__ __forceinline__ void vector_values(Int q, Int d, const Eight<T> &r, float v[8])
{
    widen(r, v);
    keep_values(q, d, v);
}
template <typename T, typename Int> __device__ __forceinline__ void store_vector(T *row, Int q, Int d, const float v[8])
{
    if (8 * q + 8 <= d) {
        Eight<T> o;
        narrow(v, o);
        store_eight(row + 8 * q, o);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (8 * q + i < d)
                store_one(row + 8 * q + i, v[i]);
    }
}

} // namespace archead
