// vecio.hpp -- loads and stores of short runs of elements at any element alignment.
//
// gfx950 takes 8- and 16-byte global accesses at every address a run of elements can
// have, so a row of odd length or an odd offset needs no scalar path: only the run that
// crosses the end of a row goes element by element.
#pragma once

#include "common.hpp"

namespace gconv {

// The dwords of a run, aligned as a 16-bit element is.
template <int DW> struct RunWords;
template <> struct RunWords<1> { typedef uint32_t type __attribute__((aligned(2))); };
template <> struct RunWords<2> { typedef uint32_t type __attribute__((ext_vector_type(2), aligned(2))); };
template <> struct RunWords<4> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2))); };
template <typename T> struct RunBits { typedef uint16_t type; };
template <> struct RunBits<float> { typedef uint32_t type; };
template <typename T, int N> struct Run { T v[N]; };
template <typename T, int N> using RunVec = typename RunWords<N * (int)sizeof(T) / 4>::type;

// N elements at src (N * sizeof(T) is 4, 8 or 16 bytes), as they are stored, of which the
// first `valid` exist; the others read as zero.  As words: where the two paths meet, the
// elements of a Run would stay in a register each.
template <typename T, int N>
__device__ __forceinline__ RunVec<T, N> load_words(const T *src, int valid)
{
    constexpr int PW = 4 / sizeof(T), NW = N / PW;
    if (valid >= N) return *reinterpret_cast<const RunVec<T, N> *>(src);
    uint32_t w[NW] = {};
    if (valid > 0) {     // every element from an address that exists
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const uint32_t x = reinterpret_cast<const typename RunBits<T>::type *>(src)[e < valid ? e : valid - 1];
            w[e / PW] |= e < valid ? x << (32 / PW * (e % PW)) : 0;
        }
    }
    return __builtin_bit_cast(RunVec<T, N>, w);
}

template <typename T, int N>
__device__ __forceinline__ Run<T, N> load_raw(const T *src, int valid)
{
    return __builtin_bit_cast(Run<T, N>, load_words<T, N>(src, valid));
}

template <typename T, int N>
__device__ __forceinline__ void load_run(const T *src, int valid, float (&f)[N])
{
    const Run<T, N> r = load_raw<T, N>(src, valid);
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = to_f32(r.v[e]);
}

// The first `valid` of N elements to dst.
template <typename T, int N>
__device__ __forceinline__ void store_raw(T *dst, int valid, const Run<T, N> &r)
{
    if (valid >= N) {
        *reinterpret_cast<RunVec<T, N> *>(dst) = __builtin_bit_cast(RunVec<T, N>, r);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e < valid) dst[e] = r.v[e];
    }
}

template <typename T, int N>
__device__ __forceinline__ void store_run(T *dst, int valid, const float (&f)[N])
{
    Run<T, N> r;
#pragma unroll
    for (int e = 0; e < N; ++e) r.v[e] = from_f32<T>(f[e]);
    store_raw<T, N>(dst, valid, r);
}

}  // namespace gconv
