// plain_common.h -- element types, row access and reductions shared by the
// plaintext-side kernels (include/ckks_plain.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "../../../include/ckks_plain.h"

namespace ckks_plain {

typedef __bf16 bf16;
typedef _Float16 f16;

__device__ __forceinline__ float to_f32(bf16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(f16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(float v) { return v; }
// to nearest, ties to even
template <typename T> __device__ __forceinline__ T from_f32(float v) { return (T)v; }

template <typename T> constexpr int VEC = 16 / sizeof(T);  // elements of a 16-byte access
template <typename T> struct VecOf { typedef T type __attribute__((ext_vector_type(16 / sizeof(T)))); };

// A row of `cols` elements over NT threads, E elements a thread.  VECTOR: 16-byte pieces dealt out
// in turn (rows have to start at multiples of 16 bytes); else single elements in turn.  Elements
// past the end read as 0 and are not written.
template <typename T, int NT, int E, bool VECTOR> struct Row {
    static constexpr int V = VECTOR ? VEC<T> : 1;
    static_assert(E % V == 0, "whole pieces");
    // column of this thread's element i
    static __device__ __forceinline__ int col(int i, int t) { return ((i / V) * NT + t) * V + i % V; }
    static __device__ __forceinline__ void load(const T *__restrict__ p, int cols, int t, float (&v)[E]) {
        if constexpr (VECTOR) {
#pragma unroll
            for (int i = 0; i < E; i += V) {
                const int c = col(i, t);
                if (c + V <= cols) {
                    const typename VecOf<T>::type w = *(const typename VecOf<T>::type *)(p + c);
#pragma unroll
                    for (int j = 0; j < V; j++) v[i + j] = to_f32(w[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < V; j++) v[i + j] = c + j < cols ? to_f32(p[c + j]) : 0.0f;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; i++) v[i] = col(i, t) < cols ? to_f32(p[col(i, t)]) : 0.0f;
        }
    }
    static __device__ __forceinline__ void store(T *__restrict__ p, int cols, int t, const float (&v)[E]) {
        if constexpr (VECTOR) {
#pragma unroll
            for (int i = 0; i < E; i += V) {
                const int c = col(i, t);
                if (c + V <= cols) {
                    typename VecOf<T>::type w;
#pragma unroll
                    for (int j = 0; j < V; j++) w[j] = from_f32<T>(v[i + j]);
                    *(typename VecOf<T>::type *)(p + c) = w;
                } else {
#pragma unroll
                    for (int j = 0; j < V; j++)
                        if (c + j < cols) p[c + j] = from_f32<T>(v[i + j]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; i++)
                if (col(i, t) < cols) p[col(i, t)] = from_f32<T>(v[i]);
        }
    }
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
    return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int m = 32; m; m >>= 1) {
        const uint32_t o = __shfl_xor(v, m);
        v = v > o ? v : o;
    }
    return v;
}

// Sum / largest over the NT threads of a row; every thread gets it.  `buf` holds a slot for each
// wave; with NT > 64 the caller gives reductions in a row different ones (two in turn: a thread
// that writes the first again has passed the second's barrier, so all have read the first).
template <int NT> __device__ __forceinline__ float row_sum(float v, float *buf) {
    v = wave_sum(v);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int w = 0; w < NT / 64; w++) v += buf[w];
    }
    return v;
}
template <int NT> __device__ __forceinline__ uint32_t row_max(uint32_t v, float *buf) {
    v = wave_max(v);
    if constexpr (NT > 64) {
        uint32_t *b = (uint32_t *)buf;
        if ((threadIdx.x & 63) == 0) b[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int w = 0; w < NT / 64; w++) v = v > b[w] ? v : b[w];
    }
    return v;
}

// The row's 8-bit form (ckks_plain_quantize_rows): scale from the largest |v| bit pattern (as
// unsigned numbers those order like the magnitudes, infinities and NaN above all), quotients in
// 32 bits.  The division by the scale is a true one: a reciprocal would move ties.
__device__ __forceinline__ float i8_scale(uint32_t max_bits) {
    return max_bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(max_bits) / 127.0f;
}
__device__ __forceinline__ int i8_of(float v, float s) {
    if (!(s > 0.0f)) return 0;  // a row of zeros, or not finite
    return (int)fminf(fmaxf(rintf(v / s), -127.0f), 127.0f);
}
template <typename R, int E>
__device__ __forceinline__ void store_i8(int8_t *__restrict__ q, int padded, int t, const float (&v)[E], float s) {
    constexpr int V = R::V;
#pragma unroll
    for (int i = 0; i < E; i += V) {
        const int c = R::col(i, t);
        if (c >= padded) continue;  // padded is a multiple of V: v is 0 from the last column on
        if constexpr (V == 1) {
            q[c] = (int8_t)i8_of(v[i], s);
        } else {
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                uint32_t w = 0;
#pragma unroll
                for (int b = 0; b < 4; b++) w |= (uint32_t)(uint8_t)i8_of(v[i + j + b], s) << (8 * b);
                *(uint32_t *)(q + c + j) = w;
            }
        }
    }
}

// Compile-time numbers and flags as arguments.
template <int N> struct Int { static constexpr int value = N; };
template <bool B> struct Flag { static constexpr bool value = B; };
// f(Int<0>), ..., f(Int<N - 1>): a loop whose counter is a constant in its body, also where the
// body is too long for the compiler to unroll a loop early enough to keep arrays in registers.
template <typename F, int... I>
__device__ __forceinline__ void for_all(F f, std::integer_sequence<int, I...>) { (f(Int<I>{}), ...); }
template <int N, typename F> __device__ __forceinline__ void for_all(F f) {
    for_all(f, std::make_integer_sequence<int, N>{});
}

// ------------------------------------------------------------------ host side

inline size_t type_size(int type) { return type == CKKS_PLAIN_F32 ? 4 : 2; }
inline bool type_ok(int type) { return type >= CKKS_PLAIN_BF16 && type <= CKKS_PLAIN_F32; }
inline bool at(const void *p, size_t align) { return ((uintptr_t)p & (align - 1)) == 0; }
inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
inline size_t span(int64_t rows, int64_t stride, int64_t cols, size_t size) {
    return rows ? ((size_t)(rows - 1) * stride + cols) * size : 0;
}
inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && na && nb && x < y + nb && y < x + na;
}
// a matrix argument: CKKS_OK or the error
inline int check_matrix(const void *p, int64_t stride, int64_t cols, size_t size) {
    if (!p || stride < cols) return CKKS_EINVAL;
    return at(p, size) ? CKKS_OK : CKKS_EALIGN;
}
inline int launched() { return hipGetLastError() == hipSuccess ? CKKS_OK : CKKS_EHIP; }

}  // namespace ckks_plain
