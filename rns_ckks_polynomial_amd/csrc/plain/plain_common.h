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

// 16 bytes of elements at any element's address (the unaligned access mode of this GPU: a load that
// straddles a cache line costs one line more, and the neighbouring lanes use it too).
template <typename T> constexpr int VEC = 16 / sizeof(T);
template <typename T> struct VecOf {
    typedef T type __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
};

// A row of `cols` elements over NT threads, E elements a thread in 16-byte pieces dealt out in turn.
// Elements past the end read as 0 and are not written.
template <typename T, int NT, int E> struct Row {
    static constexpr int V = VEC<T>;
    typedef typename VecOf<T>::type Vec;
    static_assert(E % V == 0, "whole pieces");
    // column of this thread's element i
    static __device__ __forceinline__ int col(int i, int t) { return ((i / V) * NT + t) * V + i % V; }
    struct Raw {
        Vec v[E / V];
    };
    static __device__ __forceinline__ void fetch(const T *__restrict__ p, int cols, int t, Raw &r) {
#pragma unroll
        for (int i = 0; i < E; i += V) {
            const int c = col(i, t);
            if (c + V <= cols) {
                r.v[i / V] = *(const Vec *)(p + c);
            } else {
#pragma unroll
                for (int j = 0; j < V; j++) r.v[i / V][j] = c + j < cols ? p[c + j] : (T)0.0f;
            }
        }
    }
    static __device__ __forceinline__ void widen(const Raw &r, float (&v)[E]) {
#pragma unroll
        for (int i = 0; i < E; i++) v[i] = to_f32(r.v[i / V][i % V]);
    }
    static __device__ __forceinline__ void load(const T *__restrict__ p, int cols, int t, float (&v)[E]) {
        Raw r;
        fetch(p, cols, t, r);
        widen(r, v);
    }
    static __device__ __forceinline__ void store(T *__restrict__ p, int cols, int t, const float (&v)[E]) {
#pragma unroll
        for (int i = 0; i < E; i += V) {
            const int c = col(i, t);
            if (c + V <= cols) {
                Vec w;
#pragma unroll
                for (int j = 0; j < V; j++) w[j] = from_f32<T>(v[i + j]);
                *(Vec *)(p + c) = w;
            } else {
#pragma unroll
                for (int j = 0; j < V; j++)
                    if (c + j < cols) p[c + j] = from_f32<T>(v[i + j]);
            }
        }
    }
};

// The neighbour's value that a move between lanes brings (`none` where there is no neighbour).
template <int CTRL, int ROWS> __device__ __forceinline__ uint32_t moved(uint32_t none, uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS> __device__ __forceinline__ float moved(float none, float v) {
    return __uint_as_float(moved<CTRL, ROWS>(__float_as_uint(none), __float_as_uint(v)));
}
template <int CTRL, int ROWS> __device__ __forceinline__ uint64_t moved(uint64_t none, uint64_t v) {
    return (uint64_t)moved<CTRL, ROWS>((uint32_t)(none >> 32), (uint32_t)(v >> 32)) << 32 |
           moved<CTRL, ROWS>((uint32_t)none, (uint32_t)v);
}
__device__ __forceinline__ uint32_t lane(uint32_t v, int l) { return (uint32_t)__builtin_amdgcn_readlane((int)v, l); }
__device__ __forceinline__ float lane(float v, int l) { return __uint_as_float(lane(__float_as_uint(v), l)); }
__device__ __forceinline__ uint64_t lane(uint64_t v, int l) {
    return (uint64_t)lane((uint32_t)(v >> 32), l) << 32 | lane((uint32_t)v, l);
}
// Inclusive scans over rows of 16 lanes and over the wave, in a fixed order (moves within the
// register file: an exchange through LDS takes ten times as long).
template <typename V, typename F> __device__ __forceinline__ V scan16(V v, V none, F f) {
    v = f(moved<0x111, 0xf>(none, v), v);
    v = f(moved<0x112, 0xf>(none, v), v);
    v = f(moved<0x114, 0xf>(none, v), v);
    return f(moved<0x118, 0xf>(none, v), v);
}
template <typename V, typename F> __device__ __forceinline__ V scan64(V v, V none, F f) {
    v = scan16(v, none, f);
    v = f(moved<0x142, 0xa>(none, v), v);
    return f(moved<0x143, 0xc>(none, v), v);
}
struct Larger {
    template <typename V> __device__ __forceinline__ V operator()(V a, V b) const { return a > b ? a : b; }
};
struct Sum {
    template <typename V> __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};

// Sum / largest over the NT threads of a row; every thread gets it.  `buf` holds a slot for each
// wave; with NT > 64 the caller gives reductions in a row different ones (two in turn: a thread
// that writes the first again has passed the second's barrier, so all have read the first).
template <int NT, typename V, typename F> __device__ __forceinline__ V row_all(V v, V *buf, F f) {
    v = lane(scan64(v, V(0), f), 63);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
        __syncthreads();
        v = buf[0];
#pragma unroll
        for (int w = 1; w < NT / 64; w++) v = f(v, buf[w]);
    }
    return v;
}
template <int NT> __device__ __forceinline__ float row_sum(float v, float *buf) { return row_all<NT>(v, buf, Sum{}); }
// two sums behind one barrier
template <int NT> __device__ __forceinline__ void row_sums(float &v, float &w, float *buf_v, float *buf_w) {
    v = lane(scan64(v, 0.0f, Sum{}), 63);
    w = lane(scan64(w, 0.0f, Sum{}), 63);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) buf_v[threadIdx.x >> 6] = v, buf_w[threadIdx.x >> 6] = w;
        __syncthreads();
        v = buf_v[0], w = buf_w[0];
#pragma unroll
        for (int i = 1; i < NT / 64; i++) v += buf_v[i], w += buf_w[i];
    }
}
template <int NT> __device__ __forceinline__ uint32_t row_max(uint32_t v, float *buf) {
    return row_all<NT>(v, (uint32_t *)buf, Larger{});
}

// The row's 8-bit form (ckks_plain_quantize_rows): scale from the largest |v| bit pattern (as
// unsigned numbers those order like the magnitudes, infinities and NaN above all) times 1 / 127 in
// 32 bits, as a division by a constant is usually compiled.  The division by the scale is a true
// one: a reciprocal would move ties.
__device__ __forceinline__ float i8_scale(uint32_t max_bits) {
    return max_bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(max_bits) * (1.0f / 127.0f);
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
        typedef uint32_t Words __attribute__((ext_vector_type(V / 4)));
        Words w;
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            w[j / 4] = 0;
#pragma unroll
            for (int b = 0; b < 4; b++) w[j / 4] |= (uint32_t)(uint8_t)i8_of(v[i + j + b], s) << (8 * b);
        }
        *(Words *)(q + c) = w;
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
// A grid holds fewer than 2^32 threads: f(first row, rows) for each part of the rows, `threads` a row.
template <typename F> int in_parts(int64_t rows, int threads, F f) {
    const int64_t most = ((int64_t)1 << 31) / threads / 4 * 4;  // whole workgroups, also of four rows
    for (int64_t first = 0; first < rows; first += most)
        if (int e = f(first, rows - first < most ? rows - first : most)) return e;
    return CKKS_OK;
}
inline int launched() { return hipGetLastError() == hipSuccess ? CKKS_OK : CKKS_EHIP; }

}  // namespace ckks_plain
