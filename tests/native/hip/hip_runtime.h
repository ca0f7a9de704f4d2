// Device code of one workgroup on the host, for checks without a GPU: threads are
// fibers, run in turn until all wait at a barrier; moves between lanes meet at a
// barrier of their wave.  What the plaintext-side kernels use, no more.
#pragma once
#include <ucontext.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <vector>

#define __device__
#define __global__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __shared__ static

struct Index { unsigned x, y, z; };
static Index threadIdx, blockIdx;

namespace host {
constexpr int LANES = 64;
struct Barrier {
    int size, here, turn;
};
static std::vector<ucontext_t> fibers;
static std::vector<std::vector<char>> stacks;
static std::vector<char> ended;
static std::vector<Barrier> waves;
static std::vector<uint32_t> posted;
static Barrier all;
static ucontext_t scheduler;
static std::function<void()> body;

inline void wait(Barrier &b) {
    const int turn = b.turn;
    if (++b.here == b.size) {
        b.here = 0, b.turn++;
        return;
    }
    while (b.turn == turn) swapcontext(&fibers[threadIdx.x], &scheduler);
}
inline void wave_wait() { wait(waves[threadIdx.x / LANES]); }
// v of every lane of this wave, then f(lane's value reader)
template <typename F> auto exchange(uint32_t v, F f) {
    uint32_t *wave = &posted[threadIdx.x / LANES * LANES];
    wave[threadIdx.x % LANES] = v;
    wave_wait();
    auto r = f(wave);
    wave_wait();
    return r;
}
inline void entry() {
    body();
    ended[threadIdx.x] = 1;
    for (;;) swapcontext(&fibers[threadIdx.x], &scheduler);
}
// Runs f as `threads` threads that all pass the same barriers; false if they have not ended after `turns` turns
// of all of them.
inline bool run(int threads, long turns, std::function<void()> f) {
    body = f;
    fibers.assign(threads, ucontext_t());
    stacks.resize(threads);
    ended.assign(threads, 0);
    posted.assign(threads, 0);
    all = {threads, 0, 0};
    waves.assign(threads / LANES, Barrier{LANES, 0, 0});
    for (int t = 0; t < threads; t++) {
        stacks[t].resize(1 << 16);
        getcontext(&fibers[t]);
        fibers[t].uc_stack.ss_sp = stacks[t].data();
        fibers[t].uc_stack.ss_size = stacks[t].size();
        fibers[t].uc_link = &scheduler;
        makecontext(&fibers[t], entry, 0);
    }
    for (long n = 0; n < turns; n++) {
        int left = 0;
        for (int q = 0; q < threads; q++) {
            const int t = n % 2 ? threads - 1 - q : q;  // both orders
            if (ended[t]) continue;
            left++;
            threadIdx.x = t;
            swapcontext(&scheduler, &fibers[t]);
        }
        if (!left) return true;
    }
    return false;
}
inline uint32_t update_dpp(uint32_t none, uint32_t v, int ctrl, int rows) {
    const int l = threadIdx.x % LANES;
    return exchange(v, [&](const uint32_t *wave) {
        if (!(rows >> (l / 16) & 1)) return none;
        if (ctrl >= 0x111 && ctrl <= 0x11f) return l % 16 >= ctrl - 0x110 ? wave[l - (ctrl - 0x110)] : none;
        if (ctrl == 0x142) return l >= 16 ? wave[(l & ~15) - 1] : none;
        if (ctrl == 0x143) return l >= 32 ? wave[31] : none;
        abort();
    });
}
inline uint64_t ballot(bool v) {
    return exchange(v, [](const uint32_t *wave) {
        uint64_t r = 0;
        for (int i = 0; i < LANES; i++) r |= (uint64_t)(wave[i] != 0) << i;
        return r;
    });
}
inline uint32_t bits_under_lane(uint32_t mask, uint32_t base, int first) {
    const int l = threadIdx.x % LANES - first;
    return base + __builtin_popcount(l <= 0 ? 0 : l >= 32 ? mask : mask & ((1u << l) - 1));
}
}  // namespace host

inline void __syncthreads() { host::wait(host::all); }
inline int __syncthreads_count(int v) {
    static int n;
    __syncthreads();
    if (threadIdx.x == 0) n = 0;
    __syncthreads();
    n += v != 0;
    __syncthreads();
    return n;
}
template <typename T> inline T atomicAdd(T *p, T v) { const T o = *p; *p = o + v; return o; }
template <typename T> inline T atomicMax(T *p, T v) { const T o = *p; *p = o > v ? o : v; return o; }
inline uint32_t __float_as_uint(float f) { uint32_t u; memcpy(&u, &f, 4); return u; }
inline float __uint_as_float(uint32_t u) { float f; memcpy(&f, &u, 4); return f; }
inline int __clzll(unsigned long long v) { return v ? __builtin_clzll(v) : 64; }
inline int __popc(uint32_t v) { return __builtin_popcount(v); }
inline int __popcll(uint64_t v) { return __builtin_popcountll(v); }
inline float log2_host(float v) { return log2f(v); }
#define __log2f log2_host
#define __ffsll __builtin_ffsll
#define __ballot(v) host::ballot(v)
#define __builtin_amdgcn_update_dpp(none, v, ctrl, rows, banks, bound) \
    ((int)host::update_dpp((uint32_t)(none), (uint32_t)(v), ctrl, rows))
#define __builtin_amdgcn_readlane(v, l) ((int)host::exchange((uint32_t)(v), [&](const uint32_t *wave) { return wave[(l) & 63]; }))
#define __builtin_amdgcn_readfirstlane(v) (v)
#define __builtin_amdgcn_exp2f(v) exp2f(v)
#define __builtin_amdgcn_mbcnt_lo(mask, base) host::bits_under_lane(mask, base, 0)
#define __builtin_amdgcn_mbcnt_hi(mask, base) host::bits_under_lane(mask, base, 32)
#define hipSuccess 0
inline int hipGetLastError() { return hipSuccess; }
