// sample.hip -- one token for each row of logits (include/ckks_plain.h).
#include "plain_common.h"

namespace ckks_plain {

// Order of tokens: the logit as an unsigned number of the same order, then the complement of the
// index, in one 64-bit number; 0 stands for a token that is not possible.
__device__ __forceinline__ uint32_t order_bits(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);  // -0 orders as 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_of(float z, uint32_t index) {
    return z > -INFINITY ? (uint64_t)order_bits(z) << 32 | (uint32_t)~index : 0;
}
__device__ __forceinline__ float logit_of(uint64_t order) {
    const uint32_t k = (uint32_t)(order >> 32);
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint32_t index_of(uint64_t order) { return ~(uint32_t)order; }

struct SampleArgs {
    const void *logits;
    const float *gumbel, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    const uint8_t *allowed;
    int64_t logits_stride, gumbel_stride, allowed_stride;
    int vocab, mass_bits;
    int64_t *token;
    float *logprob;
};

constexpr int NT = 1024, BINS = 2048, LIST = 4096;
constexpr uint64_t NONE = ~(uint64_t)0;

// Reductions over the workgroup's 16 waves; the same tree on every run.
template <typename V, typename F> __device__ __forceinline__ V block_reduce(V v, V *sh, F f) {
#pragma unroll
    for (int m = 32; m; m >>= 1) v = f(v, __shfl_xor(v, m));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = sh[threadIdx.x & 15];
#pragma unroll
    for (int m = 8; m; m >>= 1) v = f(v, __shfl_xor(v, m));
    return v;
}
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t smaller(uint64_t a, uint64_t b) { return a < b ? a : b; }
// Sum over the threads in front of this one; `total` over all.
__device__ __forceinline__ uint64_t block_before(uint64_t v, uint64_t *sh, uint64_t &total) {
    const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
    uint64_t s = v;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint64_t o = __shfl_up(s, m);
        if (l >= m) s += o;
    }
    __syncthreads();
    if (l == 63) sh[w] = s;
    __syncthreads();
    uint64_t before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < NT / 64; i++) {
        const uint64_t x = sh[i];
        before += i < w ? x : 0;
        total += x;
    }
    return before + s - v;
}

// One workgroup a row.  A row is read once for its largest logit and its mass (the sum of
// e = exp((z - max) / temperature)); a filter then needs the last token that stays:
//  - Bounds.  A token under the k-th largest of the threads' own maxima is not among the first k.
//    One with e < (1 - p) mass / count is not in the nucleus: all such together have less than
//    (1 - p) of the mass, so what comes before any of them has p of it.
//  - What passes the bound usually fits the list in LDS, where it is sorted: everything else is
//    decided there, without reading the row again.
//  - Where it does not fit, the last token is located by counts or masses in bins of equal width
//    over the logits, and the one bin it falls into is listed and sorted (a bin that does not
//    fit either is divided again, by the tokens' order).
// Masses are whole multiples of 2^-mass_bits where they are added by atomics or compared, so
// results do not depend on the order of anything.
template <typename T> struct Sampler {
    static constexpr int N = 16 / sizeof(T);  // logits of a vector
    typedef T Vec __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
    typedef uint8_t Mask __attribute__((ext_vector_type(16 / sizeof(T)), aligned(1)));

    const SampleArgs &a;
    const T *z;
    const uint8_t *ok;
    const float *gumbel;
    float t, c, top;  // temperature, log2(e) / temperature, the largest logit

    // f(first index, logits) for this thread's vectors; a token that is not possible has -infinity.
    // Rows need no alignment beyond their elements'.
    template <int U = 4, typename F> __device__ __forceinline__ void pass(F f) const {  // U vectors in flight
        const int whole = a.vocab / N, rest = a.vocab % N;
        for (int v = threadIdx.x; v < whole; v += U * NT) {
            Vec r[U];
            Mask m[U];
#pragma unroll
            for (int j = 0; j < U; j++) {
                const int64_t i = (int64_t)(v + j * NT < whole ? v + j * NT : v) * N;
                r[j] = *(const Vec *)(z + i);
                if (ok) m[j] = *(const Mask *)(ok + i);
            }
#pragma unroll
            for (int j = 0; j < U; j++) {
                if (v + j * NT >= whole) break;
                float x[N];
#pragma unroll
                for (int k = 0; k < N; k++) {
                    x[k] = fmaxf(to_f32(r[j][k]), -INFINITY);  // NaN: -infinity
                    if (ok) x[k] = m[j][k] ? x[k] : -INFINITY;
                }
                f((v + j * NT) * N, x);
            }
        }
        if (rest && threadIdx.x == whole % NT) {
            float x[N];
#pragma unroll
            for (int k = 0; k < N; k++) {
                const bool there = k < rest && (!ok || ok[whole * N + k]);
                x[k] = there ? fmaxf(to_f32(z[whole * N + k]), -INFINITY) : -INFINITY;
            }
            f(whole * N, x);
        }
    }
    // e in 32 bits; the quotient as a product, which moves it by about 2^-23 of the exponent
    __device__ __forceinline__ float weight(float v, float from) const {
        return __builtin_amdgcn_exp2f(fminf((v - from) * c, 0.0f));  // infinity - infinity: 1
    }
    __device__ __forceinline__ uint64_t fixed(float e) const {  // e in [0, 1], cut to a multiple
        const uint32_t b = __float_as_uint(e);
        const int x = (int)(b >> 23) - 150 + a.mass_bits;
        const uint64_t m = (b & 0x7fffff) | 0x800000;
        return b < 0x800000 || x <= -24 ? 0 : x >= 0 ? m << x : m >> -x;
    }
    __device__ __forceinline__ uint64_t mass(float v) const { return fixed(weight(v, top)); }
    // the distance to the largest logit, as defined: each step rounded to 32 bits
    __device__ __forceinline__ float part(float v) const { return v == top ? 0.0f : (v - top) / t; }
    // as `order_of`, of the score
    __device__ __forceinline__ uint64_t score(float v, uint32_t i) const {
        return (uint64_t)order_bits(part(v) + gumbel[i]) << 32 | (uint32_t)~i;
    }
};

struct SampleShared {
    uint64_t sh[16];
    float shf[16];
    uint64_t pick[4];
    uint32_t n;
    union {
        uint64_t list[LIST];
        uint64_t bins[BINS];
    };
};

// list[0..n) in falling order, for the whole workgroup; n <= LIST.
__device__ __forceinline__ void sort_list(uint64_t *list, int n) {
    int size = 2;
    while (size < n) size *= 2;
    __syncthreads();
    for (int i = n + threadIdx.x; i < size; i += NT) list[i] = 0;
    for (int run = 2; run <= size; run *= 2)
        for (int gap = run / 2; gap; gap /= 2) {
            __syncthreads();
            for (int i = threadIdx.x; i < size / 2; i += NT) {
                const int lo = 2 * i - (i & (gap - 1)), hi = lo + gap;
                const uint64_t x = list[lo], y = list[hi];
                if ((x < y) == ((lo & run) == 0)) list[lo] = y, list[hi] = x;
            }
        }
    __syncthreads();
}

// Puts the tokens for which f(logit, order) holds on the list, at most LIST; returns how many
// there are (more than LIST: at least that many).
template <typename S, typename F> __device__ __forceinline__ uint32_t gather(const S &s, SampleShared &m, F f) {
    __syncthreads();
    if (threadIdx.x == 0) m.n = 0;
    __syncthreads();
    s.pass([&](int first, const float (&x)[S::N]) {
#pragma unroll
        for (int k = 0; k < S::N; k++) {
            const uint64_t o = order_of(x[k], first + k);
            if (o && f(x[k], o) && *(volatile uint32_t *)&m.n <= LIST) {
                const uint32_t at = atomicAdd(&m.n, 1u);
                if (at < LIST) m.list[at] = o;
            }
        }
    });
    __syncthreads();
    return m.n;
}

// The order of the last token that stays, among those from `from` on with logits >= low: by count
// the want-th, by mass the last before which there is less than `want`; 0 if there are not so many.
// `above`: the mass of the tokens up to it (by count).
template <bool MASS, typename S>
__device__ __forceinline__ uint64_t locate(const S &s, SampleShared &m, uint64_t want, uint64_t from, float low, uint64_t &above) {
    const float width = (float)BINS / (s.top - fmaxf(low, s.top - 64.0f / s.c));
    uint64_t a = 0, b = 0, before = 0;  // the range of orders that is divided, and what comes before it
    for (int level = 0;; level++) {
        const int shift = level && b - a >= BINS ? 53 - __clzll(b - a) : 0;  // (b - a) >> shift < BINS
        auto bin_of = [&](float x, uint64_t o) {
            return level ? (int)((b - o) >> shift) : (int)fminf(fmaxf((s.top - x) * width, 0.0f), BINS - 1.0f);
        };
        auto inside = [&](float x, uint64_t o) { return o >= from && x >= low && (!level || (o >= a && o <= b)); };
        __syncthreads();
        for (int i = threadIdx.x; i < BINS; i += NT) m.bins[i] = 0;
        if (threadIdx.x == 0) m.pick[0] = BINS;
        __syncthreads();
        s.template pass<1>([&](int first, const float (&x)[S::N]) {
#pragma unroll
            for (int k = 0; k < S::N; k++) {
                const uint64_t o = order_of(x[k], first + k);
                if (o && inside(x[k], o))
                    atomicAdd((unsigned long long *)&m.bins[bin_of(x[k], o)],
                              (unsigned long long)(MASS ? s.mass(x[k]) : 1));
            }
        });
        __syncthreads();
        const uint64_t v0 = m.bins[2 * threadIdx.x], v1 = m.bins[2 * threadIdx.x + 1];
        uint64_t total;
        const uint64_t p = before + block_before(v0 + v1, m.sh, total);
        if (p < want && want <= p + v0 + v1) {
            const bool second = want > p + v0;
            m.pick[0] = 2 * threadIdx.x + second;
            m.pick[1] = p + (second ? v0 : 0);
        }
        __syncthreads();
        const int bin = (int)m.pick[0];
        if (bin == BINS) return 0;
        before = m.pick[1];
        const uint32_t n =
            gather(s, m, [&](float x, uint64_t o) { return inside(x, o) && bin_of(x, o) == bin; });
        if (n <= LIST) {
            sort_list(m.list, n);
            // by mass: four neighbours a thread
            uint64_t o[4], w[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint32_t at = 4 * threadIdx.x + i;
                o[i] = at < n ? m.list[at] : 0;
                w[i] = !o[i] ? 0 : MASS ? s.mass(logit_of(o[i])) : 1;
                sum += w[i];
            }
            uint64_t q = before + block_before(sum, m.sh, total);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if (q < want && want <= q + w[i]) m.pick[2] = o[i];
                q += w[i];
            }
            __syncthreads();
            const uint64_t last = m.pick[2];
            if (!MASS) {  // the mass down to it
                uint64_t sum = 0;
                s.template pass<1>([&](int first, const float (&x)[S::N]) {
#pragma unroll
                    for (int k = 0; k < S::N; k++)
                        if (order_of(x[k], first + k) >= last) sum += s.mass(x[k]);
                });
                above = block_reduce(sum, m.sh, [](uint64_t x, uint64_t y) { return x + y; });
            }
            return last;
        }
        // divide the bin by the orders that are in it
        uint64_t lowest = NONE, highest = 0;
        s.template pass<1>([&](int first, const float (&x)[S::N]) {
#pragma unroll
            for (int k = 0; k < S::N; k++) {
                const uint64_t o = order_of(x[k], first + k);
                if (!o || !inside(x[k], o) || bin_of(x[k], o) != bin) continue;
                lowest = smaller(lowest, o), highest = larger(highest, o);
            }
        });
        const uint64_t a1 = block_reduce(lowest, m.sh, smaller), b1 = block_reduce(highest, m.sh, larger);
        a = a1, b = b1;
    }
}

template <typename T> __global__ __launch_bounds__(NT) void k_sample(SampleArgs a) {
    typedef Sampler<T> S;
    constexpr int N = S::N;
    __shared__ SampleShared m;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const float temp = a.temperature[row];
    const bool greedy = !(temp > 0);
    const int k = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.0f, min_p = a.min_p ? a.min_p[row] : 0.0f;
    S s{a, (const T *)a.logits + row * a.logits_stride, a.allowed ? a.allowed + row * a.allowed_stride : nullptr,
        a.gumbel + row * a.gumbel_stride, greedy ? 1.0f : temp, 0, 0};
    // under 2^-120 the exponents of finite logits stay, and -infinity times it stays -infinity
    s.c = fmaxf(1.44269504f / s.t, 0x1p-120f);
    // the thread's largest logit, where it first occurs, and its mass from there
    float mine = -INFINITY, sum = 0;
    uint32_t where = 0xffffffffu;
    s.pass([&](int first, const float (&x)[N]) {
        float v = x[0];
#pragma unroll
        for (int i = 1; i < N; i++) v = fmaxf(v, x[i]);
        if (v > mine) sum *= s.weight(mine, v), mine = v, where = first;
        if (mine > -INFINITY) {
#pragma unroll
            for (int i = 0; i < N; i++) sum += s.weight(x[i], mine);
        }
    });
    const uint64_t best = block_reduce(order_of(mine, where), m.sh, larger);
    if (!best) {
        if (tid == 0) a.token[row] = -1, a.logprob[row] = -INFINITY;
        return;
    }
    s.top = logit_of(best);
    sum = block_reduce(mine > -INFINITY ? sum * s.weight(mine, s.top) : 0.0f, m.shf, [](float x, float y) { return x + y; });
    auto answer = [&](uint32_t token, float v) {
        a.token[row] = token;
        a.logprob[row] = s.part(v) - logf(sum);
    };
    if (greedy || k == 1 || p <= 0 || min_p > 1) {  // the first alone: it is in the vector at index_of(best)
        if (tid == 0) {
            uint32_t i = index_of(best);
            while (!(to_f32(s.z[i]) == s.top && (!s.ok || s.ok[i]))) i++;
            answer(i, s.top);
        }
        return;
    }
    const bool by_count = k > 0 && k < a.vocab, by_mass = p < 1;
    uint64_t last = 1, win = 0;  // the order of the last that stays; the best score
    if (by_count || by_mass) {
        float low = -INFINITY;
        if (by_count) {
            // the k-th largest of the threads' maxima, or a little less: by bins of equal width
            const uint64_t own = order_of(mine, 0);
            const float least = logit_of(block_reduce(own ? own : NONE, m.sh, smaller));
            const float width = 1024.0f / (s.top - least);
            const int bin = mine > -INFINITY ? (int)fminf(fmaxf((s.top - mine) * width, 0.0f), 1023.0f) : 1024;
            m.bins[tid] = 0;
            if (tid == 0) m.pick[0] = 1024;
            __syncthreads();
            if (bin < 1024) atomicAdd((unsigned long long *)&m.bins[bin], 1ull);
            __syncthreads();
            uint64_t total;
            const uint64_t v = m.bins[tid], before = block_before(v, m.sh, total);
            if (before < (uint64_t)k && (uint64_t)k <= before + v) m.pick[0] = tid;
            __syncthreads();
            const int at = (int)m.pick[0];
            if (at < 1024) low = logit_of(block_reduce(bin <= at ? own : NONE, m.sh, smaller));
        } else {
            low = s.top + (__log2f((1.0f - p) * sum / (float)a.vocab) - 0.0625f) / s.c;
        }
        // the list is tried unless nearly every thread has something for it (then it has thousands)
        const int passing = __syncthreads_count(mine > -INFINITY && mine >= low);
        uint32_t n = LIST + 1;
        if (a.vocab <= LIST || passing <= 1000) n = gather(s, m, [&](float x, uint64_t) { return x >= low; });
        const double scale = exp2((double)a.mass_bits);
        auto under = [&](double whole) { return larger(1, (uint64_t)ceil((double)p * whole)); };
        if (n <= LIST) {
            sort_list(m.list, n);
            const uint32_t stay = by_count && (uint32_t)k < n ? k : n;
            uint64_t o[4], w[4], own = 0, total;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint32_t at = 4 * tid + i;
                o[i] = at < stay ? m.list[at] : 0;
                w[i] = o[i] ? s.mass(logit_of(o[i])) : 0;
                own += w[i];
            }
            uint64_t q = block_before(own, m.sh, total);
            const uint64_t want = by_mass ? under(by_count ? (double)total : (double)sum * scale) : NONE;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float v = logit_of(o[i]);
                if (o[i] && q < want && !(min_p > 0 && s.weight(v, s.top) < min_p)) win = larger(win, s.score(v, index_of(o[i])));
                q += w[i];
            }
            win = block_reduce(win, m.sh, larger);
            if (tid == 0) answer(index_of(win), to_f32(s.z[index_of(win)]));
            return;
        }
        uint64_t whole = (uint64_t)((double)sum * scale), unused;
        if (by_count) last = larger(1, locate<false>(s, m, k, 1, low, whole));
        if (by_mass) last = larger(last, locate<true>(s, m, under((double)whole), last, low, unused));
        if (last == 1) last = order_of(low, 0xffffffffu);  // all that pass the bound
        last = larger(last, 1);
    }
    s.pass([&](int first, const float (&x)[N]) {
#pragma unroll
        for (int i = 0; i < N; i++) {
            const uint64_t o = order_of(x[i], first + i);
            if (o >= last && !(min_p > 0 && s.weight(x[i], s.top) < min_p)) win = larger(win, s.score(x[i], first + i));
        }
    });
    win = block_reduce(win, m.sh, larger);
    if (tid == 0) answer(index_of(win), to_f32(s.z[index_of(win)]));
}

}  // namespace ckks_plain

using namespace ckks_plain;

extern "C" int ckks_plain_sample_workspace_size(int64_t rows, int64_t vocab, size_t *bytes) {
    if (!bytes || rows < 0 || rows >= (int64_t)1 << 31 || vocab < 1 || vocab > 1 << 24) return CKKS_EINVAL;
    *bytes = 0;
    return CKKS_OK;
}

extern "C" int ckks_plain_sample(int type, const void *logits, int64_t logits_stride, const float *gumbel,
                                 int64_t gumbel_stride, const float *temperature, const int32_t *top_k,
                                 const float *top_p, const float *min_p, const uint8_t *allowed,
                                 int64_t allowed_stride, int64_t rows, int64_t vocab, int64_t *token, float *logprob,
                                 void *ws, size_t ws_bytes, void *stream) {
    size_t need;
    if (int e = ckks_plain_sample_workspace_size(rows, vocab, &need)) return e;
    if (!type_ok(type)) return CKKS_EINVAL;
    if (rows == 0) return CKKS_OK;
    const size_t z = type_size(type);
    if (int e = check_matrix(logits, logits_stride, vocab, z)) return e;
    if (int e = check_matrix(gumbel, gumbel_stride, vocab, 4)) return e;
    if (allowed && allowed_stride < vocab) return CKKS_EINVAL;
    if (!temperature || !token || !logprob) return CKKS_EINVAL;
    if (!at(temperature, 4) || !at(top_k, 4) || !at(top_p, 4) || !at(min_p, 4) || !at(token, 8) || !at(logprob, 4))
        return CKKS_EALIGN;
    struct { const void *p; size_t n; } in[7] = {
        {logits, span(rows, logits_stride, vocab, z)}, {gumbel, span(rows, gumbel_stride, vocab, 4)},
        {temperature, (size_t)rows * 4}, {top_k, (size_t)rows * 4}, {top_p, (size_t)rows * 4}, {min_p, (size_t)rows * 4},
        {allowed, span(rows, allowed_stride, vocab, 1)}};
    for (auto &r : in)
        if (overlap(token, rows * 8, r.p, r.n) || overlap(logprob, rows * 4, r.p, r.n)) return CKKS_EINVAL;
    if (overlap(token, rows * 8, logprob, rows * 4)) return CKKS_EINVAL;
    if (need && (!ws || ws_bytes < need)) return CKKS_EWORKSPACE;
    int bits = 0;
    while (((int64_t)1 << bits) < vocab) bits++;
    const SampleArgs a{logits, gumbel, temperature, top_p, min_p, top_k, allowed, logits_stride, gumbel_stride,
                       allowed_stride, (int)vocab, 62 - bits, token, logprob};
    auto go = [&](auto ty) {
        k_sample<decltype(ty)><<<dim3((uint32_t)rows), NT, 0, (hipStream_t)stream>>>(a);
        return launched();
    };
    return type == CKKS_PLAIN_BF16 ? go(bf16{}) : type == CKKS_PLAIN_F16 ? go(f16{}) : go(0.0f);
}
