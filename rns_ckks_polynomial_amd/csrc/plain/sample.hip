// sample.hip -- one token for each row of logits (include/ckks_plain.h).
#include <type_traits>

#include "plain_common.h"

namespace ckks_plain {

// A number of the order of a float.
__device__ __forceinline__ uint32_t order_bits(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);  // -0 orders as 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_order_bits(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }

struct SampleArgs {
    const void *logits;
    const float *gumbel, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    const uint8_t *allowed;
    int64_t logits_stride, gumbel_stride, allowed_stride;
    int vocab, index_bits;  // vocab <= 2^index_bits
    int64_t *token;
    float *logprob;
};

constexpr int NT = 1024, WAVES = NT / 64, BINS = 2048, LIST = 4096, HELD = LIST / NT;
constexpr int FINE = 8192, EACH = FINE / NT;  // counted bins, of a thread
// A bound on e is taken this much lower, in powers of two: the mass, the logarithm and the quotient are off by less
// than 2^-9 of one (2^14 additions a thread at most), and the list gets 4 % longer.
constexpr float SLACK = 0.0625f;

struct SampleShared {
    uint64_t slot[8][WAVES];
    uint64_t pick[3];
    uint32_t n, cut;
    union {
        uint64_t list[LIST];
        uint64_t bins[BINS];
        uint32_t counts[FINE];
    };
};

// One workgroup a row.  A row is read once for its largest logit and its mass (the sum of
// e = exp((z - max) / temperature)); a filter then needs the last token that stays:
//  - Bounds.  A token under the k-th largest of the threads' own maxima is not among the first k.
//    One with e < (1 - p) mass / count is not in the nucleus: all such together have less than
//    (1 - p) of the mass, so what comes before any of them has p of it.  One with e < min_p does
//    not stay.
//  - What passes the bound usually fits the list in LDS: everything else is decided there,
//    without reading the row again.
//  - A nucleus that does not fit is counted in bins of equal width over the logits.  A bin's mass
//    is its count times e of its middle, to half a bin's width; that names a few bins that may hold
//    the end of the nucleus.  The last read takes the tokens above them, adds up their exact mass
//    and lists those bins.
//  - Many tokens by count, or bins that overflow the list (runs of equal logits): the last token is
//    located by counts or masses in bins of the tokens' order, eleven bits a read.
// Masses that are added by atomics are whole multiples of a power of two and float sums go in a
// fixed order, so the result does not depend on the order of anything.
//
// 256 x 131072 bf16, top-p 0.95 of normal logits (deviation 2.5, a nucleus of 26000): 72 to 80 us for
// 290 MB from memory, three reads of the logits and the noise lines that hold a token of the nucleus;
// each read has a compute unit's vector instructions beside its loads (the waves wait in 55 % of their
// cycles).  The same rows without filters 47 us, the largest alone 16.  1 x 32768 f32, top-k 50 and
// top-p: 13 us, one read, then latency; 33 x 50021 f16, masked, min-p and top-k 1000: 21 us.  Few long
// rows leave most compute units idle: 16 x 262144 bf16 top-p 116 us.
template <typename T> struct Sampler {
    static constexpr int N = 16 / sizeof(T);  // logits of a vector
    typedef T Vec __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
    typedef uint8_t Mask __attribute__((ext_vector_type(16 / sizeof(T)), aligned(1)));
    typedef float Four __attribute__((ext_vector_type(4), aligned(4)));

    const SampleArgs &a;
    SampleShared &m;
    const T *z;
    const uint8_t *ok;
    const float *gumbel;
    int wave, slot;
    float t, c, top;   // temperature, log2(e) / temperature, the largest logit
    float sum, min_p;  // the mass
    float least;       // log2 of min_p, -infinity without

    // ---- the order of tokens: the logit as an unsigned number of the same order, without the bits
    // that its type never sets, then the complement of the index; 0: a token that is not possible
    static constexpr int UNSET = sizeof(T) == 4 ? 0 : std::is_same<T, f16>::value ? 13 : 16;
    __device__ __forceinline__ uint32_t indexes() const { return (1u << a.index_bits) - 1; }
    // the lowest and the highest order of a logit
    __device__ __forceinline__ uint64_t lowest(float v) const { return (uint64_t)(order_bits(v) >> UNSET) << a.index_bits; }
    __device__ __forceinline__ uint64_t highest(float v) const { return lowest(v) | indexes(); }
    __device__ __forceinline__ uint64_t order_of(float v, uint32_t i) const {
        return v > -INFINITY ? lowest(v) | (indexes() - i) : 0;
    }
    static __device__ __forceinline__ float of_key(uint32_t key) {
        const uint32_t k = key << UNSET;
        return of_order_bits(k & 0x80000000u ? k : k | ((1u << UNSET) - 1));
    }
    __device__ __forceinline__ float logit_of(uint64_t o) const { return of_key((uint32_t)(o >> a.index_bits)); }
    __device__ __forceinline__ uint32_t index_of(uint64_t o) const { return indexes() - ((uint32_t)o & indexes()); }

    // ---- the workgroup's reductions: one barrier each, in eight places in turn
    template <typename V, typename F> __device__ __forceinline__ V across(V v, V none, F f) {  // of each wave's v
        V *at = (V *)m.slot[slot++ & 7];
        if ((threadIdx.x & 63) == 63) at[wave] = v;
        __syncthreads();
        return scan16(at[threadIdx.x & 15], none, f);
    }
    template <typename V, typename F> __device__ __forceinline__ V all(V v, V none, F f) {
        return lane(across(scan64(v, none, f), none, f), 15);
    }
    // the sum over the threads in front of this one, and over all
    template <typename V> __device__ __forceinline__ V in_front(V v, V &total) {
        const V s = scan64(v, V(0), Sum{}), w = across(s, V(0), Sum{});
        total = lane(w, 15);
        return (wave ? lane(w, wave - 1) : V(0)) + s - v;
    }

    // ---- the row
    // f(first index, logits) for this thread's vectors; a token that is not possible has -infinity.
    // Rows need no alignment beyond their elements'.
    // NaN: -infinity.  The compiler takes a widened bfloat16 for a quiet number, so the larger of a signalling
    // NaN and -infinity would be a NaN; of bits in a float's place it assumes nothing.
    static __device__ __forceinline__ float value(T z) {
        if constexpr (std::is_same<T, bf16>::value) return upper((uint32_t)__builtin_bit_cast(uint16_t, z) << 16);
        return fmaxf(to_f32(z), -INFINITY);
    }
    static __device__ __forceinline__ float upper(uint32_t bits) { return fmaxf(__uint_as_float(bits), -INFINITY); }
    __device__ __forceinline__ void logits(const Vec &r, const Mask &k, float (&x)[N]) const {
        if constexpr (std::is_same<T, bf16>::value) {  // two of a word: a shift, and a mask
            typedef uint32_t Words __attribute__((ext_vector_type(4)));
            const Words w = __builtin_bit_cast(Words, r);
#pragma unroll
            for (int i = 0; i < N; i++) x[i] = upper(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) x[i] = value(r[i]);
        }
#pragma unroll
        for (int i = 0; i < N; i++)
            if (ok) x[i] = k[i] ? x[i] : -INFINITY;
    }
    template <typename F> __device__ __forceinline__ void rest(F f) const {  // the last, broken vector
        const int whole = a.vocab / N, rest = a.vocab % N;
        if (!rest || threadIdx.x != whole % NT) return;
        float x[N];
#pragma unroll
        for (int k = 0; k < N; k++) {
            const bool there = k < rest && (!ok || ok[whole * N + k]);
            x[k] = there ? value(z[whole * N + k]) : -INFINITY;
        }
        f(whole * N, x);
    }
    template <int U, typename F> __device__ __forceinline__ void pass(F f) const {  // U vectors in flight
        const int whole = a.vocab / N;
        for (int v = threadIdx.x; v < whole; v += U * NT) {
            Vec r[U];
            Mask k[U];
#pragma unroll
            for (int j = 0; j < U; j++) {
                const int64_t i = (int64_t)(v + j * NT < whole ? v + j * NT : v) * N;
                r[j] = *(const Vec *)(z + i);
                if (ok) k[j] = *(const Mask *)(ok + i);
            }
#pragma unroll
            for (int j = 0; j < U; j++) {
                if (v + j * NT >= whole) break;
                float x[N];
                logits(r[j], k[j], x);
                f((v + j * NT) * N, x);
            }
        }
        rest(f);
    }
    static __device__ __forceinline__ float largest(const float (&x)[N]) {
        float v = x[0];
#pragma unroll
        for (int i = 1; i < N; i++) v = fmaxf(v, x[i]);
        return v;
    }

    // ---- values
    // e in 32 bits; the quotient as a product, which moves it by about 2^-23 of the exponent
    __device__ __forceinline__ float weight(float v, float from) const {
        return __builtin_amdgcn_exp2f(fminf((v - from) * c, 0.0f));  // infinity - infinity: 1
    }
    // e in [0, 1] cut to a multiple of 2^-bits
    static __device__ __forceinline__ uint64_t fixed(float e, int bits) {
        const uint32_t b = __float_as_uint(e);
        const int x = (int)(b >> 23) - 150 + bits;
        const uint64_t v = (b & 0x7fffff) | 0x800000;
        return b < 0x800000 || x <= -24 ? 0 : x >= 0 ? v << x : v >> -x;
    }
    __device__ __forceinline__ int mass_bits() const { return 62 - a.index_bits; }  // a row's sum fits
    __device__ __forceinline__ uint64_t mass(float v) const { return fixed(weight(v, top), mass_bits()); }
    // e < min_p, by the exponents: e of a high temperature rounds to 1 where it is less, and is not min_p = 1
    __device__ __forceinline__ bool too_small(float v) const { return (v - top) * c < least; }
    // the distance to the largest logit, as defined: each step rounded to 32 bits
    __device__ __forceinline__ float part(float v) const { return v == top ? 0.0f : (v - top) / t; }
    // the score and the complement of the index: the largest is the answer
    __device__ __forceinline__ uint64_t score(float v, uint32_t i, float noise) const {
        return (uint64_t)order_bits(part(v) + noise) << 32 | (uint32_t)~i;
    }
    __device__ __forceinline__ void answer(int64_t row, uint32_t token) const {
        a.token[row] = token;
        a.logprob[row] = part(to_f32(z[token])) - logf(sum);
    }

    // ---- lists
    // Puts the tokens with logits >= low on the list, at most LIST; returns how many there are.
    __device__ __forceinline__ uint32_t gather(float low) {
        __syncthreads();
        if (threadIdx.x == 0) m.n = 0;
        __syncthreads();
        pass<4>([&](int first, const float (&x)[N]) {
            if (!(largest(x) >= low)) return;
            uint32_t hits = 0;
#pragma unroll
            for (int k = 0; k < N; k++) hits |= x[k] >= low ? 1u << k : 0;
            append(first, x, hits);
        });
        __syncthreads();
        return m.n;
    }
    // The tokens of these lanes' vectors that `hits` names go on the list: one place in the count for
    // all lanes, found by the bits of their numbers.
    __device__ __forceinline__ void append(int first, const float (&x)[N], uint32_t hits) {
#pragma unroll
        for (int k = 0; k < N; k++) hits &= x[k] > -INFINITY ? ~0u : ~(1u << k);
        const uint32_t n = __popc(hits);
        uint32_t total = 0, at = 0;
#pragma unroll
        for (int b = 0; 1 << b <= N; b++) {
            const uint64_t lanes = __ballot(n >> b & 1);
            total += __popcll(lanes) << b;
            at += before_lane(lanes) << b;
        }
        if (!total) return;
        uint32_t base = 0;
        if (before_lane(__ballot(1)) == 0) base = atomicAdd(&m.n, total);
        at += (uint32_t)__builtin_amdgcn_readfirstlane((int)base);
#pragma unroll
        for (int k = 0; k < N; k++)
            if (hits >> k & 1) {
                if (at < LIST) m.list[at] = order_of(x[k], first + k);
                at++;
            }
    }
    static __device__ __forceinline__ uint32_t before_lane(uint64_t lanes) {
        return __builtin_amdgcn_mbcnt_hi((uint32_t)(lanes >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)lanes, 0));
    }
    // where a logit lies in bins of 1 / width from the largest down (infinity - infinity: 0)
    __device__ __forceinline__ float place(float v, float width) const { return fmaxf((top - v) * width, 0.0f); }
    // The smallest logit with place < b (b >= 1, the largest logit finite: it is one), 64 candidates at
    // a time.  -infinity is none.
    __device__ __forceinline__ float edge(float b, float width) const {
        uint32_t under = order_bits(-INFINITY) >> UNSET, from = order_bits(top) >> UNSET;  // not one; one
        while (from - under > 1) {
            const uint32_t step = (from - under + 63) / 64, k = under + (threadIdx.x % 64 + 1) * step;
            const uint64_t lanes = __ballot(k >= from || place(of_key(k), width) < b);
            from = under + (uint32_t)__ffsll((unsigned long long)lanes) * step;
            under = from - step;
        }
        return of_key(from);
    }
    // the numbers of tokens with logits >= low in FINE bins of 1 / width from the largest logit down
    __device__ __forceinline__ void count(float low, float width) {
        __syncthreads();
        for (int i = threadIdx.x; i < FINE; i += NT) m.counts[i] = 0;
        __syncthreads();
        pass<4>([&](int first, const float (&x)[N]) {
#pragma unroll
            for (int i = 0; i < N; i++)
                if (x[i] >= low && x[i] > -INFINITY) atomicAdd(&m.counts[(int)fminf(place(x[i], width), FINE - 1.0f)], 1u);
        });
        __syncthreads();
    }
    // the list in registers (0 past its end); the bins take its place
    __device__ __forceinline__ void hold(uint32_t n, uint64_t (&o)[HELD]) {
#pragma unroll
        for (int i = 0; i < HELD; i++) o[i] = threadIdx.x + i * NT < n ? m.list[threadIdx.x + i * NT] : 0;
        __syncthreads();
    }
    // A listed token's count and mass in one number, 13 and 51 bits.  A mass is at most 2^LIST_BITS, so LIST
    // of them add up to 2^50 at most, and their count to 2^12: neither sum leaves its place.
    static constexpr int LIST_BITS = 38, COUNT = 51;
    static_assert(((uint64_t)LIST << LIST_BITS) < (uint64_t)1 << COUNT && LIST < 1 << (64 - COUNT), "sums fit");
    static constexpr uint64_t MASS = ((uint64_t)1 << COUNT) - 1;
    __device__ __forceinline__ uint64_t both(uint64_t o) const {
        return (uint64_t)1 << COUNT | fixed(weight(logit_of(o), top), LIST_BITS);
    }
    // Of the held tokens with orders in [from, b]: the last that stays, by count the want-th, by mass
    // the last before which there is less than `want`; `until` is what there is up to it.  0 if there
    // are not so many.
    template <bool BY_MASS>
    __device__ __forceinline__ uint64_t select(const uint64_t (&o)[HELD], uint64_t want, uint64_t from, uint64_t b,
                                               uint64_t &until) {
        uint64_t a = from, before = 0;
        auto of = [](uint64_t v) { return BY_MASS ? v & MASS : v >> COUNT; };
        for (;;) {
            const int shift = b - a >= BINS ? 53 - __clzll(b - a) : 0;  // (b - a) >> shift < BINS
            for (int i = threadIdx.x; i < BINS; i += NT) m.bins[i] = 0;
            if (threadIdx.x == 0) m.pick[0] = BINS;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < HELD; i++)
                if (o[i] >= a && o[i] <= b && o[i])
                    atomicAdd((unsigned long long *)&m.bins[(b - o[i]) >> shift], (unsigned long long)both(o[i]));
            __syncthreads();
            const uint64_t v0 = m.bins[2 * threadIdx.x], v1 = m.bins[2 * threadIdx.x + 1];
            uint64_t total;
            const uint64_t p = before + in_front(v0 + v1, total);
            if (of(p) < want && want <= of(p + v0 + v1)) {
                const bool second = want > of(p + v0);
                m.pick[0] = 2 * threadIdx.x + second;
                m.pick[1] = p + (second ? v0 : 0);
                m.pick[2] = second ? v1 : v0;
            }
            __syncthreads();
            const uint64_t bin = m.pick[0], inside = m.pick[2];
            if (bin == BINS) return 0;
            before = m.pick[1];
            b -= bin << shift;
            a = b - a >= (uint64_t)1 << shift ? b - (((uint64_t)1 << shift) - 1) : a;
            __syncthreads();
            if (!shift) {  // a bin is an order: at most six turns, whatever is on the list
                until = before + inside;
                return b;
            }
            if (inside >> COUNT == 1) {  // whose order it is
#pragma unroll
                for (int i = 0; i < HELD; i++)
                    if (o[i] >= a && o[i] <= b) m.pick[0] = o[i];
                __syncthreads();
                until = before + inside;
                const uint64_t last = m.pick[0];
                __syncthreads();
                return last;
            }
        }
    }

    // Of the row's tokens with orders in [from, b]: as `select`, with masses in multiples of
    // 2^-mass_bits, eleven bits of the order at a time.
    template <bool BY_MASS> __device__ __forceinline__ uint64_t locate(uint64_t want, uint64_t from, uint64_t b) {
        uint64_t a = from, before = 0;
        for (;;) {
            const int shift = b - a >= BINS ? 53 - __clzll(b - a) : 0;  // (b - a) >> shift < BINS
            __syncthreads();
            for (int i = threadIdx.x; i < BINS; i += NT) m.bins[i] = 0;
            if (threadIdx.x == 0) m.pick[0] = BINS;
            __syncthreads();
            pass<1>([&](int first, const float (&x)[N]) {
#pragma unroll
                for (int k = 0; k < N; k++) {
                    const uint64_t o = order_of(x[k], first + k);
                    if (o >= a && o <= b)
                        atomicAdd((unsigned long long *)&m.bins[(b - o) >> shift],
                                  (unsigned long long)(BY_MASS ? mass(x[k]) : 1));
                }
            });
            __syncthreads();
            const uint64_t v0 = m.bins[2 * threadIdx.x], v1 = m.bins[2 * threadIdx.x + 1];
            uint64_t total;
            const uint64_t p = before + in_front(v0 + v1, total);
            if (p < want && want <= p + v0 + v1) {
                const bool second = want > p + v0;
                m.pick[0] = 2 * threadIdx.x + second;
                m.pick[1] = p + (second ? v0 : 0);
            }
            __syncthreads();
            const uint64_t bin = m.pick[0];
            if (bin == BINS) return 0;
            before = m.pick[1];
            b -= bin << shift;
            if (!shift) return b;
            const uint64_t width = (uint64_t)1 << shift;
            a = b - a >= width ? b - (width - 1) : a;
        }
    }
    // the mass of the tokens with orders >= last
    __device__ __forceinline__ uint64_t mass_until(uint64_t last) {
        uint64_t v = 0;
        pass<1>([&](int first, const float (&x)[N]) {
#pragma unroll
            for (int k = 0; k < N; k++)
                if (order_of(x[k], first + k) >= last) v += mass(x[k]);
        });
        return all(v, (uint64_t)0, Sum{});
    }

    // The best score of the tokens with orders >= last, or (UNTIL) of those in bins < first_bin, whose
    // mass goes to `above`; those in [first_bin, last_bin] are listed then.
    template <bool UNTIL>
    __device__ __forceinline__ uint64_t best(uint64_t last, float width, float first_bin, float last_bin, float &above) {
        constexpr int U = 2;
        // UNTIL: tokens from `low` on stay, those from `listing` on to it are listed
        const float low = UNTIL ? first_bin >= 1 ? edge(first_bin, width) : INFINITY : last <= 1 ? -INFINITY : logit_of(last);
        const float listing = UNTIL ? edge(last_bin + 1.0f, width) : 0.0f;
        const float rt = 1.0f / t;
        // no quick score where the reciprocal of the temperature has lost digits, or off infinity
        const bool slow = !(t > 0x1p-100f && t < 0x1p100f) || top == INFINITY;
        uint64_t win = 0;
        float part_sum = 0;
        // A score is computed as defined only where a quick one comes near the best so far: the quick
        // quotient is off by less than 2^-22 of itself, a sum by 2^-23.  `quick` is that with 2^-20 of
        // both on top.
        auto consider = [&](float v, uint32_t i, float noise) {
            if (!(v >= low) || (!UNTIL && order_of(v, i) < last) || too_small(v)) return;
            const uint64_t s = score(v, i, noise);
            if (s > win) {
                win = s;
                if ((uint32_t)(s >> 32) > *(volatile uint32_t *)&m.cut) atomicMax(&m.cut, (uint32_t)(s >> 32));
            }
        };
        auto handle = [&](int first, const float (&x)[N], const float (&noise)[N]) {
            const float cut = of_order_bits(*(volatile uint32_t *)&m.cut);  // NaN before the first
            float quick = -INFINITY;
            uint32_t listed = 0;
#pragma unroll
            for (int k = 0; k < N; k++) {
                const float off = (x[k] >= low ? x[k] : -INFINITY) - top, d = off * rt, score = d + noise[k];
                if constexpr (UNTIL) {
                    part_sum += __builtin_amdgcn_exp2f(off * c);
                    listed |= x[k] >= listing && x[k] < low ? 1u << k : 0;
                }
                quick = fmaxf(quick, score + (fabsf(d) + fabsf(score)) * 0x1p-20f);
            }
            if (slow || !(quick < cut)) {
#pragma unroll
                for (int k = 0; k < N; k++) consider(x[k], first + k, noise[k]);
            }
            if (UNTIL && listed) append(first, x, listed);
        };
        const int whole = a.vocab / N;
        Vec r[U];
        Mask ks[U];
        auto fetch = [&](int v) {
#pragma unroll
            for (int j = 0; j < U; j++) {
                const int64_t i = (int64_t)(v + j * NT < whole ? v + j * NT : 0) * N;
                r[j] = *(const Vec *)(z + i);
                if (ok) ks[j] = *(const Mask *)(ok + i);
            }
        };
        if ((int)threadIdx.x < whole) fetch(threadIdx.x);
        for (int v = threadIdx.x; v < whole; v += U * NT) {
            float x[U][N], noise[U][N];
#pragma unroll
            for (int j = 0; j < U; j++) {
                logits(r[j], ks[j], x[j]);
                const float most = largest(x[j]);
                const bool need = v + j * NT < whole && most > -INFINITY && most >= low;
                if (need) {
                    const float *g = gumbel + (int64_t)(v + j * NT) * N;
#pragma unroll
                    for (int i = 0; i < N; i += 4) {
                        const Four f = *(const Four *)(g + i);
#pragma unroll
                        for (int k = 0; k < 4; k++) noise[j][i + k] = f[k];
                    }
                }
            }
            if (v + U * NT < whole) fetch(v + U * NT);  // on their way while these are handled
#pragma unroll
            for (int j = 0; j < U; j++)
                if (v + j * NT < whole) handle((v + j * NT) * N, x[j], noise[j]);
        }
        rest([&](int first, const float (&x)[N]) {
            float noise[N];
#pragma unroll
            for (int k = 0; k < N; k++) noise[k] = first + k < a.vocab ? gumbel[first + k] : 0.0f;
            handle(first, x, noise);
        });
        above = part_sum;
        return win;
    }
};

template <typename T> __global__ __launch_bounds__(NT) void k_sample(SampleArgs a) {
    typedef Sampler<T> S;
    constexpr int N = S::N;
    __shared__ SampleShared m;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const float temp = a.temperature[row];
    const bool greedy = !(temp > 0);
    const int k = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.0f;
    S s{a, m, (const T *)a.logits + row * a.logits_stride, a.allowed ? a.allowed + row * a.allowed_stride : nullptr,
        a.gumbel + row * a.gumbel_stride, (int)__builtin_amdgcn_readfirstlane(tid >> 6), 0, greedy ? 1.0f : temp};
    s.min_p = a.min_p ? a.min_p[row] : 0.0f;
    s.least = s.min_p > 0 ? log2f(s.min_p) : -INFINITY;
    // above 0 a product with -infinity stays that, up to 2^126 one with 0 stays 0 (felt by subnormal differences
    // of logits alone)
    s.c = fminf(fmaxf(1.44269504f / s.t, 0x1p-149f), 0x1p126f);
    m.counts[tid] = 0;
    if (tid == 0) m.cut = 0, m.pick[0] = NT;
    // the thread's largest logit, where it first occurs, and its mass from there
    float mine = -INFINITY, sum = 0;
    uint32_t where = 0;
    s.template pass<4>([&](int first, const float (&x)[N]) {
        const float v = S::largest(x);
        if (v > mine) sum *= s.weight(mine, v), mine = v, where = first;
        if (mine > -INFINITY) {
#pragma unroll
            for (int i = 0; i < N; i++) sum += __builtin_amdgcn_exp2f((x[i] - mine) * s.c);
        }
    });
    const uint32_t top_bits = s.all(mine > -INFINITY ? order_bits(mine) : 0u, 0u, Larger{});
    if (!top_bits) {
        if (tid == 0) a.token[row] = -1, a.logprob[row] = -INFINITY;
        return;
    }
    s.top = of_order_bits(top_bits);
    if (s.top == INFINITY) {  // infinity - infinity: each is worth 1, and nothing else anything
        sum = 0;
        s.template pass<1>([&](int first, const float (&x)[N]) {
#pragma unroll
            for (int i = 0; i < N; i++) sum += x[i] == INFINITY ? 1.0f : 0.0f;
        });
    }
    s.sum = s.all(mine > -INFINITY ? sum * s.weight(mine, s.top) : 0.0f, 0.0f, Sum{});
    if (greedy || k == 1 || p <= 0 || s.min_p > 1) {  // the first alone: it is in the first vector that holds it
        uint32_t i = ~s.all(mine == s.top ? ~where : 0u, 0u, Larger{});
        if (tid == 0) {
            while (!(to_f32(s.z[i]) == s.top && (!s.ok || s.ok[i]))) i++;
            s.answer(row, i);
        }
        return;
    }
    const bool by_count = k > 0 && k < a.vocab, by_mass = p < 1, by_size = s.min_p > 0;
    uint64_t win = 0;
    float unused;
    // what the mass in front of a token that stays is under, in multiples of 2^-bits
    auto under = [&](double whole, int bits) {
        const double w = ceil((double)p * whole * exp2((double)bits));
        return w > 1 ? (uint64_t)w : (uint64_t)1;
    };
    if (!by_count && !by_mass && !by_size) {
        win = s.template best<false>(1, 0, 0, 0, unused);
    } else {
        float low = -INFINITY;
        if (by_count) {
            // the k-th largest of the threads' maxima, or a little less: by bins of equal width
            const float least = of_order_bits(~s.all(mine > -INFINITY ? ~order_bits(mine) : 0u, 0u, Larger{}));
            const float range = s.top - least;
            if (mine > -INFINITY) atomicAdd(&m.counts[(int)fminf(fmaxf((s.top - mine) * (NT / range), 0.0f), NT - 1.0f)], 1u);
            __syncthreads();
            uint32_t total;
            const uint32_t v = m.counts[tid], before = s.in_front(v, total);
            if (before < (uint32_t)k && (uint32_t)k <= before + v) m.pick[0] = tid;
            __syncthreads();
            const int at = (int)m.pick[0];
            // The bin's lower edge, and more than it may be off by: places and differences by 2^-22 of themselves, the
            // bound by 2^-24 of the largest logit.  A part of the range, as a bin may be narrower than any number.
            if (at < NT) low = fmaxf(least, s.top - range * ((float)(at + 1) / NT) * 1.00001f - fabsf(s.top) * 1e-6f);
        } else if (by_mass) {
            low = s.top + (__log2f((1.0f - p) * s.sum / (float)a.vocab) - SLACK) / s.c;
        }
        // nothing under min_p stays; only the mass of the first k by count has it in it
        const float nucleus = low;
        if (by_size && !(by_count && by_mass)) low = fmaxf(low, s.top + (s.least - SLACK) / s.c);
        // Threads with something for the list, and which of two ways is tried by it.
        //  - Top-k.  The bound is one maximum of each thread: where half of them pass, whole vectors of neighbours
        //    (eight of 16 bits a thread) still fit the list, beyond that it may overflow, and where fewer than k
        //    threads have a token there is no bound.  Then the tokens are counted in bins down to it, or down to
        //    e = 2^-64, and the k-th one's bin is the bound.  1 x 131072 bf16, k = 600: sorted logits 35 us, 98
        //    without the count; in random order 50 us, 41 without.
        //  - A nucleus.  1000 of 1024 threads mean 1024 ln(1024 / 24) = 3840 tokens if they fall evenly, what a list
        //    just holds; above that a nucleus has thousands and the list is not tried.  256 x 131072 bf16, top-p
        //    0.95: deviation 8 (675 threads) 44.5 us, without the list 53; deviation 2.5 (all threads) 72, with a
        //    list that overflows 93.
        const int passing = __syncthreads_count(mine > -INFINITY && mine >= low);
        if (by_count && a.vocab > LIST && (passing > NT / 2 || low == -INFINITY)) {
            const float range = s.top - fmaxf(low, s.top - 64.0f / s.c);
            if (tid == 0) m.pick[0] = FINE;
            s.count(low, (float)FINE / range);
            uint32_t own = 0, total;
#pragma unroll
            for (int i = 0; i < EACH; i++) own += m.counts[EACH * tid + i];
            uint32_t before = s.in_front(own, total);
#pragma unroll
            for (int i = 0; i < EACH; i++) {
                const uint32_t v = m.counts[EACH * tid + i];
                if (before < (uint32_t)k && (uint32_t)k <= before + v) m.pick[0] = EACH * tid + i;
                before += v;
            }
            __syncthreads();
            const int at = (int)m.pick[0];
            if (at < FINE - 1)  // the last bin has what is below the range too
                low = fmaxf(low, s.top - range * ((float)(at + 1) / FINE) * 1.00001f - fabsf(s.top) * 1e-6f);
        }
        uint32_t n = LIST + 1;
        if (by_count || a.vocab <= LIST || passing <= NT - 24) n = s.gather(low);
        if (n <= 64) {  // one wave, a lane a token: its rank and the mass in front of it
            if (s.wave) return;
            const uint64_t o = (uint32_t)tid < n ? m.list[tid] : 0;
            const float noise = o ? s.gumbel[s.index_of(o)] : 0.0f;
            const uint64_t own = o ? s.both(o) : 0;
            uint64_t q = 0;
            for (uint32_t j = 0; j < n; j++) {
                const uint64_t oj = lane(o, j), vj = lane(own, j);
                q += oj > o ? vj : 0;
            }
            bool stay = o && (!by_count || (int64_t)(q >> S::COUNT) < k);
            if (by_mass) {
                const uint64_t whole = lane(scan64(stay ? own & S::MASS : 0, (uint64_t)0, Sum{}), 63);
                stay = stay && (q & S::MASS) < (by_count ? under((double)whole * exp2(-S::LIST_BITS), S::LIST_BITS)
                                                         : under((double)s.sum, S::LIST_BITS));
            }
            const float v = s.logit_of(o);
            if (stay && !s.too_small(v)) win = s.score(v, s.index_of(o), noise);
            win = lane(scan64(win, (uint64_t)0, Larger{}), 63);
            if (tid == 0) s.answer(row, s.index_of(win));
            return;
        }
        if (n <= LIST) {
            uint64_t o[HELD], last = 1, until = 0;
            s.hold(n, o);
            const uint64_t from = low > -INFINITY ? s.lowest(low) : 1, to = s.highest(s.top);
            if (by_count && (uint32_t)k < n) {
                last = s.template select<false>(o, k, from, to, until);
            } else if (by_mass) {
#pragma unroll
                for (int i = 0; i < HELD; i++) until += o[i] ? s.both(o[i]) : 0;
                until = s.all(until, (uint64_t)0, Sum{});
            }
            if (by_mass) {
                const double whole = by_count ? (double)(until & S::MASS) * exp2(-S::LIST_BITS) : (double)s.sum;
                const uint64_t l = s.template select<true>(o, under(whole, S::LIST_BITS), larger(from, last), to, until);
                last = larger(l, last);  // 0: all of them
            }
#pragma unroll
            for (int i = 0; i < HELD; i++) {
                const float v = s.logit_of(o[i]);
                if (o[i] && o[i] >= last && !s.too_small(v))
                    win = larger(win, s.score(v, s.index_of(o[i]), s.gumbel[s.index_of(o[i])]));
            }
        } else {
            uint64_t last = 1;
            bool found = false;
            if (by_mass && !by_count) {
                // Counts in bins down to the bound; a bin's mass by e of its middle, at most `off` off: half a bin, and
                // 1e-4 for the 24 additions in front of a sum, the exponentials and the mass.
                const float range = s.top - nucleus, width = (float)FINE / range;
                s.count(nucleus, width);
                const float step = range / FINE * s.c;  // of a bin, in powers of two
                const float off = __builtin_amdgcn_exp2f(0.5f * step) - 1.0f + 1e-4f, want = p * s.sum;
                float own = 0, total, v[EACH];
#pragma unroll
                for (int i = 0; i < EACH; i++) {
                    const int at = EACH * tid + i;
                    v[i] = (float)m.counts[at] * __builtin_amdgcn_exp2f(-((float)at + 0.5f) * step);
                    own += v[i];
                }
                float after = s.in_front(own, total);
                // The first bin after which there may be `want`, and the first after which there must be (the last
                // one if none: nothing under it is in the nucleus).  Each is the least over all bins, so it does
                // not matter that a thread's last sum and the next thread's first differ in their rounding.
                uint32_t may = FINE, must = FINE;
#pragma unroll
                for (int i = 0; i < EACH; i++) {
                    after += v[i];
                    if (may == FINE && after * (1 + off) >= want) may = EACH * tid + i;
                    if (must == FINE && after * (1 - off) >= want) must = EACH * tid + i;
                }
                const float first_bin = (float)~s.all(~may, 0u, Larger{});
                const float last_bin = fminf((float)~s.all(~must, 0u, Larger{}), FINE - 1.0f);
                // A bin is under 2^-7 of a power of two (the range has log2(vocab / (1 - p)) of them, 49 at most); where it
                // is not, the range is what rounding the largest logit leaves, and a few bins hold everything.  A range
                // under 2.4e-35 has no such width in 32 bits: its bins are the largest logit's and the rest.
                if (first_bin < FINE && step < 0.125f && width < INFINITY) {
                    if (tid == 0) m.n = 0;
                    __syncthreads();
                    float above;
                    win = s.template best<true>(0, width, first_bin, last_bin, above);
                    above = s.all(above, 0.0f, Sum{});
                    n = m.n;
                    if (n <= LIST) {
                        found = true;
                        uint64_t o[HELD], until;
                        s.hold(n, o);
                        const double left = (double)p * s.sum - above;
                        if (left > 0) {
                            const double w = ceil(left * exp2(S::LIST_BITS));
                            // a bin more at both ends, for what the bins' edges are off by
                            const float lo = s.top - (last_bin + 2.0f) / width, hi = s.top - (first_bin - 1.0f) / width;
                            last = s.template select<true>(o, w > 1 ? (uint64_t)w : 1, s.lowest(lo), s.highest(hi), until);
#pragma unroll
                            for (int i = 0; i < HELD; i++) {
                                const float v = s.logit_of(o[i]);
                                if (o[i] && o[i] >= last && !s.too_small(v))
                                    win = larger(win, s.score(v, s.index_of(o[i]), s.gumbel[s.index_of(o[i])]));
                            }
                        }
                    }
                }
            }
            if (!found) {
                const uint64_t from = low > -INFINITY ? s.lowest(low) : 1, to = s.highest(s.top);
                last = from;
                double whole = (double)s.sum;
                if (by_count) last = larger(last, s.template locate<false>(k, from, to));  // 0: there are not so many
                if (by_count && by_mass) whole = (double)s.mass_until(last) * exp2(-(double)s.mass_bits());
                if (by_mass) last = larger(last, s.template locate<true>(under(whole, s.mass_bits()), last, to));
                __syncthreads();
                if (tid == 0) m.cut = 0;
                __syncthreads();
                win = s.template best<false>(last, 0, 0, 0, unused);
            }
        }
    }
    win = s.all(win, (uint64_t)0, Larger{});
    if (tid == 0) s.answer(row, s.index_of(win));
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
    auto go = [&](auto ty) {
        typedef decltype(ty) T;
        return in_parts(rows, NT, [&](int64_t first, int64_t n) {
            auto from = [&](auto *p, int64_t at) { return p ? p + at : nullptr; };
            const SampleArgs a{(const T *)logits + first * logits_stride, gumbel + first * gumbel_stride,
                               temperature + first, from(top_p, first), from(min_p, first), from(top_k, first),
                               from(allowed, first * allowed_stride), logits_stride, gumbel_stride, allowed_stride,
                               (int)vocab, bits, token + first, logprob + first};
            k_sample<T><<<dim3((uint32_t)n), NT, 0, (hipStream_t)stream>>>(a);
            return launched();
        });
    };
    return type == CKKS_PLAIN_BF16 ? go(bf16{}) : type == CKKS_PLAIN_F16 ? go(f16{}) : go(0.0f);
}
