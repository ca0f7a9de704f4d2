// logprob.hip -- log probabilities of given tokens, entropy and the largest alternatives, and their gradient.
#include "plain_common.h"

namespace ckks_plain {

constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;

struct ScoreArgs {
    const void *logits;
    const int64_t *tokens;
    const float *temperature;
    const uint8_t *allowed;
    int64_t stride, allowed_stride, first;
    int vocab, top;
    float *logprob, *entropy, *largest, *log_mass;
    int64_t *top_token;
    float *top_logprob;
};

// 1 / temperature of a row: at most 2^127, so that its product with log2 e is finite.
__device__ __forceinline__ float inverse_temperature(const float *temperature, int64_t row) {
    const float t = temperature ? temperature[row] : 1.0f;
    return t > 0.0f ? fminf(1.0f / t, 0x1p127f) : 1.0f;
}
// (z - largest) factor: 0 where both are infinite; -infinity below an infinite largest logit (and of -infinity and NaN),
// also where the factor is 0, that of an infinite temperature; by its two parts where the distance of finite logits
// leaves the range of 32 bits, as its quotient by a large temperature need not.
__device__ __forceinline__ float distance_times(float z, float largest, float factor) {
    const float d = z - largest;
    if (z == largest) return 0.0f;
    if (d > -INFINITY) return d * factor;
    return z > -INFINITY && largest < INFINITY ? z * factor - largest * factor : -INFINITY;
}

constexpr int MAX_SLICES = 32, JOIN_KEYS = MAX_SLICES * CKKS_PLAIN_MAX_TOP;

// A row's given token: its logit (NaN where it is not possible), or none.  Asked for before the row is read: at the
// end, two loads one after the other took a third of the time between the last logit and the results.
struct Given {
    bool there;
    float logit;
};
template <typename T, bool MASK>
__device__ __forceinline__ Given given_token(const ScoreArgs &a, int64_t row, const T *z, const uint8_t *allowed) {
    const int64_t token = a.tokens[row];
    Given g{token >= 0 && token < a.vocab, NAN};
    if (g.there) g.logit = to_f32(z[token]);
    if (MASK && g.there && !allowed[token]) g.logit = NAN;
    return g;
}
__device__ __forceinline__ void put_score(const ScoreArgs &a, int64_t row, const Given &g, float largest, float log_mass,
                                          float mean, float inv_t) {
    a.logprob[row] = !g.there                ? 0.0f
                     : g.logit > -INFINITY ? distance_times(g.logit, largest, inv_t) - log_mass
                                             : -INFINITY;
    a.entropy[row] = log_mass > -INFINITY ? log_mass - LN2 * mean : 0.0f;  // mean: of the distances, in powers of two
    a.largest[row] = largest;
    a.log_mass[row] = log_mass;
}

// Logits c ... c + 7 of a row; -infinity or NaN where there is no possible token.
template <typename T, bool MASK> struct Logits {
    Piece<T, 8> e;
    Piece<int8_t, 8> ok;
    // STREAM: past the caches
    template <bool STREAM> __device__ __forceinline__ void fetch(const T *z, const uint8_t *allowed, int c) {  // whole
        if (STREAM) e.fetch_once(z + c);
        else e.fetch(z + c);
        if (MASK && STREAM) ok.fetch_once((const int8_t *)allowed + c);
        else if (MASK) ok.fetch((const int8_t *)allowed + c);
    }
    __device__ __forceinline__ void fetch(const T *z, const uint8_t *allowed, int c, int end) {
        e.fetch(z + c, end - c);
        if constexpr (MASK) ok.fetch((const int8_t *)allowed + c, end - c);
    }
    __device__ __forceinline__ void widen(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            f[i] = e.at(i);
            if (MASK && !ok.v[0][i]) f[i] = -INFINITY;
        }
    }
    __device__ __forceinline__ void widen(int c, int end, float (&f)[8]) const {
        widen(f);
        if (c + 8 > end) {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (c + i >= end) f[i] = -INFINITY;
        }
    }
};

constexpr int JOIN_NT = 512, CANDIDATES = 1024, FEW = 128;
constexpr float LEAST = -200.0f;  // exp2 of it is 0

// Sums of 2^x and of x 2^x over logits z, x = z scale - at, where `at` is near the largest z scale so far.
struct Mass {
    float at, mass, moment;
    __device__ __forceinline__ void shift(float d) {  // every x by d
        const float k = __builtin_amdgcn_exp2f(d);
        moment = k * (moment + d * mass);
        mass *= k;
    }
    __device__ __forceinline__ void move(float to) {
        shift(fmaxf(at - to, LEAST));
        at = to;
    }
    __device__ __forceinline__ void add(const float (&f)[8], float scale) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float x = fmaxf(__builtin_fmaf(f[i], scale, -at), LEAST);  // LEAST for -infinity and NaN
            const float e = __builtin_amdgcn_exp2f(x);
            mass += e;
            moment = __builtin_fmaf(e, x, moment);
        }
    }
};
// NaN where there is one (the instruction that lets them through takes numbers as they are loaded)
__device__ __forceinline__ float max_or_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float largest_of(const float (&f)[8]) {
    return max_or_nan(max_or_nan(max_or_nan(f[0], f[1]), max_or_nan(f[2], f[3])),
                      max_or_nan(max_or_nan(f[4], f[5]), max_or_nan(f[6], f[7])));
}
// The order of tokens as a number: by logit, then the lower index.  0 is below all.
__device__ __forceinline__ uint64_t token_key(float z, int index) { return (uint64_t)order_bits(z) << 32 | (uint32_t)~index; }
__device__ __forceinline__ float key_logit(uint64_t k) { return of_order_bits((uint32_t)(k >> 32)); }

// Alternative `rank` of a row (key 0: there is none), or of its slice.
__device__ __forceinline__ void put_top(const ScoreArgs &a, int64_t row, int rank, uint64_t key, float largest,
                                        float log_mass, float inv_t, uint64_t *keys) {
    if (keys) {
        keys[(row * gridDim.y + blockIdx.y) * a.top + rank] = key;
        return;
    }
    a.top_token[row * a.top + rank] = key ? (int64_t)(uint32_t)~(uint32_t)key : -1;
    a.top_logprob[row * a.top + rank] = key ? distance_times(key_logit(key), largest, inv_t) - log_mass : -INFINITY;
}

template <int NT> struct ScoreShared {
    uint64_t list[CANDIDATES], bound;  // the list begins as the threads' keys
    uint32_t slots[NT / 64], more[NT / 64], ranks[64], winners[NT], n_winners, n_readers, n;
    float sums[2][NT / 64];
};
// What a slice of a row leaves for the whole: these and its `top` largest keys, in order.
struct Part {
    float m, mass, moment, unused;  // 16 bytes: the keys behind the parts are aligned
};

// The rank of a key of sh.list: how many of its first n are larger.
__device__ __forceinline__ int rank_in_list(const uint64_t *list, int n, uint64_t key) {
    int r = 0;
    for (int i = 0; i < n; i++) r += list[i] > key;
    return r;
}
__device__ __forceinline__ uint64_t other_lane(uint64_t v, int far) {
    return (uint64_t)(uint32_t)__shfl_xor((int)(v >> 32), far) << 32 | (uint32_t)__shfl_xor((int)v, far);
}
// One key a lane, falling over the wave: all of them, or (from half = 32 on) of a sequence that falls and then rises.
__device__ __forceinline__ uint64_t sort_halves(uint64_t v, int l, int size, int half) {
    for (; half; half >>= 1) {
        const uint64_t w = other_lane(v, half);
        const bool low = !(l & half), falls = !(l & size);
        v = (low == falls) == (v > w) ? v : w;
    }
    return v;
}
__device__ __forceinline__ uint64_t sort_wave(uint64_t v, int l) {
    for (int size = 2; size <= 64; size *= 2) v = sort_halves(v, l, size, size / 2);
    return v;
}
// The largest 64 of two falling sequences, falling; `reversed`: the second from its end.
__device__ __forceinline__ uint64_t join_waves(uint64_t v, uint64_t reversed, int l) {
    return sort_halves(v > reversed ? v : reversed, l, 64, 32);
}
// The largest 64 of the list's first n, falling, at its front (behind the last: 0).  All threads; ends behind a barrier.
// (A rank by comparison with all n costs as many reads for each: 4096 x 1000 bf16 top 64 450 us, so 34.)
template <int NT> __device__ __forceinline__ void sort_list(uint64_t *list, int n) {
    const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
    uint64_t v = 0;
    for (int q = wave; q * 64 < n; q += NT / 64) {
        uint64_t w = sort_wave(q * 64 + l < n ? list[q * 64 + l] : 0, l);
        v = join_waves(v, other_lane(w, 63), l);
    }
    __syncthreads();
    list[threadIdx.x] = v;
    for (int s = NT / 128; s; s /= 2) {
        __syncthreads();
        if (wave < s) {
            v = join_waves(v, list[(wave + s) * 64 + 63 - l], l);
            list[wave * 64 + l] = v;
        }
    }
    __syncthreads();
}

// A workgroup reads a slice of a row once; each thread keeps the sums of what it reads.  Their `at` is the
// rounded product of its largest logit and the scale: one multiply-add gives an x, whose shift by that
// rounding is taken out at the end.  Where the products have no room (beyond 2^20, that rounding is no small
// number: infinite logits, tiny temperatures, rows of the type's lowest value) or a logit is NaN, the slice is
// read twice more, with distances to its largest logit.
//
// The alternatives:  a thread's key is its largest logit and the end of the vector where that first came, so
// at least one token is not below it.  The top-th largest of the keys of 64 groups of threads is a bound which
// at least `top` tokens pass; they are all among the tokens of threads whose largest logit passes it from its
// vector's start (`winners`, little more than `top`).  Such a thread's vector is read again, and its others where
// the largest of them may pass too (all of them would be lines of memory: 2048 x 131072 bf16 top 20 120 us, so 96).
// What passes goes on a list, and a token's rank there is its place.  Where the list is too short (runs of equal
// logits, rows in bad order), the top-th largest on it is a better bound: all that were on it below that one do not
// come back, so it ends.
//
// 2048 x 131072 bf16 top 20 takes 96 us in a loop, 100 on logits that no cache has (5.6 and 5.4 TB/s; reading alone
// reaches 6.1): memory, with the vector units busy for most of it (two of the 124 vector instructions for 16 logits
// less change nothing), and 5 us of choosing at the rows' ends.  Without alternatives 4096 x 32768 bf16 50 us
// (5.4 TB/s).  Few rows are latency: 4 x 32768 f32 top 5 7.5 us, 333 x 50021 f16 top 20 under a mask 21.5 us for 50 MB.
// The next two vectors are on their way while two are added; four or six were no faster (2048 x 131072 95 and 97 us,
// 333 x 50021 15.6 and 15.9 instead of 15.0, 1000 x 16384 9.0 and 9.1 instead of 8.4).
constexpr float ROOM = 0x1p20f;
template <typename T, bool MASK, bool TOP, bool STREAM, int NT>
__global__ __launch_bounds__(NT) void k_token_logprobs(ScoreArgs a, int slice, Part *parts, uint64_t *keys) {
    __shared__ ScoreShared<NT> sh;
    const int t = threadIdx.x;
    const int64_t row = a.first + blockIdx.x;
    const T *z = (const T *)a.logits + row * a.stride;
    const uint8_t *allowed = MASK ? a.allowed + row * a.allowed_stride : nullptr;
    Given given{};
    if (!parts) given = given_token<T, MASK>(a, row, z, allowed);
    const float inv_t = inverse_temperature(a.temperature, row), scale = inv_t * LOG2E;
    const int begin = blockIdx.y * slice, end = begin + slice < a.vocab ? begin + slice : a.vocab;
    Mass s{-ROOM, 0, 0};
    float best = -INFINITY;  // the largest; best_at: the first vector that has it
    int best_at = 0;
    float next = -INFINITY;  // the largest of the other vectors
    if (t == 0) sh.bound = 1, sh.n_winners = sh.n_readers = sh.n = 0;
    if (t < 64) sh.ranks[t] = 0;
    // two vectors at a time, the next two on their way
    auto take = [&](const float (&f)[8], int c, const float (&g)[8], int d) {
        const float v = largest_of(f), w = largest_of(g);
        if (TOP) {
            if (v > best) best_at = c;
            next = __builtin_amdgcn_fmed3f(v, best, next);
            best = max_or_nan(best, v);
            if (w > best) best_at = d;
            next = __builtin_amdgcn_fmed3f(w, best, next);
            best = max_or_nan(best, w);
        } else {
            best = max_or_nan(best, max_or_nan(v, w));
        }
        s.move(fmaxf(best * scale, -ROOM));
        s.add(f, scale);
        s.add(g, scale);
    };
    constexpr int STEP = NT * 8;
    const int whole = (end - begin) / (2 * STEP);
    int c = begin + t * 8;
    Logits<T, MASK> p, q;
    auto fetch = [&](int c) {
        p.template fetch<STREAM>(z, allowed, c);
        q.template fetch<STREAM>(z, allowed, c + STEP);
    };
    if (whole) fetch(c);
    for (int i = 0; i < whole; i++, c += 2 * STEP) {
        float f[8], g[8];
        p.widen(f);
        q.widen(g);
        if (i + 1 < whole) fetch(c + 2 * STEP);
        take(f, c, g, c + STEP);
    }
    if (c < end) {
        float f[8], g[8];
        p.fetch(z, allowed, c, end);
        p.widen(c, end, f);
        if (c + STEP < end) q.fetch(z, allowed, c + STEP, end);
        q.widen(c + STEP, end, g);
        take(f, c, g, c + STEP);
    }
    const uint32_t top_bits = row_all<NT>(best != best ? ~0u : order_bits(best), sh.slots, Larger{});
    float m = of_order_bits(top_bits);  // -infinity where nothing is possible
    if (top_bits != ~0u && fabsf(m * scale) < ROOM) {
        const float at = m * scale;
        s.move(at);
        s.shift(-__builtin_fmaf(m, scale, -at));
    } else if (m != -INFINITY) {
        best = next = -INFINITY;
        for (int c = begin + t * 8; c < end; c += STEP) {
            float f[8], v = -INFINITY;
            p.fetch(z, allowed, c, end);
            p.widen(c, end, f);
#pragma unroll
            for (int i = 0; i < 8; i++) v = fmaxf(v, f[i]);  // not NaN
            next = fmaxf(next, fminf(v, best));
            if (v > best) best = v, best_at = c;
        }
        m = of_order_bits(row_all<NT>(order_bits(best), sh.more, Larger{}));
        s.mass = s.moment = 0;
        for (int c = begin + t * 8; c < end; c += STEP) {
            float f[8];
            p.fetch(z, allowed, c, end);
            p.widen(c, end, f);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float x = fmaxf(distance_times(f[i], m, scale), LEAST);
                const float e = f[i] > -INFINITY ? __builtin_amdgcn_exp2f(x) : 0.0f;
                s.mass += e;
                s.moment += e * x;
            }
        }
    }
    row_sums<NT>(s.mass, s.moment, sh.sums[0], sh.sums[1]);
    const bool some = s.mass > 0;
    const float log_mass = some ? logf(s.mass) : -INFINITY, largest = some ? m : -INFINITY;
    if (t == 0) {
        if (parts) {
            parts[row * gridDim.y + blockIdx.y] = Part{largest, s.mass, s.moment, 0};
        } else {
            put_score(a, row, given, largest, log_mass, s.moment / s.mass, inv_t);
        }
    }
    if (!TOP) return;
    const uint64_t mine = best > -INFINITY ? token_key(best, best_at + 7) : 0;
    sh.list[t] = mine;
    __syncthreads();
    uint64_t key = 0;  // of the threads l, l + 64, ...: short rows are in all of these groups too
    for (int w = 0; w < NT / 64; w++) key = Larger{}(key, sh.list[w * 64 + (t & 63)]);
    uint32_t larger = 0;  // a part of the other groups for each wave
    for (int i = t >> 6; i < 64; i += NT / 64) larger += lane(key, i) > key;
    atomicAdd(&sh.ranks[t & 63], larger);
    __syncthreads();
    if (t < 64 && sh.ranks[t] == (uint32_t)a.top - 1 && key) sh.bound = key;
    const int steps = (end - begin + NT * 8 - 1) / (NT * 8);  // vectors of a thread
    int n;
    for (;;) {
        __syncthreads();
        const uint64_t bound = sh.bound;
        auto list_vector = [&](int c) {
            Logits<T, MASK> p;
            float f[8];
            p.fetch(z, allowed, c, end);
            p.widen(c, end, f);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint64_t key = token_key(f[i], c + i);
                if (f[i] > -INFINITY && key >= bound) {
                    const uint32_t at = atomicAdd(&sh.n, 1u);
                    if (at < CANDIDATES) sh.list[at] = key;
                }
            }
        };
        if (mine && mine + 7 >= bound) {
            // its other vectors, if one may hold a token that passes; the front of `winners` is those to read in
            // full, the back those of one vector
            if (token_key(next, 0) >= bound) sh.winners[atomicAdd(&sh.n_readers, 1u)] = t;
            else sh.winners[NT - 1 - atomicAdd(&sh.n_winners, 1u)] = best_at;
        }
        __syncthreads();
        const int jobs = (int)sh.n_readers * steps, ones = (int)sh.n_winners;
        for (int j = t; j < jobs + ones; j += NT) {
            const int c = j < jobs ? begin + (j % steps * NT + (int)sh.winners[j / steps]) * 8
                                   : (int)sh.winners[NT - 1 - (j - jobs)];
            if (c < end) list_vector(c);
        }
        __syncthreads();
        n = (int)sh.n;
        if (n <= FEW) break;
        sort_list<NT>(sh.list, n < CANDIDATES ? n : CANDIDATES);
        if (n <= CANDIDATES) break;
        if (t == 0) sh.bound = sh.list[a.top - 1], sh.n_winners = sh.n_readers = sh.n = 0;
    }
    if (n > FEW) {  // sorted
        if (t < a.top) put_top(a, row, t, sh.list[t], largest, log_mass, inv_t, keys);
        return;
    }
    if (t < n) {
        const int rank = rank_in_list(sh.list, n, sh.list[t]);
        if (rank < a.top) put_top(a, row, rank, sh.list[t], largest, log_mass, inv_t, keys);
    }
    if (t >= n && t < a.top) put_top(a, row, t, 0, largest, log_mass, inv_t, keys);
}

// A row's slices together: one workgroup a row.
template <typename T, bool MASK>
__global__ __launch_bounds__(JOIN_NT) void k_join_logprobs(ScoreArgs a, int slices, const Part *parts,
                                                            const uint64_t *keys) {
    __shared__ uint64_t list[JOIN_KEYS];
    __shared__ uint32_t slots[JOIN_NT / 64];
    __shared__ float sums[2][JOIN_NT / 64];
    const int t = threadIdx.x;
    const int64_t row = a.first + blockIdx.x;
    const T *z = (const T *)a.logits + row * a.stride;
    const uint8_t *allowed = MASK ? a.allowed + row * a.allowed_stride : nullptr;
    const float inv_t = inverse_temperature(a.temperature, row), scale = inv_t * LOG2E;
    const Given given = given_token<T, MASK>(a, row, z, allowed);
    Part p{-INFINITY, 0, 0, 0};
    if (t < slices) p = parts[row * slices + t];
    for (int i = t; i < slices * a.top; i += JOIN_NT) list[i] = keys[row * slices * a.top + i];
    const float m = of_order_bits(row_all<JOIN_NT>(order_bits(p.m), slots, Larger{}));
    Mass s{0, p.mass, p.moment};
    s.shift(fmaxf(distance_times(p.m, m, scale), LEAST));
    row_sums<JOIN_NT>(s.mass, s.moment, sums[0], sums[1]);
    const bool some = s.mass > 0;
    const float log_mass = some ? logf(s.mass) : -INFINITY, largest = some ? m : -INFINITY;
    if (t == 0) put_score(a, row, given, largest, log_mass, s.moment / s.mass, inv_t);
    if (!a.top) return;
    // Bounds that `top` keys pass: a slice's last, and the least of the slices' keys at a place that makes `top`
    // of them together.
    __shared__ uint64_t ends[2][JOIN_NT / 64];
    uint64_t last = 0, least = 0;
    if (t < slices) last = list[t * a.top + a.top - 1], least = ~list[t * a.top + (a.top - 1) / slices];
    last = row_all<JOIN_NT>(last, ends[0], Larger{});
    least = ~row_all<JOIN_NT>(least, ends[1], Larger{});
    const uint64_t bound = last > least ? last : least;
    // Each slice's keys fall: a key's place among all is where it would stand in each of them.
    for (int i = t; i < slices * a.top; i += JOIN_NT) {
        const uint64_t key = list[i];
        if (key < bound) continue;
        int rank = i % a.top;
        for (int k = 0; k < slices && rank < a.top; k++) {
            if (k == i / a.top) continue;
            int low = 0, high = a.top;  // the first `low` are larger
            while (low < high) {
                const int mid = (low + high) / 2;
                if (list[k * a.top + mid] > key || (list[k * a.top + mid] == key && k < i / a.top)) low = mid + 1;
                else high = mid;
            }
            rank += low;
        }
        if (rank < a.top) put_top(a, row, rank, key, largest, log_mass, inv_t, nullptr);
    }
}

// ------------------------------------------------------------------ gradient

struct ScoreGradArgs {
    const void *logits;
    const int64_t *tokens;
    const float *temperature, *entropy, *largest, *log_mass, *dlogprob, *dentropy;
    const uint8_t *allowed;
    void *dlogits;
    int64_t stride, allowed_stride, out_stride;
    int vocab;
};
// A piece of a row for a workgroup, GRAD_EACH vectors a thread.  With lp = ln 2 x, x = z A - B,
//   dz = p (c0 + c1 x) + [token] dlogprob / temperature,  p = 2^x,
// of which a row's constants are worked out first (B in 64 bits; what its rounding to 32 leaves is in c0 and c1).
// Where they have no room, x comes from distances as above, and 1 / temperature is multiplied last: at 1e-38 it leaves
// the range of 32 bits with a term of 4, where p is 1 and the terms' sum 0.
// Bound by memory: 4096 x 32768 bf16 88 us for 537 MB (6.1 TB/s, past the caches); 333 x 50021 f16 under a mask 18 us
// for 83 MB, in rows that start at odd elements.
constexpr int GRAD_EACH = 4, GRAD_PIECE = 256 * 8 * GRAD_EACH;
template <typename T, bool MASK, bool STREAM>
__global__ __launch_bounds__(256) void k_token_logprobs_grad(ScoreGradArgs a, int64_t last, uint32_t pieces) {
    // from the last row on: the loss has just read those, and the last-level cache may hold them
    const int64_t row = last - blockIdx.x / pieces;
    const T *z = (const T *)a.logits + row * a.stride;
    T *out = (T *)a.dlogits + row * a.out_stride;
    const uint8_t *allowed = MASK ? a.allowed + row * a.allowed_stride : nullptr;
    const float inv_t = inverse_temperature(a.temperature, row), m = a.largest[row], log_mass = a.log_mass[row];
    const float h = a.entropy[row], dh = a.dentropy ? a.dentropy[row] : 0.0f;
    const int64_t token = a.tokens[row];
    float dl = 0;
    if (a.dlogprob && token >= 0 && token < a.vocab && to_f32(z[token]) > -INFINITY && (!MASK || allowed[token]))
        dl = a.dlogprob[row];
    const int begin = (int)(blockIdx.x % pieces) * GRAD_PIECE + threadIdx.x * 8;
    const float scale = inv_t * LOG2E;
    const double exact = (double)m * scale + (double)log_mass * 1.4426950408889634074;
    const float b = (float)exact;
    const float off = (float)(exact - b), k = -__builtin_amdgcn_exp2f(-off) * inv_t;
    Logits<T, MASK> v[GRAD_EACH];
#pragma unroll
    for (int j = 0; j < GRAD_EACH; j++) {
        const int c = begin + j * 2048;
        if (c + 8 <= a.vocab) v[j].template fetch<STREAM>(z, allowed, c);
        else if (c < a.vocab) v[j].fetch(z, allowed, c, a.vocab);
    }
    const float c0 = k * (dl + dh * (h - LN2 * off)), c1 = k * dh * LN2, given = dl * inv_t;
    // nothing below overflows, not even for x = LEAST, whose p is 0 (NaN: no)
    const bool room = fabsf(b) < ROOM && fabsf(c0) + fabsf(LEAST * c1) + fabsf(given) < 0x1p126f;
#pragma unroll
    for (int j = 0; j < GRAD_EACH; j++) {
        const int c = begin + j * 2048;
        if (c >= a.vocab) break;
        float f[8];
        v[j].widen(c, a.vocab, f);
        if (room) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float x = fmaxf(__builtin_fmaf(f[i], scale, -b), LEAST);
                f[i] = __builtin_amdgcn_exp2f(x) * __builtin_fmaf(c1, x, c0);
            }
            if ((uint64_t)(token - c) < 8) {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    if (c + i == token) f[i] += given;
            }
        } else {
            // the terms cancel before 1 / temperature comes to them
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float lp = fmaxf(distance_times(f[i], m, inv_t) - log_mass, LEAST);
                const float e = f[i] > -INFINITY ? __builtin_amdgcn_exp2f(lp * LOG2E) : 0.0f;  // 0 at the bound
                const float g = e > 0.0f ? -e * (dl + dh * (lp + h)) : 0.0f;
                f[i] = (c + i == token ? g + dl : g) * inv_t;
            }
        }
        Piece<T, 8>::template store<STREAM>(out + c, a.vocab - c, f);
    }
}

// ------------------------------------------------------------------ launches

template <typename F> int by_mask(int type, bool mask, F f) {
    switch (type) {
        case CKKS_PLAIN_BF16: return mask ? f(bf16{}, Flag<true>{}) : f(bf16{}, Flag<false>{});
        case CKKS_PLAIN_F16: return mask ? f(f16{}, Flag<true>{}) : f(f16{}, Flag<false>{});
        default: return mask ? f(float{}, Flag<true>{}) : f(float{}, Flag<false>{});
    }
}
int check_score(int64_t rows, int64_t vocab) {
    if (rows < 0 || rows >= (int64_t)1 << 31 || vocab < 1) return CKKS_EINVAL;
    return vocab > (int64_t)1 << 24 ? CKKS_EUNSUPPORTED : CKKS_OK;
}
// Logits that the last-level cache (256 MB) does not hold beside their gradient go past the caches (log probabilities
// and gradient: 4096 x 32768 bf16 132 us, else 152; 1024 x 131072 134, else 152); others do not (512 x 32768 f32 40 us,
// past the caches 42; 333 x 50021 f16 under a mask 34, past them 38).
bool past_caches(int64_t rows, int64_t vocab, size_t size) { return rows * vocab * (int64_t)size > (int64_t)128 << 20; }
// Slices of a row: a workgroup for each compute unit where there are few rows, none of less than 32768 logits
// (16 x 131072 bf16 top 20: 13.7 us with four slices, 15.0 with one, 19.3 with 16; 4 x 32768 f32 top 5: 7.5 us, with
// four about 11; 200 x 131072: 15.5 us, with two 19.9).
int64_t score_slices(int64_t rows, int64_t vocab) {
    const int64_t most = vocab / 32768, want = rows ? 256 / rows : 1;
    const int64_t n = want < most ? want : most;
    return n < 1 ? 1 : n < MAX_SLICES ? n : MAX_SLICES;
}
struct Range {
    const void *p;
    size_t n;
    Range(const void *p, int64_t n) : p(p), n((size_t)n) {}
};
// the arrays that both calls read
int check_score_inputs(int type, const void *logits, int64_t stride, const int64_t *tokens, const float *temperature,
                       const uint8_t *allowed, int64_t allowed_stride, int64_t vocab) {
    if (int e = check_matrix(logits, stride, vocab, type_size(type))) return e;
    if (!tokens || (allowed && allowed_stride < vocab)) return CKKS_EINVAL;
    return at(tokens, 8) && at(temperature, 4) ? CKKS_OK : CKKS_EALIGN;
}

}  // namespace ckks_plain

using namespace ckks_plain;

extern "C" int ckks_plain_token_logprobs_workspace_size(int64_t rows, int64_t vocab, int64_t top, size_t *bytes) {
    if (!bytes || top < 0) return CKKS_EINVAL;
    if (int e = check_score(rows, vocab)) return e;
    if (top > CKKS_PLAIN_MAX_TOP) return CKKS_EUNSUPPORTED;
    const int64_t slices = score_slices(rows, vocab);
    *bytes = slices > 1 ? (size_t)(rows * slices) * (sizeof(Part) + top * 8) : 0;
    return CKKS_OK;
}

extern "C" int ckks_plain_token_logprobs(int type, const void *logits, int64_t logits_stride, const int64_t *tokens,
                                         const float *temperature, const uint8_t *allowed, int64_t allowed_stride,
                                         int64_t rows, int64_t vocab, int64_t top, float *logprob, float *entropy,
                                         float *largest, float *log_mass, int64_t *top_token, float *top_logprob,
                                         void *ws, size_t ws_bytes, void *stream) {
    size_t need;
    if (!type_ok(type)) return CKKS_EINVAL;
    if (int e = ckks_plain_token_logprobs_workspace_size(rows, vocab, top, &need)) return e;
    if (rows == 0) return CKKS_OK;
    const size_t z = type_size(type);
    if (int e = check_score_inputs(type, logits, logits_stride, tokens, temperature, allowed, allowed_stride, vocab))
        return e;
    if (!logprob || !entropy || !largest || !log_mass || (top > 0) != (top_token != nullptr) ||
        (top > 0) != (top_logprob != nullptr))
        return CKKS_EINVAL;
    if (!at(logprob, 4) || !at(entropy, 4) || !at(largest, 4) || !at(log_mass, 4) || !at(top_token, 8) ||
        !at(top_logprob, 4))
        return CKKS_EALIGN;
    const Range in[4] = {{logits, (int64_t)span(rows, logits_stride, vocab, z)}, {tokens, rows * 8}, {temperature, rows * 4},
                         {allowed, (int64_t)span(rows, allowed_stride, vocab, 1)}};
    const Range out[7] = {{logprob, rows * 4}, {entropy, rows * 4}, {largest, rows * 4}, {log_mass, rows * 4},
                          {top_token, rows * top * 8}, {top_logprob, rows * top * 4}, {ws, (int64_t)need}};
    for (int i = 0; i < 7; i++) {
        for (const Range &r : in)
            if (overlap(out[i].p, out[i].n, r.p, r.n)) return CKKS_EINVAL;
        for (int j = 0; j < i; j++)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return CKKS_EINVAL;
    }
    if (need && (!ws || ws_bytes < need)) return CKKS_EWORKSPACE;
    if (!at(ws, 16)) return CKKS_EALIGN;
    ScoreArgs a{logits, tokens, temperature, allowed, logits_stride, allowed_stride, 0, (int)vocab, (int)top,
                logprob, entropy, largest, log_mass, top_token, top_logprob};
    return by_mask(type, allowed != nullptr, [&](auto ty, auto mask) {
        typedef decltype(ty) T;
        constexpr bool MASK = decltype(mask)::value;
        const int slices = (int)score_slices(rows, vocab);
        const int slice = (int)round_up((vocab + slices - 1) / slices, 8);
        Part *parts = slices > 1 ? (Part *)ws : nullptr;
        uint64_t *keys = slices > 1 && top ? (uint64_t *)(parts + rows * slices) : nullptr;
        return in_parts(rows, 512 * slices, [&](int64_t first, int64_t n) {
            a.first = first;
            const dim3 grid((uint32_t)n, slices);
            auto go = [&](auto alternatives, auto past, auto threads) {
                constexpr int NT = decltype(threads)::value;
                k_token_logprobs<T, MASK, decltype(alternatives)::value, decltype(past)::value, NT>
                    <<<grid, NT, 0, (hipStream_t)stream>>>(a, slice, parts, keys);
                return launched();
            };
            // 512 threads where a unit has one workgroup (1 x 262144 bf16 top 64 22 us, with 256 35) and for long rows
            // (2048 x 131072 bf16 top 20 96 us, with 256 99), 256 for others (512 x 32768 f16 top 20 11.9 us, with 512
            // 12.8; 600 x 65536 21.2 and 22.6; 900 x 65536 28.5 and 34.2; 2048 x 65536 55.5 and 55.5; 4096 x 4001 top 5 22
            // and 32).  The rule goes by length alone: between a row a unit and four, long rows without a mask would be
            // faster with 256 (600 x 131072 35.9, with 512 37.8; 900 45.8 and 53.5), masked ones with 512 (333 x 50021
            // 20.9, with 512 19.8; 300 x 65536 22.3 and 21.8; 600 x 131072 53.0 and 49.6).
            auto go2 = [&](auto alternatives, auto past) {
                return n * slices <= 256 || slice > 65536 ? go(alternatives, past, Int<512>{}) : go(alternatives, past, Int<256>{});
            };
            const bool past = past_caches(rows, vocab, z);
            int e = top ? past ? go2(Flag<true>{}, Flag<true>{}) : go2(Flag<true>{}, Flag<false>{})
                        : past ? go2(Flag<false>{}, Flag<true>{}) : go2(Flag<false>{}, Flag<false>{});
            if (e) return e;
            if (slices == 1) return CKKS_OK;
            k_join_logprobs<T, MASK><<<dim3((uint32_t)n), JOIN_NT, 0, (hipStream_t)stream>>>(a, slices, parts, keys);
            return launched();
        });
    });
}

extern "C" int ckks_plain_token_logprobs_grad(int type, const void *logits, int64_t logits_stride,
                                              const int64_t *tokens, const float *temperature, const uint8_t *allowed,
                                              int64_t allowed_stride, int64_t rows, int64_t vocab,
                                              const float *entropy, const float *largest, const float *log_mass,
                                              const float *dlogprob, const float *dentropy, void *dlogits,
                                              int64_t dlogits_stride, void *stream) {
    if (!type_ok(type)) return CKKS_EINVAL;
    if (int e = check_score(rows, vocab)) return e;
    if (rows == 0) return CKKS_OK;
    const size_t z = type_size(type);
    if (int e = check_score_inputs(type, logits, logits_stride, tokens, temperature, allowed, allowed_stride, vocab))
        return e;
    if (!entropy || !largest || !log_mass) return CKKS_EINVAL;
    if (int e = check_matrix(dlogits, dlogits_stride, vocab, z)) return e;
    const int64_t r4 = rows * 4;
    const size_t ob = span(rows, dlogits_stride, vocab, z);
    const Range in[9] = {{logits, (int64_t)span(rows, logits_stride, vocab, z)}, {tokens, rows * 8}, {temperature, r4},
                         {allowed, (int64_t)span(rows, allowed_stride, vocab, 1)}, {entropy, r4}, {largest, r4},
                         {log_mass, r4}, {dlogprob, r4}, {dentropy, r4}};
    for (const Range &r : in)
        if (overlap(dlogits, ob, r.p, r.n)) return CKKS_EINVAL;
    for (const float *p : {entropy, largest, log_mass, dlogprob, dentropy})
        if (!at(p, 4)) return CKKS_EALIGN;
    const ScoreGradArgs a{logits, tokens, temperature, entropy, largest, log_mass, dlogprob, dentropy, allowed,
                          dlogits, logits_stride, allowed_stride, dlogits_stride, (int)vocab};
    return by_mask(type, allowed != nullptr, [&](auto ty, auto mask) {
        const uint32_t pieces = (uint32_t)((vocab + GRAD_PIECE - 1) / GRAD_PIECE);
        return in_parts(rows, 256 * (int)pieces, [&](int64_t first, int64_t n) {
            auto go = [&](auto past) {
                k_token_logprobs_grad<decltype(ty), decltype(mask)::value, decltype(past)::value>
                    <<<dim3((uint32_t)(n * pieces)), 256, 0, (hipStream_t)stream>>>(a, rows - 1 - first, pieces);
            };
            past_caches(rows, vocab, z) ? go(Flag<true>{}) : go(Flag<false>{});
            return launched();
        });
    });
}
