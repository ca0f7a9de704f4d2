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
// The distance of a logit to the largest, 0 also where both are infinite.
__device__ __forceinline__ float distance(float z, float largest) { return z == largest ? 0.0f : z - largest; }

// Logits c ... c + 7 of a row, -infinity where there is no possible token.
template <typename T, bool MASK>
__device__ __forceinline__ void fetch_logits(const T *z, const uint8_t *allowed, int64_t c, int64_t vocab,
                                             float (&f)[8]) {
    Eight<T> e;
    Eight<int8_t> ok;
    e.fetch(z + c, vocab - c);
    if constexpr (MASK) ok.fetch((const int8_t *)allowed + c, vocab - c);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        f[i] = e.at(i);
        if (!(c + i < vocab) || !(f[i] > -INFINITY) || (MASK && !ok.v[0][i])) f[i] = -INFINITY;
    }
}

// A workgroup a row: its largest logit, then its sums, then one read for each alternative.
constexpr int SCORE_NT = 1024;
template <typename T, bool MASK>
__global__ __launch_bounds__(SCORE_NT) void k_token_logprobs(ScoreArgs a) {
    __shared__ uint64_t buf[2][SCORE_NT / 64];
    __shared__ float sums[2][SCORE_NT / 64];
    const int64_t row = a.first + blockIdx.x;
    const T *z = (const T *)a.logits + row * a.stride;
    const uint8_t *allowed = MASK ? a.allowed + row * a.allowed_stride : nullptr;
    auto best_under = [&](uint64_t bound, uint64_t *at) {  // the largest key below it (0: none)
        uint64_t best = 0;
        for (int c = threadIdx.x * 8; c < a.vocab; c += SCORE_NT * 8) {
            float f[8];
            fetch_logits<T, MASK>(z, allowed, c, a.vocab, f);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint64_t key = (uint64_t)order_bits(f[i]) << 32 | (uint32_t)~(c + i);
                if (f[i] > -INFINITY && key < bound && key > best) best = key;
            }
        }
        return row_all<SCORE_NT>(best, at, Larger{});
    };
    const uint64_t first = best_under(~(uint64_t)0, buf[0]);
    const float m = first ? of_order_bits((uint32_t)(first >> 32)) : -INFINITY;
    const float inv_t = inverse_temperature(a.temperature, row), scale = inv_t * LOG2E;
    float mass = 0, moment = 0;
    if (first)
        for (int c = threadIdx.x * 8; c < a.vocab; c += SCORE_NT * 8) {
            float f[8];
            fetch_logits<T, MASK>(z, allowed, c, a.vocab, f);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float x = fmaxf(distance(f[i], m) * scale, -200.0f);  // 2^-200 is 0
                const float e = f[i] > -INFINITY ? __builtin_amdgcn_exp2f(x) : 0.0f;
                mass += e;
                moment += e * x;
            }
        }
    row_sums<SCORE_NT>(mass, moment, sums[0], sums[1]);
    const float log_mass = first ? logf(mass) : -INFINITY;
    if (threadIdx.x == 0) {
        const int64_t token = a.tokens[row];
        float lp = 0;
        if (token >= 0 && token < a.vocab) {
            const float v = to_f32(z[token]);
            const bool possible = v > -INFINITY && (!MASK || allowed[token]);
            lp = possible ? distance(v, m) * inv_t - log_mass : -INFINITY;
        }
        a.logprob[row] = lp;
        a.entropy[row] = first ? log_mass - LN2 * (moment / mass) : 0.0f;
        a.largest[row] = m;
        a.log_mass[row] = log_mass;
    }
    uint64_t key = first;
    for (int k = 0; k < a.top; k++) {
        if (threadIdx.x == 0) {
            a.top_token[row * a.top + k] = key ? (int64_t)(uint32_t)~(uint32_t)key : -1;
            a.top_logprob[row * a.top + k] =
                key ? distance(of_order_bits((uint32_t)(key >> 32)), m) * inv_t - log_mass : -INFINITY;
        }
        if (k + 1 < a.top && key) key = best_under(key, buf[(k + 1) % 2]);
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
// 2048 logits of a row for a workgroup.
template <typename T, bool MASK>
__global__ __launch_bounds__(256) void k_token_logprobs_grad(ScoreGradArgs a, int64_t first) {
    const int64_t row = first + blockIdx.x;
    const T *z = (const T *)a.logits + row * a.stride;
    const uint8_t *allowed = MASK ? a.allowed + row * a.allowed_stride : nullptr;
    const float inv_t = inverse_temperature(a.temperature, row), m = a.largest[row], log_mass = a.log_mass[row];
    const float h = a.entropy[row], dh = a.dentropy ? a.dentropy[row] : 0.0f;
    const int64_t token = a.tokens[row];
    float dl = 0;
    if (a.dlogprob && token >= 0 && token < a.vocab && to_f32(z[token]) > -INFINITY && (!MASK || allowed[token]))
        dl = a.dlogprob[row];
    const int64_t c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 8;
    if (c >= a.vocab) return;
    float f[8];
    fetch_logits<T, MASK>(z, allowed, c, a.vocab, f);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float lp = fmaxf(distance(f[i], m) * inv_t - log_mass, -200.0f);
        const float p = __builtin_amdgcn_exp2f(lp * LOG2E);  // 0 at the bound
        const float g = (c + i == token ? dl : 0.0f) - p * (dl + dh * (lp + h));
        f[i] = f[i] > -INFINITY ? g * inv_t : 0.0f;
    }
    Eight<T>::store((T *)a.dlogits + row * a.out_stride + c, a.vocab - c, f);
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
    *bytes = 0;
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
        return in_parts(rows, SCORE_NT, [&](int64_t first, int64_t n) {
            a.first = first;
            k_token_logprobs<decltype(ty), decltype(mask)::value>
                <<<dim3((uint32_t)n), SCORE_NT, 0, (hipStream_t)stream>>>(a);
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
    const bool in_place = dlogits == logits && dlogits_stride == logits_stride;
    for (int i = in_place; i < 9; i++)
        if (overlap(dlogits, ob, in[i].p, in[i].n)) return CKKS_EINVAL;
    for (const float *p : {entropy, largest, log_mass, dlogprob, dentropy})
        if (!at(p, 4)) return CKKS_EALIGN;
    const ScoreGradArgs a{logits, tokens, temperature, entropy, largest, log_mass, dlogprob, dentropy, allowed,
                          dlogits, logits_stride, allowed_stride, dlogits_stride, (int)vocab};
    return by_mask(type, allowed != nullptr, [&](auto ty, auto mask) {
        const uint32_t pieces = (uint32_t)((vocab + 2047) / 2048);
        return in_parts(rows, 256 * (int)pieces, [&](int64_t first, int64_t n) {
            k_token_logprobs_grad<decltype(ty), decltype(mask)::value>
                <<<dim3((uint32_t)n, pieces), 256, 0, (hipStream_t)stream>>>(a, first);
            return launched();
        });
    });
}
