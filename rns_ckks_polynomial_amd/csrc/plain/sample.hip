// sample.hip -- one token for each row of logits (include/ckks_plain.h).
#include "plain_common.h"

namespace ckks_plain {

// Tokens are ordered by one 64-bit number: the logit as an unsigned number of the same order, then
// the complement of the index; 0 stands for a token that is not possible.
__device__ __forceinline__ uint32_t order_bits(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);  // -0 orders as 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_of(float z, bool allowed, uint32_t index) {
    return allowed && z > -INFINITY ? (uint64_t)order_bits(z) << 32 | (uint32_t)~index : 0;
}

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

template <int N> __device__ __forceinline__ uint64_t block_max(uint64_t v, uint64_t *sh) {
#pragma unroll
    for (int m = 32; m; m >>= 1) {
        const uint64_t o = __shfl_xor(v, m);
        v = v > o ? v : o;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < N / 64; w++) v = v > sh[w] ? v : sh[w];
    return v;
}
template <int N> __device__ __forceinline__ uint64_t block_sum(uint64_t v, uint64_t *sh) {
#pragma unroll
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < N / 64; w++) v += sh[w];
    return v;
}

// A workgroup for each row.  Masses are whole multiples of 2^-mass_bits, so their sums are exact
// and do not depend on the order in which they are added.  The last token that stays is found by
// its order, eight bits at a time from the top: by count for top-k, then by mass for top-p.
constexpr int NT = 1024;
template <typename T> __global__ __launch_bounds__(NT) void k_sample(SampleArgs a) {
    __shared__ uint64_t sh[NT / 64], mass[256], found[3];
    __shared__ uint32_t count[256];
    const int64_t row = blockIdx.x;
    const T *z = (const T *)a.logits + row * a.logits_stride;
    const uint8_t *ok = a.allowed ? a.allowed + row * a.allowed_stride : nullptr;
    const float temp = a.temperature[row];
    const bool greedy = !(temp > 0);
    const float t = greedy ? 1.0f : temp;
    auto order = [&](int i) { return order_of(to_f32(z[i]), !ok || ok[i], i); };
    uint64_t first = 0, n = 0;
    for (int i = threadIdx.x; i < a.vocab; i += NT) {
        const uint64_t o = order(i);
        first = o > first ? o : first;
        n += o != 0;
    }
    first = block_max<NT>(first, sh);
    n = block_sum<NT>(n, sh);
    if (!first) {
        if (threadIdx.x == 0) a.token[row] = -1, a.logprob[row] = -INFINITY;
        return;
    }
    const uint32_t first_index = ~(uint32_t)first;
    const float top = to_f32(z[first_index]);
    auto part = [&](float v) { return v == top ? 0.0f : (v - top) / t; };
    auto mass_of = [&](float v) { return (uint64_t)rintf(ldexpf(expf(part(v)), a.mass_bits)); };
    uint64_t all = 0;
    for (int i = threadIdx.x; i < a.vocab; i += NT)
        if (order(i)) all += mass_of(to_f32(z[i]));
    all = block_sum<NT>(all, sh);
    uint64_t best = first;
    if (!greedy) {
        // the order of the last of the first `want` (by count), or of the last before which the mass is
        // under `want`, among those from `from` on
        auto last_of = [&](bool by_mass, uint64_t want, uint64_t from) {
            uint64_t prefix = 0, above = 0;
            for (int shift = 56; shift >= 0; shift -= 8) {
                __syncthreads();
                if (threadIdx.x < 256) mass[threadIdx.x] = 0, count[threadIdx.x] = 0;
                __syncthreads();
                for (int i = threadIdx.x; i < a.vocab; i += NT) {
                    const uint64_t o = order(i);
                    if (o < from || !o || (shift < 56 && (o >> (shift + 8)) != prefix)) continue;
                    if (by_mass)
                        atomicAdd((unsigned long long *)&mass[o >> shift & 255], (unsigned long long)mass_of(to_f32(z[i])));
                    else
                        atomicAdd(&count[o >> shift & 255], 1u);
                }
                __syncthreads();
                if (threadIdx.x == 0) {
                    int b = 255;
                    for (; b > 0; b--) {
                        const uint64_t v = by_mass ? mass[b] : count[b];
                        if (above + v >= want) break;
                        above += v;
                    }
                    found[0] = b, found[1] = above;
                }
                __syncthreads();
                prefix = prefix << 8 | found[0];
                above = found[1];
            }
            return prefix;
        };
        uint64_t last = 1;
        const int k = a.top_k ? a.top_k[row] : 0;
        if (k > 0 && (uint64_t)k < n) last = last_of(false, k, 1);
        const float p = a.top_p ? a.top_p[row] : 1.0f, m = a.min_p ? a.min_p[row] : 0.0f;
        if (p < 1) {
            uint64_t stay = 0;
            for (int i = threadIdx.x; i < a.vocab; i += NT)
                if (order(i) >= last) stay += mass_of(to_f32(z[i]));
            stay = block_sum<NT>(stay, sh);
            const double want = ceil((double)p * (double)stay);
            last = last_of(true, want < 1 ? 1 : (uint64_t)want, last);
        }
        best = 0;
        for (int i = threadIdx.x; i < a.vocab; i += NT) {
            const uint64_t o = order(i);
            if (o < last || !o) continue;
            const float d = part(to_f32(z[i]));
            if (o != first && m > 0 && !(expf(d) >= m)) continue;
            const uint64_t s = (uint64_t)order_bits(d + a.gumbel[row * a.gumbel_stride + i]) << 32 | (uint32_t)~i;
            best = s > best ? s : best;
        }
        best = block_max<NT>(best, sh);
    }
    if (threadIdx.x == 0) {
        const uint32_t token = ~(uint32_t)best;
        a.token[row] = token;
        a.logprob[row] = part(to_f32(z[token])) - (float)log((double)all * exp2(-(double)a.mass_bits));
    }
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
