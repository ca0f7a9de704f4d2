// k_token_logprobs and k_join_logprobs (csrc/plain/logprob.hip), device code on the host, where a logit's distance to the
// largest leaves the range of 32 bits and its quotient by the temperature does not, or the temperature is infinite: against
// the definition in 64 bits, where an infinite logit outweighs every finite one.
#include <algorithm>

#include "hip/hip_runtime.h"

#define __builtin_nontemporal_load(p) (*(p))
#define __builtin_nontemporal_store(v, p) (*(p) = (v))
// moves within a row of 16 lanes that the header does not have
static Index gridDim;
static uint32_t update_dpp(uint32_t none, uint32_t v, int ctrl, int rows) {
    const int l = threadIdx.x % host::LANES;
    const int from = ctrl == 0xb1 ? l ^ 1 : ctrl == 0x4e ? l ^ 2 : ctrl == 0x141 ? l ^ 7 : -1;
    if (from < 0) return host::update_dpp(none, v, ctrl, rows);
    return host::exchange(v, [&](const uint32_t *wave) { return wave[from]; });
}
static int shfl_xor(int v, int far) {
    return (int)host::exchange((uint32_t)v, [&](const uint32_t *wave) { return wave[(threadIdx.x % host::LANES) ^ far]; });
}
#define __shfl_xor shfl_xor
#undef __builtin_amdgcn_update_dpp
#define __builtin_amdgcn_update_dpp(none, v, ctrl, rows, banks, bound) \
    ((int)update_dpp((uint32_t)(none), (uint32_t)(v), ctrl, rows))
#define __builtin_amdgcn_fmed3f(a, b, c) std::max(std::min(a, b), std::min(std::max(a, b), c))
#include "device.inc"

using namespace ckks_plain;

constexpr int V = 50, TOP = 4;
static int failures, checks;

static void check(const char *what, const std::vector<float> &z, float temperature, int token, int slices) {
    std::vector<int> some;
    for (int i = 0; i < V; i++)
        if (z[i] > -INFINITY) some.push_back(i);
    std::stable_sort(some.begin(), some.end(), [&](int a, int b) { return z[a] > z[b]; });
    const double m = z[some[0]];
    auto x = [&](int i) {
        return z[i] == m ? 0.0 : m == INFINITY || !(z[i] > -INFINITY) ? -INFINITY : (z[i] - m) / temperature;
    };
    double mass = 0, entropy = 0, far = 0;
    for (int i : some) mass += std::exp(x(i));
    const double log_mass = std::log(mass);
    for (int i : some) {
        const double p = std::exp(x(i) - log_mass);
        if (p > 0) entropy -= p * (x(i) - log_mass), far -= p * x(i);
    }
    const int64_t tokens = token;
    float logprob, e, l, lm, logs[TOP];
    int64_t tops[TOP];
    Part parts[4];
    uint64_t keys[4 * TOP];
    const ScoreArgs a{z.data(), &tokens, &temperature, nullptr, V, 0, 0, V, TOP, &logprob, &e, &l, &lm, tops, logs};
    gridDim.y = slices;
    bool done = true;
    for (unsigned y = 0; y < (unsigned)slices && done; y++) {
        blockIdx = {0, y, 0};
        done = host::run(256, 100000, [&] {
            k_token_logprobs<float, false, true, false, 256>(a, slices > 1 ? 24 : 56, slices > 1 ? parts : nullptr,
                                                              slices > 1 ? keys : nullptr);
        });
    }
    blockIdx = {0, 0, 0};
    if (slices > 1 && done)
        done = host::run(JOIN_NT, 100000, [&] { k_join_logprobs<float, false>(a, slices, parts, keys); });
    // a quotient is rounded four times (difference or its two parts, reciprocal, product), exp2 and the sums of 50 terms
    // less than 60 times in all; what lies below the least number of 32 bits, -2^128 (1 - 2^-24), by more than half a step
    // of it, 2^103, rounds to -infinity there
    auto off = [&](double got, double want, double of) {
        if (want < -0x1p128 + 0x1p103) want = -INFINITY;
        return want == -INFINITY ? got != want : !(std::fabs(got - want) <= 0x1p-24 * (64 + 4 * far + 4 * of + 4 * log_mass));
    };
    bool bad = !done || l != (float)m || off(lm, log_mass, 0) ||
               off(logprob, x(token) - log_mass, x(token) > -INFINITY ? std::fabs(x(token)) : 0) ||
               off(e, entropy, 4 * far + log_mass);
    for (int i = 0; i < TOP && !bad; i++)
        bad = tops[i] != some[i] || off(logs[i], x(some[i]) - log_mass, x(some[i]) > -INFINITY ? std::fabs(x(some[i])) : 0);
    if (bad)
        printf("%s at %g, %d slices: logprob %g for %g, entropy %g for %g, log mass %g for %g, then %g for %g\n", what,
               temperature, slices, logprob, x(token) - log_mass, e, entropy, lm, log_mass, logs[1], x(some[1]) - log_mass);
    checks++;
    failures += bad;
}

int main() {
    for (float temperature : {1.0f, 1e30f, 1e38f, 2e38f, 3.4e38f, INFINITY})
        for (int slices : {1, 3})
            for (int token : {0, 13, 31, 49}) {
                std::vector<float> z(V);
                for (int i = 0; i < V; i++) z[i] = (float)(i % 7) * 0.3f - 1;
                check("small", z, temperature, token, slices);
                for (int i = 0; i < V; i++) z[i] = (float)(i % 7 - 3) * 1.1e38f;
                check("the whole range", z, temperature, token, slices);
                z[20] = NAN, z[44] = -INFINITY;
                check("the whole range beside no number", z, temperature, token, slices);
                for (int i = 0; i < V; i++) z[i] = i < 24 ? 3e38f : -3e38f;
                check("slices apart", z, temperature, token, slices);
                for (int i = 0; i < V; i++) z[i] = i == 30 ? 3.0f : -3.4e38f;
                check("the lowest value", z, temperature, token, slices);
                for (int i = 0; i < V; i++) z[i] = (float)(i % 5);
                z[13] = INFINITY;
                check("infinite", z, temperature, token, slices);
                z[49] = INFINITY;
                check("two infinite", z, temperature, token, slices);
            }
    printf(failures ? "distances: %d of %d wrong\n" : "distances: ok\n", failures, checks);
    return failures != 0;
}
