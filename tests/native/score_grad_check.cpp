// The gradient of k_token_logprobs_grad (csrc/plain/logprob.hip), device code on the host, where 1 / temperature times a
// term has no room in 32 bits, against the definition in 64 bits.
#include "hip/hip_runtime.h"

#define __builtin_nontemporal_load(p) (*(p))
#define __builtin_nontemporal_store(v, p) (*(p) = (v))
#define __builtin_amdgcn_fmed3f(a, b, c) std::max(std::min(a, b), std::min(std::max(a, b), c))
#define __shfl_xor(v, far) (v)  // of kernels that are not run here
static Index gridDim;
#include <algorithm>
#include "device.inc"

using namespace ckks_plain;

constexpr int V = 16;
constexpr double EPS = 0x1p-24, TINY = 0x1p-126;
static int failures, checks;

// The bound: x = (z - m) / t is rounded three times, log mass and entropy once each (they are given here), exp2 and the
// products less than eight times together, so p is off by (8 + 4 |x| + 4 log mass) eps and a result by that of the
// sizes of its terms, and by eps of their sum for each of the last four steps; exp2 gives 0 below 2^-126.
template <bool MASK> static void check(const float *z, float temperature, int token, float dl, float dh) {
    const double t = std::max((double)temperature, 0x1p-127);
    double m = -INFINITY, mass = 0, entropy = 0;
    const uint8_t ok[V] = {1, 1, 1, 1, 1, 1, 1, 0, 1, 1, 1, 1, 1, 1, 1, 1};
    for (int i = 0; i < V; i++)
        if (!MASK || ok[i]) m = std::max(m, (double)z[i]);
    for (int i = 0; i < V; i++)
        if (!MASK || ok[i]) mass += std::exp((z[i] - m) / t);
    const double log_mass = std::log(mass);
    for (int i = 0; i < V; i++) {
        const double lp = (z[i] - m) / t - log_mass, p = std::exp(lp);
        if ((!MASK || ok[i]) && p > 0) entropy -= p * lp;
    }
    const int64_t tokens = token;
    const float e = (float)entropy, l = (float)m, lm = (float)log_mass;
    float got[V];
    std::fill(got, got + V, -7.0f);
    const ScoreGradArgs a{z, &tokens, &temperature, &e, &l, &lm, dl ? &dl : nullptr, dh ? &dh : nullptr, ok, got, V, V, V, V};
    blockIdx = {0, 0, 0};
    bool bad = !host::run(256, 1000, [&] { k_token_logprobs_grad<float, MASK, false>(a, 0, 1); });
    for (int i = 0; i < V && !bad; i++) {
        const bool here = i == token && (!MASK || ok[token]);
        const double x = (z[i] - m) / t, lp = x - log_mass, p = !MASK || ok[i] ? std::exp(lp) : 0;
        const double given = MASK && !ok[token] ? 0 : dl;
        const double term = p > 0 ? given + dh * (lp + entropy) : 0;
        const double size = p > 0 ? p * (std::fabs(given) + std::fabs(dh) * (std::fabs(lp) + entropy)) : 0;
        const double both = size + (here ? std::fabs(given) : 0);
        const double want = ((here ? given : 0) - p * term) / t;
        const double tol = ((12 + 4 * std::fabs(p > 0 ? x : 0) + 4 * log_mass) * EPS * both +
                            TINY * (std::fabs(given) + std::fabs(dh) * (200 + entropy))) / t + TINY;
        bad = !(got[i] >= (float)(want - tol) && got[i] <= (float)(want + tol));
        if (bad) printf("z[%d] %g of largest %g at %g, token %d, dl %g dh %g: %g for %g\n", i, z[i], m, temperature, token,
                        dl, dh, got[i], want);
    }
    checks++;
    failures += bad;
}

int main() {
    for (float temperature : {1e-45f, 1e-38f, 1e-37f, 3e-36f, 1e-30f, 1.0f, 1e30f})
        for (float largest : {0.0f, -3.0f, 5.0f})
            for (float apart : {temperature, 1.0f})
                for (float dl : {0.0f, 4.0f, 50.0f, -1e4f})
                    for (float dh : {0.0f, 1.0f, -30.0f})
                        for (int token : {0, 3, 7, 9}) {
                            float z[V];  // the largest is the third, and the last again where others are near it
                            for (int i = 0; i < V; i++) z[i] = largest - apart * (float)(i * 7 % V) * 0.37f;
                            std::swap(z[0], z[3]);
                            if (apart != 1.0f) z[V - 1] = largest;
                            check<false>(z, temperature, token, dl, dh);
                            check<true>(z, temperature, token, dl, dh);
                        }
    printf(failures ? "gradient: %d of %d wrong\n" : "gradient: ok\n", failures, checks);
    return failures != 0;
}
