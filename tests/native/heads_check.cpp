// A workgroup of k_head_norm_rotate and k_head_grad (csrc/plain/heads.hip) with several steps of tokens, the last one
// short, device code on the host, against the definition in 64 bits: the angles in LDS belong to the step that reads them,
// the head fetched ahead to the next one.
#include <algorithm>

#include "hip/hip_runtime.h"

#define __builtin_nontemporal_load(p) (*(p))
#define __builtin_nontemporal_store(v, p) (*(p) = (v))
struct float2 {
    float x, y;
};
inline void sincospif(float v, float *s, float *c) { *s = (float)std::sin(M_PI * v), *c = (float)std::cos(M_PI * v); }
static uint32_t update_dpp(uint32_t none, uint32_t v, int ctrl, int rows) {
    const int l = threadIdx.x % host::LANES;
    const int from = ctrl == 0xb1 ? l ^ 1 : ctrl == 0x4e ? l ^ 2 : ctrl == 0x141 ? l ^ 7 : ctrl == 0x140 ? l ^ 15 : -1;
    if (from < 0) return host::update_dpp(none, v, ctrl, rows);
    return host::exchange(v, [&](const uint32_t *wave) { return wave[from]; });
}
static float shfl_xor(float v, int far) {
    return __uint_as_float(host::exchange(__float_as_uint(v), [&](const uint32_t *wave) {
        return wave[(threadIdx.x % host::LANES) ^ far];
    }));
}
#define __shfl_xor shfl_xor
#undef __builtin_amdgcn_update_dpp
#define __builtin_amdgcn_update_dpp(none, v, ctrl, rows, banks, bound) \
    ((int)update_dpp((uint32_t)(none), (uint32_t)(v), ctrl, rows))
#include "device.inc"

using namespace ckks_plain;

// 16 heads of 128 in 32 bits: 16 lanes a head, so each step's heads take whole workgroups
constexpr int H = 16, D = 128, R = 24;
static uint32_t state = 99;
static float rnd() { return (float)(int)(state = state * 1664525u + 1013904223u) * 0x1p-30f; }

static bool far(const char *what, const std::vector<float> &got, const std::vector<double> &want) {
    for (size_t i = 0; i < got.size(); i++)
        if (!(std::fabs(got[i] - want[i]) < 1e-5)) {
            printf("%s: element %zu is %g for %g\n", what, i, got[i], want[i]);
            return true;
        }
    return false;
}

static int check(int tokens, int step, bool interleaved) {
    std::vector<float> x(tokens * H * D), dy(x.size()), w(D), freq(R), y(x.size(), NAN), dx(x.size(), NAN), part(D, NAN);
    std::vector<int64_t> pos(tokens);
    for (float &v : x) v = rnd();
    for (float &v : dy) v = rnd();
    for (float &v : w) v = 1 + 0.1f * rnd();
    for (int i = 0; i < R; i++) freq[i] = std::pow(0.7f, i);
    for (int t = 0; t < tokens; t++) pos[t] = t * 13 - 20;
    HeadArgs a{};
    a.side[0] = {x.data(), w.data(), dy.data(), y.data(), nullptr, {H * D, D}, {H * D, D}, {H * D, D}, H, 1};
    a.positions = pos.data(), a.inv_freq = freq.data(), a.tokens = tokens, a.span = tokens;
    a.half = D / 2, a.r = R, a.step = step, a.log_l = 4, a.eps = 1e-6f, a.inv_dim = 1.0f / D, a.interleaved = interleaved;
    blockIdx = {0, 0, 0};
    if (!host::run(256, 100000, [&] { k_head_norm_rotate<float, 4, 1>(a); })) return 1;
    a.side[0].out = dx.data(), a.side[0].part = part.data();
    if (!host::run(256, 100000, [&] { k_head_grad<float, 4, 1>(a); })) return 1;

    std::vector<double> want(x.size()), want_dx(x.size()), want_part(D, 0.0);
    for (int t = 0; t < tokens; t++)
        for (int h = 0; h < H; h++) {
            const int at = (t * H + h) * D;
            double sum = 0, dot = 0, n[D], back[D];
            for (int i = 0; i < D; i++) sum += (double)x[at + i] * x[at + i];
            const double r = 1 / std::sqrt(sum / D + 1e-6);
            for (int i = 0; i < D; i++) n[i] = x[at + i] * r * w[i], back[i] = dy[at + i], want[at + i] = n[i];
            for (int i = 0; i < R; i++) {
                const int p = interleaved ? 2 * i : i, q = interleaved ? 2 * i + 1 : i + R;
                const double f = (double)pos[t] * freq[i], c = std::cos(f), s = std::sin(f);
                want[at + p] = n[p] * c - n[q] * s, want[at + q] = n[q] * c + n[p] * s;
                back[p] = dy[at + p] * c + dy[at + q] * s, back[q] = dy[at + q] * c - dy[at + p] * s;
            }
            for (int i = 0; i < D; i++) dot += back[i] * w[i] * x[at + i] * r / D;
            for (int i = 0; i < D; i++) {
                want_dx[at + i] = r * (back[i] * w[i] - x[at + i] * r * dot);
                want_part[i] += back[i] * x[at + i] * r;
            }
        }
    // numbers of about 1, at most 20 a sum in order: far from 1e-5 by roundings of 2^-24
    for (double &v : want_part) v /= tokens * H;
    for (float &v : part) v /= (float)(tokens * H);
    const bool bad = far("forward", y, want) || far("gradient", dx, want_dx) || far("weight", part, want_part);
    if (bad) printf("%d tokens, %d at a time, interleaved %d\n", tokens, step, interleaved);
    return bad;
}

int main() {
    int bad = 0;
    for (bool interleaved : {false, true})
        for (int step : {1, 2, 4})
            for (int tokens : {1, 3, 4, 9, 13}) bad += check(tokens, step, interleaved);
    printf(bad ? "heads: wrong\n" : "heads: ok\n");
    return bad;
}
