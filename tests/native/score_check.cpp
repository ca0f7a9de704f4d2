// The alternatives of k_token_logprobs (csrc/plain/logprob.hip), device code on the host: rows in orders that
// overflow its list, masks, and slices joined, against a sort.  Buffers end where the row does.
#include <algorithm>
#include <memory>

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

static uint32_t state = 12345;
static uint32_t rnd() { return state = state * 1664525u + 1013904223u; }

static int failures;
static void check(const char *what, int vocab, int top, int slices, bool masked, float (*value)(int, int)) {
    std::unique_ptr<float[]> z(new float[vocab]);
    std::unique_ptr<uint8_t[]> ok(new uint8_t[vocab]);
    std::vector<int> want;
    for (int i = 0; i < vocab; i++) {
        z[i] = value(i, vocab);
        ok[i] = !masked || rnd() >> 30 == 0;
        if (z[i] > -INFINITY && ok[i]) want.push_back(i);
    }
    std::stable_sort(want.begin(), want.end(), [&](int a, int b) { return z[a] > z[b]; });
    const int64_t token = 0;
    float logprob, entropy, largest, log_mass;
    std::unique_ptr<int64_t[]> tops(new int64_t[top]);
    std::unique_ptr<float[]> logs(new float[top]);
    std::unique_ptr<Part[]> parts(new Part[slices]);
    std::unique_ptr<uint64_t[]> keys(new uint64_t[slices * top]);
    std::fill(&tops[0], &tops[0] + top, -7);
    ScoreArgs a{z.get(), &token, nullptr, ok.get(), vocab, vocab, 0, vocab, top, &logprob, &entropy, &largest, &log_mass,
                tops.get(), logs.get()};
    const int slice = (vocab / slices + 8) / 8 * 8;
    gridDim.y = slices;
    bool done = true;
    for (unsigned y = 0; y < (unsigned)slices && done; y++) {
        blockIdx = {0, y, 0};
        Part *p = slices > 1 ? parts.get() : nullptr;
        uint64_t *k = slices > 1 ? keys.get() : nullptr;
        done = masked ? host::run(512, 20000000, [&] { k_token_logprobs<float, true, true, false, 512>(a, slice, p, k); })
                      : host::run(256, 20000000, [&] { k_token_logprobs<float, false, true, false, 256>(a, slice, p, k); });
    }
    blockIdx = {0, 0, 0};
    if (slices > 1 && done)
        done = host::run(JOIN_NT, 20000000, [&] { k_join_logprobs<float, true>(a, slices, parts.get(), keys.get()); });
    int bad = !done;
    for (int i = 0; i < top && !bad; i++) bad = tops[i] != (i < (int)want.size() ? want[i] : -1);
    double mass = 0;
    for (int i : want) mass += std::exp((double)z[i] - z[want[0]]);
    if (!bad) bad = want.empty() ? log_mass != -INFINITY : std::fabs(log_mass - std::log(mass)) > 1e-4;
    if (bad) failures++, printf("%s vocab %d top %d slices %d masked %d: wrong\n", what, vocab, top, slices, masked);
    fflush(stdout);
}

int main() {
    auto noise = [](int, int) { return (float)(int)rnd() * 1e-9f; };
    auto equal = [](int, int) { return 2.0f; };
    auto rising = [](int i, int) { return i * 1e-3f; };
    auto falling = [](int i, int) { return -i * 1e-3f; };
    // what one group of threads reads is large, and rises: all of it passes the first bound
    auto group = [](int i, int n) { return i / 8 % 256 < 8 ? 10 + i * 1e-4f : -i * 1e-4f; };
    auto lanes = [](int i, int n) { return i / 8 % 8 == 3 ? 10 + i * 1e-4f : -INFINITY; };
    auto few = [](int i, int n) { return i % 1000 == 7 ? 1.0f : -INFINITY; };
    auto none = [](int, int) { return (float)NAN; };
    auto steps = [](int i, int) { return (float)(i % 3); };
    for (int top : {1, 5, 64}) {
        for (int vocab : {1, 7, 1000, 4096, 9001, 40003}) {
            check("noise", vocab, top, 1, false, noise);
            check("equal", vocab, top, 1, false, equal);
            check("rising", vocab, top, 1, false, rising);
            check("steps", vocab, top, 1, true, steps);
        }
        for (bool masked : {false, true}) {
            check("falling", 20001, top, 1, masked, falling);
            check("group", 70001, top, 1, masked, group);
            check("lanes", 70001, top, 1, masked, lanes);
            check("few", 20001, top, 1, masked, few);
            check("none", 20001, top, 1, masked, none);
        }
        check("noise", 40003, top, 3, true, noise);
        check("equal", 40003, top, 3, true, equal);
        check("few", 40003, top, 4, true, few);
        check("none", 40003, top, 2, true, none);
    }
    printf(failures ? "score: %d wrong\n" : "score: ok\n", failures);
    return failures != 0;
}
