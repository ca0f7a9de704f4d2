// The order of tokens (k_token_order, csrc/plain/embed.hip), device code on the host, against a stable sort: all
// tokens, one token, none, more rows than a wave lists.
#include <algorithm>

#include "hip/hip_runtime.h"
static Index gridDim;
#define __shfl(v, l) (v)  // of kernels that are not run here
#define __builtin_nontemporal_load(p) (*(p))
#define __builtin_nontemporal_store(v, p) (*(p) = (v))
#define __builtin_amdgcn_fence(order, scope) host::ballot(true)  // the wave meets
#include "device.inc"

using namespace ckks_plain;

static uint32_t state = 777;
static uint32_t rnd() { return (state = state * 1664525u + 1013904223u) >> 8; }

static int check(int rows, int vocab, int log_bins, int kind) {
    std::vector<int64_t> tokens(rows);
    for (int i = 0; i < rows; i++)
        tokens[i] = kind == 0 ? (int64_t)(rnd() % (vocab + 2)) - 1 : kind == 1 ? vocab - 1 : kind == 2 ? -5
                  : kind == 3 ? (rnd() % 3 ? vocab / 2 : 0) : vocab - 1 - (int64_t)i * vocab / rows;
    std::vector<int32_t> want;
    for (int i = 0; i < rows; i++)
        if (tokens[i] >= 0 && tokens[i] < vocab) want.push_back(i);
    std::stable_sort(want.begin(), want.end(), [&](int a, int b) { return tokens[a] < tokens[b]; });
    const int64_t n = want.size();
    std::vector<int32_t> order(rows, -9), token_of(rows, -9), starts(vocab + 1, -9);
    const TokenOrder o{order.data(), token_of.data(), starts.data()};
    for (int b = 0; b < (vocab + (1 << log_bins) - 1) >> log_bins; b++) {
        blockIdx = {(unsigned)b, 0, 0};
        if (!host::run(ORDER_NT, 20000000, [&] { k_token_order(tokens.data(), rows, vocab, log_bins, o); })) return 1;
    }
    int bad = 0;
    for (int i = 0; i < rows; i++) bad += order[i] != (i < n ? want[i] : -9);
    for (int v = 0; v <= vocab; v++)
        bad += starts[v] != std::count_if(want.begin(), want.end(), [&](int i) { return tokens[i] < v; });
    for (int i = 0; i < rows; i++) bad += token_of[i] != (i < n ? tokens[want[i]] : -9);
    if (bad) printf("rows %d vocab %d bins %d kind %d: %d wrong\n", rows, vocab, 1 << log_bins, kind, bad);
    return bad != 0;
}

int main() {
    int bad = 0;
    for (int kind = 0; kind < 5; kind++) {
        bad += check(1, 1, 0, kind);
        bad += check(300, 7, 1, kind);
        bad += check(1500, 1000, 9, kind);
        bad += check(1025, 20, 3, kind);
        bad += check(17000, 50, 5, kind);
    }
    printf(bad ? "order: wrong\n" : "order: ok\n");
    return bad;
}
