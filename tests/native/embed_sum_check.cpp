// k_embed_sum (csrc/plain/embed.hip), device code on the host: a workgroup of the grid's columns that the rows of the table
// do not have ends without reading anything, the others write their columns.  The lists end where they are read last.
#include <algorithm>
#include <memory>

#include "hip/hip_runtime.h"
static Index gridDim;
#define __shfl(v, l) ((int32_t)host::exchange((uint32_t)(v), [&](const uint32_t *wave) { return wave[(l) & 63]; }))
#define __builtin_nontemporal_load(p) (*(p))
#define __builtin_nontemporal_store(v, p) (*(p) = (v))
#define __builtin_amdgcn_fence(order, scope)
#include "device.inc"

using namespace ckks_plain;

template <bool ADD, int E, int ROWS> static int check(int cols, int log_l) {
    const int turn = E << log_l, pieces = (cols + 2047) / 2048;
    const std::vector<int32_t> order{0, 1, 2}, token_of{0, 0, 2}, starts{0, 2, 2, 3};  // tokens 0 0 2 of a table of 3
    std::vector<float> drows(3 * cols), out(3 * cols, ADD ? 5.0f : NAN);
    for (size_t i = 0; i < drows.size(); i++) drows[i] = (float)(i % 97) - 40;
    gridDim = {0, (unsigned)pieces, 1};
    for (int y = 0; y < pieces; y++) {
        const bool some = y * turn < cols;
        // a workgroup without columns gets no lists: nothing of them may be read
        const EmbedSums s{some ? order.data() : nullptr, some ? token_of.data() : nullptr, some ? starts.data() : nullptr,
                          3, 3, cols, 8, 2.0f, nullptr, nullptr};
        for (int x = 0; x < (3 + ROWS - 1) / ROWS; x++) {
            blockIdx = {(unsigned)x, (unsigned)y, 0};
            if (!host::run(256, 100000, [&] {
                    k_embed_sum<float, float, ADD, E, ROWS>(s, drows.data(), cols, out.data(), cols, 0, 0, log_l);
                }))
                return 1;
        }
    }
    int bad = 0;
    const float old = ADD ? 5 : 0;
    for (int c = 0; c < cols; c++)
        bad += out[c] != old + 2 * (drows[c] + drows[cols + c]) || out[cols + c] != old || out[2 * cols + c] != old + 2 * drows[2 * cols + c];
    if (bad) printf("%d columns by %d: %d wrong\n", cols, turn, bad);
    return bad != 0;
}

int main() {
    int bad = 0;
    bad += check<false, 8, 1>(2048, 8) + check<false, 8, 1>(2047, 8) + check<true, 8, 1>(2047, 8);
    bad += check<false, 16, 1>(2051, 8) + check<false, 16, 1>(4096, 8) + check<false, 16, 1>(4099, 8);
    bad += check<false, 16, 2>(2500, 8) + check<false, 16, 1>(9001, 8);
    bad += check<true, 16, 1>(2051, 8) + check<true, 16, 1>(4099, 8) + check<true, 16, 1>(9001, 8);
    printf(bad ? "sums: wrong\n" : "sums: ok\n");
    return bad;
}
