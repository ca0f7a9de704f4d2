// matmul_i8.hip -- product of 8-bit rows with a scale for each row of both
// operands (include/ckks_plain.h).
#include "plain_common.h"

namespace ckks_plain {

typedef int v4i __attribute__((ext_vector_type(4)));

struct MatmulArgs {
    const int8_t *a, *w;
    const float *a_scale, *w_scale, *bias;
    int64_t a_stride, w_stride, out_stride;
    int rows, channels, padded;
};

// N channels of one token from their sums: the sum, the two scales, their product and the bias
// round once each in 32 bits.
template <typename T, int N>
__device__ __forceinline__ void store_sums(const MatmulArgs &m, T *out, int t, int c, float a_scale, const int (&s)[N],
                                           const float (&w_scale)[N], const float (&bias)[N]) {
    typedef T TN __attribute__((ext_vector_type(N), aligned(sizeof(T))));  // at any channel
    T *p = out + (int64_t)t * m.out_stride + c;
    TN v;
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = from_f32<T>((float)s[i] * (a_scale * w_scale[i]) + bias[i]);
    if (c + N <= m.channels) {
        *(TN *)p = v;
    } else {
#pragma unroll
        for (int i = 0; i < N; i++)
            if (c + i < m.channels) p[i] = v[i];
    }
}

// The tile of a workgroup.  Workgroups go to the eight dies in turn; each die gets a contiguous
// run of tiles, in bands of `band` token tiles with the channels running across, so that what its
// workgroups read at a time is shared in its own L2.
struct TileOrder {
    int tokens, channels, band;
    __device__ __forceinline__ void tile(int block, int &t, int &c) const {
        const int n = tokens * channels, per = n / 8, rest = n % 8, die = block % 8;
        const int i = die * per + (die < rest ? die : rest) + block / 8;
        const int b = i / (band * channels), in = i - b * band * channels;
        const int wide = tokens - b * band < band ? tokens - b * band : band;
        t = b * band + in % wide;
        c = in / wide;
    }
};

// ------------------------------------------------------------------ tiles
//
// A workgroup of four waves (2 x 2) computes BN channels x BM tokens; a wave has a quarter of
// them as 16 x 16 tiles in registers.  (On random values 16x16x64 products alone run at
// 4.0 POP/s on this GPU, 32x32x32 ones at 3.4: the accumulators move half as often for the same
// work, and under full load power sets the clock.)  The contraction goes in steps of 64 bytes:
// one is multiplied from registers, the next is read from LDS, and three more are there or on
// their way, by loads that go from memory to LDS directly.
//
// LDS layout: rows of 64 bytes in four 16-byte pieces; piece p of row r lies at p ^ turn(r).  The
// lanes that LDS serves at a time then reach all 64 banks once, whether those are 16 neighbours
// (piece p of rows 0..15) or, as the conflict counter says of this GPU, rows 0..3 and 12..15 of one
// piece with rows 4..11 of the next (p ^ (r / 4 & 3) serves the former only).  The loads write LDS
// in lane order and permute the pieces on the memory side (within a row's 64 bytes).
//
// 8192 x 8192 x 8192 on normal values, bf16 out: 440 to 490 us (2.2 to 2.5 POP/s), no LDS conflicts.  A
// compute unit is busy for 838000 cycles, so the clock is 1.8 GHz under this load; its matrix cores are
// busy in 62 % of them (the 275 us of the products alone).  A wave, one to a matrix core, issues in 36 %
// of its cycles, waits for a unit to take its instruction in 52 and for loads, LDS or the other waves in
// 12.  A tile's fill and its epilogue (16 us of 256 x 256 together, four times) are not hidden behind
// another tile's products: a second accumulator does not fit.  777 x 5003 x 2051 f16 24 to 25 us, two
// thirds of that the load of 34 steps; 64 x 8192 x 8192 16.4 us, 4.1 TB/s of weights.
constexpr int STEP = 64;
__device__ __forceinline__ int turn(int row) {  // 0, 2, 3, 1 for each four rows in turn
    const int q = row / 4 % 4;
    return q >> 1 | ((q ^ q >> 1) & 1) << 1;
}

// 64 lanes x 16 bytes from base + voff (a lane's offset) to the LDS address `lds` (of the wave) on.
// The write to LDS is counted by vmcnt, which the compiler does not see here: tile_wait orders it.
__device__ __forceinline__ void load_to_lds(const int8_t *base, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(voff), "s"(base)
                 : "memory", "m0");
}
// All of this wave's reads of LDS and all but the last `PENDING` of its loads to LDS are done, and
// then the other waves' too.
template <int PENDING> __device__ __forceinline__ void tile_wait() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(PENDING) : "memory");
}

// acc += w x a, tied to one set of accumulation registers: with all 256 of them in use, the
// compiler's own form lets a result go to other registers and pays for it with copies in the loop
// (70 in two steps of the 256 x 256 tile).  The compiler does not see a matrix product here:
// products that follow each other need no wait, results are read after mfma_done.
__device__ __forceinline__ void mfma_i8(v4i &acc, v4i w, v4i a) {
    asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(w), "v"(a));
}
// Results are there (two times 16 cycles after the last product) and may be read from here on.
__device__ __forceinline__ void not_before(v4i &acc) { asm volatile("" : "+a"(acc)); }
template <int TN, int TM> __device__ __forceinline__ void mfma_done(v4i (&acc)[TN][TM]) {
    asm volatile("s_nop 15\n\ts_nop 15");
    for_all<TN * TM>([&](auto at) { not_before(acc[decltype(at)::value / TM][decltype(at)::value % TM]); });
}

template <typename T, int BM, int BN, int SUB, int STAGES>
__global__ __launch_bounds__(256, STAGES * SUB * (BM + BN) * STEP > 80 * 1024 ? 1 : 2) void k_matmul_i8_tile(
    MatmulArgs m, T *out, TileOrder order) {
    constexpr int TN = BN / 32, TM = BM / 32, TILES = TN * TM * SUB;  // 16 x 16 tiles of a wave, and products of a stage
    constexpr int GROUPS = (BN + BM) / 16, LOADS = GROUPS * SUB / 4;  // loads of 16 rows a step; of a wave a stage
    constexpr int PLACE = (BN + BM) * STEP, STAGE = PLACE * SUB, READS = (TN + TM) * SUB;
    static_assert(GROUPS * SUB % 4 == 0 && TM % 2 == 0, "whole shares");
    // the epilogue's: 32 tokens x a wave's channels of sums, rows 16 bytes apart in the banks
    constexpr int SUMS = BN / 2 + 4;
    static_assert(4 * 32 * SUMS * 4 <= STAGES * STAGE, "the epilogue fits");
    __shared__ __attribute__((aligned(16))) int8_t lds[STAGES * STAGE];
    __shared__ float scales[BM];
    int tile_t, tile_c;
    order.tile(blockIdx.x, tile_t, tile_c);
    const int t0 = tile_t * BM, c0 = tile_c * BN;
    const int l = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int8_t *wp = m.w + (int64_t)c0 * m.w_stride, *ap = m.a + (int64_t)t0 * m.a_stride;
    const int steps = m.padded / STEP, stages = (steps + SUB - 1) / SUB;
    // A wave's load j of a stage is number 4 j + wave: steps in turn, the weights' rows first.  The
    // lane's row and piece in it; rows past the end read the last one (not stored).
    uint32_t off[LOADS];
    for_all<LOADS>([&](auto at) {
        constexpr int j = decltype(at)::value;
        const int g = (4 * j + wave) % GROUPS, r = g * 16 + l / 4;
        const bool weights = g < BN / 16;
        const int row = weights ? r : r - BN, left = weights ? m.channels - 1 - c0 : m.rows - 1 - t0;
        off[j] = (uint32_t)((row < left ? row : left) * (weights ? m.w_stride : m.a_stride)) + ((l % 4) ^ turn(r)) * 16;
    });
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t *)&lds[0];
    // load j of this wave's share of stage s, to place `place`
    auto fill_one = [&](int s, int place, auto at) {
        constexpr int j = decltype(at)::value;
        // with groups in fours, which step and operand it is does not depend on the wave
        constexpr bool FOURS = BN / 16 % 4 == 0 && GROUPS % 4 == 0;
        const int q = 4 * j + wave, sub = FOURS ? 4 * j / GROUPS : q / GROUPS;
        const int g = FOURS ? 4 * j % GROUPS + wave : q % GROUPS;
        const bool weights = FOURS ? 4 * j % GROUPS < BN / 16 : g < BN / 16;
        const int step = s * SUB + sub;  // past the last step: the last one again, which nobody multiplies
        const int64_t k = (int64_t)(SUB == 1 || step < steps ? step : steps - 1) * STEP;
        load_to_lds((weights ? wp : ap) + k, off[j],
                    __builtin_amdgcn_readfirstlane(lds0 + place * STAGE + sub * PLACE + g * 1024));
    };
    // wave's quarter; lane's row in a 16-row tile, its 16-byte piece: l / 16
    const int row_w = (wave & 1) * (BN / 2) + l % 16, row_a = BN + (wave >> 1) * (BM / 2) + l % 16;
    v4i fw[2][SUB][TN], fa[2][SUB][TM];
    v4i acc[TN][TM] = {};
    // read n of stage s into set h: for each step the weight tiles' pieces, then the tokens'
    auto read_one = [&](int s, int h, auto at) {
        constexpr int n = decltype(at)::value, sub = n / (TN + TM), i = n % (TN + TM);
        const int8_t *from = lds + s % STAGES * STAGE + sub * PLACE + ((l / 16) ^ turn(l)) * 16;
        if constexpr (i < TN)
            fw[h][sub][i] = *(const v4i *)(from + (row_w + 16 * i) * STEP);
        else
            fa[h][sub][i - TN] = *(const v4i *)(from + (row_a + 16 * (i - TN)) * STEP);
    };
    // One stage, from register set h.  First the next stage has to have arrived and the waves to have
    // read this one, whose place in LDS then takes the stage STAGES later.  Reads and loads are
    // spread over the products: a wave that issues them together waits for LDS to take them, and
    // the matrix cores with it.  The last stages load the last one again and read stale ones, which
    // nobody uses: so every stage is the same code, and the accumulators never move.
    auto stage = [&](int s, auto set) {
        constexpr int h = decltype(set)::value, HALF = TILES / 2;
        tile_wait<(STAGES - 2) * LOADS>();
        const int next = s + STAGES < stages ? s + STAGES : stages - 1;
        for_all<TILES>([&](auto at) {
            constexpr int n = decltype(at)::value, sub = n / (TN * TM), i = n % (TN * TM) / TM, j = n % TM;
            if (SUB == 1 || s * SUB + sub < steps) mfma_i8(acc[i][j], fw[h][sub][i], fa[h][sub][j]);
            for_all<READS>([&](auto r) {
                if constexpr (n == decltype(r)::value * HALF / READS) read_one(s + 1, h ^ 1, r);
            });
            for_all<LOADS>([&](auto r) {
                if constexpr (n == HALF + decltype(r)::value * HALF / LOADS) fill_one(next, s % STAGES, r);
            });
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    for_all<STAGES>([&](auto s) {
        constexpr int at = decltype(s)::value;
        for_all<LOADS>([&](auto j) { fill_one(at < stages ? at : stages - 1, at, j); });
    });
    tile_wait<(STAGES - 1) * LOADS>();
    for_all<READS>([&](auto n) { read_one(0, 0, n); });
    for (int s = 0; s < stages; s += 2) {  // one more than there are, if their number is odd: it multiplies nothing
        stage(s, Int<0>{});
        if (SUB == 1 || s + 1 < stages) stage(s + 1, Int<1>{});
    }
    // Epilogue: 32 tokens at a time through LDS (a place for each wave), so that a token's channels
    // leave in whole 16-byte pieces of neighbouring lanes.  A lane holds channels
    // 4 (l / 16) + 0..3 of token l % 16 of each tile.
    tile_wait<0>();
    mfma_done(acc);
    if (threadIdx.x < BM) scales[threadIdx.x] = m.a_scale[t0 + (int)threadIdx.x < m.rows ? t0 + threadIdx.x : m.rows - 1];
    constexpr int PER = sizeof(T) == 4 ? 4 : 8, LANES = BN / 2 / PER;  // channels a lane stores, lanes a token
    int *sums = (int *)lds + wave * 32 * SUMS;
    const int c = c0 + (wave & 1) * (BN / 2) + l % LANES * PER;
    float ws[PER], bias[PER];
#pragma unroll
    for (int i = 0; i < PER; i++) {
        ws[i] = c + i < m.channels ? m.w_scale[c + i] : 0.0f;
        bias[i] = m.bias && c + i < m.channels ? m.bias[c + i] : 0.0f;
    }
    __syncthreads();
    for_all<TM / 2>([&](auto pair) {
        constexpr int j = 2 * decltype(pair)::value;
        for_all<TN>([&](auto i) {
            constexpr int at = decltype(i)::value;
            *(v4i *)(sums + l % 16 * SUMS + 16 * at + 4 * (l / 16)) = acc[at][j];
            *(v4i *)(sums + (16 + l % 16) * SUMS + 16 * at + 4 * (l / 16)) = acc[at][j + 1];
        });
        __builtin_amdgcn_wave_barrier();
        const int tj = (wave >> 1) * (BM / 2) + 16 * j;
#pragma unroll
        for (int r = 0; r < 32; r += 64 / LANES) {
            const int t = tj + r + l / LANES;
            int v[PER];
#pragma unroll
            for (int i = 0; i < PER; i += 4)
                *(v4i *)(v + i) = *(const v4i *)(sums + (r + l / LANES) * SUMS + l % LANES * PER + i);
            if (t0 + t < m.rows) store_sums<T, PER>(m, out, t0 + t, c, scales[t], v, ws, bias);
        }
        __builtin_amdgcn_wave_barrier();
    });
}

// ------------------------------------------------------------------ few tokens
//
// For a few tokens the weights are all that has to move.  A wave takes 16 channels and all tokens
// and reads both straight into the operand registers: lane l holds 16 bytes of row l % 16 at
// 16 (l / 16) of each 64, so two loads use a row's 128 bytes; the tokens come from L2.  The waves of
// a workgroup share the channels and split the contraction (in turn, 128 bytes each); their sums
// meet in LDS.  1 x 32768 x 2048: 14.2 us, 4.7 TB/s of weights (a copy of 2 GiB moves 4.8).
constexpr int FEW = 8;       // tokens: 8 x 8192 x 8192 takes 16.6 us here and 16.3 in tiles, 1 14.2 and 16.5
constexpr int BATCH = 4;     // pieces of 128 bytes in flight
template <typename T> __global__ __launch_bounds__(512) void k_matmul_i8_few(MatmulArgs m, T *out) {
    __shared__ v4i sums[8][64];
    const int l = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6, pieces = m.padded / 128, c0 = blockIdx.x * 16;
    const int cw = c0 + l % 16, tw = l % 16;
    const int8_t *wp = m.w + (int64_t)(cw < m.channels ? cw : m.channels - 1) * m.w_stride + l / 16 * 16;
    const int8_t *ap = m.a + (int64_t)(tw < m.rows ? tw : m.rows - 1) * m.a_stride + l / 16 * 16;
    v4i acc = {0, 0, 0, 0};
    // n pieces from p on, all loads in front of the products
    auto take = [&](int p, auto count) {
        constexpr int n = decltype(count)::value;
        v4i w[n][2], a[n][2];
#pragma unroll
        for (int u = 0; u < n; u++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int64_t at = (int64_t)(p + u * waves) * 128 + h * 64;
                w[u][h] = __builtin_nontemporal_load((const v4i *)(wp + at));  // read once
                a[u][h] = *(const v4i *)(ap + at);
            }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < n; u++)
#pragma unroll
            for (int h = 0; h < 2; h++) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][h], a[u][h], acc, 0, 0, 0);
    };
    int p = wave;
    for (; p + (BATCH - 1) * waves < pieces; p += BATCH * waves) take(p, Int<BATCH>{});
    for (; p < pieces; p += waves) take(p, Int<1>{});
    sums[wave][l] = acc;
    __syncthreads();
    if (wave) return;
    for (int k = 1; k < waves; k++) acc += sums[k][l];
    // a lane has channels 4 (l / 16) + 0..3 of token l % 16
    const int t = l % 16, c = c0 + l / 16 * 4;
    if (t >= m.rows || c >= m.channels) return;
    const int s[4] = {acc[0], acc[1], acc[2], acc[3]};
    float ws[4], bias[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        ws[i] = c + i < m.channels ? m.w_scale[c + i] : 0.0f;
        bias[i] = m.bias && c + i < m.channels ? m.bias[c + i] : 0.0f;
    }
    store_sums<T, 4>(m, out, t, c, m.a_scale[t], s, ws, bias);
}

}  // namespace ckks_plain

using namespace ckks_plain;

extern "C" int ckks_plain_matmul_i8_workspace_size(int64_t rows, int64_t channels, int64_t cols, size_t *bytes) {
    if (!bytes || rows < 0 || channels < 0 || cols < 1 || cols >= 131072) return CKKS_EINVAL;
    *bytes = 0;
    return CKKS_OK;
}

constexpr int64_t MOST = ((int64_t)1 << 31) - 256;  // rows, channels

// every check of a product with rows and channels
static int check_matmul(const int8_t *a, int64_t a_stride, const float *a_scale, const int8_t *w, int64_t w_stride,
                        const float *w_scale, const float *bias, int out_type, void *out, int64_t out_stride,
                        int64_t rows, int64_t channels, int64_t cols, void *ws, size_t ws_bytes) {
    size_t need;
    if (int e = ckks_plain_matmul_i8_workspace_size(rows, channels, cols, &need)) return e;
    // 32-bit indexes of whole tiles, and of one store past them
    if (!type_ok(out_type) || rows > MOST || channels > MOST) return CKKS_EINVAL;
    const size_t z = type_size(out_type);
    const int64_t padded = round_up(cols, CKKS_PLAIN_I8_ROW);
    if (!a || !w || !a_scale || !w_scale || a_stride < padded || w_stride < padded || a_stride % CKKS_PLAIN_I8_ROW ||
        w_stride % CKKS_PLAIN_I8_ROW || a_stride >= 1 << 23 || w_stride >= 1 << 23)
        return CKKS_EINVAL;
    if (!at(a, 16) || !at(w, 16) || !at(a_scale, 4) || !at(w_scale, 4) || !at(bias, 4)) return CKKS_EALIGN;
    if (int e = check_matrix(out, out_stride, channels, z)) return e;
    const size_t ob = span(rows, out_stride, channels, z);
    if (overlap(out, ob, a, span(rows, a_stride, padded, 1)) || overlap(out, ob, w, span(channels, w_stride, padded, 1)) ||
        overlap(out, ob, a_scale, rows * 4) || overlap(out, ob, w_scale, channels * 4) ||
        overlap(out, ob, bias, channels * 4) || overlap(out, ob, ws, need))
        return CKKS_EINVAL;
    if (need && (!ws || ws_bytes < need)) return CKKS_EWORKSPACE;
    return need && !at(ws, 16) ? CKKS_EALIGN : CKKS_OK;
}

extern "C" int ckks_plain_matmul_i8(const int8_t *a, int64_t a_stride, const float *a_scale, const int8_t *w,
                                    int64_t w_stride, const float *w_scale, const float *bias, int out_type, void *out,
                                    int64_t out_stride, int64_t rows, int64_t channels, int64_t cols, void *ws,
                                    size_t ws_bytes, void *stream) {
    size_t need;
    if (int e = ckks_plain_matmul_i8_workspace_size(rows, channels, cols, &need)) return e;
    if (!type_ok(out_type)) return CKKS_EINVAL;
    if (rows == 0 || channels == 0) return CKKS_OK;
    if (int e = check_matmul(a, a_stride, a_scale, w, w_stride, w_scale, bias, out_type, out, out_stride, rows, channels,
                             cols, ws, ws_bytes))
        return e;
    const size_t z = type_size(out_type);
    const int64_t padded = round_up(cols, CKKS_PLAIN_I8_ROW);
    const MatmulArgs m{a, w, a_scale, w_scale, bias, a_stride, w_stride, out_stride, (int)rows, (int)channels,
                       (int)padded};
    auto go = [&](auto ty) {
        typedef decltype(ty) T;
        const hipStream_t st = (hipStream_t)stream;
        if (rows <= FEW && channels < (int64_t)1 << 30) {  // four threads a channel: fewer than 2^32 in all
            // up to eight waves share channels, while that does not make more than 32 a compute unit
            // and each has a batch of pieces
            const int groups = (int)((channels + 15) / 16);
            int waves = 8;
            while (waves > 1 && (groups * waves > 8192 || padded / 128 < BATCH * waves)) waves /= 2;
            k_matmul_i8_few<T><<<dim3(groups), 64 * waves, 0, st>>>(m, (T *)out);
            return launched();
        }
        auto order = [&](int bm, int bn) {
            return TileOrder{(int)((rows + bm - 1) / bm), (int)((channels + bn - 1) / bn), 8};
        };
        auto tile = [&](auto bm, auto bn, auto sub, auto stages) {
            constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value;
            const TileOrder o = order(BM, BN);
            k_matmul_i8_tile<T, BM, BN, decltype(sub)::value, decltype(stages)::value>
                <<<dim3(o.tokens * o.channels), 256, 0, st>>>(m, (T *)out, o);
        };
        // What a compute unit has to load sets the time of all tiles (35 to 57 GB/s into LDS, measured
        // from 64 x 32 to 256 x 256): rounds of tiles on 256 units times a tile's rows.  The least of
        // that; the larger of equals, which reads less in all.  777 x 5003 x 2051: 128 x 256 tiles (140)
        // 24 us, 256 x 256 (80) 36 us; 128 x 8192 x 8192: 64 x 64 (256) 29 us, 128 x 128 (64) 51 us.
        // Four steps between barriers keep the short steps of small tiles from waiting.
        constexpr int SHAPES[6][2] = {{256, 256}, {128, 256}, {128, 128}, {128, 64}, {64, 64}, {64, 32}};
        int best = 0;
        int64_t least = INT64_MAX;
        for (int i = 0; i < 6; i++) {
            const TileOrder o = order(SHAPES[i][0], SHAPES[i][1]);
            const int64_t cost = ((int64_t)o.tokens * o.channels + 255) / 256 * (SHAPES[i][0] + SHAPES[i][1]);
            if (cost < least) best = i, least = cost;
        }
        switch (best) {
            case 0: tile(Int<256>{}, Int<256>{}, Int<1>{}, Int<4>{}); break;
            case 1: tile(Int<128>{}, Int<256>{}, Int<1>{}, Int<4>{}); break;
            case 2: tile(Int<128>{}, Int<128>{}, Int<1>{}, Int<4>{}); break;
            case 3: tile(Int<128>{}, Int<64>{}, Int<2>{}, Int<4>{}); break;
            case 4: tile(Int<64>{}, Int<64>{}, Int<4>{}, Int<4>{}); break;
            default: tile(Int<64>{}, Int<32>{}, Int<4>{}, Int<4>{});
        }
        return launched();
    };
    return out_type == CKKS_PLAIN_BF16 ? go(bf16{}) : out_type == CKKS_PLAIN_F16 ? go(f16{}) : go(0.0f);
}

// the 8-bit rows, their scales, and what the product takes
static size_t linear_rows_bytes(int64_t rows, int64_t cols) {
    return (size_t)rows * round_up(cols, CKKS_PLAIN_I8_ROW) + round_up(rows * 4, 16);
}
extern "C" int ckks_plain_linear_i8_workspace_size(int64_t rows, int64_t channels, int64_t cols, size_t *bytes) {
    if (int e = ckks_plain_matmul_i8_workspace_size(rows, channels, cols, bytes)) return e;
    if (cols > CKKS_PLAIN_MAX_COLS) return CKKS_EUNSUPPORTED;
    *bytes += linear_rows_bytes(rows, cols);
    return CKKS_OK;
}
extern "C" int ckks_plain_linear_i8(int type, const void *x, int64_t x_stride, const int8_t *w, int64_t w_stride,
                                    const float *w_scale, const float *bias, int out_type, void *out,
                                    int64_t out_stride, int64_t rows, int64_t channels, int64_t cols, void *ws,
                                    size_t ws_bytes, void *stream) {
    size_t need;
    if (int e = ckks_plain_linear_i8_workspace_size(rows, channels, cols, &need)) return e;
    if (rows == 0 || channels == 0) return CKKS_OK;
    if (!type_ok(type) || rows > MOST) return CKKS_EINVAL;
    const size_t xb = span(rows, x_stride, cols, type_size(type));
    if (int e = check_matrix(x, x_stride, cols, type_size(type))) return e;
    if (!ws || ws_bytes < need) return CKKS_EWORKSPACE;
    if (!at(ws, 16)) return CKKS_EALIGN;
    // the product's own checks, before the quantiser runs
    if (!type_ok(out_type)) return CKKS_EINVAL;
    if (int e = check_matrix(out, out_stride, channels, type_size(out_type))) return e;
    const size_t ob = span(rows, out_stride, channels, type_size(out_type));
    const size_t wb = span(channels, w_stride, round_up(cols, CKKS_PLAIN_I8_ROW), 1);
    if (overlap(out, ob, x, xb) || overlap(ws, need, x, xb) || overlap(ws, need, out, ob) || overlap(ws, need, w, wb) ||
        overlap(ws, need, w_scale, channels * 4) || overlap(ws, need, bias, channels * 4))
        return CKKS_EINVAL;
    int8_t *q = (int8_t *)ws;
    const int64_t stride = round_up(cols, CKKS_PLAIN_I8_ROW);
    float *scale = (float *)(q + rows * stride);
    char *rest = (char *)ws + linear_rows_bytes(rows, cols);
    const size_t left = ws_bytes - linear_rows_bytes(rows, cols);
    if (int e = check_matmul(q, stride, scale, w, w_stride, w_scale, bias, out_type, out, out_stride, rows, channels,
                             cols, rest, left))
        return e;
    if (int e = ckks_plain_quantize_rows(type, x, x_stride, rows, cols, q, stride, scale, stream)) return e;
    return ckks_plain_matmul_i8(q, stride, scale, w, w_stride, w_scale, bias, out_type, out, out_stride, rows, channels,
                                cols, rest, left, stream);
}
