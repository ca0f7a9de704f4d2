// matmul_i8.hip -- product of 8-bit rows with a scale for each row of both
// operands (include/ckks_plain.h).
#include <type_traits>

#include "plain_common.h"

namespace ckks_plain {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

struct MatmulArgs {
    const int8_t *a, *w;
    const float *a_scale, *w_scale, *bias;
    int64_t a_stride, w_stride, out_stride;
    int rows, channels, padded;
    bool vector_out;  // four channels from a multiple of four on can be stored at once
};

// Four channels of one token from their sums: float(sum) is exact to half a step of 32 bits, and
// so is each of the products and the bias.
template <typename T>
__device__ __forceinline__ void store4(const MatmulArgs &m, T *out, int t, int c, float a_scale, int s0, int s1, int s2,
                                       int s3) {
    typedef T T4 __attribute__((ext_vector_type(4)));
    const int s[4] = {s0, s1, s2, s3};
    T *p = out + (int64_t)t * m.out_stride + c;
    if (m.vector_out && c + 4 <= m.channels) {
        T4 v;
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] = from_f32<T>((float)s[i] * (a_scale * m.w_scale[c + i]) + (m.bias ? m.bias[c + i] : 0.0f));
        *(T4 *)p = v;
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (c + i < m.channels)
                p[i] = from_f32<T>((float)s[i] * (a_scale * m.w_scale[c + i]) + (m.bias ? m.bias[c + i] : 0.0f));
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
// them as 32 x 32 tiles in registers.  The contraction goes in steps of 128 bytes, two steps in
// LDS: while one is multiplied, the other is filled by loads that go from memory to LDS directly.
//
// LDS layout: rows of 128 bytes in eight 16-byte pieces; piece p of row r lies at p ^ (r & 7), so
// the lanes that read one piece of neighbouring rows reach different banks.  The loads write LDS
// in lane order and permute the pieces on the memory side (within a row's 128 bytes).
constexpr int STEP = 128;

// 64 lanes x 16 bytes from base + voff (a lane's offset) to the LDS address `lds` (of the wave) on.
// The write to LDS is tracked by vmcnt, which the compiler does not see here: tile_wait orders it.
__device__ __forceinline__ void load_to_lds(const int8_t *base, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(voff), "s"(base)
                 : "memory", "m0");
}
// All of this wave's reads and writes of LDS are done, and then the other waves'.
__device__ __forceinline__ void tile_wait() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <typename T, int BM, int BN>
__global__ __launch_bounds__(256, BM == 256 ? 1 : 2) void k_matmul_i8_tile(MatmulArgs m, T *out, TileOrder order) {
    constexpr int TN = BN / 64, TM = BM / 64;      // 32 x 32 tiles of a wave
    constexpr int LOADS_W = BN / 32, LOADS_A = BM / 32;  // of a wave, per step
    __shared__ int8_t lds[2][(BN + BM) * STEP];
    int tile_t, tile_c;
    order.tile(blockIdx.x, tile_t, tile_c);
    const int t0 = tile_t * BM, c0 = tile_c * BN;
    const int l = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int8_t *wp = m.w + (int64_t)c0 * m.w_stride, *ap = m.a + (int64_t)t0 * m.a_stride;
    // lane's row and piece in a load of 8 rows; rows past the end read the last one (not stored)
    uint32_t off_w[LOADS_W], off_a[LOADS_A];
#pragma unroll
    for (int j = 0; j < LOADS_W; j++) {
        const int r = (j * 4 + wave) * 8 + l / 8, left = m.channels - 1 - c0;
        off_w[j] = (uint32_t)((r < left ? r : left) * m.w_stride) + ((l % 8) ^ (l / 8)) * 16;
    }
#pragma unroll
    for (int j = 0; j < LOADS_A; j++) {
        const int r = (j * 4 + wave) * 8 + l / 8, left = m.rows - 1 - t0;
        off_a[j] = (uint32_t)((r < left ? r : left) * m.a_stride) + ((l % 8) ^ (l / 8)) * 16;
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t *)&lds[0][0];
    // load j of this wave's share of the step at k
    auto fill_one = [&](int buf, int64_t k, int j) {
        const uint32_t at = __builtin_amdgcn_readfirstlane(lds0 + buf * (BN + BM) * STEP + wave * 1024);
        if (j < LOADS_W)
            load_to_lds(wp + k, off_w[j], at + j * 4096);
        else
            load_to_lds(ap + k, off_a[j - LOADS_W], at + BN * STEP + (j - LOADS_W) * 4096);
    };
    auto fill = [&](int buf, int64_t k) {
#pragma unroll
        for (int j = 0; j < LOADS_W + LOADS_A; j++) fill_one(buf, k, j);
    };
    // wave's quarter; lane's row in a 32-row tile and its 16-byte piece of slab s: 2 s + l / 32
    const int row_w = (wave & 1) * (BN / 2) + l % 32, row_a = BN + (wave >> 1) * (BM / 2) + l % 32;
    v4i fw[2][TN], fa[2][TM];
    v16i acc[TN][TM] = {};
    auto read = [&](int buf, int s, v4i (&w)[TN], v4i (&a)[TM]) {
        const int piece = ((2 * s + l / 32) ^ (l & 7)) * 16;
#pragma unroll
        for (int i = 0; i < TN; i++) w[i] = *(const v4i *)&lds[buf][(row_w + 32 * i) * STEP + piece];
#pragma unroll
        for (int i = 0; i < TM; i++) a[i] = *(const v4i *)&lds[buf][(row_a + 32 * i) * STEP + piece];
        __builtin_amdgcn_sched_barrier(0);
    };
    // a slab's products; `other(n)` runs after the n-th of them
    auto mac = [&](const v4i (&w)[TN], const v4i (&a)[TM], auto other) {
#pragma unroll
        for (int n = 0; n < TN * TM; n++) {
            const int i = n / TM, j = n % TM;
            acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[i], a[j], acc[i][j], 0, 0, 0);
            other(n);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    auto nothing = [](int) {};
    // One step: the reads of each slab are issued before the products of the slab in front of it,
    // the loads of the step after the next one between the products of the last slab.
    auto step = [&](int s, auto more, auto fill_more) {
        const int buf = s & 1;
        read(buf, 1, fw[1], fa[1]);
        mac(fw[0], fa[0], nothing);
        read(buf, 2, fw[0], fa[0]);
        mac(fw[1], fa[1], nothing);
        read(buf, 3, fw[1], fa[1]);
        mac(fw[0], fa[0], nothing);
        tile_wait();  // the other buffer is full, and nobody reads this one any more
        if constexpr (decltype(more)::value) read(buf ^ 1, 0, fw[0], fa[0]);
        mac(fw[1], fa[1], [&](int n) {
            if constexpr (decltype(fill_more)::value) {
                constexpr int PER = (LOADS_W + LOADS_A + TN * TM - 1) / (TN * TM);
#pragma unroll
                for (int j = n * PER; j < (n + 1) * PER && j < LOADS_W + LOADS_A; j++)
                    fill_one(buf, (int64_t)(s + 2) * STEP, j);
                __builtin_amdgcn_sched_barrier(0);
            }
        });
    };
    const int steps = m.padded / STEP;
    fill(0, 0);
    if (steps > 1) fill(1, STEP);
    tile_wait();
    read(0, 0, fw[0], fa[0]);
    int s = 0;
    for (; s < steps - 2; s++) step(s, std::true_type{}, std::true_type{});
    if (s < steps - 1) step(s++, std::true_type{}, std::false_type{});
    step(s, std::false_type{}, std::false_type{});
    // lane: token l % 32 of each tile, channels 8 (v / 4) + 4 (l / 32) + v % 4
#pragma unroll
    for (int j = 0; j < TM; j++) {
        const int t = t0 + (wave >> 1) * (BM / 2) + 32 * j + l % 32;
        if (t >= m.rows) continue;
        const float s = m.a_scale[t];
#pragma unroll
        for (int i = 0; i < TN; i++)
#pragma unroll
            for (int g = 0; g < 4; g++)
                store4(m, out, t, c0 + (wave & 1) * (BN / 2) + 32 * i + 8 * g + 4 * (l / 32), s, acc[i][j][4 * g],
                       acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
    }
}

}  // namespace ckks_plain

using namespace ckks_plain;

extern "C" int ckks_plain_matmul_i8_workspace_size(int64_t rows, int64_t channels, int64_t cols, size_t *bytes) {
    if (!bytes || rows < 0 || channels < 0 || cols < 1 || cols >= 131072) return CKKS_EINVAL;
    *bytes = 0;
    return CKKS_OK;
}

extern "C" int ckks_plain_matmul_i8(const int8_t *a, int64_t a_stride, const float *a_scale, const int8_t *w,
                                    int64_t w_stride, const float *w_scale, const float *bias, int out_type, void *out,
                                    int64_t out_stride, int64_t rows, int64_t channels, int64_t cols, void *ws,
                                    size_t ws_bytes, void *stream) {
    size_t need;
    if (int e = ckks_plain_matmul_i8_workspace_size(rows, channels, cols, &need)) return e;
    if (!type_ok(out_type) || rows >= (int64_t)1 << 31 || channels >= (int64_t)1 << 31) return CKKS_EINVAL;
    if (rows == 0 || channels == 0) return CKKS_OK;
    const size_t z = type_size(out_type);
    const int64_t padded = round_up(cols, CKKS_PLAIN_I8_ROW);
    if (!a || !w || !a_scale || !w_scale || a_stride < padded || w_stride < padded || a_stride % CKKS_PLAIN_I8_ROW ||
        w_stride % CKKS_PLAIN_I8_ROW)
        return CKKS_EINVAL;
    if (!at(a, 16) || !at(w, 16) || !at(a_scale, 4) || !at(w_scale, 4) || !at(bias, 4)) return CKKS_EALIGN;
    if (int e = check_matrix(out, out_stride, channels, z)) return e;
    const size_t ob = span(rows, out_stride, channels, z);
    if (overlap(out, ob, a, span(rows, a_stride, padded, 1)) || overlap(out, ob, w, span(channels, w_stride, padded, 1)) ||
        overlap(out, ob, a_scale, rows * 4) || overlap(out, ob, w_scale, channels * 4) ||
        overlap(out, ob, bias, channels * 4))
        return CKKS_EINVAL;
    if (need && (!ws || ws_bytes < need)) return CKKS_EWORKSPACE;
    const MatmulArgs m{a, w, a_scale, w_scale, bias, a_stride, w_stride, out_stride, (int)rows, (int)channels,
                       (int)padded, out_stride % 4 == 0 && at(out, 4 * z)};
    auto go = [&](auto ty) {
        typedef decltype(ty) T;
        auto tiles = [&](int bm, int bn) {
            return TileOrder{(int)((rows + bm - 1) / bm), (int)((channels + bn - 1) / bn), 8};
        };
        const TileOrder big = tiles(256, 256);
        if (big.tokens * big.channels >= 192) {
            k_matmul_i8_tile<T, 256, 256><<<dim3(big.tokens * big.channels), 256, 0, (hipStream_t)stream>>>(m, (T *)out, big);
        } else {
            const TileOrder small = tiles(128, 128);
            k_matmul_i8_tile<T, 128, 128>
                <<<dim3(small.tokens * small.channels), 256, 0, (hipStream_t)stream>>>(m, (T *)out, small);
        }
        return launched();
    };
    return out_type == CKKS_PLAIN_BF16 ? go(bf16{}) : out_type == CKKS_PLAIN_F16 ? go(f16{}) : go(0.0f);
}
