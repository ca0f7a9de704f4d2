// matmul_i8.hip -- product of 8-bit rows with a scale for each row of both
// operands (include/ckks_plain.h).
#include "plain_common.h"

namespace ckks_plain {

typedef int v4i __attribute__((ext_vector_type(4)));

// The simplest tile: a wave computes 16 channels x 16 tokens, reading both operands from memory.
// Lane l supplies 16 contraction bytes of weight row l % 16 (left) and token l % 16 (right), at
// 16 (l / 16) of each 64, and ends with channels 4 (l / 16) + v (v < 4) of token l % 16.
template <typename T>
__global__ __launch_bounds__(256) void k_matmul_i8(const int8_t *a, int64_t a_stride, const float *a_scale,
                                                   const int8_t *w, int64_t w_stride, const float *w_scale,
                                                   const float *bias, T *out, int64_t out_stride, int rows,
                                                   int channels, int padded) {
    const int l = threadIdx.x & 63, c0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 16, t0 = blockIdx.y * 16;
    const int c = c0 + l % 16, t = t0 + l % 16;
    const int8_t *wp = w + (int64_t)(c < channels ? c : channels - 1) * w_stride + l / 16 * 16;
    const int8_t *ap = a + (int64_t)(t < rows ? t : rows - 1) * a_stride + l / 16 * 16;
    v4i acc = {0, 0, 0, 0};
    for (int k = 0; k < padded; k += 64)
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(*(const v4i *)(wp + k), *(const v4i *)(ap + k), acc, 0, 0, 0);
    if (t >= rows) return;
    const float s = a_scale[t];
#pragma unroll
    for (int v = 0; v < 4; v++) {
        const int o = c0 + l / 16 * 4 + v;
        if (o < channels)
            out[(int64_t)t * out_stride + o] = from_f32<T>((float)acc[v] * (s * w_scale[o]) + (bias ? bias[o] : 0.0f));
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
    const dim3 grid((uint32_t)((channels + 63) / 64), (uint32_t)((rows + 15) / 16));
    auto go = [&](auto ty) {
        typedef decltype(ty) T;
        k_matmul_i8<T><<<grid, 256, 0, (hipStream_t)stream>>>(a, a_stride, a_scale, w, w_stride, w_scale, bias, (T *)out,
                                                               out_stride, (int)rows, (int)channels, (int)padded);
        return launched();
    };
    return out_type == CKKS_PLAIN_BF16 ? go(bf16{}) : out_type == CKKS_PLAIN_F16 ? go(f16{}) : go(0.0f);
}
