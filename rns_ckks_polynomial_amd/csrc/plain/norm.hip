// norm.hip -- residual stream and norms around a gated block: forward, 8-bit
// output, gradient, and the 8-bit form of rows.
#include "plain_common.h"

namespace ckks_plain {

// ckks_plain_norm with the column count in 32 bits
struct NormArgs {
    const void *x, *y, *nw, *nb, *bw, *bb, *gate;
    int64_t rows, x_stride, y_stride, rows_per_gate;
    int cols;
    bool layer;
    float scale, eps;
    int64_t first;  // row of the first workgroup
};

// Mean (0 for rms) and 1 / sqrt(mean square around it + eps) of a row in registers; the mean
// comes first and the squares are of differences from it, so a large mean costs no digits.
template <typename R, int NT, int E>
__device__ __forceinline__ void row_stats(const float (&v)[E], const NormArgs &a, int t, float (*buf)[16], float &mu,
                                          float &r) {
    mu = 0;
    float s = 0;
    if (a.layer) {
#pragma unroll
        for (int i = 0; i < E; i++) s += v[i];
        mu = row_sum<NT>(s, buf[0]) / (float)a.cols;
        s = 0;
    }
#pragma unroll
    for (int i = 0; i < E; i++) {
        const float d = v[i] - mu;
        if (R::col(i, t) < a.cols) s += d * d;
    }
    r = 1.0f / sqrtf(row_sum<NT>(s, buf[1]) / (float)a.cols + a.eps);
}

// One row for NT threads (four rows a workgroup where NT is one wave), held in registers from its one
// read to its one write: x, y in, h, u out, nothing else moves but the weights, which stay in L2.
// Bound by memory: 8192 x 4096 bf16, norm of the block and a gate, 46.5 us for 268 MB (5.8 TB/s: part
// comes from the last-level cache; a copy of 2 GiB moves 4.8); 1021 x 5003 f32, rows at odd strides,
// layer norm with biases, 20 us for 82 MB (4.0 TB/s: one round of workgroups, each with two means to
// wait for); 4 x 2048 bf16 2.4 to 2.8 us, all latency.
template <typename T, int NT, int E, bool I8>
__global__ __launch_bounds__(NT == 64 ? 256 : NT) void k_residual_norm(NormArgs a, T *h_out, int64_t h_stride,
                                                                      void *u_out, int64_t u_stride, float *q_scale) {
    typedef Row<T, NT, E> R;
    __shared__ float buf[5][16];
    const int t = NT == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int64_t row = a.first + (NT == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x);
    if (row >= a.rows) return;
    float x[E], n[E], w[E];
    R::load((const T *)a.x + row * a.x_stride, a.cols, t, x);
    R::load((const T *)a.y + row * a.y_stride, a.cols, t, n);
    float mu, r;
    if (a.bw) {
        row_stats<R, NT>(n, a, t, buf, mu, r);
        R::load((const T *)a.bw, a.cols, t, w);
#pragma unroll
        for (int i = 0; i < E; i++) n[i] = (n[i] - mu) * r * w[i];
        if (a.bb) {
            R::load((const T *)a.bb, a.cols, t, w);
#pragma unroll
            for (int i = 0; i < E; i++) n[i] += w[i];
        }
    }
    if (a.gate) {
        R::load((const T *)a.gate + row / a.rows_per_gate * a.cols, a.cols, t, w);
#pragma unroll
        for (int i = 0; i < E; i++) n[i] *= w[i];
    }
#pragma unroll
    for (int i = 0; i < E; i++) x[i] += a.scale * n[i];
    R::store(h_out + row * h_stride, a.cols, t, x);
    row_stats<R, NT>(x, a, t, buf + 2, mu, r);
    R::load((const T *)a.nw, a.cols, t, w);
#pragma unroll
    for (int i = 0; i < E; i++) x[i] = (x[i] - mu) * r * w[i];
    if (a.nb) {
        R::load((const T *)a.nb, a.cols, t, w);
#pragma unroll
        for (int i = 0; i < E; i++) x[i] += w[i];
    }
    if constexpr (!I8) {
        R::store((T *)u_out + row * u_stride, a.cols, t, x);
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < E; i++) {
            const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
            if (R::col(i, t) < a.cols && b > m) m = b;
        }
        const float s = i8_scale(row_max<NT>(m, buf[4]));
        if (t == 0) q_scale[row] = s;
        const int padded = (a.cols + CKKS_PLAIN_I8_ROW - 1) / CKKS_PLAIN_I8_ROW * CKKS_PLAIN_I8_ROW;
        store_i8<R>((int8_t *)u_out + row * u_stride, padded, t, x, s);
    }
}

// max |x| of a row, then its 8-bit values, the row in registers in between.  Bound by memory: 8192 x
// 8192 bf16 39 to 45 us for 201 MB (4.5 to 5.1 TB/s).  |x| is compared by its bits, where infinities
// and NaN are the largest and mark the row.
template <typename T, int NT, int E>
__global__ __launch_bounds__(NT == 64 ? 256 : NT) void k_quantize_rows(const T *x, int64_t x_stride, int64_t rows,
                                                                      int cols, int8_t *q, int64_t q_stride,
                                                                      float *q_scale) {
    typedef Row<T, NT, E> R;
    __shared__ float buf[16];
    const int t = NT == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int64_t row = NT == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    if (row >= rows) return;
    float v[E];
    R::load(x + row * x_stride, cols, t, v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < E; i++) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
        if (b > m) m = b;
    }
    const float s = i8_scale(row_max<NT>(m, buf));
    if (t == 0) q_scale[row] = s;
    store_i8<R>(q + row * q_stride, (cols + CKKS_PLAIN_I8_ROW - 1) / CKKS_PLAIN_I8_ROW * CKKS_PLAIN_I8_ROW, t, v, s);
}

// ------------------------------------------------------------------ gradient

constexpr int GRAD_E = 8;  // elements a thread

// The gradient of v -> hat = (v - mu) r from that of hat: r (g - [mean g] - hat mean(g hat)), the
// bracketed mean for the layer norm alone.
//
// A workgroup walks a range of rows and keeps the weights' sums of its columns in registers; they
// leave as one row of partial sums for each workgroup, which k_norm_grad_sum adds in a fixed order
// (no atomics: the same bits on every run).  Ranges never cross from one gate row into part of
// another: either a workgroup has whole gate groups, whose sums are then complete, or a group has
// `chunks` workgroups.
struct GradPlan {
    int64_t rows_per_gate, groups;  // without a gate: all rows, 1
    int64_t chunks;                 // workgroups of a group (1: `span` whole groups a workgroup)
    int64_t span;                   // rows of a workgroup
    int64_t blocks;
};
struct GradArgs {
    const void *dh, *du;
    void *dx, *dy;
    int64_t dh_stride, du_stride, dx_stride, dy_stride;
    float *gate;      // [groups][cols] (chunks == 1)
    float *part_gate; // [blocks][cols] (chunks > 1)
    float *part[4];   // [blocks][cols]: next_weight, next_bias, block_weight, block_bias
};

//
// FULL has means and biases; without them (the rms norm of most decoders) a third of the arithmetic
// goes, which is what bounds this kernel.  The next row's operands are fetched while a row is
// worked on.  16384 x 2048 bf16 rms, with the block's norm and a gate: 101 us for 403 MB and 25 MB of
// partial sums (4.2 TB/s), and 6.5 us to add those up.
template <typename T, int NT, int E, bool FULL>
__global__ __launch_bounds__(NT, FULL && E == 8 && NT != 768 ? 4 : 1)  // 12 waves go one workgroup a unit
void k_norm_grad(NormArgs a, GradArgs o, GradPlan p) {
    typedef Row<T, NT, E> R;
    typedef typename R::Raw Raw;
    typedef float Four __attribute__((ext_vector_type(4)));
    // The columns' sums: of next_weight, block_weight, next_bias, block_bias in this order; the first
    // IN_LDS of them there, each thread its own, the others (and the gate's) in registers.  LDS has room
    // for 16 waves' (128 KB of four) and time: 1 part in 25 of the row's from memory.  In registers they
    // leave 8 or 12 waves, or spill with 16: 8192 x 4096 bf16 layer norm with biases 167 us, so 133;
    // f32 234, so 191; 4096 x 8192 bf16 156, so 147.  Without biases they fit, up to 4096 columns.
    constexpr int IN_LDS = E > 8 ? 2 : FULL ? 4 : NT < 1024 ? 0 : 2;
    __shared__ Four sums[IN_LDS ? IN_LDS * E / 4 * NT : 1];
    __shared__ float buf[8][16];
    const int t = threadIdx.x;
    float acc[4][E] = {}, acc_g[E] = {};
#pragma unroll
    for (int i = 0; i < IN_LDS * E / 4; i++) sums[i * NT + t] = Four{0, 0, 0, 0};
    auto add = [&](auto which, auto value) {
        constexpr int K = decltype(which)::value;
        if constexpr (K < IN_LDS) {
#pragma unroll
            for (int i = 0; i < E / 4; i++) {
                Four f = sums[(K * E / 4 + i) * NT + t];
#pragma unroll
                for (int j = 0; j < 4; j++) f[j] += value(4 * i + j);
                sums[(K * E / 4 + i) * NT + t] = f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; i++) acc[K][i] += value(i);
        }
    };
    const int64_t group = p.chunks > 1 ? blockIdx.x / p.chunks : 0;
    const int64_t first = p.chunks > 1 ? group * p.rows_per_gate + blockIdx.x % p.chunks * p.span
                                       : (int64_t)blockIdx.x * p.span;
    const int64_t end = p.chunks > 1 ? (group + 1) * p.rows_per_gate : a.rows;
    const int64_t last = first + p.span < end ? first + p.span : end;
    const float inv = 1.0f / (float)a.cols;
    const bool layer = FULL && a.layer;
    // sum of squares around the mean, as row_stats; what is past the end is 0 and counts where there is no mean
    auto stats = [&](const float (&v)[E], float (*b)[16], float &mu, float &r) {
        if constexpr (FULL) {
            row_stats<R, NT>(v, a, t, b, mu, r);
        } else {
            float s = 0;
#pragma unroll
            for (int i = 0; i < E; i++) s += v[i] * v[i];
            mu = 0;
            r = 1.0f / sqrtf(row_sum<NT>(s, b[1]) * inv + a.eps);
        }
    };
    // s2's for the layer norm alone
    auto means = [&](float &s1, float &s2, float (*b)[16]) {
        if (layer) {
            row_sums<NT>(s1, s2, b[0], b[1]);
            s2 *= inv;
        } else {
            s1 = row_sum<NT>(s1, b[0]), s2 = 0;
        }
        s1 *= inv;
    };
    auto center = [](float v, float mu) { return FULL ? v - mu : v; };
    // The next row, where it fits in 128 registers (16 waves a compute unit); rows of at most 4096
    // columns without biases run with fewer waves for it.
    constexpr bool AHEAD = E == 8 && (sizeof(T) == 2 || (!FULL && NT < 1024));
    Raw rx, ry, rdu, rdh;
    auto fetch = [&](int64_t row) {
        R::fetch((const T *)a.y + row * a.y_stride, a.cols, t, ry);
        R::fetch((const T *)a.x + row * a.x_stride, a.cols, t, rx);
        R::fetch((const T *)o.du + row * o.du_stride, a.cols, t, rdu);
        if constexpr (AHEAD) R::fetch((const T *)o.dh + row * o.dh_stride, a.cols, t, rdh);
    };
    if (AHEAD && first < last) fetch(first);
    for (int64_t row = first; row < last; row++) {
        float x[E], y[E], h[E], g[E], w[E], du[E], dh[E];
        if (!AHEAD) fetch(row);
        R::widen(rx, x);
        R::widen(ry, y);
        R::widen(rdu, du);
        if constexpr (AHEAD) {
            R::widen(rdh, dh);
            if (row + 1 < last) fetch(row + 1);
        }
        float mu_y = 0, r_y = 1, mu_h, r_h;
        if (a.bw) {
            stats(y, buf, mu_y, r_y);
#pragma unroll
            for (int i = 0; i < E; i++) y[i] = center(y[i], mu_y) * r_y;  // y is its norm from here on
        }
        // h = n, and g = scale times gate
        if (a.bw) {
            R::load((const T *)a.bw, a.cols, t, w);
#pragma unroll
            for (int i = 0; i < E; i++) h[i] = y[i] * w[i];
            if (FULL && a.bb) {
                R::load((const T *)a.bb, a.cols, t, w);
#pragma unroll
                for (int i = 0; i < E; i++) h[i] += w[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; i++) h[i] = y[i];
        }
        if (a.gate) {
            R::load((const T *)a.gate + row / a.rows_per_gate * a.cols, a.cols, t, g);
#pragma unroll
            for (int i = 0; i < E; i++) g[i] *= a.scale;
        } else {
#pragma unroll
            for (int i = 0; i < E; i++) g[i] = a.scale;
        }
#pragma unroll
        for (int i = 0; i < E; i++) x[i] += g[i] * h[i];
        stats(x, buf + 2, mu_h, r_h);
        R::load((const T *)a.nw, a.cols, t, w);
        float s1 = 0, s2 = 0;
#pragma unroll
        for (int i = 0; i < E; i++) x[i] = center(x[i], mu_h) * r_h;  // x is the norm of h from here on
        add(Int<0>{}, [&](int i) { return du[i] * x[i]; });
        if constexpr (FULL) add(Int<2>{}, [&](int i) { return du[i]; });
#pragma unroll
        for (int i = 0; i < E; i++) {
            du[i] *= w[i];
            s1 += du[i] * x[i];
            if constexpr (FULL) s2 += du[i];
        }
        means(s1, s2, buf + 4);
        if constexpr (!AHEAD) R::load((const T *)o.dh + row * o.dh_stride, a.cols, t, dh);
#pragma unroll
        for (int i = 0; i < E; i++) dh[i] += r_h * (center(du[i], s2) - x[i] * s1);  // the gradient of h
#pragma unroll
        for (int i = 0; i < E; i++) {
            acc_g[i] += a.scale * dh[i] * h[i];
            g[i] *= dh[i];  // the gradient of n
        }
        R::store((T *)o.dx + row * o.dx_stride, a.cols, t, dh);
        if (a.bw) {
            R::load((const T *)a.bw, a.cols, t, w);
            s1 = 0, s2 = 0;
            add(Int<1>{}, [&](int i) { return g[i] * y[i]; });
            if constexpr (FULL) add(Int<3>{}, [&](int i) { return g[i]; });
#pragma unroll
            for (int i = 0; i < E; i++) {
                g[i] *= w[i];
                s1 += g[i] * y[i];
                if constexpr (FULL) s2 += g[i];
            }
            means(s1, s2, buf + 6);
#pragma unroll
            for (int i = 0; i < E; i++) g[i] = r_y * (center(g[i], s2) - y[i] * s1);
        }
        R::store((T *)o.dy + row * o.dy_stride, a.cols, t, g);
        if (a.gate && p.chunks == 1 && (row + 1) % a.rows_per_gate == 0) {
            float *q = o.gate + row / a.rows_per_gate * a.cols;
#pragma unroll
            for (int i = 0; i < E; i++) {
                if (R::col(i, t) < a.cols) q[R::col(i, t)] = acc_g[i];
                acc_g[i] = 0;
            }
        }
    }
    auto put = [&](float *base, auto &v) {
        if (!base) return;
        base += (int64_t)blockIdx.x * a.cols;
#pragma unroll
        for (int i = 0; i < E; i++)
            if (R::col(i, t) < a.cols) base[R::col(i, t)] = v[i];
    };
    auto put_sum = [&](float *base, auto which) {
        constexpr int K = decltype(which)::value;
        if constexpr (K < IN_LDS) {
#pragma unroll
            for (int i = 0; i < E; i++) acc[K][i] = sums[(K * E / 4 + i / 4) * NT + t][i % 4];
        }
        put(base, acc[K]);
    };
    put(o.part_gate, acc_g);
    put_sum(o.part[0], Int<0>{});
    put_sum(o.part[2], Int<1>{});
    if constexpr (FULL) {
        put_sum(o.part[1], Int<2>{});
        put_sum(o.part[3], Int<3>{});
    }
}

// out[c] = sum over b of part[b][c], 64 columns a workgroup, SLICES threads a column.  blockIdx.y:
// the weights' arrays, then the gate's groups.  Latency and L2: 1024 x 2048 of three arrays 6.5 us.
struct GradSums {
    const float *part[4];
    float *out[4];
    const float *part_gate;
    float *gate;
    int64_t blocks, chunks;
};
constexpr int SLICES = 16;
__global__ __launch_bounds__(64 * SLICES) void k_norm_grad_sum(GradSums s, int cols) {
    __shared__ float sh[SLICES][64];
    const int c = blockIdx.x * 64 + (threadIdx.x & 63), k = threadIdx.x >> 6;
    const float *part;
    float *out;
    int64_t n;
    if (blockIdx.y < 4) {
        part = s.part[blockIdx.y], out = s.out[blockIdx.y], n = s.blocks;
    } else {
        const int64_t g = blockIdx.y - 4;
        part = s.part_gate + g * s.chunks * cols, out = s.gate + g * cols, n = s.chunks;
    }
    if (!out) return;
    float v = 0;
    if (c < cols) {
        int64_t b = k;
        for (; b + 7 * SLICES < n; b += 8 * SLICES) {  // eight rows in flight
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; i++) w[i] = part[(b + i * SLICES) * cols + c];
#pragma unroll
            for (int i = 0; i < 8; i++) v += w[i];
        }
        for (; b < n; b += SLICES) v += part[b * cols + c];
    }
    sh[k][threadIdx.x & 63] = v;
    __syncthreads();
    if (k == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < SLICES; i++) v += sh[i][threadIdx.x];
        out[c] = v;
    }
}

__global__ void k_zero(float *p, size_t n) {
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x) p[i] = 0;
}

// ------------------------------------------------------------------ launches

// f(type tag, threads, elements) for the smallest row shape that holds the columns.  12 waves between 8
// and 16 are worth their code: 8192 x 10000 bf16 143 us with 16, 131 with 12; 1021 x 5003 f32 layer norm
// 19.8 and 18.3; gradient of 3118 x 5313 bf16 layer norm 147 and 136.
template <int E, typename T, typename F> int by_shape(int64_t cols, F f) {
    if (cols <= 64 * E) return f(T{}, Int<64>{}, Int<E>{});
    if (cols <= 128 * E) return f(T{}, Int<128>{}, Int<E>{});
    if (cols <= 256 * E) return f(T{}, Int<256>{}, Int<E>{});
    if (cols <= 512 * E) return f(T{}, Int<512>{}, Int<E>{});
    if (cols <= 768 * E) return f(T{}, Int<768>{}, Int<E>{});
    if (cols <= 1024 * E) return f(T{}, Int<1024>{}, Int<E>{});
    return f(T{}, Int<1024>{}, Int<16>{});
}
template <int E, typename F> int by_type(int type, int64_t cols, F f) {
    switch (type) {
        case CKKS_PLAIN_BF16: return by_shape<E, bf16>(cols, f);
        case CKKS_PLAIN_F16: return by_shape<E, f16>(cols, f);
        default: return by_shape<E, float>(cols, f);
    }
}

// Elements a thread of the kernels that walk one row: 16 leave the GPU more rows at a time (8192 x
// 4096 bf16: 53 us, with 8 57 us); where the rows do not fill it anyway, 8 are done sooner (4 x 2048:
// 2.8 us, with 16 3.2 us).
template <typename F> int by_rows(int type, int64_t rows, int64_t cols, F f) {
    return rows <= 1024 ? by_type<8>(type, cols, f) : by_type<16>(type, cols, f);
}

int check_norm(const ckks_plain_norm *p) {
    if (!p || !type_ok(p->type) || (p->kind != CKKS_PLAIN_RMS && p->kind != CKKS_PLAIN_LAYER)) return CKKS_EINVAL;
    if (p->rows < 0 || p->cols < 1 || p->groups < 0 || p->rows >= (int64_t)1 << 31) return CKKS_EINVAL;
    if (p->cols > CKKS_PLAIN_MAX_COLS) return CKKS_EUNSUPPORTED;
    if (!p->gate != (p->groups == 0) || (p->groups && p->rows % p->groups)) return CKKS_EINVAL;
    if (!p->next_weight || (p->block_bias && !p->block_weight) || !(p->eps >= 0)) return CKKS_EINVAL;
    const size_t z = type_size(p->type);
    for (const void *v : {p->next_weight, p->next_bias, p->block_weight, p->block_bias, p->gate})
        if (!at(v, z)) return CKKS_EALIGN;
    if (p->rows == 0) return CKKS_OK;
    if (int e = check_matrix(p->x, p->x_stride, p->cols, z)) return e;
    return check_matrix(p->y, p->y_stride, p->cols, z);
}
// an output's range against every input of the call
bool norm_overlap(const ckks_plain_norm *p, const void *out, size_t bytes, bool x_too) {
    const size_t z = type_size(p->type), row = p->cols * z;
    if (x_too && overlap(out, bytes, p->x, span(p->rows, p->x_stride, p->cols, z))) return true;
    if (overlap(out, bytes, p->y, span(p->rows, p->y_stride, p->cols, z))) return true;
    for (const void *v : {p->next_weight, p->next_bias, p->block_weight, p->block_bias})
        if (overlap(out, bytes, v, row)) return true;
    return overlap(out, bytes, p->gate, row * p->groups);
}
NormArgs args_of(const ckks_plain_norm *p) {
    return NormArgs{p->x, p->y, p->next_weight, p->next_bias, p->block_weight, p->block_bias, p->gate, p->rows,
                    p->x_stride, p->y_stride, p->groups ? p->rows / p->groups : p->rows, (int)p->cols,
                    p->kind == CKKS_PLAIN_LAYER, p->scale, p->eps, 0};
}
template <bool I8>
int residual_norm(const ckks_plain_norm *p, void *h, int64_t h_stride, void *u, int64_t u_stride, float *q_scale,
                  hipStream_t s) {
    if (int e = check_norm(p)) return e;
    if (p->rows == 0) return CKKS_OK;
    const size_t z = type_size(p->type);
    if (int e = check_matrix(h, h_stride, p->cols, z)) return e;
    const int64_t padded = round_up(p->cols, CKKS_PLAIN_I8_ROW);
    if (I8) {
        if (!u || !q_scale || u_stride < padded || u_stride % CKKS_PLAIN_I8_ROW) return CKKS_EINVAL;
        if (!at(u, 16) || !at(q_scale, 4)) return CKKS_EALIGN;
    } else if (int e = check_matrix(u, u_stride, p->cols, z)) {
        return e;
    }
    const size_t hb = span(p->rows, h_stride, p->cols, z);
    const size_t ub = I8 ? span(p->rows, u_stride, padded, 1) : span(p->rows, u_stride, p->cols, z);
    const bool in_place = h == p->x && h_stride == p->x_stride;
    if (norm_overlap(p, h, hb, !in_place) || norm_overlap(p, u, ub, true) || overlap(h, hb, u, ub)) return CKKS_EINVAL;
    if (I8) {
        const size_t sb = p->rows * 4;
        if (norm_overlap(p, q_scale, sb, true) || overlap(q_scale, sb, u, ub) || overlap(q_scale, sb, h, hb))
            return CKKS_EINVAL;
    }
    NormArgs a = args_of(p);
    return by_rows(p->type, p->rows, p->cols, [&](auto ty, auto nt, auto e) {
        typedef decltype(ty) T;
        constexpr int NT = decltype(nt)::value;
        return in_parts(p->rows, NT, [&](int64_t first, int64_t rows) {
            a.first = first;
            k_residual_norm<T, NT, decltype(e)::value, I8>
                <<<dim3((uint32_t)(NT == 64 ? (rows + 3) / 4 : rows)), NT == 64 ? 256 : NT, 0, s>>>(
                    a, (T *)h, h_stride, u, u_stride, q_scale);
            return launched();
        });
    });
}

// Rows of a workgroup: as many workgroups as run at a time (registers leave a compute unit 16 waves),
// so that each writes its partial sums once: 8 MB in all for each weight, whatever the columns.  (With
// 1024 workgroups for any width: 4096 x 8192 bf16 rms 177 us, now 121.)
GradPlan grad_plan(const ckks_plain_norm *p) {
    GradPlan q;
    int64_t target = 2048;  // also of one wave: more would write as much as they read
    for (int64_t cols = 128 * GRAD_E; cols < p->cols && target > 256; cols *= 2) target /= 2;
    q.groups = p->groups ? p->groups : 1;
    q.rows_per_gate = p->rows / q.groups;
    // never a few more than run at a time: 3118 x 5313 f32 layer norm took 245 us with 260 of them
    const int64_t want = p->rows > target ? (p->rows + target - 1) / target : 1;
    if (q.rows_per_gate <= want) {
        q.chunks = 1;
        q.span = q.rows_per_gate ? (want + q.rows_per_gate - 1) / q.rows_per_gate * q.rows_per_gate : 1;
        q.blocks = (p->rows + q.span - 1) / q.span;
    } else {
        q.chunks = target / q.groups;  // groups < target, as rows_per_gate > rows / target
        q.span = (q.rows_per_gate + q.chunks - 1) / q.chunks;
        q.chunks = (q.rows_per_gate + q.span - 1) / q.span;
        q.blocks = q.groups * q.chunks;
    }
    return q;
}
// partial sums of next_weight, next_bias, block_weight, block_bias, gate
void grad_parts(const ckks_plain_norm *p, const GradPlan &q, bool (&has)[5]) {
    has[0] = true;
    has[1] = p->next_bias != nullptr;
    has[2] = p->block_weight != nullptr;
    has[3] = p->block_bias != nullptr;
    has[4] = p->gate && q.chunks > 1;
}

}  // namespace ckks_plain

using namespace ckks_plain;

extern "C" int ckks_plain_residual_norm(const ckks_plain_norm *p, void *h, int64_t h_stride, void *u,
                                        int64_t u_stride, void *stream) {
    return residual_norm<false>(p, h, h_stride, u, u_stride, nullptr, (hipStream_t)stream);
}
extern "C" int ckks_plain_residual_norm_i8(const ckks_plain_norm *p, void *h, int64_t h_stride, int8_t *q,
                                           int64_t q_stride, float *q_scale, void *stream) {
    return residual_norm<true>(p, h, h_stride, q, q_stride, q_scale, (hipStream_t)stream);
}

extern "C" int ckks_plain_norm_grad_workspace_size(const ckks_plain_norm *p, size_t *bytes) {
    if (!bytes) return CKKS_EINVAL;
    if (int e = check_norm(p)) return e;
    const GradPlan q = grad_plan(p);
    bool has[5];
    grad_parts(p, q, has);
    size_t n = 0;
    for (bool b : has) n += b;
    *bytes = n * (size_t)round_up(q.blocks * p->cols * 4, 16);
    return CKKS_OK;
}

extern "C" int ckks_plain_residual_norm_grad(const ckks_plain_norm *p, const ckks_plain_norm_grads *g, void *ws,
                                             size_t ws_bytes, void *stream) {
    if (!g) return CKKS_EINVAL;
    size_t need;
    if (int e = ckks_plain_norm_grad_workspace_size(p, &need)) return e;
    const size_t z = type_size(p->type), row4 = p->cols * 4;
    float *const outs[5] = {g->next_weight, g->next_bias, g->block_weight, g->block_bias, g->gate};
    const void *const ins[5] = {p->next_weight, p->next_bias, p->block_weight, p->block_bias, p->gate};
    for (int i = 0; i < 5; i++) {
        if (!outs[i] != !ins[i]) return CKKS_EINVAL;
        if (!at(outs[i], 4)) return CKKS_EALIGN;
    }
    if (p->rows) {
        if (int e = check_matrix(g->dh, g->dh_stride, p->cols, z)) return e;
        if (int e = check_matrix(g->du, g->du_stride, p->cols, z)) return e;
        if (int e = check_matrix(g->dx, g->dx_stride, p->cols, z)) return e;
        if (int e = check_matrix(g->dy, g->dy_stride, p->cols, z)) return e;
    }
    struct { const void *p; size_t n; } w[8] = {{g->dx, span(p->rows, g->dx_stride, p->cols, z)},
                                                {g->dy, span(p->rows, g->dy_stride, p->cols, z)}, {ws, need}};
    for (int i = 0; i < 5; i++) w[3 + i] = {outs[i], i < 4 ? row4 : row4 * p->groups};
    for (int i = 0; i < 8; i++) {
        if (norm_overlap(p, w[i].p, w[i].n, true) ||
            overlap(w[i].p, w[i].n, g->dh, span(p->rows, g->dh_stride, p->cols, z)) ||
            overlap(w[i].p, w[i].n, g->du, span(p->rows, g->du_stride, p->cols, z)))
            return CKKS_EINVAL;
        for (int j = 0; j < i; j++)
            if (overlap(w[i].p, w[i].n, w[j].p, w[j].n)) return CKKS_EINVAL;
    }
    if (need && (!ws || ws_bytes < need)) return CKKS_EWORKSPACE;
    if (!at(ws, 16)) return CKKS_EALIGN;
    const hipStream_t s = (hipStream_t)stream;
    const GradPlan q = grad_plan(p);
    bool has[5];
    grad_parts(p, q, has);
    GradArgs o{g->dh, g->du, g->dx, g->dy, g->dh_stride, g->du_stride, g->dx_stride, g->dy_stride, g->gate, nullptr, {}};
    GradSums sums{};
    sums.blocks = q.blocks, sums.chunks = q.chunks;
    char *at_ws = (char *)ws;
    for (int i = 0; i < 5; i++) {
        if (!has[i]) continue;
        (i < 4 ? o.part[i] : o.part_gate) = (float *)at_ws;
        at_ws += round_up(q.blocks * p->cols * 4, 16);
    }
    for (int i = 0; i < 4; i++) sums.part[i] = o.part[i], sums.out[i] = outs[i];
    sums.part_gate = o.part_gate, sums.gate = g->gate;
    if (p->rows) {
        const NormArgs a = args_of(p);
        int e = by_type<GRAD_E>(p->type, p->cols, [&](auto ty, auto nt, auto el) {
            constexpr int NT = decltype(nt)::value, E = decltype(el)::value;
            if (a.layer || a.nb || a.bb)
                k_norm_grad<decltype(ty), NT, E, true><<<dim3((uint32_t)q.blocks), NT, 0, s>>>(a, o, q);
            else
                k_norm_grad<decltype(ty), NT, E, false><<<dim3((uint32_t)q.blocks), NT, 0, s>>>(a, o, q);
            return launched();
        });
        if (e) return e;
    }
    // without rows there are no partial sums: the sums of nothing are written
    if (p->gate && !p->rows) {
        const size_t n = (size_t)p->groups * p->cols;
        k_zero<<<dim3((uint32_t)(n < 65536 * 256 ? (n + 255) / 256 : 65536)), 256, 0, s>>>(g->gate, n);
    }
    const uint32_t gate_sums = has[4] ? (uint32_t)p->groups : 0;  // fewer than `target` of grad_plan
    k_norm_grad_sum<<<dim3((uint32_t)((p->cols + 63) / 64), 4 + gate_sums), 64 * SLICES, 0, s>>>(sums, (int)p->cols);
    return launched();
}

extern "C" int ckks_plain_quantize_rows(int type, const void *x, int64_t x_stride, int64_t rows, int64_t cols,
                                        int8_t *q, int64_t q_stride, float *q_scale, void *stream) {
    if (!type_ok(type) || rows < 0 || rows >= (int64_t)1 << 31 || cols < 1) return CKKS_EINVAL;
    if (cols > CKKS_PLAIN_MAX_COLS) return CKKS_EUNSUPPORTED;
    if (rows == 0) return CKKS_OK;
    const size_t z = type_size(type);
    const int64_t padded = round_up(cols, CKKS_PLAIN_I8_ROW);
    if (int e = check_matrix(x, x_stride, cols, z)) return e;
    if (!q || !q_scale || q_stride < padded || q_stride % CKKS_PLAIN_I8_ROW) return CKKS_EINVAL;
    if (!at(q, 16) || !at(q_scale, 4)) return CKKS_EALIGN;
    const size_t xb = span(rows, x_stride, cols, z), qb = span(rows, q_stride, padded, 1), sb = rows * 4;
    if (overlap(q, qb, x, xb) || overlap(q_scale, sb, x, xb) || overlap(q, qb, q_scale, sb)) return CKKS_EINVAL;
    return by_rows(type, rows, cols, [&](auto ty, auto nt, auto e) {
        typedef decltype(ty) T;
        constexpr int NT = decltype(nt)::value;
        return in_parts(rows, NT, [&](int64_t first, int64_t n) {
            k_quantize_rows<T, NT, decltype(e)::value>
                <<<dim3((uint32_t)(NT == 64 ? (n + 3) / 4 : n)), NT == 64 ? 256 : NT, 0, (hipStream_t)stream>>>(
                    (const T *)x + first * x_stride, x_stride, n, (int)cols, q + first * q_stride, q_stride,
                    q_scale + first);
            return launched();
        });
    });
}
