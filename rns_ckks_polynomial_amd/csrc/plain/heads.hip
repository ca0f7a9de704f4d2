// heads.hip -- queries and keys: a norm for each head and the rotation by position in one pass, and its gradient.
#include "plain_common.h"

namespace ckks_plain {

struct HeadStrides {
    int64_t token, head;
};
// One tensor of heads and what becomes of it.
struct HeadSide {
    const void *x, *weight, *dy;  // dy: the gradient of the output (gradient alone)
    void *out;                    // the output, or the gradient of x
    float *part;                  // [blocks][head_dim]: the weight's gradient from each workgroup
    HeadStrides x_strides, dy_strides, out_strides;
    int heads, blocks;
};
struct HeadArgs {
    HeadSide side[2];
    const int64_t *positions;
    const float *inv_freq;
    int64_t tokens, span;  // span: tokens of a workgroup
    int half, r;           // head_dim / 2, rotary / 2
    int step;              // tokens whose angles are in LDS at a time
    int log_l;             // threads of a head
    float eps, inv_dim;
    bool interleaved;
};

// Sum over groups of 2^log_l neighbouring lanes, the same bits in each of a group's lanes.
__device__ __forceinline__ float group_sum(float v, int log_l) {
    if (log_l > 0) v += moved<0xb1, 0xf>(0.0f, v);   // quad: neighbours
    if (log_l > 1) v += moved<0x4e, 0xf>(0.0f, v);   // quad: pairs
    if (log_l > 2) v += moved<0x141, 0xf>(0.0f, v);  // half row mirrored
    if (log_l > 3) v += moved<0x140, 0xf>(0.0f, v);  // row mirrored
    if (log_l > 4) v += __shfl_xor(v, 16);
    if (log_l > 5) v += __shfl_xor(v, 32);
    return v;
}

// A thread's share of a head: K times V pairs of dimensions, a vector of V elements `lo` and one `hi`
// each.  Pair u < r turns by angle u; the pairs behind take what is left over, half and half.
template <typename T, int V, int K> struct Head {
    typedef T Vec __attribute__((ext_vector_type(V), aligned(sizeof(T))));
    Vec lo[K], hi[K];
    // first dimension of the vectors of pair u, and the distance between them
    static __device__ __forceinline__ int place(const HeadArgs &a, int u, int &apart) {
        if (a.interleaved) {
            apart = V;
            return 2 * u;
        }
        apart = u < a.r ? a.r : a.half - a.r;
        return u < a.r ? u : a.r + u;
    }
    __device__ __forceinline__ void fetch(const HeadArgs &a, const T *p, int l) {
#pragma unroll
        for (int k = 0; k < K; k++) {
            const int u = ((k << a.log_l) + l) * V;
            if (u < a.half) {
                int apart;
                const T *q = p + place(a, u, apart);
                lo[k] = *(const Vec *)q;
                hi[k] = *(const Vec *)(q + apart);
            } else {
                lo[k] = (Vec)(T)0.0f;
                hi[k] = (Vec)(T)0.0f;
            }
        }
    }
    // the pairs' elements in 32 bits
    __device__ __forceinline__ void widen(const HeadArgs &a, float (&x)[K][V], float (&y)[K][V]) const {
#pragma unroll
        for (int k = 0; k < K; k++)
#pragma unroll
            for (int j = 0; j < V; j++) {
                if (a.interleaved) {
                    x[k][j] = to_f32(2 * j < V ? lo[k][2 * j % V] : hi[k][2 * j % V]);
                    y[k][j] = to_f32(2 * j + 1 < V ? lo[k][(2 * j + 1) % V] : hi[k][(2 * j + 1) % V]);
                } else {
                    x[k][j] = to_f32(lo[k][j]);
                    y[k][j] = to_f32(hi[k][j]);
                }
            }
    }
    static __device__ __forceinline__ void store(const HeadArgs &a, T *p, int l, const float (&x)[K][V],
                                                 const float (&y)[K][V]) {
#pragma unroll
        for (int k = 0; k < K; k++) {
            const int u = ((k << a.log_l) + l) * V;
            if (u >= a.half) continue;
            Vec lo, hi;
#pragma unroll
            for (int j = 0; j < V; j++) {
                const int i = V + j;
                lo[j] = from_f32<T>(!a.interleaved ? x[k][j] : j % 2 ? y[k][j / 2] : x[k][j / 2]);
                hi[j] = from_f32<T>(!a.interleaved ? y[k][j] : i % 2 ? y[k][i / 2] : x[k][i / 2]);
            }
            int apart;
            T *q = p + place(a, u, apart);
            *(Vec *)q = lo;
            *(Vec *)(q + apart) = hi;
        }
    }
    // the pairs turned by their angles (`sign` -1: back)
    static __device__ __forceinline__ void turn(const HeadArgs &a, const float2 *angles, int l, float sign,
                                                float (&x)[K][V], float (&y)[K][V]) {
#pragma unroll
        for (int k = 0; k < K; k++) {
            const int u = ((k << a.log_l) + l) * V;
            if (u >= a.r) continue;
#pragma unroll
            for (int j = 0; j < V; j++) {
                const float2 cs = angles[u + j];
                const float s = sign * cs.y, p = x[k][j], q = y[k][j];
                x[k][j] = p * cs.x - q * s;
                y[k][j] = q * cs.x + p * s;
            }
        }
    }
};

// cos and sin of positions[t] inv_freq[i] for the tokens [first, last).  The angle in whole turns, in 64
// bits: its fraction is what a far position leaves, and 32 bits hold it.
__device__ __forceinline__ void head_angles(const HeadArgs &a, int64_t first, int64_t last, float2 *angles) {
    for (int i = threadIdx.x; i < (int)(last - first) * a.r; i += 256) {
        const int64_t t = first + i / a.r;
        const double turns = (double)a.positions[t] * ((double)a.inv_freq[i % a.r] * 0.15915494309189533577);
        float2 cs;
        sincospif((float)(2.0 * (turns - rint(turns))), &cs.y, &cs.x);
        angles[i] = cs;
    }
}

// A workgroup's tokens on one side, `step` tokens at a time: for each head, by 2^log_l threads, fetch(token, head)
// and then, with the next head's on its way, work(token, head, angles of the token).
template <typename Fetch, typename Work>
__device__ __forceinline__ void each_head(const HeadArgs &a, int heads, int64_t block, float2 *angles, Fetch fetch,
                                          Work work) {
    const int64_t first = block * a.span;
    const int64_t last = first + a.span < a.tokens ? first + a.span : a.tokens;
    const int groups = 256 >> a.log_l, g = threadIdx.x >> a.log_l;
    for (int64_t t = first; t < last; t += a.step) {
        const int64_t end = t + a.step < last ? t + a.step : last;
        const int n = (int)(end - t) * heads;
        if (g < n) fetch(t + g / heads, g % heads);
        if (t != first) __syncthreads();  // the angles before are not read any more
        head_angles(a, t, end, angles);
        __syncthreads();
        for (int i = g; i < n; i += groups) {
            const int next = i + groups;
            work(t + i / heads, i % heads, angles + i / heads * a.r,
                 [&] { if (next < n) fetch(t + next / heads, next % heads); });
        }
    }
}

// A head is read once, into registers, and its sum goes over its own lanes: no barrier but those around the angles, which
// all heads of a token share.  Bound by memory: 8192 tokens of 32 + 8 heads of 128 bf16 34.5 us for 168 MB that no cache
// has (4.9 TB/s, as a copy).  Four tokens 3.5 us: latency.
template <typename T, int V, int K>
__global__ __launch_bounds__(256) void k_head_norm_rotate(HeadArgs a) {
    typedef Head<T, V, K> H;
    extern __shared__ float2 angles[];
    const int which = blockIdx.x >= a.side[0].blocks;
    const HeadSide &s = a.side[which];
    const int l = threadIdx.x & ((1 << a.log_l) - 1);
    H hw, hx;
    if (s.weight) hw.fetch(a, (const T *)s.weight, l);
    each_head(a, s.heads, blockIdx.x - (which ? a.side[0].blocks : 0), angles,
              [&](int64_t t, int h) {
        hx.fetch(a, (const T *)s.x + t * s.x_strides.token + h * s.x_strides.head, l);
    },
              [&](int64_t t, int h, const float2 *cs, auto fetch_next) {
        float x[K][V], y[K][V];
        hx.widen(a, x, y);
        fetch_next();
        if (s.weight) {
            float w[K][V], v[K][V], sum = 0;
#pragma unroll
            for (int k = 0; k < K; k++)
#pragma unroll
                for (int j = 0; j < V; j++) sum += x[k][j] * x[k][j] + y[k][j] * y[k][j];
            const float r = 1.0f / sqrtf(group_sum(sum, a.log_l) * a.inv_dim + a.eps);
            hw.widen(a, w, v);
#pragma unroll
            for (int k = 0; k < K; k++)
#pragma unroll
                for (int j = 0; j < V; j++) x[k][j] *= r * w[k][j], y[k][j] *= r * v[k][j];
        }
        H::turn(a, cs, l, 1.0f, x, y);
        H::store(a, (T *)s.out + t * s.out_strides.token + h * s.out_strides.head, l, x, y);
    });
}

// dn: dy turned back.  With a weight: dx = r (a - hat mean(a hat)), a = dn weight, hat = x r; the weight's
// sum of dn hat over a workgroup's heads leaves as one row of partial sums.  Bound by memory: 8192 tokens of 32 + 8 heads
// of 128 bf16 56 us for 252 MB (4.5 TB/s), and 4.6 us for the sums of the partial sums.
template <typename T, int V, int K>
__global__ __launch_bounds__(256) void k_head_grad(HeadArgs a) {
    typedef Head<T, V, K> H;
    extern __shared__ float2 angles[];
    __shared__ float sums[4][CKKS_PLAIN_MAX_HEAD];
    const int which = blockIdx.x >= a.side[0].blocks;
    const HeadSide &s = a.side[which];
    const int block = blockIdx.x - (which ? a.side[0].blocks : 0);
    const int l = threadIdx.x & ((1 << a.log_l) - 1);
    float ax[K][V] = {}, ay[K][V] = {};
    H hw, hx, hd;
    if (s.weight) hw.fetch(a, (const T *)s.weight, l);
    each_head(a, s.heads, block, angles,
              [&](int64_t t, int h) {
        hd.fetch(a, (const T *)s.dy + t * s.dy_strides.token + h * s.dy_strides.head, l);
        if (s.weight) hx.fetch(a, (const T *)s.x + t * s.x_strides.token + h * s.x_strides.head, l);
    },
              [&](int64_t t, int h, const float2 *cs, auto fetch_next) {
        float p[K][V], q[K][V], x[K][V], y[K][V];
        hd.widen(a, p, q);
        if (s.weight) hx.widen(a, x, y);
        fetch_next();
        H::turn(a, cs, l, -1.0f, p, q);
        if (s.weight) {
            float w[K][V], v[K][V], sum = 0, dot = 0;
            hw.widen(a, w, v);
#pragma unroll
            for (int k = 0; k < K; k++)
#pragma unroll
                for (int j = 0; j < V; j++) sum += x[k][j] * x[k][j] + y[k][j] * y[k][j];
            const float r = 1.0f / sqrtf(group_sum(sum, a.log_l) * a.inv_dim + a.eps);
#pragma unroll
            for (int k = 0; k < K; k++)
#pragma unroll
                for (int j = 0; j < V; j++) {
                    x[k][j] *= r, y[k][j] *= r;
                    ax[k][j] += p[k][j] * x[k][j], ay[k][j] += q[k][j] * y[k][j];
                    p[k][j] *= w[k][j], q[k][j] *= v[k][j];
                    dot += p[k][j] * x[k][j] + q[k][j] * y[k][j];
                }
            dot = group_sum(dot, a.log_l) * a.inv_dim;
#pragma unroll
            for (int k = 0; k < K; k++)
#pragma unroll
                for (int j = 0; j < V; j++) {
                    p[k][j] = r * (p[k][j] - x[k][j] * dot);
                    q[k][j] = r * (q[k][j] - y[k][j] * dot);
                }
        }
        H::store(a, (T *)s.out + t * s.out_strides.token + h * s.out_strides.head, l, p, q);
    });
    if (!s.part) return;
    // the sums of a wave's groups, in a fixed order, then of the four waves
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int k = 0; k < K; k++) {
        const int u = ((k << a.log_l) + l) * V;
        int apart;
        const int at = H::place(a, u, apart);
#pragma unroll
        for (int j = 0; j < V; j++) {
            float x = ax[k][j], y = ay[k][j];
            for (int far = 32; far >> a.log_l; far >>= 1) x += __shfl_xor(x, far), y += __shfl_xor(y, far);
            if ((threadIdx.x & 63) >> a.log_l == 0 && u < a.half) {
                sums[wave][at + (a.interleaved ? 2 * j : j)] = x;
                sums[wave][at + (a.interleaved ? 2 * j + 1 : apart + j)] = y;
            }
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.half; c += 256)
        s.part[(int64_t)block * 2 * a.half + c] = ((sums[0][c] + sums[1][c]) + sums[2][c]) + sums[3][c];
}

// out[c] = the sum of part[b][c] over b, 64 columns and a side a workgroup, 16 waves on the rows in turn.
__global__ __launch_bounds__(1024) void k_head_weight_sum(const float *part0, const float *part1, int blocks0,
                                                          int blocks1, float *out0, float *out1, int dim) {
    __shared__ float sh[16][64];
    const float *part = blockIdx.y ? part1 : part0;
    float *out = blockIdx.y ? out1 : out0;
    const int n = blockIdx.y ? blocks1 : blocks0, wave = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int c = blockIdx.x * 64 + l;
    if (!out) return;
    float v = 0;
    if (c < dim) {
        int b = wave;
        for (; b + 7 * 16 < n; b += 8 * 16) {  // eight rows in flight
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; i++) w[i] = part[(int64_t)(b + i * 16) * dim + c];
#pragma unroll
            for (int i = 0; i < 8; i++) v += w[i];
        }
        for (; b < n; b += 16) v += part[(int64_t)b * dim + c];
    }
    sh[wave][l] = v;
    __syncthreads();
    if (wave || c >= dim) return;
    for (int w = 1; w < 16; w++) v += sh[w][l];
    out[c] = v;
}

// ------------------------------------------------------------------ launches

// first and last element of a tensor of heads, as a number of bytes from its pointer
size_t head_span(int64_t tokens, int64_t heads, int64_t dim, const HeadStrides &s, size_t size) {
    return tokens && heads ? ((size_t)(tokens - 1) * s.token + (size_t)(heads - 1) * s.head + dim) * size : 0;
}
HeadStrides q_strides(const ckks_plain_heads *p) { return {p->q_token_stride, p->q_head_stride}; }
HeadStrides k_strides(const ckks_plain_heads *p) { return {p->k_token_stride, p->k_head_stride}; }
bool same(const HeadStrides &a, const HeadStrides &b) {
    return a.token == b.token && a.head == b.head;
}
int check_side(const ckks_plain_heads *p, const void *x, int64_t heads, const HeadStrides &s, bool output) {
    if (!p->tokens || !heads) return CKKS_OK;
    if (!x || (p->tokens > 1 && s.token < p->head_dim) || (heads > 1 && s.head < p->head_dim)) return CKKS_EINVAL;
    // heads within a token, or tokens within a head
    if (output && p->tokens > 1 && heads > 1 && s.token < (heads - 1) * s.head + p->head_dim &&
        s.head < (p->tokens - 1) * s.token + p->head_dim)
        return CKKS_EINVAL;
    return at(x, type_size(p->type)) ? CKKS_OK : CKKS_EALIGN;
}
int check_heads(const ckks_plain_heads *p) {
    if (!p || !type_ok(p->type) || (p->interleaved != 0 && p->interleaved != 1)) return CKKS_EINVAL;
    if (p->tokens < 0 || p->tokens >= (int64_t)1 << 31 || p->q_heads < 1 || p->k_heads < 0) return CKKS_EINVAL;
    if (p->head_dim < 2 || p->rotary < 0 || p->rotary > p->head_dim || !(p->eps >= 0)) return CKKS_EINVAL;
    if (p->head_dim % 2 || p->rotary % 2 || p->head_dim > CKKS_PLAIN_MAX_HEAD || p->q_heads > 65535 ||
        p->k_heads > 65535)
        return CKKS_EUNSUPPORTED;
    if (!p->k_heads && (p->k || p->k_weight)) return CKKS_EINVAL;
    const size_t z = type_size(p->type);
    if (!at(p->q_weight, z) || !at(p->k_weight, z) || !at(p->positions, 8) || !at(p->inv_freq, 4)) return CKKS_EALIGN;
    if (p->tokens && p->rotary && (!p->positions || !p->inv_freq)) return CKKS_EINVAL;
    if (int e = check_side(p, p->q, p->q_heads, q_strides(p), false)) return e;
    return check_side(p, p->k, p->k_heads, k_strides(p), false);
}
// A tensor of heads of a call.
struct Heads {
    const void *p;
    int64_t heads;
    HeadStrides s;
};
// Whether two share memory: their ranges, unless each token of one lies between two tokens of the other (parts of
// the rows of a joint projection).
bool share(const ckks_plain_heads *p, const Heads &a, const Heads &b) {
    const size_t z = type_size(p->type);
    if (!overlap(a.p, head_span(p->tokens, a.heads, p->head_dim, a.s, z), b.p,
                 head_span(p->tokens, b.heads, p->head_dim, b.s, z)))
        return false;
    const int64_t each = a.s.token, bytes = (const char *)b.p - (const char *)a.p;
    if (p->tokens < 2 || each != b.s.token || bytes % (int64_t)z) return true;
    const int64_t off = (bytes / (int64_t)z % each + each) % each;
    return off < (a.heads - 1) * a.s.head + p->head_dim || off + (b.heads - 1) * b.s.head + p->head_dim > each;
}
// An output against every input of the call but itself (in place).
bool heads_overlap(const ckks_plain_heads *p, const Heads &out) {
    const Heads in[2] = {{p->q, p->q_heads, q_strides(p)}, {p->k, p->k_heads, k_strides(p)}};
    for (const Heads &h : in)
        if (!(h.p == out.p && h.heads == out.heads && same(h.s, out.s)) && share(p, out, h)) return true;
    const size_t z = type_size(p->type), bytes = head_span(p->tokens, out.heads, p->head_dim, out.s, z);
    return overlap(out.p, bytes, p->q_weight, p->head_dim * z) || overlap(out.p, bytes, p->k_weight, p->head_dim * z) ||
           overlap(out.p, bytes, p->positions, p->tokens * 8) || overlap(out.p, bytes, p->inv_freq, p->rotary / 2 * 4);
}

// Pairs of a vector: as many as 16 bytes hold, or fewer, so that pairs that turn, and all pairs, are whole vectors.
int head_vector(const ckks_plain_heads *p) {
    int v = 16 / (int)type_size(p->type);
    while (v > 1 && (p->rotary / 2 % v || p->head_dim / 2 % v)) v /= 2;
    return v;
}
// f(type tag, pairs of a vector, vectors of a thread): at most 64 threads
template <typename T, typename F> int by_head(const ckks_plain_heads *p, F f) {
    const int v = head_vector(p);
    const int64_t units = p->head_dim / 2;
    if (v == 2) return units <= 128 ? f(T{}, Int<2>{}, Int<1>{}) : f(T{}, Int<2>{}, Int<2>{});
    if (v == 1)
        return units <= 64 ? f(T{}, Int<1>{}, Int<1>{}) : units <= 128 ? f(T{}, Int<1>{}, Int<2>{}) : f(T{}, Int<1>{}, Int<4>{});
    if (v == 4) return f(T{}, Int<4>{}, Int<1>{});
    return f(T{}, Int<VEC<T>>{}, Int<1>{});
}
template <typename F> int by_head(const ckks_plain_heads *p, F f) {
    switch (p->type) {
        case CKKS_PLAIN_BF16: return by_head<bf16>(p, f);
        case CKKS_PLAIN_F16: return by_head<f16>(p, f);
        default: return by_head<float>(p, f);
    }
}

// Threads of a head, tokens of a step and of a workgroup.
struct HeadPlan {
    int log_l, step, span;
    int64_t blocks;
};
HeadPlan head_plan(const ckks_plain_heads *p, bool grad) {
    HeadPlan h;
    bool wide = false;
    by_head(p, [&](auto, auto v, auto k) {
        wide = decltype(v)::value == 8;
        const int64_t share = decltype(v)::value * decltype(k)::value;
        h.log_l = 0;
        while ((share << h.log_l) < p->head_dim / 2) h.log_l++;
        return 0;
    });
    const int64_t groups = 256 >> h.log_l;
    // A step of so many tokens that all threads work out angles, and each takes a few heads behind the next's loads:
    // 8192 tokens of 32 + 8 heads of 128 bf16 in a loop 29 us in steps of four, 39 one by one (gradient 54 and 62).
    // The first step is as many tokens as it takes to give each group of threads a head of the queries (with one head of
    // 64, 64 tokens and 16 KB of angles, the most); it doubles to at most four times that while 512 workgroups a side
    // remain and the angles stay within 8 KB.  Where keys have more heads than queries, their side takes as many tokens
    // a step and so more turns: 8192 tokens of 1 + 32 heads of 128 43 us, of 32 + 1 27; of 8 + 32 32 us, of 32 + 8 29.
    const int64_t one = p->q_heads < groups ? groups / p->q_heads : 1;
    h.step = (int)one;
    while (h.step < 4 * one && h.step * p->rotary <= 1024 && p->tokens >= 1024 * (int64_t)h.step) h.step *= 2;
    // The gradient's workgroups each leave a row of partial sums: as many as run at a time (with vectors of 16-bit
    // pairs the registers leave room for four a unit, of both sides: that gradient 54 us, with 256 a side 68, with
    // 1024 55; other forms have fewer registers).
    const int64_t most = !grad ? 1 << 22 : wide ? 512 : 1024;  // workgroups of a side
    h.span = (int)((p->tokens + most * h.step - 1) / (most * h.step) * h.step);
    if (h.span < h.step) h.span = h.step;
    h.blocks = (p->tokens + h.span - 1) / h.span;
    return h;
}
HeadArgs head_args(const ckks_plain_heads *p, const HeadPlan &h) {
    HeadArgs a{};
    a.side[0].x = p->q, a.side[0].weight = p->q_weight, a.side[0].x_strides = q_strides(p);
    a.side[1].x = p->k, a.side[1].weight = p->k_weight, a.side[1].x_strides = k_strides(p);
    a.side[0].heads = (int)p->q_heads, a.side[1].heads = (int)p->k_heads;
    a.side[0].blocks = (int)h.blocks, a.side[1].blocks = p->k_heads ? (int)h.blocks : 0;
    a.positions = p->positions, a.inv_freq = p->inv_freq, a.tokens = p->tokens;
    a.half = (int)p->head_dim / 2, a.r = (int)p->rotary / 2;
    a.step = h.step, a.span = h.span, a.log_l = h.log_l;
    a.eps = p->eps, a.inv_dim = 1.0f / (float)p->head_dim, a.interleaved = p->interleaved != 0;
    return a;
}

}  // namespace ckks_plain

using namespace ckks_plain;

extern "C" int ckks_plain_head_norm_rotate(const ckks_plain_heads *p, void *q_out, int64_t q_out_token_stride,
                                           int64_t q_out_head_stride, void *k_out, int64_t k_out_token_stride,
                                           int64_t k_out_head_stride, void *stream) {
    if (int e = check_heads(p)) return e;
    const HeadStrides q_out_strides{q_out_token_stride, q_out_head_stride};
    const HeadStrides k_out_strides{k_out_token_stride, k_out_head_stride};
    if (!p->k_heads && k_out) return CKKS_EINVAL;
    if (int e = check_side(p, q_out, p->q_heads, q_out_strides, true)) return e;
    if (int e = check_side(p, k_out, p->k_heads, k_out_strides, true)) return e;
    if (p->tokens == 0) return CKKS_OK;
    const Heads q{q_out, p->q_heads, q_out_strides}, k{k_out, p->k_heads, k_out_strides};
    // in place is for the tensor itself: queries over the keys are not
    if (heads_overlap(p, q) || heads_overlap(p, k) || share(p, q, k) || (q_out && q_out == p->k) || (k_out && k_out == p->q))
        return CKKS_EINVAL;
    const HeadPlan h = head_plan(p, false);
    HeadArgs a = head_args(p, h);
    a.side[0].out = q_out, a.side[0].out_strides = q_out_strides;
    a.side[1].out = k_out, a.side[1].out_strides = k_out_strides;
    return by_head(p, [&](auto ty, auto v, auto k) {
        k_head_norm_rotate<decltype(ty), decltype(v)::value, decltype(k)::value>
            <<<dim3((uint32_t)(a.side[0].blocks + a.side[1].blocks)), 256, (size_t)a.step * a.r * 8,
               (hipStream_t)stream>>>(a);
        return launched();
    });
}

extern "C" int ckks_plain_head_grad_workspace_size(const ckks_plain_heads *p, size_t *bytes) {
    if (!bytes) return CKKS_EINVAL;
    if (int e = check_heads(p)) return e;
    const HeadPlan h = head_plan(p, true);
    *bytes = ((p->q_weight != nullptr) + (p->k_weight != nullptr)) *
             (size_t)round_up(h.blocks * p->head_dim * 4, 16);
    return CKKS_OK;
}

extern "C" int ckks_plain_head_norm_rotate_grad(const ckks_plain_heads *p, const ckks_plain_head_grads *g, void *ws,
                                                size_t ws_bytes, void *stream) {
    if (!g) return CKKS_EINVAL;
    size_t need;
    if (int e = ckks_plain_head_grad_workspace_size(p, &need)) return e;
    if (!p->q_weight != !g->q_weight || !p->k_weight != !g->k_weight) return CKKS_EINVAL;
    if (!p->k_heads && (g->dk || g->dk_in)) return CKKS_EINVAL;
    if (!at(g->q_weight, 4) || !at(g->k_weight, 4)) return CKKS_EALIGN;
    const HeadStrides dq_strides{g->dq_token_stride, g->dq_head_stride}, dk_strides{g->dk_token_stride, g->dk_head_stride};
    const HeadStrides dq_in_strides{g->dq_in_token_stride, g->dq_in_head_stride};
    const HeadStrides dk_in_strides{g->dk_in_token_stride, g->dk_in_head_stride};
    if (int e = check_side(p, g->dq, p->q_heads, dq_strides, false)) return e;
    if (int e = check_side(p, g->dk, p->k_heads, dk_strides, false)) return e;
    if (int e = check_side(p, g->dq_in, p->q_heads, dq_in_strides, true)) return e;
    if (int e = check_side(p, g->dk_in, p->k_heads, dk_in_strides, true)) return e;
    const Heads in[4] = {{p->q, p->q_heads, q_strides(p)}, {p->k, p->k_heads, k_strides(p)},
                         {g->dq, p->q_heads, dq_strides}, {g->dk, p->k_heads, dk_strides}};
    const Heads out[2] = {{g->dq_in, p->q_heads, dq_in_strides}, {g->dk_in, p->k_heads, dk_in_strides}};
    const size_t z = type_size(p->type), row = p->head_dim * z;
    auto bytes = [&](const Heads &h) { return head_span(p->tokens, h.heads, p->head_dim, h.s, z); };
    struct { const void *p; size_t n; } w[3] = {{g->q_weight, (size_t)p->head_dim * 4}, {g->k_weight, (size_t)p->head_dim * 4},
                                                {ws, need}},
                                        v[4] = {{p->q_weight, row}, {p->k_weight, row}, {p->positions, (size_t)p->tokens * 8},
                                                {p->inv_freq, (size_t)p->rotary / 2 * 4}};
    for (const Heads &o : out) {
        for (const Heads &i : in)
            if (share(p, o, i)) return CKKS_EINVAL;
        for (const auto &i : v)
            if (overlap(o.p, bytes(o), i.p, i.n)) return CKKS_EINVAL;
    }
    if (share(p, out[0], out[1])) return CKKS_EINVAL;
    for (int i = 0; i < 3; i++) {
        for (const Heads &h : in)
            if (overlap(w[i].p, w[i].n, h.p, bytes(h))) return CKKS_EINVAL;
        for (const Heads &h : out)
            if (overlap(w[i].p, w[i].n, h.p, bytes(h))) return CKKS_EINVAL;
        for (const auto &x : v)
            if (overlap(w[i].p, w[i].n, x.p, x.n)) return CKKS_EINVAL;
        for (int j = 0; j < i; j++)
            if (overlap(w[i].p, w[i].n, w[j].p, w[j].n)) return CKKS_EINVAL;
    }
    if (need && (!ws || ws_bytes < need)) return CKKS_EWORKSPACE;
    if (!at(ws, 16)) return CKKS_EALIGN;
    const HeadPlan h = head_plan(p, true);
    HeadArgs a = head_args(p, h);
    a.side[0].dy = g->dq, a.side[0].dy_strides = dq_strides;
    a.side[1].dy = g->dk, a.side[1].dy_strides = dk_strides;
    a.side[0].out = g->dq_in, a.side[0].out_strides = dq_in_strides;
    a.side[1].out = g->dk_in, a.side[1].out_strides = dk_in_strides;
    const size_t one = (size_t)round_up(h.blocks * p->head_dim * 4, 16);
    if (p->q_weight) a.side[0].part = (float *)ws;
    if (p->k_weight) a.side[1].part = (float *)((char *)ws + (p->q_weight ? one : 0));
    const hipStream_t s = (hipStream_t)stream;
    if (p->tokens) {
        int e = by_head(p, [&](auto ty, auto v, auto k) {
            k_head_grad<decltype(ty), decltype(v)::value, decltype(k)::value>
                <<<dim3((uint32_t)(a.side[0].blocks + a.side[1].blocks)), 256, (size_t)a.step * a.r * 8, s>>>(a);
            return launched();
        });
        if (e) return e;
    }
    if (!p->q_weight && !p->k_weight) return CKKS_OK;
    // without tokens the sums of nothing are written
    k_head_weight_sum<<<dim3((uint32_t)((p->head_dim + 63) / 64), 2), 1024, 0, s>>>(
        a.side[0].part, a.side[1].part, a.side[0].blocks, a.side[1].blocks, g->q_weight, g->k_weight,
        (int)p->head_dim);
    return launched();
}
