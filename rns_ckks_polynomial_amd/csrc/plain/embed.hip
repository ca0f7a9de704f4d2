// embed.hip -- rows of a table by token, and the table's gradient.
#include "plain_common.h"

namespace ckks_plain {

// out[t] = scale table[tokens[t]], 2^log_l threads of 8 elements a row, the rest of 256 threads on other
// rows.
template <typename T, typename O>
__global__ __launch_bounds__(256) void k_embed(const T *table, int64_t table_stride, const float *table_scale,
                                               int64_t vocab, int64_t cols, const int64_t *tokens, int64_t first,
                                               int64_t rows, float scale, O *out, int64_t out_stride, int log_l) {
    const int64_t row = first + ((int64_t)blockIdx.x << (8 - log_l)) + (threadIdx.x >> log_l);
    if (row >= rows) return;
    const int64_t v = tokens[row];
    const bool there = v >= 0 && v < vocab;
    if (table_scale && there) scale *= table_scale[v];
    const T *p = table + (there ? v : 0) * table_stride;
    O *o = out + row * out_stride;
    for (int64_t c = (threadIdx.x & ((1 << log_l) - 1)) * 8; c < cols; c += (int64_t)8 << log_l) {
        float f[8];
        Eight<T> e;
        e.fetch(p + c, there ? cols - c : 0);
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = there ? e.at(i) * scale : 0.0f;
        Eight<O>::store(o + c, cols - c, f);
    }
}

// ------------------------------------------------------------------ gradient

constexpr int ORDER_NT = 1024, ORDER_WAVES = ORDER_NT / 64;

// order[0 ...): the rows with a token in [0, vocab), by token and, among equals, by row; starts[v]: how
// many of them have a token below v (v <= vocab).  A workgroup has 2^log_bins tokens of the vocabulary
// and reads all rows' tokens itself, so nothing is joined between workgroups: wave w counts those of its
// part of the rows, and after a sum over waves and bins puts its rows where they belong, in order.
__global__ __launch_bounds__(ORDER_NT) void k_token_order(const int64_t *tokens, int64_t rows, int64_t vocab,
                                                          int log_bins, int32_t *order, int32_t *starts) {
    extern __shared__ uint32_t places[];  // [wave][bin]: counts, then the next place
    __shared__ uint32_t buf[ORDER_WAVES], sums[ORDER_WAVES];
    const int bins = 1 << log_bins, wave = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int64_t low = (int64_t)blockIdx.x << log_bins;
    const int64_t high = low + bins < vocab ? low + bins : vocab;
    const int64_t part = (rows + ORDER_NT - 1) / ORDER_NT * 64;
    const int64_t first = wave * part, last = first + part < rows ? first + part : rows;
    uint32_t *mine = places + (wave << log_bins);
    for (int i = threadIdx.x; i < ORDER_WAVES << log_bins; i += ORDER_NT) places[i] = 0;
    __syncthreads();
    uint32_t below = 0;
    for (int64_t i = first + l; i < last; i += 64) {
        const int64_t v = tokens[i];
        below += v >= 0 && v < low;
        if (v >= low && v < high) atomicAdd(&mine[v - low], 1u);
    }
    below = row_all<ORDER_NT>(below, buf, Sum{});  // its barrier ends the counting
    uint32_t n = 0;
    if (threadIdx.x < bins)
        for (int w = 0; w < ORDER_WAVES; w++) n += places[(w << log_bins) + threadIdx.x];
    const uint32_t upto = scan64(n, 0u, Sum{});
    if (l == 63) sums[wave] = upto;
    __syncthreads();
    uint32_t at = below + upto - n;
    for (int w = 0; w < wave; w++) at += sums[w];
    if (threadIdx.x < bins) {
        if (low + threadIdx.x < vocab) starts[low + threadIdx.x] = (int32_t)at;
        if (low + threadIdx.x == vocab - 1) starts[vocab] = (int32_t)(at + n);
        for (int w = 0; w < ORDER_WAVES; w++) {
            const uint32_t c = places[(w << log_bins) + threadIdx.x];
            places[(w << log_bins) + threadIdx.x] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t i = first + l; i - l < last; i += 64) {
        const int64_t v = i < last ? tokens[i] : -1;
        const bool in = v >= low && v < high;
        const uint32_t bin = in ? (uint32_t)(v - low) : 0;
        for (uint64_t left = __ballot(in); left;) {  // one token of the wave's at a time
            const uint32_t b = lane(bin, __ffsll((unsigned long long)left) - 1);
            const uint64_t same = __ballot(in && bin == b);
            const uint32_t place = mine[b];
            if (in && bin == b)
                order[place + __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32),
                                                        __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0))] = (int32_t)i;
            mine[b] = place + (uint32_t)__popcll(same);  // every lane the same
            left &= ~same;
        }
    }
}

// What the sums go by: order and starts above; a run is the rows of one token, in order.  Runs of more
// than `chunk` rows are cut where a multiple of it falls: a chunk's part of such a run is summed into
// parts[2 chunk] if the run holds the chunk's first place, else into parts[2 chunk + 1] (it is long, so
// it holds the first or the last), and k_embed_join adds up the parts.
struct EmbedSums {
    const int64_t *tokens;
    const int32_t *order, *starts;
    int64_t rows, vocab, cols, chunk, chunks;
    float scale;
    float *parts;
};

// The sum of rows order[from, to) at columns c ... c + 7.
template <typename T>
__device__ __forceinline__ void run_sum(const EmbedSums &s, const T *drows, int64_t stride, int64_t from, int64_t to,
                                        int64_t c, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j++) f[j] = 0;
    int64_t i = from;
    for (; i + 4 <= to; i += 4) {  // four rows in flight
        Eight<T> e[4];
#pragma unroll
        for (int k = 0; k < 4; k++) e[k].fetch(drows + s.order[i + k] * stride + c, s.cols - c);
#pragma unroll
        for (int k = 0; k < 4; k++)
#pragma unroll
            for (int j = 0; j < 8; j++) f[j] += e[k].at(j);
    }
    for (; i < to; i++) {
        Eight<T> e;
        e.fetch(drows + s.order[i] * stride + c, s.cols - c);
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] += e.at(j);
    }
}

template <typename O, bool ADD>
__device__ __forceinline__ void put_sum(O *p, int64_t left, float scale, float (&f)[8]) {
    if constexpr (ADD) {
        Eight<O> old;
        old.fetch(p, left);
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] = old.at(j) + f[j] * scale;
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] *= scale;
    }
    Eight<O>::store(p, left, f);
}

// Workgroups from `chunks` on: a row of the table for 2^log_l threads (with ADD: a place of the order,
// the first of its token).  Those before: the parts of long runs in a chunk.
template <typename T, typename O, bool ADD>
__global__ __launch_bounds__(256) void k_embed_sum(EmbedSums s, const T *drows, int64_t stride, O *out,
                                                   int64_t out_stride, int64_t first, int64_t chunks, int log_l) {
    const int lanes = 1 << log_l;
    if (blockIdx.x < chunks) {
        const int64_t from = blockIdx.x * s.chunk, n = s.starts[s.vocab];
        const int64_t to = from + s.chunk < n ? from + s.chunk : n;
        if (from >= to) return;
        const int64_t va = s.tokens[s.order[from]], vb = s.tokens[s.order[to - 1]];
        for (int k = 0; k < (va == vb ? 1 : 2); k++) {
            const int64_t v = k ? vb : va, a = s.starts[v], b = s.starts[v + 1];
            if (b - a <= s.chunk) continue;
            for (int64_t c = (int64_t)threadIdx.x * 8; c < s.cols; c += 256 * 8) {
                float f[8];
                run_sum(s, drows, stride, a > from ? a : from, b < to ? b : to, c, f);
                Eight<float>::store(s.parts + (2 * (int64_t)blockIdx.x + k) * s.cols + c, s.cols - c, f);
            }
        }
        return;
    }
    const int64_t i = first + ((blockIdx.x - chunks) << (8 - log_l)) + (threadIdx.x >> log_l);
    int64_t v = i;
    if (ADD) {
        if (i >= s.starts[s.vocab]) return;
        v = s.tokens[s.order[i]];
        if (i != s.starts[v]) return;
    } else if (i >= s.vocab) {
        return;
    }
    const int64_t a = s.starts[v], b = s.starts[v + 1];
    if (b - a > s.chunk) return;
    for (int64_t c = (int64_t)(threadIdx.x & (lanes - 1)) * 8; c < s.cols; c += (int64_t)8 << log_l) {
        float f[8];
        run_sum(s, drows, stride, a, b, c, f);
        put_sum<O, ADD>(out + v * out_stride + c, s.cols - c, s.scale, f);
    }
}

// The long run that starts in chunk blockIdx.x, if there is one: 512 columns (blockIdx.y), 16 waves on its
// parts in turn, then their sums in order.
constexpr int JOIN_COLS = 512;
template <typename O, bool ADD>
__global__ __launch_bounds__(1024) void k_embed_join(EmbedSums s, O *out, int64_t out_stride) {
    __shared__ float sh[16][JOIN_COLS];
    const int64_t j = blockIdx.x, n = s.starts[s.vocab], from = j * s.chunk;
    const int64_t to = from + s.chunk < n ? from + s.chunk : n;
    if (from >= to) return;
    const int64_t v = s.tokens[s.order[to - 1]], a = s.starts[v], b = s.starts[v + 1];
    if (b - a <= s.chunk || a < from) return;
    const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int64_t c = (int64_t)blockIdx.y * JOIN_COLS + l * 8, last = (b - 1) / s.chunk;
    float f[8] = {};
    if (c < s.cols)
        for (int64_t k = j + wave; k <= last; k += 16) {
            Eight<float> e;
            e.fetch(s.parts + (2 * k + (k == j && a > from)) * s.cols + c, s.cols - c);
#pragma unroll
            for (int i = 0; i < 8; i++) f[i] += e.at(i);
        }
#pragma unroll
    for (int i = 0; i < 8; i++) sh[wave][l * 8 + i] = f[i];
    __syncthreads();
    if (wave || c >= s.cols) return;
    for (int w = 1; w < 16; w++)
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] += sh[w][l * 8 + i];
    put_sum<O, ADD>(out + v * out_stride + c, s.cols - c, s.scale, f);
}

// ------------------------------------------------------------------ launches

// threads of 8 elements for a row: a power of two, at most a workgroup
int log_lanes(int64_t cols) {
    int l = 0;
    while (l < 8 && ((int64_t)8 << l) < cols) l++;
    return l;
}
template <typename F> int typed(int type, F f) {
    switch (type) {
        case CKKS_PLAIN_BF16: return f(bf16{});
        case CKKS_PLAIN_F16: return f(f16{});
        default: return f(float{});
    }
}
constexpr int64_t MAX_VOCAB = (int64_t)1 << 24;

int check_embed(int64_t vocab, int64_t cols, int64_t rows, int out_type) {
    if (!type_ok(out_type) || vocab < 1 || cols < 1 || rows < 0 || rows >= (int64_t)1 << 31) return CKKS_EINVAL;
    return vocab > MAX_VOCAB || cols >= (int64_t)1 << 31 ? CKKS_EUNSUPPORTED : CKKS_OK;
}
template <typename T>
int embed(const T *table, int64_t table_stride, const float *table_scale, size_t size, int64_t vocab, int64_t cols,
          const int64_t *tokens, int64_t rows, float scale, int out_type, void *out, int64_t out_stride,
          hipStream_t stream) {
    if (rows == 0) return CKKS_OK;
    const size_t z = type_size(out_type);
    if (int e = check_matrix(table, table_stride, cols, size)) return e;
    if (int e = check_matrix(out, out_stride, cols, z)) return e;
    if (!tokens) return CKKS_EINVAL;
    if (!at(tokens, 8)) return CKKS_EALIGN;
    const size_t ob = span(rows, out_stride, cols, z);
    if (overlap(out, ob, table, span(vocab, table_stride, cols, size)) || overlap(out, ob, tokens, rows * 8) ||
        overlap(out, ob, table_scale, vocab * 4))
        return CKKS_EINVAL;
    const int l = log_lanes(cols);
    return typed(out_type, [&](auto ty) {
        typedef decltype(ty) O;
        return in_parts(rows, 1 << l, [&](int64_t first, int64_t n) {
            const int64_t blocks = (n + (256 >> l) - 1) >> (8 - l);
            k_embed<T, O><<<dim3((uint32_t)blocks), 256, 0, stream>>>(table, table_stride, table_scale, vocab, cols,
                                                                      tokens, first, first + n, scale, (O *)out,
                                                                      out_stride, l);
            return launched();
        });
    });
}

// Bins of a workgroup of k_token_order: 256 workgroups, as far as LDS has room.
int log_bins(int64_t vocab) {
    int b = 2;
    while (b < 9 && ((int64_t)256 << b) < vocab) b++;
    return b;
}
// Rows of a chunk: at most 2048 chunks.
int64_t chunk_rows(int64_t rows) {
    int64_t c = 32;
    while (c * 2048 < rows) c *= 2;
    return c;
}
struct EmbedPlan {
    int64_t chunk, chunks;
    size_t order, starts, parts;  // bytes
};
EmbedPlan embed_plan(int64_t rows, int64_t vocab, int64_t cols) {
    EmbedPlan p;
    p.chunk = chunk_rows(rows);
    p.chunks = rows > p.chunk ? (rows + p.chunk - 1) / p.chunk : 0;  // without a long run none are needed
    p.order = (size_t)round_up(rows * 4, 16);
    p.starts = (size_t)round_up((vocab + 1) * 4, 16);
    p.parts = (size_t)p.chunks * 2 * cols * 4;
    return p;
}

}  // namespace ckks_plain

using namespace ckks_plain;

extern "C" int ckks_plain_embed(int type, const void *table, int64_t table_stride, int64_t vocab, int64_t cols,
                                const int64_t *tokens, int64_t rows, float scale, int out_type, void *out,
                                int64_t out_stride, void *stream) {
    if (!type_ok(type)) return CKKS_EINVAL;
    if (int e = check_embed(vocab, cols, rows, out_type)) return e;
    return typed(type, [&](auto ty) {
        typedef decltype(ty) T;
        return embed<T>((const T *)table, table_stride, nullptr, sizeof(T), vocab, cols, tokens, rows, scale, out_type,
                        out, out_stride, (hipStream_t)stream);
    });
}
extern "C" int ckks_plain_embed_i8(const int8_t *q, int64_t q_stride, const float *q_scale, int64_t vocab,
                                   int64_t cols, const int64_t *tokens, int64_t rows, float scale, int out_type,
                                   void *out, int64_t out_stride, void *stream) {
    if (int e = check_embed(vocab, cols, rows, out_type)) return e;
    if (rows && (!q_scale || q_stride % CKKS_PLAIN_I8_ROW || q_stride < round_up(cols, CKKS_PLAIN_I8_ROW)))
        return CKKS_EINVAL;
    if (rows && (!at(q, 16) || !at(q_scale, 4))) return CKKS_EALIGN;
    return embed<int8_t>(q, q_stride, q_scale, 1, vocab, cols, tokens, rows, scale, out_type, out, out_stride,
                         (hipStream_t)stream);
}

extern "C" int ckks_plain_embed_grad_workspace_size(int64_t rows, int64_t vocab, int64_t cols, size_t *bytes) {
    if (!bytes) return CKKS_EINVAL;
    if (int e = check_embed(vocab, cols, rows, CKKS_PLAIN_F32)) return e;
    const EmbedPlan p = embed_plan(rows, vocab, cols);
    *bytes = p.order + p.starts + p.parts;
    return CKKS_OK;
}

extern "C" int ckks_plain_embed_grad(int type, const void *drows, int64_t drows_stride, const int64_t *tokens,
                                     int64_t rows, int64_t vocab, int64_t cols, float scale, int out_type, void *out,
                                     int64_t out_stride, int add, void *ws, size_t ws_bytes, void *stream) {
    if (!type_ok(type)) return CKKS_EINVAL;
    size_t need;
    if (int e = check_embed(vocab, cols, rows, out_type)) return e;
    if (int e = ckks_plain_embed_grad_workspace_size(rows, vocab, cols, &need)) return e;
    if (add && rows == 0) return CKKS_OK;
    const size_t z = type_size(type), oz = type_size(out_type);
    if (int e = check_matrix(out, out_stride, cols, oz)) return e;
    if (rows) {
        if (int e = check_matrix(drows, drows_stride, cols, z)) return e;
        if (!tokens) return CKKS_EINVAL;
        if (!at(tokens, 8)) return CKKS_EALIGN;
    }
    const size_t ob = span(vocab, out_stride, cols, oz), db = span(rows, drows_stride, cols, z), tb = rows * 8;
    if (overlap(out, ob, drows, db) || overlap(out, ob, tokens, tb) || overlap(ws, need, drows, db) ||
        overlap(ws, need, tokens, tb) || overlap(ws, need, out, ob))
        return CKKS_EINVAL;
    if (!ws || ws_bytes < need) return CKKS_EWORKSPACE;
    if (!at(ws, 16)) return CKKS_EALIGN;
    const hipStream_t s = (hipStream_t)stream;
    const EmbedPlan p = embed_plan(rows, vocab, cols);
    const int b = log_bins(vocab), l = log_lanes(cols);
    char *w = (char *)ws;
    EmbedSums a{tokens, (int32_t *)w, (int32_t *)(w + p.order), rows, vocab, cols, p.chunk, p.chunks, scale,
                (float *)(w + p.order + p.starts)};
    k_token_order<<<dim3((uint32_t)((vocab + (1 << b) - 1) >> b)), ORDER_NT, (size_t)ORDER_WAVES * 4 << b, s>>>(
        tokens, rows, vocab, b, (int32_t *)a.order, (int32_t *)a.starts);
    if (int e = launched()) return e;
    return typed(type, [&](auto ty) {
        return typed(out_type, [&](auto oy) {
            typedef decltype(ty) T;
            typedef decltype(oy) O;
            auto go = [&](auto addition) {
                constexpr bool ADD = decltype(addition)::value;
                int64_t chunks = p.chunks;  // with the first part of the rows
                int e = in_parts(ADD ? rows : vocab, 1 << l, [&](int64_t first, int64_t n) {
                    const int64_t blocks = (n + (256 >> l) - 1) >> (8 - l);
                    k_embed_sum<T, O, ADD><<<dim3((uint32_t)(blocks + chunks)), 256, 0, s>>>(
                        a, (const T *)drows, drows_stride, (O *)out, out_stride, first, chunks, l);
                    chunks = 0;
                    return launched();
                });
                if (e || !p.chunks) return e;
                k_embed_join<O, ADD><<<dim3((uint32_t)p.chunks, (uint32_t)((cols + JOIN_COLS - 1) / JOIN_COLS)), 1024,
                                       0, s>>>(a, (O *)out, out_stride);
                return launched();
            };
            return add ? go(Flag<true>{}) : go(Flag<false>{});
        });
    });
}
