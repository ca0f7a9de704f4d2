// embed.hip -- rows of a table by token, and the table's gradient.
#include "plain_common.h"

namespace ckks_plain {

// Elements of a vector of types T and O: 16 bytes of the wider, so that neighbouring lanes' accesses join to
// whole lines on both sides (with 32 bytes a lane of the wider type, half a line an instruction: the table's
// gradient in f32 97 us, so ...).
template <typename T, typename O> constexpr int JOINT = 16 / (int)(sizeof(T) > sizeof(O) ? sizeof(T) : sizeof(O));

// out[t] = scale table[tokens[t]], 2^log_l threads a row, the rest of 256 threads on other rows.
template <typename T, typename O>
__global__ __launch_bounds__(256) void k_embed(const T *table, int64_t table_stride, const float *table_scale,
                                               int64_t vocab, int64_t cols, const int64_t *tokens, int64_t first,
                                               int64_t rows, float scale, O *out, int64_t out_stride, int log_l) {
    constexpr int V = JOINT<T, O>;
    const int64_t row = first + ((int64_t)blockIdx.x << (8 - log_l)) + (threadIdx.x >> log_l);
    if (row >= rows) return;
    const int64_t v = tokens[row];
    const bool there = v >= 0 && v < vocab;
    if (table_scale && there) scale *= table_scale[v];
    const T *p = table + (there ? v : 0) * table_stride;
    O *o = out + row * out_stride;
    const int64_t step = (int64_t)V << log_l;
    for (int64_t c = (threadIdx.x & ((1 << log_l) - 1)) * V; c < cols; c += 2 * step) {
        Piece<T, V> e[2];
        if (there) {
            e[0].fetch(p + c, cols - c);
            if (c + step < cols) e[1].fetch(p + c + step, cols - c - step);
        }
#pragma unroll
        for (int k = 0; k < 2; k++) {
            float f[V];
#pragma unroll
            for (int i = 0; i < V; i++) f[i] = there ? e[k].at(i) * scale : 0.0f;
            if (c + k * step < cols) Piece<O, V>::store(o + c + k * step, cols - c - k * step, f);
        }
    }
}

// ------------------------------------------------------------------ gradient

constexpr int ORDER_NT = 1024, ORDER_WAVES = ORDER_NT / 64;

// order[0 ...): the rows with a token in [0, vocab), by token and, among equals, by row; starts[v]: how
// many of them have a token below v (v <= vocab).  Of each `chunk` places, firsts and lasts: the tokens at both
// ends.
//
// A workgroup has 2^log_bins tokens of the vocabulary and reads all rows' tokens itself, so nothing is joined
// between workgroups and one launch does: wave w counts those of its part of the rows, and after a sum over
// waves and bins puts its rows where they belong, in order.  The tokens of up to HELD * 64 rows a wave stay in
// registers in between.
constexpr int HELD = 16;
constexpr uint32_t NONE = ~0u;
struct TokenOrder {
    int32_t *order, *starts, *firsts, *lasts;
    int log_chunk;
};
__device__ __forceinline__ uint32_t token_at(const int64_t *tokens, int64_t i, int64_t last, int64_t vocab) {
    const int64_t v = i < last ? tokens[i] : -1;
    return v >= 0 && v < vocab ? (uint32_t)v : NONE;
}
__global__ __launch_bounds__(ORDER_NT) void k_token_order(const int64_t *tokens, int64_t rows, int64_t vocab,
                                                          int log_bins, TokenOrder o) {
    extern __shared__ uint32_t places[];  // [wave][bin]: counts, then the next place
    __shared__ uint32_t buf[ORDER_WAVES], sums[ORDER_WAVES], ends[ORDER_WAVES];
    const uint32_t bins = 1u << log_bins, wave = threadIdx.x >> 6, l = threadIdx.x & 63;
    const uint32_t low = blockIdx.x << log_bins;
    const int64_t part = (rows + ORDER_NT - 1) / ORDER_NT * 64;
    const int64_t first = wave * part, last = first + part < rows ? first + part : rows;
    const int64_t step = HELD * 64;
    uint32_t *mine = places + (wave << log_bins);
    for (uint32_t i = threadIdx.x; i < ORDER_WAVES << log_bins; i += ORDER_NT) places[i] = 0;
    __syncthreads();
    uint32_t below = 0, all = 0, v[HELD];
    auto fetch = [&](int64_t from) {
#pragma unroll
        for (int k = 0; k < HELD; k++) v[k] = token_at(tokens, from + k * 64 + l, last, vocab);
    };
    for (int64_t i = first; i < last; i += step) {
        fetch(i);
#pragma unroll
        for (int k = 0; k < HELD; k++) {
            below += v[k] < low;
            all += v[k] != NONE;
            if (v[k] - low < bins) atomicAdd(&mine[v[k] - low], 1u);
        }
    }
    below = row_all<ORDER_NT>(below, buf, Sum{});  // its barrier ends the counting
    all = row_all<ORDER_NT>(all, ends, Sum{});
    uint32_t n = 0;
    if (threadIdx.x < bins)
        for (int w = 0; w < ORDER_WAVES; w++) n += places[(w << log_bins) + threadIdx.x];
    const uint32_t upto = scan64(n, 0u, Sum{});
    if (l == 63) sums[wave] = upto;
    __syncthreads();
    uint32_t at = below + upto - n;
    for (uint32_t w = 0; w < wave; w++) at += sums[w];
    if (threadIdx.x < bins) {
        const int64_t token = (int64_t)low + threadIdx.x;
        if (token < vocab) o.starts[token] = (int32_t)at;
        if (token == vocab - 1) o.starts[vocab] = (int32_t)all;
        if (n && o.firsts) {
            // the ends of chunks that fall into its run
            const uint32_t chunk = 1u << o.log_chunk, end = at + n;
            for (uint32_t j = (at + chunk - 1) >> o.log_chunk; j << o.log_chunk < end; j++) o.firsts[j] = (int32_t)token;
            for (uint32_t j = at >> o.log_chunk; j << o.log_chunk < end; j++)
                if (end == all || (j + 1) << o.log_chunk <= end) o.lasts[j] = (int32_t)token;
        }
        for (int w = 0; w < ORDER_WAVES; w++) {
            const uint32_t c = places[(w << log_bins) + threadIdx.x];
            places[(w << log_bins) + threadIdx.x] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t i = first; i < last; i += step) {
        if (part > step) fetch(i);
#pragma unroll
        for (int k = 0; k < HELD; k++) {
            const uint32_t bin = v[k] - low;
            const bool in = bin < bins;  // NONE: low + bins is at most 2^24 + 2^9
            for (uint64_t left = __ballot(in); left;) {  // one token of the wave's at a time
                const int leader = __ffsll((unsigned long long)left) - 1;
                const uint32_t b = lane(bin, leader), place = mine[b];
                const uint64_t same = __ballot(in && bin == b);
                if (in && bin == b)
                    o.order[place + __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32),
                                                              __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0))] =
                        (int32_t)(i + k * 64 + l);
                if (l == (uint32_t)leader) mine[b] = place + (uint32_t)__popcll(same);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the wave's other lanes read it next
                left &= ~same;
            }
        }
    }
}

// What the sums go by: order and starts above; a run is the rows of one token, in order.  Runs of more
// than `chunk` rows are cut where a multiple of it falls: a chunk's part of such a run is summed into
// parts[2 chunk] if the run holds the chunk's first place, else into parts[2 chunk + 1] (it is long, so
// it holds the first or the last), and k_embed_join adds up the parts.
struct EmbedSums {
    const int64_t *tokens;
    const int32_t *order, *starts, *firsts, *lasts;
    int64_t rows, vocab, cols, chunk, chunks;
    float scale;
    float *parts;
};

// A thread's share of a row, eight elements: vectors of V, `apart` elements from one to the next.
template <typename T, int V> struct Share {
    static constexpr int N = 8 / V;
    Piece<T, V> e[N];
    __device__ __forceinline__ void fetch(const T *row, int64_t c, int64_t apart, int64_t cols) {
#pragma unroll
        for (int n = 0; n < N; n++)
            if (c + n * apart < cols) e[n].fetch(row + c + n * apart, cols - c - n * apart);
    }
    __device__ __forceinline__ void add_to(float (&f)[N][V]) const {
#pragma unroll
        for (int n = 0; n < N; n++)
#pragma unroll
            for (int j = 0; j < V; j++) f[n][j] += e[n].at(j);
    }
    // scale f [+ what is there]
    // (a table's gradient is larger than the caches, and stores past them are faster: 268 MB in 52 us, else 70)
    template <bool ADD> static __device__ __forceinline__ void put(T *row, int64_t c, int64_t apart, int64_t cols,
                                                                    float scale, float (&f)[N][V]) {
#pragma unroll
        for (int n = 0; n < N; n++) {
            if (c + n * apart >= cols) continue;
            T *p = row + c + n * apart;
            Piece<T, V> old;
            if (ADD) old.fetch(p, cols - c - n * apart);
#pragma unroll
            for (int j = 0; j < V; j++) f[n][j] = (ADD ? old.at(j) : 0.0f) + f[n][j] * scale;
            Piece<T, V>::template store<!ADD>(p, cols - c - n * apart, f[n]);
        }
    }
};

// Adds a share of the rows order[from, to).
template <typename T, int V>
__device__ __forceinline__ void add_run(const EmbedSums &s, const T *drows, int64_t stride, int64_t from, int64_t to,
                                        int64_t c, int64_t apart, float (&f)[8 / V][V]) {
    int64_t i = from;
    for (; i + 4 <= to; i += 4) {  // four rows in flight
        Share<T, V> e[4];
#pragma unroll
        for (int k = 0; k < 4; k++) e[k].fetch(drows + s.order[i + k] * stride, c, apart, s.cols);
#pragma unroll
        for (int k = 0; k < 4; k++) e[k].add_to(f);
    }
    for (; i < to; i++) {
        Share<T, V> e;
        e.fetch(drows + s.order[i] * stride, c, apart, s.cols);
        e.add_to(f);
    }
}

// The parts of long runs in chunk j, by a workgroup.
template <typename T>
__device__ __forceinline__ void sum_parts(const EmbedSums &s, const T *drows, int64_t stride, int64_t j) {
    constexpr int V = JOINT<T, float>;
    const int64_t from = j * s.chunk, n = s.starts[s.vocab], to = from + s.chunk < n ? from + s.chunk : n;
    if (from >= to) return;
    const int64_t va = s.firsts[j], vb = s.lasts[j];
    for (int k = 0; k < (va == vb ? 1 : 2); k++) {
        const int64_t v = k ? vb : va, a = s.starts[v], b = s.starts[v + 1];
        if (b - a <= s.chunk) continue;
        for (int64_t c = (int64_t)threadIdx.x * V; c < s.cols; c += 256 * 8) {
            float f[8 / V][V] = {};
            add_run<T, V>(s, drows, stride, a > from ? a : from, b < to ? b : to, c, 256 * V, f);
            Share<float, V>::template put<false>(s.parts + (2 * j + k) * s.cols, c, 256 * V, s.cols, 1.0f, f);
        }
    }
}

// The first `chunks` workgroups: parts of long runs.  The others: 2^log_l threads on TABLE_ROWS rows of the table,
// with the first row of each run, and where those start, on their way together.
constexpr int TABLE_ROWS = 4;
template <typename T, typename O>
__global__ __launch_bounds__(256) void k_embed_table(EmbedSums s, const T *drows, int64_t stride, O *out,
                                                     int64_t out_stride, int64_t first, int64_t chunks, int log_l) {
    if (blockIdx.x < chunks) return sum_parts(s, drows, stride, blockIdx.x);
    constexpr int V = JOINT<T, O>;
    const int64_t group = ((blockIdx.x - chunks) << (8 - log_l)) + (threadIdx.x >> log_l);
    const int64_t v = first + group * TABLE_ROWS, apart = (int64_t)V << log_l;
    if (v >= s.vocab) return;
    int32_t at[TABLE_ROWS + 1], row[TABLE_ROWS];
#pragma unroll
    for (int k = 0; k <= TABLE_ROWS; k++) at[k] = s.starts[v + k < s.vocab ? v + k : s.vocab];
#pragma unroll
    for (int k = 0; k < TABLE_ROWS; k++) {
        const int32_t n = at[k + 1] - at[k];
        row[k] = n && n <= s.chunk ? s.order[at[k]] : -1;
    }
    for (int64_t c = (int64_t)(threadIdx.x & ((1 << log_l) - 1)) * V; c < s.cols; c += (int64_t)8 << log_l) {
        Share<T, V> e[TABLE_ROWS];
#pragma unroll
        for (int k = 0; k < TABLE_ROWS; k++)
            if (row[k] >= 0) e[k].fetch(drows + row[k] * stride, c, apart, s.cols);
#pragma unroll
        for (int k = 0; k < TABLE_ROWS; k++) {
            if (v + k >= s.vocab || at[k + 1] - at[k] > s.chunk) continue;
            float f[8 / V][V] = {};
            if (row[k] >= 0) {
                e[k].add_to(f);
                add_run<T, V>(s, drows, stride, at[k] + 1, at[k + 1], c, apart, f);
            }
            Share<O, V>::template put<false>(out + (v + k) * out_stride, c, apart, s.cols, s.scale, f);
        }
    }
}

// The same with the sums added to `out`: a place of the order for 2^log_l threads, the first of its token.
template <typename T, typename O>
__global__ __launch_bounds__(256) void k_embed_add(EmbedSums s, const T *drows, int64_t stride, O *out,
                                                   int64_t out_stride, int64_t first, int64_t chunks, int log_l) {
    if (blockIdx.x < chunks) return sum_parts(s, drows, stride, blockIdx.x);
    constexpr int V = JOINT<T, O>;
    const int64_t i = first + ((blockIdx.x - chunks) << (8 - log_l)) + (threadIdx.x >> log_l);
    if (i >= s.starts[s.vocab]) return;
    const int64_t v = s.tokens[s.order[i]], apart = (int64_t)V << log_l;
    if (i != s.starts[v] || s.starts[v + 1] - i > s.chunk) return;
    for (int64_t c = (int64_t)(threadIdx.x & ((1 << log_l) - 1)) * V; c < s.cols; c += (int64_t)8 << log_l) {
        float f[8 / V][V] = {};
        add_run<T, V>(s, drows, stride, i, s.starts[v + 1], c, apart, f);
        Share<O, V>::template put<true>(out + v * out_stride, c, apart, s.cols, s.scale, f);
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
    const int64_t v = s.lasts[j], a = s.starts[v], b = s.starts[v + 1];
    if (b - a <= s.chunk || a < from) return;
    const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int64_t c = (int64_t)blockIdx.y * JOIN_COLS + l * 4, last = (b - 1) / s.chunk;
    float f[2][4] = {};
    for (int64_t k = j + wave; k <= last; k += 16) {
        Share<float, 4> e{};
        e.fetch(s.parts + (2 * k + (k == j && a > from)) * s.cols, c, 256, s.cols);
        e.add_to(f);
    }
#pragma unroll
    for (int i = 0; i < 8; i++) sh[wave][i / 4 * 256 + l * 4 + i % 4] = f[i / 4][i % 4];
    __syncthreads();
    const int64_t mine = (int64_t)blockIdx.y * JOIN_COLS + threadIdx.x;
    if (threadIdx.x >= JOIN_COLS || mine >= s.cols) return;
    float sum = 0;
    for (int w = 0; w < 16; w++) sum += sh[w][threadIdx.x];
    O *p = out + v * out_stride + mine;
    *p = from_f32<O>((ADD ? to_f32(*p) : 0.0f) + sum * s.scale);
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
// Rows of a chunk, as a power of two: at most 2048 chunks.
int log_chunk_rows(int64_t rows) {
    int l = 5;
    while ((int64_t)2048 << l < rows) l++;
    return l;
}
struct EmbedPlan {
    int log_chunk;
    int64_t chunk, chunks;
    size_t order, starts, ends, parts;  // bytes
};
EmbedPlan embed_plan(int64_t rows, int64_t vocab, int64_t cols) {
    EmbedPlan p;
    p.log_chunk = log_chunk_rows(rows);
    p.chunk = (int64_t)1 << p.log_chunk;
    p.chunks = rows > p.chunk ? (rows + p.chunk - 1) / p.chunk : 0;  // without a long run none are needed
    p.order = (size_t)round_up(rows * 4, 16);
    p.starts = (size_t)round_up((vocab + 1) * 4, 16);
    p.ends = (size_t)round_up(p.chunks * 4, 16);
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
    *bytes = p.order + p.starts + 2 * p.ends + p.parts;
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
    TokenOrder o{(int32_t *)w, (int32_t *)(w + p.order), nullptr, nullptr, p.log_chunk};
    w += p.order + p.starts;
    if (p.chunks) o.firsts = (int32_t *)w, o.lasts = (int32_t *)(w + p.ends);
    const EmbedSums a{tokens, o.order, o.starts, o.firsts, o.lasts, rows, vocab, cols, p.chunk, p.chunks, scale,
                      (float *)(w + 2 * p.ends)};
    k_token_order<<<dim3((uint32_t)((vocab + (1 << b) - 1) >> b)), ORDER_NT, (size_t)ORDER_WAVES * 4 << b, s>>>(
        tokens, rows, vocab, b, o);
    if (int e = launched()) return e;
    return typed(type, [&](auto ty) {
        return typed(out_type, [&](auto oy) {
            typedef decltype(ty) T;
            typedef decltype(oy) O;
            auto go = [&](auto addition) {
                constexpr bool ADD = decltype(addition)::value;
                int64_t chunks = p.chunks;  // with the first part of the rows
                const int64_t each = ADD ? 1 : TABLE_ROWS, n = ADD ? rows : (vocab + each - 1) / each;
                int e = in_parts(n, 1 << l, [&](int64_t first, int64_t n) {
                    const dim3 grid((uint32_t)(((n + (256 >> l) - 1) >> (8 - l)) + chunks));
                    if constexpr (ADD)
                        k_embed_add<T, O><<<grid, 256, 0, s>>>(a, (const T *)drows, drows_stride, (O *)out, out_stride,
                                                               first, chunks, l);
                    else
                        k_embed_table<T, O><<<grid, 256, 0, s>>>(a, (const T *)drows, drows_stride, (O *)out,
                                                                 out_stride, first * each, chunks, l);
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
