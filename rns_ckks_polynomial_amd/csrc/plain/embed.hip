// embed.hip -- rows of a table by token, and the table's gradient.
#include "plain_common.h"

namespace ckks_plain {

// Elements of a vector of types T and O: 16 bytes of the wider, so that neighbouring lanes' accesses join to
// whole lines on both sides (with 32 bytes a lane of the wider type, half a line an instruction, the gradient of
// 16384 rows bf16 into 32768 x 2048 f32 took 119 us in its first form; 62 now).
template <typename T, typename O> constexpr int JOINT = 16 / (int)(sizeof(T) > sizeof(O) ? sizeof(T) : sizeof(O));

// out[t] = scale table[tokens[t]], 2^log_l threads a row, the rest of 256 threads on other rows.  Bound by memory:
// 16384 x 4096 bf16 33 us for 269 MB (8.1 TB/s: frequent tokens' rows come from the caches).  PAST: outputs of 64 MB
// and more are stored past the caches (so 33 us, else 40; with a norm that reads them next, 72.4 and 73.2 us at 64 MB,
// 148 and 145 at 128 MB, 19.3 and 17.7 at 16 MB).
template <typename T, typename O, bool PAST>
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
            if (c + k * step < cols) Piece<O, V>::template store<PAST>(o + c + k * step, cols - c - k * step, f);
        }
    }
}

// ------------------------------------------------------------------ gradient

constexpr int ORDER_NT = 1024, ORDER_WAVES = ORDER_NT / 64;

// order[0 ...): the rows with a token in [0, vocab), by token and, among equals, by row, and token_of these
// places; starts[v]: how many of them have a token below v (v <= vocab).
//
// A workgroup has 2^log_bins tokens of the vocabulary and reads all rows' tokens itself, so nothing is joined
// between workgroups and one launch does: wave w counts those of its part of the rows and lists its own (up to
// LISTED of them; where there are more, the part is read again), and after a sum over waves and bins puts its rows
// where they belong, in order.  Latency: 16384 tokens of 32768 8.2 us, 8191 of 20011 6.3 us (a launch, the tokens at four
// loads a turn, five barriers).  A workgroup has at most 512 tokens of the vocabulary, so beyond 131072 of them there are
// more workgroups and each still reads all rows' tokens: 16384 rows into 2^20 47 us, into 2^24 630; 131072 rows into 2^17
// 27 us, into 2^24 2500 (an order joined between workgroups would read them once).
//
// It is short code on purpose: with all of a wave's tokens in registers, and so a copy of the loops' bodies for each, 9.9
// and 7.9 us, most of the difference to fetch the instructions.
constexpr int FETCHED = 4, LISTED = 512;
constexpr uint32_t NONE = ~0u;
struct TokenOrder {
    int32_t *order, *token_of, *starts;
};
__device__ __forceinline__ uint32_t token_at(const int64_t *tokens, int64_t i, int64_t last, int64_t vocab) {
    const int64_t v = i < last ? tokens[i] : -1;
    return v >= 0 && v < vocab ? (uint32_t)v : NONE;
}
// a lane's place among the lanes of a mask
__device__ __forceinline__ uint32_t place_in(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}
__global__ __launch_bounds__(ORDER_NT) void k_token_order(const int64_t *tokens, int64_t rows, int64_t vocab,
                                                          int log_bins, TokenOrder o) {
    extern __shared__ uint32_t places[];  // [wave][bin]: counts, then the next place
    __shared__ uint32_t listed[ORDER_WAVES][LISTED];  // rows of the wave's part
    __shared__ uint16_t listed_bin[ORDER_WAVES][LISTED];
    __shared__ uint32_t buf[ORDER_WAVES], sums[ORDER_WAVES], ends[ORDER_WAVES];
    const uint32_t bins = 1u << log_bins, wave = threadIdx.x >> 6, l = threadIdx.x & 63;
    const uint32_t low = blockIdx.x << log_bins;
    const int64_t part = (rows + ORDER_NT - 1) / ORDER_NT * 64;
    const int64_t first = wave * part, last = first + part < rows ? first + part : rows;
    uint32_t *mine = places + (wave << log_bins);
    for (uint32_t i = threadIdx.x; i < ORDER_WAVES << log_bins; i += ORDER_NT) places[i] = 0;
    __syncthreads();
    uint32_t below = 0, all = 0, found = 0;
    for (int64_t i = first; i < last; i += FETCHED * 64) {
        uint32_t v[FETCHED];
#pragma unroll
        for (int k = 0; k < FETCHED; k++) v[k] = token_at(tokens, i + k * 64 + l, last, vocab);
#pragma unroll
        for (int k = 0; k < FETCHED; k++) {
            below += v[k] < low;
            all += v[k] != NONE;
            const uint32_t bin = v[k] - low;
            const bool in = bin < bins;  // not NONE: low + bins is at most 2^24 + 2^9
            const uint64_t mask = __ballot(in);
            if (!mask) continue;
            if (in) {
                const uint32_t at = found + place_in(mask);
                atomicAdd(&mine[bin], 1u);
                if (at < LISTED) listed[wave][at] = (uint32_t)(i + k * 64 + l), listed_bin[wave][at] = (uint16_t)bin;
            }
            found += (uint32_t)__popcll(mask);
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
        for (int w = 0; w < ORDER_WAVES; w++) {
            const uint32_t c = places[(w << log_bins) + threadIdx.x];
            places[(w << log_bins) + threadIdx.x] = at;
            at += c;
        }
    }
    __syncthreads();
    // up to 64 rows of the wave at a time: a lane goes behind the lanes before it that have its token
    auto put = [&](bool in, uint32_t bin, int64_t row) {
        const uint32_t place = in ? mine[bin] : 0;
        uint64_t same = __ballot(in);
        if (!same) return;
        for (int bit = 0; bit < log_bins; bit++) {
            const uint64_t ones = __ballot(bin >> bit & 1);
            same &= bin >> bit & 1 ? ones : ~ones;
        }
        if (in) {
            const uint32_t before = place_in(same);
            o.order[place + before] = (int32_t)row;
            o.token_of[place + before] = (int32_t)(low + bin);
            if (before == 0) mine[bin] = place + (uint32_t)__popcll(same);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the wave's other lanes read them next
    };
    if (found <= LISTED) {
        for (uint32_t i = 0; i < found; i += 64) {
            const bool in = i + l < found;
            put(in, in ? listed_bin[wave][i + l] : 0, in ? listed[wave][i + l] : 0);
        }
    } else {
        uint32_t next = token_at(tokens, first + l, last, vocab);
        for (int64_t i = first; i < last; i += 64) {
            const uint32_t bin = next - low;
            next = token_at(tokens, i + 64 + l, last, vocab);
            put(bin < bins, bin, i + l);
        }
    }
}

// What the sums go by: order and starts above; a run is the rows of one token, in order.  Runs of more
// than `chunk` rows are cut where a multiple of it falls: a chunk's part of such a run is summed into
// parts[2 chunk] if the run holds the chunk's first place, else into parts[2 chunk + 1] (it is long, so
// it holds the first or the last), and k_embed_join adds up the parts.  runs[chunk]: the token whose long run begins
// there, or -1.
struct EmbedSums {
    const int32_t *order, *token_of, *starts;
    int64_t rows, vocab, cols, chunk;
    float scale;
    float *parts;
    int32_t *runs;
};

// A thread's share of a row, E elements: the columns of its vectors of V.
template <int V, int E> struct Columns {
    static constexpr int N = E / V;
    int64_t at[N], cols;
    // from column c on, `apart` columns from one to the next; OVER: the last whole
    template <bool OVER> __device__ __forceinline__ void set(int64_t c, int64_t apart, int64_t n) {
        cols = n;
#pragma unroll
        for (int k = 0; k < N; k++) at[k] = c + k * apart < cols && OVER ? whole_vector<V>(c + k * apart, cols) : c + k * apart;
    }
};
template <typename T, int V, int E> struct Share {
    static constexpr int N = E / V;
    Piece<T, V> e[N];
    __device__ __forceinline__ void fetch(const T *row, const Columns<V, E> &c) {
#pragma unroll
        for (int n = 0; n < N; n++)
            if (c.at[n] < c.cols) e[n].fetch(row + c.at[n], c.cols - c.at[n]);
    }
    __device__ __forceinline__ void add_to(float (&f)[N][V]) const {
#pragma unroll
        for (int n = 0; n < N; n++)
#pragma unroll
            for (int j = 0; j < V; j++) f[n][j] += e[n].at(j);
    }
    // scale f [+ what is there]; stores of a whole table go past the caches: the gradient of 16384 rows into 268 MB
    // 63 us, else 105; of 4000 rows into 34 MB 18, else 21
    template <bool ADD>
    static __device__ __forceinline__ void put(T *row, const Columns<V, E> &c, float scale, float (&f)[N][V]) {
#pragma unroll
        for (int n = 0; n < N; n++) {
            if (c.at[n] >= c.cols) continue;
            T *p = row + c.at[n];
            Piece<T, V> old;
            if (ADD) old.fetch(p, c.cols - c.at[n]);
#pragma unroll
            for (int j = 0; j < V; j++) f[n][j] = (ADD ? old.at(j) : 0.0f) + f[n][j] * scale;
            Piece<T, V>::template store<!ADD>(p, c.cols - c.at[n], f[n]);
        }
    }
};

// Adds a share of the rows order[from, to), FLY rows in flight.  The places of 32 rows come in one load, by 32
// lanes of a row (all of a row's lanes are here), where it has as many: with a load for each, a run of 32 rows
// waited 16 times, and 8191 x 2051 f16 took 48 us.
template <typename T, int V, int E>
__device__ __forceinline__ void add_run(const EmbedSums &s, const T *drows, int64_t stride, int64_t from, int64_t to,
                                        const Columns<V, E> &c, int log_l, float (&f)[E / V][V]) {
    constexpr int FLY = sizeof(T) * E > 16 ? 4 : 8;
    const int l = threadIdx.x & 31, half = threadIdx.x & 32;
    for (int64_t base = from; base < to; base += 32) {
        const int n = to - base < 32 ? (int)(to - base) : 32;
        const int32_t mine = s.order[base + (l < n ? l : 0)];
        for (int i = 0; i < n; i += FLY) {
            Share<T, V, E> e[FLY];
#pragma unroll
            for (int k = 0; k < FLY; k++) {
                if (i + k >= n) break;
                const int32_t row = log_l >= 5 ? __shfl(mine, half + i + k) : s.order[base + i + k];
                e[k].fetch(drows + row * stride, c);
            }
#pragma unroll
            for (int k = 0; k < FLY; k++)
                if (i + k < n) e[k].add_to(f);
        }
    }
}

// The parts of long runs in chunk j, by a workgroup.
template <typename T>
__device__ __forceinline__ void sum_parts(const EmbedSums &s, const T *drows, int64_t stride, int64_t j) {
    constexpr int V = JOINT<T, float>;
    const int64_t from = j * s.chunk, n = s.starts[s.vocab], to = from + s.chunk < n ? from + s.chunk : n;
    const bool first_columns = blockIdx.y == 0 && threadIdx.x == 0;
    if (from >= to) {
        if (first_columns) s.runs[j] = -1;
        return;
    }
    const int64_t va = s.token_of[from], vb = s.token_of[to - 1];
    if (first_columns) {
        const int64_t a = s.starts[vb], b = s.starts[vb + 1];
        s.runs[j] = b - a > s.chunk && a >= from ? (int32_t)vb : -1;
    }
    for (int k = 0; k < (va == vb ? 1 : 2); k++) {
        const int64_t v = k ? vb : va, a = s.starts[v], b = s.starts[v + 1];
        if (b - a <= s.chunk) continue;
        for (int64_t first = blockIdx.y * 2048; first < s.cols; first += gridDim.y * 2048) {
            Columns<V, 8> c;
            c.template set<true>(first + threadIdx.x * V, 256 * V, s.cols);
            float f[8 / V][V] = {};
            add_run<T, V, 8>(s, drows, stride, a > from ? a : from, b < to ? b : to, c, 8, f);
            Share<float, V, 8>::template put<false>(s.parts + (2 * j + k) * s.cols, c, 1.0f, f);
        }
    }
}

// The first `chunks` workgroups: parts of long runs.  The others: 2^log_l threads for ROWS rows of the table (the
// zeros of tokens that do not occur first, which wait for nothing), or with ADD for a place of the order, the first of
// its token.
//
// Bound by memory, most of it stores: 16384 rows bf16 into 32768 x 2048 f32 48 us for 335 MB (6.9 TB/s, past the
// caches), behind 8.2 us of order and in front of 6.6 us of long runs; added to such a table 44 us for 156 MB (3.5 TB/s:
// each row of it waits for its places, its rows and what is there).  E elements a thread: 16 spare rows of just over
// 2048 columns a second turn for the rest (8191 rows f16, none of them padding, into 20011 x 2051 36.1 us, with 8 43.0), 8
// are faster for narrower ones (4096 into 32768 x 64 f32 15.3 us, with 16 17.2; 16384 into 32768 x 2048 f32 62.8, with 16
// 71.3).  Two rows of the table where they are short: 8191 rows f16 into 20011 x 2051 36.1 us, with one 39.9; 16384 bf16
// into 32768 x 2048 f32 70.1 us, with one 62.8; between them (8192 bf16 into 32768 x 1024 f32 36.6 and 36.1) it is the same.
template <typename T, typename O, bool ADD, int E, int ROWS>
__global__ __launch_bounds__(256) void k_embed_sum(EmbedSums s, const T *drows, int64_t stride, O *out,
                                                   int64_t out_stride, int64_t from, int64_t chunks, int log_l) {
    if (blockIdx.x < chunks) return sum_parts(s, drows, stride, blockIdx.x);
    constexpr int V = JOINT<T, O>;
    const int64_t group = from + ((blockIdx.x - chunks) << (8 - log_l)) + (threadIdx.x >> log_l);
    const int64_t turn = (int64_t)E << log_l;
    if (blockIdx.y * turn >= s.cols) return;  // the grid's columns go by pieces of 2048, those of the chunks
    int64_t v = group * ROWS;
    if (ADD) {
        const int64_t a = group;
        if (a >= s.rows || a >= s.starts[s.vocab]) return;
        v = s.token_of[a];
        if (a && s.token_of[a - 1] == v) return;
    } else if (v >= s.vocab) {
        return;
    }
    int32_t at[ROWS + 1];
#pragma unroll
    for (int k = 0; k <= ROWS; k++) at[k] = s.starts[v + k < s.vocab ? v + k : s.vocab];
    for (int64_t first = blockIdx.y * turn; first < s.cols; first += gridDim.y * turn) {
        Columns<V, E> c;
        c.template set<!ADD>(first + (threadIdx.x & ((1 << log_l) - 1)) * V, (int64_t)V << log_l, s.cols);
#pragma unroll
        for (int k = 0; k < ROWS; k++) {
            float f[E / V][V] = {};
            if (!ADD && v + k < s.vocab && at[k] == at[k + 1])
                Share<O, V, E>::template put<ADD>(out + (v + k) * out_stride, c, 0.0f, f);
        }
#pragma unroll
        for (int k = 0; k < ROWS; k++) {
            if (at[k] == at[k + 1] || at[k + 1] - at[k] > s.chunk) continue;
            float f[E / V][V] = {};
            add_run<T, V, E>(s, drows, stride, at[k], at[k + 1], c, log_l, f);
            Share<O, V, E>::template put<ADD>(out + (v + k) * out_stride, c, s.scale, f);
        }
    }
}

// The long run that begins in chunk blockIdx.y, if there is one: 512 columns (blockIdx.x), eight waves on its
// parts in turn, then their sums in order.  Latency, 4.1 to 6.7 us: a launch and three loads that wait for each other,
// and the parts of the longest run (with 16 waves, and each workgroup to find out whether a run begins, 10 us).  Rows of
// fewer than 512 columns leave lanes idle: 32768 rows of 64 into 1000 take it 12 us, with 16 lanes of a wave at work.
constexpr int JOIN_COLS = 512;
template <typename O, bool ADD>
__global__ __launch_bounds__(JOIN_COLS) void k_embed_join(EmbedSums s, O *out, int64_t out_stride) {
    constexpr int WAVES = JOIN_COLS / 64;
    __shared__ float sh[WAVES][JOIN_COLS];
    const int64_t j = blockIdx.y, v = s.runs[j];
    if (v < 0) return;
    const int64_t a = s.starts[v], b = s.starts[v + 1], from = j * s.chunk;
    const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int64_t c = (int64_t)blockIdx.x * JOIN_COLS + l * 4, last = (b - 1) / s.chunk;
    float f[8] = {};
    for (int64_t k = j + wave; k <= last; k += 2 * WAVES) {
        Piece<float, 4> e[2][2];
#pragma unroll
        for (int p = 0; p < 2; p++) {
            const int64_t q = k + p * WAVES;
            const float *part = s.parts + (2 * q + (q == j && a > from)) * s.cols;
            if (q <= last)
#pragma unroll
                for (int i = 0; i < 2; i++) e[p][i].fetch(part + c + i * 256, s.cols - c - i * 256);
        }
#pragma unroll
        for (int p = 0; p < 2; p++)
            if (k + p * WAVES <= last)
#pragma unroll
                for (int i = 0; i < 8; i++) f[i] += e[p][i / 4].at(i % 4);
    }
#pragma unroll
    for (int i = 0; i < 8; i++) sh[wave][i / 4 * 256 + l * 4 + i % 4] = f[i];
    __syncthreads();
    const int64_t mine = (int64_t)blockIdx.x * JOIN_COLS + threadIdx.x;
    if (mine >= s.cols) return;
    float sum = 0;
    for (int w = 0; w < WAVES; w++) sum += sh[w][threadIdx.x];
    O *p = out + v * out_stride + mine;
    *p = from_f32<O>((ADD ? to_f32(*p) : 0.0f) + sum * s.scale);
}

// ------------------------------------------------------------------ launches

// threads of `share` elements for a row: a power of two, at most a workgroup
int log_lanes(int64_t cols, int share) {
    int l = 0;
    while (l < 8 && ((int64_t)share << l) < cols) l++;
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
    const int l = log_lanes(cols, 8);
    return typed(out_type, [&](auto ty) {
        typedef decltype(ty) O;
        return in_parts(rows, 1 << l, [&](int64_t first, int64_t n) {
            const int64_t blocks = (n + (256 >> l) - 1) >> (8 - l);
            auto go = [&](auto past) {
                k_embed<T, O, decltype(past)::value><<<dim3((uint32_t)blocks), 256, 0, stream>>>(
                    table, table_stride, table_scale, vocab, cols, tokens, first, first + n, scale, (O *)out, out_stride,
                    l);
                return launched();
            };
            return rows * cols * (int64_t)z >= (int64_t)64 << 20 ? go(Flag<true>{}) : go(Flag<false>{});
        });
    });
}

// Bins of a workgroup of k_token_order: 256 workgroups, as far as LDS has room.
int log_bins(int64_t vocab) {
    int b = 0;
    while (b < 9 && ((int64_t)256 << b) < vocab) b++;
    return b;
}
// Rows of a chunk: at most 2048 chunks, so 64 at 131072 rows and more beyond.  Long runs are read by as many workgroups
// as they have chunks, and their parts by fewer: 500 rows f16 into 4001 x 1001 f32 in chunks of 8 13.4 us, of 16 14.6, of
// 32 18.2; 4000 rows bf16 into 1000 x 4096 f32 22.1, 22.7 and 29.1 us; 16384 f32 into 1000 x 512 33.9, 29.2 and 31.7 us.
int64_t chunk_rows(int64_t rows) {
    int64_t c = rows <= 2048 ? 8 : 16;
    while (c * 2048 < rows) c *= 2;
    return c;
}
struct EmbedPlan {
    int64_t chunk, chunks;
    size_t order, starts, runs, parts;  // bytes
};
EmbedPlan embed_plan(int64_t rows, int64_t vocab, int64_t cols) {
    EmbedPlan p;
    p.chunk = chunk_rows(rows);
    p.chunks = rows > p.chunk ? (rows + p.chunk - 1) / p.chunk : 0;  // without a long run none are needed
    p.order = (size_t)round_up(rows * 4, 16);
    p.starts = (size_t)round_up((vocab + 1) * 4, 16);
    p.runs = (size_t)round_up(p.chunks * 4, 16);
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
    *bytes = 2 * p.order + p.starts + p.runs + p.parts;
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
    const int b = log_bins(vocab), share = cols > 2048 ? 16 : 8, l = log_lanes(cols, share);
    char *w = (char *)ws;
    const TokenOrder o{(int32_t *)w, (int32_t *)(w + p.order), (int32_t *)(w + 2 * p.order)};
    const EmbedSums a{o.order, o.token_of, o.starts, rows, vocab, cols, p.chunk, scale,
                      (float *)(w + 2 * p.order + p.starts + p.runs), (int32_t *)(w + 2 * p.order + p.starts)};
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
                // wide rows by workgroups of 2048 columns, as far as a grid goes
                const uint32_t turns = (uint32_t)(cols > 64 * 2048 ? 64 : (cols + 2047) / 2048);
                auto sum = [&](auto elements, auto table_rows) {
                    constexpr int E = decltype(elements)::value, ROWS = decltype(table_rows)::value;
                    return in_parts(ADD ? rows : (vocab + ROWS - 1) / ROWS, turns << l, [&](int64_t first, int64_t n) {
                        k_embed_sum<T, O, ADD, E, ROWS>
                            <<<dim3((uint32_t)(((n + (256 >> l) - 1) >> (8 - l)) + chunks), turns), 256, 0, s>>>(
                                a, (const T *)drows, drows_stride, (O *)out, out_stride, first, chunks, l);
                        chunks = 0;
                        return launched();
                    });
                };
                const bool two = cols * sizeof(O) < 6144;
                int e;
                if constexpr (ADD)
                    e = share == 16 ? sum(Int<16>{}, Int<1>{}) : sum(Int<8>{}, Int<1>{});
                else if constexpr (sizeof(O) == 4)  // 16 elements: rows of 8 KB at least
                    e = share == 16 ? sum(Int<16>{}, Int<1>{}) : two ? sum(Int<8>{}, Int<2>{}) : sum(Int<8>{}, Int<1>{});
                else  // 8 elements: rows of 4 KB at most
                    e = share == 8 ? sum(Int<8>{}, Int<2>{}) : two ? sum(Int<16>{}, Int<2>{}) : sum(Int<16>{}, Int<1>{});
                if (e || !p.chunks) return e;
                // chunks, at most 2048, as the dimension of few
                k_embed_join<O, ADD><<<dim3((uint32_t)((cols + JOIN_COLS - 1) / JOIN_COLS), (uint32_t)p.chunks), JOIN_COLS,
                                       0, s>>>(a, (O *)out, out_stride);
                return launched();
            };
            return add ? go(Flag<true>{}) : go(Flag<false>{});
        });
    });
}
