// The sampler's selection from a list (csrc/plain/sample.hip, Sampler::select) as
// host code: against a sort, by count and by mass, and on lists that hold an order
// more than once, where it still has to end.
#include "sample_device.inc"

#include <algorithm>
#include <random>

using namespace ckks_plain;
static SampleArgs args;
static SampleShared shared;

// select on every thread's share of the list; ends, and all threads agree
template <bool BY_MASS> static bool select(const std::vector<uint64_t> &list, float top, uint64_t want, uint64_t &last,
                                           uint64_t &until) {
    std::vector<uint64_t> got(NT), upto(NT);
    const bool ends = host::run(NT, 3000, [&] {
        Sampler<float> s{args, shared, nullptr, nullptr, nullptr, (int)(threadIdx.x / 64), 0, 1.0f, 1.44269504f, top};
        uint64_t o[HELD], u = 0;
        for (int i = 0; i < HELD; i++) {
            const size_t at = threadIdx.x + (size_t)i * NT;
            o[i] = at < list.size() ? list[at] : 0;
        }
        const uint32_t me = threadIdx.x;
        got[me] = s.select<BY_MASS>(o, want, 1, s.highest(top), u);
        upto[me] = u;
    });
    if (!ends) return false;
    for (int t = 0; t < NT; t++)
        if (got[t] != got[0] || upto[t] != upto[0]) return false;
    last = got[0], until = upto[0];
    return true;
}

int main() {
    args.vocab = 50000, args.index_bits = 16;
    std::mt19937 rng(7);
    int bad = 0;
    for (int kind = 0; kind < 4; kind++) {  // spread, few values, all equal, one value many times
        const size_t n = kind == 2 ? (size_t)LIST : 3000 + 301 * kind;
        float top = -INFINITY;
        std::vector<float> z(n);
        for (float &v : z) {
            v = kind == 0 ? std::normal_distribution<float>()(rng) : kind == 1 ? (float)(rng() % 5) : kind == 2 ? 1.0f : rng() % 3 ? 0.5f : -(float)(rng() % 9);
            top = std::max(top, v);
        }
        Sampler<float> s{args, shared, nullptr, nullptr, nullptr, 0, 0, 1.0f, 1.44269504f, top};
        std::vector<uint64_t> list(n);
        for (size_t i = 0; i < n; i++) list[i] = s.order_of(z[i], (uint32_t)i);
        std::vector<uint64_t> sorted = list;
        std::sort(sorted.rbegin(), sorted.rend());
        std::vector<uint64_t> sums(n);
        uint64_t sum = 0;
        for (size_t i = 0; i < n; i++) sums[i] = sum += s.both(sorted[i]);
        std::shuffle(list.begin(), list.end(), rng);
        for (size_t want : {(size_t)1, (size_t)2, n / 3, n - 1, n}) {
            uint64_t last = 0, until = 0;
            if (!select<false>(list, top, want, last, until) || last != sorted[want - 1] || until != sums[want - 1])
                bad++, printf("by count: kind %d want %zu\n", kind, want);
            const uint64_t mass = sums[want - 1] & Sampler<float>::MASS;
            if (!select<true>(list, top, mass, last, until) || (until & Sampler<float>::MASS) < mass || last < sorted[want - 1])
                bad++, printf("by mass: kind %d want %zu\n", kind, want);
        }
        // the same token on the list twice and three times
        for (int twice = 0; twice < 3; twice++) {
            std::vector<uint64_t> more = list;
            more.resize(std::min<size_t>(n, LIST - 2));
            std::vector<uint64_t> order = more;
            std::sort(order.rbegin(), order.rend());
            const uint64_t again = order[twice == 0 ? 0 : twice == 1 ? order.size() / 2 : order.size() - 1];
            more.push_back(again);
            if (twice) more.push_back(again);
            order = more;
            std::sort(order.rbegin(), order.rend());
            const size_t at = std::find(order.begin(), order.end(), again) - order.begin();
            uint64_t last = 0, until = 0;
            for (size_t want : {at + 1, at + 2})
                if (!select<false>(more, top, want, last, until) || last != again)
                    bad++, printf("twice: kind %d case %d want %zu does not end at it\n", kind, twice, want);
        }
    }
    printf(bad ? "%d wrong\n" : "select: ok\n", bad);
    return bad != 0;
}
