// Host check of where a wave is in a packed batch (gdn2_packed.h), against a
// plain list of boundaries: the starts, ends and sequences that every slice of
// 8 tokens reports, for waves that walk as the kernels' do - consecutive tokens
// (the convolution's slices, its gradients' with the rows behind, the
// recurrence's chunks) and 8 of every 64 (the recurrence's groups) - and the
// starts and ranks that divide a batch into groups; and the channels of lanes.
// Built with g++ by tests/test_packed_host.py; prints "ok" and exits 0.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <numeric>
#include <random>
#include <string>
#include <vector>

#include "gdn2_packed.h"

using namespace gdn2::dev;

constexpr int R = 8;
static long failures = 0, slices = 0;
static std::string batch;

struct Batch {
    std::vector<int> cu, owner;  // owner: each token's sequence
    std::vector<char> start, last;
    Packed p;
    explicit Batch(const std::vector<int> &lens, int behind = 0)
    {
        cu.push_back(0);
        for (int l : lens) {
            owner.insert(owner.end(), l, (int)cu.size() - 1);
            cu.push_back(cu.back() + l);
        }
        const int n = cu.back();
        start.assign(n, 0);
        last.assign(n, 0);
        for (size_t s = 0; s < lens.size(); ++s)
            if (lens[s] > 0) start[cu[s]] = last[cu[s + 1] - 1] = 1;
        p = Packed{cu.data(), 0, (int)lens.size(), n + behind};
    }
    int tokens() const { return cu.back(); }
};

// One wave over [lo, hi), 8 tokens of every `step`.
static void walk(const Batch &b, const char *how, int lo, int hi, int step, bool looks_first)
{
    if (lo >= hi) return;
    Cursor cur(b.p);
    if (looks_first && cur.at(lo) != b.owner[lo] && failures++ < 20) fprintf(stderr, "%s: %s: at(%d)\n", batch.c_str(), how, lo);
    Slice<R> s;
    for (int t = lo; t < hi; t += step) {
        s.set(cur, t, hi, b.tokens());
        ++slices;
        uint32_t starts = 0, lasts = 0;
        bool ok = s.cnt == std::min(R, hi - t) && s.t0 == t;
        for (int i = 0; i < std::min(R, hi - t); ++i) {
            starts |= (uint32_t)b.start[t + i] << i;
            lasts |= (uint32_t)b.last[t + i] << i;
            ok = ok && s.seq(i) == b.owner[t + i];
        }
        if (!(ok && s.starts == starts && s.lasts == lasts) && failures++ < 20)
            fprintf(stderr, "%s: %s, [%d, %d): tokens from %d: starts %x lasts %x of %d, not %x %x of %d\n", batch.c_str(), how, lo, hi,
                    t, s.starts, s.lasts, s.seq(0), starts, lasts, b.owner[t]);
    }
}

static void check(const std::string &name, const std::vector<int> &lens, std::vector<int> groups = {})
{
    batch = name;
    const Batch b(lens, 37);
    const int T = b.tokens(), N = (int)lens.size();
    for (int n : {8, 16, 32, 64, 128, 256})
        for (int lo = 0; lo < T; lo += n) {
            walk(b, "slice", lo, std::min(lo + n, T), R, true);
            walk(b, "chunk", lo, std::min(lo + n, T), R, false);
            walk(b, "slice and 3 rows", lo, std::min(lo + n + 3, T), R, true);
        }
    walk(b, "all", 0, T, R, false);
    groups.push_back(1);
    groups.push_back(7);
    for (int g : groups) {
        int end = 0;
        for (int r = 0; r < g; ++r) {
            const int t = (int)((int64_t)b.p.T * r / g);
            const int lo = b.p.start_from(t), hi = r + 1 < g ? b.p.start_from((int)((int64_t)b.p.T * (r + 1) / g)) : T;
            int want = T;
            for (int s = N - 1; s >= 0; --s)
                if (b.cu[s] >= t) want = b.cu[s];
            if ((lo != want || lo != end) && failures++ < 20) fprintf(stderr, "%s: group %d of %d begins at %d, not %d\n", name.c_str(), r, g, lo, want);
            end = hi;
            for (int w = 0; w < 8; ++w) walk(b, "group", lo + w * R, hi, 64, false);
        }
    }
    if (N <= 64) {
        std::vector<int> order(N);
        std::iota(order.begin(), order.end(), 0);
        std::stable_sort(order.begin(), order.end(), [&](int x, int y) { return lens[x] > lens[y]; });
        for (int r = 0; r < N; ++r) {
            int lo, hi;
            b.p.by_length(r, lo, hi);
            if ((lo != b.cu[order[r]] || hi != b.cu[order[r] + 1]) && failures++ < 20)
                fprintf(stderr, "%s: rank %d is [%d, %d)\n", name.c_str(), r, lo, hi);
            for (int w = 0; w < 8; ++w) walk(b, "rank", lo + w * R, hi, 64, false);
        }
    }
}

// Every channel has a place among its own workgroup's 64 VEC, and no lane one outside.
template <int VEC>
static void check_channels(int D)
{
    const int width = 64 * VEC, blocks = (D + width - 1) / width;
    for (int b = 0; b < blocks; ++b) {
        std::vector<char> seen(width, 0);
        for (int lane = 0; lane < 64; ++lane) {
            const Channels<VEC> at(b, lane, D);
            bool ok = (int)at.col + VEC <= D && at.on == (b * width + lane * VEC < D);
            for (int v = 0; v < VEC; ++v) {
                const int c = at.place(v);
                ok = ok && c < width && (c >= 0 ? at.on && b * width + c == (int)at.col + v : !at.on || (int)at.col + v < b * width);
                if (c >= 0 && c < width) seen[c] = 1;
            }
            if (!ok && failures++ < 20) fprintf(stderr, "D = %d, block %d, lane %d of %d channels\n", D, b, lane, VEC);
        }
        for (int c = 0; c < width; ++c)
            if (seen[c] != (b * width + c < D) && failures++ < 20) fprintf(stderr, "D = %d, block %d: channel %d\n", D, b, c);
    }
}

int main()
{
    for (int D = 1; D <= 1100; ++D) {
        check_channels<1>(D);
        if (D >= 2) check_channels<2>(D);
    }
    for (int D : {2049, 4097, 8193, (1 << 20) + 1}) check_channels<2>(D);
    check("1000 of 64", std::vector<int>(1000, 64), {16});
    check("65 of 1 and one of 300", [] { std::vector<int> l(65, 1); l.push_back(300); return l; }());
    {
        std::vector<int> l(12, 20);
        l.insert(l.end(), 64, 1);
        l.insert(l.end(), 51, 8);
        l.push_back(16384);
        check("12 of 20, 64 of 1, 51 of 8, one of 16384", l);
    }
    std::mt19937 rng(1);
    auto up_to = [&](int n) { return (int)(rng() % (unsigned)n); };
    for (int n : {1, 2, 63, 64, 65, 66, 100, 127, 128, 129, 193, 256, 257, 1024, 2000, 4160})
        for (int kind = 0; kind < 6; ++kind) {
            std::vector<int> l(n);
            for (int &x : l)
                x = kind == 0 ? 8 * (1 + up_to(12)) : kind == 1 ? up_to(5) : kind == 2 ? 1 + up_to(4) : kind == 3 ? 8
                    : kind == 4 ? (up_to(3) ? 0 : 8 * up_to(4)) : up_to(60);
            if (kind == 2 && n > 65) l[n / 2] = 1000;
            check(std::to_string(n) + " sequences, kind " + std::to_string(kind), l, {2, 16, 64});
        }
    if (failures) {
        fprintf(stderr, "%ld of %ld slices\n", failures, slices);
        return 1;
    }
    printf("ok\n");
    return 0;
}
