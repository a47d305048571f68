// Where a wave is in a packed batch: which sequences begin and end among the
// tokens that it walks over, shared by the recurrence's and the convolution's
// kernels. What lanes hold and vote on is written as a function of the lane,
// so that a host program can check it against a plain list of boundaries. Not
// part of the ABI.
#pragma once

#include <stdint.h>

#include "gdn2_index.h"

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>
#define GDN2_WAVE __device__ __forceinline__
#else
#define GDN2_WAVE inline
#endif

namespace gdn2 {
namespace dev {

// An int per lane of a wave, and the votes of its lanes: f(lane).
#if defined(__HIPCC__)
struct LaneInt {
    int own;
    template <class F>
    GDN2_WAVE void set(F f) { own = f((int)(threadIdx.x & 63)); }
    GDN2_WAVE void put(int lane, int x) { own = (int)(threadIdx.x & 63) == lane ? x : own; }
    GDN2_WAVE int of(int) const { return own; }  // (of the lane that asks)
    GDN2_WAVE int read(int lane) const { return __builtin_amdgcn_readlane(own, lane); }
};
template <class F>
GDN2_WAVE uint64_t vote(F f)
{
    return __ballot(f((int)(threadIdx.x & 63)));
}
#else
struct LaneInt {
    int v[64];
    template <class F>
    void set(F f)
    {
        for (int i = 0; i < 64; ++i) v[i] = f(i);
    }
    void put(int lane, int x) { v[lane] = x; }
    int of(int lane) const { return v[lane]; }
    int read(int lane) const { return v[lane & 63]; }  // (the hardware takes the lane's low six bits)
};
template <class F>
uint64_t vote(F f)
{
    uint64_t m = 0;
    for (int i = 0; i < 64; ++i) m |= (uint64_t)(f(i) ? 1 : 0) << i;
    return m;
}
#endif

// The channels of a lane: VEC neighbouring ones from `col` on, of the 64 VEC that
// a wave takes from `base` on. With VEC = 2 and an odd D the last pair begins at
// the last channel but one, which may lie in front of `base` (D = 64 VEC k + 1).
template <int VEC>
struct Channels {
    uint32_t base, col;
    bool on;  // (lanes past the last channel read the last pair and store nothing)
    GDN2_WAVE Channels(uint32_t block, int lane, int D)
    {
        base = block * (64 * VEC);
        const uint32_t c0 = base + lane * VEC, last = (uint32_t)D - VEC;
        on = c0 < (uint32_t)D;
        col = c0 < last ? c0 : last;
    }
    // The place of channel col + v among the wave's own 64 VEC, or -1: another workgroup's, or no lane's to store.
    GDN2_WAVE int place(int v) const { return on && col + v >= base ? (int)(col + v - base) : -1; }
};

// A packed batch. Every token and sequence index that is derived from
// cu_seqlens stays in [0, T] and [0, N), whatever the array holds.
struct Packed {
    const void *cu;
    int cu64, N, T;
    GDN2_WAVE int entry(int i) const  // cu[i], in [0, T]
    {
        const int64_t v = cu_raw(cu, cu64, i);
        return (int)(v < 0 ? 0 : v > T ? T : v);
    }
    GDN2_WAVE int tokens() const { return cu ? entry(N) : T; }  // behind the last sequence's end: none
    // The first sequence start at or behind token t (the last sequence's end if there is none). Wave-uniform.
    GDN2_WAVE int start_from(int t) const
    {
        if (!cu) return t > 0 ? T : 0;
        int lo = 0, hi = N;  // starts before lo lie before t, those from hi on do not
        while (lo < hi) {
            const int step = (hi - lo + 63) / 64;
            const int c = __builtin_popcountll(vote([&](int lane) { return lo + lane * step < hi && entry(lo + lane * step) < t; }));
            if (c == 0) break;
            const int last = lo + (c - 1) * step;
            hi = step == 1 ? lo + c : last + step < hi ? last + step : hi;
            lo = last + 1;
        }
        return entry(lo < N ? lo : N);
    }
    // The tokens of the sequence of a rank by length, the longest first (N <= 64).
    GDN2_WAVE void by_length(int rank, int &lo, int &hi) const
    {
        LaneInt s, len, before;
        s.set([&](int lane) { return lane < N ? entry(lane) : 0; });
        len.set([&](int lane) {
            const int e = lane < N ? entry(lane + 1) : 0;
            return e > s.of(lane) ? e - s.of(lane) : 0;
        });
        before.set([&](int) { return 0; });
        for (int j = 0; j < N; ++j) {
            const int l = len.read(j);
            before.set([&](int lane) { return before.of(lane) + (l > len.of(lane) || (l == len.of(lane) && j < lane)); });
        }
        const int n = __builtin_ctzll(vote([&](int lane) { return lane < N && before.of(lane) == rank; }));
        lo = s.read(n);
        hi = lo + len.read(n);
    }
};

// The sequence of each token, for tokens in (mostly) rising order. A lane
// holds the end of one of 64 sequences; all members are wave-uniform else.
struct Cursor {
    Packed b;
    int base = 0, from = 0;
    LaneInt win = {};
    bool held = false;
    int n_in = 0, b_in = 0, e_in = 0;  // tokens b_in .. e_in - 1 are known to lie in sequence n_in

    GDN2_WAVE explicit Cursor(const Packed &p) : b(p) {}
    GDN2_WAVE void seek(int t)
    {
        int lo = 0, hi = b.N;  // sequences before lo end at or before t, those from hi on do not
        while (hi - lo > 64) {
            const int step = (hi - lo + 63) / 64;
            const int c =
                __builtin_popcountll(vote([&](int lane) { return lo + lane * step < hi && b.entry(lo + lane * step + 1) <= t; }));
            if (c == 0) {
                hi = lo;
                break;
            }
            const int last = lo + (c - 1) * step;
            hi = last + step < hi ? last + step : hi;
            lo = last + 1;
        }
        base = lo;
        from = t;
        win.set([&](int lane) { return base + lane < b.N ? b.entry(base + lane + 1) : INT32_MAX; });
        held = true;
    }
    // The sequence that holds token t (t < tokens()).
    GDN2_WAVE int at(int t)
    {
        if (!b.cu) return 0;
        if (!held || t < from) seek(t);
        auto ended = [&]() { return __builtin_popcountll(vote([&](int lane) { return win.of(lane) <= t; })); };
        int c = ended();
        if (c == 64) {
            seek(t);
            c = ended();
        }
        return base + c < b.N ? base + c : b.N - 1;
    }
    // Remembers that token t lies in sequence n. The lanes may have moved on to
    // later sequences since n was found (n < base): then its end is not known.
    GDN2_WAVE void inside(int n, int t)
    {
        n_in = n;
        b_in = t;
        e_in = n >= base && n - base < 64 ? win.read(n - base) : 0;
    }
};

// R tokens of one wave: [t0, t0 + cnt), which of them begin and end their
// sequences (bits), and the sequence of token i in lane i.
template <int R>
struct Slice {
    int t0, cnt;
    LaneInt nn;
    uint32_t starts, lasts;

    GDN2_WAVE void set(Cursor &cur, int t, int hi, int tokens)
    {
        t0 = t;
        cnt = hi - t < 0 ? 0 : hi - t < R ? hi - t : R;
        starts = lasts = 0;
        nn.set([](int) { return 0; });
        if (cnt == 0) return;
        if (!cur.b.cu) {
            starts = t == 0;
            lasts = t + cnt == tokens ? 1u << (cnt - 1) : 0;
            return;
        }
        if (t > cur.b_in && t + R < cur.e_in) {  // well inside a sequence
            nn.set([&](int) { return cur.n_in; });
            return;
        }
        int before = t > 0 ? cur.at(t - 1) : -1;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (i >= cnt) break;
            const int n = cur.at(t + i);
            if (n != before) {
                starts |= 1u << i;
                lasts |= i > 0 ? 1u << (i - 1) : 0;
            }
            nn.put(i, n);
            before = n;
        }
        if (t + cnt >= tokens || cur.at(t + cnt) != before) lasts |= 1u << (cnt - 1);
        cur.inside(before, t + cnt - 1);
    }
    GDN2_WAVE int seq(int i) const { return nn.read(i); }
};

}  // namespace dev
}  // namespace gdn2
