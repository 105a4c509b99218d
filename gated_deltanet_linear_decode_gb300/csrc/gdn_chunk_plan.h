// gdn_chunk_plan.h -- how gdn_attn_chunk's work is divided.  Host and device code.
//
// A unit is up to `tokens` consecutive new tokens of one sequence with one kv head's G query heads: tokens * G rows that share
// their keys, and see them up to their last token's.  Units are numbered by sequence, kv head, place in the sequence, and lie
// one after another on a line: a unit takes `cost` numbers for its begin and end, then one for every key that it sees.  The
// line is divided evenly over the workers; a tile of a unit belongs to the worker in whose share its first key's number lies,
// and a unit without keys to the one that has its first number.  (Numbers are keys, not tiles, because then what the first u
// units of a sequence take is a sum in closed form, and a worker finds its first unit by bisection.)
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define GDN_HD __host__ __device__ __forceinline__
#else
#define GDN_HD inline
#endif

namespace gdn {
namespace chunk {

GDN_HD long long least(long long a, long long b) { return a < b ? a : b; }
GDN_HD long long most(long long a, long long b) { return a > b ? a : b; }
// a / b rounded down, with the short division where it will do (a, b >= 0).
GDN_HD long long quot(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// The new tokens of one sequence: n rows from row0 on, the last n of its len tokens (len may be less than n).
struct Rows {
    int row0, n, len;
};

struct Line {
    int tokens, key_bits, cost;   // tokens of a unit, log2 of a tile's keys, numbers for a unit's begin and end

    GDN_HD int keys() const { return 1 << key_bits; }
    GDN_HD int units(const Rows& r) const { return static_cast<int>((static_cast<uint32_t>(r.n) + static_cast<uint32_t>(tokens) - 1) / static_cast<uint32_t>(tokens)); }
    // keys that unit i sees
    GDN_HD int seen(const Rows& r, int i) const {
        const long long s = least((i + 1ll) * tokens, r.n) + r.len - r.n;
        return s > 0 ? static_cast<int>(s) : 0;
    }
    // numbers of units 0..u-1 (u up to units(r))
    GDN_HD long long before(const Rows& r, int u) const {
        const int nt = units(r);
        const long long m = least(u, nt - 1), off = static_cast<long long>(r.len) - r.n;   // units that are full
        long long sum = static_cast<long long>(u) * cost;
        const long long i0 = off >= 0 ? 0 : least(m, quot(-off, tokens));   // those before see nothing
        if (i0 < m) sum += (m - i0) * off + tokens * (m * (m + 1) / 2 - i0 * (i0 + 1) / 2);
        if (u == nt && nt > 0) sum += most(r.len, 0);
        return sum;
    }
    GDN_HD long long head(const Rows& r) const { return r.n > 0 ? before(r, units(r)) : 0; }
};

// Worker w's share of `total` numbers among `workers`: [first, last).
struct Share {
    long long first, last, total;
    int workers;
    GDN_HD static Share of(long long total, int workers, int w) {
        return Share{quot(total * w, workers), quot(total * (w + 1), workers), total, workers};
    }
    // the worker that has number x
    GDN_HD int owner(long long x) const { return static_cast<int>(quot((x + 1) * workers - 1, total)); }
};
// Workers that take part: shares of less than `tile` keys would leave some of them without one.
GDN_HD int workers_of(long long total, int workers, int min_share) { return static_cast<int>(most(1, least(workers, quot(total, min_share)))); }

// A worker's part of a unit: tiles [t0, t1) of `tiles`.
struct Part {
    Rows r;
    int units;      // of the sequence and a kv head
    int b, hk, i, seen, tiles, t0, t1;
    long long at;   // the unit's first number

    GDN_HD bool whole() const { return t0 == 0 && t1 == tiles; }
};

// The tiles of the unit that the share holds; false if there is nothing of it.
GDN_HD bool clip(const Line& ln, const Share& sh, Part& c) {
    const int up = ln.keys() - 1;
    c.seen = ln.seen(c.r, c.i);
    c.tiles = static_cast<int>((static_cast<uint32_t>(c.seen) + up) >> ln.key_bits);
    const long long base = c.at + ln.cost;   // the first tile's number
    c.t0 = sh.first > base ? static_cast<int>(least(c.tiles, (sh.first - base + up) >> ln.key_bits)) : 0;
    c.t1 = sh.last > base ? static_cast<int>(least(c.tiles, (sh.last - base + up) >> ln.key_bits)) : 0;
    return c.tiles > 0 ? c.t0 < c.t1 : c.at >= sh.first && c.at < sh.last;
}

// On to the next unit with something in the share; false at the share's end.  rows(b): the Rows of sequence b.
template <class F>
GDN_HD bool next_part(const Line& ln, const Share& sh, int B, int Hkv, Part& c, F rows) {
    for (;;) {
        c.at += ln.cost + c.seen;
        if (c.at >= sh.last) return false;
        if (++c.i == c.units) {
            c.i = 0;
            if (++c.hk == Hkv) {
                c.hk = 0;
                do {
                    if (++c.b >= B) return false;
                    c.r = rows(c.b);
                } while (c.r.n == 0);
                c.units = ln.units(c.r);
            }
        }
        if (clip(ln, sh, c)) return true;
    }
}

// The unit that has number sh.first; false if none of its tiles is the share's (then next_part's is the first).  c.b, c.r are the
// sequence that has the number, `start` the number where it begins.
GDN_HD bool first_part(const Line& ln, const Share& sh, long long start, Part& c) {
    const long long head = ln.head(c.r), in = sh.first - start;
    c.hk = static_cast<int>(quot(in, head));
    const long long x = in - c.hk * head;
    c.units = ln.units(c.r);
    int lo = 0, hi = c.units;   // the last unit with before(unit) <= x
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (ln.before(c.r, mid) <= x) lo = mid;
        else hi = mid;
    }
    c.i = lo;
    c.at = sh.first - x + ln.before(c.r, lo);
    return clip(ln, sh, c);
}

}  // namespace chunk
}  // namespace gdn
