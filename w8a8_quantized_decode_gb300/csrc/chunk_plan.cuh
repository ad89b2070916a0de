// chunk_plan.cuh -- how the attention of a chunk is cut into work: integer
// arithmetic alone, for the device and for tests on the host.
//
// A tile is up to 256 / G consecutive tokens of one request with the G query
// heads of one KV head: wide with more than 128 rows, otherwise narrow. Its work
// is counted in units: a few for its queries and results and one for every block of
// 128 keys that its last token sees (one where it sees none). Tiles are
// numbered request by request, in a request KV head by KV head, in a head by their
// tokens. A part is a contiguous range of units.
#pragma once

#include <stdint.h>

// Functions that are called, not copied into each place: a launch runs most of
// them a few times, each time from a cold instruction cache.
#ifdef __CUDACC__
#define CHUNK_CALL __host__ __device__ __noinline__ static
#else
#define CHUNK_CALL inline
#endif

namespace a8w8 {
namespace chunk {

constexpr int kKeys = 128;        // keys of a block
constexpr int kTileRows = 256;    // (token, head) rows of a tile at most

// Units of a tile beside its blocks, wide and narrow. A fit over the CTAs of several
// batches, BF16 cache, in clocks: a wide tile 7000 to 11000 and 2900 to 3300 a block,
// a narrow one 2400 to 3800 and 2200 to 2800.
constexpr int kWideCost = 3, kNarrowCost = 1;
constexpr int kMinUnits = 3;      // of a part
constexpr int kSlackShare = 8, kMaxSlack = 6;

struct Req {
    int row0;   // its first row of q
    int n;      // new tokens
    int ctx;    // tokens of its context, the new ones included
};

__host__ __device__ inline int tile_tokens(int G) { return kTileRows / G; }
__host__ __device__ inline int blocks_of(long keys) {
    return keys <= kKeys ? 1 : (int)((keys + kKeys - 1) / kKeys);
}
// Tokens of tile i, and the keys that its last token sees (not positive: none).
__host__ __device__ inline int tokens_in(const Req& r, int tpt, int i) {
    const int left = r.n - i * tpt;
    return left < tpt ? left : tpt;
}
__host__ __device__ inline long keys_of(const Req& r, int tpt, int i) {
    return (long)r.ctx - r.n + (long)i * tpt + tokens_in(r, tpt, i);
}
// (tile_tokens / 2 tokens have 128 rows at most, one more has more)
__host__ __device__ inline bool is_narrow(int tokens, int tpt) { return tokens <= tpt / 2; }
__host__ __device__ inline int cost_of(bool narrow) { return narrow ? kNarrowCost : kWideCost; }
__host__ __device__ inline int tiles_of(const Req& r, int tpt) { return (r.n + tpt - 1) / tpt; }

// sum over 0 <= k < n of floor((a k + b) / m): the whole parts of a and b taken
// out, then the lattice points counted along the other axis (Graham, Knuth,
// Patashnik, Concrete Mathematics, section 3.5). n at most 2^24, a and m at
// most 256.
CHUNK_CALL long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
    long s = 0;
    while (n > 0) {
        s += (long)((unsigned long)(n - 1) * n / 2) * (a / m) + (long)n * (b / m);
        a %= m;
        b %= m;
        const unsigned top = a * n + b;
        if (top < m) break;
        n = top / m;
        b = top - n * m;
        const unsigned t = a;
        a = m;
        m = t;
    }
    return s;
}

// Units of a head's tiles before tile i; i is at most the number of tiles - 1,
// so that they all hold tpt tokens and are wide.
CHUNK_CALL long units_before(const Req& r, int tpt, int i) {
    const int base = r.ctx - r.n;
    // tiles whose last token sees a block at most: one unit each
    int one = kKeys - base < tpt ? 0 : (kKeys - base) / tpt;
    if (one > i) one = i;
    return (long)i * kWideCost +
           one + floor_sum(i - one, kKeys, tpt, base + (one + 1) * tpt + kKeys - 1);
}
// Units of a tile, and of one KV head of a request.
__host__ __device__ inline int tile_units(const Req& r, int tpt, int i) {
    return cost_of(is_narrow(tokens_in(r, tpt, i), tpt)) + blocks_of(keys_of(r, tpt, i));
}
CHUNK_CALL long head_units(const Req& r, int tpt) {
    if (r.n <= 0) return 0;
    const int last = tiles_of(r, tpt) - 1;
    return units_before(r, tpt, last) + tile_units(r, tpt, last);
}

CHUNK_CALL long div_long(long a, long b) {
    return (a | b) >> 32 ? a / b : (long)((unsigned)a / (unsigned)b);
}

// How W units are shared by at most P parts: part c begins at W c / parts, moved
// to the nearer end of the tile where that is at most `slack` units away, as a tile
// that two parts hold costs both of them: an eighth of a part, kMaxSlack at most;
// but the tile's own cost at least, so that no part begins before a tile's second
// block.
struct Shares {
    long W, share, whole;
    int parts, rest;
    __host__ __device__ Shares(long units, int P) {
        W = units;
        parts = (int)(units < (long)P * kMinUnits ? (units + kMinUnits - 1) / kMinUnits : P);
        whole = parts > 0 ? div_long(W, parts) : 0;
        rest = (int)(W - whole * parts);
        share = whole / kSlackShare < kMaxSlack ? whole / kSlackShare : kMaxSlack;
    }
    __host__ __device__ long raw(int c) const { return whole * c + rest * c / (parts > 0 ? parts : 1); }
    __host__ __device__ long slack(bool narrow) const {
        return share > cost_of(narrow) ? share : cost_of(narrow);
    }
    __host__ __device__ long snap(long u, long tile, long tile_end, bool narrow) const {
        const long s = slack(narrow);
        if (u - tile <= s && u - tile <= tile_end - u) return tile;
        return tile_end - u <= s ? tile_end : u;
    }
    // The parts kf .. kl that begin inside a tile (more than `slack` units from
    // both ends, as snap has it), given that part c does.
    __host__ __device__ void inside(long tile, long tile_end, bool narrow, int c, int& kf, int& kl) const {
        const long s = slack(narrow);
        kf = kl = c;
        while (kf > 1 && raw(kf - 1) > tile + s) --kf;
        while (kl + 1 < parts && raw(kl + 1) < tile_end - s) ++kl;
    }
};

}  // namespace chunk
}  // namespace a8w8
