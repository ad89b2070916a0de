// chunk_plan.cuh -- how the attention of a chunk is cut into work: integer
// arithmetic alone, for the device and for tests on the host.
//
// A tile is up to 256 / G consecutive tokens of one request with the G query
// heads of one KV head; a unit is one tile's work on one block of 128 keys.
// Tiles are numbered request by request, in a request KV head by KV head, in a
// head by their tokens; a tile's units are kTileCost for its queries and results
// and then the key blocks that its last token sees (one where it sees none). A
// part is a contiguous range of units.
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
constexpr int kTileCost = 1;      // units that a tile costs beside its blocks

constexpr int kSlackShare = 8, kMinSlack = 2;

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
// so that they all hold tpt tokens.
CHUNK_CALL long units_before(const Req& r, int tpt, int i) {
    const int base = r.ctx - r.n;
    // tiles whose last token sees a block at most: one unit each
    int one = kKeys - base < tpt ? 0 : (kKeys - base) / tpt;
    if (one > i) one = i;
    return one + (long)i * kTileCost +
           floor_sum(i - one, kKeys, tpt, base + (one + 1) * tpt + kKeys - 1);
}
// Units of a tile, and of one KV head of a request.
__host__ __device__ inline int tile_units(const Req& r, int tpt, int i) {
    return kTileCost + blocks_of(keys_of(r, tpt, i));
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
// to the nearer end of the tile where that is at most `slack` units away: an
// eighth of a part, as a tile that two parts hold costs both of them, and at
// least a tile's own cost, so that no part begins before a tile's first block.
struct Shares {
    long W, slack, whole;
    int parts, rest;
    __host__ __device__ Shares(long units, int P, int min_units) {
        W = units;
        parts = (int)(units < (long)P * min_units ? (units + min_units - 1) / min_units : P);
        whole = parts > 0 ? div_long(W, parts) : 0;
        rest = (int)(W - whole * parts);
        slack = whole / kSlackShare > kMinSlack ? whole / kSlackShare : kMinSlack;
    }
    __host__ __device__ long raw(int c) const { return whole * c + rest * c / (parts > 0 ? parts : 1); }
    __host__ __device__ long snap(long u, long tile, long tile_end) const {
        if (u - tile <= slack && u - tile <= tile_end - u) return tile;
        return tile_end - u <= slack ? tile_end : u;
    }
    // The parts kf .. kl that begin inside a tile (more than `slack` units from
    // both ends, as snap has it), given that part c does.
    __host__ __device__ void inside(long tile, long tile_end, int c, int& kf, int& kl) const {
        kf = kl = c;
        while (kf > 1 && raw(kf - 1) > tile + slack) --kf;
        while (kl + 1 < parts && raw(kl + 1) < tile_end - slack) ++kl;
    }
};

}  // namespace chunk
}  // namespace a8w8
