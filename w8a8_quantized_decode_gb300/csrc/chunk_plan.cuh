// chunk_plan.cuh -- how the attention of a chunk is cut into work: integer
// arithmetic alone, for the device and for tests on the host.
//
// A tile is up to 256 / G consecutive tokens of one request with the G query
// heads of one KV head: wide with more than 128 rows, otherwise narrow. Its work
// is counted in units: a few for its queries and results and one for every block of
// 128 keys that its last token sees (one where it sees none), or one more: whole
// tiles are counted together, so that the units before any of them need no sum
// over them. Tiles are numbered request by request, in a request KV head by KV
// head, in a head by their tokens. A part is a contiguous range of units.
#pragma once

#include <stdint.h>

namespace a8w8 {
namespace chunk {

constexpr int kKeys = 128;        // keys of a block
constexpr int kTileRows = 256;    // (token, head) rows of a tile at most

// Units of a tile beside its blocks, wide and narrow. A fit over the CTAs of several
// batches, BF16 cache, in clocks: a wide tile 7000 to 11000 and 2900 to 3300 a block,
// a narrow one 2400 to 3800 and 2200 to 2800.
constexpr int kWideCost = 3, kNarrowCost = 1;
constexpr int kMinUnits = 3;      // of a part
constexpr int kWideSlack = 3, kNarrowSlack = 2;    // the costs at least, see Shares

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

// Units of a head's tiles before tile i, all of them whole: with c the cost and b0 the
// first token's position, tile k sees b0 + (k + 1) tpt keys, and the sum of those over
// k < i in whole blocks and i (c + 1) are i c, the tiles' blocks and at most one more for
// each. (Where the first tokens see nothing, b0 counts as 0: see Shares.)
__host__ __device__ inline long units_before(const Req& r, int tpt, int i) {
    const long b0 = r.ctx > r.n ? r.ctx - r.n : 0;
    return (long)i * (kWideCost + 1) + (i * b0 + (long)tpt * i * (i + 1) / 2) / kKeys;
}
// Units of a tile, and of one KV head of a request.
__host__ __device__ inline long tile_units(const Req& r, int tpt, int i) {
    const int tokens = r.n - i * tpt;
    if (tokens > tpt) return units_before(r, tpt, i + 1) - units_before(r, tpt, i);
    return cost_of(is_narrow(tokens, tpt)) + blocks_of(keys_of(r, tpt, i));
}
__host__ __device__ inline long head_units(const Req& r, int tpt) {
    if (r.n <= 0) return 0;
    const int last = tiles_of(r, tpt) - 1;
    return units_before(r, tpt, last) + tile_units(r, tpt, last);
}

__host__ __device__ inline long div_long(long a, long b) {
    return (a | b) >> 32 ? a / b : (long)((unsigned)a / (unsigned)b);
}

// Whether a tile of contexts of up to nb blocks may be divided: it has more units
// than both of its ends keep.
__host__ __device__ inline bool may_divide(int nb) {
    return kWideCost + nb + 1 > 2 * kWideSlack || kNarrowCost + nb > 2 * kNarrowSlack;
}

// How W units are shared by at most P parts: part c begins at W c / parts, moved
// to the nearer end of the tile where that is at most `slack` units away, as a tile
// that two parts hold costs both of them; and so that no part begins before a tile's
// second block. (With an eighth of a part, 64 requests of 4 drafts, 4-bit: 154 us
// instead of 143; 512 tokens at 16384: 154 instead of 150.) Tiles of requests whose first tokens see nothing, where units are not
// blocks, are not divided.
struct Shares {
    long W, whole;
    int parts, rest;
    __host__ __device__ Shares(long units, int P) {
        W = units;
        parts = (int)(units < (long)P * kMinUnits ? (units + kMinUnits - 1) / kMinUnits : P);
        whole = parts > 0 ? div_long(W, parts) : 0;
        rest = (int)(W - whole * parts);
    }
    __host__ __device__ long raw(int c) const { return whole * c + rest * c / (parts > 0 ? parts : 1); }
    __host__ __device__ long slack(const Req& r, int tpt, int i) const {
        if (r.ctx < r.n) return W;
        return is_narrow(tokens_in(r, tpt, i), tpt) ? kNarrowSlack : kWideSlack;
    }
    __host__ __device__ static long snap(long u, long tile, long tile_end, long slack) {
        if (u - tile <= slack && u - tile <= tile_end - u) return tile;
        return tile_end - u <= slack ? tile_end : u;
    }
    // The parts kf .. kl that begin inside a tile (more than `slack` units from
    // both ends, as snap has it), given that part c does.
    __host__ __device__ void inside(long tile, long tile_end, long slack, int c, int& kf, int& kl) const {
        kf = kl = c;
        while (kf > 1 && raw(kf - 1) > tile + slack) --kf;
        while (kl + 1 < parts && raw(kl + 1) < tile_end - slack) ++kl;
    }
};

}  // namespace chunk
}  // namespace a8w8
