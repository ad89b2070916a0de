// The plan of the chunk attention on the host: counts of units against sums over the
// tiles, and the parts walked as the kernel does, every block once and in order.
#define __host__
#define __device__
#include "../w8a8_quantized_decode_gb300/csrc/chunk_plan.cuh"

#include <stdio.h>
#include <stdlib.h>

#include <vector>

using namespace a8w8::chunk;

static int fail(const char* what, const Req& r, int tpt, int at) {
    printf("%s: n %d ctx %d tile tokens %d at %d\n", what, r.n, r.ctx, tpt, at);
    return 1;
}

static int check(const Req& r, int G, int P) {
    const int tpt = tile_tokens(G), nt = tiles_of(r, tpt);
    std::vector<long> first;
    std::vector<int> blocks, cost;
    long sum = 0;
    for (int i = 0; i < nt; ++i) {
        const int tokens = i + 1 < nt ? tpt : r.n - i * tpt;
        const long keys = (long)r.ctx - r.n + (long)i * tpt + tokens;
        const bool narrow = tokens * G <= 128;
        const int nb = keys <= 128 ? 1 : (int)((keys + 127) / 128);
        first.push_back(sum);
        blocks.push_back(nb);
        cost.push_back(narrow ? kNarrowCost : kWideCost);
        if (units_before(r, tpt, i) != sum) return fail("units before", r, tpt, i);
        if (is_narrow(tokens, tpt) != narrow || keys_of(r, tpt, i) != keys) return fail("tile", r, tpt, i);
        const long u = tile_units(r, tpt, i), least = nb + cost[i];
        if (u < least || (r.ctx >= r.n && u > least + 1)) return fail("units", r, tpt, i);
        sum += u;
    }
    if (head_units(r, tpt) != sum) return fail("head", r, tpt, 0);
    first.push_back(sum);
    auto tile_at = [&](long u) {
        int i = 0;
        while (i + 1 < nt && first[i + 1] <= u) ++i;
        return i;
    };
    const Shares sh(sum, P);
    if (sh.parts < 1 || sh.parts > P || sh.raw(sh.parts) != sum) return fail("parts", r, tpt, P);
    std::vector<long> cut;
    auto begin_of = [&](int c, int& t) {
        const long u = sh.raw(c);
        t = tile_at(u);
        return Shares::snap(u, first[t], first[t + 1], sh.slack(r, tpt, t));
    };
    for (int c = 0, t; c < sh.parts; ++c) {
        const long v = begin_of(c, t);
        cut.push_back(v);
        if (v == first[t] || v == first[t + 1]) continue;
        if (!may_divide(blocks_of(r.ctx))) return fail("divided", r, tpt, c);
        int kf, kl;
        sh.inside(first[t], first[t + 1], sh.slack(r, tpt, t), c, kf, kl);
        for (int k = 1, o; k < sh.parts; ++k) {
            const long x = begin_of(k, o);
            const bool in = o == t && x > first[t] && x < first[t + 1];
            if (in != (k >= kf && k <= kl)) return fail("inside", r, tpt, k);
        }
    }
    cut.push_back(sum);
    int t = 0, j = 0;
    for (int c = 0; c < sh.parts; ++c) {
        long u = cut[c];
        const long u1 = cut[c + 1];
        if (u > u1) return fail("order", r, tpt, c);
        while (u < u1) {
            const int k = tile_at(u);
            const long j0 = u == first[k] ? 0 : u - first[k] - cost[k];
            long j1 = u1 - first[k] - cost[k];
            if (j1 > blocks[k]) j1 = blocks[k];
            if (k != t || j0 != j || j1 <= j0) return fail("walk", r, tpt, c);
            if (j1 == blocks[k]) u = first[k + 1], ++t, j = 0;
            else u = u1, j = (int)j1;
        }
    }
    return t == nt && j == 0 ? 0 : fail("end", r, tpt, 0);
}

int main() {
    srand(1);
    for (int it = 0; it < 6000; ++it) {
        Req r;
        r.row0 = 0;
        r.n = 1 + rand() % (it % 3 == 0 ? 3000 : 300);
        r.ctx = rand() % (it % 2 ? 5000 : 400);
        const int G = 1 + rand() % 8;
        for (int P : {152, 7, 1})
            if (check(r, G, P)) return 1;
    }
    const Req longest = {0, 1 << 24, 1 << 24}, far = {0, 1, 0x7FFFFF00};
    for (int G : {1, 5, 8})
        if (head_units(longest, tile_tokens(G)) <= 0 || check(far, G, 152)) return 1;
    printf("ok\n");
    return 0;
}
