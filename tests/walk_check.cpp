// Runs the split of chunk attention over CTAs (csrc/mk_walk.cuh) on the CPU and
// compares it with counting by hand.  The lanes of a warp are coroutines that
// meet at each exchange, as the hardware's do.  Prints "ok" and what it ran.
#include <ucontext.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <tuple>
#include <vector>

static struct {
    int x;
} threadIdx;
static ucontext_t scheduler, lanes[32];
static long long slots[2][32];
static int turn[32], done[32];
static std::vector<std::vector<char>> stacks(32, std::vector<char>(64 << 10));

#define CHECK(c, ...)                                                            \
    do {                                                                         \
        if (!(c)) {                                                              \
            printf("line %d: %s ", __LINE__, #c);                                \
            printf(__VA_ARGS__);                                                 \
            printf("\n");                                                        \
            exit(1);                                                             \
        }                                                                        \
    } while (0)

// what every lane brings; slots alternate, so that a lane that runs ahead to the
// next exchange does not overwrite what the others still read
static const long long *meet(long long v) {
    const int l = threadIdx.x, t = turn[l] ^= 1;
    slots[t][l] = v;
    swapcontext(&lanes[l], &scheduler);
    return slots[t];
}
template <class T>
static T __shfl_sync(unsigned, T v, int from) { return (T)meet(v)[from & 31]; }
template <class T>
static T __shfl_up_sync(unsigned, T v, int by) {
    const int l = threadIdx.x;
    const long long *s = meet(v);
    return (T)s[l >= by ? l - by : l];
}
template <class T>
static T __shfl_xor_sync(unsigned, T v, int by) {
    const int l = threadIdx.x;
    return (T)meet(v)[l ^ by];
}
static unsigned __ballot_sync(unsigned, bool v) {
    const long long *s = meet(v);
    unsigned r = 0;
    for (int i = 0; i < 32; ++i) r |= (unsigned)(s[i] != 0) << i;
    return r;
}
static int __all_sync(unsigned m, bool v) { return __ballot_sync(m, v) == 0xffffffffu; }
static int __ffs(unsigned v) { return __builtin_ffs((int)v); }
static int __clz(unsigned v) { return v ? __builtin_clz(v) : 32; }
static int __ldg(const int *p) { return *p; }
using std::max;
using std::min;

#include "mk_walk.cuh"

using namespace mkc;

template <int BN, int OV>
struct Run {
    typedef Walk<BN, OV> W;
    struct Call {
        const ChunkP *c;
        int tpu, hkv, grid, cta, least;
        W w[32];
        bool good[32];
    };
    static Call *call;
    static void lane() {
        const int l = threadIdx.x;
        call->good[l] = call->w[l].plan(call->c, call->tpu, call->hkv, call->grid, call->cta, call->least);
        done[l] = 1;
    }
    static void plan(Call &k) {
        call = &k;
        for (int l = 0; l < 32; ++l) {
            turn[l] = done[l] = 0;
            getcontext(&lanes[l]);
            lanes[l].uc_stack.ss_sp = stacks[l].data();
            lanes[l].uc_stack.ss_size = stacks[l].size();
            lanes[l].uc_link = &scheduler;
            makecontext(&lanes[l], lane, 0);
        }
        for (int running = 32; running;) {
            running = 0;
            for (int l = 0; l < 32; ++l) {
                if (done[l]) continue;
                threadIdx.x = l;
                swapcontext(&scheduler, &lanes[l]);
                running += !done[l];
            }
        }
    }

    // the chunk's cover by `grid` CTAs, or its refusal
    static void check(const std::vector<int> &lens, const std::vector<int> &ctxs, int tpu, int hkv, int grid, int least,
                      int max_pages, bool valid = true, const std::vector<int> *offsets = nullptr) {
        const int S = (int)lens.size();
        std::vector<int> off(S + 1, 0);
        for (int i = 0; i < S; ++i) off[i + 1] = off[i] + lens[i];
        if (offsets) off = *offsets;
        ChunkP c;
        c.off = off.data();
        c.ctx = ctxs.data();
        c.S = S;
        c.n_rows = offsets ? *std::max_element(off.begin(), off.end()) : off[S];
        c.max_pages = max_pages;
        c.max_pos = 64ll * max_pages;
        typedef std::tuple<int, int, int> Unit;              // stream, kv head, unit
        std::map<Unit, std::vector<int>> cover;              // CTA of each iteration
        std::map<Unit, std::pair<int, int>> cut;             // first CTA, followers
        long long its = 0;
        for (int i = 0; i < S; ++i)
            for (int u = 0; valid && u * tpu < lens[i]; ++u) {
                const int n = (ctxs[i] + min((u + 1) * tpu, lens[i]) + BN - 1) / BN;
                for (int h = 0; h < hkv; ++h) cover[Unit(i, h, u)].assign(n, -1);
                its += (long long)n * hkv;
            }
        Call k{&c, tpu, hkv, grid, 0, least, {}, {}};
        for (k.cta = 0; k.cta < grid; ++k.cta) {
            plan(k);
            for (int l = 0; l < 32; ++l) CHECK(k.good[l] == valid, "cta %d lane %d", k.cta, l);
            if (!valid) continue;
            int begun = 0, continued = 0;
            Seg g, o;
            for (bool more = true; more;) {
                more = k.w[0].next(g);
                if (k.cta % 16 == 0)                         // every lane walks the same way
                    for (int l = 1; l < 32; ++l) {
                        CHECK(k.w[l].next(o) == more, "lane %d", l);
                        CHECK(!more || (o.stream == g.stream && o.head == g.head && o.tok0 == g.tok0 && o.j0 == g.j0 && o.j1 == g.j1), "lane %d", l);
                    }
                if (!more) break;
                CHECK(g.stream >= 0 && g.stream < S && g.head >= 0 && g.head < hkv && g.tok0 % tpu == 0, "cta %d", k.cta);
                const Unit u(g.stream, g.head, g.tok0 / tpu);
                CHECK(cover.count(u), "stream %d unit %d", g.stream, g.tok0 / tpu);
                std::vector<int> &v = cover[u];
                CHECK(g.ntok == min(tpu, lens[g.stream] - g.tok0) && g.row0 == off[g.stream] + g.tok0, "stream %d", g.stream);
                CHECK(g.ctx == ctxs[g.stream] && g.kvlen == g.ctx + lens[g.stream] && g.nit == (int)v.size(), "stream %d", g.stream);
                CHECK(0 <= g.j0 && g.j0 < g.j1 && g.j1 <= g.nit, "%d %d of %d", g.j0, g.j1, g.nit);
                for (int j = g.j0; j < g.j1; ++j) {
                    CHECK(v[j] < 0, "iteration %d twice", j);
                    v[j] = k.cta;
                }
                // slots of a CTA: one unit that it continues, one that it leaves unfinished
                if (g.j0 > 0) CHECK(++continued == 1, "cta %d", k.cta);
                if (g.j0 == 0 && g.j1 < g.nit) {
                    CHECK(++begun == 1, "cta %d", k.cta);
                    cut[u] = std::make_pair(k.cta, g.followers);
                } else {
                    CHECK(g.followers == 0, "%d", g.followers);
                }
            }
        }
        for (auto &e : cover) {
            const std::vector<int> &v = e.second;
            for (size_t j = 0; j < v.size(); ++j) CHECK(v[j] >= 0 && (j == 0 || v[j] == v[j - 1] || v[j] == v[j - 1] + 1), "iteration %zu", j);
            const int more = v.back() - v.front();
            CHECK(more ? cut.count(e.first) && cut[e.first] == std::make_pair(v.front(), more) : !cut.count(e.first), "%d CTAs", more + 1);
        }
        ++calls;
        iterations += its;
    }
    static long long calls, iterations;
};
template <int BN, int OV> typename Run<BN, OV>::Call *Run<BN, OV>::call;
template <int BN, int OV> long long Run<BN, OV>::calls;
template <int BN, int OV> long long Run<BN, OV>::iterations;

template <int M>
static void sums(std::mt19937 &rng) {
    for (uint32_t a = 0; a <= 3 * M; a += 1 + a / 70)
        for (uint32_t b = 0; b <= 4 * M; b += 1 + b / 50) {
            long long want = 0;
            for (uint32_t n = 0; n < 70; ++n) {
                CHECK(floor_sum<M>(n, a, b) == want, "n %u a %u b %u", n, a, b);
                want += (a * n + b) / M;
            }
        }
    for (int k = 0; k < 300; ++k) {                          // up to the 32 bits that a n + b may have
        const uint32_t a = 1 + rng() % 256, n = rng() % 20000, b = rng() % (0xffffffffu - a * n);
        long long want = 0;
        for (uint32_t i = 0; i < n; ++i) want += ((uint64_t)a * i + b) / M;
        CHECK(floor_sum<M>(n, a, b) == want, "n %u a %u b %u", n, a, b);
    }
}

// all chunks of up to two streams over small lengths and contexts, and random ones
template <int BN, int OV>
static void walks(std::mt19937 &rng, int least, int rounds) {
    typedef Run<BN, OV> R;
    auto pick = [&](std::initializer_list<int> v) { return *(v.begin() + rng() % v.size()); };
    for (int l0 : {0, 1, 2, 3, 5})
        for (int l1 : {0, 1, 4})
            for (int c0 : {0, 1, BN - 1, BN, 3 * BN + 7})
                for (int grid : {1, 2, 3, 8}) R::check({l0, l1}, {c0, BN - 2}, 2, 2, grid, least, 64);
    for (int k = 0; k < rounds; ++k) {
        const int S = k % 4 == 3 ? pick({31, 32, 33, 64, 65, 97}) : 1 + rng() % 6;
        std::vector<int> lens(S), ctxs(S);
        for (int i = 0; i < S; ++i) {
            lens[i] = rng() % 4 == 0 ? rng() % 2 : rng() % (S > 6 ? 20 : 300);
            ctxs[i] = rng() % 3 == 0 ? 0 : rng() % (S > 6 ? 300 : 3000);
        }
        R::check(lens, ctxs, pick({1, 2, 3, 4, 5, 8, 10, 12, 16, 21, 32, 42, 64, 85, 128, 256}), pick({1, 2, 4, 8}),
                 pick({1, 2, 7, 152, 304}), least, 64);
    }
    R::check({0, 0, 0}, {5, 0, 9}, 16, 2, 8, least, 64);     // nothing to do
    R::check({3}, {1 << 18}, 16, 1, 304, least, 5000);       // one long axis
    R::check(std::vector<int>(700, 1), std::vector<int>(700, 70), 16, 4, 152, least, 2);
    // descriptions that no CTA may follow
    const std::vector<int> three = {0, 0, 0};
    const std::vector<std::pair<std::vector<int>, std::vector<int>>> bad = {
        {{0, 5, 3, 8}, {0, 0, 0}}, {{1, 5, 6, 8}, {0, 0, 0}}, {{0, -1, 6, 8}, {0, 0, 0}}, {{0, 8, 8, 7}, {0, 0, 0}},
        {{0, 5, 5, 8}, {0, -1, 0}}, {{0, 5, 5, 8}, {0, 129, 0}}, {{0, 5, 6, 8}, {124, 0, 0}}};
    for (auto &e : bad) R::check(three, e.second, 16, 2, 3, least, 2, false, &e.first);
    for (int S : {33, 64, 200})
        for (int at : {0, 31, 32, S - 2}) {
            std::vector<int> off(S + 1), ctx(S, 3);
            for (int i = 0; i <= S; ++i) off[i] = 2 * i;
            std::vector<int> fall = off;
            fall[at + 1] = off[at + 1] + (at + 2 <= S ? 3 : -3);
            R::check(std::vector<int>(S, 0), ctx, 16, 1, 3, least, 2, false, &fall);
            ctx[at] = -1;
            R::check(std::vector<int>(S, 0), ctx, 16, 1, 3, least, 2, false, &off);
        }
    printf("%d keys, start %d, least %d: %lld chunks, %lld iterations\n", BN, OV, least, R::calls, R::iterations);
}

int main() {
    std::mt19937 rng(1);
    sums<64>(rng);
    sums<128>(rng);
    walks<64, 1>(rng, 1, 120);     // float32
    walks<128, 3>(rng, 3, 120);    // bf16 pages
    walks<128, 5>(rng, 5, 120);    // FP8 pages
    printf("ok\n");
}
