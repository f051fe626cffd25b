// The split of a chunk's attention over CTAs.  Arithmetic and warp exchanges
// only, so that a host program can run it against counting by hand
// (tests/walk_check.cpp does).
#pragma once
#include "mk_internal.h"

namespace mkc {

// Sum over i < n of floor((a*i + b) / M), M a power of two, a*n + b < 2^32
// (Euclid's reduction: the lattice points under a line, counted by swapping the
// axes; after the first step all but n is below M)
template <int M>
__device__ __forceinline__ long long floor_sum(uint32_t n, uint32_t a, uint32_t b) {
    if (n == 0) return 0;
    long long ans = (long long)n * (n - 1) / 2 * (a / M) + (long long)n * (b / M);
    a %= M;
    b %= M;
    uint32_t y = a * n + b, m = M;
    while (y >= m) {
        n = y / m;
        b = y % m;
        const uint32_t t = m;
        m = a;
        a = t;
        // sum over i < n of floor((a*i + b) / m)
        ans += (long long)n * (n - 1) / 2 * (a / m) + (long long)n * (b / m);
        a %= m;
        b %= m;
        y = a * n + b;
    }
    return ans;
}

// a / b, in 32 bits where they fit (64-bit division is a long subroutine)
__device__ __forceinline__ long long div64(long long a, long long b) {
    return (unsigned long long)(a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// Attention work is a line of cost: stream by stream, kv head by kv head, unit
// by unit (a unit is TPU consecutive tokens of a chunk with all query heads of
// the kv head); a unit costs OV (its start and end) and then one per iteration
// of BN keys that its last token sees.  CTA c takes [c*per, (c+1)*per) of the
// line: equal shares whatever the lengths, at the price of units that are cut
// at a border.  A cut unit's parts are joined from (maximum, sum, unnormalised
// output) per row.
struct Seg {
    int stream, head, tok0, ntok;  // unit: kv head, first token in the chunk, tokens
    int row0;                      // packed row of the unit's first token
    int ctx;                       // cached positions before the chunk
    int kvlen;                     // positions of the stream after the chunk
    int j0, j1, nit;               // iterations [j0, j1), at least one, of the unit's nit
    int followers;                 // CTAs that continue the unit (only where j0 == 0)
};

template <int BN, int OV>
struct Walk {
    const ChunkP *c;
    int tpu, hkv;
    long long pos, end, per;       // next place on the line, end of this CTA's range
    // cursor
    int s, h, u, nu;               // stream, kv head, unit, units of the stream
    int j;                         // next place in the unit (OV + iteration)
    int off, len, ctx;

    __device__ __forceinline__ int unit_its(int i) const {
        const int last = min((i + 1) * tpu, len);
        return (ctx + last + BN - 1) / BN;
    }
    // cost of units 0..n-1 of one kv head
    __device__ __forceinline__ long long cost_of(int n) const {
        if (n <= 0) return 0;
        const bool whole = n == nu;  // the last unit may be short
        long long r = floor_sum<BN>(whole ? n - 1 : n, tpu, (uint32_t)ctx + tpu + BN - 1);
        if (whole) r += unit_its(n - 1);
        return r + (long long)n * OV;
    }
    __device__ __forceinline__ bool load(int i) {  // stream i; false: not a valid chunk
        s = i;
        off = __ldg(c->off + i);
        const int o1 = __ldg(c->off + i + 1);
        ctx = __ldg(c->ctx + i);
        len = o1 - off;
        nu = len > 0 ? (len + tpu - 1) / tpu : 0;
        return off >= 0 && len >= 0 && o1 <= c->n_rows && ctx >= 0 && (long long)ctx + len <= c->max_pos &&
               (i > 0 || off == 0);
    }

    // Every warp plans on its own (all lanes call; no block barrier, whose waits
    // would be most of a short call's start).  False where the chunk's
    // description is bad: the same in every warp of every CTA.  A short call runs
    // this code once and cold, so it is kept short: one place each for the sums.
    __device__ bool plan(const ChunkP *cp, int tpu_, int hkv_, int grid, int cta, int min_cost) {
        c = cp;
        tpu = tpu_;
        hkv = hkv_;
        const int lane = threadIdx.x % 32;
        long long total = 0, one = 0;         // the line's length; a kv head of this lane's stream
        bool ok = true;
        // streams 32 at a time: their sum, then the one that holds pos
        long long base = 0;
        for (int b = 0, find = 0;; b += 32) {
            if (!find || c->S > 32) {
                const bool in = b + lane < c->S, good = !in || load(b + lane);
                one = in && good ? cost_of(nu) : 0;
                ok &= good;
            }
            const long long mine = one * hkv;
            if (!find) {
                total += mine;
                if (b + 32 < c->S) continue;
                if (!__all_sync(0xffffffffu, ok)) return false;
#pragma unroll
                for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
                per = div64(total + grid - 1, grid);
                if (per < min_cost) per = min_cost;
                pos = per * cta;
                end = min(total, pos + per);
                s = c->S;
                if (pos >= end) return true;
                find = 1;
                b = -32;
                if (c->S > 32) continue;
            }
            long long x = mine;                // inclusive scan
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            const unsigned past = __ballot_sync(0xffffffffu, base + x > pos);
            if (!past) {
                if (b + 32 >= c->S) return false;  // (lengths that change during the call)
                base += __shfl_sync(0xffffffffu, x, 31);
                continue;
            }
            const int k = __ffs(past) - 1;
            long long r = pos - base - __shfl_sync(0xffffffffu, x - mine, k);
            const long long ph = __shfl_sync(0xffffffffu, one, k);
            load(max(b, 0) + k);
            h = (int)div64(r, ph);
            r -= (long long)h * ph;
            // last unit that begins at r or before: lanes try 32 places at a time
            int lo = 0, hi = nu;               // begins(lo) <= r < begins(hi)
            long long at_lo = 0;
            while (hi - lo > 1) {
                const int step = (hi - lo + 31) / 32, at = lo + step * lane;
                const long long begins = cost_of(min(at, hi));
                const int i = 31 - __clz(__ballot_sync(0xffffffffu, at < hi && begins <= r));
                at_lo = __shfl_sync(0xffffffffu, begins, i);
                lo += step * i;
                hi = min(hi, lo + step);
            }
            u = lo;
            j = (int)(r - at_lo);
            return true;
        }
    }
    // next segment of this CTA (every thread of a role walks on its own)
    __device__ __forceinline__ bool next(Seg &g) {
        while (pos < end) {
            const int nit = unit_its(u);
            const int c1 = (int)min((long long)(nit + OV), j + (end - pos));
            g.stream = s;
            g.head = h;
            g.tok0 = u * tpu;
            g.ntok = min(tpu, len - g.tok0);
            g.row0 = off + g.tok0;
            g.ctx = ctx;
            g.kvlen = ctx + len;
            g.nit = nit;
            g.j0 = max(j - OV, 0);
            g.j1 = c1 - OV;
            g.followers = g.j0 == 0 && g.j1 < nit ? (int)(div64(pos - j + nit + OV - 1, per) - div64(pos, per)) : 0;
            pos += c1 - j;
            j = 0;
            if (++u == nu) {
                u = 0;
                if (++h == hkv) {
                    h = 0;
                    do {
                        if (++s >= c->S) break;
                        load(s);
                    } while (nu == 0);
                }
            }
            if (g.j1 > g.j0) return true;  // else the share ends within the unit's start: all of it is the next CTA's
        }
        return false;
    }
};

}  // namespace mkc
