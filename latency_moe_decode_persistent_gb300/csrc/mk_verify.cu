// Verification of drafted tokens by speculative sampling.
//
// Row t of a stream has p_t = softmax(logits_t / temperature).  Draft d_i is
// accepted while u_{i-1} q_{i-1}(d_i) < p_{i-1}(d_i); the emitted token is the
// first index whose cumulative weight passes u_{T-1} times the total, with
// weights max(p_n - q_n, 0) after a rejection at row n and p_{T-1} otherwise.
//
// Where a cumulative sum over 10^5 entries crosses a random number is decided
// by its last digits: with weights good to 2^-23, one draw in some tens falls
// on the wrong side of a border.  So a weight is an integer multiple of 2^-44
// of the power of two above the row's largest, good to 2^-36 + 2^-46 |logit /
// temperature| of itself (below), and all sums are integers: exact, so
// independent of how a row is cut and of the other streams.  With
//   y = logit * (log2 e / temperature) = (k + f) / 32 + yl,  k an integer,
//   |f| <= 1/2 (a two-float product), 2^y = 2^(k div 32) T[k mod 32] e^z
// T comes from 32 entries that a warp's lanes hold (a shuffle instead of
// shared-memory reads that collide) and e^z - 1 from its Taylor terms to z^5
// (|z| < 2^-6.5, remainder 2^-48).  All in FP32 pairs (f32x2): FP64 would do
// with fewer instructions, but this GPU's FP64 rate is 1/60 of its FP32 rate,
// and conversions run at an eighth of it, so floats become integers by adding
// 3 * 2^k and taking the bits.
// Error: e^z - 1 = zh + w, w below 2^-14, is rounded to half a step of w and its
// product with T to three half steps of 2^-13 at most, together below 2^-36 of
// the weight (2^-36.3 over 400,000 neighbouring logits in an exact emulation); yl,
// within 1.5 steps of y, has 24 bits, which |y| 2^-46.4 covers.
//
// Such a weight costs some 50 instructions, so only the row that the token is
// drawn from has them.  The other rows are needed for the tests' normalisers
// alone: float32 sums (one exponential per logit, HBM-bound), good to 2^-18;
// a test that comes within 2^-16 of its border is decided by exact weights too.
//
// Two launches: float32 sums of (row, slice) over the whole GPU, then one
// cluster per stream that joins them, tests the drafts and draws the token.
//
// Measured (vocab 129280, one GB300): 1 stream of 6 rows in 14 to 17 us, of which
// the sums take 4 and the rest is a chain of meetings of the cluster; 16 streams
// of 8 rows in 39 to 46 us, sums 16 us (4.1 TB/s) and 19 us of weights per wave of
// clusters, of which a device runs 15 or 16 side by side.
#include <cooperative_groups.h>

#include "mk_chunk.cuh"

namespace {
using namespace mkc;
namespace cg = cooperative_groups;

constexpr int NT = 256, PER = 16, SLICE = NT * PER;  // phase 1: at most SLICE entries of a row per block
constexpr int CT = 1024, CW = CT / 32;               // phase 2: threads, warps per CTA
constexpr float YMAX = 131000.f;                     // |logit / temperature * log2 e| that k holds

struct Scale {
    float hi, lo;  // log2(e) / temperature
};
// in two floats: the rounded quotient, and what is left of log2(e) = 1.44269502 + 1.9259630e-8
__device__ __forceinline__ Scale scale_of(float t) {
    Scale s;
    s.hi = __fdiv_rn(1.44269502162933349609375f, t);
    s.lo = __fdiv_rn(fmaf(-s.hi, t, 1.44269502162933349609375f) + 1.925963033500975e-8f, t);
    return s;
}
// An integer above the unrounded exponent of a logit, and of any below it, from the
// rounded product y: both roundings, of the product and of hi, leave at most half
// a step and one of y, and 2^-22 |y| is two at least.  (The integer at or above y
// itself will not do: a product that is rounded down to it would weigh more than 1.)
__device__ __forceinline__ float above(float y) { return floorf(fmaf(fabsf(y), 0x1p-22f, y)) + 1.f; }
__device__ __forceinline__ bool good_t(float t) { return t >= 1e-3f && t <= 1e3f; }

using f2 = unsigned long long;  // two floats side by side
__device__ __forceinline__ f2 pk(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f2 pk(float a) { return pk(a, a); }
__device__ __forceinline__ void up(f2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 sub2(f2 a, f2 b) { return fma2(b, pk(-1.f), a); }

constexpr uint32_t C1 = 0x40400000u, C2 = 0x35400000u;  // bits of 3 and of 3 * 2^-22

// 2^(y - yref) of two logits, yref an integer above either (`above`), as (h + l) * p2,
// p2 a power of two; y below yref - range counts as yref - range (range < 126).
// All 32 lanes call; T: this lane's table entry (2^(lane/32) as two floats).
struct Pow2 {
    f2 h, l, p2;
};
__device__ __forceinline__ Pow2 powers(float l0, float l1, Scale c, int yref, float range, float2 T) {
    const f2 l = pk(l0, l1), hi = pk(c.hi), one = pk(-1.f);
    const f2 ny = mul2(l, pk(-c.hi));                       // -y, rounded
    f2 yl = fma2(l, pk(c.lo), fma2(l, hi, ny));
    float y0, y1, e0, e1;
    up(ny, y0, y1);
    up(yl, e0, e1);
    const float low = (float)yref - range;
    const bool in0 = -y0 > low, in1 = -y1 > low;            // false for -inf
    const f2 y = pk(fmaxf(-y0, low), fmaxf(-y1, low));
    yl = pk(in0 ? e0 : 0.f, in1 ? e1 : 0.f);
    const f2 tn = fma2(y, pk(32.f), pk(12582912.f));        // k + 1.5 * 2^23
    f2 f = fma2(add2(tn, pk(-12582912.f)), pk(-0.03125f), y);  // exact; 0 or at least 2 |yl|
    {
        const f2 g = add2(f, yl);                           // f + yl as (sum, rest)
        yl = fma2(sub2(g, f), one, yl);
        f = g;
    }
    const float L = 0.693147182464599609375f, Ll = -1.904654323148236e-9f;  // ln 2 as two floats
    const f2 zh = mul2(f, pk(L)), nz = mul2(f, pk(-L));
    const f2 zl = fma2(yl, pk(L), fma2(f, pk(Ll), fma2(f, pk(L), nz)));
    const f2 zz = mul2(zh, zh), ez = fma2(zh, zh, mul2(zh, nz));
    const f2 q = fma2(zh, fma2(zh, pk(0.00833333377f), pk(0.0416666679f)), pk(0.166666672f));
    f2 w = fma2(zz, mul2(zh, q), zl);                       // z^3/6 + ... and the low parts
    w = fma2(zl, zh, fma2(ez, pk(0.5f), w));
    w = fma2(zz, pk(0.5f), w);                              // e^z - 1 = zh + w
    float k0, k1;
    up(tn, k0, k1);
    const int a0 = __float_as_int(k0) - 0x4b400000 - yref * 32, a1 = __float_as_int(k1) - 0x4b400000 - yref * 32;  // <= 0
    const f2 Th = pk(__shfl_sync(0xffffffffu, T.x, a0 & 31), __shfl_sync(0xffffffffu, T.x, a1 & 31));
    const f2 Tl = pk(__shfl_sync(0xffffffffu, T.y, a0 & 31), __shfl_sync(0xffffffffu, T.y, a1 & 31));
    const f2 a = mul2(Th, zh);                              // T e^z = Th + a + b
    f2 b = fma2(Th, zh, mul2(Th, nz));
    b = add2(fma2(Tl, zh, fma2(Th, w, b)), Tl);
    const f2 g = add2(a, b);
    Pow2 r;
    r.h = add2(Th, g);
    r.l = add2(sub2(g, sub2(r.h, Th)), sub2(b, sub2(g, a)));
    r.p2 = pk(__int_as_float(((a0 & ~31) << 18) + 0x3f800000), __int_as_float(((a1 & ~31) << 18) + 0x3f800000));
    return r;
}
// Two numbers as w = (hi - C1) * 2^22 + (lo - C2) in units of 2^-44 (int32 differences)
struct W2 {
    uint32_t hi[2], lo[2];
};
// x + l * s, 0 <= x <= 1, |l * s| < 2^-23: 3 + x has steps of 2^-22, what that leaves
// (a half step and l * s) on top of 3 * 2^-22 steps of 2^-44
__device__ __forceinline__ W2 multiples(f2 x, f2 l, f2 s) {
    const f2 t1 = add2(x, pk(3.f));
    const f2 t2 = add2(fma2(l, s, sub2(x, add2(t1, pk(-3.f)))), pk(7.152557373046875e-7f));
    float u0, u1;
    W2 r;
    up(t1, u0, u1);
    r.hi[0] = __float_as_uint(u0);
    r.hi[1] = __float_as_uint(u1);
    up(t2, u0, u1);
    r.lo[0] = __float_as_uint(u0);
    r.lo[1] = __float_as_uint(u1);
    return r;
}
// weights; 0 below 2^-60
__device__ __forceinline__ W2 weights(float l0, float l1, Scale c, int yref, float2 T) {
    const Pow2 e = powers(l0, l1, c, yref, 60.f, T);
    const f2 x = mul2(e.h, e.p2);
    return multiples(x, e.l, e.p2);
}
__device__ __forceinline__ long long whole(uint32_t hi, uint32_t lo) { return ((long long)(int)hi << 22) + (int)lo; }

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__global__ void __launch_bounds__(NT) verify_sums_kernel(VerifyP p) {
    __shared__ float redm[NT / 32];
    __shared__ float reds[NT / 32];
    cudaTriggerProgrammaticLaunchCompletion();
    const int tid = threadIdx.x, lane = tid % 32, wid = tid / 32;
    const int sl = blockIdx.x, row = blockIdx.y;           // row = stream * T + t
    const int b = sl * p.slice, n = min(p.slice, p.V - b);
    const float *src = p.logits + (long long)row * p.V + b;
    float x[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = i * NT + tid < n ? __ldg(src + i * NT + tid) : -CUDART_INF_F;
    const float t = __ldg(p.temps + row / p.T);
    // an earlier call's error; what this call raises, in the draws of this launch and
    // the ones before, keeps no other stream from its answer
    const bool gone = p.first ? aborted(p.ctrl) : *(volatile const int *)p.gone != 0;
    if (p.first && sl == 0 && row == 0 && tid == 0) *p.gone = gone;
    if (__syncthreads_or(gone)) return;
    float m = -CUDART_INF_F;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        m = fmaxf(m, x[i]);
        nan |= x[i] != x[i];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) redm[wid] = m;
    nan = __syncthreads_or(nan);
    for (int i = 0; i < NT / 32; ++i) m = fmaxf(m, redm[i]);
    VerifyPart out{0.f, -CUDART_INF_F};
    const Scale c = scale_of(t);
    const float y = m * c.hi;
    // +inf or NaN in the row, or a range that k does not hold; a slice far below
    // that range (masked by the lowest float32) has no weight in any row that
    // join_row lets pass
    const bool bad = nan || !good_t(t) || !(y < YMAX);
    if (!bad && y > -YMAX - 64.f) {
        out.yref = above(y);
        // logits far below (masked ones, the padding) as one that weighs 2^-110: finite,
        // so that the product's rest stays a number
        const float far = (out.yref - 110.f) / c.hi;
        f2 acc = 0;
#pragma unroll
        for (int i = 0; i < PER; i += 2) {
            // y - yref with one rounding: the product's rest comes last
            const f2 l = pk(fmaxf(x[i], far), fmaxf(x[i + 1], far));
            const f2 ny = mul2(l, pk(-c.hi)), yl = fma2(l, pk(c.lo), fma2(l, pk(c.hi), ny));
            const f2 z = add2(fma2(ny, pk(-1.f), pk(-out.yref)), yl);
            float z0, z1;
            up(z, z0, z1);
            acc = add2(acc, pk(ex2(z0), ex2(z1)));
        }
        float s, s1;
        up(acc, s, s1);
        s = warp_sum(s + s1);
        if (lane == 0) reds[wid] = s;
        __syncthreads();
        s = 0.f;
        for (int i = 0; i < NT / 32; ++i) s += reds[i];
        out.sum = s;
    }
    if (bad) out.yref = CUDART_NAN_F;
    if (tid == 0) p.part[(long long)row * p.nsl + sl] = out;
}

struct Row {
    float sum, yref;   // sum of 2^(y - yref)
    bool bad;
};
// slices of a row joined by a warp; references are integers
__device__ Row join_row(const VerifyP &p, int row, int lane) {
    static_assert(MK_VERIFY_MAXV <= 64 * SLICE, "two slices per lane");
    VerifyPart q[2];
    float yr = -CUDART_INF_F;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k = lane + 32 * i;
        q[i] = k < p.nsl ? p.part[(long long)row * p.nsl + k] : VerifyPart{0.f, -CUDART_INF_F};
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        bad |= q[i].yref != q[i].yref;
        yr = fmaxf(yr, q[i].yref);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) yr = fmaxf(yr, __shfl_xor_sync(0xffffffffu, yr, o));
    bad = __any_sync(0xffffffffu, bad) || !(yr > -YMAX);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (!bad && q[i].sum > 0.f) s += q[i].sum * ex2(q[i].yref - yr);
    return Row{warp_sum(s), yr, bad};
}

// floor(u * r) for u in [0, 1), r >= 0
__device__ __forceinline__ long long scaled(float u, long long r) {
    if (!(u > 0.f)) return 0;
    const int e = ilogbf(u);                                  // u = m 2^(e-23), 2^23 <= m < 2^24
    const unsigned long long m = (unsigned long long)scalbnf(u, 23 - e);
    const int sh = 23 - e;                                    // >= 24
    const unsigned long long hi = __umul64hi(m, (unsigned long long)r), lo = m * (unsigned long long)r;
    if (sh < 64) return (long long)((hi << (64 - sh)) | (lo >> sh));
    return sh < 128 ? (long long)(hi >> (sh - 64)) : 0;
}

// u q S < e by two-float products: 1 and 0 where the difference passes `guard`
// times the larger side, else -1.  sh + sl: S.
__device__ __forceinline__ int test(float u, float q, float sh, float sl, float eh, float el, float guard) {
    const float uq = u * q, uql = fmaf(u, q, -uq);
    const float a = uq * sh, al = fmaf(uq, sh, -a) + (uq * sl + uql * sh);
    const float d = (a - eh) + (al - el);
    if (!(uq > 0.f)) return eh > 0.f;
    if (fabsf(d) <= guard * fmaxf(a, eh)) return -1;
    return d < 0.f;
}

// q S of two draft probabilities, S = sh + sl; beyond 1, which no weight passes, as 1
__device__ __forceinline__ W2 parts_of(float q0, float q1, f2 sh, f2 nsh, f2 sl) {
    const f2 q = pk(q0, q1), nx = mul2(q, nsh), l = fma2(q, sl, fma2(q, sh, nx));
    float x0, x1, l0, l1;
    up(nx, x0, x1);
    up(l, l0, l1);
    return multiples(pk(fminf(-x0, 1.f), fminf(-x1, 1.f)), pk(x0 >= -1.f ? l0 : 0.f, x1 >= -1.f ? l1 : 0.f), pk(1.f));
}

// Weights, below 2^45, in shared memory: 6 bytes each
struct Cache {
    uint32_t *lo;
    uint16_t *hi;
    __device__ __forceinline__ long long get(int i) const { return (long long)hi[i] << 32 | lo[i]; }
    __device__ __forceinline__ void put(int i, long long v) const {
        lo[i] = (uint32_t)v;
        hi[i] = (uint16_t)(v >> 32);
    }
};

// The row in CL * CW consecutive ranges, one per warp; a range's weights stay in
// shared memory from the first sum to the draw.
template <int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(CT) verify_draw_kernel(VerifyP p) {
    __shared__ Row rows[MK_MAXT];
    __shared__ float dh[MK_MAXT], dl[MK_MAXT];    // 2^(y - yref) of the drafts, two floats
    __shared__ float du[MK_MAXT], dq[MK_MAXT];
    __shared__ int verdict[MK_MAXT], token[MK_MAXT];
    __shared__ int wrong, odd;                    // 1: bad values, 2: bad input; a bad draft probability
    __shared__ long long warps[CW];
    __shared__ long long slots[2][CL][2];         // from every CTA, in turns: its sum of weights; what went wrong
    extern __shared__ uint32_t cache[];           // [CW][len] low halves, then high ones
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid % 32, wid = tid / 32;
    const int s = blockIdx.x / CL, rank = blockIdx.x % CL;
    const int T = p.T, V = p.V, len = p.len;
    // the drafts' own powers, each against a reference of its own, before the wait for the sums
    const float2 tab = __ldg(p.tab + lane);
    const float t = __ldg(p.temps + s);
    const float *lg = p.logits + (long long)s * T * V;
    const float *pq = p.probs ? p.probs + (long long)s * (T - 1) * V : nullptr;
    const Scale c = scale_of(t);
    float u = 0.f, ld = 0.f, qd = 1.f, ey = 0.f, eh = 0.f, el = 0.f;
    int d = 0;
    if (wid == 0) {
        if (lane < T) u = __ldg(p.uniforms + s * T + lane);
        if (lane < T - 1) {
            d = __ldg(p.tokens + s * T + lane + 1);
            if (d >= 0 && d < V) {
                ld = __ldg(lg + (long long)lane * V + d);
                if (pq) qd = __ldg(pq + (long long)lane * V + d);
            }
        }
        const bool fin = good_t(t) && fabsf(ld * c.hi) < YMAX;
        const float l = fin ? ld : 0.f;
        ey = above(l * c.hi);
        const Pow2 e = powers(l, l, c, (int)ey, 120.f, tab);
        float p2, x;
        up(e.h, eh, x);
        up(e.l, el, x);
        up(e.p2, p2, x);
        eh = fin ? eh * p2 : 0.f;
        el = fin ? el * p2 : 0.f;
    }
    if (tid == 0) odd = 0;
    cl.sync();                                    // every CTA is there to be written to
    cudaGridDependencySynchronize();
    if (wid < T) {
        const Row r = join_row(p, s * T + wid, lane);
        if (lane == 0) rows[wid] = r;
    }
    const bool gone = __syncthreads_or(tid == CT - 1 && *(volatile const int *)p.gone);
    if (wid == 0) {
        // lane i tests draft i+1
        const Row tr = rows[lane < T ? lane : 0];
        const bool in = lane < T - 1;
        const bool badin = lane < T && (!(u >= 0.f && u < 1.f) || !good_t(t) || (in && (d < 0 || d >= V)));
        const bool bad = lane < T && (tr.bad || !(qd >= 0.f && qd < CUDART_INF_F));
        // 2^(ey - yref): a token below 2^-120 of the row's largest has no probability to speak of
        const float dy = ey - tr.yref, p2 = in && dy > -120.f && dy <= 0.f ? __int_as_float(((int)dy + 127) << 23) : 0.f;
        eh *= p2;
        el *= p2;
        if (lane < T) {
            dh[lane] = eh;
            dl[lane] = el;
            du[lane] = u;
            dq[lane] = qd;
            token[lane] = in ? d : -1;
            verdict[lane] = in ? test(u, qd, tr.sum, 0.f, eh, el, 0x1p-16f) : 0;
        }
        if (in && !bad && !badin && p.accept_prob && rank == 0)
            p.accept_prob[s * (T - 1) + lane] = eh < qd * tr.sum ? __fdividef(eh, qd * tr.sum) : 1.f;
        const unsigned anybad = __ballot_sync(0xffffffffu, bad), anyin = __ballot_sync(0xffffffffu, badin);
        if (lane == 0) wrong = anyin ? 2 : anybad ? 1 : 0;
    }
    __syncthreads();
    const bool dead = gone || wrong;              // (the same in all CTAs of the cluster)
    const int b = min(V, (rank * CW + wid) * len), e = min(V, b + len);
    const Cache w{cache + wid * len, reinterpret_cast<uint16_t *>(cache + CW * len) + wid * len};
    int turn = 0;
    // sums over the cluster of the warps' values: total, and what lies before this
    // CTA; nonzero where a CTA saw trouble.  Each CTA writes to all others, so that
    // after the barrier every read is local.
    auto meet = [&](long long a, long long &total, long long &before) -> int {
        a = warp_sum(a);
        if (lane == 0) warps[wid] = a;
        __syncthreads();
        if (wid == 0) {
            const long long mine = warp_sum(lane < CW ? warps[lane] : 0);
            if (lane < CL) {
                long long *o = cl.map_shared_rank(&slots[turn][rank][0], lane);
                o[0] = mine;
                o[1] = (odd ? 1 : 0) | wrong << 1 | (gone ? 8 : 0);
            }
        }
        cl.sync();
        long long flags = 0;
        total = before = 0;
#pragma unroll
        for (int k = 0; k < CL; ++k) {
            const long long v = slots[turn][k][0];
            flags |= slots[turn][k][1];
            if (k < rank) before += v;
            total += v;
        }
        turn ^= 1;                                // the next meeting's values lie elsewhere
        return (int)flags;
    };
    // exact weights of row n into the cache, and their sum
    int n = 0;
    auto weigh = [&]() -> long long {
        const float *lrow = lg + (long long)n * V + b;
        const int yref = (int)rows[n].yref;
        long long a = 0;
        // the drafter's row, which is likely to be next, comes to L2 meanwhile
        if (pq && n < T - 1)
            for (int x = 32 * lane; x < e - b; x += 1024)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(pq + (long long)n * V + b + x));
        for (int x0 = 0; x0 < e - b; x0 += 256) {  // 8 loads of a lane in flight
            float l[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int x = x0 + 32 * i + lane;
                l[i] = b + x < e ? __ldg(lrow + x) : -CUDART_INF_F;
            }
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const int x = x0 + 32 * i + lane;
                if (x0 + 32 * i >= e - b) break;  // (len is a multiple of 64)
                const W2 v = weights(l[i], l[i + 1], c, yref, tab);
                const long long w0 = whole(v.hi[0] - C1, v.lo[0] - C2), w1 = whole(v.hi[1] - C1, v.lo[1] - C2);
                w.put(x, w0);
                w.put(x + 32, w1);
                a += w0 + w1;
            }
        }
        return a;
    };
    int trouble = 0;
    long long total = 0, before = 0;
    for (;;) {
        while (n < T - 1 && verdict[n] == 1) ++n;
        trouble = meet(dead ? 0 : weigh(), total, before);
        if (trouble || n == T - 1 || verdict[n] == 0) break;
        const float sh = __ll2float_rn(total), sl = __ll2float_rn(total - (long long)sh);
        if (test(du[n], dq[n], sh * 0x1p-44f, sl * 0x1p-44f, dh[n], dl[n], 0.f) != 1) break;
        ++n;                                      // accepted after all
    }
    // after a rejection the token is drawn from max(p - q, 0)
    if (!trouble && n < T - 1) {
        const float *qrow = pq ? pq + (long long)n * V + b : nullptr;
        const int ex = token[n];
        long long a = 0, rest, rb;
        bool nonsense = false;
        const float th = __ll2float_rn(total) * 0x1p-44f, tl = __ll2float_rn(total - __float2ll_rn(th * 0x1p44f)) * 0x1p-44f;
        const f2 sh = pk(th), nsh = pk(-th), sl = pk(tl);
        for (int x0 = lane; x0 < e - b; x0 += 256) {
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = qrow && x0 + 32 * i < e - b ? __ldg(qrow + x0 + 32 * i) : 0.f;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const int x = x0 + 32 * i;
                if (x >= e - b) break;
                long long v0 = w.get(x), v1 = w.get(x + 32);  // (len is a multiple of 64; behind the range: weight 0)
                if (qrow) {
                    nonsense |= !(q[i] >= 0.f && q[i] < CUDART_INF_F) | !(q[i + 1] >= 0.f && q[i + 1] < CUDART_INF_F);
                    const W2 y = parts_of(q[i], q[i + 1], sh, nsh, sl);
                    v0 = max(v0 - whole(y.hi[0] - C1, y.lo[0] - C2), 0ll);
                    v1 = max(v1 - whole(y.hi[1] - C1, y.lo[1] - C2), 0ll);
                } else {
                    if (b + x == ex) v0 = 0;
                    if (b + x + 32 == ex) v1 = 0;
                }
                w.put(x, v0);
                w.put(x + 32, v1);
                a += v0 + v1;
            }
        }
        if (nonsense) odd = 1;
        trouble = meet(a, rest, rb);
        if (!trouble && rest == 0) {              // p <= q everywhere: from p after all
            trouble = meet(weigh(), total, before);
        } else {
            total = rest;
            before = rb;
        }
    }
    if (trouble) {
        if (rank == 0 && tid == 0 && !(trouble & 8)) {
            p.accepted[s] = 0;
            p.token[s] = -1;
            raise(p.ctrl, trouble & 4 ? MK_ERR_BAD_INPUT : MK_ERR_RANGE, 411);
        }
        return;
    }
    // the first index whose cumulative weight passes floor(u * total): it has a
    // weight, and exactly one warp's range holds it
    const long long target = scaled(__ldg(p.uniforms + s * T + T - 1), total);
    long long cum = warp_sum(lane < wid ? warps[lane] : 0) + before;
    if (cum > target || target >= cum + warps[wid]) return;
    __syncwarp();
    for (int x = 0; x < len; x += 64) {           // 64 entries: lanes take two neighbours
        const int i = x + 2 * lane;
        const long long w0 = b + i < e ? w.get(i) : 0, w1 = b + i + 1 < e ? w.get(i + 1) : 0;
        long long at = w0 + w1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += y;
        }
        const long long all = __shfl_sync(0xffffffffu, at, 31);
        if (cum + all <= target) {
            cum += all;
            continue;
        }
        const long long c1 = cum + at - w1;
        if (c1 - w0 <= target && target < c1 + w1) {
            p.token[s] = b + i + (target < c1 ? 0 : 1);
            p.accepted[s] = n;
        }
        break;
    }
}

// entries of a warp's range, and bytes of a CTA's weights
int range_len(int V, int CL) { return ((V + CL * CW - 1) / (CL * CW) + 63) / 64 * 64; }
int cache_bytes(int V, int CL) { return 6 * CW * range_len(V, CL); }

template <int CL>
cudaError_t draw(VerifyP p, int n_streams, cudaStream_t s) {
    p.len = range_len(p.V, CL);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n_streams * CL);
    cfg.blockDim = dim3(CT);
    cfg.dynamicSmemBytes = cache_bytes(p.V, CL);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_draw_kernel<CL>, p);
}
}  // namespace

int mk_verify_slices(int V) { return (V + SLICE - 1) / SLICE; }

cudaError_t mk_verify_launch(VerifyP p, int n_streams, cudaStream_t s) {
    p.nsl = mk_verify_slices(p.V);
    p.slice = (p.V + p.nsl - 1) / p.nsl;
    verify_sums_kernel<<<dim3(p.nsl, n_streams * p.T), NT, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // A CTA fills an SM, and 7 clusters of 16 or 15 of 8 run side by side (8 and 16 on
    // some devices).  T = 8, vocab 129280: 7 streams take 27 us with 16 and 31 with 8,
    // 8 streams 33 and 31, 16 streams 61 and 49.
    return n_streams > 7 ? draw<8>(p, n_streams, s) : draw<16>(p, n_streams, s);
}

// a cluster of 16, beyond the portable size, has to fit the device, and the longest
// row's weights a cluster of 8
bool mk_verify_setup() {
    const int smem = cache_bytes(MK_VERIFY_MAXV, 16), smem8 = cache_bytes(MK_VERIFY_MAXV, 8);
    if (cudaFuncSetAttribute(verify_draw_kernel<16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaFuncSetAttribute(verify_draw_kernel<16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaFuncSetAttribute(verify_draw_kernel<8>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem8) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(CT);
    cfg.dynamicSmemBytes = smem;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, verify_draw_kernel<16>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return n >= 1;
}
