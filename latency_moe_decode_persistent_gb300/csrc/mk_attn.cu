// Attention of a chunk of new tokens over the paged cache: the fp32 kernel
// (FFMA) of the all-float32 model class, the kernel that joins the parts of
// units cut over the key axis, and the choice between the classes.
//
// out[t][h] = sum_j p_j v_j / sum_j p_j,  p_j = exp((q . k_j) / sqrt(d) - m),
// j <= position of t, with the running maximum m and sum of an online softmax.
// Statistics and outputs are held in fp32.
#include "mk_chunk.cuh"

namespace {
using namespace mkc;

constexpr int BM = 64, BN = 64;  // rows (tokens x heads of a kv head) and keys of a tile; BN is one page

// 128 threads as 16 x 8: thread (ty, tx) holds the scores of rows 4ty..4ty+3 and
// keys tx, tx+8, ..., tx+56 (consecutive lanes read consecutive key rows, padded
// so that no two share a bank), and outputs of its rows' dims 4tx..4tx+3 (+32).
// The products are bound by shared-memory reads.  A 16-byte read goes by half
// warps; here each half wants 128 bytes of K or V and two rows of q or p, so that
// 12 reads of two wavefronts feed 128 FMAs.  (With 16 x 16 threads, 4 x 4 scores
// each, 8 reads of three fed 64: chunks of 128, 1, 391 and 600 tokens over up to 1391
// keys took 61.5 us, now 57.4, of which 20 are its 1.4 G FMAs.)
constexpr int NT = 128;
template <int D>
struct Smem {
    float q[BM][D + 4], p[BM][BN + 4];
    struct {
        float k[BN][D + 4], v[BN][D + 4];
    } kv[2];
};

__device__ __forceinline__ void cp16(void *dst, const void *src, bool real) {  // 16 bytes, or zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {  // two FMAs side by side
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t both(float a) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(a));
    return r;
}
__device__ __forceinline__ float2 halves(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

template <int D, class Act, class KV>
__global__ void __launch_bounds__(NT, 2) attn_simt_kernel(ChunkP c, KvP kv, AttnWs ws, Ctrl *ctrl, const Act *q, Act *out,
                                                        int hq, int hkv) {
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(raw);
    const int tid = threadIdx.x, tx = tid % 8, ty = tid / 8;
    const int G = hq / hkv;
    static_assert(D == 64, "scale");
    constexpr int ND = D / 8, NK = BN / 8;     // output dims and keys per thread
    const bool stop = tid == 0 && aborted(ctrl);  // (read while the plan is made)
    // No least share: a small call's units are cut down to single iterations (425, 9,
    // 11 and 4 tokens in 25 us, 35 with shares of 4 and more), large ones measure alike.
    Walk<BN, 1> w;
    const bool good = w.plan(&c, BM / G, hkv, gridDim.x, blockIdx.x, 1);
    if (__syncthreads_or(stop)) return;
    if (!good) {
        if (tid == 0) raise(ctrl, MK_ERR_BAD_INPUT, 402);
        return;
    }
    if (tid == 0) {
        ws.cut[blockIdx.x].followers = 0;
        ws.odd[blockIdx.x] = 0;
    }
    float chk = 0.f;                           // becomes NaN where an output is not finite
    const float scale = 0.125f * 1.4426950408889634f;  // 1 / sqrt(64), scores in the log2 domain
    Seg g;
    while (w.next(g)) {
        const int R = g.ntok * G;
        __syncthreads();
        for (int i = tid; i < BM * (D / 4); i += NT) {
            const int r = i / (D / 4), x = i % (D / 4) * 4;
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < R) {
                const Vec<Act, 4> a = *reinterpret_cast<const Vec<Act, 4> *>(
                    q + ((long long)(g.row0 + r / G) * hq + g.head * G + r % G) * D + x);
                f = make_float4(to_f(a.v[0]), to_f(a.v[1]), to_f(a.v[2]), to_f(a.v[3]));
            }
            *reinterpret_cast<float4 *>(&sm.q[r][x]) = f;
        }
        uint64_t o[4][ND / 2];                 // pairs of neighbouring dims
        float m[4], l[4];
        int lim[4];                            // last position that the row sees
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            m[a] = -CUDART_INF_F;
            l[a] = 0.f;
            lim[a] = ty * 4 + a < R ? g.ctx + g.tok0 + (ty * 4 + a) / G : -1;
#pragma unroll
            for (int b = 0; b < ND / 2; ++b) o[a][b] = 0;
        }
        // K and V of tile j on their way to buffer j & 1: float32 by copies that run
        // beside the products, bf16 through registers until `land`.  Behind the
        // stream's end, where the page holds anything, zeros.
        constexpr bool COPY = sizeof(KV) == 4;
        constexpr int PE = 16 / sizeof(KV), NP = COPY ? 1 : 2 * BN * D / (PE * NT);  // elements of a piece, pieces in registers
        uint4 raw[NP];
        auto fetch = [&](int j) {
            const int ph = __ldg(kv.table + (long long)g.stream * c.max_pages + j);
            const bool bad = ph < 0 || ph >= kv.n_pages;
            if (bad && tid == 0) raise(ctrl, MK_ERR_BAD_INPUT, 403);
            const long long base = ((long long)(bad ? 0 : ph) * hkv + g.head) * 64 * D;
            const int valid = bad ? 0 : min(64, g.kvlen - j * BN);
            auto &buf = sm.kv[j & 1];
#pragma unroll
            for (int n = 0; n < 2 * BN * D / (PE * NT); ++n) {
                const int i = n * NT + tid, r = i / (D / PE) % BN, x = i % (D / PE) * PE;
                const bool key = i < BN * (D / PE);
                const KV *src = reinterpret_cast<const KV *>(key ? kv.k : kv.v) + base + (r < valid ? r : 0) * D + x;
                if constexpr (COPY) cp16(key ? &buf.k[r][x] : &buf.v[r][x], src, r < valid);
                else raw[n] = r < valid ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0);
            }
        };
        auto land = [&](int j) {
            if constexpr (!COPY) {
                auto &buf = sm.kv[j & 1];
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    const int i = n * NT + tid, r = i / (D / PE) % BN, x = i % (D / PE) * PE;
                    float *dst = i < BN * (D / PE) ? &buf.k[r][x] : &buf.v[r][x];
                    const Vec<KV, PE> a = *reinterpret_cast<const Vec<KV, PE> *>(&raw[n]);
#pragma unroll
                    for (int e = 0; e < PE; e += 4)
                        *reinterpret_cast<float4 *>(dst + e) = make_float4(to_f(a.v[e]), to_f(a.v[e + 1]), to_f(a.v[e + 2]), to_f(a.v[e + 3]));
                }
            }
        };
        __syncthreads();                       // the unit before has read its tiles
        if (g.j0 < g.j1) {
            fetch(g.j0);
            land(g.j0);
        }
        for (int j = g.j0; j < g.j1; ++j) {
            if (COPY) cp_wait();
            __syncthreads();                   // tile j is there, the other buffer is free
            if (j + 1 < g.j1) fetch(j + 1);
            const auto &buf = sm.kv[j & 1];
            uint64_t s2[4][NK] = {};            // even and odd dims' sums
#pragma unroll 8
            for (int x = 0; x < D; x += 4) {
                ulonglong2 qa[4];
#pragma unroll
                for (int a = 0; a < 4; ++a) qa[a] = *reinterpret_cast<const ulonglong2 *>(&sm.q[ty * 4 + a][x]);
#pragma unroll
                for (int b = 0; b < NK; ++b) {
                    const ulonglong2 kb = *reinterpret_cast<const ulonglong2 *>(&buf.k[tx + 8 * b][x]);
#pragma unroll
                    for (int a = 0; a < 4; ++a) s2[a][b] = fma2(qa[a].y, kb.y, fma2(qa[a].x, kb.x, s2[a][b]));
                }
            }
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                float mx = -CUDART_INF_F, sc[NK];
#pragma unroll
                for (int b = 0; b < NK; ++b) {
                    const float2 s = halves(s2[a][b]);
                    sc[b] = j * BN + tx + 8 * b <= lim[a] ? (s.x + s.y) * scale : -CUDART_INF_F;
                    mx = fmaxf(mx, sc[b]);
                }
#pragma unroll
                for (int s = 4; s; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
                const float mn = fmaxf(m[a], mx);
                const float ms = mn == -CUDART_INF_F ? 0.f : mn;  // nothing seen yet
                const float al = exp2f(m[a] - ms);
                float sum = 0.f;
#pragma unroll
                for (int b = 0; b < NK; ++b) {
                    const float e = exp2f(sc[b] - ms);
                    sm.p[ty * 4 + a][tx + 8 * b] = e;
                    sum += e;
                }
#pragma unroll
                for (int s = 4; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
                l[a] = l[a] * al + sum;
                m[a] = mn;
#pragma unroll
                for (int b = 0; b < ND / 2; ++b) o[a][b] = mul2(o[a][b], both(al));
            }
            __syncwarp();                      // a row's probabilities stay within its eight lanes
#pragma unroll 8
            for (int k = 0; k < BN; k += 4) {
                float4 pa[4];
#pragma unroll
                for (int a = 0; a < 4; ++a) pa[a] = *reinterpret_cast<const float4 *>(&sm.p[ty * 4 + a][k]);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int b = 0; b < ND / 4; ++b) {
                        const ulonglong2 vv = *reinterpret_cast<const ulonglong2 *>(&buf.v[k + kk][b * 32 + tx * 4]);
#pragma unroll
                        for (int a = 0; a < 4; ++a) {
                            const uint64_t pv = both(kk == 0 ? pa[a].x : kk == 1 ? pa[a].y : kk == 2 ? pa[a].z : pa[a].w);
                            o[a][2 * b] = fma2(pv, vv.x, o[a][2 * b]);
                            o[a][2 * b + 1] = fma2(pv, vv.y, o[a][2 * b + 1]);
                        }
                    }
            }
            __syncwarp();                      // read before the next tile's are written
            if (j + 1 < g.j1) land(j + 1);
        }
        // whole unit: the output; a part: (m, l, o) for the joining kernel
        const bool part = g.j0 > 0 || g.j1 < g.nit;
        const int slot = g.j0 > 0 ? 0 : 1;
        if (part && g.j0 == 0 && tid == 0) ws.cut[blockIdx.x] = CutUnit{g.row0, R, g.head, g.followers};
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const int r = ty * 4 + a;
            if (r >= R) continue;
            const float inv = part ? 1.f : kv.vs / l[a];
            if (part && tx == 0) ws.ml[((long long)blockIdx.x * 2 + slot) * ws.rows + r] = make_float2(m[a], l[a]);
#pragma unroll
            for (int b = 0; b < ND / 4; ++b) {
                const float2 x = halves(o[a][2 * b]), y2 = halves(o[a][2 * b + 1]);
                const float ov[4] = {x.x, x.y, y2.x, y2.y};
                if (part) {
                    *reinterpret_cast<float4 *>(ws.o + (((long long)blockIdx.x * 2 + slot) * ws.rows + r) * D + b * 32 + tx * 4) =
                        make_float4(ov[0], ov[1], ov[2], ov[3]);
                } else {
                    Vec<Act, 4> y;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y.v[i] = Act(ov[i] * inv);
                        chk = fmaf(ov[i] * inv, 0.f, chk);
                    }
                    *reinterpret_cast<Vec<Act, 4> *>(out + ((long long)(g.row0 + r / G) * hq + g.head * G + r % G) * D +
                                                     b * 32 + tx * 4) = y;
                }
            }
        }
    }
    if (chk != 0.f) ws.odd[blockIdx.x] = 1;    // (after the first barrier of a unit: behind the 0 above)
}

// A masked key's probability is 0, and 0 times a V that is not finite is NaN: the
// products above let such a V reach rows before it.  An output row that is not
// finite is therefore looked at again by one warp: where a masked position that
// the row's tile may have covered (at most 128 tokens and 128 keys on) holds such
// a V, the row is computed anew from the keys it sees.  Slow, and reached by such
// caches alone; the check costs the others an FMA per output.
struct Again {
    ChunkP c;
    KvP kv;
    const void *q;
    int hq, hkv;
};
// row, query head h; all lanes call.  Kept short: loops that are not unrolled and
// one cache type, because its mere presence costs a cold call of the joining
// kernel time (2 us of 35 at its first size, measured without its ever running).
template <int D, class Act, class KV>
__device__ __forceinline__ void row_again(const Again &g, Act *out, int row, int h) {
    constexpr int E = D / 32;                  // dims of a lane
    const int lane = threadIdx.x % 32;
    int s = 0;
    while (s < g.c.S && row >= __ldg(g.c.off + s + 1)) ++s;
    if (s == g.c.S) return;                    // padding
    const int off = __ldg(g.c.off + s), pos = __ldg(g.c.ctx + s) + row - off, kvlen = pos - row + __ldg(g.c.off + s + 1);
    const KV *kp = static_cast<const KV *>(g.kv.k), *vp = static_cast<const KV *>(g.kv.v);
    const Act *q = static_cast<const Act *>(g.q) + ((long long)row * g.hq + h) * D;
    const float sc = fmaxf(rsqrtf((float)D) * 1.4426950408889634f * g.kv.ks, 1.2e-38f);
    float acc[E] = {}, m = -CUDART_INF_F, l = 0.f;
    bool odd = false, masked = true;
    // 32 keys at a time, first the masked ones, then from 0 on
    for (int k0 = pos + 1, end = min(kvlen, pos + 257);; k0 += 32) {
        if (k0 >= end) {
            if (!masked) break;
            if (!__any_sync(0xffffffffu, odd)) return;
            masked = false;
            k0 = 0;
            end = pos + 1;
        }
        const int k = min(k0 + lane, end - 1), ph = __ldg(g.kv.table + (long long)s * g.c.max_pages + k / 64);
        // (the main kernel has checked the pages)
        const long long at = (((long long)min(max(ph, 0), g.kv.n_pages - 1) * g.hkv + h / (g.hq / g.hkv)) * 64 + k % 64) * D;
        float x = 0.f;
#pragma unroll 2
        for (int e = 0; e < D; e += 4) {       // a lane's key: is V finite; the score
            const Vec<KV, 4> y = *reinterpret_cast<const Vec<KV, 4> *>((masked ? vp : kp) + at + e);
            const Vec<Act, 4> z = *reinterpret_cast<const Vec<Act, 4> *>(q + e);
#pragma unroll
            for (int i = 0; i < 4; ++i) x = fmaf(masked ? 0.f : to_f(z.v[i]), to_f(y.v[i]), x);
        }
        if (masked) {
            odd |= x != 0.f;
            continue;
        }
        x = k0 + lane < end ? x * sc : -CUDART_INF_F;
        float mn = fmaxf(m, x);
#pragma unroll
        for (int o = 16; o; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        const float ms = mn == -CUDART_INF_F ? 0.f : mn, al = exp2f(m - ms), p = exp2f(x - ms);
        m = mn;
        l = l * al + p;                        // (a lane's keys)
        bool nan = true;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= al;
#pragma unroll 4
        for (int i = 0; i < min(32, end - k0); ++i) {
            const Vec<KV, E> v = *reinterpret_cast<const Vec<KV, E> *>(vp + __shfl_sync(0xffffffffu, at, i) + lane * E);
            const float pi = __shfl_sync(0xffffffffu, p, i);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(pi, to_f(v.v[e]), acc[e]);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) nan &= acc[e] != acc[e];
        if (__all_sync(0xffffffffu, nan)) break;  // it stays so
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
    for (int e = 0; e < E; ++e) out[((long long)row * g.hq + h) * D + lane * E + e] = Act(acc[e] * (g.kv.vs / l));
}

// Joins the parts of every unit that a CTA of the attention kernel began and did
// not finish: slot 1 of that CTA and slot 0 of each follower, in CTA order.  The
// work is short and bound by the latency of its dependent loads (units, then
// statistics, then outputs), so it is cut into tasks that fill the GPU in one
// round: up to JP parts, a warp has JP loads in flight over several rows; beyond,
// a block's warps share a row's parts.
constexpr int JP = 8, JT = 256, JW = JT / 32, JMAX = 512;  // parts, threads, warps; CTAs of the attention kernel at most

__device__ __forceinline__ int parts_of(const CutUnit &u) { return (1 + abs(u.followers)) << (u.followers < 0); }
__device__ __forceinline__ int rows_of_task(int parts) { return parts <= 2 ? JW * JP / 2 : parts <= 4 ? JW * JP / 4 : parts <= 8 ? JW : 1; }

// parts of a row: one per CTA, or two (negative followers: two tiles shared the
// unit's rows), the second 128 rows behind
struct Parts {
    const AttnWs *ws;
    int cta, two, n;
    __device__ __forceinline__ int slot(int i, int r) const {  // (at most 2 * JMAX slots of 256 rows)
        const int c = i >> two;
        return ((cta + c) * 2 + (c == 0)) * ws->rows + r + (two ? (i & 1) * 128 : 0);
    }
};

template <int D, class Act>
__device__ __forceinline__ float join_store(const CutUnit &u, Act *out, int hq, int G, uint32_t ginv, int r, const float *acc, float inv) {  // NaN: not finite
    constexpr int E = D / 32;
    Vec<Act, E> y;
    float chk = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        y.v[e] = Act(acc[e] * inv);
        chk = fmaf(acc[e] * inv, 0.f, chk);
    }
    const int tok = r * ginv >> 16;
    *reinterpret_cast<Vec<Act, E> *>(out + ((long long)(u.row0 + tok) * hq + u.head * G + (r - tok * G)) * D + threadIdx.x % 32 * E) = y;
    return chk;
}

// up to P = 2, 4 or 8 parts: a warp takes JP / P rows from r0 on.  A part that the
// row sees nothing of has weight 0, and its output may not be there.  One code for
// the three, lp = log2 P: a cold call pays for the kernel's length.
template <int D, class Act>
__device__ __forceinline__ float join_rows(const CutUnit &u, const Parts &ps, Act *out, int hq, int G, uint32_t ginv, int r0, int lp, float vs) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x % 32, P = 1 << lp, row = r0 + (lane >> lp), part = lane & (P - 1);
    float2 ml = make_float2(-CUDART_INF_F, 0.f);
    if (lane < JP && row < u.rows && part < ps.n) ml = ps.ws->ml[ps.slot(part, row)];
    float M = ml.x;
    for (int o = P / 2; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float f = ml.x > -CUDART_INF_F ? exp2f(ml.x - M) : 0.f;
    float L = ml.y * f;
    for (int o = P / 2; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    Vec<float, E> x[JP];
    float fk[JP], acc[E] = {}, chk = 0.f;
#pragma unroll
    for (int k = 0; k < JP; ++k) {
        fk[k] = __shfl_sync(0xffffffffu, f, k);
#pragma unroll
        for (int e = 0; e < E; ++e) x[k].v[e] = 0.f;
        if (fk[k] != 0.f) x[k] = *reinterpret_cast<const Vec<float, E> *>(ps.ws->o + (long long)ps.slot(k & (P - 1), r0 + (k >> lp)) * D + lane * E);
    }
#pragma unroll
    for (int k = 0; k < JP; ++k) {
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(x[k].v[e], fk[k], acc[e]);
        if (k % 2 == 0 || (~k & (P - 1))) continue;
        const float l = __shfl_sync(0xffffffffu, L, k);
        if (r0 + (k >> lp) < u.rows) chk += join_store<D>(u, out, hq, G, ginv, r0 + (k >> lp), acc, __fdividef(vs, l));
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
    }
    return chk;
}

__device__ __forceinline__ int unit_of(const int *upto, int n_cta, int task) {  // the first unit whose tasks end behind this one
    int lo = 0, hi = n_cta - 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (upto[mid] > task) hi = mid; else lo = mid + 1;
    }
    return lo;
}

// the rows that this warp joined (own) and those of whole units (odd)
template <int D, class Act, class KV>
__device__ __noinline__ void rows_again(const Again &g, Act *out, const CutUnit *cut, const int *upto, int base, int n_cta, bool own, bool odd) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x % 32, wid = threadIdx.x / 32, hq = g.hq, G = hq / g.hkv;
    int task = own ? blockIdx.x : base, r = 0;
    for (int row = 0, h = blockIdx.x * JW + wid;;) {  // h of all rows' heads, 152 * 24 apart
        int y, z;                              // row, head
        if (task < base) {
            const int lo = unit_of(upto, n_cta, task), per = rows_of_task(parts_of(cut[lo])), mine = max(per / JW, 1);
            const int at = (task - (lo ? upto[lo - 1] : 0)) * per + (wid * per / JW) + r;
            if (r == mine || at >= cut[lo].rows || (per < JW && wid > 0)) {  // (per = 1: warp 0's)
                task += gridDim.x;
                r = 0;
                continue;
            }
            ++r;
            y = cut[lo].row0 + at / G;
            z = cut[lo].head * G + at % G;
        } else {
            for (; h >= hq; h -= hq) ++row;
            if (!odd || row >= g.c.n_rows) break;
            y = row;
            z = h;
            h += gridDim.x * JW;
            bool joined = false;
            for (int k = lane; k < n_cta; k += 32)
                joined |= cut[k].followers && z / G == cut[k].head && y >= cut[k].row0 && y < cut[k].row0 + cut[k].rows / G;
            if (__any_sync(0xffffffffu, joined)) continue;
        }
        const Act *o = out + ((long long)y * hq + z) * D + lane * E;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x = fmaf(to_f(o[e]), 0.f, x);
        if (__any_sync(0xffffffffu, x != 0.f)) row_again<D, Act, KV>(g, out, y, z);
    }
}

template <int D, class Act, class KV>
__global__ void __launch_bounds__(JT, 3) attn_join_kernel(AttnWs ws, Ctrl *ctrl, const __grid_constant__ Again g, Act *out, int n_cta) {
    __shared__ CutUnit cut[JMAX];
    __shared__ int upto[JMAX];                 // tasks of units 0..i
    __shared__ int wsum[JW];
    __shared__ float part[JW][D], partl[JW];
    constexpr int E = D / 32;
    const int tid = threadIdx.x, lane = tid % 32, wid = tid / 32, hq = g.hq, G = hq / g.hkv;
    const float vs = g.kv.vs;
    const uint32_t ginv = 65536u / G + 1;      // r / G = r * ginv >> 16 for r < 256, G <= 128
    cudaGridDependencySynchronize();
    CutUnit u{0, 0, 0, 0};                     // one latency for the units and the abort word
    if (tid < n_cta) u = ws.cut[tid];
    bool odd = tid < n_cta && ws.odd[tid];
    if (__syncthreads_or(tid == 0 && aborted(ctrl))) return;
    int base = 0;
    for (int b = 0; b < n_cta; b += JT) {
        const int i = b + tid;
        if (b) {
            u = i < n_cta ? ws.cut[i] : CutUnit{0, 0, 0, 0};
            odd |= i < n_cta && ws.odd[i];
        }
        const int per = rows_of_task(parts_of(u));
        int x = u.followers ? (u.rows + per - 1) / per : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) wsum[wid] = x;
        __syncthreads();
        int all = 0;
        for (int k = 0; k < JW; ++k) {
            if (k < wid) x += wsum[k];
            all += wsum[k];
        }
        if (i < n_cta) {
            cut[i] = u;
            upto[i] = base + x;
        }
        base += all;
        odd = __syncthreads_or(odd);
    }
    float chk = 0.f;                           // becomes NaN where an output is not finite
    for (int task = blockIdx.x; task < base; task += gridDim.x) {
        const int lo = unit_of(upto, n_cta, task);
        const CutUnit u = cut[lo];
        const Parts ps{&ws, lo, u.followers < 0, parts_of(u)};
        const int row0 = (task - (lo ? upto[lo - 1] : 0)) * rows_of_task(ps.n);
        if (ps.n <= JP) {
            const int lp = ps.n <= 2 ? 1 : ps.n <= 4 ? 2 : 3;
            chk += join_rows<D>(u, ps, out, hq, G, ginv, row0 + (wid * JP >> lp), lp, vs);
        } else {
            // one row: warp w takes parts w, w + JW, ...; all of them the row's maximum
            float M = -CUDART_INF_F;
            for (int i = lane; i < ps.n; i += 32) M = fmaxf(M, ws.ml[ps.slot(i, row0)].x);
#pragma unroll
            for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            float acc[E] = {}, L = 0.f;
            for (int i0 = wid; i0 < ps.n; i0 += JW * JP) {
                const int mine = i0 + JW * lane;
                float f = 0.f;
                if (lane < JP && mine < ps.n) {
                    const float2 ml = ws.ml[ps.slot(mine, row0)];
                    if (ml.x > -CUDART_INF_F) f = exp2f(ml.x - M);
                    L += ml.y * f;
                }
                Vec<float, E> x[JP];
                float fk[JP];
#pragma unroll
                for (int k = 0; k < JP; ++k) {
                    fk[k] = __shfl_sync(0xffffffffu, f, k);
#pragma unroll
                    for (int e = 0; e < E; ++e) x[k].v[e] = 0.f;
                    if (fk[k] != 0.f) x[k] = *reinterpret_cast<const Vec<float, E> *>(ws.o + (long long)ps.slot(i0 + JW * k, row0) * D + lane * E);
                }
#pragma unroll
                for (int k = 0; k < JP; ++k)
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] = fmaf(x[k].v[e], fk[k], acc[e]);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll
            for (int e = 0; e < E; ++e) part[wid][lane * E + e] = acc[e];
            if (lane == 0) partl[wid] = L;
            __syncthreads();
            if (wid == 0) {
                L = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = 0.f;
                for (int k = 0; k < JW; ++k) {
                    L += partl[k];
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] += part[k][lane * E + e];
                }
                chk += join_store<D>(u, out, hq, G, ginv, row0, acc, __fdividef(vs, L));
            }
            __syncthreads();
        }
    }
    const bool own = __any_sync(0xffffffffu, chk != 0.f);
    if (own || odd) rows_again<D, Act, KV>(g, out, cut, upto, base, n_cta, own, odd);
}

template <int D, class Act, class KV>
cudaError_t join(const AttnWs &ws, Ctrl *ctrl, const Again &g, Act *out, int grid, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(3 * 152);
    cfg.blockDim = dim3(JT);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<D, Act, KV>, ws, ctrl, g, out, grid);
}

template <int D, class Act, class KV>
cudaError_t attn(const ChunkP &c, const KvP &kv, const AttnWs &ws, Ctrl *ctrl, const void *q, void *out, int hq, int hkv,
                 int grid, cudaStream_t s) {
    attn_simt_kernel<D, Act, KV><<<grid, NT, sizeof(Smem<D>), s>>>(c, kv, ws, ctrl, static_cast<const Act *>(q),
                                                                    static_cast<Act *>(out), hq, hkv);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return join<D, Act, KV>(ws, ctrl, Again{c, kv, q, hq, hkv}, static_cast<Act *>(out), grid, s);
}
template <int D, class Act, class KV>
cudaError_t setup() {
    return cudaFuncSetAttribute(attn_simt_kernel<D, Act, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(Smem<D>));
}
}  // namespace

cudaError_t mk_attn_setup(bool f32) {
    if (!f32) return mk_attn_mma_setup();
    cudaError_t e = setup<64, float, float>();
    return e != cudaSuccess ? e : setup<64, float, __nv_bfloat16>();
}
int mk_attn_ws_rows(bool f32) { return f32 ? BM : 256; }
int mk_attn_grid(bool f32, int sms) { return min(f32 ? 2 * sms : sms, JMAX); }

cudaError_t mk_attn_launch(const ChunkP &c, const KvP &kv, const AttnWs &ws, Ctrl *ctrl, const CUtensorMap *maps,
                           const void *q, void *out, int hq, int hkv, bool f32, int grid, long long timeout_ns,
                           cudaStream_t s) {
    if (f32)
        return kv.dtype == MK_DT_F32 ? attn<64, float, float>(c, kv, ws, ctrl, q, out, hq, hkv, grid, s)
                                     : attn<64, float, __nv_bfloat16>(c, kv, ws, ctrl, q, out, hq, hkv, grid, s);
    cudaError_t e = mk_attn_mma_launch(c, kv, ws, ctrl, maps, out, hq, hkv, grid, timeout_ns, s);
    if (e != cudaSuccess) return e;
    const Again g{c, kv, q, hq, hkv};
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(out);
    return kv.dtype == MK_DT_FP8E4M3 ? join<128, __nv_bfloat16, __nv_fp8_e4m3>(ws, ctrl, g, o, grid, s)
                                     : join<128, __nv_bfloat16, __nv_bfloat16>(ws, ctrl, g, o, grid, s);
}
