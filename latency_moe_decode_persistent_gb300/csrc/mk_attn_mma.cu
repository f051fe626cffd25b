// Attention of a chunk over the paged cache on the tensor cores (tcgen05), for
// head dim 128, bf16 queries, and a bf16 or FP8 E4M3 cache.
//
// A unit is two tiles (A, B) of up to 128 rows, a row being one query head of
// one token: the G heads that share a kv head lie side by side, so a tile is
// 128/G tokens.  Per 128 keys and tile: S = Q K^T (fp32 in TMEM), the softmax
// warpgroup of the tile turns its row of S into probabilities, stores them over
// S in 16 bits, and O += P V takes them from TMEM.  The two tiles alternate on
// the tensor cores: while one is in its softmax the other multiplies.
//
//   warps 0-3, 4-7   softmax of tile A, B: one row per thread; writes its output
//   warp 8           loader: K and V pages by TMA (two pages per tile)
//   warp 9           issues the MMAs
//   warps 10, 11     load Q of tile A, B
//   warps 12-15      FP8 cache only: codes -> f16 tiles for the MMAs (exact)
//
// A unit whose tokens fit one tile (decoding, short blocks) would leave the
// second idle and be bound by the chain S -> softmax -> O of the first: there
// both tiles hold the same rows and take the iterations in turn, and tile A's
// warps add B's (maximum, sum, output) to theirs through shared memory at the
// end.
//
// The online softmax keeps a reference maximum per row and moves it, with a
// rescale of O in TMEM, only when the row's maximum has grown by more than 2^8
// (bf16) or 2^4 (f16, FP8 caches): probabilities may exceed 1 by that much, and
// the rescale leaves the common path.
//
// Behind a stream's last position a page holds whatever was there: 0 * NaN must
// not reach O.  The last page's box therefore starts `sh` rows early (rows of a
// page are an axis of their own in the tensor map), so that its valid rows lie
// at the box's end and the rest is TMA's zero fill, for K and V alike.
//
// Measured (32/4 heads, one GB300; of the copy bandwidth and the cuBLAS bf16 rate):
//   one prompt of 8192 tokens, bf16      384 us   1.43 PFLOP/s, 73 %: the chain S -> softmax
//                                                 -> P -> O of two tiles, whose waits leave the
//                                                 tensor cores idle for 30 % of the kernel
//   chunks up to 2048, FP8 cache         191 us   1.08 PFLOP/s, 55 %: 3950 cycles per 128 keys of
//                                                 two tiles, against 2048 of MMAs and some 2500
//                                                 of shared memory; the widening of the codes
//                                                 lies between their arrival and the MMAs
//   16 single tokens, bf16 cache          39 us   4.0 TB/s, 59 %: this kernel 32 us (4.9 TB/s)
//   6 tokens over 65536, FP8 cache        33 us   2.0 TB/s, 30 %: this kernel 27 us; the
//                                                 widening is 1500 of 2900 cycles per 128 keys
// A split call's joining kernel takes 6 to 9 us of that, and a call's start
// (launch, plan, first tiles) 4.  On the prompt, 128 keys of two tiles take 2650
// cycles: 2048 of MMAs, and as many of shared memory; per tile 1400 of softmax and
// 1100 until the next S.  A unit's end and start cost 4500 more.
#include "mk_chunk.cuh"

namespace {
using namespace mkc;

constexpr int BN = 128;              // keys per iteration (two pages)
constexpr uint32_t TILE = 32768;     // bytes of a 128 x 128 tile of 16-bit values: two 64-column halves, 128-byte swizzle
constexpr uint32_t HALF_TILE = 16384;
constexpr uint32_t RAW_TILE = 16384; // 128 x 128 E4M3 codes

template <bool FP8>
struct Cfg {
    static constexpr int THREADS = FP8 ? 512 : 384;
    // The cost line along which the CTAs share the work: a unit's start and end count
    // as OV iterations (an FP8 cache's include the conversion of Q).  Measured with 2,
    // 3, 4, 5: a prompt of 8192 tokens, bf16, 391, 387, 388, 391 us; chunks up to 2048
    // over FP8 216, 200, 196, 192.  A CTA takes MIN_COST at least, so that small calls
    // are not cut to pieces: the mean of 44 calls of 1 to 16 streams of random lengths and
    // contexts is 29.3 us with OV + 1, 29.0 with OV, 29.3 with OV - 1; 137 tokens alone
    // take 20.5 with OV + 2, 14.4 with OV.
    static constexpr int OV = FP8 ? 5 : 3, MIN_COST = OV;
    // A row's reference maximum moves when its maximum has grown by more than GROW powers
    // of two, and its probabilities, their sum and its output are held times 2^BIAS, which
    // cancels.  In f16 2^(BIAS + GROW) may be the largest, and numbers below 2^-14 lose
    // bits: with 2^11 a key counts with all bits down to 2^-25 of its row's largest, and as
    // a multiple of 2^-35 of it below (without the bias, 65536 keys 18 nats below one whose
    // V is 0 vanished).  Moves cost time: chunks up to 2048 over FP8 take 190.5 us with a
    // GROW of 8, 190.6 with 4, 198 with 2, 207 with 1.  A bf16's range needs none of it.
    static constexpr float GROW = FP8 ? 4.f : 8.f, BIAS = FP8 ? 11.f : 0.f;
    static constexpr int RING = FP8 ? 3 : 5;        // tiles the MMAs read
    static constexpr int RAW = FP8 ? 4 : 0;         // tiles of codes
    static constexpr uint32_t Q = 0, KV = 2 * TILE, RAWS = KV + RING * TILE, BARS = RAWS + RAW * RAW_TILE;
    static constexpr uint32_t STAT = BARS + 320, MISC = STAT + 1024, TOTAL = MISC + 64;
    static constexpr int SOFT_REGS = FP8 ? 192 : 216, OTHER_REGS = FP8 ? 64 : 72;
    static_assert((SOFT_REGS * 256 + OTHER_REGS * (THREADS - 256)) <= (THREADS == 512 ? 128 : 168) * THREADS, "registers");
};

struct MmaP {
    ChunkP c;
    KvP kv;
    AttnWs ws;
    Ctrl *ctrl;
    __nv_bfloat16 *out;
    int hq, hkv, min_cost;
    int G, tpt;                          // heads per kv head, tokens per tile
    int wide_out;                        // out is 32-byte aligned
    uint32_t ginv;                       // r / G = r * ginv >> 16 for r < 128
    uint32_t tries;                      // of a wait, a microsecond or less each
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint32_t b, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(b), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(b) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(b), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t b, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.b32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok) : "r"(b), "r"(parity) : "memory");
    return ok != 0;
}
// the same, asleep for a microsecond at most
__device__ __forceinline__ bool bar_try_us(uint32_t b, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.b32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok) : "r"(b), "r"(parity), "r"(1000) : "memory");
    return ok != 0;
}
// Every wait ends: after `tries` attempts, each of which sleeps up to a
// microsecond, or once another role gave up (*gone).  A count and not a clock,
// because every wait is inlined: with a timed loop in each the kernel's code
// outgrew the instruction cache.  The first attempt has the hardware's own time
// limit, which wakes sooner: a prompt of 8192 tokens 412 us, 428 with
// the microsecond's alone.
struct Waiter {
    volatile int *gone;
    uint32_t tries;
    __device__ __forceinline__ bool one(uint32_t b, uint32_t parity) const {  // a single thread
        if (bar_try(b, parity)) return true;
        for (uint32_t n = 0; !bar_try_us(b, parity); ++n)
            if (n >= tries || *gone) {
                *gone = 1;
                return false;
            }
        return true;
    }
    __device__ __forceinline__ bool operator()(uint32_t b, uint32_t parity) const {  // a whole warp, one verdict
        return __all_sync(0xffffffffu, one(b, parity));
    }
};

__device__ __forceinline__ void tma3(uint32_t dst, const CUtensorMap *m, int x, int y, int z, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
// The MMA warp runs as a whole, with one elected lane issuing: its operands then
// come from uniform registers.  (One diverged lane, which has to move every
// descriptor there, took 90 cycles per MMA, more than the MMA's 64.)
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r;
}
// Shared-memory descriptors, 128-byte swizzle, 8-row groups 1024 bytes apart:
// low words for K-major tiles and for MN-major ones (64-column groups 16 KB
// apart along N), and the common high word
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return (addr & 0x3ffff) >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr) { return (addr & 0x3ffff) >> 4 | (HALF_TILE >> 4) << 16; }
constexpr uint32_t DESC_HI = 64u | 1u << 14 | 2u << 29;
#define MMA_SS(off, acc) \
    " add.u32 x, %1, " off ";\n add.u32 y, %2, " off ";\n mov.b64 da, {x, %5};\n mov.b64 db, {y, %5};\n" \
    " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, " acc ";\n"
#define MMA_TS(aoff, boff, acc) \
    " add.u32 x, %1, " aoff ";\n add.u32 y, %2, " boff ";\n mov.b64 db, {y, %5};\n" \
    " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, " acc ";\n"
// D = A B over 128 columns: A, B K-major in shared memory
__device__ __forceinline__ void mma8_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t elect) {
    asm volatile("{\n .reg .pred e, t, f;\n .reg .b32 x, y;\n .reg .b64 da, db;\n setp.ne.u32 e, %4, 0;\n setp.eq.u32 t, 0, 0;\n setp.ne.u32 f, 0, 0;\n"
                 MMA_SS("0", "f") MMA_SS("2", "t") MMA_SS("4", "t") MMA_SS("6", "t")
                 MMA_SS("1024", "t") MMA_SS("1026", "t") MMA_SS("1028", "t") MMA_SS("1030", "t") "}\n"
                 ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(elect), "n"(DESC_HI) : "memory");
}
// D (+)= A B over 64 keys: A in TMEM, B MN-major in shared memory
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t elect, uint32_t acc) {
    asm volatile("{\n .reg .pred e, t, f;\n .reg .b32 x, y;\n .reg .b64 db;\n setp.ne.u32 e, %4, 0;\n setp.eq.u32 t, 0, 0;\n setp.ne.u32 f, %6, 0;\n"
                 MMA_TS("0", "0", "f") MMA_TS("8", "128", "t") MMA_TS("16", "256", "t") MMA_TS("24", "384", "t") "}\n"
                 ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(elect), "n"(DESC_HI), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t elect) {
    asm volatile("{\n .reg .pred e;\n setp.ne.u32 e, %1, 0;\n"
                 " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar), "r"(elect) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define I8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void tm_ld32(uint32_t a, uint32_t *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
                 "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : R8(v, 0), R8(v, 8), R8(v, 16), R8(v, 24) : "r"(a));
}
__device__ __forceinline__ void tm_ld16(uint32_t a, uint32_t *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : R8(v, 0), R8(v, 8) : "r"(a));
}
__device__ __forceinline__ void tm_st16(uint32_t a, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
                 ::I8(v, 0), I8(v, 8), "r"(a) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two floats side by side
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_out(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// 32 bytes, a whole sector, of a lane's row
__device__ __forceinline__ void st_global32(void *p, const uint32_t *v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), I8(v, 0) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// what the roles agree on about a tile of a segment: its iterations are
// j0, j0 + step, ... below j1
struct TileSeg {
    int rows;     // rows of the tile (0: none)
    int tok0;     // its first token within the unit
    int j0, j1;
};
// both tiles on the same rows, taking turns
__device__ __forceinline__ bool dual_seg(const Seg &g, int tpt) { return g.ntok <= tpt && g.j1 - g.j0 > 1; }
__device__ __forceinline__ TileSeg tile_of(const Seg &g, int X, int tpt, int G) {
    TileSeg t;
    if (dual_seg(g, tpt)) return TileSeg{g.ntok * G, 0, g.j0 + X, g.j1};
    t.tok0 = X * tpt;
    const int n = min(max(g.ntok - t.tok0, 0), tpt);
    t.rows = n * G;
    t.j0 = g.j0;
    t.j1 = n ? min(g.j1, (g.ctx + g.tok0 + t.tok0 + n + BN - 1) / BN) : 0;
    return t;
}

template <bool FP8>
__global__ void __launch_bounds__(Cfg<FP8>::THREADS, 1)
attn_mma_kernel(const __grid_constant__ MmaP p, const __grid_constant__ CUtensorMap mapk, const __grid_constant__ CUtensorMap mapv,
                const __grid_constant__ CUtensorMap mapq) {
    using C = Cfg<FP8>;
    extern __shared__ unsigned char raw_smem[];
    unsigned char *sm = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
    const uint32_t s0 = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int G = p.G, tpt = p.tpt;
    const uint32_t ginv = p.ginv;
    const uint32_t bars = s0 + C::BARS;
    auto full = [&](int i) { return bars + 8 * i; };
    auto empty = [&](int i) { return bars + 40 + 8 * i; };
    constexpr int RAW = FP8 ? C::RAW : 1;     // (a modulus)
    auto rfull = [&](int i) { return bars + 80 + 8 * i; };
    auto rempty = [&](int i) { return bars + 112 + 8 * i; };
    auto qfull = [&](int x) { return bars + 144 + 8 * x; };
    auto sfull = [&](int x) { return bars + 160 + 8 * x; };
    auto pfull = [&](int x) { return bars + 176 + 8 * x; };
    auto ofull = [&](int x) { return bars + 192 + 8 * x; };
    const uint32_t fin = bars + 208, aready = bars + 216, bdone = bars + 224, adone = bars + 232;
    auto qfree = [&](int x) { return bars + 240 + 8 * x; };
    auto phalf = [&](int x) { return bars + 256 + 8 * x; };
    auto qraw = [&](int x) { return bars + 272 + 8 * x; };
    volatile int *misc = reinterpret_cast<volatile int *>(sm + C::MISC);  // 0: a role gave up, 1: TMEM base, 2: so did its drain

    cudaTriggerProgrammaticLaunchCompletion();  // the joining kernel may come up while this one ends
    if (warp == 8) {
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(&mapk) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(&mapv) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(&mapq) : "memory");
            for (int i = 0; i < C::RING; ++i) {
                bar_init(full(i), FP8 ? 4 : 1);
                bar_init(empty(i), 1);
            }
            for (int i = 0; i < C::RAW; ++i) {
                bar_init(rfull(i), 1);
                bar_init(rempty(i), 4);
            }
            for (int x = 0; x < 2; ++x) {
                bar_init(qfull(x), 1);
                bar_init(qfree(x), 1);
                bar_init(qraw(x), 1);
                bar_init(phalf(x), 4);
                bar_init(sfull(x), 1);
                bar_init(pfull(x), 4);
                bar_init(ofull(x), 1);
            }
            bar_init(fin, 1);
            bar_init(aready, 4);
            bar_init(bdone, 4);
            bar_init(adone, 4);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            misc[0] = misc[2] = 0;
        }
    } else if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(s0 + C::MISC + 4) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        fence_before();
    }
    const bool stop = tid == 0 && aborted(p.ctrl);  // an earlier call's error (read while the plan is made)
    Walk<BN, C::OV> w;
    const bool good = w.plan(&p.c, 2 * tpt, p.hkv, gridDim.x, blockIdx.x, p.min_cost);
    if (tid == 0) {
        if (!good) raise(p.ctrl, MK_ERR_BAD_INPUT, 402);
        p.ws.cut[blockIdx.x].followers = 0;
        p.ws.odd[blockIdx.x] = 0;
    }
    const bool idle = __syncthreads_or(stop) || !good;  // one verdict for the CTA
    fence_after();
    if (idle) w.pos = w.end = 0;
    const uint32_t tm = (uint32_t)misc[1];    // columns: S_A 0, S_B 128, O_A 256, O_B 384
    const Waiter wait{misc, p.tries};
    const uint32_t qs = s0 + C::Q, ring = s0 + C::KV;
    Seg g;

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFT_REGS));
        const int X = warp / 4, wr = warp % 4 * 32;             // tile, first row of the warp
        const uint32_t ts = tm + X * 128 + (wr << 16), to = tm + 256 + X * 128 + (wr << 16);
        // scores in the log2 domain; positive, so that it keeps -inf
        const float sc = fmaxf(0.08838834764831845f * 1.4426950408889634f * p.kv.ks, 1.2e-38f);
        uint32_t ps = 0, po = 0, pd = 0;                        // phases of sfull, ofull; of aready and bdone
        bool live = true;
        while (live && w.next(g)) {
            const bool dual = dual_seg(g, tpt);
            const TileSeg t = tile_of(g, X, tpt, G);
            const int step = dual ? 2 : 1;
            if (!t.rows) continue;
            const int r = wr + lane;
            const int unit_row = t.tok0 * G + r;
            const bool part = g.j0 > 0 || g.j1 < g.nit, mine = r < t.rows, single = g.ntok <= tpt;
            const long long slot = (long long)blockIdx.x * 2 + (g.j0 > 0 ? 0 : 1);
            // parts: rows of the unit; of a one-tile unit A's rows, then B's from 128 on
            float2 *pml = p.ws.ml + slot * p.ws.rows + (single ? X * 128 + r : unit_row);
            float *pdst = p.ws.o + (slot * p.ws.rows + (single ? X * 128 + r : unit_row)) * 128;
            if (part && g.j0 == 0 && X == 0 && r == 0)
                p.ws.cut[blockIdx.x] = CutUnit{g.row0, g.ntok * G, g.head, single ? -g.followers : g.followers};
            if (part && single && !dual && mine) pml[128] = make_float2(-CUDART_INF_F, 0.f);  // (X == 0) no B here
            if (t.j1 <= t.j0) {                                 // this part lies behind the tile's last key
                if (mine) *pml = make_float2(-CUDART_INF_F, 0.f);
                continue;
            }
            const int lim = g.ctx + g.tok0 + t.tok0 + (int)(min(r, t.rows - 1) * ginv >> 16);   // last key of the row
            const int first = g.ctx + g.tok0 + t.tok0;                          // last key of the tile's first row
            float m = -CUDART_INF_F, l = 0.f;                   // reference maximum (raw scores), sum
            for (int j = t.j0; j < t.j1; j += step) {
                if (!wait(sfull(X), ps)) { live = false; break; }
                ps ^= 1;
                fence_after();
                if (wr >= t.rows) {                             // no rows in this warp: its part of P is never read back
                    fence_before();
                    if (lane == 0) {
                        bar_arrive(phalf(X));
                        bar_arrive(pfull(X));
                    }
                    continue;
                }
                uint32_t sv[128];
#pragma unroll
                for (int b = 0; b < 4; ++b) tm_ld32(ts + 32 * b, sv + 32 * b);
                wait_ld();
                float *s = reinterpret_cast<float *>(sv);
                const int k0 = j * BN;
                if (k0 + BN - 1 > first || k0 + BN > g.kvlen) {
#pragma unroll
                    for (int b = 0; b < 4; ++b) {               // 32 columns; a page's valid rows end its box
                        const int kb = k0 + 64 * (b / 2), sh = 64 - min(max(g.kvlen - kb, 0), 64);
                        const int lo = sh - 32 * (b % 2), hi = lim - kb + lo;    // visible: lo <= c <= hi
                        uint32_t see = lo >= 32 || hi < 0 ? 0u : ~0u << max(lo, 0);
                        if (hi < 31) see &= (2u << max(hi, 0)) - 1;
#pragma unroll
                        for (int c = 0; c < 32; ++c) s[32 * b + c] = see >> c & 1 ? s[32 * b + c] : -CUDART_INF_F;
                    }
                }
                // four chains of three-input maxima
                float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int c = 4; c < 124; c += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) mx4[k] = fmaxf(fmaxf(mx4[k], s[c + 2 * k]), s[c + 2 * k + 1]);
#pragma unroll
                for (int k = 0; k < 4; ++k) mx4[k] = fmaxf(mx4[k], s[124 + k]);
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                if (__any_sync(0xffffffffu, mine && ((mx - m) * sc > C::GROW || (m == -CUDART_INF_F && mx > m)))) {
                    const float mn = fmaxf(m, mx), al = m == -CUDART_INF_F ? 0.f : ex2((m - mn) * sc);
                    m = mn;
                    l *= al;
                    if (j > t.j0) {
#pragma unroll
                        for (int b = 0; b < 8; ++b) {
                            uint32_t ov[16];
                            tm_ld16(to + 16 * b, ov);
                            wait_ld();
#pragma unroll
                            for (int c = 0; c < 16; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * al);
                            tm_st16(to + 16 * b, ov);
                        }
                    }
                }
                const float mr = m == -CUDART_INF_F ? 0.f : C::BIAS - m * sc;
                const uint64_t sc2 = f2(sc, sc), mr2 = f2(mr, mr);
                uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint32_t pv[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        float e0, e1;
                        f2_out(fma2(f2(s[32 * b + 2 * c], s[32 * b + 2 * c + 1]), sc2, mr2), e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        acc[c % 4] = add2(acc[c % 4], f2(e0, e1));
                        pv[c] = pack2<FP8>(e0, e1);
                    }
                    tm_st16(ts + 16 * b, pv);
                    if (b == 1) {                               // the first 64 keys may be multiplied
                        wait_st();
                        fence_before();
                        __syncwarp();
                        if (lane == 0) bar_arrive(phalf(X));
                    }
                }
                float l0, l1;
                f2_out(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), l0, l1);
                l += l0 + l1;
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(pfull(X));
            }
            if (!live || !wait(ofull(X), po)) break;
            po ^= 1;
            fence_after();
            if (part) {
                // the statistics and the output as they are; joined by the next kernel
                if (mine) *pml = make_float2(m * sc, l);
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    uint32_t ov[32];
                    __syncwarp();
                    tm_ld32(to + 32 * b, ov);
                    wait_ld();
                    if (mine)
#pragma unroll
                        for (int c = 0; c < 4; ++c) st_global32(pdst + 32 * b + 8 * c, ov + 8 * c);
                }
                continue;
            }
            float fa = p.kv.vs / l, fb = 0.f;                   // weights of A's and B's output
            const unsigned char *orow = sm + C::Q + r * 512;
            if (dual) {
                // B's rows go to A through the Q tiles, which no MMA reads any more: 32
                // pieces of 16 bytes, their order turned by the row so that neighbouring
                // lanes meet different banks
                float *stat = reinterpret_cast<float *>(sm + C::STAT);
                if (X == 1) {
                    if (!wait(aready, pd)) break;
#pragma unroll 1
                    for (int b = 0; b < 4; ++b) {
                        uint32_t ov[32];
                        __syncwarp();
                        tm_ld32(to + 32 * b, ov);
                        wait_ld();
                        if (mine)
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                st_shared16(smem_u32(orow) + (((8 * b + c) ^ lane) << 4),
                                            make_uint4(ov[4 * c], ov[4 * c + 1], ov[4 * c + 2], ov[4 * c + 3]));
                    }
                    stat[r] = m;
                    stat[128 + r] = l;
                    fence_async();                              // the next unit's Q comes by TMA to the same bytes
                    fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(bdone);
                    pd ^= 1;
                    continue;
                }
                if (lane == 0) bar_arrive(aready);              // A's MMAs are done
                if (!wait(bdone, pd)) break;
                pd ^= 1;
                const float mb = stat[r], lb = stat[128 + r], mn = fmaxf(m, mb);
                fa = m == -CUDART_INF_F ? 0.f : ex2((m - mn) * sc);
                fb = mb == -CUDART_INF_F ? 0.f : ex2((mb - mn) * sc);
                const float inv = p.kv.vs / (l * fa + lb * fb);
                fa *= inv;
                fb *= inv;
            }
            const int tok = r * ginv >> 16;
            float chk = 0.f;                                    // becomes NaN where an output is not finite
            __nv_bfloat16 *dst = p.out + ((long long)(g.row0 + t.tok0 + tok) * p.hq + g.head * G + (r - tok * G)) * 128;
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
                uint32_t ov[32];
                __syncwarp();
                tm_ld32(to + 32 * b, ov);
                wait_ld();
                if (mine) {
                    float o[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = __uint_as_float(ov[c]) * fa;
                    if (dual)
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const float4 x = *reinterpret_cast<const float4 *>(orow + (((8 * b + c) ^ lane) << 4));
                            o[4 * c] += x.x * fb;
                            o[4 * c + 1] += x.y * fb;
                            o[4 * c + 2] += x.z * fb;
                            o[4 * c + 3] += x.w * fb;
                        }
#pragma unroll
                    for (int c = 0; c < 32; ++c) chk = fmaf(o[c], 0.f, chk);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t y[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c) y[c] = pack2<false>(o[16 * h + 2 * c], o[16 * h + 2 * c + 1]);
                        if (p.wide_out) {
                            st_global32(dst + 32 * b + 16 * h, y);
                        } else {
                            *reinterpret_cast<uint4 *>(dst + 32 * b + 16 * h) = make_uint4(y[0], y[1], y[2], y[3]);
                            *reinterpret_cast<uint4 *>(dst + 32 * b + 16 * h + 8) = make_uint4(y[4], y[5], y[6], y[7]);
                        }
                    }
                }
            }
            if (chk != 0.f) p.ws.odd[blockIdx.x] = 1;
            if (dual) {
                fence_async();
                __syncwarp();
                if (lane == 0) bar_arrive(adone);               // the Q tiles are free again
            }
        }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
        if (warp == 8 && w.pos < w.end) {
            // loader: K and V of each iteration, in the order the MMAs take them
            int n = 0;                                          // tiles issued
            constexpr int SLOTS = FP8 ? C::RAW : C::RING;
            bool live = true;
            while (live && w.next(g)) {
                const int32_t *tab = p.kv.table + (long long)g.stream * p.c.max_pages;
                const int pages = (g.kvlen + 63) / 64;
                // K runs one iteration ahead of V, two where the tiles take turns
                const int lead = dual_seg(g, tpt) ? 2 : 1;
                int base = 2 * g.j0;                            // table entries base..base+31, one per lane, and the next 32
                int cur = base + lane < pages ? __ldg(tab + base + lane) : 0;
                int nxt = base + 32 + lane < pages ? __ldg(tab + base + 32 + lane) : 0;
                for (int i = -lead; live && i < g.j1 - g.j0; ++i) {
#pragma unroll
                    for (int kv = 1; kv >= 0; --kv) {           // V of iteration i, then K of i + lead
                        const int j = g.j0 + (kv ? i : i + lead);
                        if (j < g.j0 || j >= g.j1) continue;
                        if (2 * j >= base + 64) {               // (V of i - 1 may still lie in the window before)
                            base += 32;
                            cur = nxt;
                            nxt = base + 32 + lane < pages ? __ldg(tab + base + 32 + lane) : 0;
                        }
                        int z[2], y[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int pg = 2 * j + h, at = pg - base;
                            const int ph0 = __shfl_sync(0xffffffffu, cur, at & 31), ph1 = __shfl_sync(0xffffffffu, nxt, at & 31);
                            const int ph = at < 32 ? ph0 : ph1;
                            const bool bad = ph < 0 || ph >= p.kv.n_pages;
                            if (bad && lane == 0) raise(p.ctrl, MK_ERR_BAD_INPUT, 403);
                            z[h] = (bad ? 0 : ph) * p.hkv + g.head;
                            y[h] = bad ? -64 : min(max(g.kvlen - pg * 64, 0), 64) - 64;
                        }
                        const int s = n % SLOTS;
                        const uint32_t fb = FP8 ? rfull(s) : full(s), eb = FP8 ? rempty(s) : empty(s);
                        if (n >= SLOTS && !wait(eb, (n / SLOTS - 1) & 1)) { live = false; break; }
                        if (lane == 0) {
                            const CUtensorMap *map = kv ? &mapv : &mapk;
                            if (FP8) {
                                const uint32_t dst = s0 + C::RAWS + s * RAW_TILE;
                                bar_expect(fb, RAW_TILE);
                                tma3(dst, map, 0, y[0], z[0], fb);
                                tma3(dst + 8192, map, 0, y[1], z[1], fb);
                            } else {
                                const uint32_t dst = ring + s * TILE;
                                bar_expect(fb, TILE);
                                tma3(dst, map, 0, y[0], z[0], fb);
                                tma3(dst + HALF_TILE, map, 64, y[0], z[0], fb);
                                tma3(dst + 8192, map, 0, y[1], z[1], fb);
                                tma3(dst + HALF_TILE + 8192, map, 64, y[1], z[1], fb);
                            }
                        }
                        __syncwarp();
                        ++n;
                    }
                }
            }
            if (*wait.gone) {                                   // copies in flight end before the CTA does
                const Waiter drain{misc + 2, p.tries};
                for (int i = n > SLOTS ? n - SLOTS : 0; i < n; ++i) {
                    const int s = i % SLOTS;
                    drain(FP8 ? rfull(s) : full(s), (i / SLOTS) & 1);
                }
            }
        } else if (warp == 9) {
            // D fp32, A and B bf16 or f16, N 128, M 128; V is MN-major
            constexpr uint32_t ty = FP8 ? 0 : 1;
            constexpr uint32_t id_qk = (1u << 4) | (ty << 7) | (ty << 10) | (16u << 17) | (8u << 24), id_pv = id_qk | (1u << 16);
            const uint32_t el = elect_one();
            int slot = 0;                                       // next tile of the ring, in the loader's order
            uint32_t fph = 0;                                   // its phase
            uint32_t pq = 0, pp = 0;                            // phases of qfull, pfull (bit x)
            auto advance = [&]() {
                if (++slot == C::RING) {
                    slot = 0;
                    fph ^= 1;
                }
            };
            auto slot_wait = [&]() { return wait(full(slot), fph); };
            auto qk = [&](int x, int s, bool last) {
                mma8_ss(tm + x * 128, desc_k(qs + x * TILE), desc_k(ring + s * TILE), id_qk, el);
                mma_commit(sfull(x), el);
                if (last) mma_commit(qfree(x), el);
            };
            // O += P V, half the keys as soon as half of P is there
            auto pv = [&](int x, int s, bool acc) {
                bool r = wait(phalf(x), pp >> x & 1);
                fence_after();
                if (!r) return false;
                mma4_ts(tm + 256 + x * 128, tm + x * 128, desc_mn(ring + s * TILE), id_pv, el, acc);
                r = wait(pfull(x), pp >> x & 1);
                pp ^= 1u << x;
                fence_after();
                if (r) mma4_ts(tm + 256 + x * 128, tm + x * 128 + 32, desc_mn(ring + s * TILE) + 512, id_pv, el, 1);
                return r;
            };
            auto q_wait = [&](int x) {
                const bool r = wait(qfull(x), pq >> x & 1);
                pq ^= 1u << x;
                fence_after();
                return r;
            };
            bool ok = true;
            while (ok && w.next(g)) {
                if (dual_seg(g, tpt)) {
                    // tiles in the loader's order: K0 K1 | V0 K2 | V1 K3 | ...
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (!(ok = ok && slot_wait() && q_wait(x))) break;
                        qk(x, slot, g.j0 + x + 2 >= g.j1);
                        mma_commit(empty(slot), el);
                        advance();
                    }
                    for (int j = g.j0; ok && j < g.j1; ++j) {
                        const int x = (j - g.j0) & 1;
                        if (!(ok = slot_wait() && pv(x, slot, j > g.j0 + 1))) break;
                        if (j + 2 >= g.j1) mma_commit(ofull(x), el);
                        mma_commit(empty(slot), el);
                        advance();
                        if (j + 2 < g.j1) {
                            if (!(ok = slot_wait())) break;
                            qk(x, slot, j + 4 >= g.j1);
                            mma_commit(empty(slot), el);
                            advance();
                        }
                    }
                    continue;
                }
                const TileSeg ta = tile_of(g, 0, tpt, G), tb = tile_of(g, 1, tpt, G);
                // K of the first iteration
                ok = slot_wait();
                if (ok && g.j0 < ta.j1 && (ok = q_wait(0))) qk(0, slot, g.j0 + 1 == ta.j1);
                if (ok && g.j0 < tb.j1 && (ok = q_wait(1))) qk(1, slot, g.j0 + 1 == tb.j1);
                if (!ok) break;
                mma_commit(empty(slot), el);
                advance();
                for (int j = g.j0; j < g.j1; ++j) {
                    // V of iteration j, K of j + 1: per tile O += P V, then the next S
                    const bool more = j + 1 < g.j1;
                    const int sv = slot;
                    if (!(ok = slot_wait())) break;
                    advance();
                    if (more && !(ok = slot_wait())) break;
                    if (j < ta.j1) {
                        if (!(ok = pv(0, sv, j > g.j0))) break;
                        if (j + 1 == ta.j1) mma_commit(ofull(0), el);
                    }
                    if (j + 1 < ta.j1) qk(0, slot, j + 2 == ta.j1);
                    if (j < tb.j1) {
                        if (!(ok = pv(1, sv, j > g.j0))) break;
                        if (j + 1 == tb.j1) mma_commit(ofull(1), el);
                    }
                    mma_commit(empty(sv), el);
                    if (more) {
                        if (j + 1 < tb.j1) qk(1, slot, j + 2 == tb.j1);
                        mma_commit(empty(slot), el);
                        advance();
                    }
                }
            }
            if (*wait.gone) {                                   // MMAs in flight end before TMEM is freed
                const Waiter drain{misc + 2, p.tries};
                mma_commit(fin, el);
                drain(fin, 0);
            }
        } else {
            // warp 10 loads Q of tile A, warp 11 of tile B, as soon as the tile's last S of
            // the unit before is there: the load is done when that unit's output is.  A
            // box is the G heads of tpt tokens, which makes a tile's rows; tokens of
            // another stream behind the tile's only fill rows that nobody reads.
            const int X = warp - 10;
            const uint32_t half = G * tpt * 128;
            bool used = false, shared = false;
            uint32_t pf = 0, pd = 0, pr = 0, pl = 0;                // phases of qfree, adone, qraw; loads issued (parity)
            while (w.next(g)) {
                const TileSeg t = tile_of(g, X, tpt, G);
                if (t.j1 <= t.j0) continue;
                if (used && !wait(qfree(X), pf)) break;
                if (used) pf ^= 1;
                used = true;
                if (shared) {                                   // B's output has passed through the Q tiles
                    if (!wait(adone, pd)) break;
                    pd ^= 1;
                }
                shared = dual_seg(g, tpt) && g.j0 == 0 && g.j1 == g.nit;
                const uint32_t dst = qs + X * TILE, bar = FP8 ? qraw(X) : qfull(X);
                if (lane == 0) {
                    bar_expect(bar, 2 * half);
                    tma3(dst, &mapq, 0, g.head * G, g.row0 + t.tok0, bar);
                    tma3(dst + HALF_TILE, &mapq, 64, g.head * G, g.row0 + t.tok0, bar);
                }
                pl ^= 1;
                __syncwarp();
                if (FP8) {                                      // bf16 -> f16, the type of the widened codes
                    if (!wait(bar, pr)) break;
                    pr ^= 1;
                    bool over = false;
                    unsigned char *tile = sm + C::Q + X * TILE;
#pragma unroll 1
                    for (int h = 0; h < 2; ++h)                 // rows of a half are 128 bytes; 4 x 512 bytes at a time
                        for (int i = lane * 16; i < t.rows * 128; i += 2048) {
                            uint4 v[4];
#pragma unroll
                            for (int n = 0; n < 4; ++n)
                                if (i + 512 * n < t.rows * 128) v[n] = *reinterpret_cast<const uint4 *>(tile + h * HALF_TILE + i + 512 * n);
#pragma unroll
                            for (int n = 0; n < 4; ++n) {
                                if (i + 512 * n >= t.rows * 128) break;
                                uint32_t *u = reinterpret_cast<uint32_t *>(&v[n]);
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const float lo = __uint_as_float(u[k] << 16), hi = __uint_as_float(u[k] & 0xffff0000u);
                                    over |= fabsf(lo) > 65504.f || fabsf(hi) > 65504.f;  // (NaN stays its row's)
                                    u[k] = pack2<true>(lo, hi);
                                }
                                *reinterpret_cast<uint4 *>(tile + h * HALF_TILE + i + 512 * n) = v[n];
                            }
                        }
                    if (over) raise(p.ctrl, MK_ERR_RANGE, 404);
                    fence_async();
                    __syncwarp();
                    if (lane == 0) bar_arrive(qfull(X));
                }
            }
            if (used && *wait.gone) {                           // a copy in flight ends before the CTA does
                const Waiter drain{misc + 2, p.tries};
                drain(FP8 ? qraw(X) : qfull(X), pl ^ 1);
            }
        }
    } else if (FP8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
        // codes to f16: a thread takes 16 codes of a row.  Lanes of the right half
        // of a row write their second 16 bytes first, so that 8 lanes of a row
        // cover all banks.  (Measured against it, at chunks of 1, 517, 1300 and 2048
        // tokens over FP8 caches, 221 us: two warps a tile, the other two the next,
        // 244; K not widened but multiplied as codes by two E4M3 parts of q, 295.)
        const int ct = tid % 128, seg = ct % 8;
        int n = 0;
        bool live = true;
        while (live && w.next(g)) {
            for (int i = 0; i < 2 * (g.j1 - g.j0); ++i, ++n) {
                const int rs = n % RAW, ds = n % C::RING;
                if (!wait(rfull(rs), (n / RAW) & 1) || (n >= C::RING && !wait(empty(ds), (n / C::RING - 1) & 1))) {
                    live = false;
                    break;
                }
                const unsigned char *src = sm + C::RAWS + rs * RAW_TILE + ct / 8 * 128 + seg * 16;
                const uint32_t dst = ring + ds * TILE + seg / 4 * HALF_TILE + ct / 8 * 128;
                const int c0 = seg % 4 * 2, sw = seg / 4;
                const uint32_t o0 = ((c0 + sw) ^ ct / 8 % 8) << 4, o1 = ((c0 + 1 - sw) ^ ct / 8 % 8) << 4;
                // A short loop: unrolled, this code and the softmax's evict one another
                // from the instruction cache, and both run several times slower.
#pragma unroll 1
                for (int h = 0; h < 8; h += 4) {
                    uint4 v[4];                                 // reads in flight before the first write
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const uint4 *>(src + (h + k) * 2048);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                        uint32_t f[8];
#pragma unroll
                        for (int a = 0; a < 4; ++a)
                            asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
                                : "=r"(f[2 * a]), "=r"(f[2 * a + 1]) : "r"(u[a]));
                        const uint4 lo = make_uint4(f[0], f[1], f[2], f[3]), hi = make_uint4(f[4], f[5], f[6], f[7]);
                        st_shared16(dst + (h + k) * 2048 + o0, sw ? hi : lo);
                        st_shared16(dst + (h + k) * 2048 + o1, sw ? lo : hi);
                    }
                }
                fence_async();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(rempty(rs));
                    bar_arrive(full(ds));
                }
            }
        }
    }
    __syncwarp();
    if (*wait.gone && lane == 0) raise(p.ctrl, MK_ERR_TIMEOUT, 405);
    fence_before();
    __syncthreads();
    if (warp == 9) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
    }
}

template <bool FP8>
cudaError_t launch(const MmaP &p, const CUtensorMap *maps, int grid, cudaStream_t s) {
    attn_mma_kernel<FP8><<<grid, Cfg<FP8>::THREADS, Cfg<FP8>::TOTAL + 1024, s>>>(p, maps[0], maps[1], maps[2]);
    return cudaGetLastError();
}
template <bool FP8>
cudaError_t setup() {
    return cudaFuncSetAttribute(attn_mma_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<FP8>::TOTAL + 1024);
}
}  // namespace

cudaError_t mk_attn_mma_setup() {
    cudaError_t e = setup<false>();
    return e != cudaSuccess ? e : setup<true>();
}

cudaError_t mk_attn_mma_launch(const ChunkP &c, const KvP &kv, const AttnWs &ws, Ctrl *ctrl, const CUtensorMap *maps, void *out,
                               int hq, int hkv, int grid, long long timeout_ns, cudaStream_t s) {
    const MmaP p{c, kv, ws, ctrl, static_cast<__nv_bfloat16 *>(out), hq, hkv, kv.dtype == MK_DT_FP8E4M3 ? Cfg<true>::MIN_COST : Cfg<false>::MIN_COST,
                 hq / hkv, 128 * hkv / hq, reinterpret_cast<uintptr_t>(out) % 32 == 0, 65536u / (hq / hkv) + 1,
                 (uint32_t)(timeout_ns / 250 < 0x7fffffff ? timeout_ns / 250 : 0x7fffffff)};
    return kv.dtype == MK_DT_FP8E4M3 ? launch<true>(p, maps, grid, s) : launch<false>(p, maps, grid, s);
}
