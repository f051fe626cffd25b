// Writing a chunk's keys and values into the paged cache (RoPE, rounding to the
// cache type) and reading cached entries back.
//
// Both move every byte once and are bound by HBM; small calls by one chain of
// dependent loads (row -> stream -> page -> entry), large ones first by the
// instructions of that lookup.  So a warp looks up 32 rows at once, a lane per
// row: a binary search over the offsets, which 32 streams' worth of lanes hold
// (five shuffles; more streams search in memory).
//
// Measured (32/4 heads of 128, one GB300; of the copy bandwidth): 37319 rows
// appended to FP8 caches in 126 us (5.8 TB/s, 85 %), 2047 rows to bf16 ones in 13 us (3.1
// TB/s), 6 rows in 6 us; 39106 rows of FP8 entries read
// back in 29 us (4.2 TB/s; the kernel alone 23 us), 129 rows in 5 us.
#include "mk_chunk.cuh"

namespace {
using namespace mkc;

struct RowAt {
    int pos;    // position in the sequence; -1: row without a stream (padding) or bad input
    int phys;   // physical page
};

// stream i's part of the chunk's description, as the attention's plan checks it
__device__ __forceinline__ bool good_stream(const ChunkP &c, int i, int o0, int o1, int ctx) {
    return (i > 0 || o0 == 0) && o0 >= 0 && o1 >= o0 && o1 <= c.n_rows && ctx >= 0 && (long long)ctx + (o1 - o0) <= c.max_pos;
}

// The lanes of a warp look up packed rows r (of their own; behind the rows:
// none).  A description that is bad for any stream leaves no row (`good`: of more
// than 32 streams, which the block has checked; fewer are checked here).  Memory
// safety rests on the checks of a row's own stream: nothing is read or written
// for a row that fails one.
__device__ RowAt row_at(const ChunkP &c, const KvP &kv, Ctrl *ctrl, long long r, bool good) {
    const int lane = threadIdx.x % 32, S = c.S;
    const int last = __ldg(c.off + S);
    int s = 0, o0 = 0, o1 = 0, ctx = 0;  // the last stream that begins at r or before
    if (S <= 32) {
        const int o = lane < S ? __ldg(c.off + lane) : 0x7fffffff, cx = lane < S ? __ldg(c.ctx + lane) : 0;
        const int next = __shfl_down_sync(0xffffffffu, o, 1);
        good = __all_sync(0xffffffffu, lane >= S || good_stream(c, lane, o, lane + 1 < S ? next : last, cx));
#pragma unroll
        for (int k = 16; k; k >>= 1) {
            const int v = __shfl_sync(0xffffffffu, o, s + k);
            if (v <= r) s += k;
        }
        o0 = __shfl_sync(0xffffffffu, o, s);
        o1 = __shfl_sync(0xffffffffu, o, (s + 1) & 31);
        if (s + 1 >= S) o1 = last;
        ctx = __shfl_sync(0xffffffffu, cx, s);
    } else {
        int hi = S;
        while (hi - s > 1) {
            const int mid = (s + hi) / 2;
            if (__ldg(c.off + mid) <= r) s = mid; else hi = mid;
        }
        o0 = __ldg(c.off + s);
        o1 = __ldg(c.off + s + 1);
        ctx = __ldg(c.ctx + s);
    }
    RowAt a{-1, -1};
    if (r >= c.n_rows || (good && r >= last)) return a;  // none, or behind the last sequence
    bool bad = !good || !good_stream(c, s, o0, o1, ctx) || o0 > r || o1 <= r;
    if (!bad) {
        const int pos = ctx + (int)(r - o0), ph = __ldg(kv.table + (long long)s * c.max_pages + pos / 64);
        bad = ph < 0 || ph >= kv.n_pages;
        if (!bad) a = RowAt{pos, ph};
    }
    if (bad) raise(ctrl, MK_ERR_BAD_INPUT, 401);
    return a;
}

// 8 values to the cache type: float32, bf16 (nearest even), or the E4M3 code of
// value / scale (division in fp32, nearest even, saturating at 448), as the
// verify step stores its own entries
__device__ __forceinline__ void store8(float *p, const float *v, float) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *v, float) {
    Vec<__nv_bfloat16, 8> o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = __float2bfloat16_rn(v[i]);
    *reinterpret_cast<Vec<__nv_bfloat16, 8> *>(p) = o;
}
__device__ __forceinline__ void store8(__nv_fp8_e4m3 *p, const float *v, float scale) {
    Vec<unsigned char, 8> o;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o.v[i] = (unsigned char)__nv_cvt_float_to_fp8(v[i] / scale, __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<Vec<unsigned char, 8> *>(p) = o;
}
// A block of 8 warps takes `rb` rows: its first warp looks them up, then 8 / rb
// warps share a row, or each takes rb / 8 rows.
struct Share {
    int row, rows, part, parts;  // first row of this warp, rows between its rows, its share of a row
};
__device__ __forceinline__ Share share_of(int rb) {
    const int wid = threadIdx.x / 32, parts = rb < 8 ? 8 / rb : 1;
    return Share{wid / parts, 8 / parts, wid % parts, parts};
}

// The block's rows into `at`; false after an earlier error.  A single row is
// looked up by every warp for itself: no barrier in the shortest calls.
__device__ __forceinline__ bool rows_of(const ChunkP &c, const KvP &kv, Ctrl *ctrl, long long r0, int rb, RowAt (*at)[32]) {
    const int lane = threadIdx.x % 32, wid = threadIdx.x / 32;
    bool good = true;
    if (c.S > 32) {
        bool bad = false;
        for (int i = threadIdx.x; i < c.S; i += 256)
            bad |= !good_stream(c, i, __ldg(c.off + i), __ldg(c.off + i + 1), __ldg(c.ctx + i));
        good = !__syncthreads_or(bad);
    }
    if (rb == 1) {
        const RowAt a = row_at(c, kv, ctrl, lane < 1 ? r0 : c.n_rows, good);
        at[wid][lane] = a;
        __syncwarp();
        return !__any_sync(0xffffffffu, aborted(ctrl));
    }
    if (wid == 0) {
        const RowAt a = row_at(c, kv, ctrl, lane < rb ? r0 + lane : c.n_rows, good);
        at[0][lane] = a;
    }
    return !__syncthreads_or(threadIdx.x == 0 && aborted(ctrl));
}

// heads that the lanes of a warp hold at a time: a lane has 8 rotation pairs
// (i, i + d/2) of one
template <int D>
constexpr int HEADS = 32 / (D / 16);

template <int D, class Act, class KV>
__global__ void __launch_bounds__(256) append_kernel(ChunkP c, KvP kv, Ctrl *ctrl, const float2 *rope, const Act *qkv,
                                                     long long ld, Act *q_out, int hq, int hkv, int rb) {
    constexpr int TPR = D / 16, H = HEADS<D>;
    __shared__ RowAt at[8][32];
    const int lane = threadIdx.x % 32, x = lane % TPR, nh = hq + 2 * hkv;
    const long long r0 = (long long)blockIdx.x * rb;
    const Share sh = share_of(rb);
    const int step = sh.parts * H, h0 = sh.part * H + lane / TPR;
    if (!rows_of(c, kv, ctrl, r0, rb, at)) return;
    for (int row = sh.row; row < rb; row += sh.rows) {
        const RowAt a = at[rb == 1 ? threadIdx.x / 32 : 0][row];
        const long long r = r0 + row;
        if (a.pos < 0) continue;
        const Act *src = qkv + r * ld + x * 8;
        float cs[16];
        {
            const float4 *rp = reinterpret_cast<const float4 *>(rope + (long long)a.pos * (D / 2) + x * 8);
#pragma unroll
            for (int i = 0; i < 4; ++i) reinterpret_cast<float4 *>(cs)[i] = __ldg(rp + i);
        }
        const long long slot = ((long long)a.phys * hkv) * 64 + (a.pos % 64);
        for (int h = h0; h < nh; h += step) {
            const Vec<Act, 8> v1 = *reinterpret_cast<const Vec<Act, 8> *>(src + h * D);
            const Vec<Act, 8> v2 = *reinterpret_cast<const Vec<Act, 8> *>(src + h * D + D / 2);
            float y1[8], y2[8];
            const bool turn = h < hq + hkv;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                y1[k] = to_f(v1.v[k]);
                y2[k] = to_f(v2.v[k]);
            }
            if (turn) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float a1 = y1[k], a2 = y2[k];
                    y1[k] = a1 * cs[2 * k] - a2 * cs[2 * k + 1];
                    y2[k] = a2 * cs[2 * k] + a1 * cs[2 * k + 1];
                }
            }
            if (h < hq) {
                if (q_out) {
                    Act *o = q_out + (r * hq + h) * D + x * 8;
                    store8(o, y1, 1.f);
                    store8(o + D / 2, y2, 1.f);
                }
            } else {
                const int hh = h - (turn ? hq : hq + hkv);
                KV *o = reinterpret_cast<KV *>(turn ? kv.k : kv.v) + (slot + (long long)hh * 64) * D + x * 8;
                const float sc = turn ? kv.ks : kv.vs;
                store8(o, y1, sc);
                store8(o + D / 2, y2, sc);
            }
        }
    }
}

// N stored entries as values
template <int N>
__device__ __forceinline__ void values(const Vec<__nv_fp8_e4m3, N> &v, float *o, float sc) {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(v.v[k].__x | v.v[k + 1].__x << 8), __NV_E4M3)));
        o[k] = f.x * sc;
        o[k + 1] = f.y * sc;
    }
}
template <int N, class T>
__device__ __forceinline__ void values(const Vec<T, N> &v, float *o, float) {
#pragma unroll
    for (int k = 0; k < N; ++k) o[k] = to_f(v.v[k]);
}

// Entries back as values: code * scale, rounded once to the activation type.  A
// lane writes 16 bytes at a time.
template <int D, class Act, class KV>
__global__ void __launch_bounds__(256, 6) read_kernel(ChunkP c, KvP kv, Ctrl *ctrl, Act *k_out, Act *v_out, int hkv, int rb) {
    constexpr int N = 16 / sizeof(Act), P = D / N;  // elements of a piece, pieces of a head
    __shared__ RowAt at[8][32];
    const int lane = threadIdx.x % 32;
    const long long r0 = (long long)blockIdx.x * rb;
    if (!rows_of(c, kv, ctrl, r0, rb, at)) return;
    const Share sh = share_of(rb);
    const int per = hkv * P, step = 32 * sh.parts;
    for (int row = sh.row; row < rb; row += sh.rows) {
        const RowAt a = at[rb == 1 ? threadIdx.x / 32 : 0][row];
        if (a.pos < 0) continue;
        const long long from = ((long long)a.phys * hkv * 64 + a.pos % 64) * D, to = (r0 + row) * hkv * D;
        for (int p0 = sh.part * 32 + lane; p0 < per; p0 += step) {
            const long long o = from + (long long)(p0 / P) * 64 * D + p0 % P * N;
            const Vec<KV, N> k = *reinterpret_cast<const Vec<KV, N> *>(reinterpret_cast<const KV *>(kv.k) + o);
            const Vec<KV, N> v = *reinterpret_cast<const Vec<KV, N> *>(reinterpret_cast<const KV *>(kv.v) + o);
            float f[N];
            Vec<Act, N> y;
            values(k, f, kv.ks);
#pragma unroll
            for (int i = 0; i < N; ++i) y.v[i] = Act(f[i]);
            *reinterpret_cast<Vec<Act, N> *>(k_out + to + p0 * N) = y;
            values(v, f, kv.vs);
#pragma unroll
            for (int i = 0; i < N; ++i) y.v[i] = Act(f[i]);
            *reinterpret_cast<Vec<Act, N> *>(v_out + to + p0 * N) = y;
        }
    }
}

// rows of a block, a power of two: as many as leave three blocks for each of
// 152 SMs, up to `most`.  Measured at 37319 rows of 32/4 heads: 128 us with 16
// rows, 139 with 4; at 2047 rows: 14.3 us with 4, 22.5 with 16.
int rows_per_block(int n_rows, int most) {
    int rb = 1;
    while (rb < most && n_rows >= 2 * rb * 456) rb *= 2;
    return rb;
}

template <int D, class Act, class KV>
cudaError_t append(const ChunkP &c, const KvP &kv, Ctrl *ctrl, const float2 *rope, const void *qkv, long long ld,
                   void *q_out, int hq, int hkv, cudaStream_t s) {
    const int rb = rows_per_block(c.n_rows, 16);
    append_kernel<D, Act, KV><<<(c.n_rows + rb - 1) / rb, 256, 0, s>>>(
        c, kv, ctrl, rope, static_cast<const Act *>(qkv), ld, static_cast<Act *>(q_out), hq, hkv, rb);
    return cudaGetLastError();
}
template <int D, class Act, class KV>
cudaError_t read(const ChunkP &c, const KvP &kv, Ctrl *ctrl, void *k_out, void *v_out, int hkv, cudaStream_t s) {
    const int rb = rows_per_block(c.n_rows, 32);
    read_kernel<D, Act, KV><<<(c.n_rows + rb - 1) / rb, 256, 0, s>>>(c, kv, ctrl, static_cast<Act *>(k_out),
                                                                     static_cast<Act *>(v_out), hkv, rb);
    return cudaGetLastError();
}
}  // namespace

// activations: float32 with head dim 64 (all-float32 models), bf16 with 128
cudaError_t mk_append_launch(const ChunkP &c, const KvP &kv, Ctrl *ctrl, const float2 *rope, const void *qkv,
                             long long ld, void *q_out, int hq, int hkv, bool f32, cudaStream_t s) {
    if (f32)
        return kv.dtype == MK_DT_F32 ? append<64, float, float>(c, kv, ctrl, rope, qkv, ld, q_out, hq, hkv, s)
                                     : append<64, float, __nv_bfloat16>(c, kv, ctrl, rope, qkv, ld, q_out, hq, hkv, s);
    return kv.dtype == MK_DT_BF16
               ? append<128, __nv_bfloat16, __nv_bfloat16>(c, kv, ctrl, rope, qkv, ld, q_out, hq, hkv, s)
               : append<128, __nv_bfloat16, __nv_fp8_e4m3>(c, kv, ctrl, rope, qkv, ld, q_out, hq, hkv, s);
}
cudaError_t mk_read_launch(const ChunkP &c, const KvP &kv, Ctrl *ctrl, void *k_out, void *v_out, int hkv, bool f32,
                           cudaStream_t s) {
    if (f32)
        return kv.dtype == MK_DT_F32 ? read<64, float, float>(c, kv, ctrl, k_out, v_out, hkv, s)
                                     : read<64, float, __nv_bfloat16>(c, kv, ctrl, k_out, v_out, hkv, s);
    return kv.dtype == MK_DT_BF16 ? read<128, __nv_bfloat16, __nv_bfloat16>(c, kv, ctrl, k_out, v_out, hkv, s)
                                  : read<128, __nv_bfloat16, __nv_fp8_e4m3>(c, kv, ctrl, k_out, v_out, hkv, s);
}
