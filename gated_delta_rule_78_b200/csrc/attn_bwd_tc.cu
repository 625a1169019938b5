// Causal attention backward on the tensor cores (bf16).
//
//   p_ij = 2^(c s'_ij - lse_i log2 e),  c = scale log2 e,  s' = q k^T over the visible pairs
//   ds_ij = p_ij (do_i . v_j - delta_i),  delta_i = do_i . o_i
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
//
// Two kernels form the scores again, so that every sum stays inside one block and no result depends on
// the order of blocks: one block to 128 packed query rows walks over the keys and keeps dq in TMEM
// (3 products a tile pair); one block to 128 keys of a key head walks over the packed query rows of
// all of its query heads and keeps dk and dv in TMEM (4 products a tile pair).  One kernel with dq
// accumulated in memory would need 5 products a pair instead of 7, and fp32 atomics.  p and ds are
// rounded to bf16 for their products (up to 2^-8 of each term), everything else is fp32.
//
// o comes rounded to bf16, and what that does to delta is a fixed share of p in every ds of a row, which
// does not average out; most in a sequence's first rows, whose few weights are large.  Where all keys of
// a tile of queries are one tile, the dq kernel takes delta from the weights themselves, sum_j p_ij (do_i .
// v_j), and leaves it for the keys' kernel, which runs after it.  Relative errors of dq and dk of random
// sequences of 1 to 3 tokens: 2.8e-3 and 3.1e-3 -> 2.3e-3 and 2.5e-3, of 1500: 2.5e-3 -> 2.4e-3 (their own
// rounding alone: 1.7e-3).  (Corrected in every row by its sum of ds, which should be 0: dk is no better,
// and dq takes 303 instead of 266 us at 4 x 4096, window 2048.)
//
// Roles, 384 threads: warps 0-3 and 4-7 form p and ds of the tile's left and right 64 columns (a thread to
// a row), warp 8 issues the products, warp 9 the TMA loads, warp 10 (keys' kernel) brings the rows'
// lse and delta.  bf16 p and ds overwrite the columns of the scores that their own warps have read.
//
// A block stays on its SM and takes one tile after another, heavy ones first: while the warps finish a
// tile and write its gradients, the loads and first products of the next already run.  A block to a
// tile spent 12 of its 43 thousand cycles starting and ending (4 x 4096, window 2048).  Barriers and rings
// go on from tile to tile; every role walks through the same tiles and counts for itself.
//
// 4 x 4096, 16 heads, D = 128, window 2048: dq 268 us, dk and dv 370 us, 722 GFLOP of products in all, 1130 TFLOP/s.
#include <limits.h>

#include "attn_tc.cuh"

namespace gdn2 {
namespace {

using namespace attn;
using namespace tc;

struct BwdMaps {
    CUtensorMap q, k, v, d_o;
};
struct BwdParams {
    SeqBatch b;
    int H, Hkv, G, TQ, window, qtiles, ktiles;  // tiles of queries and of keys, over all sequences
    float scale;
    const float *lse;
    float *delta;  // [rows, H]: do . o, in a sequence's first rows then the dq kernel's
    __nv_bfloat16 *dq, *dk, *dv;
    int *status;
};

constexpr int kThreads = 384;
// Of 16 pairs of weights, those formed on the FMA pipe: the special-function unit's 16 values a clock are
// half of a tile's time, and the warps have nothing else to do meanwhile (dk/dv 375 -> 361 us, dq 271 ->
// 268 us at 4 x 4096; with 7 of 16 360 and 274; the forward's softmax, which waits for its products, gains nothing).
constexpr int kFma = 5;

// one tile by TMA: its column blocks at dst
template <int NB>
__device__ __forceinline__ void load_tile(char *dst, const CUtensorMap *map, int head, int row, uint64_t *bar)
{
#pragma unroll
    for (int b = 0; b < NB; ++b) tma_load_3d(dst + b * kBoxBytes, map, 64 * b, head, row, bar);
}

// 64 fp32 columns of this thread's row
__device__ __forceinline__ void ld64(uint32_t t, float (&s)[64])
{
    tmem_ld32(t, reinterpret_cast<uint32_t(&)[32]>(s[0]));
    tmem_ld32(t + 32, reinterpret_cast<uint32_t(&)[32]>(s[32]));
    tmem_wait_ld();
}
// 2^x of a pair, number i of a row's 32, in place; every one by ex2 where exact zeros (2^-inf) are wanted
__device__ __forceinline__ void weights(uint64_t x, int i, bool exact, float &a, float &b)
{
    if (!exact && i % 16 * kFma / 16 != (i % 16 + 1) * kFma / 16) {  // spread evenly
        ex2_fma(x, a, b);
    } else {
        unpair(x, a, b);
        a = ex2(a);
        b = ex2(b);
    }
}
// this thread's row of 64 values as bf16 into 32 columns
__device__ __forceinline__ void st64(uint32_t t, const float (&s)[64])
{
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = pack_bf16x2(s[2 * i], s[2 * i + 1]);
    tmem_st32(t, w);
    tmem_wait_st();
}
// f * (this thread's row of TMEM columns [0, n)) as bf16 at dst
template <int n> __device__ __forceinline__ void store_row(uint32_t t, float f, __nv_bfloat16 *dst, bool live)
{
#pragma unroll
    for (int q = 0; q < n / 32; ++q) {
        uint32_t w[32];
        tmem_ld32(t + 32 * q, w);
        tmem_wait_ld();
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < 32; i += 16) {
            uint32_t v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = pack_bf16x2(f * __uint_as_float(w[i + 2 * e]), f * __uint_as_float(w[i + 2 * e + 1]));
            store32(dst + 32 * q + i, v);
        }
    }
}
// ------------------------------------------------------------------ dq
// TMEM: S of even and odd key tiles, dP = dO V^T, dQ.  The tensor core forms S two tiles ahead and dP one
// ahead of the warps; K waits in shared memory from S to dQ, three stages of it.
template <int D> struct DqCfg {
    static constexpr int NB = D / 64, TILE = NB * kBoxBytes;
    static constexpr int KS = D == 128 ? 3 : 4, VS = D == 128 ? 2 : 4;
    static constexpr int SMEM = (2 + KS + VS) * TILE + 1024;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_dq_tc_kernel(const __grid_constant__ BwdMaps maps,
                                                                 const __grid_constant__ BwdParams p)
{
    using C = DqCfg<D>;
    constexpr int kTmP = 256, kTmQ = 384;
    extern __shared__ char raw[];
    char *sm = reinterpret_cast<char *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    char *sq = sm, *so = sq + C::TILE, *sk = so + C::TILE, *sv = sk + C::KS * C::TILE;
    __shared__ __align__(8) uint64_t q_full, q_empty, k_full[C::KS], k_empty[C::KS], v_full[C::VS], v_empty[C::VS], s_full[2],
        p_full, ds_ready, sum_full, done, bar_drain;
    __shared__ float s_sum[2][kBM];  // by half of the columns, and row
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    if (blockIdx.x == 0 && warp == 0) report_bad_seqlens(p.b, p.status);
    if (tid == 0) {
        s_abort = 0;
        mbar_init(&q_full, 1);
        mbar_init(&q_empty, 1);
        for (int i = 0; i < C::KS; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < C::VS; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        mbar_init(&p_full, 1);
        mbar_init(&ds_ready, 8);
        mbar_init(&sum_full, 8);
        mbar_init(&done, 1);
        mbar_init(&bar_drain, 1);
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(s_tmem);

    // The block's work, walked through by every role: its queries' first token t0 and count nt, and its n
    // key tiles from jb on.  `base` counts the key tiles before it, `num` the tiles of queries.
    struct Work {
        int hk, bos, len, t0, nt, jb, n;
    };
    auto find = [&](int w, Work &x) {
        TileRef r;
        if (!block_tile(p.b, w, p.qtiles, p.Hkv, p.window, p.TQ, false, r, x.hk)) return false;
        x.bos = r.sp.bos;
        x.len = r.sp.len;
        x.t0 = r.tile * p.TQ;
        x.nt = min(p.TQ, x.len - x.t0);
        x.jb = p.window == 0 || x.t0 < p.window ? 0 : (x.t0 - p.window + 1) / kBN;
        x.n = (x.t0 + x.nt - 1) / kBN + 1 - x.jb;
        return true;
    };
    const int works = p.qtiles * p.Hkv;
    int base = 0, num = 0;
    Work x;
    bool ok = true;

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int half = warp >> 2, row = tid & 127, tok = row / p.G;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const float c = p.scale * kLog2e;
        const uint64_t c2 = pair(c, c);
        uint32_t ones = 0;  // tiles of queries with one tile of keys, so far
        for (int i = 0, w; ok && (w = work_at(i, works)) >= 0; ++i) {
            if (w >= works || !find(w, x)) continue;
            const int pos = x.t0 + tok;
            const bool live = row < p.TQ * p.G && tok < x.nt;
            const size_t at = (size_t)(x.bos + pos) * p.H + x.hk * p.G + (row - tok * p.G);
            const float lse = live ? -p.lse[at] * kLog2e : 0.f, delta = live ? -p.delta[at] : 0.f;
            const uint64_t l2 = pair(lse, lse);
            uint64_t d2 = pair(delta, delta);
            for (int it = 0; it < x.n; ++it) {
                const int k = base + it;
                if (!(ok = wait_warp(&s_full[k & 1], (k >> 1) & 1, &s_abort, p.status))) break;
                tc_fence_after();
                float s[64], d[64];
                const uint32_t ts = tmem + 128 * (k & 1) + 64 * half + lanes;
                ld64(ts, s);
                const int k0 = (x.jb + it) * kBN;
                const bool edge = k0 + kBN - 1 > x.t0 || (p.window && x.t0 + x.nt - 1 - k0 >= p.window);
                const int most = pos - k0 - 64 * half, least = p.window ? most - p.window + 1 : 0;
                if (edge) {
#pragma unroll
                    for (int i = 0; i < 64; ++i) s[i] = i <= most && i >= least ? s[i] : -INFINITY;
                }
                if (edge) {
#pragma unroll
                    for (int i = 0; i < 64; i += 2) weights(fma2(pair(s[i], s[i + 1]), c2, l2), i / 2, true, s[i], s[i + 1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 64; i += 2) weights(fma2(pair(s[i], s[i + 1]), c2, l2), i / 2, false, s[i], s[i + 1]);
                }
                if (!(ok = wait_warp(&p_full, k & 1, &s_abort, p.status))) break;
                tc_fence_after();
                ld64(tmem + kTmP + 64 * half + lanes, d);
                if (edge) {  // values of masked keys may belong to another sequence: not 0 * (what they are)
#pragma unroll
                    for (int i = 0; i < 64; ++i) d[i] = i <= most && i >= least ? d[i] : 0.f;
                }
                if (x.n == 1) {  // delta from the row's weights: the halves' sums, by way of shared memory
                    uint64_t a2 = 0, b2 = 0;
#pragma unroll
                    for (int i = 0; i < 64; i += 4) {
                        a2 = fma2(pair(s[i], s[i + 1]), pair(d[i], d[i + 1]), a2);
                        b2 = fma2(pair(s[i + 2], s[i + 3]), pair(d[i + 2], d[i + 3]), b2);
                    }
                    float a, b;
                    unpair(add2(a2, b2), a, b);
                    s_sum[half][row] = a + b;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sum_full);
                    if (!(ok = wait_warp(&sum_full, ones & 1, &s_abort, p.status))) break;
                    // (written again after the next tile's s_full, which follows all warps' ds)
                    const float sum = a + b + s_sum[half ^ 1][row];
                    d2 = pair(-sum, -sum);
                    if (live && half == 0) p.delta[at] = sum;
                    ++ones;
                }
#pragma unroll
                for (int i = 0; i < 64; i += 2)
                    unpair(mul2(pair(s[i], s[i + 1]), add2(pair(d[i], d[i + 1]), d2)), s[i], s[i + 1]);
                st64(ts, s);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ds_ready);
            }
            if (!(ok = ok && wait_warp(&done, num & 1, &s_abort, p.status))) break;
            tc_fence_after();
            store_row<D / 2>(tmem + kTmQ + D / 2 * half + lanes, p.scale, p.dq + at * D + D / 2 * half, live);
            tc_fence_before();  // the next tile's first product comes after its ds of all warps
            base += x.n;
            ++num;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const uint32_t bq = smem_u32(sq), bo = smem_u32(so), bk = smem_u32(sk), bv = smem_u32(sv);
        constexpr uint32_t kS = idesc_bf16(128, kBN, 0, 0), kG = idesc_bf16(128, D, 0, 1);
        if (warp == 8) {
            const uint32_t leader = elect();
            auto scores = [&](int it) {
                const int k = base + it, st = k % C::KS;
                if (!wait_warp(&k_full[st], (k / C::KS) & 1, &s_abort, p.status)) return false;
                // keys past the sequence are another's: their ds is 0, but 0 * NaN is not
                if ((x.jb + it + 1) * kBN > x.len) zero_rows<C::NB>(sk + st * C::TILE, x.len - (x.jb + it) * kBN);
                tc_fence_after();
                mma_kk<D / 16>(leader, tmem + 128 * (k & 1), bq, bk + st * C::TILE, kS);
                commit(leader, &s_full[k & 1]);
                return true;
            };
            auto products = [&](int it) {
                const int k = base + it, st = k % C::VS;
                if (!wait_warp(&v_full[st], (k / C::VS) & 1, &s_abort, p.status)) return false;
                tc_fence_after();
                mma_kk<D / 16>(leader, tmem + kTmP, bo, bv + st * C::TILE, kS);
                commit(leader, &p_full);
                commit(leader, &v_empty[st]);
                if (it + 1 == x.n) commit(leader, &q_empty);  // its scores came before
                return true;
            };
            for (int i = 0, w; ok && (w = work_at(i, works)) >= 0; ++i) {
                if (w >= works || !find(w, x)) continue;
                if (!(ok = wait_warp(&q_full, num & 1, &s_abort, p.status))) break;
                ok = scores(0) && (x.n < 2 || scores(1)) && products(0);
                for (int it = 0; ok && it < x.n; ++it) {
                    const int k = base + it;
                    if (!(ok = wait_warp(&ds_ready, k & 1, &s_abort, p.status))) break;
                    tc_fence_after();
                    if (it + 1 < x.n && !(ok = products(it + 1))) break;  // what the warps wait for first
                    mma_tn<4>(leader, tmem + kTmQ, tmem + 128 * (k & 1), bk + (k % C::KS) * C::TILE, 0, kG, it > 0);
                    mma_tn<4>(leader, tmem + kTmQ, tmem + 128 * (k & 1) + 64, bk + (k % C::KS) * C::TILE, 64, kG, 1);
                    commit(leader, &k_empty[k % C::KS]);
                    if (it + 1 == x.n) commit(leader, &done);
                    if (it + 2 < x.n) ok = scores(it + 2);
                }
                base += x.n;
                ++num;
            }
            if (s_abort) drain(leader, &bar_drain);
        } else if (warp == 9) {
            int nq = 0, nk = 0, nv = 0;  // loads issued, by lane 0
            for (int i = 0, w; ok && (w = work_at(i, works)) >= 0; ++i) {
                if (w >= works || !find(w, x)) continue;
                if (lane == 0 && (nq == 0 || (ok = wait(&q_empty, (nq - 1) & 1, &s_abort, p.status)))) {
                    mbar_expect_tx(&q_full, 2 * C::NB * 128 * p.G * p.TQ);
                    load_tile<C::NB>(sq, &maps.q, x.hk * p.G, x.bos + x.t0, &q_full);
                    load_tile<C::NB>(so, &maps.d_o, x.hk * p.G, x.bos + x.t0, &q_full);
                    ++nq;
                    for (int it = 0; it < x.n; ++it) {
                        const int a = nk % C::KS, b = nv % C::VS, row = x.bos + (x.jb + it) * kBN;
                        if (nk >= C::KS && !(ok = wait(&k_empty[a], ((nk / C::KS) & 1) ^ 1, &s_abort, p.status))) break;
                        mbar_expect_tx(&k_full[a], C::TILE);
                        load_tile<C::NB>(sk + a * C::TILE, &maps.k, x.hk, row, &k_full[a]);
                        ++nk;
                        if (nv >= C::VS && !(ok = wait(&v_empty[b], ((nv / C::VS) & 1) ^ 1, &s_abort, p.status))) break;
                        mbar_expect_tx(&v_full[b], C::TILE);
                        load_tile<C::NB>(sv + b * C::TILE, &maps.v, x.hk, row, &v_full[b]);
                        ++nv;
                    }
                }
                ok = __shfl_sync(0xffffffffu, (int)ok, 0);
            }
            if (s_abort && lane == 0) {
                if (nq) mbar_wait(&q_full, (nq - 1) & 1, 1000000000ull);
                drain_ring(k_full, nk, C::KS);
                drain_ring(v_full, nv, C::VS);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ dk, dv
// Everything transposed: rows are keys, columns packed query rows.  TMEM: S^T, dP^T = V dO^T, dV, dK.
// dV += P^T dO and the next S^T run while the warps form dS^T; dK += dS^T Q and the next dP^T while they
// form the next P^T.
template <int D> struct DkvCfg {
    static constexpr int NB = D / 64, TILE = NB * kBoxBytes;
    static constexpr int ST = D == 128 ? 2 : 4;  // stages of Q and of dO
    static constexpr int SMEM = (2 + 2 * ST) * TILE + 1024;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_dkv_tc_kernel(const __grid_constant__ BwdMaps maps,
                                                                  const __grid_constant__ BwdParams p)
{
    using C = DkvCfg<D>;
    constexpr int kTmP = 128, kTmV = 256, kTmK = 384;
    extern __shared__ char raw[];
    char *sm = reinterpret_cast<char *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    char *sk = sm, *sv = sk + C::TILE, *sq = sv + C::TILE, *so = sq + C::ST * C::TILE;
    __shared__ __align__(16) float s_lse[2][kBM], s_delta[2][kBM];
    __shared__ int s_tok[kBM];  // token of a packed row within its tile
    __shared__ __align__(8) uint64_t kv_full, kv_empty, q_full[C::ST], q_empty[C::ST], o_full[C::ST], o_empty[C::ST],
        stat_full[2], stat_empty[2], s_full, d_full, p_ready, ds_ready, done, bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    if (tid == 0) {
        s_abort = 0;
        mbar_init(&kv_full, 1);
        mbar_init(&kv_empty, 1);
        for (int i = 0; i < C::ST; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_empty[i], 1);
        }
        mbar_init(&stat_full[0], 32);
        mbar_init(&stat_full[1], 32);
        mbar_init(&stat_empty[0], 8);
        mbar_init(&stat_empty[1], 8);
        mbar_init(&s_full, 1);
        mbar_init(&d_full, 1);
        mbar_init(&p_ready, 8);
        mbar_init(&ds_ready, 8);
        mbar_init(&done, 1);
        mbar_init(&bar_drain, 1);
        fence_mbar_init();
    }
    if (tid < kBM) s_tok[tid] = tid < p.TQ * p.G ? tid / p.G : INT_MAX;
    if (warp == 8) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(s_tmem);

    // The block's work, walked through by every role: the keys k0 .. of a sequence, and the n tiles of TQ
    // query tokens, from tile ib of the sequence on, that see one of them.  `base` counts the query tiles
    // before it, `num` the tiles of keys.
    struct Work {
        int hk, bos, len, k0, ib, n;
    };
    auto find = [&](int w, Work &x) {
        TileRef r;
        if (!block_tile(p.b, w, p.ktiles, p.Hkv, p.window, kBN, true, r, x.hk)) return false;
        x.bos = r.sp.bos;
        x.len = r.sp.len;
        x.k0 = r.tile * kBN;
        const int end = p.window == 0 || p.window > x.len ? x.len : min(x.len, x.k0 + kBN - 1 + p.window);
        x.ib = x.k0 / p.TQ;
        x.n = (end + p.TQ - 1) / p.TQ - x.ib;
        return true;
    };
    const int works = p.ktiles * p.Hkv;
    int base = 0, num = 0;
    Work x;
    bool ok = true;

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int half = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t ts = tmem + 64 * half + lanes, tp = tmem + kTmP + 64 * half + lanes;
        const float c = p.scale * kLog2e;
        const uint64_t c2 = pair(c, c);
        const int *toks = s_tok + 64 * half;
        for (int i = 0, w; ok && (w = work_at(i, works)) >= 0; ++i) {
            if (w >= works || !find(w, x)) continue;
            const int key = x.k0 + row;
            for (int it = 0; it < x.n; ++it) {
                const int k = base + it, st = k & 1, t0 = (x.ib + it) * p.TQ, nt = min(p.TQ, x.len - t0);
                const bool edge = x.k0 + kBN - 1 > t0 || nt * p.G < kBM || (p.window && t0 + nt - 1 - x.k0 >= p.window);
                if (!(ok = wait_warp(&stat_full[st], (k >> 1) & 1, &s_abort, p.status) &&
                           wait_warp(&s_full, k & 1, &s_abort, p.status)))
                    break;
                tc_fence_after();
                float s[64], d[64];
                ld64(ts, s);
                const float2 *lse = reinterpret_cast<const float2 *>(s_lse[st] + 64 * half);  // negative
                const float2 *delta = reinterpret_cast<const float2 *>(s_delta[st] + 64 * half);
#pragma unroll
                for (int i = 0; i < 64; i += 2)
                    weights(fma2(pair(s[i], s[i + 1]), c2, pair(lse[i / 2].x, lse[i / 2].y)), i / 2, false, s[i], s[i + 1]);
                if (edge) {  // the column's token t0 + tok sees the keys up to its own, and is one of the tile's
                    const int least = key - t0, most = p.window ? min(nt - 1, least + p.window - 1) : nt - 1;
#pragma unroll
                    for (int i = 0; i < 64; ++i) s[i] = toks[i] >= least && toks[i] <= most ? s[i] : 0.f;
                }
                st64(ts, s);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready);
                if (!(ok = wait_warp(&d_full, k & 1, &s_abort, p.status))) break;
                tc_fence_after();
                ld64(tp, d);
#pragma unroll
                for (int i = 0; i < 64; i += 2)
                    unpair(mul2(pair(s[i], s[i + 1]), add2(pair(d[i], d[i + 1]), pair(delta[i / 2].x, delta[i / 2].y))), s[i], s[i + 1]);
                st64(tp, s);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&stat_empty[st]);
                    mbar_arrive(&ds_ready);
                }
            }
            if (!(ok = ok && wait_warp(&done, num & 1, &s_abort, p.status))) break;
            tc_fence_after();
            const size_t at = ((size_t)(x.bos + key) * p.Hkv + x.hk) * D + D / 2 * half;
            store_row<D / 2>(tmem + kTmV + D / 2 * half + lanes, 1.f, p.dv + at, key < x.len);
            store_row<D / 2>(tmem + kTmK + D / 2 * half + lanes, p.scale, p.dk + at, key < x.len);
            tc_fence_before();  // the next tile's first products come after its p of all warps
            base += x.n;
            ++num;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const uint32_t bq = smem_u32(sq), bo = smem_u32(so), bk = smem_u32(sk), bv = smem_u32(sv);
        constexpr uint32_t kS = idesc_bf16(128, kBM, 0, 0), kG = idesc_bf16(128, D, 0, 1);
        if (warp == 8) {
            const uint32_t leader = elect();
            // the tile's rows past its tokens (another sequence's, or never loaded) become zeros: their p and
            // ds are 0, but 0 * NaN is not
            auto scores = [&](int it) {
                const int k = base + it, st = k % C::ST, rows = min(p.TQ, x.len - (x.ib + it) * p.TQ) * p.G;
                if (!wait_warp(&q_full[st], (k / C::ST) & 1, &s_abort, p.status)) return false;
                if (rows < kBM) zero_rows<C::NB>(sq + st * C::TILE, rows);
                tc_fence_after();
                mma_kk<D / 16>(leader, tmem, bk, bq + st * C::TILE, kS);
                commit(leader, &s_full);
                return true;
            };
            auto products = [&](int it) {
                const int k = base + it, st = k % C::ST, rows = min(p.TQ, x.len - (x.ib + it) * p.TQ) * p.G;
                if (!wait_warp(&o_full[st], (k / C::ST) & 1, &s_abort, p.status)) return false;
                if (rows < kBM) zero_rows<C::NB>(so + st * C::TILE, rows);
                tc_fence_after();
                mma_kk<D / 16>(leader, tmem + kTmP, bv, bo + st * C::TILE, kS);
                commit(leader, &d_full);
                if (it + 1 == x.n) commit(leader, &kv_empty);  // its scores came before
                return true;
            };
            for (int i = 0, w; ok && (w = work_at(i, works)) >= 0; ++i) {
                if (w >= works || !find(w, x)) continue;
                if (!(ok = wait_warp(&kv_full, num & 1, &s_abort, p.status))) break;
                ok = scores(0) && products(0);
                for (int it = 0; ok && it < x.n; ++it) {
                    const int k = base + it, st = k % C::ST;
                    if (!(ok = wait_warp(&p_ready, k & 1, &s_abort, p.status))) break;
                    tc_fence_after();
                    mma_tn<4>(leader, tmem + kTmV, tmem, bo + st * C::TILE, 0, kG, it > 0);
                    mma_tn<4>(leader, tmem + kTmV, tmem + 64, bo + st * C::TILE, 64, kG, 1);
                    commit(leader, &o_empty[st]);
                    if (it + 1 < x.n && !(ok = scores(it + 1))) break;
                    if (!(ok = wait_warp(&ds_ready, k & 1, &s_abort, p.status))) break;
                    tc_fence_after();
                    mma_tn<4>(leader, tmem + kTmK, tmem + kTmP, bq + st * C::TILE, 0, kG, it > 0);
                    mma_tn<4>(leader, tmem + kTmK, tmem + kTmP + 64, bq + st * C::TILE, 64, kG, 1);
                    commit(leader, &q_empty[st]);
                    if (it + 1 == x.n) commit(leader, &done);
                    if (it + 1 < x.n) ok = products(it + 1);
                }
                base += x.n;
                ++num;
            }
            if (s_abort) drain(leader, &bar_drain);
        } else if (warp == 9) {
            const uint32_t bytes = C::NB * 128 * p.G * p.TQ;
            int nw = 0, nq = 0, no = 0;  // loads issued, by lane 0
            for (int i = 0, w; ok && (w = work_at(i, works)) >= 0; ++i) {
                if (w >= works || !find(w, x)) continue;
                if (lane == 0 && (nw == 0 || (ok = wait(&kv_empty, (nw - 1) & 1, &s_abort, p.status)))) {
                    mbar_expect_tx(&kv_full, 2 * C::TILE);
                    load_tile<C::NB>(sk, &maps.k, x.hk, x.bos + x.k0, &kv_full);
                    load_tile<C::NB>(sv, &maps.v, x.hk, x.bos + x.k0, &kv_full);
                    ++nw;
                    for (int it = 0; it < x.n; ++it) {
                        const int a = nq % C::ST, b = no % C::ST, row = x.bos + (x.ib + it) * p.TQ;
                        if (nq >= C::ST && !(ok = wait(&q_empty[a], ((nq / C::ST) & 1) ^ 1, &s_abort, p.status))) break;
                        mbar_expect_tx(&q_full[a], bytes);
                        load_tile<C::NB>(sq + a * C::TILE, &maps.q, x.hk * p.G, row, &q_full[a]);
                        ++nq;
                        if (no >= C::ST && !(ok = wait(&o_empty[b], ((no / C::ST) & 1) ^ 1, &s_abort, p.status))) break;
                        mbar_expect_tx(&o_full[b], bytes);
                        load_tile<C::NB>(so + b * C::TILE, &maps.d_o, x.hk * p.G, row, &o_full[b]);
                        ++no;
                    }
                }
                ok = __shfl_sync(0xffffffffu, (int)ok, 0);
            }
            if (s_abort && lane == 0) {
                if (nw) mbar_wait(&kv_full, (nw - 1) & 1, 1000000000ull);
                drain_ring(q_full, nq, C::ST);
                drain_ring(o_full, no, C::ST);
            }
        } else if (warp == 10) {  // -lse (log2) and -delta of the query rows
            for (int i = 0, w; ok && (w = work_at(i, works)) >= 0; ++i) {
                if (w >= works || !find(w, x)) continue;
                for (int it = 0; it < x.n; ++it) {
                    const int k = base + it, st = k & 1, t0 = (x.ib + it) * p.TQ, nt = min(p.TQ, x.len - t0);
                    // a barrier to a stage: ds_ready's own may be two tiles further when this warp, which may have
                    // searched a long batch for its next tile, comes to look
                    if (k >= 2 && !(ok = wait_warp(&stat_empty[st], ((k >> 1) & 1) ^ 1, &s_abort, p.status))) break;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = lane + 32 * i, tok = row / p.G;
                        const bool live = row < p.TQ * p.G && tok < nt;
                        const size_t at = (size_t)(x.bos + t0 + tok) * p.H + x.hk * p.G + (row - tok * p.G);
                        s_lse[st][row] = live ? -p.lse[at] * kLog2e : 0.f;
                        s_delta[st][row] = live ? -p.delta[at] : 0.f;
                    }
                    mbar_arrive(&stat_full[st]);
                }
                base += x.n;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <typename F> cudaError_t run(F kernel, int smem, dim3 grid, const BwdMaps &maps, const BwdParams &p, cudaStream_t s)
{
    cudaError_t e = set_smem_attr(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, smem, s>>>(maps, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_bwd_tc(const AttnArgs &a, cudaStream_t s)
{
    BwdMaps maps;
    BwdParams p{};
    p.b = a.b;
    p.H = a.H;
    p.Hkv = a.Hkv;
    p.G = a.H / a.Hkv;
    p.TQ = kBM / p.G;
    p.window = a.window;
    p.scale = a.scale;
    p.lse = a.lse;
    p.delta = a.delta;
    p.dq = (__nv_bfloat16 *)a.dq;
    p.dk = (__nv_bfloat16 *)a.dk;
    p.dv = (__nv_bfloat16 *)a.dv;
    p.status = a.status;
    if (!make_head_map(&maps.q, a.q, a.b.rows, a.H, a.D, p.G, p.TQ) ||
        !make_head_map(&maps.d_o, a.d_o, a.b.rows, a.H, a.D, p.G, p.TQ) ||
        !make_head_map(&maps.k, a.k, a.b.rows, a.Hkv, a.D, 1, kBN) ||
        !make_head_map(&maps.v, a.v, a.b.rows, a.Hkv, a.D, 1, kBN))
        return cudaErrorInvalidValue;
    cudaError_t e = launch_attn_delta(false, a, s);
    if (e != cudaSuccess) return e;
    const long long nq = tile_bound(a.b, p.TQ) * a.Hkv, nk = tile_bound(a.b, kBN) * a.Hkv, sms = device_sms();
    if (nq > INT_MAX / 2 || nk > INT_MAX / 2) return cudaErrorInvalidValue;
    p.qtiles = (int)(nq / a.Hkv);
    p.ktiles = (int)(nk / a.Hkv);
    const dim3 gq((unsigned)(nq < sms ? nq : sms)), gk((unsigned)(nk < sms ? nk : sms));
    // dq first: its delta of the sequences' first rows is the better one
    if (a.D == 128) {
        e = run(attn_dq_tc_kernel<128>, DqCfg<128>::SMEM, gq, maps, p, s);
        return e != cudaSuccess ? e : run(attn_dkv_tc_kernel<128>, DkvCfg<128>::SMEM, gk, maps, p, s);
    }
    e = run(attn_dq_tc_kernel<64>, DqCfg<64>::SMEM, gq, maps, p, s);
    return e != cudaSuccess ? e : run(attn_dkv_tc_kernel<64>, DkvCfg<64>::SMEM, gk, maps, p, s);
}

}  // namespace gdn2
