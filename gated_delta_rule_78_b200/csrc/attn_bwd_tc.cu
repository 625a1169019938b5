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
// rounded to bf16 for their products (2^-9 of each term), everything else is fp32.
//
// Roles, 384 threads: warps 0-3 and 4-7 form p and ds of the tile's left and right 64 columns (a thread to
// a row), warp 8 issues the products, warp 9 the TMA loads, warp 10 (keys' kernel) brings the rows'
// lse and delta.  bf16 p and ds overwrite the columns of the scores that their own warps have read.
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
    int H, Hkv, G, TQ, window;
    float scale;
    const float *lse, *delta;
    __nv_bfloat16 *dq, *dk, *dv;
    int *status;
};

constexpr int kThreads = 384;

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
// this thread's row of 64 values as bf16 into 32 columns
__device__ __forceinline__ void st64(uint32_t t, const float (&s)[64])
{
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = pack_bf16x2(s[2 * i], s[2 * i + 1]);
    tmem_st32(t, w);
    tmem_wait_st();
}
// D (+)= A B, A = 128 x 128 bf16 left by st64 of both column halves (64 columns apart)
__device__ __forceinline__ void mma_grad(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc)
{
    mma_tn<4>(leader, d, a, b, 0, idesc, acc);
    mma_tn<4>(leader, d, a + 64, b, 64, idesc, 1);
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
// after a wait that gave up: the loads of a ring, `n` of them issued, end before the block's memory is free
__device__ __forceinline__ void drain_ring(uint64_t *full, int n, int stages)
{
    for (int i = n > stages ? n - stages : 0; i < n; ++i) mbar_wait(&full[i % stages], (i / stages) & 1, 1000000000ull);
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
    __shared__ __align__(8) uint64_t bar_q, k_full[C::KS], k_empty[C::KS], v_full[C::VS], v_empty[C::VS], s_full[2], p_full,
        ds_ready, done, bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    if (blockIdx.x == 0 && warp == 0) report_bad_seqlens(p.b, p.status);
    TileRef r;
    int hk;
    if (!block_tile(p.b, blockIdx.x, gridDim.x / p.Hkv, p.Hkv, p.window, p.TQ, false, r, hk)) return;
    const int len = r.sp.len, t0 = r.tile * p.TQ, nt = min(p.TQ, len - t0);
    const int jb = p.window == 0 || t0 < p.window ? 0 : (t0 - p.window + 1) / kBN, n = (t0 + nt - 1) / kBN + 1 - jb;

    if (tid == 0) {
        s_abort = 0;
        mbar_init(&bar_q, 1);
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

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int half = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const int tok = row / p.G, pos = t0 + tok;
        const bool live = row < p.TQ * p.G && tok < nt;
        const size_t at = (size_t)(r.sp.bos + pos) * p.H + hk * p.G + (row - tok * p.G);
        const float c = p.scale * kLog2e;
        const float lse = live ? p.lse[at] * kLog2e : 0.f, delta = live ? p.delta[at] : 0.f;
        bool ok = true;
        for (int it = 0; it < n; ++it) {
            if (!(ok = wait_warp(&s_full[it & 1], (it >> 1) & 1, &s_abort, p.status))) break;
            tc_fence_after();
            float s[64], d[64];
            const uint32_t ts = tmem + 128 * (it & 1) + 64 * half + lanes;
            ld64(ts, s);
            const int k0 = (jb + it) * kBN;
            const bool edge = k0 + kBN - 1 > t0 || (p.window && t0 + nt - 1 - k0 >= p.window);
            const int most = pos - k0 - 64 * half, least = p.window ? most - p.window + 1 : 0;
            if (edge) {
#pragma unroll
                for (int i = 0; i < 64; ++i) s[i] = i <= most && i >= least ? s[i] : -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = ex2(fmaf(s[i], c, -lse));
            if (!(ok = wait_warp(&p_full, it & 1, &s_abort, p.status))) break;
            tc_fence_after();
            ld64(tmem + kTmP + 64 * half + lanes, d);
            if (edge) {  // values of masked keys may belong to another sequence: not 0 * (what they are)
#pragma unroll
                for (int i = 0; i < 64; ++i) d[i] = i <= most && i >= least ? d[i] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] *= d[i] - delta;
            st64(ts, s);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ds_ready);
        }
        if (ok && wait_warp(&done, 0, &s_abort, p.status)) {
            tc_fence_after();
            store_row<D / 2>(tmem + kTmQ + D / 2 * half + lanes, p.scale, p.dq + at * D + D / 2 * half, live);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const uint32_t bq = smem_u32(sq), bo = smem_u32(so), bk = smem_u32(sk), bv = smem_u32(sv);
        constexpr uint32_t kS = idesc_bf16(128, kBN, 0, 0), kG = idesc_bf16(128, D, 0, 1);
        if (warp == 8) {
            const uint32_t leader = elect();
            bool ok = wait_warp(&bar_q, 0, &s_abort, p.status);
            auto scores = [&](int it) {
                const int st = it % C::KS;
                if (!wait_warp(&k_full[st], (it / C::KS) & 1, &s_abort, p.status)) return false;
                // keys past the sequence are another's: their ds is 0, but 0 * NaN is not
                if ((jb + it + 1) * kBN > len) zero_rows<C::NB>(sk + st * C::TILE, len - (jb + it) * kBN);
                tc_fence_after();
                mma_kk<D / 16>(leader, tmem + 128 * (it & 1), bq, bk + st * C::TILE, kS);
                commit(leader, &s_full[it & 1]);
                return true;
            };
            auto products = [&](int it) {
                const int st = it % C::VS;
                if (!wait_warp(&v_full[st], (it / C::VS) & 1, &s_abort, p.status)) return false;
                tc_fence_after();
                mma_kk<D / 16>(leader, tmem + kTmP, bo, bv + st * C::TILE, kS);
                commit(leader, &p_full);
                commit(leader, &v_empty[st]);
                return true;
            };
            if (ok) ok = scores(0) && products(0) && (n < 2 || scores(1));
            for (int it = 0; ok && it < n; ++it) {
                if (!(ok = wait_warp(&ds_ready, it & 1, &s_abort, p.status))) break;
                tc_fence_after();
                mma_grad(leader, tmem + kTmQ, tmem + 128 * (it & 1), bk + (it % C::KS) * C::TILE, kG, it > 0);
                commit(leader, &k_empty[it % C::KS]);
                if (it + 1 == n) commit(leader, &done);
                if (it + 1 < n) ok = products(it + 1);
                if (ok && it + 2 < n) ok = scores(it + 2);
            }
            if (s_abort) drain(leader, &bar_drain);
        } else if (warp == 9 && lane == 0) {
            mbar_expect_tx(&bar_q, 2 * C::NB * 128 * p.G * p.TQ);
            load_tile<C::NB>(sq, &maps.q, hk * p.G, r.sp.bos + t0, &bar_q);
            load_tile<C::NB>(so, &maps.d_o, hk * p.G, r.sp.bos + t0, &bar_q);
            int nk = 0, nv = 0;
            for (int it = 0; it < n; ++it) {
                const int a = it % C::KS, b = it % C::VS, row = r.sp.bos + (jb + it) * kBN;
                if (it >= C::KS && !wait(&k_empty[a], ((it / C::KS) & 1) ^ 1, &s_abort, p.status)) break;
                mbar_expect_tx(&k_full[a], C::TILE);
                load_tile<C::NB>(sk + a * C::TILE, &maps.k, hk, row, &k_full[a]);
                ++nk;
                if (it >= C::VS && !wait(&v_empty[b], ((it / C::VS) & 1) ^ 1, &s_abort, p.status)) break;
                mbar_expect_tx(&v_full[b], C::TILE);
                load_tile<C::NB>(sv + b * C::TILE, &maps.v, hk, row, &v_full[b]);
                ++nv;
            }
            if (s_abort) {
                mbar_wait(&bar_q, 0, 1000000000ull);
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
    __shared__ int s_pos[2][kBM];
    __shared__ __align__(8) uint64_t bar_kv, q_full[C::ST], q_empty[C::ST], o_full[C::ST], o_empty[C::ST], stat_full[2], s_full,
        p_full, p_ready, ds_ready, done, bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    TileRef r;
    int hk;
    if (!block_tile(p.b, blockIdx.x, gridDim.x / p.Hkv, p.Hkv, p.window, kBN, true, r, hk)) return;
    const int len = r.sp.len, k0 = r.tile * kBN;
    // query tokens that see a key of this tile: k0 .. end - 1, in tiles of TQ from the sequence's start
    const int end = p.window == 0 || p.window > len ? len : min(len, k0 + kBN - 1 + p.window);
    const int ib = k0 / p.TQ, n = (end + p.TQ - 1) / p.TQ - ib;

    if (tid == 0) {
        s_abort = 0;
        mbar_init(&bar_kv, 1);
        for (int i = 0; i < C::ST; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_empty[i], 1);
        }
        mbar_init(&stat_full[0], 32);
        mbar_init(&stat_full[1], 32);
        mbar_init(&s_full, 1);
        mbar_init(&p_full, 1);
        mbar_init(&p_ready, 8);
        mbar_init(&ds_ready, 8);
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

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int half = warp >> 2, row = tid & 127, key = k0 + row;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t ts = tmem + 64 * half + lanes, tp = tmem + kTmP + 64 * half + lanes;
        const float c = p.scale * kLog2e;
        bool ok = true;
        for (int it = 0; it < n; ++it) {
            const int st = it & 1, t0 = (ib + it) * p.TQ, nt = min(p.TQ, len - t0);
            const bool edge = k0 + kBN - 1 > t0 || nt * p.G < kBM || (p.window && t0 + nt - 1 - k0 >= p.window);
            if (!(ok = wait_warp(&stat_full[st], (it >> 1) & 1, &s_abort, p.status) &&
                       wait_warp(&s_full, it & 1, &s_abort, p.status)))
                break;
            tc_fence_after();
            float s[64], d[64];
            ld64(ts, s);
            const float *lse = s_lse[st] + 64 * half, *delta = s_delta[st] + 64 * half;
            const int *pos = s_pos[st] + 64 * half;
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = ex2(fmaf(s[i], c, -lse[i]));
            if (edge) {  // pos is -1 for columns that hold no row
#pragma unroll
                for (int i = 0; i < 64; ++i) s[i] = key <= pos[i] && (p.window == 0 || pos[i] - key < p.window) ? s[i] : 0.f;
            }
            st64(ts, s);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready);
            if (!(ok = wait_warp(&p_full, it & 1, &s_abort, p.status))) break;
            tc_fence_after();
            ld64(tp, d);
#pragma unroll
            for (int i = 0; i < 64; ++i) d[i] = s[i] * (d[i] - delta[i]);
            st64(tp, d);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ds_ready);
        }
        if (ok && wait_warp(&done, 0, &s_abort, p.status)) {
            tc_fence_after();
            const size_t at = ((size_t)(r.sp.bos + key) * p.Hkv + hk) * D + D / 2 * half;
            store_row<D / 2>(tmem + kTmV + D / 2 * half + lanes, 1.f, p.dv + at, key < len);
            store_row<D / 2>(tmem + kTmK + D / 2 * half + lanes, p.scale, p.dk + at, key < len);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const uint32_t bq = smem_u32(sq), bo = smem_u32(so), bk = smem_u32(sk), bv = smem_u32(sv);
        constexpr uint32_t kS = idesc_bf16(128, kBM, 0, 0), kG = idesc_bf16(128, D, 0, 1);
        if (warp == 8) {
            const uint32_t leader = elect();
            bool ok = wait_warp(&bar_kv, 0, &s_abort, p.status);
            // the tile's rows past its tokens (another sequence's, or never loaded) become zeros: their p and
            // ds are 0, but 0 * NaN is not
            auto scores = [&](int it) {
                const int st = it % C::ST, rows = min(p.TQ, len - (ib + it) * p.TQ) * p.G;
                if (!wait_warp(&q_full[st], (it / C::ST) & 1, &s_abort, p.status)) return false;
                if (rows < kBM) zero_rows<C::NB>(sq + st * C::TILE, rows);
                tc_fence_after();
                mma_kk<D / 16>(leader, tmem, bk, bq + st * C::TILE, kS);
                commit(leader, &s_full);
                return true;
            };
            auto products = [&](int it) {
                const int st = it % C::ST, rows = min(p.TQ, len - (ib + it) * p.TQ) * p.G;
                if (!wait_warp(&o_full[st], (it / C::ST) & 1, &s_abort, p.status)) return false;
                if (rows < kBM) zero_rows<C::NB>(so + st * C::TILE, rows);
                tc_fence_after();
                mma_kk<D / 16>(leader, tmem + kTmP, bv, bo + st * C::TILE, kS);
                commit(leader, &p_full);
                return true;
            };
            if (ok) ok = scores(0) && products(0);
            for (int it = 0; ok && it < n; ++it) {
                const int st = it % C::ST;
                if (!(ok = wait_warp(&p_ready, it & 1, &s_abort, p.status))) break;
                tc_fence_after();
                mma_grad(leader, tmem + kTmV, tmem, bo + st * C::TILE, kG, it > 0);
                commit(leader, &o_empty[st]);
                if (it + 1 < n && !(ok = scores(it + 1))) break;
                if (!(ok = wait_warp(&ds_ready, it & 1, &s_abort, p.status))) break;
                tc_fence_after();
                mma_grad(leader, tmem + kTmK, tmem + kTmP, bq + st * C::TILE, kG, it > 0);
                commit(leader, &q_empty[st]);
                if (it + 1 == n) commit(leader, &done);
                if (it + 1 < n) ok = products(it + 1);
            }
            if (s_abort) drain(leader, &bar_drain);
        } else if (warp == 9 && lane == 0) {
            mbar_expect_tx(&bar_kv, 2 * C::TILE);
            load_tile<C::NB>(sk, &maps.k, hk, r.sp.bos + k0, &bar_kv);
            load_tile<C::NB>(sv, &maps.v, hk, r.sp.bos + k0, &bar_kv);
            const uint32_t bytes = C::NB * 128 * p.G * p.TQ;
            int nq = 0, no = 0;
            for (int it = 0; it < n; ++it) {
                const int st = it % C::ST, row = r.sp.bos + (ib + it) * p.TQ;
                const uint32_t par = ((it / C::ST) & 1) ^ 1;
                if (it >= C::ST && !wait(&q_empty[st], par, &s_abort, p.status)) break;
                mbar_expect_tx(&q_full[st], bytes);
                load_tile<C::NB>(sq + st * C::TILE, &maps.q, hk * p.G, row, &q_full[st]);
                ++nq;
                if (it >= C::ST && !wait(&o_empty[st], par, &s_abort, p.status)) break;
                mbar_expect_tx(&o_full[st], bytes);
                load_tile<C::NB>(so + st * C::TILE, &maps.d_o, hk * p.G, row, &o_full[st]);
                ++no;
            }
            if (s_abort) {
                mbar_wait(&bar_kv, 0, 1000000000ull);
                drain_ring(q_full, nq, C::ST);
                drain_ring(o_full, no, C::ST);
            }
        } else if (warp == 10) {  // lse (log2), delta and position of the query rows
            for (int it = 0; it < n; ++it) {
                const int st = it & 1, t0 = (ib + it) * p.TQ, nt = min(p.TQ, len - t0);
                // the warps have read the stage's former rows once their ds is ready
                if (it >= 2 && !wait_warp(&ds_ready, it & 1, &s_abort, p.status)) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = lane + 32 * i, tok = row / p.G;
                    const bool live = tok < nt;
                    const size_t at = (size_t)(r.sp.bos + t0 + tok) * p.H + hk * p.G + (row - tok * p.G);
                    s_lse[st][row] = live ? p.lse[at] * kLog2e : 0.f;
                    s_delta[st][row] = live ? p.delta[at] : 0.f;
                    s_pos[st][row] = live ? t0 + tok : -1;
                }
                mbar_arrive(&stat_full[st]);
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
    const long long nq = tile_bound(a.b, p.TQ) * a.Hkv, nk = tile_bound(a.b, kBN) * a.Hkv;
    if (nq > INT_MAX || nk > INT_MAX) return cudaErrorInvalidValue;
    const dim3 gq((unsigned)nq), gk((unsigned)nk);
    if (a.D == 128) {
        e = run(attn_dkv_tc_kernel<128>, DkvCfg<128>::SMEM, gk, maps, p, s);
        return e != cudaSuccess ? e : run(attn_dq_tc_kernel<128>, DqCfg<128>::SMEM, gq, maps, p, s);
    }
    e = run(attn_dkv_tc_kernel<64>, DkvCfg<64>::SMEM, gk, maps, p, s);
    return e != cudaSuccess ? e : run(attn_dq_tc_kernel<64>, DqCfg<64>::SMEM, gq, maps, p, s);
}

}  // namespace gdn2
