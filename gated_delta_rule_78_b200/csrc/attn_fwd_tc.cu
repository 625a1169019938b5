// Causal attention forward on the tensor cores (bf16): whole sequences (keys by TMA) and the newest
// tokens of sequences over a paged cache (keys gathered page by page).
//
//   s_ij = scale q_i . k_j (visible j),  o_i = sum_j 2^(c s'_ij - m_i) v_j / l_i with c = scale log2 e
//
// One pass over the keys with a running reference m_i and sum l_i.  The reference follows the
// maximum only when a row's maximum has grown by more than 2^8 since: sums and outputs then stay
// far from overflow in fp32, and the accumulator is rescaled a few times a row instead of once a
// tile.  The weights are rounded to bf16 for the second product (their sum l_i is of the unrounded
// ones); that costs up to 2^-8 of each weight, no more than the rounding of o.
//
// A block owns two tiles A and B of 128 packed query rows.  Roles: warps 0-3 and 4-7 the softmax of
// A and of B (a thread to a row), warp 8 the products, warp 9 the TMA loads, warps 9-11 (paged)
// the gather of pages.  The tensor core works on one tile's S = Q K^T and O += P V while the other
// tile's warps form its weights.  TMEM: S_A, S_B (128 columns each), O_A, O_B (D columns each).
// With D = 128 that is all of it: P overwrites its own S, and the next S waits for P V.  With D = 64 P
// has 64 columns of its own, and the next S is formed as soon as the warps hold this one in registers.
//
// 4 x 4096, 16 heads, D = 128, window 2048: 219 us, 206 GFLOP, 940 TFLOP/s.  A step (a key tile for A and B) takes 1.9 us
// of which the products are 1.5: with D = 128 S of the next tile cannot start before this P V, and the two
// tiles' softmax fills only most of that gap.  With D = 64 it takes 1.7 us, bound by the warps: 16 exponentials a
// clock are 70% of it.
#include <limits.h>

#include "attn_tc.cuh"

namespace gdn2 {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

namespace attn {

bool make_head_map(CUtensorMap *m, const void *ptr, long long rows, int heads, int D, int box_heads, int box_rows)
{
    static EncodeTiledFn enc = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return (EncodeTiledFn) nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)heads * D * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    const cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn

namespace {

using namespace attn;
using namespace tc;

template <int D> struct Cfg {
    static constexpr int NB = D / 64;                      // column blocks of a tile
    static constexpr int TILE = NB * kBoxBytes;            // bytes of a 128-row tile
    static constexpr int ST = D == 128 ? 2 : 4;            // stages of K and of V
    static constexpr int SMEM = 2 * TILE + 2 * ST * TILE + 1024;  // kPagedE4m3: and the raw rows
};
template <int D> constexpr int kRawBytes = 64 * D;  // e4m3 rows of a step of the gather, three steps of them
constexpr int kTmS = 0, kTmO = 256, kTmP = 384;  // TMEM columns: S_A, S_B; O_A, O_B; P_A, P_B (D = 64)
constexpr int kThreads = 384, kGather = 3;  // threads; warps that gather pages
constexpr float kGrow = 8.f;         // growth of the maximum (log2) that moves the reference

struct FwdMaps {
    CUtensorMap q, k, v;
};
struct FwdParams {
    SeqBatch b;
    int H, Hkv, G, TQ, window, splits;
    float scale;
    __nv_bfloat16 *o;
    float *lse;
    int *status;
    PagedCache c;       // paged only, as is the rest
    int box;            // rows of a box of a page
    float *part_o, *part_l;
};

// The key tiles that a block works on, and each query tile's share of them.
struct Ranges {
    int first, kvlen;        // position of the sequence's query token 0; keys
    int least;               // the first key that a query of the block sees: pages wholly before it may be another's by now
    int t0[2], n[2];         // first token of tile A / B in the sequence, tokens in it
    int beg[2], end[2];      // its key tiles
    int jb, je;              // their union
};
__device__ __forceinline__ Ranges make_ranges(const FwdParams &p, const TileRef &r, int kvlen, int split)
{
    Ranges g;
    g.kvlen = kvlen;
    g.first = kvlen - r.sp.len;
    g.least = p.window ? max(0, g.first + 2 * r.tile * p.TQ - p.window + 1) : 0;
    int lo = INT_MAX, hi = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        g.t0[x] = (2 * r.tile + x) * p.TQ;
        g.n[x] = min(p.TQ, r.sp.len - g.t0[x]);
        g.beg[x] = g.end[x] = 0;
        if (g.n[x] <= 0) continue;
        const int low = g.first + g.t0[x], high = low + g.n[x] - 1;
        g.beg[x] = p.window == 0 || low < p.window ? 0 : (low - p.window + 1) / kBN;
        g.end[x] = high / kBN + 1;
        lo = min(lo, g.beg[x]);
        hi = max(hi, g.end[x]);
    }
    if (p.splits > 1) {  // this block's share of the union
        const int per = (hi - lo + p.splits - 1) / p.splits;
        lo += split * per;
        hi = min(hi, lo + per);
    }
    g.jb = INT_MAX;
    g.je = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        g.beg[x] = max(g.beg[x], lo);
        g.end[x] = min(g.end[x], hi);
        if (g.beg[x] >= g.end[x]) {
            g.beg[x] = g.end[x] = 0;
            continue;
        }
        g.jb = min(g.jb, g.beg[x]);
        g.je = max(g.je, g.end[x]);
    }
    if (g.je == 0) g.jb = 0;
    return g;
}

// Where the keys come from: whole sequences by TMA; a paged cache's bf16 rows by TMA, in boxes of as
// many rows as divide both a page and a tile (8 at least: a swizzle atom); pages of other sizes, and
// e4m3 rows, by ordinary asynchronous copies.
enum { kWhole, kPaged, kPagedAny, kPagedE4m3 };

template <int D, int kind>
__global__ void __launch_bounds__(kThreads, 1) attn_fwd_tc_kernel(const __grid_constant__ FwdMaps maps,
                                                                          const __grid_constant__ FwdParams p)
{
    using C = Cfg<D>;
    constexpr bool kSep = D == 64;  // P beside S
    constexpr bool paged = kind != kWhole, e4m3 = kind == kPagedE4m3, gather = kind >= kPagedAny;
    constexpr int SS = C::ST + 2;  // stages of the scales: see the gather
    extern __shared__ char raw[];
    char *sm = reinterpret_cast<char *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    char *sq = sm, *sk = sm + 2 * C::TILE, *sv = sk + C::ST * C::TILE;
    __shared__ __align__(8) uint64_t bar_q, k_full[C::ST], k_empty[C::ST], v_full[C::ST], v_empty[C::ST], s_full[2],
        s_free[2], p_ready[2][2], o_done[2], bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ float s_ks[e4m3 ? SS : 1][kBN], s_vs[e4m3 ? SS : 1][kBN];
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

    if (blockIdx.x == 0 && warp == 0) report_bad_seqlens(p.b, p.status);
    TileRef r;
    int hk, split = 0;
    if constexpr (paged) {
        hk = blockIdx.x % p.Hkv;
        split = blockIdx.x / p.Hkv;
        const int rank = split / p.splits;
        split -= rank * p.splits;
        if (!find_long_tile(p.b, p.c.kv_lens, rank, 2 * p.TQ, r)) return;
    } else {
        if (!block_tile(p.b, blockIdx.x, gridDim.x / p.Hkv, p.Hkv, p.window, 2 * p.TQ, false, r, hk)) return;
    }
    int kvlen = r.sp.len;
    if (paged) {
        kvlen = p.c.kv_lens[r.seq];
        if (kvlen < r.sp.len || kvlen > (long long)p.c.width * p.c.page) {
            if (tid == 0) atomicExch(p.status, kStatusBadPages);
            return;
        }
    }
    const Ranges g = make_ranges(p, r, kvlen, split);

    if (tid == 0) {
        s_abort = 0;
        mbar_init(&bar_q, 1);
        mbar_init(&bar_drain, 1);
        for (int i = 0; i < C::ST; ++i) {
            mbar_init(&k_full[i], gather ? kGather * 32 : 1);
            mbar_init(&v_full[i], gather ? kGather * 32 : 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s_full[x], 1);
            mbar_init(&s_free[x], 4);
            mbar_init(&p_ready[x][0], 4);
            mbar_init(&p_ready[x][1], 4);
            mbar_init(&o_done[x], 1);
        }
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

    if (warp < 8) {  // ---- softmax of tile A (warps 0-3) or B (4-7): thread = row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int x = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
        const uint32_t ts = tmem + kTmS + 128 * x + lanes, to = tmem + kTmO + D * x + lanes;
        const uint32_t tp = kSep ? tmem + kTmP + 64 * x + lanes : ts;
        const int beg = x ? g.beg[1] : g.beg[0], end = x ? g.end[1] : g.end[0], nt = x ? g.n[1] : g.n[0];
        const int tok0 = x ? g.t0[1] : g.t0[0], tok = row / p.G, gq = row - tok * p.G;
        const int low = g.first + tok0, high = low + nt - 1, pos = low + tok;
        const float c = p.scale * kLog2e;
        float m = -INFINITY, l = 0.f;  // reference in units of s, sum of the weights relative to it
        bool ok = true;
        uint32_t ph = 0;
        for (int j = beg; j < end; ++j, ph ^= 1) {
            if (!(ok = wait_warp(&s_full[x], ph, &s_abort, p.status))) break;
            tc_fence_after();
            float s[128];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, reinterpret_cast<uint32_t(&)[32]>(s[32 * q]));
            tmem_wait_ld();
            if constexpr (kSep) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_free[x]);
            }
            const int k0 = j * kBN;
            if constexpr (e4m3) {
                const float *ks = s_ks[(j - g.jb) % SS];
#pragma unroll
                for (int i = 0; i < 128; ++i) s[i] *= ks[i];
            }
            const bool edge = k0 + kBN - 1 > low || (p.window && k0 <= high - p.window);
            if (edge) {
                const int most = pos - k0, least = p.window ? most - p.window + 1 : 0;
#pragma unroll
                for (int i = 0; i < 128; ++i) s[i] = i <= most && i >= least ? s[i] : -INFINITY;
            }
            float t0 = fmaxf(s[0], s[1]), t1 = fmaxf(s[2], s[3]), t2 = fmaxf(s[4], s[5]), t3 = fmaxf(s[6], s[7]);
#pragma unroll
            for (int i = 8; i < 128; i += 8) {
                t0 = max3(t0, s[i], s[i + 1]);
                t1 = max3(t1, s[i + 2], s[i + 3]);
                t2 = max3(t2, s[i + 4], s[i + 5]);
                t3 = max3(t3, s[i + 6], s[i + 7]);
            }
            const float top = fmaxf(max3(t0, t1, t2), t3);
            const bool grow = (top - m) * c > kGrow;  // true for the row's first visible key (m = -inf)
            const bool move = __any_sync(0xffffffffu, grow);
            // P beside S: the former product has to be done with O before it is scaled, and with P before the
            // next is stored, which by then is half formed (waited for before the weights: 419 us against 379 at 8192
            // tokens, 32 heads on 8).  Otherwise its commit came before this S.
            bool done = !kSep || j == beg;
            auto former = [&] { return done || (done = ok = wait_warp(&o_done[x], ph ^ 1, &s_abort, p.status)); };
            if (move && !former()) break;
            if (move) {
                const float f = grow ? ex2((m - top) * c) : 1.f;
                if (grow) m = top;
                l *= f;
                if (j > beg) {
                    tc_fence_after();
#pragma unroll
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t w[32];
                        tmem_ld32(to + 32 * q, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
                        tmem_st32(to + 32 * q, w);
                    }
                }
            }
            const float off = m == -INFINITY ? 0.f : -m * c;  // no key visible yet: all weights 0
            const uint64_t c2 = pair(c, c), off2 = pair(off, off);
            uint64_t sum0 = 0, sum1 = 0;
            // weights of a quarter of the keys, handed over as they are formed: the product starts on the
            // first while the next are formed
            auto weights = [&](int h, uint32_t (&w)[16]) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float a, b;
                    unpair(fma2(pair(s[32 * h + 2 * i], s[32 * h + 2 * i + 1]), c2, off2), a, b);
                    a = ex2(a);
                    b = ex2(b);
                    if (i & 1) sum1 = add2(sum1, pair(a, b));
                    else sum0 = add2(sum0, pair(a, b));
                    if constexpr (e4m3) {
                        const float *vs = s_vs[(j - g.jb) % SS] + 32 * h;
                        w[i] = pack_bf16x2(a * vs[2 * i], b * vs[2 * i + 1]);
                    } else {
                        w[i] = pack_bf16x2(a, b);
                    }
                }
            };
            auto hand_over = [&](int h) {
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[x][h]);
            };
            uint32_t w0[16], w1[16];
            weights(0, w0);
            weights(1, w1);
            if (!former()) break;
            tmem_st16(tp, w0);
            tmem_st16(tp + 16, w1);
            hand_over(0);
            weights(2, w0);
            tmem_st16(tp + 32, w0);
            weights(3, w1);
            tmem_st16(tp + 48, w1);
            hand_over(1);
            float a, b, d, e;
            unpair(sum0, a, b);
            unpair(sum1, d, e);
            l += (a + b) + (d + e);
        }
        const bool any = beg < end;
        if (any && ok) ok = wait_warp(&o_done[x], kSep ? ph ^ 1 : 0, &s_abort, p.status);
        if (ok && nt > 0) {  // (warp-uniform) o = O / l
            tc_fence_after();
            const bool live = row < p.TQ * p.G && tok < nt;
            const size_t at = (size_t)(r.sp.bos + tok0 + tok) * p.H + hk * p.G + gq;
            const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            const float lse = l > 0.f || l != l ? (m * c + __log2f(l)) * kLn2 : -INFINITY;
            const size_t base = p.splits > 1 ? ((size_t)split * p.b.rows * p.H + at) : at;
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
                uint32_t w[32];
                if (any) {
                    tmem_ld32(to + 32 * q, w);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] = any ? __float_as_uint(__uint_as_float(w[i]) * inv) : 0u;
                if (!live) continue;
                const size_t ch = base * D + 32 * q;
                if (p.splits > 1) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        const uint32_t v[8] = {w[i], w[i + 1], w[i + 2], w[i + 3], w[i + 4], w[i + 5], w[i + 6], w[i + 7]};
                        store32(p.part_o + ch + i, v);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 16) {
                        uint32_t v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[e] = pack_bf16x2(__uint_as_float(w[i + 2 * e]), __uint_as_float(w[i + 2 * e + 1]));
                        store32(p.o + ch + i, v);
                    }
                }
            }
            if (live) {
                if (p.splits > 1) p.part_l[base] = lse;
                else if (p.lse) p.lse[base] = lse;
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const uint32_t bq = smem_u32(sq), bk = smem_u32(sk), bv = smem_u32(sv);
        if (warp == 8) {  // ---- the products
            constexpr uint32_t kS = idesc_bf16(128, kBN, 0, 0), kO = idesc_bf16(128, D, 0, 1);
            bool ok = g.je > g.jb && wait_warp(&bar_q, 0, &s_abort, p.status);
            const uint32_t leader = elect();
            uint32_t ph[2] = {0, 0};
            const int jb = uniform(g.jb), je = uniform(g.je), kvlen = uniform(g.kvlen);
            const int beg[2] = {uniform(g.beg[0]), uniform(g.beg[1])}, end[2] = {uniform(g.end[0]), uniform(g.end[1])};
            // S of tile x for key tile `nx` in the ring
            auto scores = [&](int x, int nx) {
                tc_fence_after();
                mma_kk<D / 16>(leader, tmem + kTmS + 128 * x, bq + x * C::TILE, bk + (nx % C::ST) * C::TILE, kS);
                commit(leader, &s_full[x]);
            };
            // O += P V of tile x and key tile j = jb + it
            auto output = [&](int x, int j, int it) {
                const uint32_t tp = tmem + (kSep ? kTmP + 64 * x : kTmS + 128 * x);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!wait_warp(&p_ready[x][h], ph[x], &s_abort, p.status)) return false;
                    tc_fence_after();
                    mma_tn<4>(leader, tmem + kTmO + D * x, tp + 32 * h, bv + (it % C::ST) * C::TILE, 64 * h, kO, j > beg[x] || h);
                }
                ph[x] ^= 1;
                if (kSep || j + 1 == end[x]) commit(leader, &o_done[x]);
                return true;
            };
            auto have_v = [&](int it) {
                if (!wait_warp(&v_full[it % C::ST], (it / C::ST) & 1, &s_abort, p.status)) return false;
                if (kind == kPagedAny) fence_proxy_async_smem();  // the copies are ordinary writes to shared memory
                // rows past the sequence hold other sequences' values: 0 * NaN is not 0
                if (!gather && (jb + it + 1) * kBN > kvlen) zero_rows<C::NB>(sv + (it % C::ST) * C::TILE, kvlen - (jb + it) * kBN);
                return true;
            };
            auto have_k = [&](int nx) {
                if (!wait_warp(&k_full[nx % C::ST], (nx / C::ST) & 1, &s_abort, p.status)) return false;
                if (kind == kPagedAny) fence_proxy_async_smem();
                return true;
            };
            for (int j = jb - 1; ok && j < je; ++j) {
                const int it = j - jb, nx = it + 1;  // key tile j and the next one in the rings
                const bool now = j >= jb, next = j + 1 < je;
                if constexpr (kSep) {
                    if (next && !(ok = have_k(nx))) break;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (!(j + 1 >= beg[x] && j + 1 < end[x])) continue;
                        if (j >= beg[x] && !(ok = wait_warp(&s_free[x], ph[x], &s_abort, p.status))) break;
                        scores(x, nx);
                    }
                    if (!ok) break;
                    if (next) commit(leader, &k_empty[nx % C::ST]);
                    if (now && !(ok = have_v(it))) break;
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        if (j >= beg[x] && j < end[x] && !(ok = output(x, j, it))) break;
                    if (!ok) break;
                    if (now) commit(leader, &v_empty[it % C::ST]);
                } else {
                    if (now && !(ok = have_v(it))) break;
                    if (next && !(ok = have_k(nx))) break;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (j >= beg[x] && j < end[x] && !(ok = output(x, j, it))) break;
                        if (j + 1 >= beg[x] && j + 1 < end[x]) scores(x, nx);
                    }
                    if (!ok) break;
                    if (now) commit(leader, &v_empty[it % C::ST]);
                    if (next) commit(leader, &k_empty[nx % C::ST]);
                }
            }
            if (s_abort) drain(leader, &bar_drain);
        } else if (warp == 9 && g.je > g.jb) {  // ---- TMA loads
            int nk = 0, nv = 0;
            if (lane == 0) {
                prefetch_tmap(&maps.q);
                uint32_t bytes = 0;
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (g.n[x] > 0) bytes += C::NB * 128 * p.G * p.TQ;
                mbar_expect_tx(&bar_q, bytes);
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (g.n[x] > 0)
#pragma unroll
                        for (int b = 0; b < C::NB; ++b)
                            tma_load_3d(sq + x * C::TILE + b * kBoxBytes, &maps.q, 64 * b, hk * p.G, r.sp.bos + g.t0[x], &bar_q);
            }
            if constexpr (kind == kWhole) {
                for (int j = g.jb; lane == 0 && j < g.je; ++j) {
                    const int it = j - g.jb, s = it % C::ST;
                    const uint32_t par = ((it / C::ST) & 1) ^ 1;
                    if (it >= C::ST && !wait(&k_empty[s], par, &s_abort, p.status)) break;
                    mbar_expect_tx(&k_full[s], C::TILE);
#pragma unroll
                    for (int b = 0; b < C::NB; ++b)
                        tma_load_3d(sk + s * C::TILE + b * kBoxBytes, &maps.k, 64 * b, hk, r.sp.bos + j * kBN, &k_full[s]);
                    ++nk;
                    if (it >= C::ST && !wait(&v_empty[s], par, &s_abort, p.status)) break;
                    mbar_expect_tx(&v_full[s], C::TILE);
#pragma unroll
                    for (int b = 0; b < C::NB; ++b)
                        tma_load_3d(sv + s * C::TILE + b * kBoxBytes, &maps.v, 64 * b, hk, r.sp.bos + j * kBN, &v_full[s]);
                    ++nv;
                }
            }
            if constexpr (kind == kPaged) {  // a box to a lane: column block `blk` of rows seg * box ..
                __syncwarp();
                const int seg = lane / C::NB, blk = lane % C::NB, off = blk * kBoxBytes + seg * p.box * 128;
                const bool live = seg * p.box < kBN;
                const int *table = p.c.table + (size_t)r.seq * p.c.width;
                // its row in the cache, past the end (zeros) for what the sequence lacks or the window has left behind
                auto row_of = [&](int j) {
                    const int at = j * kBN + seg * p.box, none = p.c.num_pages * p.c.page;
                    if (!live || at >= g.kvlen || at + p.box <= g.least) return none;
                    const int pg = at / p.c.page, id = table[pg];
                    if (id >= 0 && id < p.c.num_pages) return id * p.c.page + (at - pg * p.c.page);
                    atomicExch(p.status, kStatusBadPages);
                    return none;
                };
                int row = row_of(g.jb);
                for (int j = g.jb; j < g.je; ++j) {
                    const int it = j - g.jb, s = it % C::ST;
                    const uint32_t par = ((it / C::ST) & 1) ^ 1;
                    const int next = j + 1 < g.je ? row_of(j + 1) : 0;
                    if (it >= C::ST && !wait_warp(&k_empty[s], par, &s_abort, p.status)) break;
                    if (lane == 0) mbar_expect_tx(&k_full[s], C::TILE);
                    __syncwarp();
                    if (live) tma_load_3d(sk + s * C::TILE + off, &maps.k, 64 * blk, hk, row, &k_full[s]);
                    ++nk;
                    if (it >= C::ST && !wait_warp(&v_empty[s], par, &s_abort, p.status)) break;
                    if (lane == 0) mbar_expect_tx(&v_full[s], C::TILE);
                    __syncwarp();
                    if (live) tma_load_3d(sv + s * C::TILE + off, &maps.v, 64 * blk, hk, row, &v_full[s]);
                    ++nv;
                    row = next;
                }
            }
            // after a wait that gave up, loads in flight end before the block's memory is free
            if (s_abort) {
                mbar_wait(&bar_q, 0, 1000000000ull);
                for (int i = max(0, nk - C::ST); i < nk; ++i) mbar_wait(&k_full[i % C::ST], (i / C::ST) & 1, 1000000000ull);
                for (int i = max(0, nv - C::ST); i < nv; ++i) mbar_wait(&v_full[i % C::ST], (i / C::ST) & 1, 1000000000ull);
            }
        }
        if constexpr (gather) {
            if (warp >= 9) {  // ---- the gather of cache rows
                __syncwarp();
                const int w = warp - 9;
                const int *table = p.c.table + (size_t)r.seq * p.c.width;
                constexpr int CH = e4m3 ? D / 16 : D / 8, RP = 32 / CH;  // 16-byte chunks of a row, rows a pass
                const int ch = lane % CH;
                // rows lane + 32 i of a key tile: their slots in the cache, -1 past the sequence and before the window
                auto find_slots = [&](int j, int (&slot)[4]) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = j * kBN + 32 * i + lane;
                        slot[i] = -1;
                        if (at >= g.kvlen || at < g.least) continue;
                        const int pg = at / p.c.page, id = table[pg];
                        if (id >= 0 && id < p.c.num_pages) slot[i] = id * p.c.page + (at - pg * p.c.page);
                        else atomicExch(p.status, kStatusBadPages);
                    }
                };
                // copies this warp's share of 64 rows, slots s0 and s1 of each lane; put(row) says where a chunk goes
                auto copy = [&](int s0, int s1, const void *cache, auto put) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll 4
                        for (int q = (w + i) % kGather; q < CH; q += kGather) {  // 32 rows are CH passes
                            const int in = q * RP + lane / CH, s = __shfl_sync(0xffffffffu, i ? s1 : s0, in);
                            const char *from = static_cast<const char *>(cache) + ((size_t)max(s, 0) * p.Hkv + hk) * (CH * 16) + ch * 16;
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(put(32 * i + in))), "l"(from),
                                         "r"(s >= 0 ? 16 : 0)
                                         : "memory");
                        }
                };
                int slot[4];
                bool ok = true;
                if constexpr (!e4m3) {
                    // straight into the tiles; a stage's barrier counts every thread's copies as they land
                    for (int j = g.jb; ok && j < g.je; ++j) {
                        const int it = j - g.jb, st = it % C::ST;
                        const uint32_t par = ((it / C::ST) & 1) ^ 1;
                        find_slots(j, slot);
#pragma unroll 1
                        for (int isv = 0; isv < 2; ++isv) {
                            if (it >= C::ST && !(ok = wait_warp(isv ? &v_empty[st] : &k_empty[st], par, &s_abort, p.status))) break;
                            char *dst = (isv ? sv : sk) + st * C::TILE + (ch >> 3) * kBoxBytes;
                            const void *cache = isv ? p.c.v : p.c.k;
                            copy(slot[0], slot[1], cache, [&](int row) { return dst + sw128(row, (ch & 7) * 16); });
                            copy(slot[2], slot[3], cache, [&](int row) { return dst + sw128(64 + row, (ch & 7) * 16); });
                            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                                             smem_u32(isv ? &v_full[st] : &k_full[st]))
                                         : "memory");
                        }
                    }
                } else {
                    // by way of raw rows in shared memory, 64 a step (K, K, V, V of a tile), two steps' copies in
                    // flight while a third becomes bf16; a lane converts the chunks that it has copied
                    char *raw8 = sv + C::ST * C::TILE;
                    auto fetch = [&](int h) {
                        if (h < 4 * (g.je - g.jb)) {
                            if (!(h & 3)) find_slots(g.jb + h / 4, slot);
                            char *dst = raw8 + h % 3 * kRawBytes<D> + ch * 16;
                            copy(h & 1 ? slot[2] : slot[0], h & 1 ? slot[3] : slot[1], h & 2 ? p.c.v : p.c.k,
                                 [&](int row) { return dst + row * D; });
                        }
                        asm volatile("cp.async.commit_group;" ::: "memory");
                    };
                    fetch(0);
                    fetch(1);
                    for (int h = 0; ok && h < 4 * (g.je - g.jb); ++h) {
                        const int it = h / 4, isv = h & 2, st = it % C::ST;
                        if (!(h & 1) && it >= C::ST &&
                            !(ok = wait_warp(isv ? &v_empty[st] : &k_empty[st], ((it / C::ST) & 1) ^ 1, &s_abort, p.status)))
                            break;
                        if (!(h & 3)) {
                            // Stage it % SS of the scales is free: with key stage `it` empty S of tile it - ST is
                            // formed, before which the weights of tile it - ST - 2 = it - SS were handed over (with
                            // P over S even those of the tile after).
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (i % kGather != w) continue;
                                const size_t from = (size_t)max(slot[i], 0) * p.Hkv + hk;
                                s_ks[it % SS][32 * i + lane] = slot[i] >= 0 ? p.c.ks[from] : 0.f;
                                s_vs[it % SS][32 * i + lane] = slot[i] >= 0 ? p.c.vs[from] : 0.f;
                            }
                        }
                        fetch(h + 2);
                        asm volatile("cp.async.wait_group 2;" ::: "memory");
                        const char *src = raw8 + h % 3 * kRawBytes<D> + ch * 16;
                        char *dst = (isv ? sv : sk) + st * C::TILE + (ch >> 2) * kBoxBytes;
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll 2
                            for (int q = (w + i) % kGather; q < CH; q += kGather) {
                                const int in = 32 * i + q * RP + lane / CH, row = 64 * (h & 1) + in;
                                const uint4 x = *reinterpret_cast<const uint4 *>(src + in * D);
                                uint32_t z[8];
                                e4m3x4_bf16(x.x, z[0], z[1]);
                                e4m3x4_bf16(x.y, z[2], z[3]);
                                e4m3x4_bf16(x.z, z[4], z[5]);
                                e4m3x4_bf16(x.w, z[6], z[7]);
                                *reinterpret_cast<uint4 *>(dst + sw128(row, (ch & 3) * 32)) = make_uint4(z[0], z[1], z[2], z[3]);
                                *reinterpret_cast<uint4 *>(dst + sw128(row, (ch & 3) * 32 + 16)) = make_uint4(z[4], z[5], z[6], z[7]);
                            }
                        fence_proxy_async_smem();
                        if (h & 1) mbar_arrive(isv ? &v_full[st] : &k_full[st]);
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
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

template <int D, int kind> cudaError_t run(const FwdMaps &maps, const FwdParams &p, dim3 grid, cudaStream_t s)
{
    auto kernel = attn_fwd_tc_kernel<D, kind>;
    constexpr int smem = Cfg<D>::SMEM + (kind == kPagedE4m3 ? 3 * kRawBytes<D> : 0);
    cudaError_t e = set_smem_attr(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, smem, s>>>(maps, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_fwd_tc(const AttnArgs &a, cudaStream_t s)
{
    FwdMaps maps;
    FwdParams p{};
    p.b = a.b;
    p.H = a.H;
    p.Hkv = a.Hkv;
    p.G = a.H / a.Hkv;
    p.TQ = kBM / p.G;
    p.window = a.window;
    p.splits = 1;
    p.scale = a.scale;
    p.o = (__nv_bfloat16 *)a.o;
    p.lse = a.lse;
    p.status = a.status;
    if (!make_head_map(&maps.q, a.q, a.b.rows, a.H, a.D, p.G, p.TQ) ||
        !make_head_map(&maps.k, a.k, a.b.rows, a.Hkv, a.D, 1, kBN) ||
        !make_head_map(&maps.v, a.v, a.b.rows, a.Hkv, a.D, 1, kBN))
        return cudaErrorInvalidValue;
    const long long blocks = tile_bound(a.b, 2 * p.TQ) * a.Hkv;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks);
    return a.D == 128 ? run<128, kWhole>(maps, p, grid, s) : run<64, kWhole>(maps, p, grid, s);
}

cudaError_t launch_attn_cached_tc(const CachedArgs &a, cudaStream_t s)
{
    FwdMaps maps;
    FwdParams p{};
    p.b = a.b;
    p.H = a.H;
    p.Hkv = a.Hkv;
    p.G = a.H / a.Hkv;
    p.TQ = kBM / p.G;
    p.window = a.window;
    p.splits = a.splits;
    p.scale = a.scale;
    p.o = (__nv_bfloat16 *)a.o;
    p.lse = a.lse;
    p.status = a.status;
    p.c = a.c;
    p.part_o = a.part_o;
    p.part_l = a.part_l;
    if (!make_head_map(&maps.q, a.q, a.b.rows, a.H, a.D, p.G, p.TQ)) return cudaErrorInvalidValue;
    maps.k = maps.v = maps.q;  // not read, but by kPaged
    p.box = kBN;
    while (p.box > 1 && a.c.page % p.box) p.box >>= 1;
    if (!a.c.e4m3 && p.box >= 8 &&
        (!make_head_map(&maps.k, a.c.k, (long long)a.c.num_pages * a.c.page, a.Hkv, a.D, 1, p.box) ||
         !make_head_map(&maps.v, a.c.v, (long long)a.c.num_pages * a.c.page, a.Hkv, a.D, 1, p.box)))
        return cudaErrorInvalidValue;
    const long long blocks = tile_bound(a.b, 2 * p.TQ) * a.Hkv * a.splits;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks);
    if (a.c.e4m3) return a.D == 128 ? run<128, kPagedE4m3>(maps, p, grid, s) : run<64, kPagedE4m3>(maps, p, grid, s);
    if (p.box >= 8) return a.D == 128 ? run<128, kPaged>(maps, p, grid, s) : run<64, kPaged>(maps, p, grid, s);
    return a.D == 128 ? run<128, kPagedAny>(maps, p, grid, s) : run<64, kPagedAny>(maps, p, grid, s);
}

}  // namespace gdn2
