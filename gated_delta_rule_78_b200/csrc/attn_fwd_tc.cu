// Causal attention forward on the tensor cores (bf16): whole sequences (keys by TMA) and the newest
// tokens of sequences over a paged cache (keys gathered page by page).
//
//   s_ij = scale q_i . k_j (visible j),  o_i = sum_j 2^(c s'_ij - m_i) v_j / l_i with c = scale log2 e
//
// One pass over the keys with a running reference m_i and sum l_i.  The reference follows the
// maximum only when a row's maximum has grown by more than 2^8 since: sums and outputs then stay
// far from overflow in fp32, and the accumulator is rescaled a few times a row instead of once a
// tile.  The weights are rounded to bf16 for the second product (their sum l_i is of the unrounded
// ones); that costs 2^-9 of each weight, no more than the rounding of o.
//
// A block owns two tiles A and B of 128 packed query rows.  Roles: warps 0-3 and 4-7 the softmax of
// A and of B (a thread to a row), warp 8 the products, warp 9 the TMA loads, warps 12-15 (paged
// only) the gather of pages.  The tensor core works on one tile's S = Q K^T and O += P V while the
// other tile's warps form its weights; P overwrites its own S in TMEM.  TMEM: S_A, S_B (128 columns
// each), O_A, O_B (D columns each).
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
    static constexpr int SMEM = 2 * TILE + 2 * ST * TILE + 1024;
};
constexpr int kTmS = 0, kTmO = 256;  // TMEM columns: S_A, S_B; O_A, O_B
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
    PagedCache c;       // paged only
    float *part_o, *part_l;
};

// The key tiles that a block works on, and each query tile's share of them.
struct Ranges {
    int first, kvlen;        // position of the sequence's query token 0; keys
    int t0[2], n[2];         // first token of tile A / B in the sequence, tokens in it
    int beg[2], end[2];      // its key tiles
    int jb, je;              // their union
};
__device__ __forceinline__ Ranges make_ranges(const FwdParams &p, const TileRef &r, int kvlen, int split)
{
    Ranges g;
    g.kvlen = kvlen;
    g.first = kvlen - r.sp.len;
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

// Where the keys come from: whole sequences by TMA, or a paged cache's bf16 or e4m3 rows
enum { kWhole, kPaged, kPagedE4m3 };

template <int D, int kind>
__global__ void __launch_bounds__(kind != kWhole ? 512 : 384, 1) attn_fwd_tc_kernel(const __grid_constant__ FwdMaps maps,
                                                                          const __grid_constant__ FwdParams p)
{
    using C = Cfg<D>;
    constexpr bool paged = kind != kWhole, e4m3 = kind == kPagedE4m3;
    constexpr int SS = C::ST + 1;  // stages of the scales: see the gather
    extern __shared__ char raw[];
    char *sm = reinterpret_cast<char *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    char *sq = sm, *sk = sm + 2 * C::TILE, *sv = sk + C::ST * C::TILE;
    __shared__ __align__(8) uint64_t bar_q, k_full[C::ST], k_empty[C::ST], v_full[C::ST], v_empty[C::ST], s_full[2],
        p_ready[2], o_done[2], bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ float s_ks[e4m3 ? SS : 1][kBN], s_vs[e4m3 ? SS : 1][kBN];
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && warp == 0) report_bad_seqlens(p.b, p.status);
    TileRef r;
    if (!find_tile(p.b, gridDim.x - 1 - blockIdx.x, 2 * p.TQ, r)) return;
    int kvlen = r.sp.len;
    if (paged) {
        kvlen = p.c.kv_lens[r.seq];
        if (kvlen < r.sp.len || kvlen > (long long)p.c.width * p.c.page) {
            if (tid == 0) atomicExch(p.status, kStatusBadPages);
            return;
        }
    }
    const Ranges g = make_ranges(p, r, kvlen, blockIdx.z);
    const int hk = blockIdx.y;

    if (tid == 0) {
        s_abort = 0;
        mbar_init(&bar_q, 1);
        mbar_init(&bar_drain, 1);
        for (int i = 0; i < C::ST; ++i) {
            mbar_init(&k_full[i], paged ? 128 : 1);
            mbar_init(&v_full[i], paged ? 128 : 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s_full[x], 1);
            mbar_init(&p_ready[x], 4);
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
        if constexpr (paged) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int x = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
        const uint32_t ts = tmem + kTmS + 128 * x + lanes, to = tmem + kTmO + D * x + lanes;
        const int tok = row / p.G, gq = row - tok * p.G;
        const int pos = g.first + g.t0[x] + tok;
        const int low = g.first + g.t0[x], high = low + g.n[x] - 1;
        const float c = p.scale * kLog2e;
        float m = -INFINITY, l = 0.f;  // reference in units of s, sum of the weights relative to it
        bool ok = true;
        uint32_t ph = 0;
        for (int j = g.beg[x]; j < g.end[x]; ++j, ph ^= 1) {
            if (!(ok = wait_warp(&s_full[x], ph, &s_abort, p.status))) break;
            tc_fence_after();
            float s[128];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, reinterpret_cast<uint32_t(&)[32]>(s[32 * q]));
            tmem_wait_ld();
            const int k0 = j * kBN;
            const float *vs = s_vs[0];
            if constexpr (e4m3) {
                const float *ks = s_ks[(j - g.jb) % SS];
                vs = s_vs[(j - g.jb) % SS];
#pragma unroll
                for (int i = 0; i < 128; ++i) s[i] *= ks[i];
            }
            if (k0 + kBN - 1 > low || (p.window && k0 <= high - p.window)) {
                const int most = pos - k0, least = p.window ? most - p.window + 1 : 0;
#pragma unroll
                for (int i = 0; i < 128; ++i) s[i] = i <= most && i >= least ? s[i] : -INFINITY;
            }
            float t0 = s[0], t1 = s[1], t2 = s[2], t3 = s[3];
#pragma unroll
            for (int i = 4; i < 128; i += 4) {
                t0 = fmaxf(t0, s[i]);
                t1 = fmaxf(t1, s[i + 1]);
                t2 = fmaxf(t2, s[i + 2]);
                t3 = fmaxf(t3, s[i + 3]);
            }
            const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3));
            const bool grow = (top - m) * c > kGrow;  // true for the row's first visible key (m = -inf)
            if (__any_sync(0xffffffffu, grow)) {
                const float f = grow ? ex2((m - top) * c) : 1.f;
                if (grow) m = top;
                l *= f;
                if (j > g.beg[x]) {  // the previous product is done: its commit came before this S
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
            float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float a = ex2(fmaf(s[64 * q + 2 * i], c, off)), b = ex2(fmaf(s[64 * q + 2 * i + 1], c, off));
                    sum0 += a;
                    sum1 += b;
                    if constexpr (e4m3) w[i] = pack_bf16x2(a * vs[64 * q + 2 * i], b * vs[64 * q + 2 * i + 1]);
                    else w[i] = pack_bf16x2(a, b);
                }
                tmem_st32(ts + 32 * q, w);
            }
            l += sum0 + sum1;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[x]);
        }
        const bool any = g.beg[x] < g.end[x];
        if (any && ok) ok = wait_warp(&o_done[x], 0, &s_abort, p.status);
        if (ok && g.n[x] > 0) {  // (warp-uniform) o = O / l
            tc_fence_after();
            const bool live = row < p.TQ * p.G && tok < g.n[x];
            const size_t at = (size_t)(r.sp.bos + g.t0[x] + tok) * p.H + hk * p.G + gq;
            const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            const float lse = l > 0.f || l != l ? (m * c + __log2f(l)) * kLn2 : -INFINITY;
            const size_t base = p.splits > 1 ? ((size_t)blockIdx.z * p.b.rows * p.H + at) : at;
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
                if (p.splits > 1) {
                    float *dst = p.part_o + base * D + 32 * q;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        const uint32_t v[8] = {w[i], w[i + 1], w[i + 2], w[i + 3], w[i + 4], w[i + 5], w[i + 6], w[i + 7]};
                        store32(dst + i, v);
                    }
                } else {
                    __nv_bfloat16 *dst = p.o + base * D + 32 * q;
#pragma unroll
                    for (int i = 0; i < 32; i += 16) {
                        uint32_t v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[e] = pack_bf16x2(__uint_as_float(w[i + 2 * e]), __uint_as_float(w[i + 2 * e + 1]));
                        store32(dst + i, v);
                    }
                }
            }
            if (live) {
                if (p.splits > 1) p.part_l[base] = lse;
                else if (p.lse) p.lse[base] = lse;
            }
        }
    } else if (warp < 12) {
        if constexpr (paged) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const uint32_t bq = smem_u32(sq), bk = smem_u32(sk), bv = smem_u32(sv);
        if (warp == 8) {  // ---- the products
            constexpr uint32_t kS = idesc_bf16(128, kBN, 0, 0), kO = idesc_bf16(128, D, 0, 1);
            bool ok = g.je > g.jb && wait_warp(&bar_q, 0, &s_abort, p.status);
            const uint32_t leader = elect();
            uint32_t ph[2] = {0, 0};
            const int jb = uniform(g.jb), je = uniform(g.je), kvlen = uniform(g.kvlen);
            const int beg[2] = {uniform(g.beg[0]), uniform(g.beg[1])}, end[2] = {uniform(g.end[0]), uniform(g.end[1])};
            for (int j = jb - 1; ok && j < je; ++j) {
                const int it = j - jb, nx = it + 1;  // key tile j and the next one in the rings
                bool have_v = false, have_k = false;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (j >= beg[x] && j < end[x]) {
                        if (!have_v) {
                            if (!(ok = wait_warp(&v_full[it % C::ST], (it / C::ST) & 1, &s_abort, p.status))) break;
                            // rows past the sequence hold other sequences' values: 0 * NaN is not 0
                            if (!paged && (j + 1) * kBN > kvlen) zero_rows<C::NB>(sv + (it % C::ST) * C::TILE, kvlen - j * kBN);
                            have_v = true;
                        }
                        if (!(ok = wait_warp(&p_ready[x], ph[x], &s_abort, p.status))) break;
                        ph[x] ^= 1;
                        tc_fence_after();
                        mma_tn<32>(leader, tmem + kTmO + D * x, tmem + kTmS + 128 * x, bv + (it % C::ST) * C::TILE, kO, j > beg[x]);
                        if (j + 1 == end[x]) commit(leader, &o_done[x]);
                    }
                    if (j + 1 >= beg[x] && j + 1 < end[x]) {
                        if (!have_k) {
                            if (!(ok = wait_warp(&k_full[nx % C::ST], (nx / C::ST) & 1, &s_abort, p.status))) break;
                            have_k = true;
                        }
                        tc_fence_after();
                        mma_kk<D / 16>(leader, tmem + kTmS + 128 * x, bq + x * C::TILE, bk + (nx % C::ST) * C::TILE, kS);
                        commit(leader, &s_full[x]);
                    }
                }
                if (ok) {
                    if (have_v) commit(leader, &v_empty[it % C::ST]);
                    if (have_k) commit(leader, &k_empty[nx % C::ST]);
                }
            }
            if (s_abort) drain(leader, &bar_drain);
        } else if (warp == 9 && lane == 0 && g.je > g.jb) {  // ---- TMA loads
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
            bool ok = true;
            int nk = 0, nv = 0;
            if constexpr (!paged) {
                for (int j = g.jb; ok && j < g.je; ++j) {
                    const int it = j - g.jb, s = it % C::ST;
                    const uint32_t par = ((it / C::ST) & 1) ^ 1;
                    if (it >= C::ST && !(ok = wait(&k_empty[s], par, &s_abort, p.status))) break;
                    mbar_expect_tx(&k_full[s], C::TILE);
#pragma unroll
                    for (int b = 0; b < C::NB; ++b)
                        tma_load_3d(sk + s * C::TILE + b * kBoxBytes, &maps.k, 64 * b, hk, r.sp.bos + j * kBN, &k_full[s]);
                    ++nk;
                    if (it >= C::ST && !(ok = wait(&v_empty[s], par, &s_abort, p.status))) break;
                    mbar_expect_tx(&v_full[s], C::TILE);
#pragma unroll
                    for (int b = 0; b < C::NB; ++b)
                        tma_load_3d(sv + s * C::TILE + b * kBoxBytes, &maps.v, 64 * b, hk, r.sp.bos + j * kBN, &v_full[s]);
                    ++nv;
                }
            }
            // after a wait that gave up, loads in flight end before the block's memory is free
            if (s_abort) {
                mbar_wait(&bar_q, 0, 1000000000ull);
                for (int i = max(0, nk - C::ST); i < nk; ++i) mbar_wait(&k_full[i % C::ST], (i / C::ST) & 1, 1000000000ull);
                for (int i = max(0, nv - C::ST); i < nv; ++i) mbar_wait(&v_full[i % C::ST], (i / C::ST) & 1, 1000000000ull);
            }
        }
    } else if constexpr (paged) {  // ---- the gather of cache rows, 32 rows of a tile to a warp
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        const int w4 = warp - 12;
        const int *table = p.c.table + (size_t)r.seq * p.c.width;
        // row w4 * 32 + lane of key tile j: its slot in the cache, -1 past the sequence
        auto slot_of = [&](int j) {
            const int at = j * kBN + w4 * 32 + lane;
            if (at >= g.kvlen) return -1;
            const int pg = at / p.c.page, id = table[pg];
            if (id < 0 || id >= p.c.num_pages) {
                atomicExch(p.status, kStatusBadPages);
                return -1;
            }
            return id * p.c.page + (at - pg * p.c.page);
        };
        bool ok = true;
        for (int j = g.jb; ok && j < g.je; ++j) {
            const int it = j - g.jb, st = it % C::ST;
            const uint32_t par = ((it / C::ST) & 1) ^ 1;
            const int slot = slot_of(j);
            if (it >= C::ST && !(ok = wait_warp(&k_empty[st], par, &s_abort, p.status))) break;
            if constexpr (e4m3) {
                // Stage it % SS of the scales is free: key stage `it` being empty, tile it - ST has been
                // multiplied, for which the softmax of tile it - ST - 1 = it - SS was done.
                s_ks[it % SS][w4 * 32 + lane] = slot >= 0 ? p.c.ks[(size_t)slot * p.Hkv + hk] : 0.f;
                s_vs[it % SS][w4 * 32 + lane] = slot >= 0 ? p.c.vs[(size_t)slot * p.Hkv + hk] : 0.f;
            }
#pragma unroll 1
            for (int isv = 0; isv < 2; ++isv) {
                if (isv && it >= C::ST && !(ok = wait_warp(&v_empty[st], par, &s_abort, p.status))) break;
                char *dst = (isv ? sv : sk) + st * C::TILE;
                const char *src = static_cast<const char *>(isv ? p.c.v : p.c.k);
                if constexpr (!e4m3) {
                    constexpr int CH = D / 8, RP = 32 / CH;  // 16-byte chunks of a row, rows a pass
                    const int ch = lane % CH;
#pragma unroll
                    for (int i = 0; i < 32 / RP; ++i) {
                        const int row = i * RP + lane / CH, s = __shfl_sync(0xffffffffu, slot, row);
                        const char *from = src + (((size_t)max(s, 0) * p.Hkv + hk) * D + ch * 8) * 2;
                        const uint32_t to = smem_u32(dst + (ch >> 3) * kBoxBytes) + sw128(w4 * 32 + row, (ch & 7) * 16);
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(s >= 0 ? 16 : 0)
                                     : "memory");
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    // the copies before these have landed: V of the tile before, or K of this one
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                    fence_proxy_async_smem();
                    if (isv) mbar_arrive(&k_full[st]);
                    else if (it > 0) mbar_arrive(&v_full[(it - 1) % C::ST]);
                } else {
                    constexpr int CH = D / 16, RP = 32 / CH;  // 16 channels of 8 bits a lane
                    const int ch = lane % CH;
                    uint4 x[32 / RP];
#pragma unroll
                    for (int i = 0; i < 32 / RP; ++i) {
                        const int s = __shfl_sync(0xffffffffu, slot, i * RP + lane / CH);
                        x[i] = make_uint4(0, 0, 0, 0);
                        if (s >= 0) x[i] = *reinterpret_cast<const uint4 *>(src + ((size_t)s * p.Hkv + hk) * D + ch * 16);
                    }
#pragma unroll
                    for (int i = 0; i < 32 / RP; ++i) {
                        const int row = w4 * 32 + i * RP + lane / CH;
                        uint32_t y[8];
                        e4m3x4_bf16(x[i].x, y[0], y[1]);
                        e4m3x4_bf16(x[i].y, y[2], y[3]);
                        e4m3x4_bf16(x[i].z, y[4], y[5]);
                        e4m3x4_bf16(x[i].w, y[6], y[7]);
                        char *to = dst + (ch >> 2) * kBoxBytes;
                        *reinterpret_cast<uint4 *>(to + sw128(row, (ch & 3) * 32)) = make_uint4(y[0], y[1], y[2], y[3]);
                        *reinterpret_cast<uint4 *>(to + sw128(row, (ch & 3) * 32 + 16)) = make_uint4(y[4], y[5], y[6], y[7]);
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(isv ? &v_full[st] : &k_full[st]);
                }
            }
        }
        if constexpr (!e4m3) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            fence_proxy_async_smem();
            if (ok && g.je > g.jb) mbar_arrive(&v_full[(g.je - 1 - g.jb) % C::ST]);
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
    cudaError_t e = set_smem_attr(reinterpret_cast<const void *>(kernel), Cfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kind != kWhole ? 512 : 384, Cfg<D>::SMEM, s>>>(maps, p);
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
    const dim3 grid((unsigned)tile_bound(a.b, 2 * p.TQ), (unsigned)a.Hkv);
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
    maps.k = maps.v = maps.q;  // not read
    const dim3 grid((unsigned)tile_bound(a.b, 2 * p.TQ), (unsigned)a.Hkv, (unsigned)a.splits);
    if (a.c.e4m3) return a.D == 128 ? run<128, kPagedE4m3>(maps, p, grid, s) : run<64, kPagedE4m3>(maps, p, grid, s);
    return a.D == 128 ? run<128, kPaged>(maps, p, grid, s) : run<64, kPaged>(maps, p, grid, s);
}

}  // namespace gdn2
