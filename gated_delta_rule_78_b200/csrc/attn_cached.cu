// Attention of each sequence's newest tokens over the paged cache, few rows to a key head (decode
// steps), and the joining of parts.
//
// A decode step reads every visible key and value once and computes 4 D flop a pair for the G query
// heads of a key head: it is bound by memory.  A block takes 8 packed query rows (row r is token r / G,
// head r % G; 16 where sequences bring more than 8) and one part of the key axis; its 4 warps take key
// steps in turn, each with a ring of its own of cp.async stages, so that no warp waits for another
// until the end, where their sums are joined in shared memory.
//
// Products are m16n8k16 on transposed operands: S^T = K Q^T and O^T = V^T P^T, keys and channels in the
// 16 rows and queries in the 8 columns.  The other way round a decode step's few queries leave three
// quarters of the 16 rows empty, with twice the products, registers and exponentials.  (A 128-row tile of
// the fifth-generation tensor core would be emptier still, and the time is the loads'.)
//
// e4m3 rows go to shared memory as they are and become f16 in registers, one conversion to two values
// (by way of f32 to bf16 it would be four).  f16 holds every e4m3 value.  Its range asks for care on
// the other side: a query row is brought below 2^14 by a power of two (exact, but for channels below
// 2^-28 of the row's largest), and a key's weight p_j scale_j, e4m3's scale of the value with it, is kept
// below 2^14 by a reference of its own, which like the softmax's follows the largest when that has grown
// by 2^8: weights are off by 2^-11 of themselves or 2^-31 of the largest.
//
// Cut into parts, each part writes its normalised output and log-sum; a second kernel joins them,
// in a fixed order.
//
// 256 sequences of 256 to 8192 keys, 16 heads on 4, D = 128, e4m3: 129 us with the joining's 5 (4.7 TB/s; sequences
// alike, 2048 keys each: 98 us).  One sequence over 32768 keys, bf16: 18.5 and 5 us, launch and latency.
#include "attn_tc.cuh"

namespace gdn2 {
namespace {

using attn::ex2;
using attn::kLn2;
using attn::kLog2e;
using tc::pack_bf16x2;
using tc::smem_u32;

constexpr int kWarps = 4;
constexpr int kManyRows = 1024;  // rows of outputs that fill the SMs at a warp to a row
constexpr float kGrow = 8.f;    // growth of the maximum (log2) that moves the reference
constexpr float kWeight = 6.f;  // e4m3: log2 of the weight at the reference

template <int D, bool e4m3, int NQ> struct Cfg {
    static constexpr int ROWS = 8 * NQ;                    // query rows
    static constexpr int STEP = e4m3 ? 32 : 16;            // keys of a warp's step
    static constexpr int ROW = D * (e4m3 ? 1 : 2);         // bytes of a cache row
    static constexpr int TILE = STEP * ROW;                // a warp's K (or V) stage
    static constexpr int SCALES = e4m3 ? 2 * STEP * 4 : 0;
    static constexpr int STAGE = 2 * TILE + SCALES;
    static constexpr int ST = D == 128 ? (e4m3 ? 2 : 3) : (e4m3 ? 3 : 4);
    static constexpr int RING = kWarps * ST * STAGE;
    static constexpr int MERGE = kWarps * ROWS * (D + 4) * 4;  // the warps' outputs, over the rings
    static constexpr int SMEM = RING > MERGE ? RING : MERGE;
};

struct Params {
    SeqBatch b;
    int H, Hkv, G, window, splits, piece;
    float scale;
    PagedCache c;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    float *lse, *part_o, *part_l;
    int *status;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Four e4m3 values as two pairs of f16 (exact).
__device__ __forceinline__ void e4m3x4_f16(uint32_t x, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// the transpose of an 8 x 8 matrix of 16-bit values, a row to four lanes
__device__ __forceinline__ uint32_t transpose(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 16-byte chunk c of row r of a stage whose rows are 64, 128 or 256 bytes; the chunk index is
// permuted by the row so that the 8 rows of an ldmatrix lie in different banks
template <int ROW> __device__ __forceinline__ uint32_t chunk(int r, int c)
{
    if constexpr (ROW == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    else return r * ROW + ((c ^ (r & 7)) << 4);
}

// Block x < n is the first tile of sequence x; the others are the further tiles of sequences with
// more than `rows` rows, in order.  By a whole warp.
__device__ __forceinline__ bool find_rows(const Params &p, int x, int rows, TileRef &r)
{
    if (x < p.b.n) {
        r.seq = x;
        r.tile = 0;
        r.sp = batch_span(p.b, x);
        return r.sp.len > 0;
    }
    int e = x - p.b.n;
    const int lane = threadIdx.x & 31;
    for (int base = 0; base < p.b.n; base += 32) {
        SeqSpan sp = {0, -1};
        if (base + lane < p.b.n) sp = batch_span(p.b, base + lane);
        const int more = sp.len > 0 ? (int)(((long long)sp.len * p.G + rows - 1) / rows) - 1 : 0;
        int sum = more;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, m);
            if (lane >= m) sum += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, sum > e);
        if (hit) {
            const int src = __ffs(hit) - 1;
            r.seq = base + src;
            r.tile = 1 + e - __shfl_sync(0xffffffffu, sum - more, src);
            r.sp.bos = __shfl_sync(0xffffffffu, sp.bos, src);
            r.sp.len = __shfl_sync(0xffffffffu, sp.len, src);
            return true;
        }
        e -= __shfl_sync(0xffffffffu, sum, 31);
    }
    return false;
}

template <int D, bool e4m3, int NQ>
__global__ void __launch_bounds__(kWarps * 32) attn_rows_kernel(const __grid_constant__ Params p)
{
    using C = Cfg<D, e4m3, NQ>;
    constexpr int kStep = C::STEP, KT = kStep / 16, kRows = C::ROWS;  // keys of a step, tiles of 16 of them, query rows
    extern __shared__ __align__(128) char sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && warp == 0) report_bad_seqlens(p.b, p.status);
    TileRef r;
    if (!find_rows(p, blockIdx.x, kRows, r)) return;
    const int kvlen = p.c.kv_lens[r.seq];
    if (kvlen < r.sp.len || kvlen > (long long)p.c.width * p.c.page) {  // before any difference, which could wrap
        if (tid == 0) atomicExch(p.status, kStatusBadPages);
        return;
    }
    const int first = kvlen - r.sp.len;
    const int hk = blockIdx.y, r0 = r.tile * kRows, rows = min(kRows, r.sp.len * p.G - r0);
    // keys that this tile's rows see, and this block's part of them
    const int low = first + r0 / p.G, high = first + (r0 + rows - 1) / p.G;
    const int lo = p.window == 0 || low < p.window ? 0 : low - p.window + 1;
    const int kb = lo + (int)blockIdx.z * p.piece, ke = min(high + 1, kb + p.piece);
    const size_t part = (size_t)blockIdx.z * p.b.rows * p.H;
    auto row_at = [&](int row) {  // [rows, H] index of the tile's row
        const int rr = r0 + row, tok = rr / p.G;
        return (size_t)(r.sp.bos + tok) * p.H + hk * p.G + (rr - tok * p.G);
    };
    if (kb >= ke) {  // nothing in this part (one part alone has keys: part_l may be null then)
        if (p.splits > 1 && tid < rows) p.part_l[part + row_at(tid)] = -INFINITY;
        return;
    }

    const int *table = p.c.table + (size_t)r.seq * p.c.width;
    char *ring = sm + warp * C::ST * C::STAGE;
    const int nsteps = (ke - kb + kStep - 1) / kStep, mine = nsteps > warp ? (nsteps - warp + kWarps - 1) / kWarps : 0;
    // The keys of this warp's step i, from kb + kStep (warp + 4 i) on, go into its stage i % ST; rows past
    // the part and rows of bad pages become zeros.  Lane l looks up row l % kStep: `pg` and `in` are its
    // page and place for the next step to load, carried from step to step without a division, and `id` is
    // that page's table entry, read a step ahead.
    constexpr int CH = C::ROW / 16, RP = 32 / CH;
    const int ch = lane % CH;
    const char *kbase = (const char *)p.c.k + (size_t)hk * C::ROW + ch * 16, *vbase = (const char *)p.c.v + (size_t)hk * C::ROW + ch * 16;
    const uint32_t rowbytes = (uint32_t)p.Hkv * C::ROW;
    const uint32_t to0 = smem_u32(ring) + chunk<C::ROW>(lane / CH, ch);
    int at = kb + kStep * warp + lane % kStep, pg = at / p.c.page, in = at - pg * p.c.page;
    const int dpg = kStep * kWarps / p.c.page, din = kStep * kWarps - dpg * p.c.page;
    int id = at < ke ? table[pg] : -1;
    auto load = [&](int i) {
        if (i < mine) {
            int slot = -1;
            if (at < ke) {
                if (id >= 0 && id < p.c.num_pages) slot = id * p.c.page + in;
                else atomicExch(p.status, kStatusBadPages);
            }
            at += kStep * kWarps;
            pg += dpg;
            in += din;
            if (in >= p.c.page) {
                in -= p.c.page;
                ++pg;
            }
            id = at < ke ? table[pg] : -1;
            const uint32_t st = (uint32_t)(i % C::ST) * C::STAGE;
#pragma unroll
            for (int x = 0; x < kStep / RP; ++x) {
                const int s = __shfl_sync(0xffffffffu, slot, x * RP + lane / CH);
                const size_t off = (size_t)(uint32_t)max(s, 0) * rowbytes;
                // the chunk permutation repeats every 8 rows
                const uint32_t to = RP % 8 == 0 ? to0 + st + x * RP * C::ROW : smem_u32(ring) + st + chunk<C::ROW>(x * RP + lane / CH, ch);
                const uint32_t n = s >= 0 ? 16 : 0;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(kbase + off), "r"(n) : "memory");
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + C::TILE), "l"(vbase + off), "r"(n) : "memory");
            }
            if constexpr (e4m3) {
                const size_t off = (size_t)max(slot, 0) * p.Hkv + hk;
                const uint32_t to = smem_u32(ring) + st + 2 * C::TILE + 4 * lane, n = slot >= 0 ? 4 : 0;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(p.c.ks + off), "r"(n) : "memory");
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + 4 * kStep), "l"(p.c.vs + off), "r"(n) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < C::ST - 1; ++i) load(i);

    // Q fragments: column g of each tile of 8 queries.  e4m3 keys come four channels to a lane (see below),
    // so there a lane's k indices 2t, 2t+1, 2t+8, 2t+9 stand for channels 4t .. 4t+3; a sum has no order.
    uint32_t qf[D / 16][NQ][2];
    float cq[NQ][2];  // scale log2 e (and a row's power of two) of columns 2t, 2t + 1
    int pos[NQ][2];   // their positions
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const __nv_bfloat16 *q = p.q + row_at(min(g + 8 * n, rows - 1)) * D;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                qf[k][n][e] = *reinterpret_cast<const uint32_t *>(q + 16 * k + (e4m3 ? 4 * t + 2 * e : 2 * t + 8 * e));
        float back = 1.f;
        if constexpr (e4m3) {  // f16 of q 2^-x, x from the row's largest finite exponent
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t w = qf[k][n][e], lo = (w >> 7) & 0xffu, hi = (w >> 23) & 0xffu;
                    top = max(top, max(lo < 255u ? lo : 0u, hi < 255u ? hi : 0u));
                }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int x = min(max((int)top - 127 - 13, -120), 120);
            const float f = __uint_as_float((uint32_t)(127 - x) << 23);
            back = __uint_as_float((uint32_t)(127 + x) << 23);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t w = qf[k][n][e];
                    qf[k][n][e] = pack_f16x2(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
                }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int row = 2 * t + x + 8 * n;
            cq[n][x] = p.scale * kLog2e * __shfl_sync(0xffffffffu, back, 4 * (2 * t + x));
            pos[n][x] = row < rows ? first + (r0 + row) / p.G : -1;
        }
    }

    // m: reference of the sums l, wm: of the outputs o (the same without a scale of values); log2.  All of a
    // column's lanes hold the same references, each its own keys' share of the sum.
    float o[D / 16][NQ][4], m[NQ][2], wm[NQ][2], l[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][n][e] = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            m[n][x] = wm[n][x] = -INFINITY;
            l[n][x] = 0.f;
        }
    }
    const int edge = min(ke, low + 1);  // keys below it are seen by every row, but for a window
    for (int i = 0; i < mine; ++i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(C::ST - 2) : "memory");
        __syncwarp();
        load(i + C::ST - 1);
        const uint32_t sk = smem_u32(ring + (i % C::ST) * C::STAGE), sv = sk + C::TILE;
        float s[KT][NQ][4] = {};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t b[4];
            if constexpr (!e4m3) {
                // matrices: keys 0-7 / 8-15 (lane bit 3) x channels 16k .. +7 / +8 .. +15 (lane bit 4)
                ldm4(b, sk + chunk<C::ROW>((lane & 7) + (lane & 8), 2 * k + (lane >> 4)));
#pragma unroll
                for (int n = 0; n < NQ; ++n) mma_bf16(s[0][n], b, qf[k][n][0], qf[k][n][1]);
            } else {
                // keys 0-7 .. 24-31 (lane / 8) x the 16 channels of step k: a lane gets channels 4t .. 4t + 3
                // of keys g, g + 8, ..
                ldm4(b, sk + chunk<C::ROW>(lane, k));
#pragma unroll
                for (int h = 0; h < KT; ++h) {
                    uint32_t a[4];
                    e4m3x4_f16(b[2 * h], a[0], a[2]);
                    e4m3x4_f16(b[2 * h + 1], a[1], a[3]);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) mma_f16(s[h][n], a, qf[k][n][0], qf[k][n][1]);
                }
            }
        }
        // s[h][n][e]: key 16 h + g + 8 (e / 2), query 8 n + 2t + e % 2
        const float *sc = reinterpret_cast<const float *>(ring + (i % C::ST) * C::STAGE + 2 * C::TILE);
        float lv[KT][2];  // log2 of the values' scales
#pragma unroll
        for (int h = 0; h < KT; ++h)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float f = 1.f;
                if constexpr (e4m3) {
                    f = sc[16 * h + 8 * y + g];
                    lv[h][y] = __log2f(sc[kStep + 16 * h + 8 * y + g]);
                }
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x) s[h][n][2 * y + x] *= e4m3 ? f * cq[n][x] : cq[n][x];
            }
        // only the steps at the part's ends, the newest keys and a window's edge hide a key from a row
        const int kstep = kb + kStep * (warp + kWarps * i);
        if (kstep + kStep > edge || (p.window && kstep <= high - p.window)) {
#pragma unroll
            for (int h = 0; h < KT; ++h)
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = kstep + 16 * h + g + 8 * (e >> 1), row = pos[n][e & 1];
                        const bool vis = key <= row && key < ke && (p.window == 0 || key > row - p.window);
                        s[h][n][e] = vis ? s[h][n][e] : -INFINITY;
                    }
        }
        bool move = false, grow[NQ][2], wgrow[NQ][2];
        float top[NQ][2], wtop[NQ][2];  // the largest score; the largest log2 weight (e4m3: with the value's scale)
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float a = m[n][x], w = wm[n][x];
#pragma unroll
                for (int h = 0; h < KT; ++h)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        a = fmaxf(a, s[h][n][2 * y + x]);
                        if constexpr (e4m3) w = fmaxf(w, s[h][n][2 * y + x] + lv[h][y]);
                    }
#pragma unroll
                for (int z = 4; z < 32; z <<= 1) {
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, z));
                    if constexpr (e4m3) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, z));
                }
                top[n][x] = a;
                wtop[n][x] = e4m3 ? w : a;
                grow[n][x] = a - m[n][x] > kGrow;  // true for the row's first visible key (m = -inf)
                wgrow[n][x] = e4m3 ? w - wm[n][x] > kGrow : grow[n][x];
                move |= grow[n][x] || wgrow[n][x];
            }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (grow[n][x]) {
                        l[n][x] *= ex2(m[n][x] - top[n][x]);
                        m[n][x] = top[n][x];
                    }
                    const float f = wgrow[n][x] ? ex2(wm[n][x] - wtop[n][x]) : 1.f;
                    if (wgrow[n][x]) wm[n][x] = wtop[n][x];
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        o[d][n][x] *= f;
                        o[d][n][2 + x] *= f;
                    }
                }
        }
        uint32_t pf[KT][NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            float off[2], woff[2];  // no key visible yet: all weights 0
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                off[x] = m[n][x] == -INFINITY ? 0.f : m[n][x];
                woff[x] = wm[n][x] == -INFINITY ? 0.f : wm[n][x] - kWeight;
            }
#pragma unroll
            for (int h = 0; h < KT; ++h)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float a = ex2(s[h][n][2 * y] - off[0]), b = ex2(s[h][n][2 * y + 1] - off[1]);
                    l[n][0] += a;
                    l[n][1] += b;
                    if constexpr (e4m3) {
                        a = ex2(s[h][n][2 * y] + lv[h][y] - woff[0]);
                        b = ex2(s[h][n][2 * y + 1] + lv[h][y] - woff[1]);
                        pf[h][n][y] = transpose(pack_f16x2(a, b));
                    } else {
                        pf[h][n][y] = transpose(pack_bf16x2(a, b));
                    }
                }
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            uint32_t b[4];
            if constexpr (!e4m3) {
                // keys 0-7 / 8-15 (lane bit 4) x channels 16d .. +7 / +8 .. +15 (lane bit 3), transposed
                ldm4t(b, sv + chunk<C::ROW>((lane & 7) + ((lane >> 1) & 8), 2 * d + ((lane >> 3) & 1)));
#pragma unroll
                for (int n = 0; n < NQ; ++n) mma_bf16(o[d][n], b, pf[0][n][0], pf[0][n][1]);
            } else {
                // keys 0-7 .. 24-31 x 16 channels 16d .. in pairs of bytes: a lane gets channels 2g and 2g + 1 of
                // keys 2t and 2t + 1 (+ 8, ..), so rows 0-7 of the output tile are the even channels, 8-15 the odd
                ldm4t(b, sv + chunk<C::ROW>(lane, d));
#pragma unroll
                for (int h = 0; h < KT; ++h) {
                    uint32_t a[4];
                    e4m3x4_f16(__byte_perm(b[2 * h], 0, 0x3120), a[0], a[1]);
                    e4m3x4_f16(__byte_perm(b[2 * h + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) mma_f16(o[d][n], a, pf[h][n][0], pf[h][n][1]);
                }
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // the joining kernel may be brought to the SMs; it waits there for this one's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // ---- the warps' sums joined: O and (m, l) of each warp over the rings
    __syncthreads();
    float *so = reinterpret_cast<float *>(sm);
    __shared__ float s_m[kWarps][kRows], s_w[kWarps][kRows], s_l[kWarps][kRows];
    constexpr int OS = D + 4;
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int row = 8 * n + 2 * t + x;
            float *dst = so + (warp * kRows + row) * OS;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                if constexpr (e4m3) {
                    *reinterpret_cast<float2 *>(dst + 16 * d + 2 * g) = make_float2(o[d][n][x], o[d][n][2 + x]);
                } else {
                    dst[16 * d + g] = o[d][n][x];
                    dst[16 * d + 8 + g] = o[d][n][2 + x];
                }
            }
            float sum = l[n][x];
#pragma unroll
            for (int z = 4; z < 32; z <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, z);
            if (g == 0) {
                s_m[warp][row] = m[n][x];
                s_w[warp][row] = e4m3 ? wm[n][x] - kWeight : m[n][x];
                s_l[warp][row] = sum;
            }
        }
    __syncthreads();
    for (int i = tid; i < rows * (D / 4); i += kWarps * 32) {
        const int row = i / (D / 4), ch = i % (D / 4) * 4;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][row]);
        const float base = top == -INFINITY ? 0.f : top;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            // a value's scale can be far from 1, so that 2^(s_w - base) alone may leave fp32's range where
            // its product with o does not: half of it on either side
            const float f = ex2(0.5f * (s_w[w][row] - base));
            const float4 v = *reinterpret_cast<const float4 *>(so + (w * kRows + row) * OS + ch);
            sum += ex2(s_m[w][row] - base) * s_l[w][row];
            acc.x += f * v.x * f;
            acc.y += f * v.y * f;
            acc.z += f * v.z * f;
            acc.w += f * v.w * f;
        }
        const bool some = sum > 0.f || sum != sum;
        const float inv = some ? 1.f / sum : 0.f, lse = some ? (top + __log2f(sum)) * kLn2 : -INFINITY;
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        const size_t at = row_at(row);
        if (p.splits > 1) {
            *reinterpret_cast<float4 *>(p.part_o + (part + at) * D + ch) = acc;
            if (ch == 0) p.part_l[part + at] = lse;
        } else {
            *reinterpret_cast<uint2 *>(p.o + at * D + ch) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
            if (ch == 0 && p.lse) p.lse[at] = lse;
        }
    }
}

// o = sum_z e^(lse_z - top) o_z / sum_z e^(lse_z - top) over the parts z, in a fixed order.  A warp
// to a (token, head) row, or a block of 8 warps where there are many parts (few rows, then: the warps
// take every 8th part).  Rows of no sequence, or of one that was skipped, are left as they are.
template <int D, int W> __global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ Params p)
{
    constexpr int E = D / 32, kAhead = 4;
    __shared__ float s_top[8], s_sum[8], s_acc[W > 1 ? 8 : 1][D];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for all of the parts
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = W > 1 ? warp : 0;
    const long long at = W > 1 ? blockIdx.x : (long long)blockIdx.x * 8 + warp;
    const long long n = p.b.rows * p.H;
    if (at >= n) return;
    SeqSpan sp;
    const int seq = find_seq(p.b, (int)(at / p.H), sp);
    if (seq < 0) return;
    const int kvlen = p.c.kv_lens[seq];
    if (kvlen < sp.len || kvlen > (long long)p.c.width * p.c.page) return;
    float acc[E] = {}, top = -INFINITY, sum = 0.f;
    for (int z0 = w; z0 < p.splits; z0 += 32 * W) {
        const int zl = z0 + W * lane;
        const float mine = zl < p.splits ? p.part_l[(size_t)zl * n + at] : -INFINITY;
        float t = mine;
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, m));
        t = fmaxf(t, top);
        const float old = top == -INFINITY ? 0.f : ex2((top - t) * kLog2e);
        const float wt = mine == -INFINITY ? 0.f : ex2((mine - t) * kLog2e);  // NaN stays NaN
        top = t;
        sum = sum * old + wt;  // lane by lane, summed at the end
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= old;
        const int cnt = min(32, (p.splits - z0 + W - 1) / W);
        for (int z = 0; z < cnt; z += kAhead) {
            float v[kAhead][E], f[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                f[i] = __shfl_sync(0xffffffffu, wt, (z + i) & 31);
                if (z + i >= cnt) f[i] = 0.f;
                const float *src = p.part_o + ((size_t)(z0 + W * (z + i)) * n + at) * D + lane * E;
#pragma unroll
                for (int e = 0; e < E; e += 2) {  // an empty part has written no output
                    const float2 x = f[i] != 0.f ? *reinterpret_cast<const float2 *>(src + e) : make_float2(0.f, 0.f);
                    v[i][e] = x.x;
                    v[i][e + 1] = x.y;
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += f[i] * v[i][e];
        }
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if constexpr (W > 1) {
        if (lane == 0) {
            s_top[warp] = top;
            s_sum[warp] = sum;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int i = 0; i < W; ++i) top = fmaxf(top, s_top[i]);
        sum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float f = s_top[i] == -INFINITY ? 0.f : ex2((s_top[i] - top) * kLog2e);
            sum += f * s_sum[i];
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += f * s_acc[i][lane * E + e];
        }
    }
    const bool any = sum > 0.f || sum != sum;
    const float inv = any ? 1.f / sum : 0.f;
    __nv_bfloat16 *dst = p.o + at * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t *>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (p.lse && lane == 0) p.lse[at] = any ? top + __log2f(sum) * kLn2 : -INFINITY;
}

template <int D, bool e4m3, int NQ> cudaError_t run(const Params &p, dim3 grid, cudaStream_t s)
{
    auto kernel = attn_rows_kernel<D, e4m3, NQ>;
    using C = Cfg<D, e4m3, NQ>;
    cudaError_t e = set_smem_attr(reinterpret_cast<const void *>(kernel), C::SMEM);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kWarps * 32, C::SMEM, s>>>(p);
    return cudaGetLastError();
}
template <int NQ> cudaError_t run(int D, bool e4m3, const Params &p, dim3 grid, cudaStream_t s)
{
    if (e4m3) return D == 128 ? run<128, true, NQ>(p, grid, s) : run<64, true, NQ>(p, grid, s);
    return D == 128 ? run<128, false, NQ>(p, grid, s) : run<64, false, NQ>(p, grid, s);
}

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

}  // namespace

namespace {

constexpr int kMostSplits = 256;
// Packed rows a sequence and key head, on average, up to which the rows kernel runs (see cached_plan).
long long rows_limit(bool e4m3) { return e4m3 ? 64 : 16; }
// The keys that a sequence's new rows see at most.
long long visible_keys(long long rows, int window, long long capacity)
{
    return window > 0 && window + rows < capacity ? window + rows : capacity;
}
int clamp_splits(long long want, long long most)
{
    if (want > most) want = most;
    return (int)(want > kMostSplits ? kMostSplits : want < 1 ? 1 : want);
}
int rows_splits(long long n, int Hkv, long long keys)
{
    // Two waves of blocks (one sequence over 32768 keys: 1 wave 24, 2 24, 4 28), and ragged lengths: no block
    // reads more than 2048 keys, as far as kMostSplits goes (64 sequences of 64 to 8192 keys, e4m3: 39; 1024 40;
    // any number 55)
    const long long two = ceil_div(2LL * device_sms(), n * Hkv), even = ceil_div(keys, 2048);
    return clamp_splits(two > even ? two : even, keys / 256);
}
int tile_splits(long long n, long long rows, int G, int Hkv, long long keys)
{
    // As many parts as blocks run at once, if sequences are alike.  512 tokens over 32768 keys: 4 parts 132,
    // 5 (a second wave) 193, 8 142; 128 tokens: 16 parts 51, 13 59, 8 72; 4 x 512 over 16384, 128 blocks
    // of their own: 1 part 227, 2 252.
    const long long blocks = n * ((rows * G + 256LL * n - 1) / (256LL * n)) * Hkv;
    return clamp_splits(device_sms() / blocks, keys / 512);
}

}  // namespace

// Measured with H = 16, Hkv = 4, D = 128, times in us with the join; D = 64 and other groups go by the same rules.
CachedPlan cached_plan(bool e4m3, int n, long long rows, int H, int Hkv, int window, long long capacity)
{
    const int G = H / Hkv;
    CachedPlan plan;
    // Rows a sequence and key head, on average: few leave the step bound by the cache's bytes, and the
    // tensor core's tile of 128 rows empty; the rows kernel reads the keys once to every 16.  Rows kernel against
    // tiles, 8 sequences over 8192 keys: 16 rows 40 and 59, 20 rows 52 and 42, 32 rows 58 and 43; 64 over 2048:
    // 32 rows 104 and 71 (but 2 over 2048: 16 and 18).  e4m3, whose bytes are half and whose tiles wait for their
    // conversion, 8 over 8192: 32 rows 49 and 102, 64 rows 80 and 103, 128 rows 144 and 104.
    plan.tc = rows * G > rows_limit(e4m3) * n;
    const long long keys = visible_keys(rows, window, capacity);
    plan.splits = plan.tc ? tile_splits(n, rows, G, Hkv, keys) : rows_splits(n, Hkv, keys);
    return plan;
}

// Partial outputs and log-sums: `parts` (part, row) pairs, or none if there is one part only.
size_t cached_workspace_bytes(long long parts, int H, int D) { return (size_t)parts * H * (D + 1) * sizeof(float); }

// The most (part, row) pairs that any call of up to n sequences, `rows` rows and `capacity` positions plans.
// Both kinds of splits grow with the keys, so with the rows where nothing else changes, and with the capacity.
long long cached_most_parts(bool e4m3, int n, long long rows, int H, int Hkv, int window, long long capacity)
{
    const int G = H / Hkv, sms = device_sms();
    long long most = 0;
    auto count = [&](long long r, long long splits) { most = splits > 1 && splits * r > most ? splits * r : most; };
    // Rows kernel: x sequences take up to `limit` rows; more sequences have fewer parts, until two waves are one
    // block each (a last x is the number of sequences itself), and no more rows once all are taken.
    for (long long x = 1; x <= n; ++x) {
        if (x * Hkv > 2LL * sms) x = n;
        const long long limit = rows_limit(e4m3) * x / G, r = limit < rows ? limit : rows;
        if (r > 0) count(r, rows_splits(x, Hkv, visible_keys(r, window, capacity)));
        if (r == rows) break;
    }
    // Tiles: of all numbers of sequences one has the fewest blocks to the same rows; b blocks a key head hold up
    // to 256 b rows, and leave one part each from half of the SMs on.
    for (long long b = 1; b * Hkv <= sms / 2; ++b) {
        const long long limit = 256 * b / G, r = limit < rows ? limit : rows;
        if (r * G > rows_limit(e4m3)) count(r, tile_splits(1, r, G, Hkv, visible_keys(r, window, capacity)));
        if (r == rows) break;
    }
    return most;
}

cudaError_t launch_attn_cached(const CachedArgs &a, bool use_tc, cudaStream_t s)
{
    Params p{};
    p.b = a.b;
    p.H = a.H;
    p.Hkv = a.Hkv;
    p.G = a.H / a.Hkv;
    p.window = a.window;
    p.splits = a.splits;
    p.scale = a.scale;
    p.c = a.c;
    p.q = (const __nv_bfloat16 *)a.q;
    p.o = (__nv_bfloat16 *)a.o;
    p.lse = a.lse;
    p.part_o = a.part_o;
    p.part_l = a.part_l;
    p.status = a.status;
    cudaError_t e;
    if (use_tc) {
        e = launch_attn_cached_tc(a, s);
    } else {
        // more than 8 rows a sequence, on average (64 sequences over 4096 keys: 12 rows 111 us, by eights 139; 4 rows
        // 108, by eights 105)
        const bool wide = a.b.rows * p.G > 8LL * a.b.n;
        const int rows = wide ? 16 : 8;
        long long keys = (long long)a.c.width * a.c.page;
        if (a.window > 0 && a.window + rows < keys) keys = a.window + rows;
        p.piece = ceil_div(ceil_div(keys, a.splits), 128) * 128;  // whole steps of the four warps
        const long long tiles = a.b.n + a.b.rows * p.G / rows;
        if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
        const dim3 grid((unsigned)tiles, (unsigned)a.Hkv, (unsigned)a.splits);
        e = wide ? run<2>(a.D, a.c.e4m3, p, grid, s) : run<1>(a.D, a.c.e4m3, p, grid, s);
    }
    if (e != cudaSuccess || a.splits == 1) return e;
    const long long rows = a.b.rows * a.H;
    // 8 warps to a row where parts are many and rows too few to fill the SMs (16 rows, 37 parts: 24 us in all,
    // a warp to a row 38; 2048 rows, 16 parts: 52 and 50; 32768 rows: 454 and 379)
    const bool wide = a.splits > 8 && rows <= kManyRows;
    cudaLaunchAttribute early;  // launched while the last parts are written: one sequence over 32768 keys 2 us sooner
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(wide ? rows : (rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    if (wide) e = a.D == 128 ? cudaLaunchKernelEx(&cfg, attn_join_kernel<128, 8>, p) : cudaLaunchKernelEx(&cfg, attn_join_kernel<64, 8>, p);
    else e = a.D == 128 ? cudaLaunchKernelEx(&cfg, attn_join_kernel<128, 1>, p) : cudaLaunchKernelEx(&cfg, attn_join_kernel<64, 1>, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace gdn2
