// Shared declarations of the attention layer's operators: the rotation prologue (rope.cu), causal
// attention over whole sequences (attn_simt.cu, attn_fwd_tc.cu, attn_bwd_tc.cu), the paged cache
// (kv_cache.cu) and attention over it (attn_cached.cu).
#pragma once

#include <limits.h>

#include "gdn2_internal.cuh"

namespace gdn2 {

// Pairs of fp32 values: one instruction to two of them.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// A batch of sequences.  Fixed length (cu == null): n sequences of T tokens.  Packed: sequence i is
// rows cu[i] .. cu[i + 1] of `rows` token rows; rows behind cu[n] belong to no sequence.
struct SeqBatch {
    const int *cu;
    int n, T;
    long long rows;
};

// First row and token count of sequence i; len = -1 where cu is invalid (nothing is read or
// written for such a sequence).
__device__ __forceinline__ SeqSpan batch_span(const SeqBatch &b, int i)
{
    if (!b.cu) return {i * b.T, b.T};
    const int b0 = b.cu[i], b1 = b.cu[i + 1];
    if (b0 < 0 || b1 < b0 || b1 > b.rows || (i == 0 && b0 != 0)) return {0, -1};
    return {b0, b1 - b0};
}

// The tile'th tile (of `per` tokens) over all sequences in order, found by one whole warp: 32
// sequences' tile counts at a time, their running sum by shuffles.  False past the last tile.
struct TileRef {
    int seq, tile;  // sequence, and the tile within it
    SeqSpan sp;
};
__device__ __forceinline__ bool find_tile(const SeqBatch &b, int tile, int per, TileRef &r)
{
    if (!b.cu) {
        const int nt = (b.T + per - 1) / per;
        r.seq = tile / nt;
        r.tile = tile - r.seq * nt;
        r.sp = {r.seq * b.T, b.T};
        return r.seq < b.n;
    }
    const int lane = threadIdx.x & 31;
    for (int base = 0; base < b.n; base += 32) {
        SeqSpan sp = {0, -1};
        if (base + lane < b.n) sp = batch_span(b, base + lane);
        const int nt = sp.len > 0 ? (sp.len + per - 1) / per : 0;
        int sum = nt;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, m);
            if (lane >= m) sum += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, sum > tile);
        if (hit) {
            const int src = __ffs(hit) - 1;
            r.seq = base + src;
            r.tile = tile - __shfl_sync(0xffffffffu, sum - nt, src);
            r.sp.bos = __shfl_sync(0xffffffffu, sp.bos, src);
            r.sp.len = __shfl_sync(0xffffffffu, sp.len, src);
            return true;
        }
        tile -= __shfl_sync(0xffffffffu, sum, 31);
    }
    return false;
}
// The rank'th tile in order of falling cost, so that the last blocks to run are the short ones.  A
// tile costs the more the further it lies from its sequence's start (causal queries: the keys before
// it) or, with from_end, from its end (keys: the queries after it): all sequences' tiles at the
// greatest distance come first, then the next ones.  More than 32 packed sequences: in the batch's
// order, their tiles are many and alike.  By a whole warp.
__device__ __forceinline__ bool find_heavy_tile(const SeqBatch &b, int rank, int per, bool from_end, TileRef &r)
{
    if (!b.cu) {
        const int nt = (b.T + per - 1) / per, d = nt - 1 - rank / b.n;
        r.seq = rank % b.n;
        r.tile = from_end ? nt - 1 - d : d;
        r.sp = {r.seq * b.T, b.T};
        return d >= 0;
    }
    if (b.n > 32) return find_tile(b, rank, per, r);
    const int lane = threadIdx.x & 31;
    SeqSpan sp = {0, -1};
    if (lane < b.n) sp = batch_span(b, lane);
    const int nt = sp.len > 0 ? (sp.len + per - 1) / per : 0;
    auto beyond = [&](int d) { return __reduce_add_sync(0xffffffffu, max(nt - d, 0)); };  // tiles at distance >= d
    int lo = 0, hi = __reduce_max_sync(0xffffffffu, nt);
    if (beyond(0) <= rank) return false;
    while (hi - lo > 1) {  // beyond(lo) > rank >= beyond(hi)
        const int mid = (lo + hi) >> 1;
        if (beyond(mid) > rank) lo = mid;
        else hi = mid;
    }
    const unsigned who = __ballot_sync(0xffffffffu, nt > lo);
    r.seq = __fns(who, 0, rank - beyond(lo + 1) + 1);
    r.sp.bos = __shfl_sync(0xffffffffu, sp.bos, r.seq);
    r.sp.len = __shfl_sync(0xffffffffu, sp.len, r.seq);
    r.tile = from_end ? __shfl_sync(0xffffffffu, nt, r.seq) - 1 - lo : lo;
    return true;
}
// The same where a tile's cost is its sequence's `len` of keys: the longest sequences' tiles first.
__device__ __forceinline__ bool find_long_tile(const SeqBatch &b, const int *lens, int rank, int per, TileRef &r)
{
    if (b.n > 32) return find_tile(b, rank, per, r);
    const int lane = threadIdx.x & 31;
    SeqSpan sp = {0, -1};
    if (lane < b.n) sp = batch_span(b, lane);
    const int nt = sp.len > 0 ? (sp.len + per - 1) / per : 0, len = nt ? lens[lane] : INT_MIN;
    int before = 0;  // tiles of longer sequences
    for (int i = 0; i < b.n; ++i) {
        const int l = __shfl_sync(0xffffffffu, len, i), n = __shfl_sync(0xffffffffu, nt, i);
        if (l > len || (l == len && i < lane)) before += n;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, rank >= before && rank < before + nt);
    if (!hit) return false;
    r.seq = __ffs(hit) - 1;
    r.tile = rank - __shfl_sync(0xffffffffu, before, r.seq);
    r.sp.bos = __shfl_sync(0xffffffffu, sp.bos, r.seq);
    r.sp.len = __shfl_sync(0xffffffffu, sp.len, r.seq);
    return true;
}
// upper bound of the number of tiles over all sequences
inline long long tile_bound(const SeqBatch &b, int per)
{
    return b.cu ? b.rows / per + b.n : (long long)b.n * ((b.T + per - 1) / per);
}
// The sequence that holds row t, by a whole warp: 32 boundaries at a time, a ballot a step.
// -1 for rows behind the last sequence and for an invalid cu around t.  An entry outside [0, rows] may lead the
// ballots to a sequence that it makes invalid, from any row: then all are looked through, a step of 32 each.
__device__ __forceinline__ int find_seq(const SeqBatch &b, int t, SeqSpan &sp)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = b.n;  // the sequence is one of lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool le = lane * step < n && b.cu[i] <= t;  // sequence i starts at or before t
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int last = m ? 31 - __clz(m) : 0;
        n = min(step, n - last * step);
        lo += last * step;
    }
    // sequences of no tokens share their start with the one after them, which the last ballot took
    sp = batch_span(b, lo);
    for (int base = 0; sp.len < 0 && base < b.n; base += 32) {
        SeqSpan x = {0, -1};
        if (base + lane < b.n) x = batch_span(b, base + lane);
        const unsigned hit = __ballot_sync(0xffffffffu, x.len > 0 && t >= x.bos && t - x.bos < x.len);
        if (!hit) continue;
        lo = base + __ffs(hit) - 1;
        sp.bos = __shfl_sync(0xffffffffu, x.bos, lo - base);
        sp.len = __shfl_sync(0xffffffffu, x.len, lo - base);
    }
    return sp.len > 0 && t >= sp.bos && t < sp.bos + sp.len ? lo : -1;
}

// One warp of one block of a launch checks cu once; an invalid entry sets the status word.
__device__ __forceinline__ void report_bad_seqlens(const SeqBatch &b, int *status)
{
    if (!b.cu) return;
    bool bad = false;
    for (int i = threadIdx.x & 31; i < b.n; i += 32) bad |= batch_span(b, i).len < 0;
    if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) atomicExch(status, kStatusBadSeqlens);
}

// Causal attention over whole sequences.  q, o [rows, H, D]; k, v [rows, Hkv, D]; lse [rows, H];
// query head h reads key head h / (H / Hkv).  A query at position i sees the keys j <= i, with
// window > 0 only those with j > i - window.
struct AttnArgs {
    SeqBatch b;
    int H, Hkv, D, window;
    float scale;
    const void *q, *k, *v;
    void *o;           // forward: output; backward: input
    float *lse;        // forward: output, may be null; backward: input
    const void *d_o;   // backward only, as are the rest
    void *dq, *dk, *dv;
    float *delta;      // [rows, H] workspace: sum over channels of d_o * o
    int *status;
};
cudaError_t launch_attn_fwd_simt(const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attn_bwd_simt(const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attn_fwd_tc(const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attn_bwd_tc(const AttnArgs &a, cudaStream_t s);
cudaError_t launch_attn_delta(bool fp32, const AttnArgs &a, cudaStream_t s);

struct RopeArgs {
    int interleaved, norm, H, Hkv, D, rot;
    long long n;  // token rows
    const void *q, *k;
    const float *wq, *wk;  // may be null (ones)
    const int *pos;
    const float *inv;
    float eps, rot_scale;
    void *qo, *ko;               // forward outputs
    const void *dqo, *dko;       // backward inputs
    void *dq, *dk;               // backward outputs
    float *dwq, *dwk, *partial;  // backward weight gradients and their per-block sums
};
int rope_bwd_blocks(long long n);       // of n token rows' backward pass, a row of `partial` each
int rope_bwd_most_blocks(long long n);  // ... of any pass of up to n token rows
cudaError_t launch_rope(bool bwd, bool fp32, const RopeArgs &a, cudaStream_t s);

// The paged cache: k and v [num_pages, page, Hkv, D] (bf16, or e4m3 with one fp32 scale per row
// and head, [num_pages, page, Hkv]).  Position p of sequence i is row p % page of page
// table[i * width + p / page].  Sequence i holds kv_lens[i] positions, of which its rows in the
// batch are the last.
struct PagedCache {
    int e4m3, num_pages, page, width;
    const int *table, *kv_lens;
    void *k, *v;
    float *ks, *vs;
};
cudaError_t launch_cache_copy(bool read, const SeqBatch &b, int Hkv, int D, const PagedCache &c, void *k, void *v,
                              int *status, cudaStream_t s);

struct CachedArgs {
    SeqBatch b;
    int H, Hkv, D, window;
    float scale;
    PagedCache c;
    const void *q;
    void *o;
    float *lse;               // may be null
    int splits;               // parts that the key axis is cut into
    float *part_o, *part_l;   // workspace of splits > 1: [splits][rows, H] x (D values of o; log-sum)
    int *status;
};
// How many parts the key axis is cut into, and whether the tensor-core kernel runs, from sizes alone.
struct CachedPlan {
    bool tc;
    int splits;
};
CachedPlan cached_plan(bool e4m3, int n, long long rows, int H, int Hkv, int window, long long capacity);
long long cached_most_parts(bool e4m3, int n, long long rows, int H, int Hkv, int window, long long capacity);
size_t cached_workspace_bytes(long long parts, int H, int D);
cudaError_t launch_attn_cached(const CachedArgs &a, bool tc, cudaStream_t s);
cudaError_t launch_attn_cached_tc(const CachedArgs &a, cudaStream_t s);

int device_sms();

}  // namespace gdn2
