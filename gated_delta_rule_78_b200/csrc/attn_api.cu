// C ABI of the attention layer's operators: argument checks, workspaces, dispatch.  Declarations and
// the contract of every entry point are in include/gdn2.h.
#include <limits.h>
#include <math.h>

#include <initializer_list>

#include "attn.cuh"

namespace {

using namespace gdn2;

gdn2_status from_cuda(cudaError_t e) { return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA; }

gdn2_status check_ptrs(std::initializer_list<const void *> required, std::initializer_list<const void *> optional = {})
{
    for (const void *p : required)
        if (!p) return GDN2_ERR_NULL;
    for (const void *p : required)
        if ((uintptr_t)p & 15u) return GDN2_ERR_ALIGN;
    for (const void *p : optional)
        if (p && ((uintptr_t)p & 15u)) return GDN2_ERR_ALIGN;
    return GDN2_OK;
}

// Heads and sizes of one operator: `rows` token rows in all.
gdn2_status check_heads(gdn2_dtype dt, long long rows, int H, int Hkv, int D)
{
    if (dt != GDN2_F32 && dt != GDN2_BF16) return GDN2_ERR_DTYPE;
    if (rows < 0 || H <= 0 || Hkv <= 0 || D <= 0) return GDN2_ERR_SHAPE;
    if ((D != 64 && D != 128) || H > 65535) return GDN2_ERR_UNSUPPORTED;
    // rows are TMA coordinates and (row, head) pairs 32-bit indices; differences of positions and a
    // window below the longest sequence stay inside 32 bits too
    if (rows * H > INT_MAX || rows * Hkv > INT_MAX || rows > (1LL << 30)) return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}
// ... of attention: grouped heads, window, scale
gdn2_status check_attn(gdn2_dtype dt, long long rows, int H, int Hkv, int D, int window, float scale)
{
    const gdn2_status st = check_heads(dt, rows, H, Hkv, D);
    if (st != GDN2_OK) return st;
    if (H % Hkv != 0 || window < 0 || !(scale > 0.f) || !(scale < INFINITY)) return GDN2_ERR_SHAPE;
    if (H / Hkv > 64) return GDN2_ERR_UNSUPPORTED;  // a tile holds a token's whole group
    return GDN2_OK;
}
// a window that no sequence of `longest` tokens reaches is none
int effective_window(int window, long long longest) { return window >= longest ? 0 : window; }

gdn2_status check_rope(int flags, gdn2_dtype dt, int N, int H, int Hkv, int D, int rot, float eps, float rot_scale)
{
    if (flags & ~(GDN2_ROPE_RMSNORM | GDN2_ROPE_INTERLEAVED)) return GDN2_ERR_UNSUPPORTED;
    const gdn2_status st = check_heads(dt, N, H, Hkv, D);
    if (st != GDN2_OK) return st;
    if (rot < 0 || rot > D || rot % 2 != 0 || !(eps >= 0.f) || !(eps < INFINITY) || !(fabsf(rot_scale) < INFINITY))
        return GDN2_ERR_SHAPE;
    return GDN2_OK;
}
size_t rope_partial_bytes(int blocks, int D) { return (size_t)2 * blocks * D * sizeof(float); }

gdn2_status attn_fwd(gdn2_dtype dt, const SeqBatch &b, int H, int Hkv, int D, int window, float scale, const void *q,
                     const void *k, const void *v, void *o, float *lse, void *stream)
{
    const gdn2_status st = check_ptrs({q, k, v, o}, {lse});
    if (st != GDN2_OK) return st;
    window = effective_window(window, b.cu ? b.rows : b.T);
    AttnArgs a{};
    a.b = b;
    a.H = H; a.Hkv = Hkv; a.D = D; a.window = window; a.scale = scale;
    a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
    a.status = status_word();
    if (!a.status) return GDN2_ERR_CUDA;
    return from_cuda(dt == GDN2_F32 ? launch_attn_fwd_simt(a, (cudaStream_t)stream) : launch_attn_fwd_tc(a, (cudaStream_t)stream));
}
gdn2_status attn_bwd(gdn2_dtype dt, const SeqBatch &b, int H, int Hkv, int D, int window, float scale, const void *q,
                     const void *k, const void *v, const void *o, const float *lse, const void *d_o, void *dq, void *dk,
                     void *dv, void *workspace, size_t ws_bytes, void *stream)
{
    gdn2_status st = check_ptrs({q, k, v, o, lse, d_o, dq, dk, dv});
    if (st != GDN2_OK) return st;
    if (!workspace || ws_bytes < (size_t)b.rows * H * sizeof(float)) return GDN2_ERR_WORKSPACE;
    if ((st = check_ptrs({workspace})) != GDN2_OK) return st;
    window = effective_window(window, b.cu ? b.rows : b.T);
    AttnArgs a{};
    a.b = b;
    a.H = H; a.Hkv = Hkv; a.D = D; a.window = window; a.scale = scale;
    a.q = q; a.k = k; a.v = v; a.o = const_cast<void *>(o); a.lse = const_cast<float *>(lse); a.d_o = d_o;
    a.dq = dq; a.dk = dk; a.dv = dv; a.delta = (float *)workspace;
    a.status = status_word();
    if (!a.status) return GDN2_ERR_CUDA;
    return from_cuda(dt == GDN2_F32 ? launch_attn_bwd_simt(a, (cudaStream_t)stream) : launch_attn_bwd_tc(a, (cudaStream_t)stream));
}

// The cache's sizes; slots (page, row in it) are 32-bit.
gdn2_status check_cache(gdn2_cache_type type, gdn2_dtype dt, int N, int total_T, int Hkv, int D, int max_pages,
                        int num_pages, int page_size)
{
    if (type != GDN2_CACHE_BF16 && type != GDN2_CACHE_E4M3) return GDN2_ERR_DTYPE;
    const gdn2_status st = check_heads(dt, total_T, Hkv, Hkv, D);
    if (st != GDN2_OK) return st;
    if (N <= 0 || max_pages <= 0 || num_pages <= 0 || page_size <= 0) return GDN2_ERR_SHAPE;
    if (dt != GDN2_BF16) return GDN2_ERR_UNSUPPORTED;
    if ((long long)max_pages * page_size > (1LL << 30) || (long long)num_pages * page_size > INT_MAX)
        return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}
PagedCache make_cache(gdn2_cache_type type, int max_pages, int num_pages, int page_size, const int *block_table,
                      const int *kv_lens, const void *k, const void *v, const float *ks, const float *vs)
{
    return PagedCache{type == GDN2_CACHE_E4M3, num_pages, page_size, max_pages, block_table, kv_lens,
                      const_cast<void *>(k), const_cast<void *>(v), const_cast<float *>(ks), const_cast<float *>(vs)};
}
gdn2_status cache_copy(bool read, gdn2_cache_type type, gdn2_dtype dt, int N, int total_T, int Hkv, int D,
                       const int *cu_seqlens, const int *kv_lens, const int *block_table, int max_pages, int num_pages,
                       int page_size, void *k, void *v, void *k_cache, void *v_cache, float *k_scale, float *v_scale,
                       void *stream)
{
    gdn2_status st = check_cache(type, dt, N, total_T, Hkv, D, max_pages, num_pages, page_size);
    if (st != GDN2_OK) return st;
    if (total_T == 0) return GDN2_OK;
    st = check_ptrs({cu_seqlens, kv_lens, block_table, k, v, k_cache, v_cache});
    if (st == GDN2_OK && type == GDN2_CACHE_E4M3) st = check_ptrs({k_scale, v_scale});
    if (st != GDN2_OK) return st;
    int *status = status_word();
    if (!status) return GDN2_ERR_CUDA;
    return from_cuda(launch_cache_copy(read, SeqBatch{cu_seqlens, N, 0, total_T}, Hkv, D,
                                       make_cache(type, max_pages, num_pages, page_size, block_table, kv_lens, k_cache,
                                                  v_cache, k_scale, v_scale),
                                       k, v, status, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

gdn2_status gdn2_qk_rope(int flags, gdn2_dtype dt, int N, int H, int Hkv, int D, int rot, const void *q, const void *k,
                         const float *q_weight, const float *k_weight, const int *positions, const float *inv_freq,
                         float eps, float rot_scale, void *q_out, void *k_out, void *stream)
{
    gdn2_status st = check_rope(flags, dt, N, H, Hkv, D, rot, eps, rot_scale);
    if (st != GDN2_OK || N == 0) return st;
    st = check_ptrs({q, k, q_out, k_out}, {q_weight, k_weight});
    if (st == GDN2_OK && rot > 0) st = check_ptrs({positions, inv_freq});
    if (st != GDN2_OK) return st;
    RopeArgs a{};
    a.interleaved = flags & GDN2_ROPE_INTERLEAVED; a.norm = flags & GDN2_ROPE_RMSNORM;
    a.n = N; a.H = H; a.Hkv = Hkv; a.D = D; a.rot = rot;
    a.q = q; a.k = k; a.wq = q_weight; a.wk = k_weight; a.pos = positions; a.inv = inv_freq;
    a.eps = eps; a.rot_scale = rot_scale; a.qo = q_out; a.ko = k_out;
    return from_cuda(launch_rope(false, dt == GDN2_F32, a, (cudaStream_t)stream));
}

gdn2_status gdn2_qk_rope_bwd(int flags, gdn2_dtype dt, int N, int H, int Hkv, int D, int rot, const void *q,
                             const void *k, const float *q_weight, const float *k_weight, const int *positions,
                             const float *inv_freq, float eps, float rot_scale, const void *d_q_out,
                             const void *d_k_out, void *dq, void *dk, float *dq_weight, float *dk_weight,
                             void *workspace, size_t ws_bytes, void *stream)
{
    gdn2_status st = check_rope(flags, dt, N, H, Hkv, D, rot, eps, rot_scale);
    if (st != GDN2_OK) return st;
    const bool norm = flags & GDN2_ROPE_RMSNORM, want_w = norm && (dq_weight || dk_weight);
    st = check_ptrs({}, {dq_weight, dk_weight});
    if (st != GDN2_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    if (N == 0) {  // no rows: the weights' gradients are empty sums
        cudaError_t e = cudaSuccess;
        if (want_w && dq_weight) e = cudaMemsetAsync(dq_weight, 0, D * sizeof(float), s);
        if (e == cudaSuccess && want_w && dk_weight) e = cudaMemsetAsync(dk_weight, 0, D * sizeof(float), s);
        return from_cuda(e);
    }
    st = check_ptrs({d_q_out, d_k_out, dq, dk}, {q_weight, k_weight});
    if (st == GDN2_OK && norm) st = check_ptrs({q, k});
    if (st == GDN2_OK && rot > 0) st = check_ptrs({positions, inv_freq});
    if (st != GDN2_OK) return st;
    if (want_w) {
        if (!workspace || ws_bytes < rope_partial_bytes(rope_bwd_blocks(N), D)) return GDN2_ERR_WORKSPACE;
        if ((st = check_ptrs({workspace})) != GDN2_OK) return st;
    }
    RopeArgs a{};
    a.interleaved = flags & GDN2_ROPE_INTERLEAVED; a.norm = norm;
    a.n = N; a.H = H; a.Hkv = Hkv; a.D = D; a.rot = rot;
    a.q = q; a.k = k; a.wq = q_weight; a.wk = k_weight; a.pos = positions; a.inv = inv_freq;
    a.eps = eps; a.rot_scale = rot_scale; a.dqo = d_q_out; a.dko = d_k_out; a.dq = dq; a.dk = dk;
    a.dwq = dq_weight; a.dwk = dk_weight; a.partial = want_w ? (float *)workspace : nullptr;
    return from_cuda(launch_rope(true, dt == GDN2_F32, a, s));
}

size_t gdn2_qk_rope_workspace_size(int flags, gdn2_dtype dt, int N, int H, int Hkv, int D)
{
    if (check_rope(flags, dt, N, H, Hkv, D, 0, 0.f, 1.f) != GDN2_OK) return 0;
    return flags & GDN2_ROPE_RMSNORM ? rope_partial_bytes(rope_bwd_most_blocks(N), D) : 0;
}

gdn2_status gdn2_attn_fwd(gdn2_dtype dt, int B, int T, int H, int Hkv, int D, int window, float scale, const void *q,
                          const void *k, const void *v, void *o, float *lse, void *stream)
{
    if (B <= 0 || T < 0) return GDN2_ERR_SHAPE;
    const long long rows = (long long)B * T;
    const gdn2_status st = check_attn(dt, rows, H, Hkv, D, window, scale);
    if (st != GDN2_OK || T == 0) return st;
    return attn_fwd(dt, SeqBatch{nullptr, B, T, rows}, H, Hkv, D, window, scale, q, k, v, o, lse, stream);
}

gdn2_status gdn2_attn_fwd_varlen(gdn2_dtype dt, int N, int total_T, int H, int Hkv, int D, int window, float scale,
                                 const int *cu_seqlens, const void *q, const void *k, const void *v, void *o,
                                 float *lse, void *stream)
{
    if (N <= 0) return GDN2_ERR_SHAPE;
    gdn2_status st = check_attn(dt, total_T, H, Hkv, D, window, scale);
    if (st != GDN2_OK || total_T == 0) return st;
    if ((st = check_ptrs({cu_seqlens})) != GDN2_OK) return st;
    return attn_fwd(dt, SeqBatch{cu_seqlens, N, 0, total_T}, H, Hkv, D, window, scale, q, k, v, o, lse, stream);
}

gdn2_status gdn2_attn_bwd(gdn2_dtype dt, int B, int T, int H, int Hkv, int D, int window, float scale, const void *q,
                          const void *k, const void *v, const void *o, const float *lse, const void *d_o, void *dq,
                          void *dk, void *dv, void *workspace, size_t ws_bytes, void *stream)
{
    if (B <= 0 || T < 0) return GDN2_ERR_SHAPE;
    const long long rows = (long long)B * T;
    const gdn2_status st = check_attn(dt, rows, H, Hkv, D, window, scale);
    if (st != GDN2_OK || T == 0) return st;
    return attn_bwd(dt, SeqBatch{nullptr, B, T, rows}, H, Hkv, D, window, scale, q, k, v, o, lse, d_o, dq, dk, dv,
                    workspace, ws_bytes, stream);
}

gdn2_status gdn2_attn_bwd_varlen(gdn2_dtype dt, int N, int total_T, int H, int Hkv, int D, int window, float scale,
                                 const int *cu_seqlens, const void *q, const void *k, const void *v, const void *o,
                                 const float *lse, const void *d_o, void *dq, void *dk, void *dv, void *workspace,
                                 size_t ws_bytes, void *stream)
{
    if (N <= 0) return GDN2_ERR_SHAPE;
    gdn2_status st = check_attn(dt, total_T, H, Hkv, D, window, scale);
    if (st != GDN2_OK || total_T == 0) return st;
    if ((st = check_ptrs({cu_seqlens})) != GDN2_OK) return st;
    return attn_bwd(dt, SeqBatch{cu_seqlens, N, 0, total_T}, H, Hkv, D, window, scale, q, k, v, o, lse, d_o, dq, dk, dv,
                    workspace, ws_bytes, stream);
}

size_t gdn2_attn_workspace_size(gdn2_dtype dt, int N, int T, int H, int Hkv, int D)
{
    const long long rows = (long long)N * T;
    if (N <= 0 || T < 0 || check_attn(dt, rows, H, Hkv, D, 0, 1.f) != GDN2_OK) return 0;
    return (size_t)rows * H * sizeof(float);
}

gdn2_status gdn2_cache_write(gdn2_cache_type type, gdn2_dtype dt, int N, int total_T, int Hkv, int D,
                             const int *cu_seqlens, const int *kv_lens, const int *block_table, int max_pages,
                             int num_pages, int page_size, const void *k, const void *v, void *k_cache, void *v_cache,
                             float *k_scale, float *v_scale, void *stream)
{
    return cache_copy(false, type, dt, N, total_T, Hkv, D, cu_seqlens, kv_lens, block_table, max_pages, num_pages,
                      page_size, const_cast<void *>(k), const_cast<void *>(v), k_cache, v_cache, k_scale, v_scale, stream);
}

gdn2_status gdn2_cache_read(gdn2_cache_type type, gdn2_dtype dt, int N, int total_T, int Hkv, int D,
                            const int *cu_seqlens, const int *kv_lens, const int *block_table, int max_pages,
                            int num_pages, int page_size, const void *k_cache, const void *v_cache,
                            const float *k_scale, const float *v_scale, void *k, void *v, void *stream)
{
    return cache_copy(true, type, dt, N, total_T, Hkv, D, cu_seqlens, kv_lens, block_table, max_pages, num_pages,
                      page_size, k, v, const_cast<void *>(k_cache), const_cast<void *>(v_cache),
                      const_cast<float *>(k_scale), const_cast<float *>(v_scale), stream);
}

size_t gdn2_attn_cached_workspace_size(gdn2_dtype dt, int N, int total_T, int H, int Hkv, int D, int window,
                                       int max_pages, int page_size)
{
    if (check_attn(dt, total_T, H, Hkv, D, window, 1.f) != GDN2_OK || total_T == 0 ||
        check_cache(GDN2_CACHE_BF16, dt, N, total_T, Hkv, D, max_pages, 1, page_size) != GDN2_OK)
        return 0;
    const long long capacity = (long long)max_pages * page_size;
    window = effective_window(window, capacity);
    long long most = 0;  // for either type of cache
    for (bool e4m3 : {false, true}) {
        const long long parts = cached_most_parts(e4m3, N, total_T, H, Hkv, window, capacity);
        most = parts > most ? parts : most;
    }
    return cached_workspace_bytes(most, H, D);
}

gdn2_status gdn2_attn_cached(gdn2_cache_type type, gdn2_dtype dt, int N, int total_T, int H, int Hkv, int D,
                             int window, float scale, const int *cu_seqlens, const int *kv_lens,
                             const int *block_table, int max_pages, int num_pages, int page_size, const void *q,
                             const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
                             void *o, float *lse, void *workspace, size_t ws_bytes, void *stream)
{
    gdn2_status st = check_attn(dt, total_T, H, Hkv, D, window, scale);
    if (st == GDN2_OK) st = check_cache(type, dt, N, total_T, Hkv, D, max_pages, num_pages, page_size);
    if (st != GDN2_OK || total_T == 0) return st;
    st = check_ptrs({cu_seqlens, kv_lens, block_table, q, k_cache, v_cache, o}, {lse});
    if (st == GDN2_OK && type == GDN2_CACHE_E4M3) st = check_ptrs({k_scale, v_scale});
    if (st != GDN2_OK) return st;
    window = effective_window(window, (long long)max_pages * page_size);
    const CachedPlan plan = cached_plan(type == GDN2_CACHE_E4M3, N, total_T, H, Hkv, window, (long long)max_pages * page_size);
    if (plan.splits > 1) {
        const size_t need = cached_workspace_bytes((long long)plan.splits * total_T, H, D);
        if (!workspace || ws_bytes < need) return GDN2_ERR_WORKSPACE;
        if ((st = check_ptrs({workspace})) != GDN2_OK) return st;
    }
    CachedArgs a{};
    a.b = SeqBatch{cu_seqlens, N, 0, total_T};
    a.H = H; a.Hkv = Hkv; a.D = D; a.window = window; a.scale = scale; a.q = q; a.o = o; a.lse = lse;
    a.c = make_cache(type, max_pages, num_pages, page_size, block_table, kv_lens, k_cache, v_cache, k_scale, v_scale);
    a.splits = plan.splits;
    a.part_o = (float *)workspace;
    a.part_l = a.part_o ? a.part_o + (size_t)plan.splits * total_T * H * D : nullptr;
    a.status = status_word();
    if (!a.status) return GDN2_ERR_CUDA;
    return from_cuda(launch_attn_cached(a, plan.tc, (cudaStream_t)stream));
}

}  // extern "C"
