// Causal attention in fp32 on the CUDA cores: the fp32 path of gdn2_attn_fwd / gdn2_attn_bwd.
//
//   forward   s_ij = scale q_i . k_j over the visible j, one pass with a running maximum and sum:
//             o_i = sum_j e^(s_ij - m_i) v_j / l_i,  lse_i = m_i + ln l_i
//   backward  p_ij = e^(s_ij - lse_i),  delta_i = do_i . o_i,  ds_ij = p_ij (do_i . v_j - delta_i)
//             dv_j = sum_i p_ij do_i,  dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
//
// A block owns 32 queries, or for dk and dv 16 or 32 keys, and walks over the other side in tiles of 64.  Its
// groups of 4 threads to a row take the tiles in turn, each with shared memory of its own, and add up at
// the end, in order: an fp32 batch is mostly a small one, whose few blocks would otherwise leave an SM two
// warps to a scheduler.  The next tile's loads run behind this one's arithmetic, each as soon as its buffer
// is free.  A thread forms 4 x 4 scores and 4 rows x D / 16 channels of each product, two values to an
// instruction, with 16-byte loads of both operands from shared memory: 12 wavefronts of them to 32 pairs of
// FMAs of a warp, 16 of its scheduler's cycles, so bound by both pipes at once.  The backward runs two kernels,
// so that no sum depends on the order in which blocks run.
//
// 2 x 500 tokens, 4 heads on 2, D = 64: forward 24 us, delta 2, dk and dv 45, dq 30: a block's two or three tiles
// one after another.  8 x 2048, 16 heads, D = 128: forward 4.5 ms, 31 TFLOP/s, backward 13.8 ms.
#include "attn.cuh"

namespace gdn2 {
namespace {

constexpr int BQ = 32, BC = 64;  // queries of a block (keys of one: 16 or 32), columns of a tile

// shared-memory rows of D + 4 floats: 16-byte aligned, eight rows' 16 bytes in different banks
template <int D> constexpr int kStride = D + 4;
constexpr int kPs = BC + 4;

// rows [0, n) of a [n][D] tile (zeros from `rows` on), by the `threads` threads numbered tid
template <int D, int n>
__device__ __forceinline__ void load_tile(float *dst, const float *src, int rows, size_t stride, int tid, int threads)
{
    for (int i = tid; i < n * D / 4; i += threads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) v = *reinterpret_cast<const float4 *>(src + (size_t)r * stride + c);
        *reinterpret_cast<float4 *>(dst + r * kStride<D> + c) = v;
    }
}
// the same by asynchronous copies, which the thread waits for itself
template <int D, int n>
__device__ __forceinline__ void fetch_tile(float *dst, const float *src, int rows, size_t stride, int tid, int threads)
{
    for (int i = tid; i < n * D / 4; i += threads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst + r * kStride<D> + c)),
                     "l"(r < rows ? src + (size_t)r * stride + c : src), "r"(r < rows ? 16 : 0)
                     : "memory");
    }
}
__device__ __forceinline__ void fetch_one(float *dst, const float *src, bool live)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void fetched() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int n> __device__ __forceinline__ void group_sync(int group) { asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + group), "n"(n) : "memory"); }

// acc[i][j] = A[4 ty + i] . B[tx + 16 j] over D channels: even and odd ones in the halves of a pair
template <int D>
__device__ __forceinline__ void dot_tile(float (&acc)[4][4], const float *A, const float *B, int ty, int tx)
{
    uint64_t sum[4][4] = {};
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        ulonglong2 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const ulonglong2 *>(A + (4 * ty + i) * kStride<D> + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const ulonglong2 *>(B + (tx + 16 * j) * kStride<D> + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[i][j] = fma2(x[i].y, y[j].y, fma2(x[i].x, y[j].x, sum[i][j]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo, hi;
            unpair(sum[i][j], lo, hi);
            acc[i][j] = lo + hi;
        }
}

// acc[i][n] += sum over the 64 columns t of P[4 ty + i][t] * X[t][64 (n / 4) + 4 tx + n % 4]
template <int D>
__device__ __forceinline__ void mul_tile(float (&acc)[4][D / 16], const float *P, const float *X, int ty, int tx)
{
    uint64_t sum[4][D / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < D / 32; ++n) sum[i][n] = pair(acc[i][2 * n], acc[i][2 * n + 1]);
#pragma unroll 2
    for (int t = 0; t < BC; t += 4) {
        float p[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float4 *>(p[i]) = *reinterpret_cast<const float4 *>(P + (4 * ty + i) * kPs + t);
#pragma unroll
        for (int z = 0; z < 4; ++z)
#pragma unroll
            for (int n = 0; n < D / 64; ++n) {
                const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(X + (t + z) * kStride<D> + 64 * n + 4 * tx);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t p2 = pair(p[i][z], p[i][z]);
                    sum[i][2 * n] = fma2(p2, x.x, sum[i][2 * n]);
                    sum[i][2 * n + 1] = fma2(p2, x.y, sum[i][2 * n + 1]);
                }
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < D / 32; ++n) unpair(sum[i][n], acc[i][2 * n], acc[i][2 * n + 1]);
}

__device__ __forceinline__ bool visible(int i, int j, int len, int window)
{
    return j <= i && i < len && (window == 0 || i - j < window);
}

// This thread's 4 x D / 16 sums as a row-major [rows][D] tile, and the sum of the groups' tiles, group 0 first.
// The caller's barriers lie between.
template <int D> __device__ __forceinline__ void put_sums(float *dst, const float (&acc)[4][D / 16], int ty, int tx)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < D / 64; ++n)
            *reinterpret_cast<float4 *>(dst + (4 * ty + i) * D + 64 * n + 4 * tx) =
                make_float4(acc[i][4 * n], acc[i][4 * n + 1], acc[i][4 * n + 2], acc[i][4 * n + 3]);
}
template <int D, int BR, int NG>
__device__ __forceinline__ void store_sums(float *out, size_t stride, const float *sums, size_t gap, float f, int rows)
{
    for (int i = threadIdx.x; i < BR * D / 4; i += NG * 4 * BR) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        if (r >= rows) continue;
        float4 a = *reinterpret_cast<const float4 *>(sums + r * D + c);
#pragma unroll
        for (int g = 1; g < NG; ++g) {
            const float4 b = *reinterpret_cast<const float4 *>(sums + g * gap + r * D + c);
            a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
        }
        *reinterpret_cast<float4 *>(out + (size_t)r * stride + c) = make_float4(f * a.x, f * a.y, f * a.z, f * a.w);
    }
}

// Groups and shared memory (floats): the block's rows, then each group's column tiles, scores and, for dk
// and dv, the queries' lse and delta.
template <int D> struct Fwd {
    static constexpr int NG = D == 64 ? 4 : 2, ROWS = BQ * kStride<D>, GROUP = 2 * BC * kStride<D> + BQ * kPs;
    static constexpr int SMEM = (ROWS + NG * GROUP) * 4;
};
template <int D> struct Dq {
    static constexpr int NG = D == 64 ? 4 : 2, ROWS = 2 * BQ * kStride<D>, GROUP = 2 * BC * kStride<D> + BQ * kPs;
    static constexpr int SMEM = (ROWS + NG * GROUP) * 4;
};
template <int D, int BK> struct Dkv {
    static constexpr int NG = D == 128 ? 2 : BK == 16 ? 4 : 3, ROWS = 2 * BK * kStride<D>, GROUP = 2 * BC * kStride<D> + 2 * BK * kPs + 2 * BC;
    static constexpr int SMEM = (ROWS + NG * GROUP) * 4;
};

template <int D> __global__ void __launch_bounds__(Fwd<D>::NG * 4 * BQ) attn_fwd_kernel(const AttnArgs a)
{
    using C = Fwd<D>;
    extern __shared__ __align__(16) float sm[];
    const int tid = threadIdx.x % (4 * BQ), group = threadIdx.x / (4 * BQ), tx = tid & 15, ty = tid >> 4;
    float *Q = sm, *mine = sm + C::ROWS + group * C::GROUP, *K = mine, *V = K + BC * kStride<D>, *P = V + BC * kStride<D>;
    __shared__ float s_m[C::NG][BQ], s_l[C::NG][BQ];
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) report_bad_seqlens(a.b, a.status);
    TileRef r;
    if (!find_heavy_tile(a.b, blockIdx.x, BQ, false, r)) return;
    const int h = blockIdx.y, hk = h / (a.H / a.Hkv), q0 = r.tile * BQ, len = r.sp.len;
    const size_t qs = (size_t)a.H * D, ks = (size_t)a.Hkv * D, qoff = (size_t)(r.sp.bos + q0) * qs + h * D;
    const float *k = (const float *)a.k + (size_t)r.sp.bos * ks + hk * D;
    const float *v = (const float *)a.v + (size_t)r.sp.bos * ks + hk * D;
    const int last = min(q0 + BQ, len) - 1, jb = a.window == 0 || q0 < a.window ? 0 : (q0 - a.window + 1) / BC;
    auto fetch = [&](float *dst, const float *src, int j) {
        if (j * BC <= last) fetch_tile<D, BC>(dst, src + (size_t)j * BC * ks, len - j * BC, ks, tid, 4 * BQ);
    };
    fetch(K, k, jb + group);
    load_tile<D, BQ>(Q, (const float *)a.q + qoff, len - q0, qs, threadIdx.x, C::NG * 4 * BQ);
    fetched();
    __syncthreads();
    fetch(V, v, jb + group);
    float o[4][D / 16] = {}, m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
    for (int j = jb + group; j * BC <= last; j += C::NG) {  // K is there, V on its way
        float s[4][4];
        dot_tile<D>(s, Q, K, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = q0 + 4 * ty + i;
            float top = m[i];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                s[i][n] = visible(row, j * BC + tx + 16 * n, len, a.window) ? s[i][n] * a.scale : -INFINITY;
                top = fmaxf(top, s[i][n]);
            }
#pragma unroll
            for (int x = 8; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float base = top == -INFINITY ? 0.f : top;  // nothing visible so far
            const float f = expf(m[i] - base);
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float p = expf(s[i][n] - base);
                sum += p;
                P[(4 * ty + i) * kPs + tx + 16 * n] = p;
            }
#pragma unroll
            for (int x = 8; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            l[i] = l[i] * f + sum;
            m[i] = top;
#pragma unroll
            for (int n = 0; n < D / 16; ++n) o[i][n] *= f;
        }
        fetched();
        group_sync<4 * BQ>(group);
        fetch(K, k, j + C::NG);
        mul_tile<D>(o, P, V, ty, tx);
        fetched();
        group_sync<4 * BQ>(group);
        fetch(V, v, j + C::NG);
    }
    // ---- the groups' sums joined
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (tx == 0) {
            s_m[group][4 * ty + i] = m[i];
            s_l[group][4 * ty + i] = l[i];
        }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int g = 0; g < C::NG; ++g) top = fmaxf(top, s_m[g][4 * ty + i]);
        if (top == -INFINITY) top = 0.f;  // a row past the sequence
#pragma unroll
        for (int g = 0; g < C::NG; ++g) sum += expf(s_m[g][4 * ty + i] - top) * s_l[g][4 * ty + i];
        const float f = expf(m[i] - top) / sum;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) o[i][n] *= f;
        const int row = q0 + 4 * ty + i;
        if (a.lse && group == 0 && tx == 0 && row < len) a.lse[(size_t)(r.sp.bos + row) * a.H + h] = top + logf(sum);
    }
    put_sums<D>(mine, o, ty, tx);
    __syncthreads();
    store_sums<D, BQ, C::NG>((float *)a.o + qoff, qs, sm + C::ROWS, C::GROUP, 1.f, len - q0);
}

// delta[row, h] = sum over channels of d_o * o; 16 bytes a lane, as many lanes to a (row, head) as it
// has of them, both loads in flight at once.  Bound by memory.
template <typename T, int D> __global__ void __launch_bounds__(256) attn_delta_kernel(const AttnArgs a)
{
    constexpr int V = 16 / sizeof(T), L = D / V;
    const long long n = a.b.rows * a.H, i = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long row = i / L;
    float sum = 0.f;
    if (row < n) {
        const uint4 x = reinterpret_cast<const uint4 *>(a.o)[i], y = reinterpret_cast<const uint4 *>(a.d_o)[i];
        const T *xs = reinterpret_cast<const T *>(&x), *ys = reinterpret_cast<const T *>(&y);
#pragma unroll
        for (int e = 0; e < V; ++e) sum += to_f<T>(xs[e]) * to_f<T>(ys[e]);
    }
#pragma unroll
    for (int m = L / 2; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (row < n && threadIdx.x % L == 0) a.delta[row] = sum;
}

template <int D> __global__ void __launch_bounds__(Dq<D>::NG * 4 * BQ) attn_dq_kernel(const AttnArgs a)
{
    using C = Dq<D>;
    extern __shared__ __align__(16) float sm[];
    const int tid = threadIdx.x % (4 * BQ), group = threadIdx.x / (4 * BQ), tx = tid & 15, ty = tid >> 4;
    float *Q = sm, *O = sm + BQ * kStride<D>, *mine = sm + C::ROWS + group * C::GROUP, *K = mine, *V = K + BC * kStride<D>, *S = V + BC * kStride<D>;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) report_bad_seqlens(a.b, a.status);
    TileRef r;
    if (!find_heavy_tile(a.b, blockIdx.x, BQ, false, r)) return;
    const int h = blockIdx.y, hk = h / (a.H / a.Hkv), q0 = r.tile * BQ, len = r.sp.len;
    const size_t qs = (size_t)a.H * D, ks = (size_t)a.Hkv * D;
    const size_t qoff = (size_t)(r.sp.bos + q0) * qs + h * D, koff = (size_t)r.sp.bos * ks + hk * D;
    const int last = min(q0 + BQ, len) - 1, jb = a.window == 0 || q0 < a.window ? 0 : (q0 - a.window + 1) / BC;
    auto fetch = [&](float *dst, const void *src, int j) {
        if (j * BC <= last) fetch_tile<D, BC>(dst, (const float *)src + koff + (size_t)j * BC * ks, len - j * BC, ks, tid, 4 * BQ);
    };
    fetch(V, a.v, jb + group);
    load_tile<D, BQ>(Q, (const float *)a.q + qoff, len - q0, qs, threadIdx.x, C::NG * 4 * BQ);
    load_tile<D, BQ>(O, (const float *)a.d_o + qoff, len - q0, qs, threadIdx.x, C::NG * 4 * BQ);
    float lse[4], delta[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = q0 + 4 * ty + i;
        const size_t at = (size_t)(r.sp.bos + row) * a.H + h;
        lse[i] = row < len ? a.lse[at] : 0.f;
        delta[i] = row < len ? a.delta[at] : 0.f;
    }
    fetched();
    __syncthreads();
    fetch(K, a.k, jb + group);
    float dq[4][D / 16] = {};
    for (int j = jb + group; j * BC <= last; j += C::NG) {  // V is there, K on its way
        float s[4][4], dp[4][4];
        dot_tile<D>(dp, O, V, ty, tx);
        fetched();
        group_sync<4 * BQ>(group);
        fetch(V, a.v, j + C::NG);
        dot_tile<D>(s, Q, K, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const bool vis = visible(q0 + 4 * ty + i, j * BC + tx + 16 * n, len, a.window);
                S[(4 * ty + i) * kPs + tx + 16 * n] = vis ? expf(s[i][n] * a.scale - lse[i]) * (dp[i][n] - delta[i]) : 0.f;
            }
        group_sync<4 * BQ>(group);
        mul_tile<D>(dq, S, K, ty, tx);
        fetched();
        group_sync<4 * BQ>(group);
        fetch(K, a.k, j + C::NG);
    }
    put_sums<D>(mine, dq, ty, tx);
    __syncthreads();
    store_sums<D, BQ, C::NG>((float *)a.dq + qoff, qs, sm + C::ROWS, C::GROUP, a.scale, len - q0);
}

// Rows are keys, columns queries: the groups take the (query head, query tile) pairs in turn.
template <int D, int BK> __global__ void __launch_bounds__(Dkv<D, BK>::NG * 4 * BK) attn_dkv_kernel(const AttnArgs a)
{
    using C = Dkv<D, BK>;
    extern __shared__ __align__(16) float sm[];
    const int tid = threadIdx.x % (4 * BK), group = threadIdx.x / (4 * BK), tx = tid & 15, ty = tid >> 4;
    float *K = sm, *V = sm + BK * kStride<D>, *mine = sm + C::ROWS + group * C::GROUP, *Q = mine, *O = Q + BC * kStride<D>;
    float *P = O + BC * kStride<D>, *S = P + BK * kPs, *lse = S + BK * kPs, *delta = lse + BC;
    TileRef r;
    if (!find_heavy_tile(a.b, blockIdx.x, BK, true, r)) return;
    const int hk = blockIdx.y, heads = a.H / a.Hkv, k0 = r.tile * BK, len = r.sp.len;
    const size_t qs = (size_t)a.H * D, ks = (size_t)a.Hkv * D;
    const size_t koff = (size_t)(r.sp.bos + k0) * ks + hk * D;
    // queries k0 .. the last that still sees the tile's last key
    const int end = a.window == 0 || a.window > len ? len : min(len, k0 + BK - 1 + a.window), tiles = (end - k0 + BC - 1) / BC;
    auto fetch = [&](float *dst, const void *src, int i) {
        if (i >= heads * tiles) return;
        const int h = hk * heads + i / tiles, q0 = k0 + i % tiles * BC;
        fetch_tile<D, BC>(dst, (const float *)src + (size_t)(r.sp.bos + q0) * qs + h * D, len - q0, qs, tid, 4 * BK);
    };
    auto fetch_stats = [&](int i) {
        if (i >= heads * tiles || tid >= BC) return;
        const int h = hk * heads + i / tiles, q = k0 + i % tiles * BC + tid;
        const size_t at = (size_t)(r.sp.bos + min(q, len - 1)) * a.H + h;
        fetch_one(lse + tid, a.lse + at, q < len);
        fetch_one(delta + tid, a.delta + at, q < len);
    };
    fetch(O, a.d_o, group);
    fetch_stats(group);
    load_tile<D, BK>(K, (const float *)a.k + koff, len - k0, ks, threadIdx.x, C::NG * 4 * BK);
    load_tile<D, BK>(V, (const float *)a.v + koff, len - k0, ks, threadIdx.x, C::NG * 4 * BK);
    fetched();
    __syncthreads();
    fetch(Q, a.q, group);
    float dk[4][D / 16] = {}, dv[4][D / 16] = {};
    for (int i = group; i < heads * tiles; i += C::NG) {  // O, lse and delta are there, Q on its way
        const int q0 = k0 + i % tiles * BC;
        float s[4][4], dp[4][4];
        dot_tile<D>(dp, V, O, ty, tx);
        fetched();
        group_sync<4 * BK>(group);
        dot_tile<D>(s, K, Q, ty, tx);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int c = tx + 16 * n, at = (4 * ty + x) * kPs + c;
                const bool vis = visible(q0 + c, k0 + 4 * ty + x, len, a.window);
                const float p = vis ? expf(s[x][n] * a.scale - lse[c]) : 0.f;
                P[at] = p;
                S[at] = vis ? p * (dp[x][n] - delta[c]) : 0.f;
            }
        group_sync<4 * BK>(group);
        mul_tile<D>(dv, P, O, ty, tx);
        group_sync<4 * BK>(group);
        fetch(O, a.d_o, i + C::NG);
        fetch_stats(i + C::NG);
        mul_tile<D>(dk, S, Q, ty, tx);
        fetched();
        group_sync<4 * BK>(group);
        fetch(Q, a.q, i + C::NG);
    }
    put_sums<D>(mine, dk, ty, tx);
    put_sums<D>(mine + BK * D, dv, ty, tx);
    __syncthreads();
    store_sums<D, BK, C::NG>((float *)a.dk + koff, ks, sm + C::ROWS, C::GROUP, a.scale, len - k0);
    store_sums<D, BK, C::NG>((float *)a.dv + koff, ks, sm + C::ROWS + BK * D, C::GROUP, 1.f, len - k0);
}

template <typename F> cudaError_t run(F kernel, int smem, int threads, dim3 grid, const AttnArgs &a, cudaStream_t s)
{
    cudaError_t e = set_smem_attr(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, threads, smem, s>>>(a);
    return cudaGetLastError();
}
template <int D, int BK> cudaError_t run_dkv(const AttnArgs &a, cudaStream_t s)
{
    const dim3 grid((unsigned)tile_bound(a.b, BK), (unsigned)a.Hkv);
    return run(attn_dkv_kernel<D, BK>, Dkv<D, BK>::SMEM, Dkv<D, BK>::NG * 4 * BK, grid, a, s);
}
template <int D> cudaError_t run_bwd(const AttnArgs &a, cudaStream_t s)
{
    // 16 keys to a block where 32 would not fill the SMs twice (2 x 500, 2 key heads, d 64: dk and dv 45 us against
    // 76); else 32, which read each query tile half as often (8 x 2048, 16 heads, d 128: 13.8 ms against 17.3)
    const bool few = tile_bound(a.b, 32) * a.Hkv < 2LL * device_sms();
    cudaError_t e = few ? run_dkv<D, 16>(a, s) : run_dkv<D, 32>(a, s);
    const dim3 grid((unsigned)tile_bound(a.b, BQ), (unsigned)a.H);
    return e != cudaSuccess ? e : run(attn_dq_kernel<D>, Dq<D>::SMEM, Dq<D>::NG * 4 * BQ, grid, a, s);
}

}  // namespace

cudaError_t launch_attn_fwd_simt(const AttnArgs &a, cudaStream_t s)
{
    const dim3 grid((unsigned)tile_bound(a.b, BQ), (unsigned)a.H);
    return a.D == 128 ? run(attn_fwd_kernel<128>, Fwd<128>::SMEM, Fwd<128>::NG * 4 * BQ, grid, a, s)
                      : run(attn_fwd_kernel<64>, Fwd<64>::SMEM, Fwd<64>::NG * 4 * BQ, grid, a, s);
}

cudaError_t launch_attn_delta(bool fp32, const AttnArgs &a, cudaStream_t s)
{
    const long long lanes = a.b.rows * a.H * (a.D * (fp32 ? 4 : 2) / 16);
    const unsigned grid = (unsigned)((lanes + 255) / 256);
    if (fp32) (a.D == 128 ? attn_delta_kernel<float, 128> : attn_delta_kernel<float, 64>)<<<grid, 256, 0, s>>>(a);
    else (a.D == 128 ? attn_delta_kernel<__nv_bfloat16, 128> : attn_delta_kernel<__nv_bfloat16, 64>)<<<grid, 256, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_attn_bwd_simt(const AttnArgs &a, cudaStream_t s)
{
    cudaError_t e = launch_attn_delta(true, a, s);
    if (e != cudaSuccess) return e;
    return a.D == 128 ? run_bwd<128>(a, s) : run_bwd<64>(a, s);
}

}  // namespace gdn2
