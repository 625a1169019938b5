// Causal attention in fp32 on the CUDA cores: the fp32 path of gdn2_attn_fwd / gdn2_attn_bwd.
//
//   forward   s_ij = scale q_i . k_j over the visible j, one pass with a running maximum and sum:
//             o_i = sum_j e^(s_ij - m_i) v_j / l_i,  lse_i = m_i + ln l_i
//   backward  p_ij = e^(s_ij - lse_i),  delta_i = do_i . o_i,  ds_ij = p_ij (do_i . v_j - delta_i)
//             dv_j = sum_i p_ij do_i,  dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
//
// 64 x 64 tiles, 256 threads, a 4 x 4 block of the scores to a thread; every product reads its two
// operands from shared memory, the accumulators stay in registers.  Bound by the FP32 pipe and by
// shared-memory loads (2 16-byte loads to 16 FMAs).  The backward runs two kernels, one to a query
// tile (dq), one to a key tile (dk, dv, over all query heads of its key head), so that no sum
// depends on the order in which blocks run.
#include "attn.cuh"

namespace gdn2 {
namespace {

constexpr int BT = 64, kThreads = 256;

// shared-memory rows of D + 4 floats: 16-byte aligned, and 16 rows apart in different banks
template <int D> constexpr int kStride = D + 4;
constexpr int kPs = BT + 4;

template <int D>
__device__ __forceinline__ void load_tile(float *dst, const float *src, int rows, size_t stride)
{
    for (int i = threadIdx.x; i < BT * D / 4; i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) v = *reinterpret_cast<const float4 *>(src + (size_t)r * stride + c);
        *reinterpret_cast<float4 *>(dst + r * kStride<D> + c) = v;
    }
}

// acc[i][j] += A[ty + 16 i] . B[tx + 16 j] over D channels
template <int D>
__device__ __forceinline__ void dot_tile(float (&acc)[4][4], const float *A, const float *B, int ty, int tx)
{
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(A + (ty + 16 * i) * kStride<D> + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * kStride<D> + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
                acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
                acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
                acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
            }
    }
}

// acc[i][n] += sum over the 64 rows t of P(ty + 16 i, t) * X[t][4 tx + (n & 3) + 64 (n / 4)]
// P is row-major [64][kPs]; kT reads it transposed.
template <int D, bool kT>
__device__ __forceinline__ void mul_tile(float (&acc)[4][D / 16], const float *P, const float *X, int ty, int tx)
{
#pragma unroll 4
    for (int t = 0; t < BT; ++t) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = kT ? P[t * kPs + ty + 16 * i] : P[(ty + 16 * i) * kPs + t];
#pragma unroll
        for (int n = 0; n < D / 64; ++n) {
            const float4 x = *reinterpret_cast<const float4 *>(X + t * kStride<D> + 64 * n + 4 * tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i][4 * n] = fmaf(p[i], x.x, acc[i][4 * n]);
                acc[i][4 * n + 1] = fmaf(p[i], x.y, acc[i][4 * n + 1]);
                acc[i][4 * n + 2] = fmaf(p[i], x.z, acc[i][4 * n + 2]);
                acc[i][4 * n + 3] = fmaf(p[i], x.w, acc[i][4 * n + 3]);
            }
        }
    }
}

__device__ __forceinline__ bool visible(int i, int j, int len, int window)
{
    return j <= i && i < len && (window == 0 || i - j < window);
}
// first key tile that any of the queries from q0 on sees
__device__ __forceinline__ int first_key_tile(int q0, int window)
{
    return window == 0 || q0 < window ? 0 : (q0 - window + 1) / BT;
}

template <int D> constexpr int fwd_smem() { return (3 * BT * kStride<D> + BT * kPs) * 4; }
template <int D> constexpr int bwd_smem() { return (4 * BT * kStride<D> + 2 * BT * kPs + 2 * BT) * 4; }

template <int D> __global__ void __launch_bounds__(kThreads) attn_fwd_kernel(const AttnArgs a)
{
    extern __shared__ float sm[];
    float *Q = sm, *K = Q + BT * kStride<D>, *V = K + BT * kStride<D>, *P = V + BT * kStride<D>;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) report_bad_seqlens(a.b, a.status);
    TileRef r;
    if (!find_tile(a.b, gridDim.x - 1 - blockIdx.x, BT, r)) return;
    const int h = blockIdx.y, hk = h / (a.H / a.Hkv), tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int q0 = r.tile * BT, len = r.sp.len;
    const size_t qs = (size_t)a.H * D, ks = (size_t)a.Hkv * D;
    const float *q = (const float *)a.q + (size_t)r.sp.bos * qs + h * D;
    const float *k = (const float *)a.k + (size_t)r.sp.bos * ks + hk * D;
    const float *v = (const float *)a.v + (size_t)r.sp.bos * ks + hk * D;
    load_tile<D>(Q, q + (size_t)q0 * qs, len - q0, qs);
    float o[4][D / 16] = {}, m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
    const int last = min(q0 + BT, len) - 1;
    for (int j = first_key_tile(q0, a.window); j * BT <= last; ++j) {
        __syncthreads();
        load_tile<D>(K, k + (size_t)j * BT * ks, len - j * BT, ks);
        load_tile<D>(V, v + (size_t)j * BT * ks, len - j * BT, ks);
        __syncthreads();
        float s[4][4] = {};
        dot_tile<D>(s, Q, K, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = q0 + ty + 16 * i;
            float top = m[i];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                s[i][n] = visible(row, j * BT + tx + 16 * n, len, a.window) ? s[i][n] * a.scale : -INFINITY;
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
                P[(ty + 16 * i) * kPs + tx + 16 * n] = p;
            }
#pragma unroll
            for (int x = 8; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            l[i] = l[i] * f + sum;
            m[i] = top;
#pragma unroll
            for (int n = 0; n < D / 16; ++n) o[i][n] *= f;
        }
        __syncthreads();
        mul_tile<D, false>(o, P, V, ty, tx);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = q0 + ty + 16 * i;
        if (row >= len) continue;
        const float inv = 1.f / l[i];
        float *dst = (float *)a.o + ((size_t)(r.sp.bos + row) * a.H + h) * D;
#pragma unroll
        for (int n = 0; n < D / 64; ++n)
            *reinterpret_cast<float4 *>(dst + 64 * n + 4 * tx) =
                make_float4(o[i][4 * n] * inv, o[i][4 * n + 1] * inv, o[i][4 * n + 2] * inv, o[i][4 * n + 3] * inv);
        if (a.lse && tx == 0) a.lse[(size_t)(r.sp.bos + row) * a.H + h] = m[i] + logf(l[i]);
    }
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

// p and ds of one tile, from the scores s and the products dp = do . v, into P and S
__device__ __forceinline__ void softmax_grad(const AttnArgs &a, float (&s)[4][4], float (&dp)[4][4], int q0, int k0,
                                             int len, const float *lse, const float *delta, float *P, float *S, int ty,
                                             int tx)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int c = tx + 16 * n;
            const float p = visible(q0 + r, k0 + c, len, a.window) ? expf(s[i][n] * a.scale - lse[r]) : 0.f;
            P[r * kPs + c] = p;
            S[r * kPs + c] = p == 0.f ? 0.f : p * (dp[i][n] - delta[r]);
        }
    }
}
// lse and delta of the query tile's rows
__device__ __forceinline__ void load_stats(const AttnArgs &a, const TileRef &r, int q0, int h, float *lse, float *delta)
{
    if (threadIdx.x < BT) {
        const int row = q0 + threadIdx.x;
        const size_t at = (size_t)(r.sp.bos + row) * a.H + h;
        lse[threadIdx.x] = row < r.sp.len ? a.lse[at] : 0.f;
        delta[threadIdx.x] = row < r.sp.len ? a.delta[at] : 0.f;
    }
}
template <int D>
__device__ __forceinline__ void store_rows(float *dst, size_t stride, const float (&acc)[4][D / 16], float f, int rows,
                                           int ty, int tx)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (ty + 16 * i >= rows) continue;
#pragma unroll
        for (int n = 0; n < D / 64; ++n)
            *reinterpret_cast<float4 *>(dst + (size_t)(ty + 16 * i) * stride + 64 * n + 4 * tx) =
                make_float4(f * acc[i][4 * n], f * acc[i][4 * n + 1], f * acc[i][4 * n + 2], f * acc[i][4 * n + 3]);
    }
}

template <int D> __global__ void __launch_bounds__(kThreads) attn_dq_kernel(const AttnArgs a)
{
    extern __shared__ float sm[];
    constexpr int TS = BT * kStride<D>;
    float *Q = sm, *O = Q + TS, *K = O + TS, *V = K + TS, *P = V + TS, *S = P + BT * kPs, *lse = S + BT * kPs, *delta = lse + BT;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) report_bad_seqlens(a.b, a.status);
    TileRef r;
    if (!find_tile(a.b, gridDim.x - 1 - blockIdx.x, BT, r)) return;
    const int h = blockIdx.y, hk = h / (a.H / a.Hkv), tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int q0 = r.tile * BT, len = r.sp.len;
    const size_t qs = (size_t)a.H * D, ks = (size_t)a.Hkv * D;
    const size_t qoff = (size_t)(r.sp.bos + q0) * qs + h * D, koff = (size_t)r.sp.bos * ks + hk * D;
    load_tile<D>(Q, (const float *)a.q + qoff, len - q0, qs);
    load_tile<D>(O, (const float *)a.d_o + qoff, len - q0, qs);
    load_stats(a, r, q0, h, lse, delta);
    float dq[4][D / 16] = {};
    const int last = min(q0 + BT, len) - 1;
    for (int j = first_key_tile(q0, a.window); j * BT <= last; ++j) {
        __syncthreads();
        load_tile<D>(K, (const float *)a.k + koff + (size_t)j * BT * ks, len - j * BT, ks);
        load_tile<D>(V, (const float *)a.v + koff + (size_t)j * BT * ks, len - j * BT, ks);
        __syncthreads();
        float s[4][4] = {}, dp[4][4] = {};
        dot_tile<D>(s, Q, K, ty, tx);
        dot_tile<D>(dp, O, V, ty, tx);
        softmax_grad(a, s, dp, q0, j * BT, len, lse, delta, P, S, ty, tx);
        __syncthreads();
        mul_tile<D, false>(dq, S, K, ty, tx);
    }
    store_rows<D>((float *)a.dq + qoff, qs, dq, a.scale, len - q0, ty, tx);
}

template <int D> __global__ void __launch_bounds__(kThreads) attn_dkv_kernel(const AttnArgs a)
{
    extern __shared__ float sm[];
    constexpr int TS = BT * kStride<D>;
    float *Q = sm, *O = Q + TS, *K = O + TS, *V = K + TS, *P = V + TS, *S = P + BT * kPs, *lse = S + BT * kPs, *delta = lse + BT;
    TileRef r;
    if (!find_tile(a.b, blockIdx.x, BT, r)) return;
    const int hk = blockIdx.y, group = a.H / a.Hkv, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int k0 = r.tile * BT, len = r.sp.len;
    const size_t qs = (size_t)a.H * D, ks = (size_t)a.Hkv * D;
    const size_t koff = (size_t)(r.sp.bos + k0) * ks + hk * D;
    load_tile<D>(K, (const float *)a.k + koff, len - k0, ks);
    load_tile<D>(V, (const float *)a.v + koff, len - k0, ks);
    float dk[4][D / 16] = {}, dv[4][D / 16] = {};
    // queries k0 .. the last that still sees the tile's last key
    const int end = a.window == 0 || a.window > len ? len : min(len, k0 + BT - 1 + a.window);
    for (int h = hk * group; h < (hk + 1) * group; ++h)
        for (int q0 = k0; q0 < end; q0 += BT) {
            __syncthreads();
            const size_t qoff = (size_t)(r.sp.bos + q0) * qs + h * D;
            load_tile<D>(Q, (const float *)a.q + qoff, len - q0, qs);
            load_tile<D>(O, (const float *)a.d_o + qoff, len - q0, qs);
            load_stats(a, r, q0, h, lse, delta);
            __syncthreads();
            float s[4][4] = {}, dp[4][4] = {};
            dot_tile<D>(s, Q, K, ty, tx);
            dot_tile<D>(dp, O, V, ty, tx);
            softmax_grad(a, s, dp, q0, k0, len, lse, delta, P, S, ty, tx);
            __syncthreads();
            mul_tile<D, true>(dv, P, O, ty, tx);
            mul_tile<D, true>(dk, S, Q, ty, tx);
        }
    store_rows<D>((float *)a.dk + koff, ks, dk, a.scale, len - k0, ty, tx);
    store_rows<D>((float *)a.dv + koff, ks, dv, 1.f, len - k0, ty, tx);
}

template <typename F> cudaError_t run(F kernel, int smem, dim3 grid, const AttnArgs &a, cudaStream_t s)
{
    cudaError_t e = set_smem_attr(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_fwd_simt(const AttnArgs &a, cudaStream_t s)
{
    const dim3 grid((unsigned)tile_bound(a.b, BT), (unsigned)a.H);
    return a.D == 128 ? run(attn_fwd_kernel<128>, fwd_smem<128>(), grid, a, s)
                      : run(attn_fwd_kernel<64>, fwd_smem<64>(), grid, a, s);
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
    const unsigned tiles = (unsigned)tile_bound(a.b, BT);
    const dim3 gq(tiles, (unsigned)a.H), gk(tiles, (unsigned)a.Hkv);
    if (a.D == 128) {
        e = run(attn_dq_kernel<128>, bwd_smem<128>(), gq, a, s);
        return e != cudaSuccess ? e : run(attn_dkv_kernel<128>, bwd_smem<128>(), gk, a, s);
    }
    e = run(attn_dq_kernel<64>, bwd_smem<64>(), gq, a, s);
    return e != cudaSuccess ? e : run(attn_dkv_kernel<64>, bwd_smem<64>(), gk, a, s);
}

}  // namespace gdn2
