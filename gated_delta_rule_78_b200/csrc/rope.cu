// The attention layers' prologue: per-head RMS norm of q and k and the rotation by position, in one
// pass, and its backward pass.
//
//   forward   n = x rsqrt(mean x^2 + eps) w           (w per channel, 1 without a weight)
//             y = n with its first `rot` channels rotated in pairs by pos * inv_freq[i]:
//             (a, b) -> f (a cos - b sin, b cos + a sin), f = rot_scale
//   backward  u = the rotation's transpose applied to dy
//             dw = sum over rows of u x r,  r = rsqrt(mean x^2 + eps)
//             dx = r (u w - x r^2 mean(u w x))
//
// Both are bound by memory: x is read and y written once (backward: x and dy read, dx written).
// A warp owns a token and walks over its heads, as many lanes to a row as it has 16-byte vectors
// (bf16: 16 for D = 128, 8 for D = 64; fp32: twice that), so that the token's cosines and sines
// stay in registers for all of its heads.  The angle is formed and reduced modulo 2 pi in 64
// bits: pos * inv_freq in fp32 would be off by 2^-24 of an angle of up to 10^5.
#include "attn.cuh"

namespace gdn2 {
namespace {

constexpr int kWarps = 8;
constexpr int kShareBelow = 2048;  // tokens

template <typename T> struct Vec;
template <> struct Vec<float> { static constexpr int n = 4; };
template <> struct Vec<__nv_bfloat16> { static constexpr int n = 8; };

template <typename T> __device__ __forceinline__ uint4 load_raw(const T *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ void unpack(const uint4 &v, float (&f)[4])
{
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(const uint4 &v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store_vec(float *p, const float (&f)[4])
{
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// cos and sin of pos * inv, times f.  The product of an int and a float is exact in 64 bits, and so
// is the angle modulo a turn to about 1e-12; the remainder lies in [-pi, pi], where sincosf needs
// no long reduction.
__device__ __forceinline__ void angle(int pos, float inv, float f, float &c, float &s)
{
    const double a = (double)pos * (double)inv;
    const double turns = rint(a * 0.15915494309189535);
    const double r = fma(-turns, 6.283185307179586, a);
    sincosf((float)r, &s, &c);
    c *= f;
    s *= f;
}

// kSwap: pairs (i, i + rot / 2) whose halves are whole vectors, exchanged between lanes by a
// shuffle; kPair: interleaved pairs, both in one lane's vector; kAny: half layout with a rot / 2
// that ends inside a vector, exchanged through shared memory.
enum { kPair, kSwap, kAny };

// Rotates this lane's vector f (channels ch .. ch + V - 1 of its row) in place; the backward's
// transpose comes as negated sines.
template <int V, int mode>
__device__ __forceinline__ void rotate(float (&f)[V], const float (&c)[V], const float (&s)[V], int ch, int rot,
                                       float *buf, int lane)
{
    if constexpr (mode == kPair) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float a = f[e], b = f[e + 1];
            f[e] = a * c[e] - b * s[e];
            f[e + 1] = b * c[e] + a * s[e];
        }
    } else {
        // c = 1, s = 0 past rot; s is negative in the lower half
        const int half = rot >> 1;
        float o[V];
        if constexpr (mode == kSwap) {
            const int step = half / V;  // lanes between a channel and its partner
            const int src = ch < half ? lane + step : lane - step;
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = __shfl_sync(0xffffffffu, f[e], src & 31);
        } else {
            // row buffer of the lanes that share this row: channel ch + e at buf[ch + e]
            __syncwarp();
#pragma unroll
            for (int e = 0; e < V; ++e) buf[ch + e] = f[e];
            __syncwarp();
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int i = ch + e;
                o[e] = i < half ? buf[i + half] : i < rot ? buf[i - half] : 0.f;
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = f[e] * c[e] + (s[e] != 0.f ? o[e] * s[e] : 0.f);
    }
}

template <typename T, int D, int mode, bool bwd>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const RopeArgs a)
{
    constexpr int V = Vec<T>::n, L = D / V, R = 32 / L;  // elements per lane, lanes per row, rows per warp pass
    constexpr int U = bwd ? 2 : 4;                       // passes whose loads are in flight together
    __shared__ float sbuf[mode == kAny ? kWarps * R * D : 1];
    __shared__ float2 scs[kWarps][D / 2];
    __shared__ float sw[bwd ? kWarps * R : 1][bwd ? D : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ch = (lane % L) * V, sub = lane / L, half = a.rot >> 1;
    float *buf = sbuf + (mode == kAny ? (warp * R + sub) * D : 0);
    float wt[2][V], dw[2][V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        wt[0][e] = a.norm && a.wq ? a.wq[ch + e] : 1.f;
        wt[1][e] = a.norm && a.wk ? a.wk[ch + e] : 1.f;
        dw[0][e] = dw[1][e] = 0.f;
    }
    // Few tokens: the warps of a block share one token's heads (a decode step then fills the SMs);
    // many: a warp to a token, whose angles are formed once.
    const int share = a.n < kShareBelow ? kWarps : 1, heads = a.H + a.Hkv;
    const int first = share == 1 ? 0 : warp * R, step = share == 1 ? R : kWarps * R;
    const long long per = kWarps / share;
    for (long long t0 = (long long)blockIdx.x * per; t0 < a.n; t0 += (long long)gridDim.x * per) {
        const long long t = t0 + (share == 1 ? warp : 0);
        if (t >= a.n) break;
        const int pos = a.rot ? a.pos[t] : 0;
        uint4 xr[U], gr[U];  // vectors of the next U passes, as loaded
        auto fetch = [&](int h0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * step + sub;
                xr[u] = gr[u] = make_uint4(0, 0, 0, 0);
                if (h >= heads) continue;
                const bool isk = h >= a.H;
                const size_t off = ((size_t)t * (isk ? a.Hkv : a.H) + (isk ? h - a.H : h)) * D + ch;
                if (!bwd || a.norm) xr[u] = load_raw(static_cast<const T *>(isk ? a.k : a.q) + off);
                if (bwd) gr[u] = load_raw(static_cast<const T *>(isk ? a.dko : a.dqo) + off);
            }
        };
        fetch(first);
        // the token's angles, two or one to a lane
        __syncwarp();
        for (int i = lane; i < half; i += 32) {
            float c, s;
            angle(pos, a.inv[i], a.rot_scale, c, s);
            scs[warp][i] = make_float2(c, bwd ? -s : s);
        }
        __syncwarp();
        float c[V], s[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int i = ch + e;
            const int at = mode == kPair ? i >> 1 : i < half ? i : i - half;
            const float2 cs = i < a.rot ? scs[warp][at] : make_float2(1.f, 0.f);
            c[e] = cs.x;
            s[e] = mode != kPair && i < half ? -cs.y : cs.y;
        }
        for (int h0 = first; h0 < heads; h0 += U * step) {
            uint4 xn[U], gn[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                xn[u] = xr[u];
                gn[u] = gr[u];
            }
            if (h0 + U * step < heads) fetch(h0 + U * step);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * step + sub;
                if (h0 + u * step >= heads) break;  // the whole warp's pass
                const bool live = h < heads, isk = h >= a.H;
                const size_t off = ((size_t)t * (isk ? a.Hkv : a.H) + (live ? (isk ? h - a.H : h) : 0)) * D + ch;
                float x[V], g[V];
                unpack(xn[u], x);
                if (bwd) unpack(gn[u], g);
                float r = 1.f;
                if (a.norm) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < V; ++e) ss += x[e] * x[e];
#pragma unroll
                    for (int m = L / 2; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                    r = rsqrtf(ss * (1.f / D) + a.eps);
                }
                if constexpr (!bwd) {
                    if (a.norm) {
#pragma unroll
                        for (int e = 0; e < V; ++e) x[e] = x[e] * r * (isk ? wt[1][e] : wt[0][e]);
                    }
                    rotate<V, mode>(x, c, s, ch, a.rot, buf, lane);
                    if (live) store_vec(static_cast<T *>(isk ? a.ko : a.qo) + off, x);
                } else {
                    rotate<V, mode>(g, c, s, ch, a.rot, buf, lane);
                    if (a.norm) {
                        float dot = 0.f;
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            x[e] *= r;  // the normalised row
                            const float ux = g[e] * x[e];
                            dw[0][e] += isk ? 0.f : ux;
                            dw[1][e] += isk ? ux : 0.f;
                            g[e] *= isk ? wt[1][e] : wt[0][e];
                            dot += g[e] * x[e];
                        }
#pragma unroll
                        for (int m = L / 2; m >= 1; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
                        dot *= 1.f / D;
#pragma unroll
                        for (int e = 0; e < V; ++e) g[e] = r * (g[e] - x[e] * dot);
                    }
                    if (live) store_vec(static_cast<T *>(isk ? a.dk : a.dq) + off, g);
                }
            }
        }
    }
    if constexpr (bwd) {
        if (!a.partial) return;
        // the block's sums, over its warps in order, into its row of `partial` [2][blocks][D]
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < V; ++e) sw[warp * R + sub][ch + e] = dw[which][e];
            __syncthreads();
            for (int i = threadIdx.x; i < D; i += kWarps * 32) {
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps * R; ++w) sum += sw[w][i];
                a.partial[((size_t)which * gridDim.x + blockIdx.x) * D + i] = sum;
            }
        }
    }
}

// dw[which][ch] = the sum over the blocks' rows of `partial`, in a fixed order.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float *partial, int blocks, int D, float *dwq, float *dwk)
{
    __shared__ float sm[32][33];
    const int which = blockIdx.y, ch = blockIdx.x * 32 + threadIdx.x;
    const float *p = partial + (size_t)which * blocks * D + ch;
    float sum = 0.f;
    for (int b = threadIdx.y; b < blocks; b += 32) sum += p[(size_t)b * D];
    sm[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    float v = sm[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    float *dst = which ? dwk : dwq;
    if (threadIdx.x == 0 && dst) dst[blockIdx.x * 32 + threadIdx.y] = v;
}

unsigned rope_grid(long long n)
{
    const long long want = n < kShareBelow ? n : (n + kWarps - 1) / kWarps;
    const long long most = (long long)device_sms() * 4;
    return (unsigned)(want < most ? want : most);
}

template <typename T, int D, bool bwd> void run(const RopeArgs &a, unsigned grid, cudaStream_t s)
{
    const int half = a.rot >> 1;
    if (a.interleaved || a.rot == 0) rope_kernel<T, D, kPair, bwd><<<grid, kWarps * 32, 0, s>>>(a);
    else if (half % Vec<T>::n == 0) rope_kernel<T, D, kSwap, bwd><<<grid, kWarps * 32, 0, s>>>(a);
    else rope_kernel<T, D, kAny, bwd><<<grid, kWarps * 32, 0, s>>>(a);
}

}  // namespace

int device_sms()
{
    static const int sms = [] {  // of the first device asked: every B200 has as many
        int dev = 0, n = 148;
        if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        return n > 0 ? n : 148;
    }();
    return sms;
}

int rope_bwd_blocks(long long n) { return n > 0 ? (int)rope_grid(n) : 0; }

cudaError_t launch_rope(bool bwd, bool fp32, const RopeArgs &a, cudaStream_t s)
{
    const unsigned grid = rope_grid(a.n);
    if (a.D == 128) {
        if (fp32) bwd ? run<float, 128, true>(a, grid, s) : run<float, 128, false>(a, grid, s);
        else bwd ? run<__nv_bfloat16, 128, true>(a, grid, s) : run<__nv_bfloat16, 128, false>(a, grid, s);
    } else {
        if (fp32) bwd ? run<float, 64, true>(a, grid, s) : run<float, 64, false>(a, grid, s);
        else bwd ? run<__nv_bfloat16, 64, true>(a, grid, s) : run<__nv_bfloat16, 64, false>(a, grid, s);
    }
    if (bwd && a.partial)
        rope_dw_kernel<<<dim3(a.D / 32, 2), dim3(32, 32), 0, s>>>(a.partial, (int)grid, a.D, a.dwq, a.dwk);
    return cudaGetLastError();
}

}  // namespace gdn2
