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
// (bf16: 16 for D = 128, 8 for D = 64; fp32: twice that), four rows' loads in flight to a lane, so that
// the token's cosines and sines stay in registers for all of its heads.  They are multiplied by the
// weights first, and the partner channel comes as it was loaded: y_e = r (x_e (c_e w_e) + x_p (s_e w_p)).
// The angle is formed and reduced modulo 2 pi in 64 bits: pos * inv_freq in fp32 would be off by
// 2^-24 of an angle of up to 10^5.
//
// 32768 tokens, 16 + 16 heads, D = 128, bf16: forward 101 us (5.3 TB/s), backward 173 us (4.7 TB/s) and 3 us
// for the weights' sums.  The rest to the copy rate is the norm's two dependent passes over registers, and in the
// backward the registers of four rows of x and dy, which leave two blocks to an SM.
#include "attn.cuh"

namespace gdn2 {
namespace {

constexpr int kWarps = 8;
constexpr int kShareBelow = 512;  // tokens

template <typename T> constexpr int kVec = 16 / sizeof(T);  // elements of a 16-byte vector

// V elements as V / 2 pairs of fp32
__device__ __forceinline__ void unpack(const uint4 &v, uint64_t (&f)[2])
{
    f[0] = pair(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = pair(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void unpack(const uint4 &v, uint64_t (&f)[4])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack(const uint64_t (&f)[2])
{
    float a, b, c, d;
    unpair(f[0], a, b);
    unpair(f[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}
__device__ __forceinline__ uint4 pack(const uint64_t (&f)[4])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        unpair(f[i], a, b);
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(b), "f"(a));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float sum_of(uint64_t x)
{
    float a, b;
    unpair(x, a, b);
    return a + b;
}

// cos and sin of pos * inv, times f.  The product of an int and a float is exact in 64 bits for positions below
// 2^29, beyond them off by 2^-53 of itself.  The rounded 2 pi adds 2.5e-16 a turn: 4e-12 at an angle of 10^5, 8e-8
// at 2^31, where the product's 1.2e-7 comes on top.  The remainder lies in [-pi, pi], where sincosf needs no long
// reduction.
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

// the channel that channel i is rotated with (itself past rot)
template <int mode> __device__ __forceinline__ int partner(int i, int rot)
{
    if (i >= rot) return i;
    return mode == kPair ? i ^ 1 : i < (rot >> 1) ? i + (rot >> 1) : i - (rot >> 1);
}
// The partners of this lane's channels ch .. ch + V - 1, of vector x as it was loaded.  buf: kAny's
// buffer of this lane's row.
template <typename T, int mode>
__device__ __forceinline__ uint4 partners(const uint4 &x, int ch, int rot, T *buf, int lane)
{
    constexpr int V = kVec<T>;
    if constexpr (mode == kPair) {
        if (ch >= rot) return x;
        uint4 y;
        if constexpr (V == 8) y = make_uint4(__byte_perm(x.x, 0, 0x1032), __byte_perm(x.y, 0, 0x1032), __byte_perm(x.z, 0, 0x1032), __byte_perm(x.w, 0, 0x1032));
        else y = make_uint4(x.y, x.x, x.w, x.z);
        if (ch + V > rot) {  // the rotated part ends inside the vector, after whole pairs
            uint32_t *ys = reinterpret_cast<uint32_t *>(&y);
            const uint32_t *xs = reinterpret_cast<const uint32_t *>(&x);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (ch + e * (V / 4) >= rot) ys[e] = xs[e];
        }
        return y;
    } else if constexpr (mode == kSwap) {
        const int step = (rot >> 1) / V;  // lanes between a channel and its partner
        const int src = ch >= rot ? lane : ch < (rot >> 1) ? lane + step : lane - step;
        return make_uint4(__shfl_sync(0xffffffffu, x.x, src), __shfl_sync(0xffffffffu, x.y, src),
                          __shfl_sync(0xffffffffu, x.z, src), __shfl_sync(0xffffffffu, x.w, src));
    } else {
        __syncwarp();
        *reinterpret_cast<uint4 *>(buf + ch) = x;
        __syncwarp();
        uint4 y;
        T *ys = reinterpret_cast<T *>(&y);
#pragma unroll
        for (int e = 0; e < V; ++e) ys[e] = buf[partner<mode>(ch + e, rot)];
        return y;
    }
}

template <typename T, int D, int mode, bool bwd>
__global__ void __launch_bounds__(kWarps * 32, bwd ? 2 : 3) rope_kernel(const RopeArgs a)
{
    constexpr int V = kVec<T>, P = V / 2, L = D / V, R = 32 / L;  // elements and pairs per lane, lanes per row, rows per pass
    constexpr int U = 4;                                           // passes whose loads are in flight together
    __shared__ __align__(16) T sbuf[mode == kAny ? kWarps * R * D : 8];
    __shared__ float2 scs[kWarps][D / 2];
    __shared__ uint64_t sdw[bwd ? 2 : 1][bwd ? kWarps : 1][bwd ? P : 1][32];  // weight gradients, a lane's own sums
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ch = (lane % L) * V, sub = lane / L, half = a.rot >> 1;
    T *buf = sbuf + (mode == kAny ? (warp * R + sub) * D : 0);
    if constexpr (bwd) {
#pragma unroll
        for (int e = 0; e < P; ++e) sdw[0][warp][e][lane] = sdw[1][warp][e][lane] = 0;
    }
    // Few tokens: the warps of a block share one token's heads (a decode step then fills the SMs);
    // many: a warp to a token, whose angles are formed once.  16 + 16 heads, D = 128, shared against not: 256
    // tokens 6.8 us and 9.6, 384 8.2 and 9.7, 512 11.8 and 10.0, 2048 27 and 13.
    const int share = a.n < kShareBelow ? kWarps : 1;
    const int first = share == 1 ? 0 : warp * R, step = share == 1 ? R : kWarps * R;
    const long long per = kWarps / share;
    for (long long t0 = (long long)blockIdx.x * per; t0 < a.n; t0 += (long long)gridDim.x * per) {
        const long long t = t0 + (share == 1 ? warp : 0);
        if (t >= a.n) break;
        const int pos = a.rot ? a.pos[t] : 0;
        uint4 xr[U], gr[U];
        auto fetch = [&](int isk, int h0) {
            const int heads = isk ? a.Hkv : a.H;
            const T *x = static_cast<const T *>(isk ? a.k : a.q) + (size_t)t * heads * D + ch;
            const T *g = static_cast<const T *>(isk ? a.dko : a.dqo) + (size_t)t * heads * D + ch;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * step + sub;
                xr[u] = gr[u] = make_uint4(0, 0, 0, 0);
                if (h < heads && (!bwd || a.norm)) xr[u] = *reinterpret_cast<const uint4 *>(x + (size_t)h * D);
                if (bwd && h < heads) gr[u] = *reinterpret_cast<const uint4 *>(g + (size_t)h * D);
            }
        };
        fetch(0, first);
        // the token's angles, two or one to a lane, while the first rows come
        __syncwarp();
        for (int i = lane; i < half; i += 32) {
            float c, s;
            angle(pos, a.inv[i], a.rot_scale, c, s);
            scs[warp][i] = make_float2(c, bwd ? -s : s);
        }
        __syncwarp();
#pragma unroll 1
        for (int isk = 0; isk < 2; ++isk) {
            const int heads = isk ? a.Hkv : a.H;
            T *y = static_cast<T *>(bwd ? (isk ? a.dk : a.dq) : (isk ? a.ko : a.qo)) + (size_t)t * heads * D + ch;
            const float *w = a.norm ? (isk ? a.wk : a.wq) : nullptr;
            // own and partner's factors; forward: with the weights of the channels they multiply
            uint64_t own[P], oth[P], wt[P], dw[P];
#pragma unroll
            for (int e = 0; e < P; ++e) {
                float c[2], s[2], f[2];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int i = ch + 2 * e + z;
                    const float2 cs = i < a.rot ? scs[warp][mode == kPair ? i >> 1 : i < half ? i : i - half] : make_float2(1.f, 0.f);
                    f[z] = w ? w[i] : 1.f;
                    c[z] = cs.x;
                    s[z] = (mode == kPair ? !(i & 1) : i < half) ? -cs.y : cs.y;
                    if (!bwd && w) {
                        c[z] *= f[z];
                        s[z] *= w[partner<mode>(i, a.rot)];
                    }
                }
                own[e] = pair(c[0], c[1]);
                oth[e] = pair(s[0], s[1]);
                wt[e] = pair(f[0], f[1]);
                dw[e] = 0;
            }
            for (int h0 = first; h0 < heads; h0 += U * step) {
                if (isk || h0 > first) fetch(isk, h0);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = h0 + u * step + sub;
                    if (h0 + u * step >= heads) break;  // the whole warp's pass
                    uint64_t f[P], o[P];
                    unpack(xr[u], f);
                    float r = 1.f;
                    if (a.norm) {
                        uint64_t s2 = mul2(f[0], f[0]);
#pragma unroll
                        for (int e = 1; e < P; ++e) s2 = fma2(f[e], f[e], s2);
                        float ss = sum_of(s2);
#pragma unroll
                        for (int m = L / 2; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                        r = rsqrtf(ss * (1.f / D) + a.eps);
                        if (bwd && h >= heads) r = 0.f;  // zeros past the heads: not 0 * inf in dw where eps is 0
                    }
                    const uint64_t r2 = pair(r, r);
                    if constexpr (!bwd) {
                        unpack(partners<T, mode>(xr[u], ch, a.rot, buf, lane), o);
#pragma unroll
                        for (int e = 0; e < P; ++e) f[e] = mul2(fma2(o[e], oth[e], mul2(f[e], own[e])), r2);
                        if (h < heads) *reinterpret_cast<uint4 *>(y + (size_t)h * D) = pack(f);
                    } else {
                        uint64_t u2[P];
                        unpack(gr[u], u2);
                        unpack(partners<T, mode>(gr[u], ch, a.rot, buf, lane), o);
                        uint64_t d2 = 0;
#pragma unroll
                        for (int e = 0; e < P; ++e) {
                            u2[e] = fma2(o[e], oth[e], mul2(u2[e], own[e]));
                            if (a.norm) {
                                const uint64_t ux = mul2(u2[e], f[e]);
                                dw[e] = fma2(ux, r2, dw[e]);
                                d2 = fma2(ux, wt[e], d2);
                            }
                        }
                        if (a.norm) {  // dx = u (r w) - x (r^3 / D sum u w x); r^3 alone leaves fp32's range where r does not
                            float dot = sum_of(d2);
#pragma unroll
                            for (int m = L / 2; m >= 1; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
                            dot = dot * r * r * r * (-1.f / D);
                            const uint64_t k2 = pair(dot, dot);
#pragma unroll
                            for (int e = 0; e < P; ++e) u2[e] = fma2(u2[e], mul2(wt[e], r2), mul2(f[e], k2));
                        }
                        if (h < heads) *reinterpret_cast<uint4 *>(y + (size_t)h * D) = pack(u2);
                    }
                }
            }
            if constexpr (bwd) {
#pragma unroll
                for (int e = 0; e < P; ++e) sdw[isk][warp][e][lane] = add2(sdw[isk][warp][e][lane], dw[e]);
            }
        }
    }
    if constexpr (bwd) {
        if (!a.partial) return;
        // the block's sums, over its warps and their rows of a pass in order, into its row of `partial` [2][blocks][D]
        __syncthreads();
        for (int i = threadIdx.x; i < D; i += kWarps * 32) {  // two channels of q or k
            const int which = i / (D / 2), c = i - which * (D / 2);
            uint64_t sum = 0;
#pragma unroll
            for (int w = 0; w < kWarps * R; ++w) sum = add2(sum, sdw[which][w / R][c % P][w % R * L + c / P]);
            *reinterpret_cast<uint64_t *>(a.partial + ((size_t)which * gridDim.x + blockIdx.x) * D + 2 * c) = sum;
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

// Many tokens: as many blocks as run at once (`per` to an SM), so that none starts late (32768 tokens, bf16: three
// and two blocks to an SM 102 and 171 us, six 104 and 177, a warp to a token 112 and 204).
unsigned rope_grid(long long n, int per)
{
    if (n < kShareBelow) return (unsigned)n;
    const long long want = (n + kWarps - 1) / kWarps, most = (long long)device_sms() * per;
    return (unsigned)(want < most ? want : most);
}
constexpr int kBwdPerSm = 2;  // of every backward kernel, and the rows of the weight gradients' partial sums

template <typename T, int D, int mode, bool bwd> cudaError_t run(const RopeArgs &a, cudaStream_t s)
{
    auto kernel = rope_kernel<T, D, mode, bwd>;
    static const int per = [&] {
        int n = 0;
        if (bwd || cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kWarps * 32, 0) != cudaSuccess || n < 1) n = kBwdPerSm;
        return n;
    }();
    kernel<<<rope_grid(a.n, per), kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T, int D, bool bwd> cudaError_t run(const RopeArgs &a, cudaStream_t s)
{
    const int half = a.rot >> 1;
    if (a.interleaved || a.rot == 0) return run<T, D, kPair, bwd>(a, s);
    return half % kVec<T> == 0 ? run<T, D, kSwap, bwd>(a, s) : run<T, D, kAny, bwd>(a, s);
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

int rope_bwd_blocks(long long n) { return n > 0 ? (int)rope_grid(n, kBwdPerSm) : 0; }
// The grid falls where warps stop sharing a token (511 tokens 511 blocks, 512 tokens 64); from there on it grows.
int rope_bwd_most_blocks(long long n)
{
    const int own = rope_bwd_blocks(n), shared = rope_bwd_blocks(n < kShareBelow ? n : kShareBelow - 1);
    return own > shared ? own : shared;
}

cudaError_t launch_rope(bool bwd, bool fp32, const RopeArgs &a, cudaStream_t s)
{
    cudaError_t e;
    if (a.D == 128) {
        if (fp32) e = bwd ? run<float, 128, true>(a, s) : run<float, 128, false>(a, s);
        else e = bwd ? run<__nv_bfloat16, 128, true>(a, s) : run<__nv_bfloat16, 128, false>(a, s);
    } else {
        if (fp32) e = bwd ? run<float, 64, true>(a, s) : run<float, 64, false>(a, s);
        else e = bwd ? run<__nv_bfloat16, 64, true>(a, s) : run<__nv_bfloat16, 64, false>(a, s);
    }
    if (e != cudaSuccess || !bwd || !a.partial) return e;
    rope_dw_kernel<<<dim3(a.D / 32, 2), dim3(32, 32), 0, s>>>(a.partial, rope_bwd_blocks(a.n), a.D, a.dwq, a.dwk);
    return cudaGetLastError();
}

}  // namespace gdn2
