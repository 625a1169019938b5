// Keys and values of new tokens written into a paged cache, and read back from it.
//
//   bf16   the row as it is
//   e4m3   scale = amax / 448 over the row's finite channels (fp32), value = e4m3(x / scale), rounded
//          to nearest even; read back as bf16(value * scale).  A row of zeros has scale 0 and reads
//          back as zeros; an infinity or NaN reads back as NaN, its row's other channels as usual.
//
// Bound by memory, and for a decode step by latency: one launch, a warp to a token's row of 256 or
// 128 bytes per head and tensor, 16 bytes a lane.
//
// 32768 tokens, 8 heads, D = 128: bf16 44 us either way (6.0 TB/s), e4m3 written 79 us (bound by the divisions, two for
// each pair of values), read 38 us.
#include <cuda_fp8.h>

#include "attn.cuh"

namespace gdn2 {
namespace {

constexpr int kWarps = 8;
constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

struct CopyArgs {
    SeqBatch b;
    int Hkv, chunks;  // chunks: warps to a token, each a share of its rows
    PagedCache c;
    void *k, *v;
    int *status;
};

template <int D, bool e4m3, bool read>
__global__ void __launch_bounds__(kWarps * 32) cache_copy_kernel(const CopyArgs a)
{
    constexpr int L = D / 8, R = 32 / L;  // lanes to a row (8 channels each), rows a pass
    constexpr int U = e4m3 && !read ? 1 : 4;  // passes whose loads are in flight together
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && threadIdx.x < 32) report_bad_seqlens(a.b, a.status);
    const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const long long t = w / a.chunks;
    if (t >= a.b.rows) return;
    SeqSpan sp;
    const int n = find_seq(a.b, (int)t, sp);
    if (n < 0) return;
    const int kv = a.c.kv_lens[n], pos = kv - sp.len + ((int)t - sp.bos);
    const int pg = pos / a.c.page;
    bool ok = kv >= sp.len && kv <= (long long)a.c.width * a.c.page;  // else the whole sequence is skipped
    const int page = ok ? a.c.table[(size_t)n * a.c.width + pg] : -1;
    ok = ok && page >= 0 && page < a.c.num_pages;
    if (!ok) {
        if (lane == 0) atomicExch(a.status, kStatusBadPages);
        return;
    }
    const size_t slot = ((size_t)page * a.c.page + (pos - pg * a.c.page)) * a.Hkv;  // row of head 0
    const int ch = (lane % L) * 8;
    const int step = a.chunks * R;
    for (int r0 = (int)(w - t * a.chunks) * R; r0 < 2 * a.Hkv; r0 += U * step) {
        char *tok[U], *cell[U];
        float *scale[U];
        uint4 x[U];
        float sc[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {  // all loads first
            const int row = r0 + u * step + lane / L;
            live[u] = row < 2 * a.Hkv;
            const bool isv = live[u] && row >= a.Hkv;
            const int h = live[u] ? (isv ? row - a.Hkv : row) : 0;
            tok[u] = static_cast<char *>(isv ? a.v : a.k) + (((size_t)t * a.Hkv + h) * D + ch) * 2;
            cell[u] = static_cast<char *>(isv ? a.c.v : a.c.k) + ((slot + h) * D + ch) * (e4m3 ? 1 : 2);
            if constexpr (e4m3) scale[u] = (isv ? a.c.vs : a.c.ks) + slot + h;
            x[u] = make_uint4(0, 0, 0, 0);
            sc[u] = 0.f;
            if (!live[u]) continue;
            if constexpr (!read) {
                x[u] = *reinterpret_cast<const uint4 *>(tok[u]);
            } else if constexpr (!e4m3) {
                x[u] = *reinterpret_cast<const uint4 *>(cell[u]);
            } else {
                const uint2 y = *reinterpret_cast<const uint2 *>(cell[u]);
                x[u].x = y.x;
                x[u].y = y.y;
                sc[u] = *scale[u];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (r0 + u * step >= 2 * a.Hkv) break;  // the whole warp's pass
            if constexpr (!e4m3) {
                if (live[u]) *reinterpret_cast<uint4 *>(read ? tok[u] : cell[u]) = x[u];
            } else if constexpr (read) {
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t two = ((i < 2 ? x[u].x : x[u].y) >> (16 * (i & 1))) & 0xffffu;
                    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
                    const float2 f = __half22float2(__half2(hr));  // exact
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(f.y * sc[u]), "f"(f.x * sc[u]));
                }
                if (live[u]) *reinterpret_cast<uint4 *>(tok[u]) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
                const uint32_t xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                float f[8], top = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[2 * i] = bf_lo(xs[i]);
                    f[2 * i + 1] = bf_hi(xs[i]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float m = fabsf(f[i]);
                    top = m < INFINITY ? fmaxf(top, m) : top;  // false for NaN too
                }
#pragma unroll
                for (int m = L / 2; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
                // a true division, so that the row's largest value is 448 exactly; a row whose
                // scale underflows (amax below 448 * 2^-149) holds zeros
                const float q = __fdiv_rn(top, kE4m3Max);
                uint32_t y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float p[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float v = f[2 * i + j];
                        p[j] = fabsf(v) < INFINITY ? (q > 0.f ? __fdiv_rn(v, q) : 0.f) : NAN;
                    }
                    y[i] = __nv_cvt_float2_to_fp8x2(make_float2(p[0], p[1]), __NV_SATFINITE, __NV_E4M3);
                }
                if (live[u]) {
                    *reinterpret_cast<uint2 *>(cell[u]) = make_uint2(y[0] | y[1] << 16, y[2] | y[3] << 16);
                    if (lane % L == 0) *scale[u] = q;
                }
            }
        }
    }
}

template <int D> void run(bool read, const CopyArgs &a, unsigned grid, cudaStream_t s)
{
    if (a.c.e4m3) (read ? cache_copy_kernel<D, true, true> : cache_copy_kernel<D, true, false>)<<<grid, kWarps * 32, 0, s>>>(a);
    else (read ? cache_copy_kernel<D, false, true> : cache_copy_kernel<D, false, false>)<<<grid, kWarps * 32, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_cache_copy(bool read, const SeqBatch &b, int Hkv, int D, const PagedCache &c, void *k, void *v,
                              int *status, cudaStream_t s)
{
    const int R = 32 / (D / 8);
    // A warp moves four passes of rows, whose loads are in flight together; writing e4m3, whose divisions leave no
    // registers for that, one while there are few (8 heads, D = 128, one pass a warp against four: 256 tokens 4.5 us
    // and 7.5, 2048 10.4 and 9.7, 32768 114 and 79).
    const int passes = (2 * Hkv + R - 1) / R;
    const int chunks = !read && c.e4m3 && b.rows * passes <= (1 << 12) ? passes : (passes + 3) / 4;
    CopyArgs a{b, Hkv, chunks, c, k, v, status};
    const long long blocks = (b.rows * chunks + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (D == 128) run<128>(read, a, (unsigned)blocks, s);
    else run<64>(read, a, (unsigned)blocks, s);
    return cudaGetLastError();
}

}  // namespace gdn2
