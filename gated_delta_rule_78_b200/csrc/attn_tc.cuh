// Pieces shared by the tensor-core attention kernels (attn_fwd_tc.cu, attn_bwd_tc.cu): tile sizes,
// the packing of query rows, bounded waits, and the bf16 tiles' products.
//
// Query rows are packed by key head: row r of a tile of kBM rows is token r / G, query head r % G of
// the G = H / Hkv heads that read one key head, so one key tile serves all of them (a tile holds
// kTQ = kBM / G tokens; rows past kTQ * G are not used).  A packed tile arrives by one TMA box of
// (64 channels, G heads, kTQ tokens) per 64 channels.
#pragma once

#include <cuda_fp16.h>

#include "attn.cuh"
#include "tc_util.cuh"

namespace gdn2 {
namespace attn {

constexpr int kBM = 128, kBN = 128;      // query rows and keys of a tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kBoxBytes = kBM * 128;     // 128 rows of 64 bf16 channels (one SW128 column block)

// A bounded wait that every role of a block leaves once one of them has given up.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort, int *status)
{
    if (tc::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = tc::global_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 16; ++i)
            if (tc::mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (tc::global_ns() - t0 > 2000000000ull) {
            *abort = 1;
            atomicExch(status, kStatusTimeout);
            return false;
        }
    }
}

// ... by a whole warp, with one answer for all of its lanes
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort, int *status)
{
    return __all_sync(0xffffffffu, wait(bar, parity, abort, status));
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
// Warp-uniform copies: the tensor core's instructions take their operands from uniform registers, and the
// compiler keeps them there only where it can see that control flow and values are uniform.  A product
// issued under `lane == 0` instead took 75 cycles, more than it runs.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// tcgen05.mma and commit by the lane that `leader` marks, in code that the whole warp runs
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 q, %0, 0;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%1], %2, %3, %4, p;\n\t}"
        ::"r"(leader), "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 q, %0, 0;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], %3, %4, p;\n\t}"
        ::"r"(leader), "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %0, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}"
        ::"r"(leader), "r"(tc::smem_u32(bar))
        : "memory");
}

// After a wait that gave up: products in flight end before the block frees its memory.
__device__ __forceinline__ void drain(uint32_t leader, uint64_t *bar)
{
    commit(leader, bar);
    tc::mbar_wait(bar, 0, 1000000000ull);
    __syncwarp();
}

// after a wait that gave up: the loads of a ring, `n` of them issued, end before the block's memory is free
__device__ __forceinline__ void drain_ring(uint64_t *full, int n, int stages)
{
    for (int i = n > stages ? n - stages : 0; i < n; ++i) tc::mbar_wait(&full[i % stages], (i / stages) & 1, 1000000000ull);
}

// D (128 x N, fp32, TMEM) = A (128 x 16 ks) B^T: both operands K-major SW128 tiles in column blocks of 64
// channels, of 128 rows.
template <int kSteps>
__device__ __forceinline__ void mma_kk(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc)
{
    const uint64_t da = tc::sdesc_sw128(a, 16, 1024), db = tc::sdesc_sw128(b, 16, 1024);
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) {  // offsets in the descriptors' units of 16 bytes
        const uint64_t in = (ks & 3) * 2;
        mma_ss(leader, d, da + (ks >> 2) * (kBoxBytes >> 4) + in, db + (ks >> 2) * (kBoxBytes >> 4) + in, idesc, ks > 0);
    }
}
// D (128 x N) (+)= A B with A (128 x 16 ks, bf16, 8 columns a step) in TMEM and B the same number of rows, from
// `row` on, of a tile [128 rows][N channels] in shared memory, N-major.
template <int kSteps>
__device__ __forceinline__ void mma_tn(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, int row, uint32_t idesc, uint32_t acc)
{
    const uint64_t db = tc::sdesc_sw128(b + row * 128, kBoxBytes, 1024);
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) mma_ts(leader, d, a + 8 * ks, db + ks * 128, idesc, ks > 0 ? 1u : acc);
}
// Zeros in rows [from, 128) of an SW128 tile of kBlocks column blocks, by one warp, visible to the
// tensor core's reads that the warp issues afterwards.
template <int kBlocks> __device__ __forceinline__ void zero_rows(char *tile, int from)
{
    const int lane = threadIdx.x & 31;
    for (int i = from * 8 + lane; i < kBN * 8; i += 32)
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) *reinterpret_cast<uint4 *>(tile + b * kBoxBytes + i * 16) = make_uint4(0, 0, 0, 0);
    tc::fence_proxy_async_smem();
    __syncwarp();
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// the larger of two values, NaN where one is
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// 2^x of two values on the FMA pipe, for x in [-126, 127] (below: as -126; NaN: infinite in bf16).  x = n + f, n its nearest
// integer, found by adding 1.5 * 2^23; 2^f on [-1/2, 1/2] by its interpolant of degree 5 at Chebyshev nodes with
// the constant term set to 1, so that whole powers are exact (2.1e-7 relative, the interpolant itself 1.0e-7; in
// fp32 2.7e-7); n is added to the exponent.
__device__ __forceinline__ void ex2_fma(uint64_t x, float &a, float &b)
{
    float x0, x1;
    unpair(x, x0, x1);
    x = pair(max_nan(x0, -126.f), max_nan(x1, -126.f));
    const uint64_t magic = pair(12582912.f, 12582912.f), minus = pair(-12582912.f, -12582912.f);
    const uint64_t t = add2(x, magic), n = add2(t, minus);
    const uint64_t f = fma2(n, pair(-1.f, -1.f), x);
    constexpr float k[6] = {1.f, 0.693147182f, 0.240221068f, 0.0555035695f, 0.00967603177f, 0.00133908633f};
    uint64_t y = pair(k[5], k[5]);
#pragma unroll
    for (int i = 4; i >= 0; --i) y = fma2(y, f, pair(k[i], k[i]));
    float y0, y1, t0, t1;
    unpair(y, y0, y1);
    unpair(t, t0, t1);
    a = __int_as_float(__float_as_int(y0) + (__float_as_int(t0) << 23));
    b = __int_as_float(__float_as_int(y1) + (__float_as_int(t1) << 23));
}

// Four e4m3 values as two pairs of bf16 (exact: e4m3 -> f16 -> f32 -> bf16).
__device__ __forceinline__ void e4m3x4_bf16(uint32_t x, uint32_t &lo, uint32_t &hi)
{
    uint32_t h0, h1;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(h0), "=r"(h1)
        : "r"(x));
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&h0));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&h1));
    lo = tc::pack_bf16x2(f0.x, f0.y);
    hi = tc::pack_bf16x2(f1.x, f1.y);
}

// The tile and key head of block `block` of a grid of tiles * Hkv blocks.  Without a window tiles differ
// in cost by their length: the heavy ones first, all heads' together.  With a window almost all cost
// the same, and a head's neighbouring tiles, which share most of their keys, run together: K and V of
// all heads at once do not stay in L2 (4 x 4096, 16 heads, window 2048: forward, dk/dv and dq take
// 8 to 10% longer heavy-first; the other way round a causal dk/dv at d = 64 takes 40% longer).
__device__ __forceinline__ bool block_tile(const SeqBatch &b, int block, int tiles, int Hkv, int window, int per, bool from_end,
                                           TileRef &r, int &head)
{
    bool ok;
    if (window) {
        head = block / tiles;
        const int i = block - head * tiles;
        ok = find_tile(b, from_end ? i : tiles - 1 - i, per, r);
    } else {
        head = block % Hkv;
        ok = find_heavy_tile(b, block / Hkv, per, from_end, r);
    }
    head = uniform(head);
    r.tile = uniform(r.tile);
    r.sp.len = uniform(r.sp.len);
    return ok;
}

// The block's k'th piece of work where pieces lie in order of falling cost: back and forth, so that no
// block gets the heaviest of every round (dk/dv at d = 64, packed: 127 us forth only).  Past the
// last piece's round -1; a number of `works` or more is no work, but others may follow.
__device__ __forceinline__ int work_at(int k, int works)
{
    const int g = gridDim.x;
    return (long long)k * g >= works ? -1 : k * g + (k & 1 ? g - 1 - (int)blockIdx.x : (int)blockIdx.x);
}

// TMA view of a bf16 [rows][heads][D] tensor: boxes of (64 channels, box_heads, box_rows).
bool make_head_map(CUtensorMap *m, const void *ptr, long long rows, int heads, int D, int box_heads, int box_rows);

// 32 bytes in one store, in two where p is aligned to 16 bytes only (as a caller's tensor may be)
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8])
{
    if (((uintptr_t)p & 31) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        uint4 *d = static_cast<uint4 *>(p);
        d[0] = make_uint4(w[0], w[1], w[2], w[3]);
        d[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

}  // namespace attn
}  // namespace gdn2
