// kv_q8.cu -- the 8-bit KV cache's rows: bf16 blocks to e4m3 codes with one
// power-of-two scale each (ts_kv_quantize_q8), and selected rows back to
// bf16 (ts_kv_gather_q8).
//
// A block is 64 rows of one KV head of K or of V.  Its scale is 2^e, e the
// least exponent (at least kMinExp) with max|x| <= 448 * 2^e, stored as the
// byte e + 127; code = x * 2^-e rounded to e4m3 (nearest, ties to even).
// Dividing by a power of two is exact, so a code carries one rounding, and
// code * scale is a bf16 number again (4 significant bits), exactly.  A
// block that holds an infinity or a NaN gets the byte 255 and zero codes:
// every reader takes it for NaN.
//
// Both kernels are bound by HBM (long ones) or launch latency (a step's):
// every value is read once, 16 bytes a thread at a time.  32768 rows of 8 heads
// of 128 (201 MB) are quantised in 29.5 us (6.8 TB/s, part of it still in L2
// from call to call); 4096 rows of each of 8 heads out of 102400 positions (25 MB)
// gathered in 5.5 us; one block takes 2.0 us.
#include <cuda_fp8.h>
#include <math.h>

#include "attn_q8.cuh"

namespace ts {
namespace {

constexpr int kThreads = 256;

// Grid (block, KV head, K or V).  The block's values stay in registers
// between the maximum and the conversion.
template <int D>
__global__ void __launch_bounds__(kThreads)
kv_quantize_kernel(QuantArgs a)
{
    constexpr int kUnits = kQ8Block * D / 16;            // 16 values each
    constexpr int kPer = (kUnits + kThreads - 1) / kThreads;
    static_assert(kUnits % kThreads == 0, "whole rounds");
    __shared__ uint32_t top[kThreads / 32];
    const int64_t blk = blockIdx.x;
    const int g = blockIdx.y;
    const __nv_bfloat16 *src = (blockIdx.z ? a.v : a.k) +
                               ((int64_t)g * a.src_cap + blk * kQ8Block) * D;
    const int64_t row = a.dst_row + blk * kQ8Block;
    uint8_t *dst = (blockIdx.z ? a.v8 : a.k8) + ((int64_t)g * a.q8_cap + row) * D;
    uint4 x[kPer][2];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint4 *p = reinterpret_cast<const uint4 *>(src) + 2 * (i * kThreads + threadIdx.x);
        x[i][0] = __ldg(p);
        x[i][1] = __ldg(p + 1);
    }
    // magnitudes order as their bit patterns, infinities and NaN on top
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&x[i][0]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
    }
    m = max(m & 0xFFFFu, m >> 16);
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0)
        top[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
        m = max(m, top[w]);
    const bool fine = m < 0x7F80u;
    // m = 1.f * 2^k: 448 = 1.75 * 2^8, and 1.75 is mantissa 0x60 of 7 bits
    int e = (int)(m >> 7) - 127 - 8 + ((m & 0x7Fu) > 0x60u ? 1 : 0);
    e = e < kQ8MinExp ? kQ8MinExp : e;
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);   // -e in [-120, 100]
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&x[i][0]);
        uint32_t out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 u = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(w + 2 * j));
            const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(w + 2 * j + 1));
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(u.x * inv, u.y * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v.x * inv, v.y * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            out[j] = fine ? (lo | (hi << 16)) : 0u;
        }
        reinterpret_cast<uint4 *>(dst)[i * kThreads + threadIdx.x] =
            make_uint4(out[0], out[1], out[2], out[3]);
    }
    if (threadIdx.x == 0) {
        uint8_t *sc = (blockIdx.z ? a.v_scale : a.k_scale) + (int64_t)g * (a.q8_cap / kQ8Block);
        sc[row / kQ8Block] = fine ? (uint8_t)(e + 127) : 255;
    }
}

// Grid (rows, KV head, K or V): a thread takes 8 values of a kept row.
template <int D>
__global__ void __launch_bounds__(kThreads)
kv_gather_kernel(GatherQ8Args a)
{
    constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
    const int g = blockIdx.y, li = threadIdx.x % kLanes;
    const int t = blockIdx.x * kRows + threadIdx.x / kLanes;
    if (t >= a.n_keep)
        return;
    const bool is_v = blockIdx.z != 0;
    const int n = a.idx[(int64_t)g * a.n_keep + t];
    uint4 out = make_uint4(0u, 0u, 0u, 0u);
    if (n < 0 || n >= a.c.n_q8 + a.c.n_tail) {
        if (li == 0)
            record_status(reinterpret_cast<WorkspaceHeader *>(a.workspace), TS_ERR_DEVICE_ARG);
    } else if (n >= a.c.n_q8) {
        const __nv_bfloat16 *p = (is_v ? a.c.v_tail : a.c.k_tail) +
                                 ((int64_t)g * a.c.tail_cap + (n - a.c.n_q8)) * D;
        out = *(reinterpret_cast<const uint4 *>(p) + li);
    } else {
        const uint8_t *p = (is_v ? a.c.v8 : a.c.k8) + ((int64_t)g * a.c.q8_cap + n) * D;
        const uint2 w = *(reinterpret_cast<const uint2 *>(p) + li);
        const float f = q8_factor((is_v ? a.c.v_scale : a.c.k_scale)[(int64_t)g * (a.c.q8_cap / kQ8Block) +
                                                                     n / kQ8Block]);
        out.x = q8_pair(w.x, f);
        out.y = q8_pair(w.x >> 16, f);
        out.z = q8_pair(w.y, f);
        out.w = q8_pair(w.y >> 16, f);
    }
    __nv_bfloat16 *dst = (is_v ? a.v_partial : a.k_partial) + ((int64_t)g * a.partial_cap + t) * D;
    *(reinterpret_cast<uint4 *>(dst) + li) = out;
}

}  // namespace

cudaError_t kv_quantize_launch(const QuantArgs &a, cudaStream_t stream)
{
    const dim3 grid(a.n_rows / kQ8Block, a.n_heads_kv, 2);
    if (a.head_dim == 128)
        kv_quantize_kernel<128><<<grid, kThreads, 0, stream>>>(a);
    else
        kv_quantize_kernel<64><<<grid, kThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        count_launches(1);
    return e;
}

cudaError_t kv_gather_q8_launch(const GatherQ8Args &a, cudaStream_t stream)
{
    const int rows = kThreads / (a.head_dim / 8);
    const dim3 grid((a.n_keep + rows - 1) / rows, a.n_heads_kv, 2);
    if (a.head_dim == 128)
        kv_gather_kernel<128><<<grid, kThreads, 0, stream>>>(a);
    else
        kv_gather_kernel<64><<<grid, kThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        count_launches(1);
    return e;
}

}  // namespace ts
