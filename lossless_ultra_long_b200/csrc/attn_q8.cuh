// attn_q8.cuh -- the 8-bit KV cache as the kernels see it: blocks of 64
// rows of e4m3 codes with one power-of-two scale per block and KV head,
// followed by a bf16 tail that holds the newest context rows and the draft
// tree's rows.
#pragma once

#include <cuda_fp8.h>

#include "sm100.cuh"
#include "ts_internal.cuh"

namespace ts {

constexpr int kQ8Block = TS_Q8_BLOCK;   // rows that share a scale
// least exponent of a scale: magnitudes below 2^-100 * 2^-10 round to zero
constexpr int kQ8MinExp = -100;

struct Q8Cache {
    const uint8_t *k8, *v8;             // [Hkv, q8_cap, D] e4m3
    const uint8_t *k_scale, *v_scale;   // [Hkv, q8_cap / 64]: 2^(byte - 127), 255: NaN
    int64_t q8_cap;
    const __nv_bfloat16 *k_tail, *v_tail;   // [Hkv, tail_cap, D]
    int64_t tail_cap;
    int n_q8, n_tail;                   // context rows in 8 bits (a multiple of 64), in the tail
};

struct QuantArgs {
    const __nv_bfloat16 *k, *v;   // first row to quantise; src_cap rows per head apart
    int64_t src_cap;
    int n_heads_kv, head_dim, n_rows;
    uint8_t *k8, *v8, *k_scale, *v_scale;
    int64_t q8_cap, dst_row;
};

struct GatherQ8Args {
    Q8Cache c;
    int n_heads_kv, head_dim;
    const int32_t *idx;   // [Hkv, n_keep]
    int n_keep;
    __nv_bfloat16 *k_partial, *v_partial;
    int64_t partial_cap;
    void *workspace;
};

struct AttnQ8Args {
    Q8Cache c;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    float *root_scores;   // fp32 [Hq, n_q8 + n_tail], base 2, or null
    int n_heads_q, n_heads_kv, head_dim, n_tree;
    float scale_log2;
    void *workspace;
};

cudaError_t kv_quantize_launch(const QuantArgs &a, cudaStream_t stream);
cudaError_t kv_gather_q8_launch(const GatherQ8Args &a, cudaStream_t stream);

size_t attn_q8_workspace_bytes(int n_heads_q, int n_heads_kv, int head_dim, int n_q8, int n_tail,
                               int n_tree, int num_sms);
cudaError_t attn_q8_launch(const AttnQ8Args &a, const TreeMasks &masks, int num_sms,
                           cudaStream_t stream);

// head_dim 128 on the tcgen05 tensor cores (one cooperative launch)
bool attn_q8_t128_eligible(int n_heads_q, int n_heads_kv, int head_dim, int n_q8, int n_tail,
                           int n_tree, int num_sms);
size_t attn_q8_t128_workspace_bytes(int n_heads_q, int n_heads_kv, int n_q8, int n_tail, int n_tree,
                                    int num_sms);
cudaError_t attn_q8_t128_launch(const AttnQ8Args &a, const TreeMasks &masks, int num_sms,
                                cudaStream_t stream);

// Both attention kernels' workspaces: header, this region (four counters per
// set of splits that meet, the tcgen05 kernel's; zero between calls, so that one
// workspace serves calls of any shape), then scratch.
constexpr size_t kQ8SyncBytes = 4096;
constexpr int kQ8MaxSets = (int)kQ8SyncBytes / 16;

// Bounded wait until the int32 at p (written by other CTAs) reaches target.
__device__ __forceinline__ bool wait_count_bounded(const int32_t *p, int target,
                                                   volatile uint32_t *abort, WorkspaceHeader *ws)
{
    const long long t0 = clock64();
    for (;;) {
        int32_t v;
        asm volatile("ld.acquire.gpu.global.b32 %0, [%1];\n" : "=r"(v) : "l"(p) : "memory");
        if (v >= target)
            return true;
        if (clock64() - t0 > sm100::kWaitCycles) {
            *abort = 1u;
            record_status(ws, TS_ERR_TIMEOUT);
            return false;
        }
        __nanosleep(64);
    }
}

// the factor a scale byte stands for (bytes below the least scale read as
// it), its exponent, and its inverse; 255 is NaN
__device__ __forceinline__ float q8_factor(uint32_t byte)
{
    return __uint_as_float(byte == 255u ? 0x7FC00000u : max(byte, (uint32_t)(kQ8MinExp + 127)) << 23);
}
__device__ __forceinline__ float q8_log2(uint32_t byte)
{
    return byte == 255u ? __uint_as_float(0x7FC00000u) : (float)max((int)byte - 127, kQ8MinExp);
}
__device__ __forceinline__ float q8_inverse(uint32_t byte)
{
    // 2^-127, the inverse of the largest, is a subnormal
    return __uint_as_float(byte == 255u   ? 0x7FC00000u
                           : byte == 254u ? 0x00400000u
                                          : (254u - max(byte, (uint32_t)(kQ8MinExp + 127))) << 23);
}

// two codes (low byte first) times f, rounded to bf16 (exactly, for a power
// of two inside bf16's normal range)
__device__ __forceinline__ uint32_t q8_pair(uint32_t two, float f)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3);
    const float2 x = __half22float2(__half2(h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(x.x * f, x.y * f);
    return *reinterpret_cast<const uint32_t *>(&b);
}

}  // namespace ts
