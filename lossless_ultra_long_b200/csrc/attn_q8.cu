// attn_q8.cu -- tree-verify attention over the 8-bit KV cache, on warp-level
// mma.sync: the general kernel (any head_dim 64/128, group, tree size and
// context length), and the dispatch between it and the tcgen05 kernel.
//
// For node i and head h, over the context and the node's root path:
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(c s_b(j) q.k8_j - m)
// where k8 are the e4m3 codes of block b(j), s_b its power-of-two scale and
// c = softmax scale * log2 e.  A scale belongs to 64 rows of a head, so it
// leaves both products: QK^T runs on the codes and the scores are multiplied
// by c s_b; the weights are multiplied by V's scale before PV.  Codes are
// bf16 numbers (4 significant bits), so both products are exact up to their
// fp32 accumulation and, for PV, the two bf16 parts of P.
//
// Bound: short contexts, where a call is a chain of latencies (the launch, one
// or two tiles, the combine): 8 heads of 64 over 2, 13 nodes, 2048 positions
// 9.0 us; one node, 212 positions 7.6 us.
//
// Work split: grid (splits, Hkv, row blocks).  A CTA streams a contiguous
// range of tiles: a tile is one 64-row block of the 8-bit cache or 64 rows
// of the bf16 tail (context, then the tree).  cp.async brings the bytes into
// a three-stage ring; a block's codes are turned into bf16 rows in a work
// tile, a tail tile is used where it lies.  Only tail tiles evaluate masks.
// A tail row of K or of V that holds an infinity or a NaN is kept out of its
// product (0 * NaN would reach rows that do not see it) and turns the rows that do
// see its position into NaN.
#include <math.h>

#include "attn_q8.cuh"

namespace ts {
namespace {

constexpr int kTile = kQ8Block;
constexpr int kStages = 3;
constexpr int kMaxWarps = 12;    // 192 query rows per CTA
// Contexts of at most so many tiles are one split: two tiles in turn cost less
// than the meeting of two splits.  Four tiles (212 positions, D = 64) are
// 6.5 us as four splits with their combine and 10.2 us as one split.
constexpr int kOneSplit = 2;

__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid)
{
    const int n = valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n));
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2,
                                        uint32_t &r3)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2,
                                          uint32_t &r3)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// (lo, hi) floats -> bf16x2 of their rounding, and bf16x2 of the remainders
__device__ __forceinline__ void split_bf16(float lo, float hi, uint32_t &big, uint32_t &small)
{
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    const float2 back = __bfloat1622float2(h);
    __nv_bfloat162 r = __floats2bfloat162_rn(lo - back.x, hi - back.y);
    big = *reinterpret_cast<uint32_t *>(&h);
    small = *reinterpret_cast<uint32_t *>(&r);
}
// byte offset of 16-byte chunk `c` of bf16 tile row `r`
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c)
{
    return static_cast<uint32_t>(r * (D * 2) + ((c ^ (r & 7)) << 4));
}
// whether a 32-bit word of two bf16 values holds an infinity or a NaN
__device__ __forceinline__ bool odd_pair(uint32_t w)
{
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

template <int D>
struct Shape {
    static constexpr int kTileBytes = kTile * D * 2;   // K or V of a tile in bf16
    static constexpr int kSmem = (kStages + 1) * 2 * kTileBytes;
};

// Output row: out = sum_s 2^(m_s - M) acc_s / sum_s 2^(m_s - M) l_s.  A split
// whose row saw nothing has m = -inf; its l is 0, or NaN where the row saw a
// value that is no number there.
constexpr int kB = 12;   // splits whose loads a warp has in flight together

__device__ __forceinline__ float row_max(const float *ws_ml, int row, int rows_all, int n_split)
{
    float M = -INFINITY;
    for (int s = threadIdx.x & 31; s < n_split; s += 32)
        M = fmaxf(M, __ldcg(ws_ml + ((size_t)s * rows_all + row) * 2));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    return M;
}

// Adds splits s0, s0 + step, ... of a row to a warp's acc (D / 32 elements a
// lane) and L.
template <int D>
__device__ __forceinline__ void add_splits(const float *ws_o, const float *ws_ml, int row, int rows_all,
                                           int s0, int step, int n_split, float M, float (&acc)[D / 32],
                                           float &L)
{
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    for (; s0 < n_split; s0 += kB * step) {
        float2 ml[kB];
        float x[kB][PER];
#pragma unroll
        for (int u = 0; u < kB; ++u) {
            ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < PER; ++e)
                x[u][e] = 0.f;
            if (s0 + u * step < n_split) {
                const size_t at = (size_t)(s0 + u * step) * rows_all + row;
                ml[u] = __ldcg(reinterpret_cast<const float2 *>(ws_ml + at * 2));
                const float *src = ws_o + at * D + lane * PER;
                if constexpr (PER == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
                    x[u][0] = v.x; x[u][1] = v.y; x[u][2] = v.z; x[u][3] = v.w;
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
                    x[u][0] = v.x; x[u][1] = v.y;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kB; ++u) {
            const float w = ml[u].x == -INFINITY ? 0.f : exp2f(ml[u].x - M);
            L += w * ml[u].y;
#pragma unroll
            for (int e = 0; e < PER; ++e)
                acc[e] += w * x[u][e];
        }
    }
}

template <int D>
__device__ __forceinline__ void write_row(__nv_bfloat16 *out, int row, const float (&acc)[D / 32], float L)
{
    const float inv = 1.f / L;
    __nv_bfloat162 *dst = reinterpret_cast<__nv_bfloat162 *>(out + (size_t)row * D +
                                                             (threadIdx.x & 31) * (D / 32));
#pragma unroll
    for (int e = 0; e < D / 64; ++e)
        dst[e] = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
}

template <int D>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
attn_q8_kernel(AttnQ8Args a, TreeMasks masks, int tiles_per_split, int n_split, int meet)
{
    extern __shared__ __align__(128) unsigned char smem[];
    // tail tile: rows with a value that is no number, and those of K among them
    __shared__ unsigned long long odd_rows, odd_keys;
    __shared__ uint32_t gave_up;
    constexpr int TB = Shape<D>::kTileBytes;
    const Q8Cache &kc = a.c;

    if (threadIdx.x == 0) {
        gave_up = 0u;
        sm100::launch_dependents();
    }
    sm100::grid_dependency_wait();   // what the previous kernel wrote
    const int split = blockIdx.x, g = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nthreads = blockDim.x;
    const int G = a.n_heads_q / a.n_heads_kv;
    const int R = G * a.n_tree;
    const int n_blocks = kc.n_q8 / kTile;
    const int tail_rows = kc.n_tail + a.n_tree;
    const int n_tiles_all = n_blocks + (tail_rows + kTile - 1) / kTile;
    const int t_begin = split * tiles_per_split;
    const int n_tiles = min(t_begin + tiles_per_split, n_tiles_all) - t_begin;

    const uint8_t *k8 = kc.k8 + (int64_t)g * kc.q8_cap * D, *v8 = kc.v8 + (int64_t)g * kc.q8_cap * D;
    const uint8_t *ksc = kc.k_scale + (int64_t)g * (kc.q8_cap / kTile);
    const uint8_t *vsc = kc.v_scale + (int64_t)g * (kc.q8_cap / kTile);
    const __nv_bfloat16 *kt = kc.k_tail + (int64_t)g * kc.tail_cap * D;
    const __nv_bfloat16 *vt = kc.v_tail + (int64_t)g * kc.tail_cap * D;
    unsigned char *work = smem + kStages * 2 * TB;
    const uint32_t sbase = smem_u32(smem);

    auto load_tile = [&](int t_local, int stage) {
        const int tile = t_begin + t_local;
        const uint32_t ks = sbase + stage * 2 * TB, vs = ks + TB;
        if (tile < n_blocks) {
            // codes as they lie: rows of D bytes
            const int64_t off = (int64_t)tile * kTile * D;
            for (int c = threadIdx.x; c < kTile * D / 16; c += nthreads) {
                cp_async16(ks + 16 * c, k8 + off + 16 * c, true);
                cp_async16(vs + 16 * c, v8 + off + 16 * c, true);
            }
            return;
        }
        constexpr int CH = D / 8;
        const int r0 = (tile - n_blocks) * kTile;
        for (int c = threadIdx.x; c < kTile * CH; c += nthreads) {
            const int r = c / CH, ch = c % CH;
            const bool ok = r0 + r < tail_rows;
            const int64_t off = (int64_t)(ok ? r0 + r : 0) * D + ch * 8;
            cp_async16(ks + swz<D>(r, ch), kt + off, ok);
            cp_async16(vs + swz<D>(r, ch), vt + off, ok);
        }
    };

#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        if (s < n_tiles)
            load_tile(s, s);
        cp_async_commit();
    }

    // ---- this warp's 16 rows: Q fragments stay in registers
    const int row_base = blockIdx.z * blockDim.x / 2 + warp * 16;  // 16 rows per warp
    const int qr = lane >> 2, qc = (lane & 3) * 2;
    int rnode[2], rhead[2];
    bool rvalid[2];
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
        const int r = row_base + qr + hi * 8;
        rvalid[hi] = r < R;
        const int rr = rvalid[hi] ? r : 0;
        rnode[hi] = rr / G;
        rhead[hi] = g * G + rr % G;
    }
    uint32_t qa[D / 16][4];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
            const __nv_bfloat16 *qrow =
                a.q + ((int64_t)rnode[hi] * a.n_heads_q + rhead[hi]) * D + kk * 16 + qc;
            qa[kk][hi] = rvalid[hi] ? *reinterpret_cast<const uint32_t *>(qrow) : 0u;
            qa[kk][2 + hi] = rvalid[hi] ? *reinterpret_cast<const uint32_t *>(qrow + 8) : 0u;
        }
    }
    const unsigned long long anc0 = masks.anc[rnode[0]], anc1 = masks.anc[rnode[1]];
    const int n_ctx = kc.n_q8 + kc.n_tail;

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
        o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};

    for (int t = 0; t < n_tiles; ++t) {
        cp_async_wait<kStages - 2>();
        __syncthreads();   // also: the work tile and odd_rows of tile t - 1 are free
        if (t + kStages - 1 < n_tiles)
            load_tile(t + kStages - 1, (t + kStages - 1) % kStages);
        cp_async_commit();

        const int tile = t_begin + t, stage = t % kStages;
        unsigned char *raw = smem + stage * 2 * TB;
        const bool q8 = tile < n_blocks;
        float sk = 1.f, sv = 1.f;
        uint32_t ks, vs;
        unsigned long long odd = 0ull, odd_k = 0ull;
        if (q8) {
            sk = q8_factor(ksc[tile]);
            sv = q8_factor(vsc[tile]);
            // codes -> bf16 rows: 16 codes are two 16-byte chunks
            for (int u = threadIdx.x; u < 2 * kTile * D / 16; u += nthreads) {
                const int which = u / (kTile * D / 16), c = u % (kTile * D / 16);
                const int r = c / (D / 16), ch = 2 * (c % (D / 16));
                const uint4 w = *reinterpret_cast<const uint4 *>(raw + which * TB + 16 * c);
                unsigned char *dst = work + which * TB;
                *reinterpret_cast<uint4 *>(dst + swz<D>(r, ch)) =
                    make_uint4(q8_pair(w.x, 1.f), q8_pair(w.x >> 16, 1.f), q8_pair(w.y, 1.f),
                               q8_pair(w.y >> 16, 1.f));
                *reinterpret_cast<uint4 *>(dst + swz<D>(r, ch + 1)) =
                    make_uint4(q8_pair(w.z, 1.f), q8_pair(w.z >> 16, 1.f), q8_pair(w.w, 1.f),
                               q8_pair(w.w >> 16, 1.f));
            }
            ks = smem_u32(work);
        } else {
            // rows with an infinity or a NaN leave their product
            if (threadIdx.x == 0)
                odd_rows = odd_keys = 0ull;
            __syncthreads();
            for (int c = threadIdx.x; c < kTile * D / 4; c += nthreads) {
                const int which = c / (kTile * D / 8), ch = c % (kTile * D / 8);
                const int r = ch / (D / 8);
                const uint4 w = *reinterpret_cast<const uint4 *>(raw + which * TB + 16 * ch);
                if (odd_pair(w.x) || odd_pair(w.y) || odd_pair(w.z) || odd_pair(w.w)) {
                    atomicOr(&odd_rows, 1ull << r);
                    if (which == 0)
                        atomicOr(&odd_keys, 1ull << r);
                }
            }
            __syncthreads();
            odd = odd_rows;
            odd_k = odd_keys;
            if (odd) {
                // (a key whose value is no number still has its score)
                for (int c = threadIdx.x; c < kTile * D / 4; c += nthreads) {
                    const int which = c / (kTile * D / 8), ch = c % (kTile * D / 8);
                    if (((which ? odd : odd_k) >> (ch / (D / 8))) & 1ull)
                        *reinterpret_cast<uint4 *>(raw + which * TB + 16 * ch) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
            }
            ks = smem_u32(raw);
        }
        vs = ks + TB;
        __syncthreads();
        const int mrow = lane & 7, mat = lane >> 3;

        float s[kTile / 8][4];
#pragma unroll
        for (int i = 0; i < kTile / 8; ++i)
            s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
            for (int np = 0; np < kTile / 16; ++np) {
                uint32_t b0, b1, b2, b3;
                const int tok = np * 16 + (mat >> 1) * 8 + mrow;
                ldsm_x4(ks + swz<D>(tok, kk * 2 + (mat & 1)), b0, b1, b2, b3);
                mma_bf16(s[2 * np], qa[kk], b0, b1);
                mma_bf16(s[2 * np + 1], qa[kk], b2, b3);
            }
        }

        // scale to base 2, mask, online softmax.  Row i sees tail position
        // r0 + p (p < 64) iff bit p of vis
        const int r0 = (tile - n_blocks) * kTile;
        unsigned long long vis[2] = {~0ull, ~0ull};
        if (!q8) {
            const int d = kc.n_tail - r0;   // context rows of this tile, before the tree's
            const unsigned long long ctx = d >= 64 ? ~0ull : (d > 0 ? (1ull << d) - 1ull : 0ull);
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const unsigned long long anc = hi ? anc1 : anc0;   // no bits at or past n_tree
                unsigned long long v = ctx;
                if (d <= 0)
                    v |= -d < 64 ? anc >> (-d) : 0ull;
                else if (d < 64)
                    v |= anc << d;
                vis[hi] = v;
                if (v & odd)
                    l_run[hi] = __uint_as_float(0x7FC00000u);
            }
        }
        const float sc = a.scale_log2 * sk;
        const int pos0 = q8 ? tile * kTile : kc.n_q8 + r0;
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nt = 0; nt < kTile / 8; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int hi = e >> 1, p = nt * 8 + qc + (e & 1);
                float x = s[nt][e] * sc;
                if (a.root_scores && rnode[hi] == 0 && rvalid[hi] && pos0 + p < n_ctx)
                    a.root_scores[(int64_t)rhead[hi] * n_ctx + pos0 + p] =
                        (odd_k >> p) & 1ull ? __uint_as_float(0x7FC00000u) : x;
                if (!q8 && !((vis[hi] >> p) & 1ull))
                    x = -INFINITY;
                s[nt][e] = x;
                mx[hi] = fmaxf(mx[hi], x);
            }
        }
        float corr[2], mref[2];
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
            mx[hi] = fmaxf(mx[hi], __shfl_xor_sync(0xffffffffu, mx[hi], 1));
            mx[hi] = fmaxf(mx[hi], __shfl_xor_sync(0xffffffffu, mx[hi], 2));
            const float m_new = fmaxf(m_run[hi], mx[hi]);
            mref[hi] = m_new == -INFINITY ? 0.f : m_new;
            corr[hi] = exp2f(m_run[hi] - mref[hi]);
            m_run[hi] = m_new;
            l_run[hi] *= corr[hi];
        }
#pragma unroll
        for (int nt = 0; nt < kTile / 8; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p = exp2f(s[nt][e] - mref[e >> 1]);
                l_run[e >> 1] += p;
                s[nt][e] = p * sv;
            }
        }
#pragma unroll
        for (int dt = 0; dt < D / 8; ++dt) {
            o[dt][0] *= corr[0];
            o[dt][1] *= corr[0];
            o[dt][2] *= corr[1];
            o[dt][3] *= corr[1];
        }

        // O += P V, with P = P_hi + P_lo (two bf16 parts, ~16 significant bits)
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk) {
            uint32_t pa[4], pl[4];
            split_bf16(s[2 * kk][0], s[2 * kk][1], pa[0], pl[0]);
            split_bf16(s[2 * kk][2], s[2 * kk][3], pa[1], pl[1]);
            split_bf16(s[2 * kk + 1][0], s[2 * kk + 1][1], pa[2], pl[2]);
            split_bf16(s[2 * kk + 1][2], s[2 * kk + 1][3], pa[3], pl[3]);
#pragma unroll
            for (int dp = 0; dp < D / 16; ++dp) {
                uint32_t b0, b1, b2, b3;
                const int tok = kk * 16 + (mat & 1) * 8 + mrow;
                ldsm_x4_t(vs + swz<D>(tok, dp * 2 + (mat >> 1)), b0, b1, b2, b3);
                mma_bf16(o[2 * dp], pa, b0, b1);
                mma_bf16(o[2 * dp + 1], pa, b2, b3);
                mma_bf16(o[2 * dp], pl, b0, b1);
                mma_bf16(o[2 * dp + 1], pl, b2, b3);
            }
        }
    }
    cp_async_wait<0>();

    // ---- epilogue
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
        l_run[hi] += __shfl_xor_sync(0xffffffffu, l_run[hi], 1);
        l_run[hi] += __shfl_xor_sync(0xffffffffu, l_run[hi], 2);
    }
    const int rows_all = a.n_tree * a.n_heads_q;
    float *ws_o = reinterpret_cast<float *>(reinterpret_cast<char *>(a.workspace) + kHeaderBytes + kQ8SyncBytes);
    float *ws_ml = ws_o + (size_t)n_split * rows_all * D;
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
        if (!rvalid[hi])
            continue;
        const int orow = rnode[hi] * a.n_heads_q + rhead[hi];
        if (n_split == 1) {
            const float inv = 1.f / l_run[hi];
            __nv_bfloat16 *dst = a.out + (int64_t)orow * D;
#pragma unroll
            for (int dt = 0; dt < D / 8; ++dt)
                *reinterpret_cast<__nv_bfloat162 *>(dst + dt * 8 + qc) =
                    __floats2bfloat162_rn(o[dt][2 * hi] * inv, o[dt][2 * hi + 1] * inv);
        } else {
            float *dst = ws_o + ((size_t)split * rows_all + orow) * D;
#pragma unroll
            for (int dt = 0; dt < D / 8; ++dt)
                *reinterpret_cast<float2 *>(dst + dt * 8 + qc) =
                    make_float2(o[dt][2 * hi], o[dt][2 * hi + 1]);
            if ((lane & 3) == 0)
                *reinterpret_cast<float2 *>(ws_ml + ((size_t)split * rows_all + orow) * 2) =
                    make_float2(m_run[hi], l_run[hi]);
        }
    }
    if (!meet)
        return;

    // ---- few splits and rows (a cooperative launch): once every split of
    // these rows has arrived, each folds every n_split-th row
    WorkspaceHeader *hdr = reinterpret_cast<WorkspaceHeader *>(a.workspace);
    int32_t *ctr = reinterpret_cast<int32_t *>(reinterpret_cast<char *>(a.workspace) + kHeaderBytes) +
                   4 * (g * gridDim.z + blockIdx.z);
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();   // the partials before the arrival
        atomicAdd(&ctr[1], 1);
        wait_count_bounded(&ctr[1], n_split, &gave_up, hdr);
    }
    __syncthreads();
    const int row0 = blockIdx.z * nthreads / 2, row1 = min(R, row0 + nthreads / 2);
    if (!*(volatile uint32_t *)&gave_up) {
        for (int r = row0 + split + warp * n_split; r < row1; r += (nthreads / 32) * n_split) {
            const int row = (r / G) * a.n_heads_q + g * G + r % G;
            float acc[D / 32] = {}, L = 0.f;
            add_splits<D>(ws_o, ws_ml, row, rows_all, 0, 1, n_split,
                          row_max(ws_ml, row, rows_all, n_split), acc, L);
            write_row<D>(a.out, row, acc, L);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(&ctr[2], 1) == n_split - 1) {
        atomicExch(&ctr[1], 0);
        atomicExch(&ctr[2], 0);
    }
}

// The combine as a launch of its own (dependent: it starts while the splits
// run), `per_row` warps to a row.
template <int D>
__global__ void __launch_bounds__(256)
attn_q8_combine_kernel(const float *__restrict__ ws_o, const float *__restrict__ ws_ml,
                       __nv_bfloat16 *out, int rows_all, int n_split, int per_row)
{
    constexpr int PER = D / 32;
    __shared__ float part[8][32][PER + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp % per_row;
    const int row = blockIdx.x * (8 / per_row) + warp / per_row;
    sm100::launch_dependents();
    sm100::grid_dependency_wait();   // the splits' partials
    float acc[PER] = {}, L = 0.f;
    if (row < rows_all)
        add_splits<D>(ws_o, ws_ml, row, rows_all, w, per_row, n_split,
                      row_max(ws_ml, row, rows_all, n_split), acc, L);
    if (per_row > 1) {
#pragma unroll
        for (int e = 0; e < PER; ++e)
            part[warp][lane][e] = acc[e];
        part[warp][lane][PER] = L;
        __syncthreads();
        if (w == 0)
            for (int v = 1; v < per_row; ++v) {
#pragma unroll
                for (int e = 0; e < PER; ++e)
                    acc[e] += part[warp + v][lane][e];
                L += part[warp + v][lane][PER];
            }
    }
    if (row < rows_all && w == 0)
        write_row<D>(out, row, acc, L);
}

struct SplitPlan {
    int warps, row_blocks, n_split, tiles_per_split;
    bool meet;   // the splits combine their rows themselves
};

SplitPlan make_plan(int n_heads_q, int n_heads_kv, int head_dim, int n_q8, int n_tail, int n_tree, int num_sms)
{
    SplitPlan p;
    const int R = (n_heads_q / n_heads_kv) * n_tree;
    const int warps_needed = (R + 15) / 16;
    p.row_blocks = (warps_needed + kMaxWarps - 1) / kMaxWarps;
    p.warps = (warps_needed + p.row_blocks - 1) / p.row_blocks;
    const int n_tiles = n_q8 / kTile + (n_tail + n_tree + kTile - 1) / kTile;
    int want = num_sms / (n_heads_kv * p.row_blocks);
    want = want < 1 ? 1 : (want > n_tiles ? n_tiles : want);
    if (n_tiles <= kOneSplit)
        want = 1;
    p.tiles_per_split = (n_tiles + want - 1) / want;
    p.n_split = (n_tiles + p.tiles_per_split - 1) / p.tiles_per_split;
    // One launch, without a combine of its own, for heads of 64 where a warp has no
    // more than one row to fold, of no more splits than it loads at once: it spares
    // the host a launch.  8 heads of 64 over 2, T = 1, 212 positions, one launch
    // against two: a loop of calls 9.2 to 10.2 us against 10.4 to 10.6, but one call
    // waited for 22 against 21 and the GPU's time 7.6 against 6.5 (the cooperative
    // launch and the splits' meeting).  T = 13 there, four rows a warp, 14.5 against
    // 10.0 in a loop; heads of 128, 4 over 4, 265 positions, 12.3 against 10.5.
    const int warps = p.warps < 4 ? 4 : p.warps;
    p.meet = head_dim == 64 && p.n_split > 1 && p.n_split <= kB && R <= p.n_split * warps * p.row_blocks &&
             n_heads_kv * p.row_blocks <= kQ8MaxSets;
    return p;
}

// Whether the tcgen05 kernel is the faster one.  This one's time grows with the
// tiles a split takes in turn, from a short start; the other's start (TMEM,
// barriers, the tail's keys, the meeting of the splits) costs 13 us or more
// whatever the length.  Heads of 128, this kernel against the other: up to two
// tiles in turn, 32 heads over 8 at 2048 positions T = 1 14.1 and 16.7 us,
// T = 40 21.0 and 23.4; 8 over 1 at 16K T = 1 17.1 and 22.7; three, 32 over 8
// at 2.5K T = 40 25.0 and 23.5 (T = 1 15.3 and 17.0), 32 over 32 at 768 T = 1 19.6
// and 16.5, 8 over 1 at 12K T = 40 27.2 and 23.3.
bool long_enough(const SplitPlan &p) { return p.tiles_per_split > 2; }

template <int D>
cudaError_t launch_d(const AttnQ8Args &a, const TreeMasks &masks, const SplitPlan &p,
                     cudaStream_t stream)
{
    const int smem = Shape<D>::kSmem;
    cudaError_t e = cudaFuncSetAttribute(attn_q8_kernel<D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.n_split, a.n_heads_kv, p.row_blocks);
    // at least 4 warps: they also turn the codes into bf16
    cfg.blockDim = dim3((p.warps < 4 ? 4 : p.warps) * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    // cooperative where the splits wait for one another (at most one CTA per SM)
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeCooperative;
    at[1].val.cooperative = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.meet ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, attn_q8_kernel<D>, a, masks, p.tiles_per_split, p.n_split, (int)p.meet);
    if (e == cudaSuccess)
        e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    count_launches(1);
    if (p.meet || p.n_split == 1)
        return e;
    const int rows_all = a.n_tree * a.n_heads_q;
    const float *ws_o = reinterpret_cast<const float *>(
        reinterpret_cast<const char *>(a.workspace) + kHeaderBytes + kQ8SyncBytes);
    const float *ws_ml = ws_o + (size_t)p.n_split * rows_all * D;
    // warps to a row: a round of loads each
    const int per_row = p.n_split <= kB ? 1 : p.n_split <= 2 * kB ? 2 : p.n_split <= 4 * kB ? 4 : 8;
    const int rows_cta = 8 / per_row;
    return launch_pdl(attn_q8_combine_kernel<D>, dim3((rows_all + rows_cta - 1) / rows_cta), dim3(256), 0,
                      stream, ws_o, ws_ml, a.out, rows_all, p.n_split, per_row);
}

}  // namespace

size_t attn_q8_workspace_bytes(int n_heads_q, int n_heads_kv, int head_dim, int n_q8, int n_tail,
                               int n_tree, int num_sms)
{
    const SplitPlan p = make_plan(n_heads_q, n_heads_kv, head_dim, n_q8, n_tail, n_tree, num_sms);
    size_t bytes = kHeaderBytes + kQ8SyncBytes +
                   align_up((size_t)p.n_split * n_tree * n_heads_q * (head_dim + 2) * sizeof(float), 256);
    // large enough for whichever kernel the launch picks
    if (long_enough(p) &&
        attn_q8_t128_eligible(n_heads_q, n_heads_kv, head_dim, n_q8, n_tail, n_tree, num_sms)) {
        const size_t t = attn_q8_t128_workspace_bytes(n_heads_q, n_heads_kv, n_q8, n_tail, n_tree, num_sms);
        bytes = t > bytes ? t : bytes;
    }
    return bytes;
}

cudaError_t attn_q8_launch(const AttnQ8Args &a, const TreeMasks &masks, int num_sms,
                           cudaStream_t stream)
{
    const SplitPlan p = make_plan(a.n_heads_q, a.n_heads_kv, a.head_dim, a.c.n_q8, a.c.n_tail, a.n_tree, num_sms);
    // the tcgen05 kernel needs scores that grow with the products, and leaves
    // root scores for groups of up to 8 heads
    if (long_enough(p) && a.scale_log2 > 0.f && (!a.root_scores || a.n_heads_q / a.n_heads_kv <= 8) &&
        attn_q8_t128_eligible(a.n_heads_q, a.n_heads_kv, a.head_dim, a.c.n_q8, a.c.n_tail, a.n_tree,
                              num_sms))
        return attn_q8_t128_launch(a, masks, num_sms, stream);
    return a.head_dim == 128 ? launch_d<128>(a, masks, p, stream)
                             : launch_d<64>(a, masks, p, stream);
}

}  // namespace ts
