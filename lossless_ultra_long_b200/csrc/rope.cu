// rope.cu -- rotary position embedding of a step's queries and keys, with
// the append of its K/V rows to a cache (ts_rope_append), and the
// frequency tables of the scaled forms (ts_rope_inv_freq, host code).
//
// Pair j of a head is turned by the angle pos * f_j: (u, w) -> m (u cos -
// w sin, w cos + u sin).  Pairs are (j, j + rot/2) or, interleaved,
// (2j, 2j + 1); elements at or past `rot` pass through.  A tree node's
// position is pos0 + its depth, a prompt token's pos0 + its index.
//
// The angle is formed in 64 bits: at position 1e5 a binary32 product is off
// by up to 4e-3 radians.  It is reduced to a fraction of a turn there, and
// sincospi of that fraction in binary32 is off by ~2^-23, far below the one
// rounding of the result to bf16 (2^-8 relative).
//
// Bound: HBM on a prompt (every value read once and written once), launch
// latency on a step.
#include <math.h>

#include "ts_internal.cuh"

namespace ts {
namespace {

constexpr int kThreads = 256;

struct Depths {
    uint8_t depth[TS_MAX_TREE];
};

// One head's row of a token: where it comes from and where it goes.
struct RowPtr {
    const __nv_bfloat16 *src;
    __nv_bfloat16 *dst;
    bool turn;
};

__device__ __forceinline__ RowPtr row_ptr(const RopeArgs &a, int tok, int h)
{
    RowPtr r;
    if (h < a.n_heads_q) {
        r.src = a.q + tok * a.q_stride + (int64_t)h * a.head_dim;
        r.dst = a.q_out + ((int64_t)tok * a.n_heads_q + h) * a.head_dim;
        r.turn = true;
        return r;
    }
    h -= a.n_heads_q;
    r.turn = h < a.n_heads_kv;
    const int g = r.turn ? h : h - a.n_heads_kv;
    r.src = (r.turn ? a.k + tok * a.k_stride : a.v + tok * a.v_stride) + (int64_t)g * a.head_dim;
    r.dst = (r.turn ? a.k_cache : a.v_cache) +
            ((int64_t)g * a.kv_cap + a.row0 + tok) * a.head_dim;
    return r;
}

__device__ __forceinline__ void turn2(float u, float w, float c, float s, float &x, float &y)
{
    x = u * c - w * s;
    y = w * c + u * s;
}

// Eight pairs held as u[8] = a's values and w[8] = b's.
__device__ __forceinline__ void turn8(uint4 &a, uint4 &b, const float *cs, const float *sn)
{
    uint32_t *pa = reinterpret_cast<uint32_t *>(&a), *pb = reinterpret_cast<uint32_t *>(&b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 u = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(pa + i));
        const float2 w = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(pb + i));
        float x0, y0, x1, y1;
        turn2(u.x, w.x, cs[2 * i], sn[2 * i], x0, y0);
        turn2(u.y, w.y, cs[2 * i + 1], sn[2 * i + 1], x1, y1);
        *reinterpret_cast<__nv_bfloat162 *>(pa + i) = __floats2bfloat162_rn(x0, x1);
        *reinterpret_cast<__nv_bfloat162 *>(pb + i) = __floats2bfloat162_rn(y0, y1);
    }
}

// Grid (token, head group).  The token's angles are formed once per CTA;
// then each thread moves units of 16 bytes (two of them where a pair's
// halves lie apart).  VEC: interleaved pairs, or halves that start on a
// 16-byte boundary; otherwise one pair or one element per unit.
template <bool VEC>
__global__ void __launch_bounds__(kThreads)
rope_append_kernel(RopeArgs a, Depths depths, int heads_per_cta)
{
    __shared__ __align__(16) float cs[64], sn[64];
    const int tok = blockIdx.x;
    const int half = a.rot_dim / 2, D = a.head_dim;
    if (threadIdx.x < half) {
        const int64_t pos = a.pos0 + (a.tree ? depths.depth[tok] : tok);
        const double turns = (double)pos * (double)a.inv_freq[threadIdx.x] * 0.15915494309189535;
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[threadIdx.x] = c * a.mscale;
        sn[threadIdx.x] = s * a.mscale;
    }
    __syncthreads();
    const int heads = a.n_heads_q + 2 * a.n_heads_kv;
    const int h0 = blockIdx.y * heads_per_cta, h1 = min(h0 + heads_per_cta, heads);
    if (VEC) {
        // a row is D/8 chunks of 8 elements.  Half layout: chunk c < half/8
        // also takes chunk c + half/8; those partners are no unit of their own
        const int chunks = D / 8;
        const int hc = a.interleaved ? 0 : half / 8;
        for (int u = threadIdx.x; u < (h1 - h0) * chunks; u += kThreads) {
            const int c = u % chunks;
            const RowPtr r = row_ptr(a, tok, h0 + u / chunks);
            const uint4 *src = reinterpret_cast<const uint4 *>(r.src);
            uint4 *dst = reinterpret_cast<uint4 *>(r.dst);
            if (!r.turn) {
                dst[c] = src[c];
            } else if (!a.interleaved) {
                if (c < hc) {
                    uint4 x = src[c], y = src[c + hc];
                    turn8(x, y, cs + 8 * c, sn + 8 * c);
                    dst[c] = x;
                    dst[c + hc] = y;
                } else if (c >= 2 * hc) {
                    dst[c] = src[c];
                }
            } else {
                uint4 x = src[c];
                uint32_t *p = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = 4 * c + i;
                    if (j < half) {
                        const float2 v = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(p + i));
                        float y0, y1;
                        turn2(v.x, v.y, cs[j], sn[j], y0, y1);
                        *reinterpret_cast<__nv_bfloat162 *>(p + i) = __floats2bfloat162_rn(y0, y1);
                    }
                }
                dst[c] = x;
            }
        }
    } else {
        // half layout whose halves start anywhere: unit j < half is a pair,
        // the rest single elements from rot on
        const int units = D - half;
        for (int u = threadIdx.x; u < (h1 - h0) * units; u += kThreads) {
            const int j = u % units;
            const RowPtr r = row_ptr(a, tok, h0 + u / units);
            if (j < half) {
                const float x = __bfloat162float(r.src[j]), w = __bfloat162float(r.src[j + half]);
                float y0 = x, y1 = w;
                if (r.turn)
                    turn2(x, w, cs[j], sn[j], y0, y1);
                r.dst[j] = __float2bfloat16_rn(y0);
                r.dst[j + half] = __float2bfloat16_rn(y1);
            } else {
                r.dst[j + half] = r.src[j + half];
            }
        }
    }
}

}  // namespace

cudaError_t rope_append_launch(const RopeArgs &a, const int32_t *parent, int num_sms,
                               cudaStream_t stream)
{
    Depths d = {};
    if (parent)
        for (int i = 1; i < a.n_tok; ++i)
            d.depth[i] = (uint8_t)(d.depth[parent[i]] + 1);
    const int heads = a.n_heads_q + 2 * a.n_heads_kv;
    // a step has few tokens: its heads go to several CTAs
    int groups = (2 * num_sms + a.n_tok - 1) / a.n_tok;
    groups = groups > heads ? heads : groups;
    const int per = (heads + groups - 1) / groups;
    const dim3 grid(a.n_tok, (heads + per - 1) / per);
    const bool vec = a.interleaved || (a.rot_dim / 2) % 8 == 0;
    if (vec)
        rope_append_kernel<true><<<grid, kThreads, 0, stream>>>(a, d, per);
    else
        rope_append_kernel<false><<<grid, kThreads, 0, stream>>>(a, d, per);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        count_launches(1);
    return e;
}

}  // namespace ts

extern "C" int ts_rope_inv_freq(float *inv_freq, int rot_dim, double base, int kind,
                                const double *params, float *mscale)
{
    if (!inv_freq || !mscale || rot_dim < 0 || rot_dim % 2 || !(base > 1.0) || !isfinite(base) ||
        kind < TS_ROPE_PLAIN || kind > TS_ROPE_YARN || (kind != TS_ROPE_PLAIN && !params))
        return TS_ERR_INVALID_ARG;
    static const int n_params[] = {0, 1, 4, 4};
    for (int i = 0; i < n_params[kind]; ++i)
        if (!isfinite(params[i]) || !(params[i] > 0.0))
            return TS_ERR_INVALID_ARG;
    const double pi = 3.14159265358979323846;
    const int half = rot_dim / 2;
    double lo = 0.0, hi = 0.0;
    *mscale = 1.0f;
    if (kind == TS_ROPE_WAVELENGTH && !(params[2] > params[1]))
        return TS_ERR_INVALID_ARG;
    if (kind == TS_ROPE_YARN) {
        // the pair index at which a frequency makes `r` turns over the
        // original context: rot * ln(ctx / (2 pi r)) / (2 ln base)
        const double k = rot_dim / (2.0 * log(base));
        lo = floor(k * log(params[1] / (2.0 * pi * params[2])));
        hi = ceil(k * log(params[1] / (2.0 * pi * params[3])));
        lo = lo < 0.0 ? 0.0 : lo;
        hi = hi > rot_dim - 1 ? rot_dim - 1 : hi;
        if (hi - lo < 1e-3)
            hi = lo + 1e-3;
        if (params[0] > 1.0)
            *mscale = (float)(0.1 * log(params[0]) + 1.0);
    }
    for (int j = 0; j < half; ++j) {
        double f = pow(base, -2.0 * j / rot_dim);
        if (kind == TS_ROPE_LINEAR) {
            f /= params[0];
        } else if (kind == TS_ROPE_WAVELENGTH) {
            // turns over the original context: below `low` stretched by the
            // factor, above `high` kept, linear between
            double s = (params[3] * f / (2.0 * pi) - params[1]) / (params[2] - params[1]);
            s = s < 0.0 ? 0.0 : (s > 1.0 ? 1.0 : s);
            f = f * (s + (1.0 - s) / params[0]);
        } else if (kind == TS_ROPE_YARN) {
            double r = (j - lo) / (hi - lo);
            r = r < 0.0 ? 0.0 : (r > 1.0 ? 1.0 : r);
            f = f * ((1.0 - r) + r / params[0]);
        }
        inv_freq[j] = (float)f;
    }
    return TS_OK;
}
