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

// Cosines and sines (times mscale) of tokens tok0 .. tok0 + n_tok - 1 into
// shared memory, [token][rot / 2], a pair per thread and round.
__device__ __forceinline__ void form_angles(const RopeArgs &a, const Depths &depths, int tok0, int n_tok,
                                            float *cs, float *sn)
{
    const int half = a.rot_dim / 2;
    for (int i = threadIdx.x; i < n_tok * half; i += kThreads) {
        const int t = i / half;
        const int64_t pos = a.pos0 + (a.tree ? depths.depth[tok0 + t] : tok0 + t);
        const double turns = (double)pos * (double)__ldg(a.inv_freq + (i - t * half)) * 0.15915494309189535;
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[i] = c * a.mscale;
        sn[i] = s * a.mscale;
    }
    __syncthreads();
}

// Grid (run of tokens, head group): 16-byte chunks, for interleaved pairs, or
// halves that start on a chunk.  A row is D / 8 chunks; with halves apart,
// unit c < hc = rot / 16 is the chunks c and c + hc (a turned row's pairs),
// unit c >= hc the chunk c + hc.  A thread has kUnits units' loads in flight,
// the first of them while the run's angles are formed.
// HBM-bound on a prompt: on 8190 tokens of 56 heads of 128 (235 MB) a CTA per
// token took 86-95 us, each waiting for its own angles; runs of tokens 53 us.
constexpr int kUnits = 4, kMaxAngles = 512;
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads)
rope_append_kernel(RopeArgs a, Depths depths, int toks_per_cta, int heads_per_cta)
{
    __shared__ __align__(16) float cs[kMaxAngles], sn[kMaxAngles];
    constexpr int kChunks = D / 8;
    const int half = a.rot_dim / 2;
    const int hc = INTER ? 0 : half / 8, upr = kChunks - hc;   // units per row
    const int tok0 = blockIdx.x * toks_per_cta, n_tok = min(toks_per_cta, a.n_tok - tok0);
    const int h0 = blockIdx.y * heads_per_cta;
    const int n_heads = min(heads_per_cta, a.n_heads_q + 2 * a.n_heads_kv - h0);
    const int units = n_tok * n_heads * upr;
    // quotients by products: half a unit off any border is more than their rounding
    const float inv_upr = 1.f / (float)upr, inv_heads = 1.f / (float)n_heads;
    bool angles = false;
    for (int u0 = threadIdx.x; u0 < units || !angles; u0 += kUnits * kThreads) {
        uint4 x[kUnits], y[kUnits];
        __nv_bfloat16 *dst[kUnits];
        int c[kUnits], at[kUnits];   // at: the token's angles, or -1
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int u = u0 + i * kThreads;
            if (u < units) {
                const int row = (int)(((float)u + 0.5f) * inv_upr);
                const int t = (int)(((float)row + 0.5f) * inv_heads);
                c[i] = u - row * upr;
                const RowPtr r = row_ptr(a, tok0 + t, h0 + row - t * n_heads);
                const uint4 *src = reinterpret_cast<const uint4 *>(r.src);
                dst[i] = r.dst;
                at[i] = r.turn ? t * half : -1;
                if (c[i] < hc)
                    x[i] = __ldcs(src + c[i]);
                y[i] = __ldcs(src + c[i] + hc);
            }
        }
        if (!angles)
            form_angles(a, depths, tok0, n_tok, cs, sn);
        angles = true;
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            if (u0 + i * kThreads >= units)
                continue;
            uint4 *out = reinterpret_cast<uint4 *>(dst[i]);
            if (INTER) {
                if (at[i] >= 0) {
                    uint32_t *p = reinterpret_cast<uint32_t *>(&y[i]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int j = 4 * c[i] + k;
                        if (j < half) {
                            const float2 v = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(p + k));
                            float y0, y1;
                            turn2(v.x, v.y, cs[at[i] + j], sn[at[i] + j], y0, y1);
                            *reinterpret_cast<__nv_bfloat162 *>(p + k) = __floats2bfloat162_rn(y0, y1);
                        }
                    }
                }
            } else if (c[i] < hc) {
                if (at[i] >= 0)
                    turn8(x[i], y[i], cs + at[i] + 8 * c[i], sn + at[i] + 8 * c[i]);
                out[c[i]] = x[i];
            }
            out[c[i] + hc] = y[i];
        }
    }
}

// Halves that start anywhere: unit j < half is a pair, the rest single
// elements from rot on.
__global__ void __launch_bounds__(kThreads)
rope_append_any_kernel(RopeArgs a, Depths depths, int heads_per_cta)
{
    __shared__ float cs[64], sn[64];
    const int tok = blockIdx.x, half = a.rot_dim / 2;
    form_angles(a, depths, tok, 1, cs, sn);
    const int heads = a.n_heads_q + 2 * a.n_heads_kv;
    const int h0 = blockIdx.y * heads_per_cta, h1 = min(h0 + heads_per_cta, heads);
    const int units = a.head_dim - half;
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
    if (!a.interleaved && (a.rot_dim / 2) % 8 != 0) {
        rope_append_any_kernel<<<dim3(a.n_tok, (heads + per - 1) / per), kThreads, 0, stream>>>(a, d, per);
    } else {
        // runs of tokens as long as their angles fit and every SM keeps four CTAs
        const int half = a.rot_dim / 2;
        int run = half > 0 ? kMaxAngles / half : 8;
        run = run > 8 ? 8 : run;
        const int fit = a.n_tok / (4 * num_sms);
        run = fit < run ? (fit < 1 ? 1 : fit) : run;
        const dim3 grid((a.n_tok + run - 1) / run, (heads + per - 1) / per);
        if (a.head_dim == 128 && a.interleaved)
            rope_append_kernel<128, true><<<grid, kThreads, 0, stream>>>(a, d, run, per);
        else if (a.head_dim == 128)
            rope_append_kernel<128, false><<<grid, kThreads, 0, stream>>>(a, d, run, per);
        else if (a.interleaved)
            rope_append_kernel<64, true><<<grid, kThreads, 0, stream>>>(a, d, run, per);
        else
            rope_append_kernel<64, false><<<grid, kThreads, 0, stream>>>(a, d, run, per);
    }
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
