// attn_q8_t128.cu -- tree-verify attention over the 8-bit KV cache on the
// 5th-generation tensor cores (head_dim 128): split-KV, 128-position tiles.
//
// Products, for the R = G*T query rows of a KV head and one tile:
//   S_b  = Q_b K^T     kind::f8f6f4 on the codes as they lie in HBM.  A bf16
//                      query is the sum of an e4m3 and an e5m2 number: with
//                      its row scaled to at most 448, hi = e4m3(q) keeps 4 of
//                      the 8 significant bits and lo = e5m2(q - hi) holds
//                      what is left (an integer of 0..8 units of the last
//                      bit, which 3 bits represent), down to 2^-16 of the
//                      scaled row.  So S = hi K^T + lo K^T costs what one
//                      bf16 product costs, and K is never converted.
//   O^T += V^T P^T     kind::f16 on bf16: V's codes are bf16 numbers;
//                      the converter warps write them out once per tile.
// The scales (a power of two per 64 rows) never touch the products' inputs:
// K's multiplies the score inside the exponent's FMA, V's is added to the
// exponent, so the weight leaves as p * s_v with its one rounding to bf16,
// and each block's sum is multiplied back by 1 / s_v.
//
// A tail tile (bf16 rows: newest context, tree) goes through the same
// products: the converter warps scale its keys, each row by a power of two of its
// own (no row takes another's bits, whatever its size), split them like the
// queries into an e4m3 and an e5m2 tile (two K slots, four products), and copy V;
// the scores take the keys' scales where the masks are evaluated.  Rows with an
// infinity or a NaN are zeroed there and noted; a query row that sees one gets a NaN
// sum.
//
// Softmax layout, reference maximum (fixed at a row's first tile), partials, and
// the combine by the splits themselves follow the bf16 kernel in attn_t128.cu;
// a split whose row sum outgrows the reference by 2^63 is recomputed exactly.
// The result is rounded to bf16, as coarse as the weights' own rounding, so rows
// that rest on few positions need no second look.
//
// Which split takes a tile depends on its index alone (HandOut), from the end
// of the cache backwards: a row's reference and the order of its sums are the
// same in every call, and so is the result, bit for bit.  (Tiles handed out at
// run time move the result by the order of the sums and the rounding of a weight
// to bf16, up to 2^-8 of it from call to call.)
//
// CTA = (split, KV head, node group), 20 warps, one CTA per SM:
//   warp 0      root scores out of S        warp 1  QK issuer, TMEM
//   warp 2      PV issuer                   warp 3  takes tiles, TMA producer
//   warps 4-15  softmax, as many as the rows need; the others and
//   warps 16-19 V's codes to bf16
// P^T is double-buffered, and with one query block (R <= 128) S too, so a
// tile's exponentials overlap the previous tile's PV and the next one's QK.
// With at most 64 query rows one warpgroup is enough for a tile, but its chain
// of waits and loads is longer than the tile's stream from HBM: two softmax
// warpgroups then take tiles in turn, each with its own reference,
// O^T and P^T, and their partials are merged before they leave.
// TMEM: O^T in [0, 192), Q_0 (hi, lo) in [192, 256), S in [256, 512).
//
// What bounds it, at 102400 positions (8 KV heads, 210 MB: 32 us of HBM time):
// up to 16 query rows a head 51 us, the conversion of V the largest part (8 us
// without it) and shared memory, of which a tile moves some 150 KB; 52 rows 57
// us; 160 rows 95 us, the exponentials and the order of the tiles' steps (two
// query blocks leave room for one bf16 V tile).  32 KV heads of 4 rows (839 MB)
// 186 us, on the 128 SMs that 32 heads divide into.  Under calls without a pause
// the clock falls to 1.65 GHz at the power limit (59, 111 and 223 us).
//
// Every wait is bounded (about a second): on expiry the kernel records
// TS_ERR_TIMEOUT in the workspace status word, all roles leave their loops,
// and TMEM is freed before the CTA exits.
#include <math.h>

#include "attn_common.cuh"
#include "attn_q8.cuh"
#include "sm100.cuh"

namespace ts {

// from attn_dispatch.cu
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace {

using namespace sm100;

constexpr int kD = 128;
constexpr int kTileN = 128;                  // KV positions per tile
constexpr int kBlockM = 128;                 // query rows per QK block (TMEM lanes)
constexpr int kRawBytes = kTileN * kD;       // codes of K (or V) of a tile: 16 KB
constexpr int kBoxBytes = kTileN * 64 * 2;   // one 64-column half of a bf16 V tile
constexpr int kVbBytes = 2 * kBoxBytes;
constexpr int kThreads = 640;                // 20 warps
constexpr int kMaxStages = 5;
constexpr int kMaxRows = 192;
constexpr int kQCol = 192;                   // Q of block 0: hi 32 columns, lo 32 columns
constexpr int kSCol = 256;                   // S slots: 128 columns each
constexpr int kTmemCols = 512;
constexpr int kQ1Bytes = 2 * kBlockM * kD;   // Q of block 1 in shared memory: hi, lo
constexpr float kMaxRowSum = 9.223372036854775808e18f;   // 2^63
// 8-bit tiles that the others stream while a split makes its tail tile ready.
// 102400 positions of 8 heads, 3, 4, 5, 6 of them: one query row a head 54.0, 52.8,
// 52.1, 51.0 us, 40 nodes 97.1, 95.5, 95.8, 95.1
constexpr int kTailCost = 6;
constexpr int kTailWarps = 4;                // warps 16-19, which also turn the tail tiles
constexpr size_t kSmemLimit = 232448;        // dynamic shared memory per CTA
constexpr int kBarQuery = 1;                 // named barrier: query rows in place
constexpr int kBarOut = 2;                   // named barrier: O^T staged, or merged, in shared memory
constexpr int kTileRing = 16;                // entries of the tile rings (> any role's lead)
static_assert(kTileRing == 1 << 4, "indexed by shifts");
constexpr int kBarRows = 5;                  // named barrier: row_scale is written (for warp 0)
constexpr int kBarQLoads = 3;                // named barrier: the query rows are read
constexpr int kBarScales = 4;                // named barrier: the scale bytes are in shared memory
constexpr int kQLoadThreads = 32 * 9;        // warps 4-11 arrive, K's producer waits
constexpr int kMaxGz = kQ8MaxSets;           // (KV head, node group) pairs: counters in the workspace

constexpr int kTailMark = 1 << 20, kEndMark = -(1 << 30);

struct Bars {
    uint64_t full_k[kMaxStages];
    uint64_t empty_k[kMaxStages];
    uint64_t full_v[kMaxStages];    // codes of V landed (or: a tail tile)
    uint64_t empty_v[kMaxStages];
    uint64_t s_full[2];             // QK landed: by block, or (one block) by tile in turn
    uint64_t s_free[2];             // its readers hold S in registers
    uint64_t vb_full[2];            // V in bf16
    uint64_t sm_done[2];            // per P^T slot: P^T is written
    uint64_t pv_done[2];            // per P^T slot: PV is complete
    uint64_t o_final;
    uint64_t drain[2];
    uint64_t conv;                  // the converter warps meet (tail tiles)
    uint64_t info[kTileRing];       // tile_of, scale_of of that tile are written
    uint64_t tail_slots[kTileRing]; // a tail tile's K slots are free, entry_of is written
    // per tile, at [t & (kTileRing - 1)]: its index (-1 after the last); a tail
    // tile's first K ring entry, at [t & 3]
    volatile int32_t tile_of[kTileRing];
    volatile int32_t entry_of[4];
    uint32_t bad[4][4];             // tail tile t % 4: rows with a value that is no number
    uint32_t bad_k[4][4];
    uint32_t tmem_base;
    uint32_t abort;
    int32_t overflow;
};

struct Aux {
    Bars bar;
    // per tile and half, posted with tile_of: K's scale (1 on a tail tile), V's
    // as an exponent, V's inverse, and (as an int) how many of the half's positions
    // are context, kTailMark added on a tail tile, or kEndMark.  A block that is
    // NaN, in K or V, has a NaN exponent and inverse: its weights and sums are NaN.
    float4 scale_of[kTileRing][2];
    unsigned long long anc[TS_MAX_TREE];
    float2 ml[2][64];               // (m, l) of each group's rows, to be merged
    float row_scale[kMaxRows];      // softmax scale * log2 e * the query row's scale
    uint8_t key_exp[4][kTileN];     // tail tile t % 4: the keys' scales 2^(byte - 127)
};
constexpr size_t kAuxBytes = (sizeof(Aux) + 15) / 16 * 16;

struct Layout {
    int r_pad, stages_k, stages_v, stages_vb;
    size_t q1_off, p_off, vb_off, k_off, v_off, sc_off, aux_off, smem_bytes;
};

__host__ __device__ inline int q8_row_of(int n, int R)
{
    return R > kBlockM ? (n < kBlockM ? (R - kBlockM) + n : n - kBlockM) : n;
}

__host__ __device__ inline Layout q8_layout(int rows, int n_blk)
{
    Layout L;
    L.r_pad = (rows + 15) / 16 * 16;
    L.q1_off = 0;
    L.p_off = rows > kBlockM ? kQ1Bytes : 0;
    // the P^T tiles, then 1 KB that rows past the query rows are written to
    L.vb_off = L.p_off + (size_t)L.r_pad * 512 + 1024;
    L.stages_vb = rows > kBlockM ? 1 : 2;
    L.k_off = L.vb_off + (size_t)L.stages_vb * kVbBytes;
    // the scale bytes of every block of the head, K's then V's
    const size_t sc_bytes = ((size_t)2 * n_blk + 15) / 16 * 16;
    const size_t fixed = 1024 + L.k_off + sc_bytes + kAuxBytes;
    int stages = fixed > kSmemLimit ? 0 : (int)((kSmemLimit - fixed) / kRawBytes);
    stages = stages > 2 * kMaxStages ? 2 * kMaxStages : stages;
    L.stages_v = stages / 2;
    L.stages_k = stages - L.stages_v;   // at least 2: a tail tile takes two
    L.v_off = L.k_off + (size_t)L.stages_k * kRawBytes;
    L.aux_off = L.v_off + (size_t)L.stages_v * kRawBytes;
    L.sc_off = L.aux_off + kAuxBytes;
    L.smem_bytes = 1024 + L.sc_off + sc_bytes;
    return L;
}

// Instruction descriptor of kind::f8f6f4, fp32 accumulation, K-major
// operands; a5 / b5: that operand is e5m2 instead of e4m3.
constexpr uint32_t idesc_f8(int m, int n, int a5, int b5)
{
    return (1u << 4) | ((uint32_t)a5 << 7) | ((uint32_t)b5 << 10) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}

// The products of one tile, eight instructions each.  Shared-memory
// descriptors are given by their low words; the high words are the same for
// every operand here (swizzle, version, 1024-byte groups).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

// S (+)= (Q_hi + Q_lo) K^T, Q's codes in TMEM (hi, lo: 32 columns each).
__device__ __forceinline__ void mma_qk_ts(uint32_t d, uint32_t q, uint32_t k, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n .reg .pred p, o;\n .reg .b64 x, y;\n .reg .b32 s, t, u;\n setp.eq.u32 o, 0, 0;\n"
        " setp.ne.b32 p, %4, 0;\n or.b32 u, %3, 128;\n"
        " add.u32 s, %1, 0;\n add.u32 t, %2, 0;\n mov.b64 y, {t, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [s], y, %3, p;\n"
        " add.u32 s, %1, 8;\n add.u32 t, %2, 2;\n mov.b64 y, {t, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [s], y, %3, o;\n"
        " add.u32 s, %1, 16;\n add.u32 t, %2, 4;\n mov.b64 y, {t, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [s], y, %3, o;\n"
        " add.u32 s, %1, 24;\n add.u32 t, %2, 6;\n mov.b64 y, {t, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [s], y, %3, o;\n"
        " add.u32 s, %1, 32;\n add.u32 t, %2, 0;\n mov.b64 y, {t, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [s], y, u, o;\n"
        " add.u32 s, %1, 40;\n add.u32 t, %2, 2;\n mov.b64 y, {t, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [s], y, u, o;\n"
        " add.u32 s, %1, 48;\n add.u32 t, %2, 4;\n mov.b64 y, {t, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [s], y, u, o;\n"
        " add.u32 s, %1, 56;\n add.u32 t, %2, 6;\n mov.b64 y, {t, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [s], y, u, o;\n"
        "}\n" ::"r"(d), "r"(q), "r"(k), "r"(idesc), "r"(acc), "r"(kDescHi)
        : "memory");
}

// The same with Q's codes in shared memory (hi, then lo: 16 KB each).
__device__ __forceinline__ void mma_qk_ss(uint32_t d, uint32_t q, uint32_t k, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n .reg .pred p, o;\n .reg .b64 x, y;\n .reg .b32 s, t, u;\n setp.eq.u32 o, 0, 0;\n"
        " setp.ne.b32 p, %4, 0;\n or.b32 u, %3, 128;\n"
        " add.u32 s, %1, 0;\n add.u32 t, %2, 0;\n mov.b64 y, {t, %5};\n"
        " mov.b64 x, {s, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n"
        " add.u32 s, %1, 2;\n add.u32 t, %2, 2;\n mov.b64 y, {t, %5};\n"
        " mov.b64 x, {s, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, o;\n"
        " add.u32 s, %1, 4;\n add.u32 t, %2, 4;\n mov.b64 y, {t, %5};\n"
        " mov.b64 x, {s, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, o;\n"
        " add.u32 s, %1, 6;\n add.u32 t, %2, 6;\n mov.b64 y, {t, %5};\n"
        " mov.b64 x, {s, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, o;\n"
        " add.u32 s, %1, 1024;\n add.u32 t, %2, 0;\n mov.b64 y, {t, %5};\n"
        " mov.b64 x, {s, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, u, o;\n"
        " add.u32 s, %1, 1026;\n add.u32 t, %2, 2;\n mov.b64 y, {t, %5};\n"
        " mov.b64 x, {s, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, u, o;\n"
        " add.u32 s, %1, 1028;\n add.u32 t, %2, 4;\n mov.b64 y, {t, %5};\n"
        " mov.b64 x, {s, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, u, o;\n"
        " add.u32 s, %1, 1030;\n add.u32 t, %2, 6;\n mov.b64 y, {t, %5};\n"
        " mov.b64 x, {s, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, u, o;\n"
        "}\n" ::"r"(d), "r"(q), "r"(k), "r"(idesc), "r"(acc), "r"(kDescHi)
        : "memory");
}

// O^T (+)= V^T P^T; p0, p1: P^T of the tile's first and second 64 positions.
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t v, uint32_t p0, uint32_t p1, uint32_t idesc,
                                       uint32_t acc)
{
    asm volatile(
        "{\n .reg .pred p, o;\n .reg .b64 x, y;\n .reg .b32 s, t;\n setp.eq.u32 o, 0, 0;\n"
        " setp.ne.b32 p, %5, 0;\n"
        " add.u32 s, %1, 0;\n add.u32 t, %2, 0;\n mov.b64 x, {s, %6};\n mov.b64 y, {t, %6};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n"
        " add.u32 s, %1, 128;\n add.u32 t, %2, 2;\n mov.b64 x, {s, %6};\n mov.b64 y, {t, %6};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, o;\n"
        " add.u32 s, %1, 256;\n add.u32 t, %2, 4;\n mov.b64 x, {s, %6};\n mov.b64 y, {t, %6};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, o;\n"
        " add.u32 s, %1, 384;\n add.u32 t, %2, 6;\n mov.b64 x, {s, %6};\n mov.b64 y, {t, %6};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, o;\n"
        " add.u32 s, %1, 512;\n add.u32 t, %3, 0;\n mov.b64 x, {s, %6};\n mov.b64 y, {t, %6};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, o;\n"
        " add.u32 s, %1, 640;\n add.u32 t, %3, 2;\n mov.b64 x, {s, %6};\n mov.b64 y, {t, %6};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, o;\n"
        " add.u32 s, %1, 768;\n add.u32 t, %3, 4;\n mov.b64 x, {s, %6};\n mov.b64 y, {t, %6};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, o;\n"
        " add.u32 s, %1, 896;\n add.u32 t, %3, 6;\n mov.b64 x, {s, %6};\n mov.b64 y, {t, %6};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, o;\n"
        "}\n" ::"r"(d), "r"(v), "r"(p0), "r"(p1), "r"(idesc), "r"(acc), "r"(kDescHi)
        : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// 16 TMEM lanes x 64 columns, the layout of tmem_ld16x256_x16; waits.
__device__ __forceinline__ void tmem_ld16x256_x8(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// 16 TMEM lanes x 32 columns, the same layout; the registers hold the values
// after tmem_ld_wait16.
__device__ __forceinline__ void tmem_ld16x256_x4(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                   "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// 8 consecutive 32-bit TMEM columns of this thread's lane; waits.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
}

// 16 consecutive 32-bit TMEM columns of this thread's lane; not waited.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

// A place in a ring of n slots and its phase, advanced by counting: the
// quotients t / n and t % n by a run-time n, several per tile and warp, cost
// more instructions than the softmax.
struct Ring {
    int n, i;
    uint32_t ph;
    __device__ __forceinline__ explicit Ring(int slots) : n(slots), i(0), ph(0) {}
    __device__ __forceinline__ void next()
    {
        if (++i == n) {
            i = 0;
            ph ^= 1u;
        }
    }
};

// sm100's bounded waits with a uniform fast path: one try, one vote, no
// divergent branch (a satisfied wait is taken several times per tile).
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile uint32_t *abort,
                                       WorkspaceHeader *ws)
{
    return wait_bounded(bar, parity, abort, ws);
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t *abort,
                                          WorkspaceHeader *ws)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
        return true;
    return __all_sync(0xffffffffu, wait_slow(bar, parity, abort, ws));
}
__device__ __forceinline__ bool lane_wait(uint32_t bar, uint32_t parity, volatile uint32_t *abort,
                                          WorkspaceHeader *ws)
{
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort, ws);
}

// Four values (times f) as e4m3 codes, and what that leaves as e5m2 codes.
__device__ __forceinline__ void split_8(float a, float b, float c, float d, float f, uint32_t &hi,
                                        uint32_t &lo)
{
    const float2 x = make_float2(a * f, b * f), y = make_float2(c * f, d * f);
    const uint32_t h0 = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
    const uint32_t h1 = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
    const float2 bx = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h0, __NV_E4M3)));
    const float2 by = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h1, __NV_E4M3)));
    const uint32_t l0 = __nv_cvt_float2_to_fp8x2(make_float2(x.x - bx.x, x.y - bx.y), __NV_SATFINITE, __NV_E5M2);
    const uint32_t l1 = __nv_cvt_float2_to_fp8x2(make_float2(y.x - by.x, y.y - by.y), __NV_SATFINITE, __NV_E5M2);
    hi = h0 | (h1 << 16);
    lo = l0 | (l1 << 16);
}

// Eight bf16 values (16 bytes) split: two words of hi, two of lo.
__device__ __forceinline__ void split_16b(const uint4 &u, float f, uint2 &hi, uint2 &lo)
{
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
    const float2 c = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.z));
    const float2 d = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.w));
    split_8(a.x, a.y, b.x, b.y, f, hi.x, lo.x);
    split_8(c.x, c.y, d.x, d.y, f, hi.y, lo.y);
}

// Largest magnitude of a bf16 pair-wise maximum word, as bits.
__device__ __forceinline__ uint32_t top_of(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }
__device__ __forceinline__ uint32_t top_word(const uint4 &u)
{
    return __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu),
                    __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
}

// Exponent e of the scale 2^e that brings a largest magnitude (bf16 bits,
// finite) to at most 448; 0 for an all-zero row.
__device__ __forceinline__ int split_exp(uint32_t top)
{
    const int e = (int)(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0);
    return top == 0 ? 0 : max(e, -126);
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Four codes -> two bf16 pairs (low codes first).  The seven low bits of a
// code, shifted to bf16's exponent and mantissa, are its magnitude times
// 2^-120 (subnormals included); NaN codes read as 480.  With a code in the
// low byte of each half word, code * 16 + sign * 0x7800 puts the magnitude at
// bit 4 and the sign at bit 15: two multiply-adds a pair, which leave the
// integer pipe, the busiest one, to the softmax.
__device__ __forceinline__ uint32_t code_pair(uint32_t two)
{
    const uint32_t a = two * 16u + (two & 0x00800080u) * 240u;
    const uint32_t f = 0x7B807B80u;   // 2^120
    const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&f));
    return *reinterpret_cast<const uint32_t *>(&x);
}
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w)
{
    return make_uint2(code_pair(__byte_perm(w, 0u, 0x4140)), code_pair(__byte_perm(w, 0u, 0x4342)));
}

// A half tile's 64 positions that a row sees: the first d, then the bits of
// anc (its root path).
__device__ __forceinline__ unsigned long long row_vis(unsigned long long anc, int d)
{
    if (d >= 64)
        return ~0ull;
    return d > 0 ? ((1ull << d) - 1ull) | (anc << d) : (d > -64 ? anc >> -d : 0ull);
}

// s0 += the low bf16 value of w, s1 += the high one.
__device__ __forceinline__ void add_pair(float &s0, float &s1, uint32_t w)
{
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %1, h, %1;}"
        : "+f"(s0), "+f"(s1) : "r"(w));
}

// Weights 2^(x * c + n) of the 2 J scores a thread holds of row E / 2 (E = 0:
// row A, E = 2: row B) of 8 J positions, packed to bf16 pairs; adds the rounded
// weights to sum0 and sum1, so that a rounding moves the result only by how far its
// position's value lies from the result.
template <int E, int J>
__device__ __forceinline__ void exp_row(const uint32_t (&r)[4 * J], float c, float n, uint32_t (&p)[J],
                                        float &sum0, float &sum1)
{
    const uint64_t c2 = pack2(c, c), n2 = pack2(n, n);
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint64_t y = fma2(pack2(__uint_as_float(r[4 * j + E]), __uint_as_float(r[4 * j + E + 1])),
                                c2, n2);
        float y0, y1;
        unpack2(y, y0, y1);
        const float x0 = ex2(y0), x1 = ex2(y1);
        const __nv_bfloat162 hv = __floats2bfloat162_rn(x0, x1);
        p[j] = *reinterpret_cast<const uint32_t *>(&hv);
        add_pair(sum0, sum1, p[j]);
    }
}

// Maximum of the scores that a thread holds of row A (E = 0) or B (E = 2).
template <int E, int J>
__device__ __forceinline__ float part_max(const uint32_t (&r)[4 * J])
{
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < J; ++j)
        m = max3f(m, __uint_as_float(r[4 * j + E]), __uint_as_float(r[4 * j + E + 1]));
    return m;
}

// The kernel's workspace, after the header and the counters.
struct Q8Sync {
    int32_t *sync;    // [Hkv * groups][4]: unused, arrivals, finished combines, unused;
                      // zero when a call starts, and again when it ends
    float *part;      // acc fp32 [n_split][T*Hq][128], then (m, l) fp32 [n_split][T*Hq][2]
    int32_t *flags;   // [n_split][Hkv * groups]: some row's sum outgrew its reference
};

// Which split streams which tile of a head, by counting alone.  The nt tail tiles
// come first, one per split and round; the `busy` splits of the last such round are
// kTailCost 8-bit tiles behind the others (the tail's keys are split and its masks
// evaluated), so the others take so many rounds ahead of them.  The rest goes round
// all splits, what is left of the last round to the last ones.  Tiles are taken from
// the end of the cache backwards.  Every split has a tile as long as there are no
// more splits than tiles.
struct HandOut {
    int n_split, nq, n_tiles, tail_rounds, busy, ahead, full, left;
    __device__ __forceinline__ HandOut(int n_split_, int nq_, int n_tiles_) : n_split(n_split_), nq(nq_), n_tiles(n_tiles_)
    {
        const int nt = n_tiles - nq;
        tail_rounds = (nt + n_split - 1) / n_split;
        busy = nt - (tail_rounds - 1) * n_split;
        ahead = min(nq, kTailCost * (n_split - busy));
        full = (nq - ahead) / n_split;
        left = nq - ahead - full * n_split;
    }
    // the r-th tile of a split, negative from its end on
    __device__ __forceinline__ int tile(int split, int r) const
    {
        const bool late = split < busy;
        int i = r - tail_rounds + (late ? 0 : 1);
        if (i < 0)
            return n_tiles - 1 - (r * n_split + split);
        if (!late) {
            const int k = i * (n_split - busy) + split - busy;
            if (i < kTailCost)
                return k < ahead ? nq - 1 - k : -1;
            i -= kTailCost;
        }
        const int s = i < full ? split : split - (n_split - left);
        return i > full || s < 0 ? -1 : nq - 1 - (ahead + i * n_split + s);
    }
    // the split that has tile t
    __device__ __forceinline__ int split_of(int t) const
    {
        if (t >= nq)
            return (n_tiles - 1 - t) % n_split;
        int k = nq - 1 - t;
        if (k < ahead)
            return busy + k % (n_split - busy);
        k -= ahead;
        return k < full * n_split ? k % n_split : k - full * n_split + n_split - left;
    }
};

// Adds one tile to half a row's running exact partial (m, l, acc): fp32
// online softmax on CUDA cores, one warp; a lane holds dims 4 lane .. + 3 of
// the products with K, and dims 64 half + 2 lane, + 1 of V.
__device__ __noinline__ void tile_exact(const AttnQ8Args &a, unsigned long long anc, int row, int half, int g,
                                        int tile, int nq, float &m, float &l, float (&acc)[2])
{
    const int lane = threadIdx.x & 31, dv = 64 * half + 2 * lane;
    const Q8Cache &kc = a.c;
    const uint2 qb = *reinterpret_cast<const uint2 *>(a.q + (size_t)row * kD + 4 * lane);
    const float2 q0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&qb.x));
    const float2 q1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&qb.y));
    const bool q8 = tile < nq;
    const int r0 = q8 ? tile * kTileN : (tile - nq) * kTileN;
    const int n = min(kTileN, (q8 ? kc.n_q8 : kc.n_tail + a.n_tree) - r0);
    auto two = [](uint32_t codes) {
        return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xFFFFu), __NV_E4M3)));
    };
    for (int i = 0; i < n; ++i) {
        float2 k0, k1, v;
        float sk = 1.f;
        if (q8) {
            const int64_t at = (int64_t)g * kc.q8_cap + r0 + i;
            const int64_t blk = (int64_t)g * (kc.q8_cap / kQ8Block) + (r0 + i) / kQ8Block;
            const float sv = q8_factor(kc.v_scale[blk]);
            sk = q8_factor(kc.k_scale[blk]);
            const uint32_t kw = *reinterpret_cast<const uint32_t *>(kc.k8 + at * kD + 4 * lane);
            k0 = two(kw);
            k1 = two(kw >> 16);
            v = two(*reinterpret_cast<const uint16_t *>(kc.v8 + at * kD + dv));
            v.x *= sv;
            v.y *= sv;
        } else {
            const int tp = r0 + i - kc.n_tail;
            if (tp >= 0 && !((anc >> tp) & 1ull))
                continue;
            const int64_t at = (int64_t)g * kc.tail_cap + r0 + i;
            const uint2 kb = *reinterpret_cast<const uint2 *>(kc.k_tail + at * kD + 4 * lane);
            const uint2 vb = *reinterpret_cast<const uint2 *>(kc.v_tail + at * kD + 4 * lane);
            // a key or a value that is no number, anywhere in its row
            if (__any_sync(0xffffffffu, top_of(top_word(make_uint4(kb.x, kb.y, vb.x, vb.y))) >= 0x7F80u)) {
                l = __uint_as_float(0x7FC00000u);
                continue;
            }
            k0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&kb.x));
            k1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&kb.y));
            v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(kc.v_tail + at * kD + dv));
        }
        float s = q0.x * k0.x + q0.y * k0.y + q1.x * k1.x + q1.y * k1.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= sk * a.scale_log2;
        if (s > m) {
            const float f = m == -INFINITY ? 0.f : exp2f(m - s);
            l *= f;
            acc[0] *= f;
            acc[1] *= f;
            m = s;
        }
        const float p = exp2f(s - m);
        l += p;
        acc[0] += p * v.x;
        acc[1] += p * v.y;
    }
}

// Half an output row (64 dims from 64 `half` on), by one warp: out = sum
// 2^(m - M) acc / sum 2^(m - M) l over the splits, a flagged split recomputed
// exactly.  (Half a row, so that every split's values are in flight at once:
// the time here is round trips.)
__device__ __forceinline__ void combine_row(const AttnQ8Args &a, const TreeMasks &masks, int row, int half,
                                            int g, int gz, int n_gz, int n_split, int nq,
                                            int n_tiles_all, const Q8Sync &sy)
{
    const int rows_all = a.n_tree * a.n_heads_q;
    const int lane = threadIdx.x & 31;
    const float *ws_o = sy.part;
    const float2 *ws_ml = reinterpret_cast<const float2 *>(ws_o + (size_t)n_split * rows_all * kD);
    auto ml_of = [&](int s) { return __ldcg(ws_ml + (size_t)s * rows_all + row); };
    auto acc_of = [&](int s) {
        return __ldcg(reinterpret_cast<const float2 *>(ws_o + ((size_t)s * rows_all + row) * kD) + 32 * half + lane);
    };
    constexpr int kB = 18;
    float2 x[kB];
    float2 mine = lane < n_split ? ml_of(lane) : make_float2(-INFINITY, 0.f);
    bool any = lane < n_split && __ldcg(sy.flags + (size_t)lane * n_gz + gz) != 0;
#pragma unroll
    for (int u = 0; u < kB; ++u)
        x[u] = u < n_split ? acc_of(u) : make_float2(0.f, 0.f);
    float M = mine.x;
    for (int s = 32 + lane; s < n_split; s += 32) {
        any |= __ldcg(sy.flags + (size_t)s * n_gz + gz) != 0;
        M = fmaxf(M, ml_of(s).x);
    }
    any = __any_sync(0xffffffffu, any);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float acc[2] = {0.f, 0.f};
    float L = 0.f;
    if (!any) {
        // lane s holds split s's weight.  A split that saw nothing (m = -inf)
        // has l = 0 and acc = 0, or l = NaN; a NaN reference keeps its NaN
        for (int s0 = 0; s0 < n_split; s0 += 32) {
            const float2 ml = s0 == 0 ? mine
                              : s0 + lane < n_split ? ml_of(s0 + lane) : make_float2(-INFINITY, 0.f);
            const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
            L += w * ml.y;
            for (int u0 = 0; u0 < 32 && s0 + u0 < n_split; u0 += kB) {
                if (s0 + u0 > 0) {
#pragma unroll
                    for (int u = 0; u < kB; ++u)
                        x[u] = u0 + u < 32 && s0 + u0 + u < n_split ? acc_of(s0 + u0 + u) : make_float2(0.f, 0.f);
                }
#pragma unroll
                for (int u = 0; u < kB; ++u) {
                    // (past the last: a zero, times some weight that is not used)
                    const float wu = __shfl_sync(0xffffffffu, w, (u0 + u) & 31);
                    acc[0] += wu * x[u].x;
                    acc[1] += wu * x[u].y;
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            L += __shfl_xor_sync(0xffffffffu, L, o);
    } else {
        const HandOut hand(n_split, nq, n_tiles_all);
        float Mr = -INFINITY;
        for (int s = 0; s < n_split; ++s) {
            float ms = -INFINITY, ls = 0.f, as[2] = {0.f, 0.f};
            if (__ldcg(sy.flags + (size_t)s * n_gz + gz) != 0) {
                for (int t0 = 0; t0 < n_tiles_all; t0 += 32) {
                    const int t = t0 + lane;
                    uint32_t bits = __ballot_sync(0xffffffffu, t < n_tiles_all && hand.split_of(t) == s);
                    while (bits) {
                        const int tt = t0 + __ffs(bits) - 1;
                        bits &= bits - 1;
                        tile_exact(a, masks.anc[row / a.n_heads_q], row, half, g, tt, nq, ms, ls, as);
                    }
                }
            } else {
                const float2 ml = ml_of(s);
                const float2 y = acc_of(s);
                ms = ml.x;
                ls = ml.y;
                as[0] = y.x;
                as[1] = y.y;
            }
            if (ms == -INFINITY) {
                L += ls;   // nothing seen: 0, or NaN
                continue;
            }
            const float Mn = fmaxf(Mr, ms);
            const float fa = Mr == -INFINITY ? 1.f : exp2f(Mr - Mn);   // L may hold a NaN
            const float fb = exp2f(ms - Mn);
            L = L * fa + ls * fb;
            acc[0] = acc[0] * fa + as[0] * fb;
            acc[1] = acc[1] * fa + as[1] * fb;
            Mr = Mn;
        }
    }
    const float inv = 1.f / L;
    *reinterpret_cast<__nv_bfloat162 *>(a.out + (size_t)row * kD + 64 * half + 2 * lane) =
        __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv);
}

// The keys of tail tile t into its two K slots, by the converters' 128 threads,
// a row each: scaled to at most 448 by a power of two (noted in key_exp), split
// into e4m3 and e5m2 codes; notes the rows with an infinity or a NaN, and zeroes
// the keys among them (a key whose value is no number still has its score).  False
// when a wait ran out.
__device__ __noinline__ bool tail_keys(const AttnQ8Args &a, Aux *aux, unsigned char *sK, int SK, int g,
                                       int nq, int t, int &met, volatile uint32_t *abort,
                                       WorkspaceHeader *hdr)
{
    Bars *bar = &aux->bar;
    const Q8Cache &kc = a.c;
    const int tid = threadIdx.x & 127, lane = threadIdx.x & 31, w = tid >> 5;
    const int row = (bar->tile_of[t & (kTileRing - 1)] - nq) * kTileN + tid;
    const bool have = row < kc.n_tail + a.n_tree;
    const int64_t at = ((int64_t)g * kc.tail_cap + row) * kD;
    const uint4 *kr = reinterpret_cast<const uint4 *>(kc.k_tail + at);
    const uint4 *vr = reinterpret_cast<const uint4 *>(kc.v_tail + at);
    uint32_t tk = 0, tv = 0;
    if (have) {
#pragma unroll 8
        for (int c = 0; c < kD / 8; ++c) {
            tk = __vmaxu2(tk, top_word(__ldg(kr + c)));
            tv = __vmaxu2(tv, top_word(__ldg(vr + c)));
        }
    }
    tk = top_of(tk);
    tv = top_of(tv);
    const bool bad_k = tk >= 0x7F80u, bad = bad_k || tv >= 0x7F80u;
    const uint32_t wk = __ballot_sync(0xffffffffu, bad_k), wb = __ballot_sync(0xffffffffu, bad);
    const int e = bad_k ? 0 : split_exp(tk);
    if (!warp_wait(smem_addr(&bar->tail_slots[t & (kTileRing - 1)]), (t >> 4) & 1, abort, hdr))
        return false;
    // Tile t - 4's notes are read until now at the latest.  These two K slots are
    // free: with at most five, QK of tile t - 2 is complete, and it waited until
    // tile t - 4's S was read, by warp 0 too, which reads them before it says so.
    // The softmax reads them before PV of that tile, and this warp waited for PV of
    // a later one.
    static_assert(kMaxStages <= 5, "a later QK than tile t - 4's successor in its S slot");
    if (lane == 0) {
        bar->bad_k[t & 3][w] = wk;
        bar->bad[t & 3][w] = wb;
    }
    aux->key_exp[t & 3][tid] = (uint8_t)(e + 127);
    const int e0 = bar->entry_of[t & 3];
    unsigned char *khi = sK + (e0 % SK) * kRawBytes, *klo = sK + ((e0 + 1) % SK) * kRawBytes;
    const float f = two_to(-e);
#pragma unroll 2
    for (int c = 0; c < kD / 16; ++c) {   // 16 codes a step
        uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
        if (have && !bad_k) {
            uint2 h0, l0, h1, l1;
            split_16b(__ldg(kr + 2 * c), f, h0, l0);
            split_16b(__ldg(kr + 2 * c + 1), f, h1, l1);
            hi = make_uint4(h0.x, h0.y, h1.x, h1.y);
            lo = make_uint4(l0.x, l0.y, l1.x, l1.y);
        }
        const int off = tid * 128 + ((c ^ (tid & 7)) << 4);
        *reinterpret_cast<uint4 *>(khi + off) = hi;
        *reinterpret_cast<uint4 *>(klo + off) = lo;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0)
        mbar_arrive(smem_addr(&bar->conv));
    if (!warp_wait(smem_addr(&bar->conv), met++ & 1, abort, hdr))
        return false;
    if (tid == 0) {
        mbar_arrive(smem_addr(&bar->full_k[e0 % SK]));
        mbar_arrive(smem_addr(&bar->full_k[(e0 + 1) % SK]));
    }
    __syncwarp();
    return true;
}

// The values of tail tile t (rows that are none, or noted by tail_keys, as
// zeros) into a bf16 V tile, by the same 128 threads.
__device__ __noinline__ void tail_values(const AttnQ8Args &a, Bars *bar, unsigned char *vb, int g, int nq,
                                         int tile, int t)
{
    const Q8Cache &kc = a.c;
    const int tid = threadIdx.x & 127;
    const int row = (tile - nq) * kTileN + tid;
    const bool use = row < kc.n_tail + a.n_tree && !((bar->bad[t & 3][tid >> 5] >> (tid & 31)) & 1u);
    const uint4 *vr = reinterpret_cast<const uint4 *>(kc.v_tail + ((int64_t)g * kc.tail_cap + row) * kD);
#pragma unroll 4
    for (int c = 0; c < kD / 8; ++c)
        *reinterpret_cast<uint4 *>(vb + (c >> 3) * kBoxBytes + tid * 128 + (((c & 7) ^ (tid & 7)) << 4)) =
            use ? __ldg(vr + c) : make_uint4(0u, 0u, 0u, 0u);
}

// (lane quarter, unit of 16 lanes) pairs that hold query rows of a block of
// `rows` rows in runs of rq per quarter.
__device__ __forceinline__ int active_units(int rows, int rq)
{
    int n = 0;
    for (int q = 0; q < 4; ++q)
        n += (max(0, min(rq, rows - q * rq)) + 15) / 16;
    return n;
}

// The kernel's three forms by the query rows of a CTA: up to 64 (one block,
// two groups of four softmax warps), up to 128 (one block, eight warps), up
// to 192 (two blocks, twelve warps).
template <int N>
struct Const {
    static constexpr int value = N;
};

template <int MODE>
struct Form {
    static constexpr int NB = MODE == 2 ? 2 : 1;     // query blocks
    static constexpr int NG = MODE == 0 ? 2 : 1;     // softmax groups
    static constexpr int U = MODE + 1;               // softmax warps per lane quarter and group
    static constexpr int U0 = MODE == 0 ? 1 : 2;     // of these in block 0
    static constexpr int SVB = MODE == 2 ? 1 : 2;    // bf16 V slots
    // K's loads from warp 0 instead of warp 3, when it has no root scores to
    // read: with V's they cost their warp 1500 cycles a tile, about what a tile
    // takes up to 64 rows (T = 13: 58 us against 65; with the root scores in the
    // same warp 84 against 67)
    static constexpr bool kSplit = MODE == 0;
    static constexpr int n_conv = kThreads / 32 - 4 - 4 * U * NG;   // converter warps, the last ones
};

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
attn_q8_t128_kernel(const __grid_constant__ CUtensorMap tmap_k,
                    const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ AttnQ8Args a,
                    const __grid_constant__ TreeMasks masks, int n_split, int nodes_per_group,
                    Q8Sync sy)
{
    const Q8Cache &kc = a.c;
    const int G = a.n_heads_q / a.n_heads_kv;
    const int node0 = blockIdx.z * nodes_per_group;
    const int T = min(nodes_per_group, a.n_tree - node0);
    const int R = G * T;
    using F = Form<MODE>;
    constexpr int NB = F::NB, NG = F::NG, U = F::U, SVB = F::SVB, n_conv = F::n_conv, NP = 2;
    const int R0 = R < kBlockM ? R : kBlockM, R1 = R - R0;
    // rows per lane quarter: a quarter of the block's, but at least 8 while
    // that needs no more warps (a warp takes 8 rows as fast as one), so that
    // the root node's rows 0..G-1, G <= 8, are the last block's first lanes
    const int rq0 = max((R0 + 3) / 4, min(R0, 8)), rq1 = max((R1 + 3) / 4, min(R1, 8));
    // (quarter, unit) pairs with query rows: their warps arrive on the barriers
    const int act0 = active_units(R0, rq0), act1 = active_units(R1, rq1);
    const bool rs_warp0 = a.root_scores != nullptr && node0 == 0;
    const bool k_split = F::kSplit && !rs_warp0;
    const int n_blk = kc.n_q8 / kQ8Block;
    const Layout lay = q8_layout(R, n_blk);
    const int SK = lay.stages_k, SV = lay.stages_v, r_pad = lay.r_pad;
    constexpr int SI = NB == 2 ? 1 : NP;   // one block: S barriers of tile t are [t % SI], its slot t & 1

    extern __shared__ unsigned char smem_raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char *sQ1 = base + lay.q1_off;
    unsigned char *sP = base + lay.p_off;
    unsigned char *sVb = base + lay.vb_off;
    unsigned char *sK = base + lay.k_off;
    unsigned char *sV = base + lay.v_off;
    Aux *aux = reinterpret_cast<Aux *>(base + lay.aux_off);
    uint8_t *s_scale = base + lay.sc_off;   // [2][n_blk]: K's bytes, V's
    Bars *bar = &aux->bar;
    WorkspaceHeader *hdr = reinterpret_cast<WorkspaceHeader *>(a.workspace);
    volatile uint32_t *abort = &bar->abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x, g = blockIdx.y;
    const int n_ctx = kc.n_q8 + kc.n_tail;
    const int tail_rows = kc.n_tail + a.n_tree;
    const int nq = (kc.n_q8 + kTileN - 1) / kTileN;
    const int n_tiles_all = nq + (tail_rows + kTileN - 1) / kTileN;
    const int gz = g * gridDim.z + blockIdx.z;

    if (threadIdx.x == 0) {
        for (int s = 0; s < SK; ++s) {
            mbar_init(smem_addr(&bar->full_k[s]), 1);
            mbar_init(smem_addr(&bar->empty_k[s]), 1);
        }
        for (int s = 0; s < SV; ++s) {
            mbar_init(smem_addr(&bar->full_v[s]), 1);
            mbar_init(smem_addr(&bar->empty_v[s]), n_conv);
        }
        const int rs = rs_warp0 ? 1 : 0;
        mbar_init(smem_addr(&bar->conv), kTailWarps);
        mbar_init(smem_addr(&bar->vb_full[0]), n_conv);
        mbar_init(smem_addr(&bar->vb_full[1]), n_conv);
        mbar_init(smem_addr(&bar->drain[0]), 1);
        mbar_init(smem_addr(&bar->drain[1]), 1);
        for (int i = 0; i < kTileRing; ++i) {
            mbar_init(smem_addr(&bar->info[i]), 1);
            mbar_init(smem_addr(&bar->tail_slots[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&bar->s_full[i]), 1);
            mbar_init(smem_addr(&bar->s_free[i]), NB == 1 ? act0 + rs : (i == 0 ? act0 : act1 + rs));
            mbar_init(smem_addr(&bar->sm_done[i]), act0 + act1);
            mbar_init(smem_addr(&bar->pv_done[i]), 1);
        }
        mbar_init(smem_addr(&bar->o_final), 1);
        bar->abort = 0u;
        bar->overflow = 0;
        fence_mbar_init();
        launch_dependents();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&bar->tmem_base), kTmemCols);
        tmem_relinquish();
    }
    if (warp == 3 && lane == 0 && nq > 0) {
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // a programmatic dependent: what follows reads the previous kernel's results
    grid_dependency_wait();
    const uint32_t tmem = bar->tmem_base;

    // node of row m (m < 192, G <= 128: half a unit off any border is far more
    // than the product's rounding), and its row of q and out
    const float inv_G = 1.f / (float)G;
    auto node_of = [&](int m) { return (int)(((float)m + 0.5f) * inv_G); };
    auto orow = [&](int m) {
        const int node = node_of(m);
        return (node0 + node) * a.n_heads_q + g * G + (m - node * G);
    };
    auto q_row = [&](int m) { return reinterpret_cast<const uint4 *>(a.q + (int64_t)orow(m) * kD); };

    if (warp < 4) {
        if (warp == 2)
            for (int i = lane; i < a.n_tree; i += 32)
                aux->anc[i] = masks.anc[i];
        if (warp == 1 || warp == 2) {
            tc_fence_before();
            named_bar_sync(kBarQuery, 32 * (2 + 4 * U * NG));
            tc_fence_after();
        }
        // K's loads: step t issues tile t's (a tail tile takes two slots, which the
        // converters fill)
        const uint64_t pol = l2_evict_first_policy();
        Ring rk(SK);
        int ke = 0, k_tma = -1;   // K ring entries used; the last that was a TMA load
        bool k_end = false;       // the end marker is on its way
        auto k_step = [&](int t) {
            const int at = t & (kTileRing - 1);
            if (k_split && !warp_wait(smem_addr(&bar->info[at]), (t >> 4) & 1, abort, hdr))
                return false;
            const int tile = bar->tile_of[at];
            const bool tail = tile >= nq;
            for (int part = 0; part < (tail ? 2 : 1); ++part, ++ke, rk.next()) {
                const int s = rk.i;
                if (ke >= SK && !warp_wait(smem_addr(&bar->empty_k[s]), rk.ph ^ 1, abort, hdr))
                    return false;
                if (lane == 0) {
                    const uint32_t fb = smem_addr(&bar->full_k[s]);
                    if (tile < 0) {
                        mbar_arrive(fb);   // no tile left: the QK issuer passes it on
                    } else if (!tail) {
                        mbar_arrive_expect_tx(fb, kRawBytes);
                        tma_load_3d_hint(smem_addr(sK + s * kRawBytes), &tmap_k, 0, tile * kTileN, g, fb, pol);
                        k_tma = ke;
                    } else if (part == 1) {
                        bar->entry_of[t & 3] = ke - 1;
                        mbar_arrive(smem_addr(&bar->tail_slots[at]));
                    }
                }
            }
            k_end = __any_sync(0xffffffffu, tile < 0);
            return true;
        };
        auto k_drain = [&]() {   // our own copies land before the CTA exits
            if (lane == 0 && *abort)
                for (int t = max(0, k_tma - SK + 1); t <= k_tma; ++t)
                    wait_drain(smem_addr(&bar->full_k[t % SK]), (t / SK) & 1);
        };
        if (warp == 3) {
            // ------------------------------------------------ tiles, TMA producer
            if (!k_split)   // (the query rows first, as below)
                named_bar_sync(kBarQLoads, kQLoadThreads);
            named_bar_sync(kBarScales, 32 * (n_conv + 1));
            // Four lanes post a tile each (index, scales), a few tiles ahead of the
            // loads
            constexpr int kRound = 4;
            // tile t of this CTA
            auto post = [&](int t, int tile) {
                if (lane >= kRound)
                    return;
                const int at = t & (kTileRing - 1);
                const bool tail = tile >= nq;
                bar->tile_of[at] = max(tile, -1);
                // context positions from the tile's first on
                const int left = tail ? kc.n_tail - (tile - nq) * kTileN : kc.n_q8 - tile * kTileN;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // (127, a factor of one, past the last block and on a tail tile)
                    const int b = 2 * tile + h;
                    const bool have = tile >= 0 && b < n_blk;
                    const uint32_t kb = have ? s_scale[b] : 127u;
                    const uint32_t vb = kb == 255u ? 255u : (have ? s_scale[n_blk + b] : 127u);
                    aux->scale_of[at][h] =
                        make_float4(q8_factor(kb), q8_log2(vb), q8_inverse(vb),
                                    __int_as_float(tile < 0 ? kEndMark
                                                            : min(max(left - 64 * h, -kTileN), 64) +
                                                                  (tail ? kTailMark : 0)));
                }
                if (tile < 0)   // (the second group's end)
                    aux->scale_of[(t + 1) & (kTileRing - 1)][0].w = __int_as_float(kEndMark);
            };
            const HandOut hand(n_split, nq, n_tiles_all);
            int posted = 0;
            bool more = true;
            auto post_round = [&]() {
                const int tile = hand.tile(split, posted + (lane & (kRound - 1)));
                more = __shfl_sync(0xffffffffu, tile, kRound - 1) >= 0;
                post(posted + lane, tile);
                __syncwarp();
                if (lane == 0)
                    for (int i = 0; i < kRound; ++i)
                        mbar_arrive(smem_addr(&bar->info[(posted + i) & (kTileRing - 1)]));
                posted += kRound;
            };
            post_round();
            Ring rv(SV);
            int v_tma = -1;
            for (int step = 0;; ++step) {
                // V one tile behind K where both are this warp's
                const int t = k_split ? step : step - 1;
                if (more && posted - t <= 2)
                    post_round();
                if (!k_split && !k_end && !k_step(step))
                    break;
                if (t < 0)
                    continue;
                const int tile = bar->tile_of[t & (kTileRing - 1)];
                int ok = 1;
                if (lane == 0) {
                    if (t >= SV)
                        ok = lane_wait(smem_addr(&bar->empty_v[rv.i]), rv.ph ^ 1, abort, hdr);
                    if (ok) {
                        const uint32_t fb = smem_addr(&bar->full_v[rv.i]);
                        if (tile < 0 || tile >= nq) {
                            mbar_arrive(fb);   // the end, or a tail tile: the converters read it themselves
                        } else {
                            mbar_arrive_expect_tx(fb, kRawBytes);
                            tma_load_3d_hint(smem_addr(sV + rv.i * kRawBytes), &tmap_v, 0, tile * kTileN, g, fb,
                                             pol);
                            v_tma = t;
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok || tile < 0)
                    break;
                rv.next();
            }
            if (!k_split)
                k_drain();
            if (lane == 0 && *abort)   // our own copies land before the CTA exits
                for (int t = max(0, v_tma - SV + 1); t <= v_tma; ++t)
                    wait_drain(smem_addr(&bar->full_v[t % SV]), (t / SV) & 1);
            __syncwarp();
        } else if (warp == 0) {
            if (k_split) {
                // -------------------------------------------- TMA producer of K
                // (the query rows first: not behind every CTA's first ring)
                named_bar_sync(kBarQLoads, kQLoadThreads);
                for (int t = 0; !k_end && k_step(t); ++t) {
                }
                k_drain();
            }
            // ------------------------------------------------ root node's scores out of S
            const int r = lane >> 2;
            const bool mine = r < G;
            const int c0 = 2 * (lane & 3);
            float rsc = 0.f;
            float *dst_row = a.root_scores + (size_t)(g * G + (mine ? r : 0)) * n_ctx;
            const bool vec = ((reinterpret_cast<uintptr_t>(a.root_scores) | (uintptr_t)n_ctx * 4) & 7) == 0;
            if (rs_warp0) {
                named_bar_sync(kBarRows, 32 * (1 + 4 * U * NG));
                rsc = aux->row_scale[NB == 2 ? kBlockM + (mine ? r : 0) : (mine ? r : 0)];
            }
            Ring rs(SI);
            for (int t = 0; rs_warp0; ++t, rs.next()) {
                const int slot = NB == 2 ? 1 : (t & 1), sb = NB == 2 ? 1 : rs.i;
                if (!warp_wait(smem_addr(&bar->s_full[sb]), rs.ph, abort, hdr))
                    break;
                const int tile = bar->tile_of[t & (kTileRing - 1)];
                if (tile < 0)
                    break;
                tc_fence_after();
                const bool q8 = tile < nq;
                const int r0 = (q8 ? tile : tile - nq) * kTileN;
                const int left = (q8 ? kc.n_q8 : kc.n_tail) - r0;   // context positions here
                const int pos0 = q8 ? r0 : kc.n_q8 + r0;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const int lh = left - 64 * h;
                    if (lh <= 0)
                        break;   // uniform: nothing of the context from here on
                    uint32_t rr[32];
                    tmem_ld16x256_x8(tmem + kSCol + 128 * slot + 64 * h, rr);
                    float *dst = dst_row + pos0 + 64 * h + c0;
                    if (mine && !q8) {
                        // a tail tile: the keys have a scale each
                        const unsigned long long nan = bar->bad_k[t & 3][2 * h] |
                                                       ((unsigned long long)bar->bad_k[t & 3][2 * h + 1] << 32);
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const int p = 8 * (k >> 1) + c0 + (k & 1);
                            const float f = rsc * two_to(aux->key_exp[t & 3][64 * h + p] - 127);
                            if (p < lh)
                                dst[8 * (k >> 1) + (k & 1)] =
                                    (nan >> p) & 1ull ? __uint_as_float(0x7FC00000u)
                                                      : __uint_as_float(rr[4 * (k >> 1) + (k & 1)]) * f;
                        }
                    } else if (mine) {
                        const float f = rsc * aux->scale_of[t & (kTileRing - 1)][h].x;
                        if (vec && lh >= 64) {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                *reinterpret_cast<float2 *>(dst + 8 * j) =
                                    make_float2(__uint_as_float(rr[4 * j]) * f,
                                                __uint_as_float(rr[4 * j + 1]) * f);
                        } else {
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const int p = 8 * (k >> 1) + c0 + (k & 1);
                                if (p < lh)
                                    dst[8 * (k >> 1) + (k & 1)] = __uint_as_float(rr[4 * (k >> 1) + (k & 1)]) * f;
                            }
                        }
                    }
                    __syncwarp();   // the next TMEM load is the whole warp's
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&bar->s_free[sb]));
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------ QK issuer
            // (the whole warp keeps the loop, so that descriptors stay uniform;
            // one elected lane issues)
            const uint32_t kd0 = (uint32_t)sdesc_sw128(smem_addr(sK), 16, 1024);
            const uint32_t qd0 = (uint32_t)sdesc_sw128(smem_addr(sQ1), 16, 1024);
            const bool leader = elect_one();
            // rb: S barrier of tile t; rf: of the tile before it in its slot
            // rp: P^T slot of tile t - 2
            Ring rk(SK), rb(SI), rf(SI), rp(2);
            for (int t = 0;; ++t) {
                if (!warp_wait(smem_addr(&bar->full_k[rk.i]), rk.ph, abort, hdr))
                    break;
                const int tile = bar->tile_of[t & (kTileRing - 1)];
                if (__any_sync(0xffffffffu, tile < 0)) {
                    // the end, to each block or each group, once its readers are
                    // past the barrier's last phase
                    for (int i = 0; i < (NB == 2 ? 2 : NG); ++i) {
                        const int sb = NB == 2 ? i : rb.i, before = NB == 2 ? t - 1 : t + i - SI;
                        // (one phase before this barrier's next)
                        if (before >= 0 && !warp_wait(smem_addr(&bar->s_free[sb]), rb.ph ^ 1, abort, hdr))
                            break;
                        if (leader)
                            mbar_arrive(smem_addr(&bar->s_full[sb]));
                        if (NB == 1)
                            rb.next();
                    }
                    break;
                }
                const bool two = __any_sync(0xffffffffu, tile >= nq);
                const int k0 = rk.i;
                rk.next();
                bool ok = !two || warp_wait(smem_addr(&bar->full_k[rk.i]), rk.ph, abort, hdr);
                const int k1 = rk.i;
                if (two)
                    rk.next();
                // one group: S(t) stands for its P^T slot, too (PV(t - 2) is done)
                if (NG == 1 && t >= 2) {
                    ok = ok && warp_wait(smem_addr(&bar->pv_done[rp.i]), rp.ph, abort, hdr);
                    rp.next();
                }
                for (int b = 0; b < NB && ok; ++b) {
                    const int slot = NB == 2 ? b : (t & 1), sb = NB == 2 ? b : rb.i;
                    // the tile before it in this slot is in its readers' registers
                    if (t >= (NB == 2 ? 1 : 2) &&
                        !warp_wait(smem_addr(&bar->s_free[NB == 2 ? b : rf.i]), rf.ph, abort, hdr)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + kSCol + 128 * slot;
                    constexpr uint32_t id = idesc_f8(kBlockM, kTileN, 0, 0);
                    // K's codes (hi, then lo on a tail tile), each times Q's hi and lo
                    uint32_t kd = kd0 + (uint32_t)k0 * (kRawBytes >> 4);
                    if (leader) {
                        if (b == 0)
                            mma_qk_ts(d, tmem + kQCol, kd, id, 0);
                        else
                            mma_qk_ss(d, qd0, kd, id, 0);
                    }
                    if (two) {
                        kd = kd0 + (uint32_t)k1 * (kRawBytes >> 4);
                        if (leader) {
                            if (b == 0)
                                mma_qk_ts(d, tmem + kQCol, kd, id | (1u << 10), 1);
                            else
                                mma_qk_ss(d, qd0, kd, id | (1u << 10), 1);
                        }
                    }
                    if (leader)
                        mma_commit(smem_addr(&bar->s_full[sb]));
                }
                if (!ok)
                    break;
                if (leader) {
                    mma_commit(smem_addr(&bar->empty_k[k0]));
                    if (two)
                        mma_commit(smem_addr(&bar->empty_k[k1]));
                }
                rb.next();
                if (t >= (NB == 2 ? 1 : 2))
                    rf.next();
            }
            if (leader) {
                mma_commit(smem_addr(&bar->drain[0]));
                wait_drain(smem_addr(&bar->drain[0]), 0);
            }
            __syncwarp();
        } else {
            // ------------------------------------------------ PV issuer
            const uint32_t idesc = idesc_bf16(kD, r_pad, 1, 0);
            const uint32_t vd0 = (uint32_t)sdesc_sw128(smem_addr(sVb), kBoxBytes, 1024);
            const uint32_t pd0 = (uint32_t)sdesc_sw128(smem_addr(sP), 16, 1024);
            const uint32_t p_half = (uint32_t)r_pad * 128;
            const bool leader = elect_one();
            Ring rp(NP), rvb(SVB);
            for (int t = 0;; ++t, rp.next(), rvb.next()) {
                if (!warp_wait(smem_addr(&bar->info[t & (kTileRing - 1)]), (t >> 4) & 1, abort, hdr))
                    break;
                if (__any_sync(0xffffffffu, bar->tile_of[t & (kTileRing - 1)] < 0)) {
                    if (leader)
                        mma_commit(smem_addr(&bar->o_final));   // after the last PV
                    break;
                }
                const int ps = rp.i, s = rvb.i;
                if (!warp_wait(smem_addr(&bar->vb_full[s]), rvb.ph, abort, hdr) ||
                    !warp_wait(smem_addr(&bar->sm_done[ps]), rp.ph, abort, hdr))
                    break;
                tc_fence_after();
                const uint32_t vd = vd0 + (uint32_t)s * (kVbBytes >> 4);
                const uint32_t pd = pd0 + (uint32_t)ps * (uint32_t)(r_pad * 16);
                if (leader) {
                    mma_pv(tmem + (NG == 2 ? 64 * ps : 0), vd, pd, pd + (p_half >> 4), idesc,
                           t >= NG ? 1u : 0u);
                    mma_commit(smem_addr(&bar->pv_done[ps]));
                }
            }
            if (leader) {
                mma_commit(smem_addr(&bar->drain[1]));
                wait_drain(smem_addr(&bar->drain[1]), 0);
            }
            __syncwarp();
        }
    } else if (warp >= kThreads / 32 - n_conv) {
        // ------------------------------------------------ converters
        const int tid = threadIdx.x - 32 * (kThreads / 32 - n_conv), rows = 2 * n_conv;   // rows per step
        // every scale byte of the head, for the producer (one look-up per tile
        // in HBM would cost it more than the tile's stream)
        {
            const uint8_t *ksc = kc.k_scale + (int64_t)g * (kc.q8_cap / kQ8Block);
            const uint8_t *vsc = kc.v_scale + (int64_t)g * (kc.q8_cap / kQ8Block);
            for (int i = tid; i < n_blk; i += 32 * n_conv) {
                s_scale[i] = __ldg(ksc + i);
                s_scale[n_blk + i] = __ldg(vsc + i);
            }
            named_bar_arrive(kBarScales, 32 * (n_conv + 1));
        }
        // this thread's share of V's codes: a column chunk and every `rows`-th
        // row, all with the same row mod 8
        const int ch = tid & 15, r0 = tid >> 4;
        const uint32_t c_dst = (uint32_t)((ch >> 3) * kBoxBytes + r0 * 128 + (((ch & 7) ^ (r0 & 7)) << 4));
        int met = 0;   // meetings of the converters over tail tiles
        bool tail = true;
        Ring rv(SV), rvb(SVB), rpv(NP);   // rpv: PV of the tile before in the bf16 slot
        for (int t = 0;; ++t, rv.next(), rvb.next()) {
            // tail tiles, if any, come first, and their keys before their values
            if (tail) {
                if (!warp_wait(smem_addr(&bar->info[t & (kTileRing - 1)]), (t >> 4) & 1, abort, hdr))
                    break;
                tail = __any_sync(0xffffffffu, bar->tile_of[t & (kTileRing - 1)] >= nq);
                if (tail && warp >= 16 && !tail_keys(a, aux, sK, SK, g, nq, t, met, abort, hdr))
                    break;
            }
            if (!warp_wait(smem_addr(&bar->full_v[rv.i]), rv.ph, abort, hdr))
                break;
            const int tile = bar->tile_of[t & (kTileRing - 1)];
            if (tile < 0)
                break;
            if (t >= SVB) {
                if (!warp_wait(smem_addr(&bar->pv_done[rpv.i]), rpv.ph, abort, hdr))
                    break;
                rpv.next();
            }
            unsigned char *vb = sVb + rvb.i * kVbBytes;
            if (!tail) {
                const unsigned char *src = sV + rv.i * kRawBytes + 8 * tid;
                unsigned char *dst = vb + c_dst;
                // two steps' loads before their stores (which could alias them as
                // far as the compiler knows); more at once is slower, as the code
                // then drives the softmax's out of the instruction cache
#pragma unroll 1
                for (int r = r0; r < kTileN; r += 2 * rows) {
                    uint2 w[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        w[i] = *reinterpret_cast<const uint2 *>(src + i * rows * kD);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint2 x = codes_to_bf16(w[i].x), y = codes_to_bf16(w[i].y);
                        *reinterpret_cast<uint4 *>(dst + i * rows * 128) = make_uint4(x.x, x.y, y.x, y.y);
                    }
                    src += 2 * rows * kD;
                    dst += 2 * rows * 128;
                }
            } else if (warp >= 16) {
                tail_values(a, bar, vb, g, nq, tile, t);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_addr(&bar->vb_full[rvb.i]));
                mbar_arrive(smem_addr(&bar->empty_v[rv.i]));
            }
        }
    } else {
        // ---- query rows of this KV head: row n = node * G + (head - g*G),
        // block 0 into TMEM lanes (warps 4-7), block 1 into the shared-memory
        // A tile (warps 8-11), each split into hi and lo codes
        // (rows that are none keep whatever is there: their scores go nowhere).
        // Sixteen lanes read a row (a thread per row took 8000 cycles at T = 40,
        // scattered loads and a long chain each); block 0's codes pass through
        // the P^T tiles, as TMEM wants a row per lane
        {
            constexpr int n_sm = 4 * U * NG;   // softmax warps
            const int l16 = lane & 15;
            bool first = true;
            for (int k0 = 2 * (warp - 4); k0 < R || first; k0 += 4 * 2 * n_sm) {
                uint4 u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = k0 + 2 * n_sm * i + (lane >> 4);
                    u[i] = n < R ? __ldg(q_row(q8_row_of(n, R)) + l16) : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = k0 + 2 * n_sm * i + (lane >> 4);
                    uint32_t top = top_word(u[i]);
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1)
                        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
                    top = top_of(top);
                    const bool bad = top >= 0x7F80u;
                    const int e = bad ? 0 : split_exp(top);
                    uint2 hi, lo;
                    split_16b(u[i], two_to(-e), hi, lo);
                    if (n < R) {
                        if (l16 == 0)
                            aux->row_scale[n] = bad ? __uint_as_float(0x7FC00000u) : a.scale_log2 * two_to(e);
                        // row n's codes: hi in chunks 0-7 of 16 bytes, lo in 8-15
                        if (NB == 1 || n < kBlockM) {
                            unsigned char *row = sP + n * 256 + 8 * (l16 & 1);
                            *reinterpret_cast<uint2 *>(row + (((l16 >> 1) ^ (n & 15)) << 4)) = hi;
                            *reinterpret_cast<uint2 *>(row + (((8 + (l16 >> 1)) ^ (n & 15)) << 4)) = lo;
                        } else {
                            const int n1 = n - kBlockM, q1 = n1 / rq1, m = q1 * 32 + n1 - q1 * rq1;
                            unsigned char *row = sQ1 + m * 128 + (((l16 >> 1) ^ (m & 7)) << 4) + 8 * (l16 & 1);
                            *reinterpret_cast<uint2 *>(row) = hi;
                            *reinterpret_cast<uint2 *>(row + kBlockM * kD) = lo;
                        }
                    }
                }
                if (first && warp < 12)
                    named_bar_arrive(kBarQLoads, kQLoadThreads);
                first = false;
            }
            if (NB == 2)
                fence_proxy_async_smem();
            named_bar_sync(kBarOut, 32 * n_sm);
            if (NB == 1 || warp < 8 || warp >= 12) {
                // two warps per lane quarter, 64 dims each
                const int q = warp & 3, h = warp >= 8 ? 1 : 0;
                const int n = q * rq0 + lane;
                const bool valid = lane < rq0 && n < R0;
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const unsigned char *row = sP + (valid ? n : 0) * 256;
                    const int x = valid ? n & 15 : 0;
                    const uint4 a4 = *reinterpret_cast<const uint4 *>(row + (((4 * h + c) ^ x) << 4));
                    const uint4 b4 = *reinterpret_cast<const uint4 *>(row + (((8 + 4 * h + c) ^ x) << 4));
                    hi[4 * c] = a4.x; hi[4 * c + 1] = a4.y; hi[4 * c + 2] = a4.z; hi[4 * c + 3] = a4.w;
                    lo[4 * c] = b4.x; lo[4 * c + 1] = b4.y; lo[4 * c + 2] = b4.z; lo[4 * c + 3] = b4.w;
                }
                const uint32_t qa = tmem + ((uint32_t)(q * 32) << 16) + kQCol + 16 * h;
                __syncwarp();
                tmem_st16(qa, hi);
                tmem_st16(qa + 32, lo);
                tmem_st_wait();
            }
        }
        tc_fence_before();
        if (rs_warp0)
            named_bar_arrive(kBarRows, 32 * (1 + 4 * U * NG));
        named_bar_sync(kBarQuery, 32 * (2 + 4 * U * NG));
        tc_fence_after();
        if ((warp - 4) / 4 < U * NG) {
            // ------------------------------------------------ softmax
            const int q = warp & 3, j = NG == 2 ? 0 : (warp - 4) >> 2;
            const int grp = NG == 2 ? (warp - 4) >> 2 : 0;
            const int b = j < F::U0 ? 0 : 1;
            const int lb = 16 * (b == 0 ? j : j - F::U0);  // unit's first lane in the quarter
            const int Rb = b == 0 ? R0 : R1, rqb = b == 0 ? rq0 : rq1;
            const int iA = lb + (lane >> 2), iB = iA + 8;
            const bool vA = iA < rqb && q * rqb + iA < Rb;
            const bool vB = iB < rqb && q * rqb + iB < Rb;
            const bool hasA = __any_sync(0xffffffffu, vA), hasB = __any_sync(0xffffffffu, vB);
            const int nA = kBlockM * b + q * rqb + iA, nB = nA + 8;
            const uint32_t s_addr = tmem + ((uint32_t)(32 * q + lb) << 16) + kSCol;
            const int c0 = 2 * (lane & 3);
            const int nbase = kBlockM * b + q * rqb + lb;
            const int nvA = max(0, min(8, min(rqb - lb, Rb - q * rqb - lb)));
            const int nvB = max(0, min(8, min(rqb - lb - 8, Rb - q * rqb - lb - 8)));
            // this lane's P^T rows of the unit's halves A and B (stmatrix: lane
            // l gives the address of row l % 8); rows that are none go to the
            // scratch kilobyte
            const uint32_t p_addr = smem_addr(sP);
            const uint32_t p_scratch = p_addr + (uint32_t)r_pad * 256 * NP;
            const int rl = lane & 7, pnA = nbase + rl, pnB = pnA + 8;
            const bool okA = rl < nvA, okB = rl < nvB;
            const uint32_t p_rowA = okA ? p_addr + (uint32_t)((pnA >> 3) * 1024 + (pnA & 7) * 128) : p_scratch;
            const uint32_t p_rowB = okB ? p_addr + (uint32_t)((pnB >> 3) * 1024 + (pnB & 7) * 128) : p_scratch;
            const uint32_t p_half = (uint32_t)r_pad * 128;
            const uint32_t p_stepA = okA ? p_half : 0u, p_stepB = okB ? p_half : 0u;
            const int rxA = okA ? pnA & 7 : 0, rxB = okB ? pnB & 7 : 0;
            const float rsA = vA ? aux->row_scale[nA] : 1.f, rsB = vB ? aux->row_scale[nB] : 1.f;
            const unsigned long long ancA = aux->anc[node0 + (vA ? node_of(q8_row_of(nA, R)) : 0)];
            const unsigned long long ancB = aux->anc[node0 + (vB ? node_of(q8_row_of(nB, R)) : 0)];
            // references, negated (2^(x + n)); sums, NaN from the start for a
            // query row that is none (its scale is NaN)
            float mA = -INFINITY, mB = -INFINITY, nmA = 0.f, nmB = 0.f;
            float lA = rsA == rsA ? 0.f : rsA, lB = rsB == rsB ? 0.f : rsB;
            bool fresh = true;   // some row has no reference yet (uniform)
            bool ok = true;
            // S barriers and P^T slots, fixed for a group (phases alternate) or by
            // tile
            Ring rsb(NG == 2 || NB == 2 ? 1 : 2), rps(NG == 2 ? 1 : 2);
            // Part of a half tile in registers (8 J positions, from the half's
            // 32 odd on): weights to P^T
            auto part = [&](auto &r, auto jc, auto special, int odd, int left, int t, int h, float cA, float cB, float ve,
                            float (&sum)[4], uint32_t atA, uint32_t atB) {
                constexpr int J = decltype(jc)::value;
                constexpr bool kSpecial = decltype(special)::value != 0;
                if (kSpecial && (left < 64 || left > kTailMark / 2)) {
                    // masked: the first positions of the half are context, then (a
                    // tail tile) come the tree's, of which a row sees its path
                    const bool tail = left > kTailMark / 2;
                    const int d = tail ? left - kTailMark : left;
                    if (tail) {
                        // the keys have a scale each: the scores in full, before the
                        // masks (a query row that is none has a NaN for its scale)
                        const uint8_t *ke = aux->key_exp[t & 3] + 64 * h + 32 * odd + c0;
#pragma unroll
                        for (int w = 0; w < J; ++w) {
                            const uint32_t two = *reinterpret_cast<const uint16_t *>(ke + 8 * w);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float f = __uint_as_float(((two >> (8 * i)) & 0xFFu) << 23);
                                r[4 * w + i] = __float_as_uint(__uint_as_float(r[4 * w + i]) * fmaxf(rsA * f, 0.f));
                                r[4 * w + 2 + i] =
                                    __float_as_uint(__uint_as_float(r[4 * w + 2 + i]) * fmaxf(rsB * f, 0.f));
                            }
                        }
                        cA = cB = 1.f;
                    }
                    const unsigned long long wA = row_vis(tail ? ancA : 0ull, d);
                    const unsigned long long wB = row_vis(tail ? ancB : 0ull, d);
#pragma unroll
                    for (int w = 0; w < J / 4; ++w) {
                        const uint32_t qA = (uint32_t)(wA >> (32 * (odd + w))) >> c0;
                        const uint32_t qB = (uint32_t)(wB >> (32 * (odd + w))) >> c0;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int bit = 8 * (k >> 1) + (k & 1), e = 16 * w + 4 * (k >> 1) + (k & 1);
                            if (!((qA >> bit) & 1u))
                                r[e] = __float_as_uint(-INFINITY);
                            if (!((qB >> bit) & 1u))
                                r[e + 2] = __float_as_uint(-INFINITY);
                        }
                    }
                    if (tail) {
                        // a row that sees a value that is no number
                        const unsigned long long bw =
                            bar->bad[t & 3][2 * h] | ((unsigned long long)bar->bad[t & 3][2 * h + 1] << 32);
                        if (wA & bw)
                            lA = __uint_as_float(0x7FC00000u);
                        if (wB & bw)
                            lB = __uint_as_float(0x7FC00000u);
                    }
                }
                if (kSpecial && fresh) {
                    // a row that has seen nothing yet takes this part's max,
                    // rounded up to an integer, as its reference
                    float yA = part_max<0, J>(r) * cA, yB = part_max<2, J>(r) * cB;
                    yA = fmaxf(yA, __shfl_xor_sync(0xffffffffu, yA, 1));
                    yB = fmaxf(yB, __shfl_xor_sync(0xffffffffu, yB, 1));
                    yA = fmaxf(yA, __shfl_xor_sync(0xffffffffu, yA, 2));
                    yB = fmaxf(yB, __shfl_xor_sync(0xffffffffu, yB, 2));
                    if (mA == -INFINITY)
                        mA = ceilf(yA);
                    if (mB == -INFINITY)
                        mB = ceilf(yB);
                    nmA = mA == -INFINITY ? 0.f : -mA;
                    nmB = mB == -INFINITY ? 0.f : -mB;
                    fresh = __any_sync(0xffffffffu, (vA && mA == -INFINITY) || (vB && mB == -INFINITY));
                }
                uint32_t pA[J], pB[J];
                exp_row<0, J>(r, cA, nmA + ve, pA, sum[0], sum[1]);
                if (hasB)
                    exp_row<2, J>(r, cB, nmB + ve, pB, sum[2], sum[3]);
                if (NG == 2 && h == 0 && t >= 2 &&
                    !warp_wait(smem_addr(&bar->pv_done[grp]), rps.ph ^ 1, abort, hdr))
                    ok = false;
#pragma unroll
                for (int w = 0; w < J / 4; ++w)
                    stmatrix_x4(atA + (uint32_t)(((4 * (odd + w) + (lane >> 3)) ^ rxA) << 4), pA[4 * w],
                                pA[4 * w + 1], pA[4 * w + 2], pA[4 * w + 3]);
                if (hasB) {
#pragma unroll
                    for (int w = 0; w < J / 4; ++w)
                        stmatrix_x4(atB + (uint32_t)(((4 * (odd + w) + (lane >> 3)) ^ rxB) << 4), pB[4 * w],
                                    pB[4 * w + 1], pB[4 * w + 2], pB[4 * w + 3]);
                }
            };
            // One tile's scores to weights.  The halves are its two scale blocks;
            // one copy of the code serves both (the loop must stay inside the
            // instruction cache).  With a warp or two per sub-partition a half at
            // once has the longer independent stretches; with more, quarters, each
            // on its way while the one before is turned to weights, hide the loads
            // (measured with fewer other gains: T = 13 66 us against 71, T = 40 98
            // against 104).
            auto pass = [&](auto special, const float4 *scl, uint32_t s0, int t, uint32_t atA, uint32_t atB,
                            uint32_t bar_free) {
                uint32_t r0[NG == 2 ? 32 : 16];
                [[maybe_unused]] uint32_t r1[16];
                if constexpr (NG == 1) {
                    tmem_ld16x256_x4(s0, r0);
                    tmem_ld_wait16(r0);
                }
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const float4 sc = scl[h];
                    if constexpr (NG == 1)
                        tmem_ld16x256_x4(s0 + 64 * h + 32, r1);
                    else
                        tmem_ld16x256_x8(s0 + 64 * h, r0);
                    // factor of the scores: never zero, as a masked score is -inf
                    constexpr float kTiny = 1.17549435e-38f;
                    const float cA = fmaxf(rsA * sc.x, kTiny), cB = fmaxf(rsB * sc.x, kTiny);
                    const int left = __float_as_int(sc.w);
                    float sum[4] = {};
                    if constexpr (NG == 1) {
                        part(r0, Const<4>(), special, 0, left, t, h, cA, cB, sc.y, sum, atA, atB);
                        tmem_ld_wait16(r1);
                    }
                    if (h == 0) {
                        if constexpr (NG == 1)
                            tmem_ld16x256_x4(s0 + 64, r0);
                    } else {
                        // S is in registers: QK of a later tile may overwrite it
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(bar_free);
                    }
                    if constexpr (NG == 1)
                        part(r1, Const<4>(), special, 1, left, t, h, cA, cB, sc.y, sum, atA, atB);
                    else
                        part(r0, Const<8>(), special, 0, left, t, h, cA, cB, sc.y, sum, atA, atB);
                    lA += (sum[0] + sum[1]) * sc.z;
                    lB += (sum[2] + sum[3]) * sc.z;
                    atA += p_stepA;
                    atB += p_stepB;
                    if constexpr (NG == 1)
                        if (h == 0)
                            tmem_ld_wait16(r0);
                }
            };
            for (int t = grp; hasA; t += NG, rsb.next(), rps.next()) {
                const int ps = NG == 2 ? grp : rps.i;
                const int slot = NB == 2 ? b : (t & 1), sb = NB == 2 ? b : (NG == 2 ? grp : rsb.i);
                // (with one group S(t) in place also says that this P^T slot is
                // free; with two that would tie a group to its own PV)
                if (!warp_wait(smem_addr(&bar->s_full[sb]), rsb.ph, abort, hdr)) {
                    ok = false;
                    break;
                }
                const float4 *scl = aux->scale_of[t & (kTileRing - 1)];
                const int w0 = __float_as_int(scl[0].w), w1 = __float_as_int(scl[1].w);
                if (w0 == kEndMark)
                    break;
                tc_fence_after();
                const uint32_t atA = p_rowA + 2 * ps * p_stepA, atB = p_rowB + 2 * ps * p_stepB;
                // masks and references only where a tile asks for them
                if (fresh || w0 != 64 || w1 != 64)
                    pass(Const<1>(), scl, s_addr + 128 * slot, t, atA, atB, smem_addr(&bar->s_free[sb]));
                else
                    pass(Const<0>(), scl, s_addr + 128 * slot, t, atA, atB, smem_addr(&bar->s_free[sb]));
                if (!ok)
                    break;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&bar->sm_done[ps]));
            }
            // ---- (m, l) of each row (four threads' partial sums), then O^T
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
                lA += __shfl_xor_sync(0xffffffffu, lA, o);
                lB += __shfl_xor_sync(0xffffffffu, lB, o);
            }
            // a sum past 2^63 flags the split for the exact recompute (NaN
            // stays NaN)
            const bool over = (vA && lA > kMaxRowSum) || (vB && lB > kMaxRowSum);
            if (__any_sync(0xffffffffu, over) && lane == 0)
                bar->overflow = 1;
            const int rows_all = a.n_tree * a.n_heads_q;
            float *ws_o = sy.part;
            float2 *ws_ml = reinterpret_cast<float2 *>(ws_o + (size_t)n_split * rows_all * kD);
            const size_t part_row = (size_t)split * rows_all;
            auto orow_of = [&](int n) { return orow(q8_row_of(n, R)); };
            if (ok && (lane & 3) == 0) {
                if (vA) {
                    if (NG == 2)
                        aux->ml[grp][nA] = make_float2(mA, lA);
                    else
                        ws_ml[part_row + orow_of(nA)] = make_float2(mA, lA);
                }
                if (vB) {
                    if (NG == 2)
                        aux->ml[grp][nB] = make_float2(mB, lB);
                    else
                        ws_ml[part_row + orow_of(nB)] = make_float2(mB, lB);
                }
            }
            // O^T out of TMEM into shared memory in output order, from the P^T
            // tiles on (all of it is free after the last PV; one group's rows
            // are as large as two P^T tiles), then one bulk copy per node
            unsigned char *stage = sP + (size_t)grp * R * kD * 4;
            const bool have_o = ok && warp_wait(smem_addr(&bar->o_final), 0, abort, hdr);
            if (have_o) {
                tc_fence_after();
                for (int c = 32 * j; c < r_pad; c += 32 * U) {
                    // (steps of eight columns: short code, run once)
                    float *dst = reinterpret_cast<float *>(stage) + (size_t)q8_row_of(c, R) * kD + 32 * q + lane;
#pragma unroll 1
                    for (int c8 = 0; c8 < 32 && c + c8 < R; c8 += 8, dst += 8 * kD) {
                        uint32_t o[8];
                        tmem_ld8(tmem + ((uint32_t)(32 * q) << 16) + 64 * grp + c + c8, o);
                        const int nv = R - c - c8;   // query rows among these
#pragma unroll
                        for (int jj = 0; jj < 8; ++jj)
                            if (jj < nv)
                                dst[jj * kD] = __uint_as_float(o[jj]);
                    }
                }
            }
            fence_proxy_async_smem();
            named_bar_sync(kBarOut, 128 * U * NG);   // every softmax warp, whatever its path
            if (NG == 2) {
                // the groups' partials into one (all of a row's by one warp)
                for (int r = warp - 4; r < R && !*abort; r += 8) {
                    const float2 p0 = aux->ml[0][r], p1 = aux->ml[1][r];
                    const float M = fmaxf(p0.x, p1.x);
                    // a group that saw nothing (m = -inf) has l = 0, or NaN, and any O
                    const float w0 = p0.x == -INFINITY ? 0.f : exp2f(p0.x - M);
                    const float w1 = p1.x == -INFINITY ? 0.f : exp2f(p1.x - M);
                    float4 *o = reinterpret_cast<float4 *>(sP) + r * (kD / 4) + lane;
                    float4 x = w0 != 0.f ? *o : make_float4(0.f, 0.f, 0.f, 0.f);
                    const float4 y = w1 != 0.f ? o[R * (kD / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
                    x.x = w0 * x.x + w1 * y.x;
                    x.y = w0 * x.y + w1 * y.y;
                    x.z = w0 * x.z + w1 * y.z;
                    x.w = w0 * x.w + w1 * y.w;
                    *o = x;
                    if (lane == 0)
                        ws_ml[part_row + orow_of(r)] = make_float2(M, w0 * p0.y + w1 * p1.y);
                }
                fence_proxy_async_smem();
                named_bar_sync(kBarOut, 128 * U * NG);
            }
            if (!*abort && lane == 0) {
                const int sw = warp - 4, n_sw = 4 * U * NG;
                for (int node = sw; node < T; node += n_sw)
                    bulk_store(ws_o + (part_row + (size_t)(node0 + node) * a.n_heads_q + g * G) * kD,
                               smem_addr(sP) + (uint32_t)(node * G * kD * 4), (uint32_t)(G * kD * 4));
                bulk_commit();
                bulk_wait_all();
                fence_proxy_async_global();
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }

    // ---- combine: once every split of this (head, group) has arrived, each
    // folds half rows split, split + n_split, ... (one warp each)
    const int n_gz = a.n_heads_kv * gridDim.z;
    int32_t *ctr = sy.sync + 4 * gz;
    if (threadIdx.x == 0) {
        sy.flags[(size_t)split * n_gz + gz] = bar->overflow;
        __threadfence();   // partials and flag before the arrival
        atomicAdd(&ctr[1], 1);
        wait_count_bounded(&ctr[1], n_split, abort, hdr);
    }
    __syncthreads();
    if (!*abort) {
        for (int u = split + warp * n_split; u < 2 * R; u += (kThreads / 32) * n_split) {
            const int m = u >> 1;
            combine_row(a, masks, orow(m), u & 1, g, gz, n_gz,
                        n_split, nq, n_tiles_all, sy);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(&ctr[2], 1) == n_split - 1) {
        atomicExch(&ctr[1], 0);
        atomicExch(&ctr[2], 0);
    }
}

struct T128Plan {
    int n_split, node_groups, nodes_per_group;
    size_t part, flags, total;
};

T128Plan q8_plan(int n_heads_q, int n_heads_kv, int n_q8, int n_tail, int n_tree, int num_sms)
{
    T128Plan p;
    const int G = n_heads_q / n_heads_kv, rows = G * n_tree;
    // (warp 0 reads the root node's G rows out of the last block: where they
    // would lie in both, two groups)
    const bool one = rows <= kMaxRows && !(G <= 8 && rows > kBlockM && rows < kBlockM + G);
    p.node_groups = one ? 1 : (rows + kBlockM - 1) / kBlockM;
    p.nodes_per_group = (n_tree + p.node_groups - 1) / p.node_groups;
    // whole nodes per CTA: a group's rows must fit one block
    if (p.node_groups > 1 && p.nodes_per_group * G > kBlockM)
        p.nodes_per_group = kBlockM / G;
    p.node_groups = (n_tree + p.nodes_per_group - 1) / p.nodes_per_group;
    const int n_tiles = (n_q8 + kTileN - 1) / kTileN + (n_tail + n_tree + kTileN - 1) / kTileN;
    int want = num_sms / (n_heads_kv * p.node_groups);
    want = want < 1 ? 1 : want;
    want = want > n_tiles ? n_tiles : want;
    p.n_split = want;
    const size_t n_gz = (size_t)n_heads_kv * p.node_groups;
    p.part = kHeaderBytes + kQ8SyncBytes;
    p.flags = p.part + align_up((size_t)p.n_split * n_tree * n_heads_q * (kD + 2) * sizeof(float), 256);
    p.total = p.flags + align_up((size_t)p.n_split * n_gz * sizeof(int32_t), 256);
    return p;
}

bool encode_codes_map(CUtensorMap *m, const void *ptr, int rows, int64_t cap, int n_heads_kv,
                      bool swizzled)
{
    auto enc = tensor_map_encoder();
    if (!enc)
        return false;
    const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)rows, (cuuint64_t)n_heads_kv};
    const cuuint64_t strides[2] = {(cuuint64_t)kD, (cuuint64_t)cap * kD};
    const cuuint32_t box[3] = {kD, kTileN, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool attn_q8_t128_eligible(int n_heads_q, int n_heads_kv, int head_dim, int n_q8, int n_tail,
                           int n_tree, int num_sms)
{
    // a CTA takes whole tree nodes: one node's G rows must fit one block;
    // one CTA per SM, all resident
    if (head_dim != kD || n_heads_q / n_heads_kv > kBlockM)
        return false;
    const T128Plan p = q8_plan(n_heads_q, n_heads_kv, n_q8, n_tail, n_tree, num_sms);
    const long long gz = (long long)n_heads_kv * p.node_groups;
    // the scale bytes of a long head leave room for the rings
    const Layout lay = q8_layout(n_heads_q / n_heads_kv * p.nodes_per_group, n_q8 / kQ8Block);
    return gz <= kMaxGz && gz * p.n_split <= num_sms && lay.stages_k >= 2 && lay.stages_v >= 1;
}

size_t attn_q8_t128_workspace_bytes(int n_heads_q, int n_heads_kv, int n_q8, int n_tail, int n_tree,
                                    int num_sms)
{
    return q8_plan(n_heads_q, n_heads_kv, n_q8, n_tail, n_tree, num_sms).total;
}

cudaError_t attn_q8_t128_launch(const AttnQ8Args &a, const TreeMasks &masks, int num_sms,
                                cudaStream_t stream)
{
    const T128Plan p = q8_plan(a.n_heads_q, a.n_heads_kv, a.c.n_q8, a.c.n_tail, a.n_tree, num_sms);
    CUtensorMap mk = {}, mv = {};
    if (a.c.n_q8 > 0 &&
        (!encode_codes_map(&mk, a.c.k8, a.c.n_q8, a.c.q8_cap, a.n_heads_kv, true) ||
         !encode_codes_map(&mv, a.c.v8, a.c.n_q8, a.c.q8_cap, a.n_heads_kv, false)))
        return cudaErrorInvalidValue;
    // by the rows of the first node group, the largest
    const int rows = (a.n_heads_q / a.n_heads_kv) * p.nodes_per_group;
    const auto kernel = rows <= 64        ? attn_q8_t128_kernel<0>
                        : rows <= kBlockM ? attn_q8_t128_kernel<1>
                                          : attn_q8_t128_kernel<2>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemLimit);
    if (e != cudaSuccess)
        return e;
    char *ws = reinterpret_cast<char *>(a.workspace);
    Q8Sync sy;
    sy.sync = reinterpret_cast<int32_t *>(ws + kHeaderBytes);
    sy.part = reinterpret_cast<float *>(ws + p.part);
    sy.flags = reinterpret_cast<int32_t *>(ws + p.flags);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.n_split, a.n_heads_kv, p.node_groups);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemLimit;   // each group lays out its own rows' share
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kernel, mk, mv, a, masks, p.n_split, p.nodes_per_group, sy);
    if (e == cudaSuccess)
        e = cudaGetLastError();
    if (e == cudaSuccess)
        count_launches(1);
    return e;
}

}  // namespace ts
