// Backward pass of the block-sparse attention (attn.cu): dQ, dK, dV from
// Q, K, V, O, dO and the forward's log-sum-exp.
//
// Mathematics, per (b, h), on the kept real (query t, key u) pairs:
//   P = exp2(scale log2e S - lse2),  S = Q K^T           (computed again)
//   dP = dO V^T,  dS = P (dP - delta),  delta_t = dO_t . O_t
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K
//
// Two passes over the pairs, one that keeps a query tile in place and sums dQ
// over its kept key blocks, then one that keeps a key tile in place and sums
// dK and dV over the query blocks that keep it.  S and dP are formed in both:
// the other way, one pass, adds dQ up in memory by atomics, whose order would
// change the result's bits, or stores dS (32 KB a pair of blocks).  Every sum
// here runs in one CTA in list order.
//
// delta.  dP - delta cancels where a softmax is concentrated, and dO . O from
// the bf16 O is then too coarse: with scores of standard deviation 3 the
// gradients' error against 64 bits was 1.7 times that of rounding the result
// (1.41 is the rounding of dS and the result).  The query pass therefore
// starts from delta0 = dO . O and sums the exact delta_t = sum_u P_tu dP_tu
// on the way, which the key pass reads.  Its own dQ is put right at the end,
//   dQ = scale (sum_u dS0_tu k_u - (delta - delta0) sum_u P_tu k_u),
// with a product more, in the tiles that need it.  delta0's error is about
// 2^-9 |dO| |O| / sqrt(3 D) and dP_tu - delta_t = dO_t . (v_u - O_t) about
// |dO| |v_u - O| / sqrt(D), so that it adds |O| / min_u |v_u - O| roundings to
// the result at most.  Tiles with a row of |O|^2 > GRAD_EXACT min |v_u|^2, u
// the tokens of the tile's listed blocks, take the product.  With 1/16,
// |v_u - O| >= 3 |O| in the others, and their error is at most
// sqrt(2 + 1/9) = 1.45 roundings.  (The head's mean |v|^2 in the minimum's
// place let a few large values, even of blocks that no list holds, turn the
// product off where the softmax was concentrated: 2.3 to 3.1 roundings a row at
// scores of standard deviation 3.)
//
// Both passes are one kernel, grad_kernel<D, KV>, one CTA of 640 threads per
// SM (it holds all 512 tensor-memory columns):
//   warp 0      producer: takes items, TMA-loads the item's own tile pair
//               (KV: K and V; else Q and dO), streams the first tensor of the
//               other side (KV: Q; else K) in chunks of 128 rows and writes
//               each chunk's masks
//   warp 2      producer of the other streamed tensor (KV: dO; else V)
//   warps 1, 3  issue the MMAs
//   warps 4..19 four groups of four warps; a thread has one row of the
//               128-row tile and a quarter of the chunk's 128 columns: P and dS
//               are formed from the fp32 S and dP in tensor memory and go
//               back there as bf16, where they are the A operand of the
//               accumulating products
// KV: rows are keys, columns queries (S^T, dP^T); columns' statistics come
// with the stream.  Else rows are queries with their statistics in registers.
// Per chunk i, in tensor memory (all 512 columns):
//   S(i) -> P(i) over it, A0 += P(i) B;   dP(i) -> dS(i) over it, A1 += dS(i) B0
// with KV: A0 = dV (B = dO), A1 = dK; else A0 = sum P k (B = B0), A1 = dQ.  A
// query tile without A0 has a second dP buffer in its place, and S(i + 1) and
// dP(i + 1) run ahead of the arithmetic.
//
// bs < 128: as in the forward, a tile holds G = 128 / bs consecutive blocks
// and walks the union of their lists; a chunk packs 128 / bs listed blocks and
// each row sees only the columns of blocks that its own block is paired with.
//
// What bounds it.  A 720p layer (40 heads, 13.8 million pairs of 128-token
// blocks, D = 128) takes 321 to 330 ms by the board: 902 TFLOP/s counted as five products,
// 1264 as the seven that run, 92% of what a large matrix product sustains under the
// board's power limit (1368); the clock settles at 1.7 GHz and falls when the
// pipe is kept busier, so a form with 10% fewer clocks a chunk (P and dS both
// over dP, S free at once) took the same time.  Steps at 480p, 4 heads: one
// issuing lane, descriptors put together at each use 9.5 ms; masks out of the
// common body, two issuers 9.0 (with the exact delta's product); that product
// where it is needed only, dP double buffered 7.75; four warpgroups of
// arithmetic instead of two 7.7 (blocks of 64: 1.31 to 1.10 ms); issuers from
// uniform registers 7.1 to 7.5 (by the board).  Rows that see none of a chunk's
// columns skip its arithmetic: 344 to 275 us for lists of 5% of 448 blocks of 32.
#include <cuda.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "fvattn_train.h"
#include "ptx.cuh"
#include "sync.cuh"
#include "tmap.cuh"

namespace fv {

constexpr int GRAD_GROUPS = 4;    // warpgroups of arithmetic, 32 columns of a chunk each
constexpr int GRAD_WARPS = 4 * GRAD_GROUPS;
constexpr int GRAD_THREADS = 128 * (1 + GRAD_GROUPS);
// The first streamed tensor is held from S to the last product of its chunk,
// over one and a half chunks' time: a stage more.
constexpr int GRAD_STAGES0 = 3, GRAD_STAGES1 = 2;
constexpr uint32_t GRAD_TMEM = 512;
constexpr float GRAD_EXACT = 1.f / 16.f;
// An entry of the work order: tile | its list's length << 12 | GRAD_FLAG if it is a query tile that needs the
// exact delta (at most 2560 blocks: 12 bits each).
constexpr int GRAD_FLAG = 1 << 30;
constexpr int GRAD_GROUP = 8;     // blocks per tile at bs = 16
// Register split (setmaxnreg): the launch gives 96 a thread; one warpgroup
// of producers and issuers at LOW, the arithmetic at HIGH.
constexpr int GRAD_LAUNCH_REGS = 96, GRAD_LOW = 64, GRAD_HIGH = 104;
static_assert(128 * (GRAD_LOW + GRAD_GROUPS * GRAD_HIGH) <= GRAD_THREADS * GRAD_LAUNCH_REGS, "register split");

// Tensor-memory columns: S (P over it), dP (dS over it), the two accumulators.
constexpr uint32_t T_S = 0, T_DP = 128, T_A0 = 256, T_A1 = 384;

struct GradArgs {
    Geo g;
    int G, ngroups;
    const uint32_t* ul;       // [B*H][ngroups][nb] this pass's lists: block | membership bits << 24
    const int32_t* order;     // [B*H][ngroups] a head's tiles, longest list first
    int* counter;
    const int32_t* ext;       // [nb] real extent of each block
    const float* nlse2;       // [B*H][Npad] -lse * log2(e); -inf for rows that take no part
    float* ndelta;            // [B*H][Npad] -delta: read by KV; else -delta0, replaced by the exact one
    __nv_bfloat16* out0;      // KV: dV; else dQ
    __nv_bfloat16* out1;      // KV: dK
    float scale, scale_log2;
    int total_items;
    int oob_row;              // a row index past the end of every operand (reads as zero)
    unsigned long long wait_limit_ns;
};

struct __align__(16) GradCtrl {
    // KV: the chunks' column statistics, -lse2 of the first ring's stages and then -delta of the second's.
    // Else: each column group's sum of P dP by row
    float stat[GRAD_STAGES0 + GRAD_STAGES1][128];
    uint32_t mask[GRAD_STAGES0][8];                              // 4 words of columns that are tokens, then a
                                                                 // byte a slot: blocks of the tile paired with it
    unsigned long long a_full, a_empty;                          // the item's own tile pair
    unsigned long long b0_full[GRAD_STAGES0], b0_empty[GRAD_STAGES0];
    unsigned long long b1_full[GRAD_STAGES1], b1_empty[GRAD_STAGES1];
    unsigned long long s_full[2], dp_full[2], ds_full[2];        // by the chunk's parity: their waiters may lag by one
    unsigned long long p_full[2];                                // by the piece; without A0 both say that S has been read
    unsigned long long sum_full;
    unsigned long long acc_full, acc_free;
    unsigned long long item_full[2], item_empty[2];
    unsigned long long drain[2];
    int item[2][4];            // bh, tile, list length, 0: end, 1: without A0, 2: with A0
    uint32_t tmem_base;
    int abort_flag;
};

template <int D>
struct GradSmem {
    static constexpr uint32_t TILE = 128u * D * 2u;
    static constexpr uint32_t A0 = 0, A1 = TILE, B0 = 2 * TILE, B1 = B0 + GRAD_STAGES0 * TILE;
    static constexpr uint32_t CTRL = B1 + GRAD_STAGES1 * TILE;
    static constexpr uint32_t TOTAL = CTRL + static_cast<uint32_t>(sizeof(GradCtrl));
    // at least 120 KB, so that two CTAs never share an SM's tensor memory
    static constexpr uint32_t ALLOC = TOTAL > 120u * 1024u ? TOTAL : 120u * 1024u;
    static_assert(ALLOC <= 232448u, "shared-memory layout too large");
};

// Real extent of a block, packed nf | ny << 8 | nx << 16.
__device__ __forceinline__ int grad_extent(const Geo& g, int block) {
    block = tile_of_block(g, block);
    const int bx = block % g.nbx;
    const int rest = block / g.nbx;
    const int by = rest % g.nby;
    const int bf = rest / g.nby;
    return min(g.tf, g.F - bf * g.tf) | (min(g.th, g.Hs - by * g.th) << 8) | (min(g.tw, g.Ws - bx * g.tw) << 16);
}

// One slot of a chunk: its block (-1: none) and membership bits.
__device__ __forceinline__ int grad_slot(const uint32_t* ul, int e, int cnt, uint32_t& mem) {
    mem = 0u;
    if (e >= cnt) return -1;
    const uint32_t v = ul[e];
    mem = v >> 24;
    return static_cast<int>(v & 0xFFFFFFu);
}

// Columns 32 w .. of a chunk that a row of the tile's block tb sees: those of
// slots whose block is paired with tb, and tokens (unless `all`).  lbs =
// log2(bs).
__device__ __forceinline__ uint32_t grad_mask(const uint32_t* m, int lbs, int tb, int w, bool all) {
    const uint32_t pad = m[w];
    const uint2 by = *reinterpret_cast<const uint2*>(m + 4);
    const unsigned long long mem = ((static_cast<unsigned long long>(by.y) << 32) | by.x) >> tb;
    const uint32_t lo = static_cast<uint32_t>(mem >> (8 * ((w * 32) >> lbs))) & 1u;
    const uint32_t hi = static_cast<uint32_t>(mem >> (8 * ((w * 32 + 16) >> lbs))) & 1u;   // another slot at bs = 16
    const uint32_t mw = (lo ? 0x0000FFFFu : 0u) | (hi ? 0xFFFF0000u : 0u);
    return all ? mw : mw & pad;
}

// Which of a chunk's columns a warp's rows see: the arithmetic's three bodies.
enum GradColumns { ALL, SOME, NOTHING };
template <GradColumns C>
using Body = std::integral_constant<GradColumns, C>;

template <int D, bool KV>
__global__ void __launch_bounds__(GRAD_THREADS, 1)
    grad_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1, const GradArgs a) {
    using L = GradSmem<D>;
    constexpr int NS0 = GRAD_STAGES0, NS1 = GRAD_STAGES1;
    extern __shared__ __align__(1024) unsigned char smem[];
    if (smem_u32(smem) & 1023u) {   // the 128-byte swizzle needs 1024-byte aligned tiles
        pdl_wait();
        if (threadIdx.x == 0) record_status(FVATTN_ERR_UNSUPPORTED);
        return;
    }
    GradCtrl& ctl = *reinterpret_cast<GradCtrl*>(smem + L::CTRL);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const Geo& g = a.g;
    const int bs = g.bs;
    const int bpc = 128 / bs, lbs = 31 - __clz(bs);
    volatile int* abort_flag = &ctl.abort_flag;
    const unsigned long long wlim = a.wait_limit_ns;

    {   // rows that no load of the first item fills must be finite
        uint4* z = reinterpret_cast<uint4*>(smem);
        for (uint32_t i = threadIdx.x; i < L::CTRL / 16u; i += GRAD_THREADS) z[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&ctl.a_full), 1);
        mbar_init(smem_u32(&ctl.a_empty), 2);
        for (int s = 0; s < NS0; ++s) {
            mbar_init(smem_u32(&ctl.b0_full[s]), 1);
            mbar_init(smem_u32(&ctl.b0_empty[s]), (KV ? 1 : 2) + GRAD_WARPS);   // commits of its last products, the arithmetic
        }
        for (int s = 0; s < NS1; ++s) {
            mbar_init(smem_u32(&ctl.b1_full[s]), 1);
            mbar_init(smem_u32(&ctl.b1_empty[s]), KV ? 1 + GRAD_WARPS : 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&ctl.s_full[s]), 1);
            mbar_init(smem_u32(&ctl.dp_full[s]), 1);
            mbar_init(smem_u32(&ctl.p_full[s]), GRAD_WARPS);
            mbar_init(smem_u32(&ctl.ds_full[s]), GRAD_WARPS);
            mbar_init(smem_u32(&ctl.item_full[s]), 1);
            mbar_init(smem_u32(&ctl.item_empty[s]), 2 + 1 + GRAD_WARPS);   // issuers, second producer, arithmetic
        }
        mbar_init(smem_u32(&ctl.sum_full), GRAD_WARPS);
        mbar_init(smem_u32(&ctl.acc_full), 2);
        mbar_init(smem_u32(&ctl.acc_free), GRAD_WARPS);
        for (int s = 0; s < 2; ++s) mbar_init(smem_u32(&ctl.drain[s]), 1);
        ctl.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmA0);
        prefetch_tmap(&tmA1);
        prefetch_tmap(&tmB0);
        prefetch_tmap(&tmB1);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&ctl.tmem_base), GRAD_TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem_base;
    pdl_wait();              // the lists, the statistics, and for KV the query pass's delta
    pdl_launch_dependents();

    if (warp >= 4) {
        regs_inc<GRAD_HIGH>();
        // =========================== arithmetic: P, dS, epilogue
        const int w = (warp - 4) >> 2;              // columns 32 w ..
        const int quad = warp & 3;
        const int row = quad * 32 + lane;
        const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const uint32_t sbuf = trow + T_S + static_cast<uint32_t>(w) * 32u;
        const int tb = row / bs;                    // this row's block in the tile
        const unsigned long long sl2x2 = f2_pack(a.scale_log2, a.scale_log2);
        int item_seq = 0;
        uint32_t n_seq = 0;     // items with at least one chunk
        uint32_t c = 0;         // chunks
        bool ok = true;
        while (ok) {
            const int slot = item_seq & 1;
            if (!wait_warp(smem_u32(&ctl.item_full[slot]), (item_seq >> 1) & 1, abort_flag, wlim)) break;
            const int bh = ctl.item[slot][0];
            const int u = ctl.item[slot][1];
            const int cnt = ctl.item[slot][2];
            const int kind = ctl.item[slot][3];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl.item_empty[slot]));
            if (!kind) break;
            const bool two = KV || kind == 2;
            const int nc = (cnt + bpc - 1) / bpc;
            const int blk0 = u * a.G;
            const bool in_tile = row < min(a.G, g.nb - blk0) * bs;
            const long long grow = static_cast<long long>(bh) * g.Npad + static_cast<long long>(blk0) * bs + row;
            // KV: whether this key row is a token.  Else: the query row's statistics (-inf takes P to 0).
            bool live = in_tile;
            unsigned long long nl2 = 0ull, nd2 = 0ull;
            float nd = 0.f;
            unsigned long long sum2 = 0ull;             // sum of P dP: two partial sums
            // Padding keys are zero rows of K and V: their P, exp2(-lse2), multiplies zeros wherever it
            // goes, and needs a mask only where it could overflow.
            bool all = true;
            if (KV) {
                int f_, y_, x_;
                live = live && token_of_pos(g, static_cast<long long>(blk0) * bs + row, f_, y_, x_);
            } else {
                const float nl = in_tile ? a.nlse2[grow] : -INFINITY;
                if (in_tile) nd = a.ndelta[grow];
                live = nl != -INFINITY;
                nl2 = f2_pack(nl, nl);
                nd2 = f2_pack(nd, nd);
                all = __all_sync(0xffffffffu, !(nl > 60.f));
            }
            for (int i = 0; i < nc; ++i, ++c) {
                const uint32_t st0 = c % NS0, st1 = c % NS1, par = c & 1, ph = (c >> 1) & 1;
                const uint32_t dpbuf = trow + (!two && (i & 1) ? T_A0 : T_DP) + static_cast<uint32_t>(w) * 32u;
                if (!wait_warp2(smem_u32(&ctl.b0_full[st0]), (c / NS0) & 1, smem_u32(&ctl.s_full[par]), ph, abort_flag,
                                wlim)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t pv[32];                    // S, then P, of this row
                tmem_ld32(sbuf, pv);
                uint32_t mw = grad_mask(ctl.mask[st0], lbs, tb, w, all);   // columns that the row sees
                const bool full = __all_sync(0xffffffffu, mw == 0xFFFFFFFFu), none = __all_sync(0xffffffffu, mw == 0u);
                tmem_wait_ld();
                // The chunk's arithmetic is there without masks, with a select an element, and for rows that see
                // none of its columns (with blocks of 32 or more one of the first and last holds for a whole
                // warp).  One body that tests for masks on the way took twice the time, masks or not.
                auto chunk = [&](auto body, auto with_a0) {
                    constexpr bool FULL = decltype(body)::value == ALL, NONE = decltype(body)::value == NOTHING;
                    constexpr bool TWO = decltype(with_a0)::value;
                    // several bodies for the compiler too, which else moves the loads of all before the branch
                    if constexpr (FULL)
                        asm volatile("// every column" ::: "memory");
                    else if constexpr (NONE)
                        asm volatile("// no column" ::: "memory");
                    else
                        asm volatile("// masks" ::: "memory");
                    if constexpr (!TWO) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(smem_u32(&ctl.p_full[0]));
                            mbar_arrive(smem_u32(&ctl.p_full[1]));
                            mbar_arrive(smem_u32(&ctl.b0_empty[st0]));
                        }
                    }
                    const ulonglong2* nls = reinterpret_cast<const ulonglong2*>(&ctl.stat[st0][w * 32]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {   // P over S, for half of its product
                        uint32_t pk[8];
#pragma unroll
                        for (int e = h * 16; e < h * 16 + 16; e += 4) {
                            ulonglong2 add = make_ulonglong2(nl2, nl2);
                            if (KV) add = nls[e >> 2];
#pragma unroll
                            for (int z = 0; z < 4; z += 2) {
                                float x0 = 0.f, x1 = 0.f;
                                if (!NONE) {
                                    f2_unpack(f2_fma(f2_pack(__uint_as_float(pv[e + z]), __uint_as_float(pv[e + z + 1])),
                                                     sl2x2, z ? add.y : add.x), x0, x1);
                                    x0 = ex2_approx(x0);
                                    x1 = ex2_approx(x1);
                                }
                                if (!FULL && !NONE) {
                                    x0 = (mw & (1u << (e + z))) ? x0 : 0.f;
                                    x1 = (mw & (1u << (e + z + 1))) ? x1 : 0.f;
                                }
                                pv[e + z] = __float_as_uint(x0);
                                pv[e + z + 1] = __float_as_uint(x1);
                                if (TWO) pk[((e + z) >> 1) & 7] = pack_bf16x2(x0, x1);
                            }
                        }
                        if constexpr (TWO) {
                            tmem_st8(sbuf + h * 8u, pk);
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) {
                                mbar_arrive(smem_u32(&ctl.p_full[h]));
                                if (h == 1) mbar_arrive(smem_u32(&ctl.b0_empty[st0]));
                            }
                        }
                    }
                    if (KV) {
                        if (!wait_warp2(smem_u32(&ctl.b1_full[st1]), (c / NS1) & 1, smem_u32(&ctl.dp_full[par]), ph,
                                        abort_flag, wlim))
                            return false;
                    } else if (!wait_warp(smem_u32(&ctl.dp_full[par]), ph, abort_flag, wlim)) {
                        return false;
                    }
                    tc_fence_after();
                    uint32_t dv[32], ds[16];
                    if (!NONE) {
                        tmem_ld32(dpbuf, dv);
                        tmem_wait_ld();
                    }
                    // (the bits' tests are made again: kept from above they would take 32 registers)
                    if (!FULL) asm volatile("" : "+r"(mw));
                    const ulonglong2* nds = reinterpret_cast<const ulonglong2*>(&ctl.stat[NS0 + st1][w * 32]);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        ulonglong2 add = make_ulonglong2(nd2, nd2);
                        if (KV) add = nds[e >> 2];
#pragma unroll
                        for (int z = 0; z < 4; z += 2) {
                            if (NONE) {
                                ds[(e + z) >> 1] = 0u;
                                continue;
                            }
                            float x0 = __uint_as_float(dv[e + z]), x1 = __uint_as_float(dv[e + z + 1]);
                            if (!FULL && !KV) {   // nothing of a masked pair enters the sum
                                x0 = (mw & (1u << (e + z))) ? x0 : 0.f;
                                x1 = (mw & (1u << (e + z + 1))) ? x1 : 0.f;
                            }
                            const unsigned long long dp2 = f2_pack(x0, x1);
                            const unsigned long long p2 = f2_pack(__uint_as_float(pv[e + z]), __uint_as_float(pv[e + z + 1]));
                            if (!KV) sum2 = f2_fma(p2, dp2, sum2);
                            f2_unpack(f2_mul(f2_add(dp2, z ? add.y : add.x), p2), x0, x1);
                            if (!FULL && KV) {    // 0 whatever dP and the column's statistics hold
                                x0 = (mw & (1u << (e + z))) ? x0 : 0.f;
                                x1 = (mw & (1u << (e + z + 1))) ? x1 : 0.f;
                            }
                            ds[(e + z) >> 1] = pack_bf16x2(x0, x1);
                        }
                    }
                    tmem_st16(dpbuf, ds);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&ctl.ds_full[par]));
                        if (KV) mbar_arrive(smem_u32(&ctl.b1_empty[st1]));
                    }
                    return true;
                };
                auto either = [&](auto with_a0) {
                    return full   ? chunk(Body<ALL>{}, with_a0)
                           : none ? chunk(Body<NOTHING>{}, with_a0)
                                  : chunk(Body<SOME>{}, with_a0);
                };
                if (two)
                    ok = either(std::true_type{});
                else if constexpr (!KV)
                    ok = either(std::false_type{});
                if (!ok) break;
            }
            if (!ok) break;
            // ---- epilogue.  KV: groups 0 and 1 write a half of dV each, 2 and 3 of dK; else each a quarter of dQ.
            float fix = 0.f;     // delta0 - delta
            if (nc > 0) {
                if (!KV) {
                    float s0, s1;
                    f2_unpack(sum2, s0, s1);
                    // the sums of the item before have been read
                    if (n_seq > 0 && !wait_warp(smem_u32(&ctl.acc_free), (n_seq - 1) & 1, abort_flag, wlim)) break;
                    ctl.stat[w][row] = s0 + s1;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&ctl.sum_full));
                    if (!wait_warp(smem_u32(&ctl.sum_full), n_seq & 1, abort_flag, wlim)) break;
                    const float nd1 = -((ctl.stat[0][row] + ctl.stat[1][row]) + (ctl.stat[2][row] + ctl.stat[3][row]));
                    fix = nd1 - nd;
                    if (live && w == 0) a.ndelta[grow] = nd1;
                }
                if (!wait_warp(smem_u32(&ctl.acc_full), n_seq & 1, abort_flag, wlim)) break;
                tc_fence_after();
            }
            const bool first_out = KV && w < 2;
            const float f = first_out ? 1.f : a.scale;
            __nv_bfloat16* dst = (KV && !first_out ? a.out1 : a.out0) + grow * D;
            const uint32_t acc = trow + (first_out ? T_A0 : T_A1);
            constexpr int COLS = KV ? D / 2 : D / 4;       // of a thread
            constexpr int STEP = COLS < 32 ? COLS : 32;
#pragma unroll 1
            for (int q = 0; q < COLS / STEP; ++q) {
                const uint32_t col = static_cast<uint32_t>(KV ? w & 1 : w) * COLS + q * STEP;
                uint32_t r[STEP];
                if (nc > 0) {   // (rows that take no part may hold anything: they get zero)
                    tmem_ld(acc + col, r);
                    if (!KV && two) {
                        uint32_t pk[STEP];
                        tmem_ld(trow + T_A0 + col, pk);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < STEP; ++e)
                            r[e] = __float_as_uint(fmaf(fix, __uint_as_float(pk[e]), __uint_as_float(r[e])));
                    } else {
                        tmem_wait_ld();
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < STEP; ++e) r[e] = 0u;
                }
                if (in_tile) {
#pragma unroll
                    for (int v8 = 0; v8 < STEP / 8; ++v8) {
                        uint32_t o[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            o[k] = live ? pack_bf16x2(__uint_as_float(r[v8 * 8 + 2 * k]) * f,
                                                      __uint_as_float(r[v8 * 8 + 2 * k + 1]) * f)
                                        : 0u;
                        *reinterpret_cast<uint4*>(dst + col + v8 * 8) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
            }
            if (nc > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl.acc_free));
                ++n_seq;
            }
            ++item_seq;
        }
    } else {
        regs_dec<GRAD_LOW>();
        if (warp == 0) {
            // =========================== producer: items, own tiles, first streamed tensor, masks
            int c_slot[4], c_of[4], c_oy[4], c_ox[4];   // column q*32 + lane of a chunk
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int col = q * 32 + lane;
                c_slot[q] = col / bs;
                const int off = col - c_slot[q] * bs;
                c_ox[q] = off % g.tw;
                c_oy[q] = (off / g.tw) % g.th;
                c_of[q] = off / (g.tw * g.th);
            }
            int item_seq = 0;
            uint32_t n_seq = 0, c = 0;
            bool ok = true;
            while (ok) {
                const int slot = item_seq & 1;
                if (!wait_warp(smem_u32(&ctl.item_empty[slot]), ((item_seq >> 1) & 1) ^ 1, abort_flag, wlim)) break;
                int t = static_cast<int>(blockIdx.x);          // the first; then the next that nobody has taken
                if (item_seq > 0) {
                    if (lane == 0) t = atomicAdd(a.counter, 1) + static_cast<int>(gridDim.x);
                    t = __shfl_sync(0xffffffffu, t, 0);
                }
                if (t >= a.total_items) {
                    if (lane == 0) {
                        ctl.item[slot][3] = 0;
                        mbar_arrive(smem_u32(&ctl.item_full[slot]));
                    }
                    break;
                }
                const int bh = t / a.ngroups;
                const int entry = a.order[t];
                const int u = entry & 0xFFF, cnt = (entry >> 12) & 0xFFF;
                const long long unit = static_cast<long long>(bh) * a.ngroups + u;
                if (lane == 0) {
                    ctl.item[slot][0] = bh;
                    ctl.item[slot][1] = u;
                    ctl.item[slot][2] = cnt;
                    ctl.item[slot][3] = KV || (entry & GRAD_FLAG) ? 2 : 1;
                    mbar_arrive(smem_u32(&ctl.item_full[slot]));
                }
                ++item_seq;
                const int nc = (cnt + bpc - 1) / bpc;
                if (nc == 0) continue;
                const int blk0 = u * a.G;
                const int nq = min(a.G, g.nb - blk0);
                const int row_base = bh * static_cast<int>(g.Npad);
                if (!wait_warp(smem_u32(&ctl.a_empty), (n_seq & 1) ^ 1, abort_flag, wlim)) break;
                ++n_seq;
                if (lane == 0) mbar_arrive_expect_tx(smem_u32(&ctl.a_full), static_cast<uint32_t>(2 * nq * bs * D * 2));
                __syncwarp();
                if (lane < nq) {
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) {
                        const uint32_t off = h * 16384u + static_cast<uint32_t>(lane * bs) * 128u;
                        tma_load_2d(sbase + L::A0 + off, &tmA0, h * 64, row_base + (blk0 + lane) * bs, smem_u32(&ctl.a_full));
                        tma_load_2d(sbase + L::A1 + off, &tmA1, h * 64, row_base + (blk0 + lane) * bs, smem_u32(&ctl.a_full));
                    }
                }
                const uint32_t* ul = a.ul + unit * g.nb;
                // a chunk's blocks, membership bits and real extents are looked up a chunk ahead
                uint32_t m_next = 0u;
                int j_next = lane < bpc ? grad_slot(ul, lane, cnt, m_next) : -1;
                int e_next = !KV && j_next >= 0 ? a.ext[j_next] : 0;
                for (int i = 0; i < nc; ++i, ++c) {
                    const int st = c % NS0;
                    const uint32_t mem = m_next;
                    const int j = j_next, ext = e_next;
                    if (i + 1 < nc) {
                        j_next = lane < bpc ? grad_slot(ul, (i + 1) * bpc + lane, cnt, m_next) : -1;
                        e_next = !KV && j_next >= 0 ? a.ext[j_next] : 0;
                    }
                    if (!wait_warp(smem_u32(&ctl.b0_empty[st]), ((c / NS0) & 1) ^ 1, abort_flag, wlim)) {
                        ok = false;
                        break;
                    }
                    // columns that are tokens (query rows take no part through their statistics), and which
                    // blocks of the tile each slot's block is paired with
                    uint32_t pad[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int e = __shfl_sync(0xffffffffu, ext, c_slot[q]);
                        pad[q] = KV ? 0xFFFFFFFFu
                                    : __ballot_sync(0xffffffffu, (c_of[q] < (e & 255)) && (c_oy[q] < ((e >> 8) & 255)) &&
                                                                     (c_ox[q] < (e >> 16)));
                    }
                    const uint32_t byte = mem << (8 * (lane & 3));
                    const uint32_t m0 = __reduce_or_sync(0xffffffffu, lane < 4 ? byte : 0u);
                    const uint32_t m1 = __reduce_or_sync(0xffffffffu, lane >= 4 && lane < 8 ? byte : 0u);
                    if (lane == 0) {
                        *reinterpret_cast<uint4*>(&ctl.mask[st][0]) = make_uint4(pad[0], pad[1], pad[2], pad[3]);
                        *reinterpret_cast<uint2*>(&ctl.mask[st][4]) = make_uint2(m0, m1);
                    }
                    const uint32_t bar = smem_u32(&ctl.b0_full[st]);
                    const int nblk = min(bpc, cnt - i * bpc);
                    if (lane == 0)
                        mbar_arrive_expect_tx(bar, L::TILE + (KV ? static_cast<uint32_t>(nblk * bs * 4) : 0u));
                    __syncwarp();
                    if (lane < bpc) {
                        // a slot without a block is filled with zeros (a row past the end): P is 0 there, and
                        // 0 times what an earlier chunk left could be NaN
                        const int r = j >= 0 ? row_base + j * bs : a.oob_row;
                        const uint32_t dst = sbase + L::B0 + st * L::TILE + static_cast<uint32_t>(lane * bs) * 128u;
#pragma unroll
                        for (int h = 0; h < D / 64; ++h) tma_load_2d(dst + h * 16384u, &tmB0, h * 64, r, bar);
                        if (KV && j >= 0)
                            bulk_load(smem_u32(&ctl.stat[st][lane * bs]), a.nlse2 + r, static_cast<uint32_t>(bs * 4), bar);
                    }
                }
            }
            if (lane == 0) {   // no copy into shared memory outlives the CTA
                if (n_seq > 0) wait_bar_drain(smem_u32(&ctl.a_full), (n_seq - 1) & 1, wlim);
                for (int st = 0; st < NS0; ++st) {
                    const uint32_t fills = c > static_cast<uint32_t>(st) ? (c - st + NS0 - 1) / NS0 : 0u;
                    if (fills > 0) wait_bar_drain(smem_u32(&ctl.b0_full[st]), (fills - 1) & 1, wlim);
                }
            }
            __syncwarp();
        } else if (warp == 2) {
            // =========================== producer of the second streamed tensor
            int item_seq = 0;
            uint32_t c = 0;
            bool ok = true;
            while (ok) {
                const int slot = item_seq & 1;
                if (!wait_warp(smem_u32(&ctl.item_full[slot]), (item_seq >> 1) & 1, abort_flag, wlim)) break;
                const int bh = ctl.item[slot][0];
                const int u = ctl.item[slot][1];
                const int cnt = ctl.item[slot][2];
                const int valid = ctl.item[slot][3];
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl.item_empty[slot]));
                if (!valid) break;
                ++item_seq;
                const int nc = (cnt + bpc - 1) / bpc;
                const int row_base = bh * static_cast<int>(g.Npad);
                const uint32_t* ul = a.ul + (static_cast<long long>(bh) * a.ngroups + u) * g.nb;
                uint32_t mem = 0u;
                int j_next = lane < bpc ? grad_slot(ul, lane, cnt, mem) : -1;
                for (int i = 0; i < nc; ++i, ++c) {
                    const int st = c % NS1;
                    const int j = j_next;
                    if (i + 1 < nc) j_next = lane < bpc ? grad_slot(ul, (i + 1) * bpc + lane, cnt, mem) : -1;
                    if (!wait_warp(smem_u32(&ctl.b1_empty[st]), ((c / NS1) & 1) ^ 1, abort_flag, wlim)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_u32(&ctl.b1_full[st]);
                    const int nblk = min(bpc, cnt - i * bpc);
                    if (lane == 0)
                        mbar_arrive_expect_tx(bar, L::TILE + (KV ? static_cast<uint32_t>(nblk * bs * 4) : 0u));
                    __syncwarp();
                    if (lane < bpc) {
                        const int r = j >= 0 ? row_base + j * bs : a.oob_row;
                        const uint32_t dst = sbase + L::B1 + st * L::TILE + static_cast<uint32_t>(lane * bs) * 128u;
#pragma unroll
                        for (int h = 0; h < D / 64; ++h) tma_load_2d(dst + h * 16384u, &tmB1, h * 64, r, bar);
                        if (KV && j >= 0)
                            bulk_load(smem_u32(&ctl.stat[NS0 + st][lane * bs]), a.ndelta + r, static_cast<uint32_t>(bs * 4), bar);
                    }
                }
            }
            if (lane == 0) {
                for (int st = 0; st < NS1; ++st) {
                    const uint32_t fills = c > static_cast<uint32_t>(st) ? (c - st + NS1 - 1) / NS1 : 0u;
                    if (fills > 0) wait_bar_drain(smem_u32(&ctl.b1_full[st]), (fills - 1) & 1, wlim);
                }
            }
            __syncwarp();
        } else {
            // =========================== MMA issuers (warps 1 and 3)
            // Warp 1: A0 += P(i-1) B, S(i).  Warp 3: A1 += dS(i-1) B0, dP(i).  In each the second product
            // overwrites columns that the first reads: one thread's MMAs keep their order.  While one
            // thread waits on its barriers the other's MMAs run; with a single issuer the pipe ran dry at
            // every wait (4200 clocks a chunk where its four products take 2048).  The exponentials wait for
            // A0 and S only, so warp 3 holds its products back until S(i) is done: 3400 to 3000 clocks.
            // The whole warp walks the loop, so that addresses and descriptors are warp-uniform values.
            {
                constexpr uint32_t ID_SS = idesc_bf16_f32(128, 128, false);
                constexpr uint32_t ID_ACC = idesc_bf16_f32(128, D, true);
                // A descriptor's upper half is one constant for all operands and the lower half holds the
                // address: one add an operand.
                constexpr uint32_t HI = (1024u >> 4) | (1u << 14) | (2u << 29);
                const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
                // C = own tile (A, K-major) x streamed chunk (B, K-major)
                auto product = [&](uint32_t d, uint32_t abase, uint32_t bbase) {
                    abase = (abase >> 4) | (1u << 16);
                    bbase = (bbase >> 4) | (1u << 16);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * 16384u + (kk & 3) * 32u) >> 4;
                            mma_bf16_ss(d, desc_of(abase + off, HI), desc_of(bbase + off, HI), ID_SS, kk > 0 ? 1u : 0u);
                        }
                    }
                    __syncwarp();
                };
                // acc += A (bf16 in tensor memory, the 32 columns of K of group z in 16 at 32 z) x chunk (B, its
                // 128 rows are K): the steps of one 16-column piece of each group
                auto accumulate = [&](uint32_t d, uint32_t abuf, uint32_t bbase, uint32_t piece, bool first) {
                    bbase = (bbase >> 4) | ((16384u >> 4) << 16);
                    if (elect_one()) {
#pragma unroll
                        for (uint32_t z = 0; z < 4; ++z)
                            mma_bf16_ts(d, abuf + z * 32u + piece * 8u,
                                        desc_of(bbase + (((z * 2u + piece) * 2048u) >> 4), HI), ID_ACC,
                                        (z > 0 || !first) ? 1u : 0u);
                    }
                    __syncwarp();
                };
                auto commit = [&](unsigned long long* bar) {
                    if (elect_one()) mma_commit(smem_u32(bar));
                    __syncwarp();
                };
                bool ok = true;
                auto need = [&](uint32_t bar, uint32_t parity) {
                    if (ok) ok = wait_warp(bar, parity, abort_flag, wlim);
                    return ok;
                };
                int item_seq = 0;
                uint32_t n_seq = 0, c = 0;
                const bool first_role = __shfl_sync(0xffffffffu, warp, 0) == 1;
                while (ok) {
                    const int slot = item_seq & 1;
                    if (!need(smem_u32(&ctl.item_full[slot]), (item_seq >> 1) & 1)) break;
                    const int kind = __shfl_sync(0xffffffffu, ctl.item[slot][3], 0);
                    const int cnt = __shfl_sync(0xffffffffu, ctl.item[slot][2], 0);
                    if (lane == 0) mbar_arrive(smem_u32(&ctl.item_empty[slot]));
                    if (!kind) break;
                    const bool two = KV || kind == 2;
                    ++item_seq;
                    const int nc = (cnt + bpc - 1) / bpc;
                    if (nc == 0) continue;
                    if (!need(smem_u32(&ctl.a_full), n_seq & 1)) break;
                    if (first_role) {
                        for (int i = 0; i <= nc; ++i, ++c) {
                            const uint32_t cp = c - 1;
                            const uint32_t st0 = c % NS0, sp = cp % (KV ? NS1 : NS0);
                            if (i < nc && !need(smem_u32(&ctl.b0_full[st0]), (c / NS0) & 1)) break;
                            if (two && i > 0) {
                                if (i == 1 && !need(smem_u32(&ctl.acc_free), (n_seq & 1) ^ 1)) break;
                                if (KV && !need(smem_u32(&ctl.b1_full[sp]), (cp / NS1) & 1)) break;
                                const uint32_t b = sbase + (KV ? L::B1 : L::B0) + sp * L::TILE;
#pragma unroll
                                for (uint32_t piece = 0; piece < 2; ++piece) {
                                    if (!need(smem_u32(&ctl.p_full[piece]), cp & 1)) break;
                                    tc_fence_after();
                                    accumulate(tm + T_A0, tm + T_S, b, piece, piece == 0 && i == 1);
                                }
                                if (!ok) break;
                                commit(KV ? &ctl.b1_empty[sp] : &ctl.b0_empty[sp]);
                            }
                            if (i == nc) break;
                            // S: the arithmetic has read the chunk before's (it may be another kind of item's)
                            if ((!two || i == 0) && c > 0 && !need(smem_u32(&ctl.p_full[0]), cp & 1)) break;
                            tc_fence_after();
                            product(tm + T_S, sbase + L::A0, sbase + L::B0 + st0 * L::TILE);
                            commit(&ctl.s_full[c & 1]);
                            if (!two) commit(&ctl.b0_empty[st0]);
                            if (i == nc - 1) commit(&ctl.a_empty);
                        }
                    } else {
                        for (int i = 0; i <= nc; ++i, ++c) {
                            const uint32_t cp = c - 1;
                            const uint32_t st1 = c % NS1, sp = cp % NS0;
                            if (i < nc && !need(smem_u32(&ctl.b1_full[st1]), (c / NS1) & 1)) break;
                            // the accumulators, and without A0 the second dP buffer in its columns
                            if (i == 1 && !need(smem_u32(&ctl.acc_free), (n_seq & 1) ^ 1)) break;
                            auto dp = [&]() {
                                tc_fence_after();
                                product(tm + (!two && (i & 1) ? T_A0 : T_DP), sbase + L::A1, sbase + L::B1 + st1 * L::TILE);
                                commit(&ctl.dp_full[c & 1]);
                                if (!KV) commit(&ctl.b1_empty[st1]);
                                if (i == nc - 1) commit(&ctl.a_empty);
                            };
                            if (!two && i < nc) dp();
                            if (i > 0) {
                                if (!need(smem_u32(&ctl.b0_full[sp]), (cp / NS0) & 1)) break;
                                if (!need(smem_u32(&ctl.ds_full[cp & 1]), (cp >> 1) & 1)) break;
                                if (two && i < nc && !need(smem_u32(&ctl.s_full[c & 1]), (c >> 1) & 1)) break;
                                tc_fence_after();
                                const uint32_t ds = tm + (!two && !(i & 1) ? T_A0 : T_DP);
                                const uint32_t b = sbase + L::B0 + sp * L::TILE;
                                accumulate(tm + T_A1, ds, b, 0, i == 1);
                                accumulate(tm + T_A1, ds, b, 1, false);
                                commit(&ctl.b0_empty[sp]);
                            }
                            if (i == nc) break;
                            if (two) dp();
                        }
                    }
                    if (!ok) break;
                    // Two arrivals an item.  Without A0 both are warp 3's: warp 1, which has no part in the
                    // accumulators then, may be an item of one chunk ahead, and its arrival for that one would
                    // count for this.
                    if (two || !first_role) commit(&ctl.acc_full);
                    if (!two && !first_role) commit(&ctl.acc_full);
                    ++n_seq;
                }
                // every MMA this thread issued has completed before the tensor memory is released
                commit(&ctl.drain[first_role ? 0 : 1]);
                wait_bar_drain(smem_u32(&ctl.drain[first_role ? 0 : 1]), 0, wlim);
            }
            __syncwarp();
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, GRAD_TMEM);
}

// ------------------------------------------------------------------ statistics, lists, work order

// First `stat_blocks` CTAs: -lse * log2(e) and -dO . O of every row (one warp
// per 8 rows; 16 bytes of O and dO a lane), the former -inf for padding rows
// and rows that keep no block, so that their P is 0; and for each 8 rows the
// largest |O|^2 and the least |v|^2 of a token (inf without one).  The others: one warp
// per (b, h, query block) writes its kv list as a bit row; those of the first
// head write the blocks' extents.
template <int D>
__global__ void __launch_bounds__(256) grad_prep_kernel(Geo g, int stat_blocks, int nwords,
                                                        const uint4* o, const uint4* dout, const uint4* v,
                                                        const float* lse, const int32_t* kv_idx, const int32_t* kv_cnt,
                                                        float* __restrict__ nlse2, float* __restrict__ ndelta,
                                                        float2* __restrict__ norms, uint32_t* __restrict__ bits,
                                                        int32_t* __restrict__ ext) {
    extern __shared__ uint32_t gp_bits[];   // [8][nwords]
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (static_cast<int>(blockIdx.x) < stat_blocks) {
        constexpr int LPR = D / 8;           // lanes a row
        constexpr int RPI = 32 / LPR;        // rows an iteration
        const long long rows = static_cast<long long>(g.B) * g.H * g.Npad;
        const long long row0 = (static_cast<long long>(blockIdx.x) * 8 + warp) * 8;
        if (row0 >= rows) return;
        uint4 x[8 / RPI], y[8 / RPI], z[8 / RPI];   // Npad is a multiple of 16: the 8 rows exist
#pragma unroll
        for (int i = 0; i < 8 / RPI; ++i) {
            const long long at = (row0 + i * RPI) * LPR + lane;
            x[i] = o[at];
            y[i] = dout[at];
            z[i] = v[at];
        }
        int f_, y_, x_;
        const bool token = lane < 8 && token_of_pos(g, (row0 + lane) % g.Npad, f_, y_, x_);
        const uint32_t tokens = __ballot_sync(0xffffffffu, token);
        float o2max = 0.f, v2min = INFINITY;
#pragma unroll
        for (int i = 0; i < 8 / RPI; ++i) {
            const uint32_t xa[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, ya[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
            const uint32_t za[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
            float s = 0.f, o2 = 0.f, v2 = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float x0 = __uint_as_float(xa[k] << 16), x1 = __uint_as_float(xa[k] & 0xFFFF0000u);
                const float z0 = __uint_as_float(za[k] << 16), z1 = __uint_as_float(za[k] & 0xFFFF0000u);
                s = fmaf(x0, __uint_as_float(ya[k] << 16), s);
                s = fmaf(x1, __uint_as_float(ya[k] & 0xFFFF0000u), s);
                o2 = fmaf(x0, x0, fmaf(x1, x1, o2));
                v2 = fmaf(z0, z0, fmaf(z1, z1, v2));
            }
#pragma unroll
            for (int d = LPR / 2; d > 0; d >>= 1) {
                s += __shfl_xor_sync(0xffffffffu, s, d);
                o2 += __shfl_xor_sync(0xffffffffu, o2, d);
                v2 += __shfl_xor_sync(0xffffffffu, v2, d);
            }
            o2max = fmaxf(o2max, o2);
            if ((tokens >> (i * RPI + lane / LPR)) & 1u) v2min = fminf(v2min, v2);
            if (lane % LPR == 0) ndelta[row0 + i * RPI + lane / LPR] = -s;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            o2max = fmaxf(o2max, __shfl_xor_sync(0xffffffffu, o2max, d));
            v2min = fminf(v2min, __shfl_xor_sync(0xffffffffu, v2min, d));
        }
        if (lane == 0) norms[row0 / 8] = make_float2(o2max, v2min);
        if (lane < 8) {
            const long long r = row0 + lane;
            const float l = lse[r];
            nlse2[r] = token && l != -INFINITY ? -l * 1.4426950408889634f : -INFINITY;
        }
        return;
    }
    const long long unit = (static_cast<long long>(blockIdx.x) - stat_blocks) * 8 + warp;
    if (unit >= static_cast<long long>(g.B) * g.H * g.nb) return;
    if (unit < g.nb && lane == 0) ext[unit] = grad_extent(g, static_cast<int>(unit));
    uint32_t* mine = gp_bits + warp * nwords;
    for (int i = lane; i < nwords; i += 32) mine[i] = 0u;
    __syncwarp();
    int cnt = kv_cnt[unit];
    if (cnt < 0 || cnt > g.nb) {
        if (lane == 0) record_status(FVATTN_ERR_BOUNDS);
        cnt = cnt < 0 ? 0 : g.nb;
    }
    const int32_t* list = kv_idx + unit * g.nb;
    for (int e = lane; e < cnt; e += 32) {
        const int j = list[e];
        if (j < 0 || j >= g.nb) {
            record_status(FVATTN_ERR_BOUNDS);
            continue;
        }
        if (atomicOr(&mine[j >> 5], 1u << (j & 31)) & (1u << (j & 31))) record_status(FVATTN_ERR_BOUNDS);
    }
    __syncwarp();
    for (int i = lane; i < nwords; i += 32) bits[unit * nwords + i] = mine[i];
}

// The blocks that a tile of G blocks is paired with, ascending, each with its
// membership bits above bit 24 (bit t: paired with the tile's block t); the
// list's length.  Direction 0: a query tile u and key blocks, from the rows of
// the bit matrix, with `least` the least of the listed blocks' vmin; 1 (keys):
// a key tile and query blocks, from its columns.  One warp.
__device__ __forceinline__ int grad_list(const Geo& g, int G, int nwords, const uint32_t* mat, bool keys,
                                         int u, const float* vmin, float& least, uint32_t* __restrict__ dst) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    least = INFINITY;
    if (!keys) {
        const int q0 = u * G, nq = min(G, g.nb - q0);
        for (int w0 = 0; w0 < nwords; w0 += 32) {
            uint32_t row[GRAD_GROUP];           // lane l has word w0 + l of the tile's rows
#pragma unroll
            for (int t = 0; t < GRAD_GROUP; ++t)
                row[t] = t < nq && w0 + lane < nwords ? mat[static_cast<long long>(q0 + t) * nwords + w0 + lane] : 0u;
            for (int k = 0; k < min(32, nwords - w0); ++k) {   // a word at a time, lane b its bit b
                uint32_t mem = 0u;
#pragma unroll
                for (int t = 0; t < GRAD_GROUP; ++t)
                    if (t < G) mem |= ((__shfl_sync(0xffffffffu, row[t], k) >> lane) & 1u) << t;
                const uint32_t any = __ballot_sync(0xffffffffu, mem != 0u);
                if (mem) {
                    const int j = (w0 + k) * 32 + lane;
                    dst[base + __popc(any & ((1u << lane) - 1u))] = static_cast<uint32_t>(j) | (mem << 24);
                    least = fminf(least, vmin[j]);
                }
                base += __popc(any);
            }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, d));
    } else {
        const int wd = (u * G) >> 5, sh = (u * G) & 31;   // G divides 32: one word holds the tile's columns
        const uint32_t ones = (1u << G) - 1u;
        for (int i0 = 0; i0 < g.nb; i0 += 32) {
            const int i = i0 + lane;
            const uint32_t mem = i < g.nb ? (mat[static_cast<long long>(i) * nwords + wd] >> sh) & ones : 0u;
            const uint32_t any = __ballot_sync(0xffffffffu, mem != 0u);
            if (mem) dst[base + __popc(any & ((1u << lane) - 1u))] = static_cast<uint32_t>(i) | (mem << 24);
            base += __popc(any);
        }
    }
    return base;
}

// One CTA per (direction, b, h): the lists of the head's tiles, and the tiles
// by list length, longest first (a counting sort; which of two equal tiles
// comes first changes only the schedule), query tiles that need the exact
// delta with GRAD_FLAG.  The first CTA of a direction resets its item counter.
constexpr int LISTS_THREADS = 1024;

__global__ void __launch_bounds__(LISTS_THREADS) grad_lists_kernel(Geo g, int G, int ngroups, int nwords,
                                                                   const uint32_t* bits, const float2* norms,
                                                                   uint32_t* __restrict__ ulq, uint32_t* __restrict__ ulk,
                                                                   int32_t* __restrict__ ordq, int32_t* __restrict__ ordk,
                                                                   int* __restrict__ counters) {
    const int BH = g.B * g.H, nb = g.nb;
    extern __shared__ int go_start[];   // [nb + 1], then by tile [ngroups] the lists' lengths, by block [nb] and by
                                        // tile [ngroups] the least |v|^2 and the largest |O|^2
    int* cnt = go_start + nb + 1;
    float* vmin = reinterpret_cast<float*>(cnt + ngroups);
    float* omax = vmin + nb;
    pdl_launch_dependents();
    pdl_wait();
    const int dir = static_cast<int>(blockIdx.x) / BH, bh = static_cast<int>(blockIdx.x) - dir * BH;
    const long long unit0 = static_cast<long long>(bh) * ngroups;
    int32_t* ord = (dir ? ordk : ordq) + unit0;
    if (bh == 0 && threadIdx.x == 0) counters[dir] = 0;
    if (dir == 0) {
        norms += static_cast<long long>(bh) * (g.Npad / 8);
        const int n = g.bs / 8;
        for (int i = threadIdx.x; i < nb; i += LISTS_THREADS) {
            float x = INFINITY;
            for (int k = 0; k < n; ++k) x = fminf(x, norms[i * n + k].y);
            vmin[i] = x;
        }
        for (int i = threadIdx.x; i < ngroups; i += LISTS_THREADS) {
            float x = 0.f;
            for (int k = i * G * n; k < min(i * G + G, nb) * n; ++k) x = fmaxf(x, norms[k].x);
            omax[i] = x;
        }
        __syncthreads();
    }
    for (int u = threadIdx.x >> 5; u < ngroups; u += LISTS_THREADS / 32) {
        float least;
        const int n = grad_list(g, G, nwords, bits + static_cast<long long>(bh) * nb * nwords, dir != 0, u, vmin, least,
                                (dir ? ulk : ulq) + (unit0 + u) * nb);
        // (in a list's length: whether its tile needs the exact delta)
        if ((threadIdx.x & 31) == 0) cnt[u] = n | (dir == 0 && !(omax[u] <= GRAD_EXACT * least) ? GRAD_FLAG : 0);
    }
    for (int i = threadIdx.x; i <= nb; i += blockDim.x) go_start[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < ngroups; i += blockDim.x) atomicAdd(&go_start[nb - (cnt[i] & ~GRAD_FLAG)], 1);
    __syncthreads();
    if (threadIdx.x < 32) {   // exclusive scan over descending lengths
        int base = 0;
        for (int i0 = 0; i0 <= nb; i0 += 32) {
            const int i = i0 + threadIdx.x;
            const int c = i <= nb ? go_start[i] : 0;
            int incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (static_cast<int>(threadIdx.x) >= o) incl += y;
            }
            if (i <= nb) go_start[i] = base + incl - c;
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ngroups; i += blockDim.x) {
        const int n = cnt[i] & ~GRAD_FLAG;
        ord[atomicAdd(&go_start[nb - n], 1)] = i | (n << 12) | (cnt[i] & GRAD_FLAG);
    }
}

// ------------------------------------------------------------------ host side

struct GradWs {
    size_t nlse2, ndelta, norms, bits, ulq, ulk, ordq, ordk, ext, counters, total;
    int G, ngroups, nwords;
};

static GradWs grad_ws(const fvattn_geom& g) {
    auto al = [](size_t x) { return (x + 255) / 256 * 256; };
    GradWs w;
    const size_t BH = static_cast<size_t>(g.B) * g.H, nb = static_cast<size_t>(g.nb);
    w.G = g.bs > 0 ? 128 / g.bs : 1;
    w.ngroups = (g.nb + w.G - 1) / w.G;
    w.nwords = (g.nb + 31) / 32;
    const size_t units = BH * w.ngroups;
    w.nlse2 = 0;
    w.ndelta = w.nlse2 + al(4 * BH * g.Npad);
    w.norms = w.ndelta + al(4 * BH * g.Npad);
    w.bits = w.norms + al(BH * g.Npad);
    w.ulq = w.bits + al(4 * BH * nb * w.nwords);
    w.ulk = w.ulq + al(4 * units * nb);
    w.ordq = w.ulk + al(4 * units * nb);
    w.ordk = w.ordq + al(4 * units);
    w.ext = w.ordk + al(4 * units);
    w.counters = w.ext + al(4 * nb);
    w.total = w.counters + 256;
    return w;
}

template <int D, bool KV>
static int launch_grad(const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b0, const CUtensorMap& b1,
                       const GradArgs& args, int grid, int dev, cudaStream_t s) {
    using L = GradSmem<D>;
    static std::atomic<unsigned long long> ready{0};   // devices on which the kernel has its shared memory
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if ((ready.load(std::memory_order_relaxed) & bit) == 0ull) {
        if (!cuda_ok(cudaFuncSetAttribute(grad_kernel<D, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          static_cast<int>(L::ALLOC))))
            return FVATTN_ERR_CUDA;
        // setmaxnreg waits for ever for registers that the CTA was not launched with
        cudaFuncAttributes fa;
        if (!cuda_ok(cudaFuncGetAttributes(&fa, grad_kernel<D, KV>))) return FVATTN_ERR_CUDA;
        if (static_cast<long long>(fa.numRegs) * GRAD_THREADS < 128ll * (GRAD_LOW + GRAD_GROUPS * GRAD_HIGH))
            return FVATTN_ERR_UNSUPPORTED;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_after(grad_kernel<D, KV>, static_cast<unsigned>(grid), GRAD_THREADS, L::ALLOC, s, a0, a1, b0, b1, args);
}

template <int D>
static int grad_launches(const Geo& g, const GradWs& wl, const void* q_t, const void* k_t, const void* v_t,
                         const void* o_t, const void* do_t, const float* lse, const int32_t* kv_idx,
                         const int32_t* kv_cnt, float scale, void* dq_t, void* dk_t, void* dv_t, char* ws,
                         cudaStream_t s) {
    const int BH = g.B * g.H;
    const long long rows = static_cast<long long>(BH) * g.Npad;
    float* nlse2 = reinterpret_cast<float*>(ws + wl.nlse2);
    float* ndelta = reinterpret_cast<float*>(ws + wl.ndelta);
    float2* norms = reinterpret_cast<float2*>(ws + wl.norms);
    uint32_t* bits = reinterpret_cast<uint32_t*>(ws + wl.bits);
    uint32_t* ulq = reinterpret_cast<uint32_t*>(ws + wl.ulq);
    uint32_t* ulk = reinterpret_cast<uint32_t*>(ws + wl.ulk);
    int32_t* ordq = reinterpret_cast<int32_t*>(ws + wl.ordq);
    int32_t* ordk = reinterpret_cast<int32_t*>(ws + wl.ordk);
    int32_t* ext = reinterpret_cast<int32_t*>(ws + wl.ext);
    int* counters = reinterpret_cast<int*>(ws + wl.counters);

    CUtensorMap tq, tk, tv, tdo;
    auto tmap = [&](CUtensorMap* m, const void* base) {
        return make_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, static_cast<unsigned long long>(rows), D, 64u,
                            static_cast<unsigned>(g.bs));
    };
    if (!tmap(&tq, q_t) || !tmap(&tk, k_t) || !tmap(&tv, v_t) || !tmap(&tdo, do_t)) return FVATTN_ERR_CUDA;
    int dev = 0, nsm = 0;
    if (!cuda_ok(cudaGetDevice(&dev)) ||
        !cuda_ok(cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev)))
        return FVATTN_ERR_CUDA;

    const int stat_blocks = static_cast<int>((rows + 63) / 64);
    const int bit_blocks = static_cast<int>((static_cast<long long>(BH) * g.nb + 7) / 8);
    int rc = launch_after(grad_prep_kernel<D>, static_cast<unsigned>(stat_blocks + bit_blocks), 256,
                          sizeof(uint32_t) * 8 * wl.nwords, s, g, stat_blocks, wl.nwords, static_cast<const uint4*>(o_t),
                          static_cast<const uint4*>(do_t), static_cast<const uint4*>(v_t), lse, kv_idx, kv_cnt, nlse2,
                          ndelta, norms, bits, ext);
    if (rc != FVATTN_OK) return rc;
    rc = launch_after(grad_lists_kernel, static_cast<unsigned>(2 * BH), LISTS_THREADS,
                          sizeof(int) * (2 * g.nb + 1 + 2 * wl.ngroups), s, g, wl.G, wl.ngroups, wl.nwords, bits, norms, ulq,
                          ulk, ordq, ordk, counters);
    if (rc != FVATTN_OK) return rc;

    GradArgs a;
    a.g = g;
    a.G = wl.G;
    a.ngroups = wl.ngroups;
    a.ext = ext;
    a.nlse2 = nlse2;
    a.ndelta = ndelta;
    a.scale = scale;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.total_items = BH * wl.ngroups;
    a.oob_row = static_cast<int>(rows);
    a.wait_limit_ns = WAIT_LIMIT_NS;
    const int grid = nsm < a.total_items ? nsm : a.total_items;
    a.ul = ulq;
    a.order = ordq;
    a.counter = counters;
    a.out0 = static_cast<__nv_bfloat16*>(dq_t);
    a.out1 = nullptr;
    rc = launch_grad<D, false>(tq, tdo, tk, tv, a, grid, dev, s);
    if (rc != FVATTN_OK) return rc;
    a.ul = ulk;
    a.order = ordk;
    a.counter = counters + 1;
    a.out0 = static_cast<__nv_bfloat16*>(dv_t);
    a.out1 = static_cast<__nv_bfloat16*>(dk_t);
    return launch_grad<D, true>(tk, tv, tq, tdo, a, grid, dev, s);
}

}  // namespace fv

using namespace fv;

extern "C" size_t fvattn_sparse_attn_bwd_workspace_size(const fvattn_geom* gp) {
    if (!gp) return 0;
    return grad_ws(*gp).total;
}

extern "C" int fvattn_sparse_attn_bwd(const fvattn_geom* gp, const void* q_t, const void* k_t, const void* v_t,
                                      const void* o_t, const void* do_t, const float* lse, const int32_t* kv_idx,
                                      const int32_t* kv_cnt, float scale, void* dq_t, void* dk_t, void* dv_t,
                                      void* workspace, size_t ws_bytes, fvattn_stream_t stream) {
    const void* ptrs[] = {q_t, k_t, v_t, o_t, do_t, lse, kv_idx, kv_cnt, dq_t, dk_t, dv_t, workspace};
    if (!gp) return FVATTN_ERR_INVALID;
    for (const void* p : ptrs)
        if (!p || (reinterpret_cast<uintptr_t>(p) & 15u) != 0) return FVATTN_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FVATTN_ERR_INVALID;
    if (!isfinite(scale) || !(scale > 0.f)) return FVATTN_ERR_INVALID;
    if (gp->D != 64 && gp->D != 128) return FVATTN_ERR_UNSUPPORTED;
    if (gp->bs != 16 && gp->bs != 32 && gp->bs != 64 && gp->bs != 128) return FVATTN_ERR_UNSUPPORTED;
    if (gp->nb <= 0 || gp->nb > 2560) return FVATTN_ERR_UNSUPPORTED;
    const long long rows = static_cast<long long>(gp->B) * gp->H * gp->Npad;
    if (rows >= (1ll << 31)) return FVATTN_ERR_UNSUPPORTED;
    const GradWs wl = grad_ws(*gp);
    if (ws_bytes < wl.total) return FVATTN_ERR_INVALID;
    const Geo g = to_geo(*gp);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    return gp->D == 128 ? grad_launches<128>(g, wl, q_t, k_t, v_t, o_t, do_t, lse, kv_idx, kv_cnt, scale, dq_t, dk_t,
                                             dv_t, ws, s)
                        : grad_launches<64>(g, wl, q_t, k_t, v_t, o_t, do_t, lse, kv_idx, kv_cnt, scale, dq_t, dk_t,
                                            dv_t, ws, s);
}

int fv::take_status_grad() { return fv::take_tu_status(); }
