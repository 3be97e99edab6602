// A paged cache of keys and values: append with rotation, and the attention
// of one new token a sequence over it.
//
// Append moves every new key, value and query once: a bit copy of V and
// (a, b) -> (a c - b s, a s + b c) on the pairs of K and Q, bound by memory.
// One CTA a token, eight CTAs an SM: two frames of 1560 tokens with 40 query
// and 40 key heads of 128 take 35.9 us, 5.4 TB/s read and written.  (Loads for
// four heads in flight a thread cost CTAs an SM, and 42 us; four tokens a CTA
// likewise, 41 to 49.)  A single token takes 2.5 us.
//
// Attention of one token reads each cached key and value once for a handful
// of multiply-adds: bound by memory too, so the kernel's whole form follows
// from keeping enough of the cache in flight, on every SM until the end.  The
// tokens of a sequence are split into parts of one size; an item is a part of
// one key head of one sequence, and 2 persistent CTAs an SM take the items
// that exist (from the lengths, on the device) in turn.  In a CTA a producer
// warp TMA-loads 64-token tiles of K and V through the page table into a ring
// of shared memory and runs on into the next item; four warps take 16 tokens
// of a tile each and keep an online softmax of their own (running maximum,
// sum and O in registers), and the four are joined at the item's end.  The
// heads that share a key head ride along in one product:
//   S^T [16 tokens x 8 heads] = K Q^T,  O^T [D x 8 heads] += V^T P^T
// with mma.sync.m16n8k16 (8 heads an N tile; a tcgen05 tile would have 128
// rows of which one to sixteen hold a query).  The parts' (maximum, sum, O)
// are joined in part order by a second small kernel.  40 heads over 32760
// tokens: 108 us, 6.2 TB/s; 24 ragged sequences up to 9000 tokens, 16-token
// pages: 86 us, 5.5 TB/s (103 with a CTA for a third of the longest length).
#include <cuda.h>

#include <atomic>

#include "common.cuh"
#include "fvattn_cache.h"
#include "ptx.cuh"
#include "sync.cuh"
#include "tmap.cuh"

namespace fv {

// ------------------------------------------------------------------ append

struct AppendArgs {
    int Hq, Hkv, page, pages, B, width, axes;
    int pair_end[3];              // first pair past each axis
    int rot_rows, halves, fill;
    long long k_stride, v_stride, q_stride, q_out_stride;
    const int32_t *cu, *lens, *table, *pos;
    const float* rot;
    const __nv_bfloat16 *k, *v, *q;
    __nv_bfloat16 *q_out, *k_pages, *v_pages;
};

// A thread moves 16 elements (eight pairs, two 16-byte vectors) of one head.
template <int D>
__global__ void __launch_bounds__(256) cache_append_kernel(const AppendArgs a) {
    constexpr int UPH = D / 16;          // such units a head
    __shared__ __align__(16) float cs[D];
    __shared__ int s_ok;
    __shared__ long long s_row;          // first element of the token's row in its page (head 0)
    const long long t = blockIdx.x;
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    bool bad = false;                    // a position outside the rotation table
    if (tid < 32) {
        // the token's sequence: how many sequences end at or before it
        int b = 0;
        if (a.cu) {
            for (int i = tid; i < a.B; i += 32) b += a.cu[i + 1] <= t;
            b = __reduce_add_sync(0xffffffffu, b);
        } else {
            b = t < a.B ? static_cast<int>(t) : a.B;
        }
        if (tid == 0) {
            int ok = 0;
            long long row = -1;
            const int bb = min(b, a.B - 1);      // (the three loads together, whether the row has a sequence or not)
            const long long first = a.cu ? a.cu[bb] : t, end = a.cu ? a.cu[bb + 1] : t + 1;
            const int len = a.lens[bb];
            if (b < a.B && first <= t) {         // rows outside the sequences are none's
                const long long n = len - (end - t);
                int pg = -1;
                if (n >= 0 && n < static_cast<long long>(a.width) * a.page)
                    pg = a.table[static_cast<long long>(b) * a.width + n / a.page];
                if (pg >= 0 && pg < a.pages) {
                    row = (static_cast<long long>(pg) * a.Hkv * a.page + n % a.page) * D;
                    ok = 1;
                } else {
                    record_status(FVATTN_ERR_BOUNDS);
                }
            }
            s_ok = ok;
            s_row = row;
        }
    } else if (a.rot && tid - 32 < D) {
        // this token's cosines and sines, by the pair's axis
        const int e = tid - 32, i = e < D / 2 ? e : e - D / 2;
        int ax = 0;
        while (ax < a.axes - 1 && i >= a.pair_end[ax]) ++ax;
        // rows outside the sequences have no position to read
        const bool live = a.cu ? t >= a.cu[0] && t < a.cu[a.B] : t < a.B;
        const int n = live ? a.pos[t * a.axes + ax] : 0;
        if (n >= 0 && n < a.rot_rows) {
            cs[e] = a.rot[static_cast<long long>(n) * D + e];
        } else {
            record_status(FVATTN_ERR_BOUNDS);
            bad = true;
        }
    }
    if (__syncthreads_or(bad) || !s_ok) {
        if (a.fill)                      // nobody else has written this row of q_out
            for (int i = blockIdx.y * 256 + tid; i < a.Hq * D / 8; i += gridDim.y * 256)
                reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride)[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int u = tid % UPH;
    const int step = a.halves ? D / 2 : 8;       // distance of the unit's two vectors
    const int e0 = a.halves ? 8 * u : 16 * u;
    float c[8], s[8];
    if (a.rot) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = cs[8 * u + i];
            s[i] = cs[D / 2 + 8 * u + i];
        }
    }
    const int heads = a.Hq + 2 * a.Hkv;
    const int per = 256 / UPH;
    for (int vh = blockIdx.y * per + tid / UPH; vh < heads; vh += gridDim.y * per) {
        const bool is_q = vh < a.Hq, is_v = vh >= a.Hq + a.Hkv;
        const int h = is_q ? vh : (is_v ? vh - a.Hq - a.Hkv : vh - a.Hq);
        const __nv_bfloat16* src = is_q ? a.q + t * a.q_stride : (is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride);
        src += static_cast<long long>(h) * D + e0;
        __nv_bfloat16* dst = is_q ? a.q_out + t * a.q_out_stride + static_cast<long long>(h) * D
                                  : (is_v ? a.v_pages : a.k_pages) + s_row + static_cast<long long>(h) * a.page * D;
        dst += e0;
        // (read once: evict-first loads leave L2 to the pages, 2 to 7% of the time)
        uint4 x = __ldcs(reinterpret_cast<const uint4*>(src));
        uint4 y = __ldcs(reinterpret_cast<const uint4*>(src + step));
        if (a.rot && !is_v) {
            uint32_t xe[4] = {x.x, x.y, x.z, x.w}, ye[4] = {y.x, y.y, y.z, y.w};
            if (a.halves) {      // x holds the pairs' first elements, y the second
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a0 = __uint_as_float(xe[i] << 16), a1 = __uint_as_float(xe[i] & 0xFFFF0000u);
                    const float b0 = __uint_as_float(ye[i] << 16), b1 = __uint_as_float(ye[i] & 0xFFFF0000u);
                    xe[i] = pack_bf16x2(a0 * c[2 * i] - b0 * s[2 * i], a1 * c[2 * i + 1] - b1 * s[2 * i + 1]);
                    ye[i] = pack_bf16x2(a0 * s[2 * i] + b0 * c[2 * i], a1 * s[2 * i + 1] + b1 * c[2 * i + 1]);
                }
            } else {             // each 32-bit word is one pair
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a0 = __uint_as_float(xe[i] << 16), b0 = __uint_as_float(xe[i] & 0xFFFF0000u);
                    const float a1 = __uint_as_float(ye[i] << 16), b1 = __uint_as_float(ye[i] & 0xFFFF0000u);
                    xe[i] = pack_bf16x2(a0 * c[i] - b0 * s[i], a0 * s[i] + b0 * c[i]);
                    ye[i] = pack_bf16x2(a1 * c[4 + i] - b1 * s[4 + i], a1 * s[4 + i] + b1 * c[4 + i]);
                }
            }
            x = make_uint4(xe[0], xe[1], xe[2], xe[3]);
            y = make_uint4(ye[0], ye[1], ye[2], ye[3]);
        }
        *reinterpret_cast<uint4*>(dst) = x;
        *reinterpret_cast<uint4*>(dst + step) = y;
    }
}

// ------------------------------------------------------------------ attention of one token

constexpr int DEC_TILE = 64;            // tokens a ring stage
constexpr int DEC_WARPS = 4;            // arithmetic warps: two take a tile, 32 tokens each
constexpr int DEC_THREADS = 32 * (DEC_WARPS + 1);
constexpr int DEC_CTAS = 2;             // CTAs an SM
constexpr int DEC_MAX_PARTS = 256;

template <int D>
struct DecSmem {
    static constexpr uint32_t TILE = DEC_TILE * D * 2u;          // D/64 halves of 8 KB, 128-byte swizzled rows
    static constexpr int STAGES = D == 128 ? 3 : 6;              // 96 KB a CTA
    static constexpr uint32_t K = 0, V = STAGES * TILE;
    static constexpr uint32_t JO = 2 * STAGES * TILE;            // [warp][8 heads][64] a piece of the four warps' O
    static constexpr uint32_t JM = JO + DEC_WARPS * 8 * 64 * 4u; // [warp][8] maximum, then sum
    static constexpr uint32_t BARS = JM + 2 * DEC_WARPS * 8 * 4u;
    static constexpr uint32_t ITEM = BARS + 8u * (3 * STAGES + 6);   // 2 x 4 words
    static constexpr uint32_t TOTAL = ITEM + 32u;
    static_assert(DEC_CTAS * (TOTAL + 1024u) <= 233472u, "shared memory of an SM");
};

struct DecArgs {
    int B, Hq, Hkv, group, gchunks, page, pages, width, tokens, parts;
    long long longest, q_stride;
    const __nv_bfloat16* q;
    const int32_t *table, *lens;
    float scale_log2;
    __nv_bfloat16* o;
    float* lse;
    float2* part_ml;       // [B][Hq][parts] (maximum in log2 units, sum)
    float* part_o;         // [B][Hq][parts][D], relative to the maximum
};

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A sequence's length, range-checked.
__device__ __forceinline__ int cache_len(const DecArgs& a, int b) {
    const int n = a.lens[b];
    const long long cap = min(a.longest, static_cast<long long>(a.width) * a.page);
    if (n < 0 || n > cap) {
        record_status(FVATTN_ERR_BOUNDS);
        return n < 0 ? 0 : static_cast<int>(cap);
    }
    return n;
}

// NT: tiles of 8 query heads (heads that share this key head, up to 16 a CTA).
template <int D, int NT>
__global__ void __launch_bounds__(DEC_THREADS, DEC_CTAS)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const DecArgs a) {
    using L = DecSmem<D>;
    constexpr int NS = L::STAGES;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ int s_abort;
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    if (sbase & 1023u) {   // the 128-byte swizzle needs 1024-byte aligned tiles
        pdl_wait();
        if (threadIdx.x == 0) record_status(FVATTN_ERR_UNSUPPORTED);
        return;
    }
    // Tile k is in stage k % NS and lands on full barrier k % NB.  NB is even: a barrier's tiles all belong to
    // one pair of warps, which waits for each of its phases (with a barrier a stage it would miss every second
    // one, and a wait on the parity would return for the phase two uses before).
    constexpr int NB = 2 * NS;
    unsigned long long* full = reinterpret_cast<unsigned long long*>(smem + L::BARS);
    unsigned long long* empty = full + NB;
    unsigned long long* item_full = empty + NS;      // [2]
    unsigned long long* item_empty = item_full + 2;  // [2]
    unsigned long long* join_full = item_empty + 2;  // the warps' parts are in shared memory
    unsigned long long* join_free = join_full + 1;   // and have been read
    int* items = reinterpret_cast<int*>(smem + L::ITEM);   // [2]: sequence, head chunk, first token, past the last (-1: end)
    volatile int* abort_flag = &s_abort;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NB; ++s) mbar_init(smem_u32(full + s), 1);
        for (int s = 0; s < NS; ++s) mbar_init(smem_u32(empty + s), DEC_WARPS / 2);
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(item_full + s), 1);
            mbar_init(smem_u32(item_empty + s), DEC_WARPS);
        }
        mbar_init(smem_u32(join_full), DEC_WARPS);
        mbar_init(smem_u32(join_free), DEC_WARPS);
        s_abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    const int HG = a.Hkv * a.gchunks;

    if (warp == DEC_WARPS) {
        // =========================== producer: items, tiles
        const int box = min(a.page, DEC_TILE);           // rows a load
        const int boxes = DEC_TILE / box;
        int b0 = 0, len = 0, seq = 0;
        uint32_t it = 0;
        long long before = 0, incl = 0;                  // items of the sequences before b0; of b0 .. b0 + lane
        auto chunk = [&]() {                             // the items of 32 sequences, one a lane
            len = b0 + lane < a.B ? cache_len(a, b0 + lane) : 0;
            long long n = (static_cast<long long>(len) + a.tokens - 1) / a.tokens;
            if (a.parts == 1 && b0 + lane < a.B) n = 1;  // an empty sequence is answered here
            incl = n * HG;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += y;
            }
        };
        chunk();
        bool ok = true;
        for (long long j = blockIdx.x; ok; j += gridDim.x) {
            long long total = __shfl_sync(0xffffffffu, incl, 31);
            while (j >= before + total && b0 + 32 < a.B) {
                before += total;
                b0 += 32;
                chunk();
                total = __shfl_sync(0xffffffffu, incl, 31);
            }
            const bool end = j >= before + total;
            // the first sequence whose items end after j
            const int sel = end ? 0 : __ffs(static_cast<int>(__ballot_sync(0xffffffffu, j < before + incl))) - 1;
            const long long upto = __shfl_sync(0xffffffffu, incl, sel > 0 ? sel - 1 : 0);
            const long long local = j - before - (sel > 0 ? upto : 0);
            const int b = b0 + sel, hg = static_cast<int>(local % HG);
            const int t0 = static_cast<int>(local / HG) * a.tokens;
            const int blen = __shfl_sync(0xffffffffu, len, sel);
            const int t1 = blen - t0 > a.tokens ? t0 + a.tokens : blen;
            const int slot = seq & 1;
            if (!wait_warp(smem_u32(item_empty + slot), ((seq >> 1) & 1) ^ 1, abort_flag)) break;
            if (lane == 0) {
                items[slot * 4] = b;
                items[slot * 4 + 1] = hg;
                items[slot * 4 + 2] = t0;
                items[slot * 4 + 3] = end ? -1 : t1;
                mbar_arrive(smem_u32(item_full + slot));
            }
            if (end) break;
            ++seq;
            const int hk = hg / a.gchunks;
            const int32_t* row = a.table + static_cast<long long>(b) * a.width;
            // a lane's page of the tile at t; looked up a tile ahead of its use
            auto page_of = [&](int t) {
                const int tok = t + lane * box;
                return lane < boxes && tok < t1 ? row[tok / a.page] : 0;
            };
            int next = page_of(t0);
            for (int t = t0; t < t1; t += DEC_TILE, ++it) {
                const int st = it % NS;
                const int tok = t + lane * box;
                const bool mine = lane < boxes && tok < t1;
                int pg = next;
                if (t1 - t > DEC_TILE) next = page_of(t + DEC_TILE);
                if (pg < 0 || pg >= a.pages) {
                    record_status(FVATTN_ERR_BOUNDS);
                    pg = 0;
                }
                if (!wait_warp(smem_u32(empty + st), ((it / NS) & 1) ^ 1, abort_flag)) {
                    ok = false;
                    break;
                }
                const int nbox = __popc(__ballot_sync(0xffffffffu, mine));
                const uint32_t bar = smem_u32(full + it % NB);
                if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(2 * nbox * box * D * 2));
                __syncwarp();
                if (mine) {
                    const int r = (pg * a.Hkv + hk) * a.page + tok % a.page;
                    const uint32_t off = st * L::TILE + static_cast<uint32_t>(lane * box) * 128u;
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) {
                        tma_load_2d(sbase + L::K + off + h * 8192u, &tmK, h * 64, r, bar);
                        tma_load_2d(sbase + L::V + off + h * 8192u, &tmV, h * 64, r, bar);
                    }
                }
            }
        }
        // no copy outlives the CTA
        if (lane == 0)
            for (uint32_t k = 0; k < NB && k < it; ++k) wait_bar_drain(smem_u32(full + k), ((it - 1 - k) / NB) & 1);
        __syncwarp();
        return;
    }

    // =========================== arithmetic: 32 tokens of every second tile
    const int g = lane >> 2, tq = lane & 3;
    float* jo = reinterpret_cast<float*>(smem + L::JO);
    float* jm = reinterpret_cast<float*>(smem + L::JM);
    float* jl = jm + DEC_WARPS * 8;
    uint32_t it = 0, joins = 0;
    for (int seq = 0;; ++seq) {
        const int slot = seq & 1;
        if (!wait_warp(smem_u32(item_full + slot), (seq >> 1) & 1, abort_flag)) return;
        const int b = items[slot * 4], hg = items[slot * 4 + 1], t0 = items[slot * 4 + 2], t1 = items[slot * 4 + 3];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(item_empty + slot));
        if (t1 < 0) return;
        const int hk = hg / a.gchunks, gc = hg - hk * a.gchunks;
        const int head0 = hk * a.group + gc * 16;                 // first query head of the item
        const int nheads = min(16, a.group - gc * 16);

        float o[NT][D / 16][4];
        float m[NT][2], l[NT][2];
        uint32_t qf[NT][D / 16][2];        // Q^T: head g of the tile, elements 2 tq .. of each 16
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][d][i] = 0.f;
            const int h = n * 8 + g;
            const __nv_bfloat16* qr = a.q + static_cast<long long>(b) * a.q_stride + static_cast<long long>(head0 + h) * D;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    qf[n][kk][i] = h < nheads ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + i * 8 + 2 * tq) : 0u;
        }
        const uint32_t tiles = static_cast<uint32_t>((t1 - t0 + DEC_TILE - 1) / DEC_TILE);
        for (uint32_t i = (it ^ static_cast<uint32_t>(warp >> 1)) & 1u; i < tiles; i += 2) {
            const uint32_t k = it + i;
            const int st = k % NS;
            if (!wait_warp(smem_u32(full + k % NB), (k / NB) & 1, abort_flag)) return;
            const int left = t1 - (t0 + static_cast<int>(i) * DEC_TILE + (warp & 1) * 32);   // of 32 tokens that exist
            if (left > 0) {
                const uint32_t kt = sbase + L::K + st * L::TILE, vt = sbase + L::V + st * L::TILE;
                float s[2][NT][4];        // two rows of 16 tokens
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int n = 0; n < NT; ++n) s[z][n][0] = s[z][n][1] = s[z][n][2] = s[z][n][3] = 0.f;
                {
                    const int r = (warp & 1) * 32 + (lane & 15);
                    const uint32_t rb = kt + static_cast<uint32_t>(r) * 128u;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            uint32_t af[4];
                            ldsm_x4(af, rb + z * 2048u + (kk >> 2) * 8192u + ((((kk & 3) * 2 + (lane >> 4)) ^ (r & 7)) * 16u));
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma_16816(s[z][n], af, qf[n][kk][0], qf[n][kk][1]);
                        }
                }
                // row z, token g: s[z][.][0..1], token g + 8: s[z][.][2..3]; heads 2 tq, 2 tq + 1 of the tile
                uint32_t pb[2][NT][2];
                bool same = true;
                float alpha[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            s[z][n][i] = z * 16 + g < left ? s[z][n][i] * a.scale_log2 : -INFINITY;
                            s[z][n][2 + i] = z * 16 + g + 8 < left ? s[z][n][2 + i] * a.scale_log2 : -INFINITY;
                            mx = fmax3(mx, s[z][n][i], s[z][n][2 + i]);
                        }
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                        const float mn = fmaxf(m[n][i], mx);
                        const float ref = mn == -INFINITY ? 0.f : mn;      // scores of -inf only: P is 0
                        alpha[n][i] = ex2_approx(m[n][i] - ref);
                        same = same && mn == m[n][i];
                        float sum = 0.f;
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            s[z][n][i] = ex2_approx(s[z][n][i] - ref);
                            s[z][n][2 + i] = ex2_approx(s[z][n][2 + i] - ref);
                            sum += s[z][n][i] + s[z][n][2 + i];
                        }
                        l[n][i] = l[n][i] * alpha[n][i] + sum;
                        m[n][i] = mn;
                    }
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        pb[z][n][0] = movm_t(pack_bf16x2(s[z][n][0], s[z][n][1]));
                        pb[z][n][1] = movm_t(pack_bf16x2(s[z][n][2], s[z][n][3]));
                    }
                }
                if (!__all_sync(0xffffffffu, same)) {     // a maximum moved: O to the new one
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int d = 0; d < D / 16; ++d)
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[n][d][i] *= alpha[n][i & 1];
                }
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int lz = left - z * 16;
                    // values of tokens that do not exist are taken as 0 (0 times what is there could be NaN);
                    // lane words hold tokens 2 tq, 2 tq + 1 (words 0, 1) and 8 further (words 2, 3)
                    const uint32_t k0 = (2 * tq < lz ? 0x0000FFFFu : 0u) | (2 * tq + 1 < lz ? 0xFFFF0000u : 0u);
                    const uint32_t k1 = (2 * tq + 8 < lz ? 0x0000FFFFu : 0u) | (2 * tq + 9 < lz ? 0xFFFF0000u : 0u);
                    const int r = (warp & 1) * 32 + z * 16 + (lane & 7) + ((lane >> 4) & 1) * 8;
                    const uint32_t rb = vt + static_cast<uint32_t>(r) * 128u;
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        uint32_t af[4];
                        ldsm_x4_t(af, rb + (d >> 2) * 8192u + ((((d & 3) * 2 + ((lane >> 3) & 1)) ^ (r & 7)) * 16u));
                        if (lz < 16) {
                            af[0] &= k0;
                            af[1] &= k0;
                            af[2] &= k1;
                            af[3] &= k1;
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_16816(o[n][d], af, pb[z][n][0], pb[z][n][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(empty + st));
        }
        it += tiles;

        // ---- join the four warps, 8 heads and 64 elements at a time
        const int part = t0 / a.tokens;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n * 8 >= nheads) break;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], d);
#pragma unroll
            for (int e0 = 0; e0 < D; e0 += 64) {
                if (joins > 0 && !wait_warp(smem_u32(join_free), (joins - 1) & 1, abort_flag)) return;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int h = 2 * tq + i;
                    if (g == 0) {
                        jm[warp * 8 + h] = m[n][i];
                        jl[warp * 8 + h] = l[n][i];
                    }
                    // (element e of head h at e + 8 (h / 2), so that the four heads' lanes meet other banks)
                    float* dst = jo + (warp * 8 + h) * 64;
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        dst[(d * 16 + g + 8 * tq) & 63] = o[n][e0 / 16 + d][i];
                        dst[(d * 16 + 8 + g + 8 * tq) & 63] = o[n][e0 / 16 + d][2 + i];
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(join_full));
                if (!wait_warp(smem_u32(join_full), joins & 1, abort_flag)) return;
                const int count = min(8, nheads - n * 8) * 64;
                for (int i = threadIdx.x; i < count; i += 32 * DEC_WARPS) {
                    const int h = i >> 6, e = i & 63, d = e0 + e, at8 = (e + 8 * (h >> 1)) & 63;
                    float mx = -INFINITY;
#pragma unroll
                    for (int w = 0; w < DEC_WARPS; ++w) mx = fmaxf(mx, jm[w * 8 + h]);
                    const float ref = mx == -INFINITY ? 0.f : mx;
                    float sum = 0.f, acc = 0.f;
#pragma unroll
                    for (int w = 0; w < DEC_WARPS; ++w) {
                        const float f = ex2_approx(jm[w * 8 + h] - ref);
                        sum += jl[w * 8 + h] * f;
                        acc += jo[(w * 8 + h) * 64 + at8] * f;
                    }
                    const long long at = static_cast<long long>(b) * a.Hq + head0 + n * 8 + h;
                    if (a.parts == 1) {
                        a.o[at * D + d] = __float2bfloat16(sum == 0.f ? 0.f : acc / sum);
                        if (a.lse && d == 0) a.lse[at] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
                    } else {
                        const long long pt = at * a.parts + part;
                        a.part_o[pt * D + d] = acc;
                        if (d == 0) a.part_ml[pt] = make_float2(mx, sum);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(join_free));
                ++joins;
            }
        }
    }
}

// One CTA of W warps per (sequence, query head): join the parts that hold
// tokens.  Warp w takes parts w, w + W, .. in order, and the W are added in
// order.  (A single head of 100000 tokens, 224 parts: 9 us with four warps.)
template <int D, int W>
__global__ void __launch_bounds__(32 * W) cache_join_kernel(const DecArgs a) {
    constexpr int V = D / 32;          // elements a lane
    __shared__ float s_o[W][D], s_l[W];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long at = blockIdx.x;
    pdl_wait();
    const int len = cache_len(a, static_cast<int>(at / a.Hq));
    const int n = static_cast<int>((static_cast<long long>(len) + a.tokens - 1) / a.tokens);
    const float2* ml = a.part_ml + at * a.parts;
    const float* po = a.part_o + at * a.parts * D;
    float mx = -INFINITY;
    for (int p = lane; p < n; p += 32) mx = fmaxf(mx, ml[p].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    const float ref = mx == -INFINITY ? 0.f : mx;
    float acc[V], sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll 8
    for (int p = warp; p < n; p += W) {
        const float2 x = ml[p];
        const float f = ex2_approx(x.x - ref);
        sum += x.y * f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += po[static_cast<long long>(p) * D + i * 32 + lane] * f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) s_o[warp][i * 32 + lane] = acc[i];
    if (lane == 0) s_l[warp] = sum;
    __syncthreads();
    if (threadIdx.x < D) {
        const int d = threadIdx.x;
        float v = 0.f;
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            v += s_o[w][d];
            sum += s_l[w];
        }
        a.o[at * D + d] = __float2bfloat16(sum == 0.f ? 0.f : v / sum);
        if (a.lse && d == 0) a.lse[at] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
    }
}

// ------------------------------------------------------------------ host side

static bool cache_ok(const fvattn_cache* c) {
    return c && c->k && c->v && ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15u) == 0 &&
           c->k != c->v && c->pages > 0 && c->Hkv > 0;
}

static bool cache_supported(int D, int page) {
    return (D == 64 || D == 128) && (page == 16 || page == 32 || page == 64 || page == 128);
}

static bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static bool on4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The split: parts of one size, so many tokens that the items fill the GPU's
// CTA slots once, but no more than 512 (1024 where over eight query heads
// share a key head, whose partial results weigh more): several items a slot
// even out ragged lengths, and the ring runs on from one to the next.  With
// 512 and 1024: 24 ragged sequences, 4 heads a key head 88.3 and 92.6 us; 48
// sequences, 8 heads 47.6 and 51.2; 8 long ones, 16 heads 48.6 and 39.6; 40
// heads over 32760 tokens alike.  (256: 88.9, and 123 for 110 in the last.)  At
// least 128 tokens, and at most DEC_MAX_PARTS parts.
static int split_parts(int B, int Hq, int Hkv, long long longest, int nsm, int* tokens) {
    const int group = Hq / Hkv;
    const long long base = static_cast<long long>(B) * Hkv * ((group + 15) / 16);
    const long long slots = static_cast<long long>(nsm) * DEC_CTAS;
    const long long most = group > 8 ? 1024 : 512;
    const double once = static_cast<double>(longest) * static_cast<double>(base) / static_cast<double>(slots);
    long long tk = once > static_cast<double>(most) ? most : static_cast<long long>(once);
    if (tk < 128) tk = 128;
    const long long least = (longest + DEC_MAX_PARTS - 1) / DEC_MAX_PARTS;
    if (tk < least) tk = least;
    tk = (tk + DEC_TILE - 1) / DEC_TILE * DEC_TILE;
    *tokens = static_cast<int>(tk);
    const long long parts = (longest + tk - 1) / tk;
    return parts < 1 ? 1 : static_cast<int>(parts);
}

static size_t attn_ws(int B, int Hq, int D, int parts) {
    if (parts < 2) return 0;
    const size_t n = static_cast<size_t>(B) * Hq * parts;
    return (n * 8 + 255) / 256 * 256 + n * D * 4;
}

// The current device and its SMs (148 without a device: sizes are asked for on
// machines without one too).
static int current_sms(int* device = nullptr) {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (!cuda_ok(cudaGetDevice(&dev))) return 148;
    if (device) *device = dev;
    if (dev >= 0 && dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (!cuda_ok(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) || n <= 0) return 148;
    if (dev >= 0 && dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <int D, int NT>
static int launch_cache_attn(const CUtensorMap& tk, const CUtensorMap& tv, const DecArgs& a, int B, int dev, int nsm,
                             cudaStream_t s) {
    using L = DecSmem<D>;
    static std::atomic<unsigned long long> ready{0};   // devices on which the kernel has its shared memory
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if ((ready.load(std::memory_order_relaxed) & bit) == 0ull) {
        if (!cuda_ok(cudaFuncSetAttribute(cache_attn_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          static_cast<int>(L::TOTAL))))
            return FVATTN_ERR_CUDA;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    const long long items = static_cast<long long>(B) * a.Hkv * a.gchunks * a.parts;
    const long long slots = static_cast<long long>(nsm) * DEC_CTAS;
    const int rc = launch_after(cache_attn_kernel<D, NT>, dim3(static_cast<unsigned>(items < slots ? items : slots)), DEC_THREADS,
                                L::TOTAL, s, tk, tv, a);
    if (rc != FVATTN_OK || a.parts == 1) return rc;
    const dim3 heads(static_cast<unsigned>(B) * static_cast<unsigned>(a.Hq));
    return a.parts > 32 ? launch_after(cache_join_kernel<D, 16>, heads, 512, 0, s, a)
                        : launch_after(cache_join_kernel<D, 4>, heads, 128, 0, s, a);
}

}  // namespace fv

using namespace fv;

static int append_impl(const fvattn_cache* c, int B, long long rows, const int32_t* cu, const int32_t* lens,
                       const int32_t* table, int width, const void* k, long long k_stride, const void* v,
                       long long v_stride, const void* q, long long q_stride, int Hq, void* q_out,
                       long long q_out_stride, const fvattn_rotation* rot, int fill, fvattn_stream_t stream) {
    if (!cache_ok(c) || B < 1 || rows < 0 || rows > 0x7fffffffll || width < 1 || !lens || !table || !k || !v)
        return FVATTN_ERR_INVALID;
    if (!cache_supported(c->D, c->page)) return FVATTN_ERR_UNSUPPORTED;
    if (!cu && rows < B) return FVATTN_ERR_INVALID;
    if (!on16(k) || !on16(v) || !on4(lens) || !on4(table) || (cu && !on4(cu))) return FVATTN_ERR_INVALID;
    const long long kv_row = static_cast<long long>(c->Hkv) * c->D;
    if (k_stride < kv_row || v_stride < kv_row || k_stride % 8 || v_stride % 8) return FVATTN_ERR_INVALID;
    if ((q == nullptr) != (q_out == nullptr)) return FVATTN_ERR_INVALID;
    if (q) {
        const long long q_row = static_cast<long long>(Hq) * c->D;
        if (Hq < 1 || !on16(q) || !on16(q_out) || q_stride < q_row || q_out_stride < q_row || q_stride % 8 ||
            q_out_stride % 8)
            return FVATTN_ERR_INVALID;
    }
    AppendArgs a = {};
    if (rot) {
        if (!rot->table || !on16(rot->table) || !rot->pos || !on4(rot->pos) || rot->rows < 1 || rot->axes < 1 ||
            rot->axes > 3 || (rot->halves != 0 && rot->halves != 1))
            return FVATTN_ERR_INVALID;
        int end = 0;
        for (int i = 0; i < rot->axes; ++i) {
            if (rot->pairs[i] < 0 || rot->pairs[i] > c->D / 2) return FVATTN_ERR_INVALID;
            end += rot->pairs[i];
            a.pair_end[i] = end;
        }
        if (end != c->D / 2) return FVATTN_ERR_INVALID;
        a.axes = rot->axes;
        a.rot_rows = rot->rows;
        a.halves = rot->halves;
        a.rot = rot->table;
        a.pos = rot->pos;
    }
    if (rows == 0) return FVATTN_OK;
    a.fill = fill;
    a.Hq = q ? Hq : 0;
    a.Hkv = c->Hkv;
    a.page = c->page;
    a.pages = c->pages;
    a.B = B;
    a.width = width;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_stride = q_stride;
    a.q_out_stride = q_out_stride;
    a.cu = cu;
    a.lens = lens;
    a.table = table;
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_out = static_cast<__nv_bfloat16*>(q_out);
    a.k_pages = static_cast<__nv_bfloat16*>(c->k);
    a.v_pages = static_cast<__nv_bfloat16*>(c->v);
    // Below 512 tokens a token's heads go over several CTAs, from there on one CTA takes them a pass after the other
    // (which looks up the token's page and position once).  One CTA a token and spread, 40 + 40 + 40 heads of 128:
    // 1 token 3.74 and 2.60 us, 148 5.31 and 4.46, 384 9.4 and 7.0, 512 9.5 and 9.1, 700 9.7 and 11.4, 1500 15.8
    // and 21.1; 32 + 8 + 8 heads: 384 5.5 and 4.3, 512 5.7 and 6.0, 1500 8.9 and 11.0.
    const int per = 256 / (c->D / 16);
    const int passes = (a.Hq + 2 * a.Hkv + per - 1) / per;
    const dim3 grid(static_cast<unsigned>(rows), rows < 512 ? static_cast<unsigned>(passes < 64 ? passes : 64) : 1u);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return c->D == 128 ? launch_after(cache_append_kernel<128>, grid, 256, 0, s, a)
                       : launch_after(cache_append_kernel<64>, grid, 256, 0, s, a);
}

extern "C" int fvattn_cache_append(const fvattn_cache* c, int B, long long rows, const int32_t* cu,
                                   const int32_t* lens, const int32_t* table, int width, const void* k,
                                   long long k_stride, const void* v, long long v_stride, const void* q,
                                   long long q_stride, int Hq, void* q_out, long long q_out_stride,
                                   const fvattn_rotation* rot, fvattn_stream_t stream) {
    return append_impl(c, B, rows, cu, lens, table, width, k, k_stride, v, v_stride, q, q_stride, Hq, q_out, q_out_stride,
                       rot, 0, stream);
}

extern "C" int fvattn_cache_append_fresh(const fvattn_cache* c, int B, long long rows, const int32_t* cu,
                                         const int32_t* lens, const int32_t* table, int width, const void* k,
                                         long long k_stride, const void* v, long long v_stride, const void* q,
                                         long long q_stride, int Hq, void* q_out, long long q_out_stride,
                                         const fvattn_rotation* rot, fvattn_stream_t stream) {
    if (!q || q == q_out) return FVATTN_ERR_INVALID;
    return append_impl(c, B, rows, cu, lens, table, width, k, k_stride, v, v_stride, q, q_stride, Hq, q_out, q_out_stride,
                       rot, 1, stream);
}

extern "C" int fvattn_cache_attn_parts(int B, int Hq, int Hkv, int D, long long longest, int* tokens) {
    if (B < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv || (D != 64 && D != 128) || longest < 0 || longest > 0x7fffffffll - 128)
        return 0;
    int tk = 0;
    const int parts = split_parts(B, Hq, Hkv, longest, current_sms(), &tk);
    if (tokens) *tokens = tk;
    return parts;
}

extern "C" size_t fvattn_cache_attn_workspace_size(int B, int Hq, int Hkv, int D, long long longest) {
    const int parts = fvattn_cache_attn_parts(B, Hq, Hkv, D, longest, nullptr);
    return attn_ws(B, Hq, D, parts);
}

extern "C" int fvattn_cache_attn(const fvattn_cache* c, int B, int Hq, const void* q, long long q_stride,
                                 const int32_t* table, int width, const int32_t* lens, long long longest, float scale,
                                 void* o, float* lse, void* workspace, size_t ws_bytes, fvattn_stream_t stream) {
    if (!cache_ok(c) || B < 1 || B > 65535 || width < 1 || !q || !table || !lens || !o) return FVATTN_ERR_INVALID;
    if (!cache_supported(c->D, c->page)) return FVATTN_ERR_UNSUPPORTED;
    if (Hq < c->Hkv || Hq % c->Hkv || longest < 0 || longest > 0x7fffffffll - 128) return FVATTN_ERR_INVALID;
    if (!on16(q) || !on16(o) || !on4(table) || !on4(lens) || (lse && !on4(lse))) return FVATTN_ERR_INVALID;
    if (q_stride < static_cast<long long>(Hq) * c->D || q_stride % 8) return FVATTN_ERR_INVALID;
    if (!isfinite(scale) || !(scale > 0.f)) return FVATTN_ERR_INVALID;
    const long long rows = static_cast<long long>(c->pages) * c->Hkv * c->page;
    if (rows >= (1ll << 31)) return FVATTN_ERR_UNSUPPORTED;
    DecArgs a = {};
    a.Hq = Hq;
    a.Hkv = c->Hkv;
    a.group = Hq / c->Hkv;
    a.gchunks = (a.group + 15) / 16;
    if (static_cast<long long>(a.Hkv) * a.gchunks > 65535 || static_cast<long long>(B) * Hq > 0x7fffffffll)
        return FVATTN_ERR_UNSUPPORTED;
    int dev = 0;
    const int nsm = current_sms(&dev);
    a.B = B;
    a.parts = split_parts(B, Hq, c->Hkv, longest, nsm, &a.tokens);
    if (a.parts > 1) {
        if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
            ws_bytes < attn_ws(B, Hq, c->D, a.parts))
            return FVATTN_ERR_INVALID;
        const size_t n = static_cast<size_t>(B) * Hq * a.parts;
        a.part_ml = static_cast<float2*>(workspace);
        a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + (n * 8 + 255) / 256 * 256);
    }
    a.page = c->page;
    a.pages = c->pages;
    a.width = width;
    a.longest = longest;
    a.q_stride = q_stride;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.table = table;
    a.lens = lens;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.o = static_cast<__nv_bfloat16*>(o);
    a.lse = lse;
    CUtensorMap tk, tv;
    const unsigned box = static_cast<unsigned>(c->page < DEC_TILE ? c->page : DEC_TILE);
    if (!make_tmap_2d(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c->k, static_cast<unsigned long long>(rows),
                      static_cast<unsigned long long>(c->D), 64u, box) ||
        !make_tmap_2d(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c->v, static_cast<unsigned long long>(rows),
                      static_cast<unsigned long long>(c->D), 64u, box))
        return FVATTN_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool two = a.group > 8;
    if (c->D == 128)
        return two ? launch_cache_attn<128, 2>(tk, tv, a, B, dev, nsm, s) : launch_cache_attn<128, 1>(tk, tv, a, B, dev, nsm, s);
    return two ? launch_cache_attn<64, 2>(tk, tv, a, B, dev, nsm, s) : launch_cache_attn<64, 1>(tk, tv, a, B, dev, nsm, s);
}

int fv::take_status_cache() { return fv::take_tu_status(); }
