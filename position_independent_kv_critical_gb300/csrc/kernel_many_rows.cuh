// Attention of requests with more than a few new rows (prompt chunks) over their pages.
//
// The same sums as kernel_few_rows.cuh; here a key meets up to thousands of rows, so the tensor cores
// bound it.  Three launches: chunk_rotate_kernel rotates the chunk's queries and, once, the keys of the
// requests' pages into the workspace (fp16, slot order, slots that take no part zeroed); a key tile is
// visited by every pair of row tiles of its request, and rotating it at each visit costs more than
// writing and re-reading it once (the page-reading fused attention of this library, which does rotate
// in the kernel, takes twice as long).  The values stay in the pool: many_rows_kernel copies a key
// tile's eight pages straight from it.  A request whose rows fit one tile (128: a long draft, a short
// chunk) visits each key once: its keys are not rotated beforehand but copied from their pages and rotated
// in shared memory by the warps that would have tile B (24 requests of 6 k tokens with 64 rows: 262 -> 194
// us; 152 without the rotation's arithmetic, 91 at the copy rate.  One warp a sub-partition rotates and
// one has the softmax, so latencies bind: a third stage for keys and values changed nothing).
//
// many_rows_kernel: one block an SM; a run is two 128-row tiles A and B of one (request, kv head) --
// row m of a tile is token m / g, query head m % g of the kv head -- against the 128-key tiles its last
// row sees.  All runs' key tiles, in (request, kv head, row pair, tile) order, are dealt to the blocks
// in contiguous parts of equal weight by pcf_chunk_tables, whatever the lengths; a block passes on what it has of
// the runs it shares with its neighbours (two at most) and many_join_kernel adds those up in a fixed
// order.
//   warps 0-3   softmax of tile A, warps 4-7 of tile B (or the rotation): S row from TMEM, causal cut and exclusion bits,
//               online softmax (lazy rescale), P -> TMEM over the S columns, O epilogue
//   warps 8/11  Q K^T issue for tile A / B (warp 8 also owns the TMEM allocation)
//   warps 12/13 P V issue for tile A / B
//   warp  9     runs in order, Q and K tiles (TMA), exclusion bits of a tile
//   warp  10    V tiles: a page and half per TMA copy; rows of slots that hold nothing are zeroed
// A key tile is worked in two 64-key halves, S double-buffered per row tile: P(q) V runs, then Q K(q+2)
// goes into the buffer P(q) came from, while the softmax works on S(q+1).  TMEM: tile t's S halves at
// columns t*128 + {0, 64}, O_A at 256, O_B at 384; P (bf16 pairs) overwrites the S half it came from and
// is the A operand of O += P V (M = 128, N = d, K = 64 keys).
//
// The sum of a row's weights takes them unrounded, unlike the few-row kernel's: where one key dominates, the
// result is its value within half a bf16 step and the final rounding.
//
// Measured: 2048 tokens behind 32 k (32/8 heads, d 128; 1.13 TFLOP): 841 us a call of all launches, 1348 TFLOP/s
// or 71 % of a large product's burst rate, 94 % of the time in this kernel; 907 to 915 us, 1240 TFLOP/s, where
// such calls run for seconds and the power cap lowers the clock.  The chain S -> softmax -> P -> P V -> next Q K^T
// through the two halves bounds it (the tensor pipe is busy 62 % of the time), not the exponentials (31 % of
// their unit) or the copies.  Six chunks of 100 to 700 tokens beside 26 single tokens: 58 % of 276 us.
// d = 64: 717 us, 791 TFLOP/s: as many scores, each with half the products.
#pragma once
#include "chunk_format.h"
#include "kernel_attn.cuh"
#include "kernel_chunk_tables.cuh"
#include "kernel_few_rows.cuh"
#include "ptx.cuh"

namespace pcf {

// ------------------------------------------------------------------ rotation
// A block takes 16 rows at a time: a page of a request (every kv head) or 16 rows of the chunk (every
// query head).  Thread (r, c) turns the 16-byte chunks c and c + d/16 of row r, at one angle for all
// heads, so the table is read once a row; four heads' loads are in flight a thread.  Bound by HBM (reads
// the keys, writes them once): 4 % of a call with 2 k rows behind 33 k tokens, 11 % of one with six chunks.
// fp16: 11 bits of a rotated value instead of bf16's 8, with its range checked.
struct RotateParams {
    const int32_t* plan;
    const __nv_bfloat16* q;
    const __nv_bfloat16* k_pool;
    const int32_t* block_table;
    const int32_t* page_pos;
    const uint16_t* excl;
    const int32_t* row_pos;
    const float* rope;
    __half* q_rot;              // [Hkv][max_rows][g][D], scaled by log2(e) / sqrt(d)
    __half* k_rot;              // [Hkv][pages][16][D]
    int64_t q_stride;
    int32_t n, max_pages, max_rows, hq, hkv, n_phys, max_pos, tag, total_pages;
};

template <int D>
__global__ void __launch_bounds__(256) chunk_rotate_kernel(const RotateParams p) {
    constexpr int CPR = D / 16;
    constexpr int LANES = 256 / (kPage * CPR);   // heads side by side
    grid_dep_wait();
    grid_dep_launch();
    if (!plan_fits(p.plan, p.tag)) return;
    const int32_t* seq = p.plan + plan_array(CA_SEQ, p.n);
    const int32_t* add = p.plan + plan_array(CA_NEW, p.n);
    const int32_t* kpage = p.plan + plan_array(CA_KPAGE, p.n);
    const int32_t rows = p.plan[C_ROWS], pages = kpage[p.n];
    if (p.plan[plan_array(CA_MANY, p.n) + p.n] == 0) return;      // no request with many rows
    const int c = threadIdx.x % CPR, r = threadIdx.x / CPR % kPage, h0 = threadIdx.x / (CPR * kPage);
    const int g = p.hq / p.hkv, gs = __ffs(g) - 1;
    const int q_blocks = (rows + kPage - 1) / kPage;
    float big = 0.f, nan = 0.f;   // largest magnitude; NaN where a value is
    for (int t = blockIdx.x; t < pages + q_blocks; t += gridDim.x) {
        const bool is_k = t < pages;
        const __nv_bfloat16* src = nullptr;      // row of head 0
        int64_t src_head, dst_head = 0;
        __half* dst = nullptr;
        int32_t pos = 0;
        bool have = true;                        // else zeros
        int heads;
        float scale = 1.f;
        if (is_k) {
            const int b = row_request(kpage, p.n, t);
            const int pg = t - kpage[b];
            const int64_t e = (int64_t)b * p.max_pages + pg;
            const int32_t ph = p.block_table[e], pp = p.page_pos[e];
            const uint32_t ex = p.excl ? p.excl[e] : 0u;
            have = !(ex >> r & 1u) && pg * kPage + r < seq[b] + add[b];
            if (ph < 0 || ph >= p.n_phys || pp < 0 || pp > p.max_pos - kPage) {
                set_dev_error(kDevErrBounds);
                have = false;
            }
            pos = pp + r;
            heads = p.hkv;
            src = p.k_pool + ((int64_t)ph * p.hkv * kPage + r) * D;
            src_head = kPage * D;
            dst = p.k_rot + ((int64_t)t * kPage + r) * D;
            dst_head = (int64_t)p.total_pages * kPage * D;
        } else {
            const int32_t row = (t - pages) * kPage + r;
            if (row >= rows) continue;
            pos = p.row_pos[row];
            if (pos < 0 || pos >= p.max_pos) {
                set_dev_error(kDevErrBounds);
                have = false;
            }
            heads = p.hq;
            src = p.q + row * p.q_stride;
            src_head = D;
            dst = p.q_rot + (int64_t)row * g * D;
            scale = 1.4426950408889634f * (D == 128 ? 0.08838834764831845f : 0.125f);   // log2(e) / sqrt(d)
        }
        float4 cs[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            cs[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (have) cs[e] = reinterpret_cast<const float4*>(p.rope + (int64_t)pos * D + 16 * c)[e];
            cs[e].x *= scale;
            cs[e].y *= scale;
            cs[e].z *= scale;
            cs[e].w *= scale;
        }
        for (int h = h0; h < heads; h += 4 * LANES) {
            uint4 lo[4], hi[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
                if (have && h + i * LANES < heads) {
                    const __nv_bfloat16* x = src + (h + i * LANES) * src_head;
                    lo[i] = *reinterpret_cast<const uint4*>(x + 8 * c);
                    hi[i] = *reinterpret_cast<const uint4*>(x + D / 2 + 8 * c);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int hh = h + i * LANES;
                if (hh >= heads) break;
                const uint32_t ia[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w}, ib[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
                uint32_t oa[4], ob[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a0 = bf16_lo(ia[e]), a1 = bf16_hi(ia[e]), b0 = bf16_lo(ib[e]), b1 = bf16_hi(ib[e]);
                    const float y0 = fmaf(a0, cs[e].x, -b0 * cs[e].y), y1 = fmaf(a1, cs[e].z, -b1 * cs[e].w);
                    nan = fmaf(y0 + y1, 0.f, nan);    // (a NaN in b shows in a's rotation too)
                    oa[e] = pack_f16x2_track(y0, y1, big);
                    ob[e] = pack_f16x2_track(fmaf(b0, cs[e].x, a0 * cs[e].y), fmaf(b1, cs[e].z, a1 * cs[e].w), big);
                }
                __half* o = is_k ? dst + hh * dst_head
                                 : dst + (int64_t)(hh >> gs) * p.max_rows * g * D + (hh & (g - 1)) * D;
                *reinterpret_cast<uint4*>(o + 8 * c) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
                *reinterpret_cast<uint4*>(o + D / 2 + 8 * c) = make_uint4(ob[0], ob[1], ob[2], ob[3]);
            }
        }
    }
    if (!(big < kF16Limit) || nan != nan) set_dev_error(kDevErrRange);
}

// ------------------------------------------------------------------ attention
struct ManyParams {
    const int32_t* plan;
    const int32_t* block_table;
    const int32_t* page_pos;
    const uint16_t* excl;       // or null
    const float* rope;
    __nv_bfloat16* out;
    float* part_o;              // [blocks][2][256][D]
    float2* part_ml;            // [blocks][2][256]
    int4* desc;                 // [blocks][2]: a run begun here that goes on: {last block << 8 | 255, first token, kv head, 0},
                                //   {new tokens, first row, 0, 0}
    int32_t n, max_pages, max_rows, hq, hkv, n_phys, max_pos, workers, blocks, tag, total_pages;
};

constexpr int kManyThreads = 448;
constexpr int kPairRows = 2 * kTileRows;

// One run, or the part of one this block has, as warp 9 hands it to the others.
struct ManyItem {
    int32_t req;                // < 0: no more
    int32_t kvh, pair;
    int32_t jb, n_loc;          // its key tiles
    int32_t seq, add, row_base, kpage;
    int32_t slot;               // partial result, or -1: the whole run
    int32_t single;             // all rows fit tile A: keys straight from the pages, rotated here
};

template <int D>
struct ManySmem {
    static constexpr int kHalves = D / 64;
    static constexpr int kQ = kTileRows * D * 2;
    static constexpr int kK = kTileKeys * D * 2;
    static constexpr int oK = 2 * kQ;
    static constexpr int oV = oK + 2 * kK;
    static constexpr int oMask = oV + 2 * kK;          // [2 stages] 128 exclusion bits
    static constexpr int oBar = oMask + 2 * 16;
    static constexpr int kNumBars = 48;
    static constexpr int oMisc = oBar + kNumBars * 8;
    static constexpr int oItem = oMisc + 64;
    static constexpr int kBytes = oItem + 2 * (int)sizeof(ManyItem);
    static constexpr int kAlloc = kBytes + 1024;
    static_assert(kAlloc <= 232448, "more dynamic shared memory than a GB300 block can have");
};

// A wait sees the parity of a phase only, so a phase may end at most once before each of its waiters has
// passed it.  What keeps each barrier to that:
//   Q, K, V, M, ITEM  a copy goes into a stage again only behind the stage's EMPTY, which every waiter on
//                     its FULL (RAW, ROT) has arrived on, whichever kind of run the tile belongs to;
//   S_FULL, P_FULL    the next Q K^T into a half waits for the P V that read it, that one for the P of every
//                     thread that read S;
//   PV_DONE           waited for by the next Q K^T into the half, and by softmax threads that rescale: those
//                     have seen S(h), whose Q K^T waited for P V(h - 2), and P V(h + 1) needs their P(h + 1);
//   O_DONE, O_FREE    take turns: every P V of a run, then every thread's epilogue, then the next run's P V.
//                     They count the runs their row tile takes part in.  Runs of one row tile are none of tile
//                     B's: an arrival for it then would be ordered behind V tiles only, not behind the P V of
//                     the run before, nor the waits for that run's result.
enum : int {
    MB_Q_FULL = 0, MB_Q_EMPTY = 1,
    MB_K_FULL = 2,      // [2]
    MB_K_EMPTY = 4,     // [2] both Q K^T that read the stage are done
    MB_V_FULL = 6,      // [2] the V tile is ready to be read
    MB_V_RAW = 8,       // [2] the copy of a V tile with rows to be zeroed landed
    MB_V_EMPTY = 10,    // [2]
    MB_M_FULL = 12,     // [2] the tile's exclusion bits (only where the call has them)
    MB_M_EMPTY = 14,    // [2] both softmax groups have read them
    MB_S_FULL = 16,     // [4] per (row tile, S half)
    MB_P_FULL = 20,     // [4]
    MB_PV_DONE = 24,    // [4]
    MB_O_DONE = 28,     // [2]
    MB_O_FREE = 30,     // [2]
    MB_DRAIN = 32,      // [4]
    MB_ITEM_FULL = 36,  // [2]
    MB_ITEM_EMPTY = 38, // [2]
    MB_K_RAW = 40,      // [2] single: the tile's pages landed
    MB_K_ROT = 42       // [2] single: rotated in place (every thread of warps 4-7)
};

// Larger of two fp16 and of the magnitudes of two others, NaN where one is.
__device__ __forceinline__ uint32_t max_abs_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b32 t;\n\tabs.f16x2 t, %2;\n\tmax.NaN.f16x2 %0, %1, t;\n\t}\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Warps 4-7 on a single-tile run: every key tile rotated in place, bf16 in, fp16 out.  Thread t has 16-byte
// chunk pair c (dimensions 8 c .. and d/2 + 8 c ..) of N consecutive keys of page t / 16: their angles
// start from the cos/sin row of the first one's position and advance by one position, a rotation by
// table row 1, from key to key.  Slots that take no part become zeros (they may hold anything).  A tile
// is rotated once for all its rows, beside the softmax of tile A: 3500 of the 4650 cycles a tile takes, the
// softmax 2500 of them.  Whether every result is finite is kept as the largest packed fp16 magnitudes (200 ->
// 194 us against a test of the fp32 values).  More code is slower, the roles' loops compete for the
// instruction cache: the next key loaded ahead 202 us, four keys unrolled instead of two 300.
template <int D>
__device__ __forceinline__ bool rotate_tiles(const ManyParams& prm, const ManyItem& w, uint8_t* stages, int stage_bytes,
                                             const uint16_t* s_mask, uint64_t* bars, int kc, int (&raw_n)[2], int t,
                                             int lane, volatile int* abort_flag) {
    constexpr int CP = D / 16, N = D / 16;              // chunk pairs of a row; keys a thread (16 threads a page)
    const int page = t / 16, c = t % 16 % CP, r0 = t % 16 / CP * N;
    const uint32_t o_hi = D == 128 ? 16384u : 0u;
    const int c_hi = D == 128 ? c : c + 4;
    const bool masked = prm.excl != nullptr;
    const int n_slots = w.seq + w.add, n_pages = pages_of(n_slots);
    const int32_t* pos_row = prm.page_pos + (int64_t)w.req * prm.max_pages;
    auto position = [&](int j) { return pos_row[min(j * kPagesPerTile + page, n_pages - 1)]; };
    auto in_table = [&](int32_t pos) { return pos >= 0 && pos <= prm.max_pos - kPage; };
    auto row_of = [&](int32_t pos, float4 (&v)[4]) {
        const float4* src = reinterpret_cast<const float4*>(prm.rope + (int64_t)(in_table(pos) ? pos + r0 : 0) * D + 16 * c);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = src[e];
    };
    uint64_t STC[4], STS[4];
    {
        const float4* one = reinterpret_cast<const float4*>(prm.rope + D + 16 * c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 v = one[e];
            STC[e] = f2_pack(v.x, v.z);
            STS[e] = f2_pack(v.y, v.w);
        }
    }
    // the position of a tile's page is loaded two tiles ahead, its cos/sin row one
    int32_t pos = position(w.jb), pos_n = position(w.jb + 1);
    float4 cs[4];
    row_of(pos, cs);
    uint32_t big = 0;                 // largest magnitudes, NaN where one was
    for (int jj = 0; jj < w.n_loc; ++jj, ++kc) {
        const int ks = kc & 1, first = (w.jb + jj) * kTileKeys + page * kPage;
        uint32_t gone = 0;
        if (!in_table(pos)) {
            set_dev_error(kDevErrBounds);
            gone = 0xFFFFu;
        }
        const int have = min(max(n_slots - first, 0), kPage);
        gone |= 0xFFFFu & ~((1u << have) - 1u);
        uint64_t C[4], S[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            C[e] = f2_pack(cs[e].x, cs[e].z);
            S[e] = f2_pack(cs[e].y, cs[e].w);
        }
        pos = pos_n;
        pos_n = position(w.jb + jj + 2);
        row_of(pos, cs);
        bool ok = mbar_wait(&bars[MB_K_RAW + ks], raw_n[ks]++ & 1, abort_flag);
        if (masked) {
            ok = ok && mbar_wait(&bars[MB_M_FULL + ks], (kc >> 1) & 1, abort_flag);
            if (__all_sync(0xffffffffu, ok)) gone |= s_mask[ks * 8 + page];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[MB_M_EMPTY + ks]);
        }
        if (!__all_sync(0xffffffffu, ok)) return false;
        uint8_t* stage = stages + ks * stage_bytes;
#pragma unroll 2
        for (int r = 0; r < N; ++r) {
            const int key = page * kPage + r0 + r;
            uint4* plo = reinterpret_cast<uint4*>(stage + sw128_off(key, c));
            uint4* phi = reinterpret_cast<uint4*>(stage + o_hi + sw128_off(key, c_hi));
            uint4 a = *plo, b = *phi;
            if (gone >> (r0 + r) & 1u) a = b = make_uint4(0, 0, 0, 0);
            const uint32_t ia[4] = {a.x, a.y, a.z, a.w}, ib[4] = {b.x, b.y, b.z, b.w};
            uint32_t oa[4], ob[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t A = bf16x2_to_f2(ia[e]), B = bf16x2_to_f2(ib[e]), minus = f2_pack(-1.f, -1.f);
                float y0, y1, z0, z1;
                f2_unpack(f2_fma(f2_mul(B, S[e]), minus, f2_mul(A, C[e])), y0, y1);   // a cos - b sin
                f2_unpack(f2_fma(A, S[e], f2_mul(B, C[e])), z0, z1);                   // b cos + a sin
                oa[e] = pack_f16x2_inf(y0, y1);
                ob[e] = pack_f16x2_inf(z0, z1);
                big = max_abs_f16x2(max_abs_f16x2(big, oa[e]), ob[e]);
                // one position further
                const uint64_t cn = f2_fma(f2_mul(S[e], STS[e]), minus, f2_mul(C[e], STC[e]));
                S[e] = f2_fma(C[e], STS[e], f2_mul(S[e], STC[e]));
                C[e] = cn;
            }
            *plo = make_uint4(oa[0], oa[1], oa[2], oa[3]);
            *phi = make_uint4(ob[0], ob[1], ob[2], ob[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(&bars[MB_K_ROT + ks]);
    }
    if ((big & 0x7C00u) == 0x7C00u || (big & 0x7C000000u) == 0x7C000000u) set_dev_error(kDevErrRange);   // not finite
    return true;
}

template <int D>
__global__ void __launch_bounds__(kManyThreads)
many_rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_kpool, const __grid_constant__ CUtensorMap tm_v,
                 const ManyParams prm) {
    using SM = ManySmem<D>;
    constexpr int H = SM::kHalves;
    constexpr int kReaders = 13;   // softmax warps, issuers, V producer
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    auto sQ = [&](int t) { return smem + t * SM::kQ; };
    auto sK = [&](int st) { return smem + SM::oK + st * SM::kK; };
    auto sV = [&](int st) { return smem + SM::oV + st * SM::kK; };
    uint16_t* s_mask = reinterpret_cast<uint16_t*>(smem + SM::oMask);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM::oBar);
    int32_t* misc = reinterpret_cast<int32_t*>(smem + SM::oMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
    ManyItem* slots = reinterpret_cast<ManyItem*>(smem + SM::oItem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        mbar_init(&bars[MB_Q_FULL], 1);
        mbar_init(&bars[MB_Q_EMPTY], 2);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars[MB_K_FULL + s], 1);
            mbar_init(&bars[MB_K_EMPTY + s], 2);
            mbar_init(&bars[MB_V_FULL + s], 1);
            mbar_init(&bars[MB_V_RAW + s], 1);
            mbar_init(&bars[MB_V_EMPTY + s], 2);
            mbar_init(&bars[MB_M_FULL + s], 1);
            mbar_init(&bars[MB_M_EMPTY + s], 8);
            mbar_init(&bars[MB_O_DONE + s], 1);
            mbar_init(&bars[MB_O_FREE + s], 128);
            mbar_init(&bars[MB_ITEM_FULL + s], 1);
            mbar_init(&bars[MB_ITEM_EMPTY + s], kReaders);
            mbar_init(&bars[MB_K_RAW + s], 1);
            mbar_init(&bars[MB_K_ROT + s], 128);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars[MB_S_FULL + i], 1);
            mbar_init(&bars[MB_P_FULL + i], 128);
            mbar_init(&bars[MB_PV_DONE + i], 1);
            mbar_init(&bars[MB_DRAIN + i], 1);
        }
        fence_mbar_init();
        misc[4] = 0;
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_kpool);
        prefetch_tmap(&tm_v);
    }
    grid_dep_wait();
    grid_dep_launch();
    const int4* entry = reinterpret_cast<const int4*>(prm.plan + plan_many(prm.n, prm.workers)) + 2 * blockIdx.x;
    const int4 share = entry[1];
    const int weight = share.y == prm.tag ? share.x : 0;
    if (warp == kWarpMma) {
        tmem_alloc(reinterpret_cast<uint32_t*>(misc), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(misc[0]);

    const int32_t* plan = prm.plan;
    const int g = prm.hq / prm.hkv, gs = __ffs(g) - 1;
    const int tpt = kTileRows >> gs, tpp = 2 * tpt;      // tokens of a row tile, of a pair
    const bool masked = prm.excl != nullptr;

    auto take_item = [&](int it, ManyItem& w) -> bool {
        if (!mbar_wait(&bars[MB_ITEM_FULL + (it & 1)], (it >> 1) & 1, abort_flag)) return false;
        w = slots[it & 1];
        return true;
    };

    if (weight == 0) {             // nothing to do for the whole block
        if (tid == 0) prm.desc[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    } else if (warp == kWarpTma) {
        // ------------------------------------------------------------ runs, Q and K tiles
        const int32_t* seq = plan + plan_array(CA_SEQ, prm.n);
        const int32_t* add = plan + plan_array(CA_NEW, prm.n);
        const int32_t* row = plan + plan_array(CA_ROW, prm.n);
        const int32_t* many = plan + plan_array(CA_MANY, prm.n);
        const int32_t* kpage = plan + plan_array(CA_KPAGE, prm.n);
        const int4 start = entry[0];
        int left = weight;
        int begins = share.z;              // weight of the run's beginning, where that is in this share
        int32_t req = start.x, kvh = start.y, pair = start.z, tile = start.w;
        int kc = 0, last_k[2] = {-1, -1}, last_q = -1, raw_n[2] = {0, 0}, full_n[2] = {0, 0};   // copies of either kind a stage took
        bool ok = true;
        int4 desc = make_int4(0, 0, 0, 0), desc_rows = desc;
        for (int it = 0; ok; ++it) {
            ManyItem w;
            left -= begins;
            w.req = left > 0 ? req : -1;
            w.kvh = kvh;
            w.pair = pair;
            w.jb = tile;
            w.n_loc = w.seq = w.add = w.row_base = w.kpage = 0;
            w.slot = -1;
            w.single = 0;
            if (left > 0) {
                w.seq = seq[req];
                w.add = add[req];
                w.row_base = row[req];
                w.kpage = kpage[req];
                w.single = w.add << gs <= kTileRows;
                const int all = many_tiles(w.seq, w.add, tpp, pair);
                w.n_loc = min(all - tile, left);
                left -= w.n_loc;
                if (w.n_loc < all) w.slot = 2 * blockIdx.x + (tile == 0 ? 1 : 0);
                if (tile == 0 && w.n_loc < all) {
                    // the block that holds the run's last tile
                    const int32_t u = many[req] + kvh * ((many[req + 1] - many[req]) / prm.hkv) +
                                      (int32_t)many_weight(w.seq, tpp, pair) + kPairWeight + all - 1;
                    desc = make_int4(Deal(many[prm.n], prm.blocks).owner(u) << 8 | 0xFF, pair * tpp, kvh, 0);
                    desc_rows = make_int4(w.add, w.row_base, 0, 0);
                }
            }
            if (lane == 0) {
                ok = it < 2 || mbar_wait(&bars[MB_ITEM_EMPTY + (it & 1)], ((it >> 1) - 1) & 1, abort_flag);
                if (ok) {
                    slots[it & 1] = w;
                    mbar_arrive(&bars[MB_ITEM_FULL + (it & 1)]);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok || w.req < 0) break;
            if (lane == 0) {
                const int32_t qy = (w.kvh * prm.max_rows + w.row_base + w.pair * tpp) * g;
                if (it > 0) ok = mbar_wait(&bars[MB_Q_EMPTY], (it - 1) & 1, abort_flag);
                if (ok) {
                    mbar_arrive_expect_tx(&bars[MB_Q_FULL], (w.single ? 1 : 2) * SM::kQ);
                    for (int t = 0; t < (w.single ? 1 : 2); ++t)
                        for (int hb = 0; hb < H; ++hb)
                            tma_load_2d(sQ(t) + hb * 16384, &tm_q, &bars[MB_Q_FULL], hb * 64, qy + t * kTileRows);
                    last_q = it;
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            const uint16_t* ex = masked ? prm.excl + (int64_t)w.req * prm.max_pages : nullptr;
            const int32_t* table = prm.block_table + (int64_t)w.req * prm.max_pages;
            const int n_pages = pages_of(w.seq + w.add), m = lane % kPagesPerTile, hb_l = lane / kPagesPerTile;
            int32_t ph_n = w.single ? table[min(w.jb * kPagesPerTile + m, n_pages - 1)] : 0;
            for (int jj = 0; jj < w.n_loc; ++jj, ++kc) {
                const int j = w.jb + jj, ks = kc & 1;
                int32_t ph = ph_n;
                if (ph < 0 || ph >= prm.n_phys) {
                    set_dev_error(kDevErrBounds);
                    ph = 0;
                }
                if (w.single && jj + 1 < w.n_loc) ph_n = table[min((j + 1) * kPagesPerTile + m, n_pages - 1)];
                uint32_t bits = 0;
                if (masked && lane < kPagesPerTile) {
                    const int pg = j * kPagesPerTile + lane;
                    if (pg < prm.max_pages) bits = ex[pg];
                }
                if (lane == 0) {
                    ok = kc < 2 || mbar_wait(&bars[MB_K_EMPTY + ks], ((kc >> 1) - 1) & 1, abort_flag);
                    if (ok && w.single) {
                        mbar_arrive_expect_tx(&bars[MB_K_RAW + ks], H * 16384);
                    } else if (ok) {
                        mbar_arrive_expect_tx(&bars[MB_K_FULL + ks], H * 16384);
                        const int32_t y = w.kvh * prm.total_pages * kPage + w.kpage * kPage + j * kTileKeys;
                        for (int hb = 0; hb < H; ++hb)
                            tma_load_2d(sK(ks) + hb * 16384, &tm_k, &bars[MB_K_FULL + ks], hb * 64, y);
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                if (w.single) {
                    if (lane < kPagesPerTile * H)
                        tma_load_2d(sK(ks) + hb_l * 16384 + m * (kPage * 128), &tm_kpool, &bars[MB_K_RAW + ks], hb_l * 64,
                                    (ph * prm.hkv + w.kvh) * kPage);
                    ++raw_n[ks];
                } else {
                    last_k[ks] = full_n[ks]++;
                }
                if (masked) {
                    ok = kc < 2 || mbar_wait(&bars[MB_M_EMPTY + ks], ((kc >> 1) - 1) & 1, abort_flag);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    if (lane < kPagesPerTile) s_mask[ks * 8 + lane] = (uint16_t)bits;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[MB_M_FULL + ks]);
                }
            }
            // the next run
            tile = 0;
            begins = kPairWeight;
            if (w.jb + w.n_loc == many_tiles(w.seq, w.add, tpp, pair) && ++pair == many_pairs(w.add, tpp)) {
                pair = 0;
                if (++kvh == prm.hkv) {
                    kvh = 0;
                    do { ++req; } while (req < prm.n && many[req + 1] == many[req]);
                }
            }
        }
        if (lane == 0) {
            prm.desc[2 * blockIdx.x] = ok ? desc : make_int4(0, 0, 0, 0);
            prm.desc[2 * blockIdx.x + 1] = desc_rows;
            if (last_q >= 0) mbar_drain(&bars[MB_Q_FULL], last_q & 1);
            for (int s = 0; s < 2; ++s) {
                if (last_k[s] >= 0) mbar_drain(&bars[MB_K_FULL + s], last_k[s] & 1);
                if (raw_n[s] > 0) mbar_drain(&bars[MB_K_RAW + s], (raw_n[s] - 1) & 1);
            }
        }
    } else if (warp == kWarpTmaV) {
        // ------------------------------------------------------------ V tiles
        // Lane 8 hb + m copies half hb of page m of the tile (a page behind the last one repeats it).
        // A tile with slots that take no part for any row -- excluded, or behind the last token --
        // lands on a barrier of this warp, which zeroes their rows (they may hold anything, and a
        // weight of zero does not silence a NaN) before it hands the tile on.
        int vc = 0, raw_n[2] = {0, 0};
        int last_v[2] = {-1, -1};        // last copy that landed on V_FULL itself
        bool ok = true;
        for (int it = 0; ok; ++it) {
            ManyItem w;
            ok = take_item(it, w);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[MB_ITEM_EMPTY + (it & 1)]);
            if (w.req < 0) break;
            const int n_slots = w.seq + w.add, n_pages = pages_of(n_slots);
            const int32_t* table = prm.block_table + (int64_t)w.req * prm.max_pages;
            const uint16_t* ex = masked ? prm.excl + (int64_t)w.req * prm.max_pages : nullptr;
            const int m = lane % kPagesPerTile, hb = lane / kPagesPerTile;
            int32_t ph_n = 0;
            uint32_t gone_n = 0;
            auto meta = [&](int j) {     // page m of tile j: its physical page, its slots without a part
                const int pg = j * kPagesPerTile + m;
                ph_n = table[min(pg, n_pages - 1)];
                const int have = min(max(n_slots - pg * kPage, 0), kPage);
                gone_n = 0xFFFFu & ~((1u << have) - 1u);
                if (ph_n < 0 || ph_n >= prm.n_phys) {    // (reported with its key; finite data instead)
                    ph_n = 0;
                    gone_n = 0xFFFFu;
                }
                if (masked && pg < n_pages) gone_n |= ex[pg];
            };
            meta(w.jb);
            for (int jj = 0; jj < w.n_loc; ++jj, ++vc) {
                const int vs = vc & 1;
                const int32_t ph = ph_n;
                const uint32_t gone = gone_n;
                const bool dirty = __any_sync(0xffffffffu, gone != 0u);
                uint64_t* bar = &bars[(dirty ? MB_V_RAW : MB_V_FULL) + vs];
                if (lane == 0) {
                    ok = vc < 2 || mbar_wait(&bars[MB_V_EMPTY + vs], ((vc >> 1) - 1) & 1, abort_flag);
                    if (ok) mbar_arrive_expect_tx(bar, H * 16384);
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                if (lane < kPagesPerTile * H)
                    tma_load_2d(sV(vs) + hb * 16384 + m * (kPage * 128), &tm_v, bar, hb * 64,
                                (ph * prm.hkv + w.kvh) * kPage);
                if (jj + 1 < w.n_loc) meta(w.jb + jj + 1);
                if (!dirty) {
                    last_v[vs] = vc;
                } else {
                    ok = mbar_wait(bar, raw_n[vs] & 1, abort_flag);
                    ++raw_n[vs];
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    // lanes m, m + 8, m + 16, m + 24 share page m's rows
                    for (uint32_t rest = gone; rest != 0u; rest &= rest - 1u) {
                        const int r = m * kPage + __ffs(rest) - 1;
                        for (int ch = lane / kPagesPerTile; ch < D / 8; ch += 32 / kPagesPerTile)
                            *reinterpret_cast<uint4*>(sV(vs) + (ch >> 3) * 16384 + sw128_off(r, ch & 7)) =
                                make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[MB_V_FULL + vs]);
                }
            }
        }
        if (lane == 0) {
            for (int s = 0; s < 2; ++s) {
                if (last_v[s] >= 0 && last_v[s] >= vc - 2) mbar_drain(&bars[MB_V_FULL + s], (last_v[s] >> 1) & 1);
                if (!ok && raw_n[s] > 0) mbar_drain(&bars[MB_V_RAW + s], (raw_n[s] - 1) & 1);
            }
        }
    } else if (warp >= kWarpMma) {
        // ------------------------------------------------------------ MMA issuers (8, 11: Q K^T; 12, 13: P V)
        const bool qk_role = warp == kWarpMma || warp == kWarpMmaB;
        const int t = (warp == kWarpMma || warp == kWarpPvA) ? 0 : 1;
        const uint32_t leader = lane == 0 ? 1u : 0u;
        int hq = 0, kc = 0, own = 0;                     // own: runs the row tile took part in
        int raw_n[2] = {0, 0}, full_n[2] = {0, 0};       // K tiles of either kind a stage held before
        bool ok = true;
        for (int it = 0; ok; ++it) {
            ManyItem w;
            ok = __all_sync(0xffffffffu, take_item(it, w));
            if (!ok) break;
            __syncwarp();
            if (leader) mbar_arrive(&bars[MB_ITEM_EMPTY + (it & 1)]);
            if (w.req < 0) break;
            const int nq = 2 * w.n_loc;
            auto wait_k = [&](int ks) {
                return w.single ? mbar_wait(&bars[MB_K_ROT + ks], raw_n[ks]++ & 1, abort_flag)
                                : mbar_wait(&bars[MB_K_FULL + ks], full_n[ks]++ & 1, abort_flag);
            };
            if (w.single && t == 1) {
                // tile B is not there: its issuers only take their part in the hand-offs of queries, keys and values
                for (int j = 0; ok && j < w.n_loc; ++j) {
                    const int kt = kc + j;
                    ok = __all_sync(0xffffffffu, qk_role ? wait_k(kt & 1)
                                                         : mbar_wait(&bars[MB_V_FULL + (kt & 1)], (kt >> 1) & 1, abort_flag));
                    if (ok && leader) mbar_arrive(&bars[(qk_role ? MB_K_EMPTY : MB_V_EMPTY) + (kt & 1)]);
                }
                if (ok && qk_role) ok = __all_sync(0xffffffffu, mbar_wait(&bars[MB_Q_FULL], it & 1, abort_flag));
                if (ok && qk_role && leader) mbar_arrive(&bars[MB_Q_EMPTY]);
                kc += w.n_loc;
                continue;
            }
            if (qk_role) {
                constexpr uint32_t idesc_qk = idesc_f16(128, 64);
                const uint32_t aQ = desc_sw128_lo(smem_u32(sQ(t)), 16);
                ok = __all_sync(0xffffffffu, mbar_wait(&bars[MB_Q_FULL], it & 1, abort_flag));
                for (int q = 0; ok && q < nq; ++q) {
                    const int hg = hq + q, kt = kc + (q >> 1), h = q & 1;
                    ok = __all_sync(0xffffffffu,
                                    (h == 1 || wait_k(kt & 1)) &&
                                        (hg < 2 || mbar_wait(&bars[MB_PV_DONE + 2 * t + (hg & 1)],
                                                             ((hg - 2) >> 1) & 1, abort_flag)));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t aK = desc_sw128_lo(smem_u32(sK(kt & 1)) + h * 64 * 128, 16);
                    const uint32_t tS = tmem + t * 128 + (hg & 1) * 64;
#pragma unroll
                    for (int k4 = 0; k4 < D / 64; ++k4)
                        mma_ss_k4(leader, tS, aQ + k4 * 1024, aK + k4 * 1024, kDescSw128Hi, idesc_qk, k4 > 0 ? 1u : 0u);
                    mma_commit_by(leader, &bars[MB_S_FULL + 2 * t + (hg & 1)]);
                    if (h == 1) mma_commit_by(leader, &bars[MB_K_EMPTY + (kt & 1)]);
                }
                if (ok) mma_commit_by(leader, &bars[MB_Q_EMPTY]);
            } else {
                constexpr uint32_t idesc_pv = idesc_bf16(128, D, true);
                const uint32_t tO = tmem + kTmemO + t * 128;
                for (int q = 0; ok && q < nq; ++q) {
                    const int hg = hq + q, kt = kc + (q >> 1), h = q & 1;
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(&bars[MB_P_FULL + 2 * t + (hg & 1)], (hg >> 1) & 1, abort_flag) &&
                                        (h == 1 || mbar_wait(&bars[MB_V_FULL + (kt & 1)], (kt >> 1) & 1, abort_flag)) &&
                                        (q > 0 || own == 0 ||
                                         mbar_wait(&bars[MB_O_FREE + t], (own - 1) & 1, abort_flag)));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t aV = desc_sw128_lo(smem_u32(sV(kt & 1)) + h * 64 * 128, 16384);
                    const uint32_t tP = tmem + t * 128 + (hg & 1) * 64;
                    mma_ts_k4(leader, tO, tP, aV, kDescSw128Hi, idesc_pv, q > 0 ? 1u : 0u);
                    mma_commit_by(leader, &bars[MB_PV_DONE + 2 * t + (hg & 1)]);
                    if (h == 1) mma_commit_by(leader, &bars[MB_V_EMPTY + (kt & 1)]);
                }
                if (ok) mma_commit_by(leader, &bars[MB_O_DONE + t]);
            }
            hq += nq;
            kc += w.n_loc;
            ++own;
        }
        const int di = (qk_role ? 0 : 2) + t;
        mma_commit_by(leader, &bars[MB_DRAIN + di]);
        if (leader) mbar_drain(&bars[MB_DRAIN + di], 0);
    } else {
        // ------------------------------------------------------------ softmax (warps 0-7)
        const int t = warp >> 2;
        const int m = tid - t * 128;                       // row of the tile = TMEM lane
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tO = tmem + lane_addr + kTmemO + t * 128;
        int hq = 0, kc = 0, own = 0;
        int raw_n[2] = {0, 0};
        float nan = 0.f;                                   // NaN where a result is not finite
        bool ok = true;
        for (int it = 0; ok; ++it) {
            ManyItem w;
            ok = take_item(it, w);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[MB_ITEM_EMPTY + (it & 1)]);
            if (w.req < 0) break;
            if (w.single && t == 1) {
                ok = rotate_tiles<D>(prm, w, sK(0), SM::kK, s_mask, bars, kc, raw_n, m, lane, abort_flag);
                if (!ok) break;
                kc += w.n_loc;
                continue;
            }
            const int tok = w.pair * tpp + t * tpt + (m >> gs);
            const bool valid = tok < w.add;
            const int limit = w.seq + min(tok, w.add - 1) + 1;   // slots the row sees
            float m_run = -INFINITY, l_run = 0.f;
            const int nq = 2 * w.n_loc;
            uint4 mask = make_uint4(0, 0, 0, 0);
            for (int q = 0; q < nq; ++q) {
                const int hg = hq + q, h = q & 1, ks = (kc + (q >> 1)) & 1;
                const uint32_t tS = tmem + lane_addr + t * 128 + (hg & 1) * 64;
                ok = mbar_wait(&bars[MB_S_FULL + 2 * t + (hg & 1)], (hg >> 1) & 1, abort_flag);
                if (masked && h == 0) ok = ok && mbar_wait(&bars[MB_M_FULL + ks], ((kc + (q >> 1)) >> 1) & 1, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                if (masked && h == 0) {
                    mask = *reinterpret_cast<const uint4*>(s_mask + ks * 8);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[MB_M_EMPTY + ks]);
                }
                const int cut = limit - (w.jb + (q >> 1)) * kTileKeys - 64 * h;   // the half's keys [0, cut) are seen
                const uint32_t m0 = h ? mask.z : mask.x, m1 = h ? mask.w : mask.y;
                const bool full = __all_sync(0xffffffffu, cut >= 64 && (m0 | m1) == 0u);
                uint32_t sv[64];
                tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
                tmem_ld_wait();
                if (!full) {
                    // keys behind the row's own token and excluded ones: score -inf
                    const uint32_t hide0 = m0 | (cut >= 32 ? 0u : cut <= 0 ? ~0u : ~0u << cut);
                    const uint32_t hide1 = m1 | (cut >= 64 ? 0u : cut <= 32 ? ~0u : ~0u << (cut - 32));
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        if (hide0 >> e & 1u) sv[e] = __float_as_uint(-INFINITY);
                        if (hide1 >> e & 1u) sv[32 + e] = __float_as_uint(-INFINITY);
                    }
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 64; e += 8) {
                    m4[0] = max3f(m4[0], __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                    m4[1] = max3f(m4[1], __uint_as_float(sv[e + 2]), __uint_as_float(sv[e + 3]));
                    m4[2] = max3f(m4[2], __uint_as_float(sv[e + 4]), __uint_as_float(sv[e + 5]));
                    m4[3] = max3f(m4[3], __uint_as_float(sv[e + 6]), __uint_as_float(sv[e + 7]));
                }
                const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                const float m_new = fmaxf(m_run, mx);
                const bool need = m_new > m_run + 8.0f;     // lazy rescale: keep P <= 2^8
                const float alpha = need ? ex2(m_run - m_new) : 1.0f;
                if (need) { l_run *= alpha; m_run = m_new; }
                const float msub = m_run == -INFINITY ? 0.f : m_run;
                const uint64_t negm2 = f2_pack(-msub, -msub);
                uint64_t acc2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    float d0, d1;
                    f2_unpack(f2_add(f2_pack(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), negm2), d0, d1);
                    const float p0 = ex2(d0), p1 = ex2(d1);
                    acc2[e & 1] = f2_add(acc2[e & 1], f2_pack(p0, p1));
                    pk[e] = pack_bf16x2(p0, p1);   // bf16 like the values they meet (an MMA's operands share a type)
                }
                tmem_st32(tS, pk);
                float a0, a1, b0, b1;
                f2_unpack(acc2[0], a0, a1);
                f2_unpack(acc2[1], b0, b1);
                l_run += (a0 + b0) + (a1 + b1);
                if (q > 0 && __any_sync(0xffffffffu, need)) {
                    // every earlier P V of this tile must be done before O is rescaled
                    ok = mbar_wait(&bars[MB_PV_DONE + 2 * t + ((hg - 1) & 1)], ((hg - 1) >> 1) & 1, abort_flag);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t o[32];
                        tmem_ld32(tO + cc * 32, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st32(tO + cc * 32, o);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bars[MB_P_FULL + 2 * t + (hg & 1)]);
            }
            if (!ok) break;
            // epilogue: O / l, or the part's sums as they are
            ok = mbar_wait(&bars[MB_O_DONE + t], own & 1, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            tc_fence_after();
            if (w.slot >= 0) {
                const int64_t prow = (int64_t)w.slot * kPairRows + t * kTileRows + m;
                if (valid) prm.part_ml[prow] = make_float2(m_run, l_run);
#pragma unroll 1
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[32];
                    tmem_ld32(tO + cc * 32, o);
                    tmem_ld_wait();
                    if (valid) {
                        float* dst = prm.part_o + prow * D + cc * 32;
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<uint4*>(dst + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
            } else {
                const float inv = l_run > 0.f ? 1.0f / l_run : 0.f;
#pragma unroll 1
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[32];
                    tmem_ld32(tO + cc * 32, o);
                    tmem_ld_wait();
                    if (valid) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) nan = fmaf(__uint_as_float(o[e]), 0.f, nan);
                        __nv_bfloat16* dst = prm.out + ((int64_t)(w.row_base + tok) * prm.hq + w.kvh * g + (m & (g - 1))) * D + cc * 32;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint4 v;
                            v.x = pack_bf16x2(__uint_as_float(o[8 * e + 0]) * inv, __uint_as_float(o[8 * e + 1]) * inv);
                            v.y = pack_bf16x2(__uint_as_float(o[8 * e + 2]) * inv, __uint_as_float(o[8 * e + 3]) * inv);
                            v.z = pack_bf16x2(__uint_as_float(o[8 * e + 4]) * inv, __uint_as_float(o[8 * e + 5]) * inv);
                            v.w = pack_bf16x2(__uint_as_float(o[8 * e + 6]) * inv, __uint_as_float(o[8 * e + 7]) * inv);
                            *reinterpret_cast<uint4*>(dst + 8 * e) = v;
                        }
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(&bars[MB_O_FREE + t]);
            hq += nq;
            kc += w.n_loc;
            ++own;
        }
        if (nan != nan) set_dev_error(kDevErrRange);       // (a value that takes part is not finite)
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Blocks (j, y) add up the run that block j of many_rows_kernel began and left open, 8 rows of it each:
// its part, then those of the blocks behind up to the run's last.  A launch of its own, as the parts (up to
// 128 KB each) take the whole device's loads: the block that brings the last part adding them up instead, as
// the few-row kernel does with its 8 KB, took 28 us for nine short chunks against 22, 283 against 275 mixed.
template <int D>
__global__ void __launch_bounds__(256) many_join_kernel(const ManyParams p) {
    constexpr int ROWS = 256 / (D / 4);
    grid_dep_wait();
    grid_dep_launch();
    const int j = blockIdx.x;
    const int4 d = p.desc[2 * j], rows = p.desc[2 * j + 1];
    if (d.x == 0) return;
    const int last = d.x >> 8;
    const int g = p.hq / p.hkv, gs = __ffs(g) - 1;
    const int r = blockIdx.y * ROWS + threadIdx.x / (D / 4), f = threadIdx.x % (D / 4);
    const int tok = d.y + (r >> gs);
    if (tok >= rows.x) return;
    float top = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b0 = j; b0 <= last; b0 += 2) {            // two parts' loads in flight: most runs have no more
        float2 ml[2];
        float4 v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // (behind the last part: that part again, without weight -- other memory may hold NaN)
            const int b = min(b0 + i, last);
            const int64_t row = ((int64_t)b * 2 + (b == j ? 1 : 0)) * kPairRows + r;
            ml[i] = p.part_ml[row];
            v[i] = *reinterpret_cast<const float4*>(p.part_o + row * D + 4 * f);
            if (b0 + i > last) ml[i].x = -INFINITY;
        }
        add_parts(ml, v, top, l, acc);
    }
    const float odd = not_finite(acc, 0.f);
    if (odd != odd) set_dev_error(kDevErrRange);
    const float inv = l > 0.f ? 1.0f / l : 0.f;
    const int64_t row = (int64_t)(rows.y + tok) * p.hq + d.z * g + (r & (g - 1));
    *reinterpret_cast<uint2*>(p.out + row * D + 4 * f) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

}  // namespace pcf
