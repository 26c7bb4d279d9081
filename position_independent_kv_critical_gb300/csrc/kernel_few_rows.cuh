// Attention of requests with few new rows (single tokens, drafts) over their pages.
//
// Row i is token s + t of request b (s tokens held before the chunk): for query head h of kv head
// h / g, over the slots j <= s + t of b whose page does not exclude them,
//   out = sum_j softmax_j((R_pos(i) q) . (R_(page_pos + r) k_j) / sqrt(d)) v_j,
// a row with no slot left giving zeros.
//
// What bounds it: every (page, kv head) -- 16 keys and values, 4 d bytes a token -- is read once and
// meets at most 32 rows, so HBM bounds it and the arithmetic only has to keep out of the way.  One
// block an SM, eight warps, each a worker of its own: the units of all requests, in (request, kv
// head, page) order, are dealt to the workers in equal contiguous runs by pcf_chunk_tables, whatever
// the lengths.  A worker keeps a ring of units in flight (its lane 0 copies K and V of a page by
// TMA, 128-byte swizzled, and the cos/sin row of the page's first position), so no warp waits for
// another and an SM has 8 x (stages - 1) units, 130 KB, on the way.
//
// The keys are rotated in registers: the fragment of mma.m16n8k16's B operand (k = d, n = keys)
// that ldmatrix gives a thread holds dimensions i and i + d/2 of the same key, so a pair turns inside
// one thread.  The angle of slot r is that of the page's first position plus r steps:
// (C + iS)(c_r + i s_r) with the table row copied beside the page and rows 0..15 kept in shared
// memory -- four more multiply-adds a pair instead of sixteen table rows (8 KB at d = 128, as much as
// the unit itself) a page.  S = Q K^T (fp16), the running maximum and sum of the softmax in registers
// (rescaled only when the maximum grows by more than 2^8), P in bf16 as the A operand of O += P V:
// the accumulator layout of S is the A layout of the next product, nothing goes through memory.  The
// sum takes the rounded weights, so a row with one dominant key is exact.  With 16 or 32 rows a tile
// mma.sync is the right size (64 tensor-pipe cycles of the some 350 an SM has per unit at full HBM
// rate); a tcgen05 tile of 128 rows would be nine tenths padding.
//
// A run of a (request, kv head) that lies within one worker is written out directly.  Otherwise the
// block joins its warps' partial results through shared memory and passes on at most two (the run
// it shares with the block before and with the block behind), which few_join_kernel adds up: every
// sum in a fixed order, so results do not depend on timing.
#pragma once
#include "chunk_format.h"
#include "kernel_chunk_tables.cuh"
#include "ptx.cuh"

namespace pcf {

struct FewParams {
    const int32_t* plan;
    const __nv_bfloat16* q;
    const int32_t* block_table;
    const int32_t* page_pos;
    const uint16_t* excl;       // or null
    const int32_t* row_pos;
    const float* rope;
    __nv_bfloat16* out;
    float* worker_o;            // [workers][16 MT][D]
    float* block_o;             // [blocks][2][16 MT][D]
    float2* block_ml;           // [blocks][2][16 MT]
    int4* block_desc;           // [blocks]: a run that starts here and goes on: {last block << 8 | 255, rows, kv head, first row}
    int64_t q_stride;
    int32_t n, max_pages, max_rows, hq, hkv, n_phys, max_pos, blocks;
};

constexpr int kFewThreads = kFewWarps * 32;

template <int D, int MT>
struct FewSmem {
    static constexpr int kHalf = kPage * 128;                       // 16 rows of 64 elements
    static constexpr int kK = kPage * D * 2;
    static constexpr int kSlot = 2 * kK;
    static constexpr int kCs = D * 4;                               // cos/sin row
    static constexpr int kQ = MT == 2 ? MT * (D / 16) * 512 : 0;    // A fragments of a warp's rows
    static constexpr int kTabRow = D * 4 + 64;                      // rows 64 bytes apart modulo 128
    static constexpr int kMl = 2 * 16 * MT * 8;
    static constexpr int kFixed = kPage * kTabRow + kFewWarps * (kQ + kMl + 2 * 16) + 1024 + 64;
    static constexpr int kPerStage = kFewWarps * (kSlot + kCs + 16);
    static constexpr int kFit = (232448 - kFixed) / kPerStage;
    static constexpr int kStages = kFit < 6 ? kFit : 6;
    static_assert(kStages >= 2, "the ring needs two stages");
    static_assert(kStages * kSlot >= 16 * MT * D * 4, "a worker's partial result fits its ring");
    static constexpr int oCs = kFewWarps * kStages * kSlot;
    static constexpr int oTab = oCs + kFewWarps * kStages * kCs;
    static constexpr int oQ = oTab + kPage * kTabRow;
    static constexpr int oMl = oQ + kFewWarps * kQ;
    static constexpr int oDesc = oMl + kFewWarps * kMl;
    static constexpr int oBar = oDesc + kFewWarps * 2 * 16;
    static constexpr int oMeta = oBar + kFewWarps * kStages * 8;
    static constexpr int oAbort = oMeta + kFewWarps * kStages * 4;
    static constexpr int kBytes = oAbort + 16;
    static constexpr int kAlloc = kBytes + 1024;
    static_assert(kAlloc <= 232448, "more dynamic shared memory than a GB300 block can have");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Where a worker stands in the units: page `page` of `pages` of kv head `kvh` of request `req`.
struct FewCursor {
    int32_t req, kvh, page, pages;
    __device__ __forceinline__ void open(const int32_t* seq, const int32_t* add) { pages = pages_of(seq[req] + add[req]); }
    // one unit on; the next request is the next one with few rows (units left guarantee there is one)
    __device__ __forceinline__ void step(const int32_t* few, const int32_t* seq, const int32_t* add, int32_t hkv, int32_t n) {
        if (++page < pages) return;
        page = 0;
        if (++kvh < hkv) return;
        kvh = 0;
        do { ++req; } while (req < n && few[req + 1] == few[req]);
        if (req < n) open(seq, add);
    }
};

template <int D, int MT>
__global__ void __launch_bounds__(kFewThreads, 1)
few_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const FewParams p) {
    using SM = FewSmem<D, MT>;
    constexpr int NS = SM::kStages;
    constexpr int KS = D / 16;       // k steps of Q K^T
    constexpr int NT = D / 8;        // 8-column tiles of O
    constexpr int J = D / 16;        // 8-frequency chunks: chunk j turns with chunk j + J
    constexpr int ROWS = 16 * MT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = lane >> 2, c = lane & 3;     // fragment coordinates
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM::oBar) + warp * NS;
    volatile uint32_t* meta = reinterpret_cast<volatile uint32_t*>(smem + SM::oMeta) + warp * NS;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM::oAbort);
    uint8_t* ring = smem + warp * NS * SM::kSlot;
    uint8_t* ring_cs = smem + SM::oCs + warp * NS * SM::kCs;
    float2* s_ml = reinterpret_cast<float2*>(smem + SM::oMl);       // [warp][first, last][row]
    volatile int32_t* s_desc = reinterpret_cast<volatile int32_t*>(smem + SM::oDesc);   // [warp][2][4]
    if (lane == 0) {
        for (int s = 0; s < NS; ++s) mbar_init(&bars[s], 1);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        for (int i = 0; i < 8; ++i) s_desc[warp * 8 + i] = 0;
        if (warp == 0) *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
    const int32_t* plan = p.plan;
    const int32_t* seq = plan + plan_array(CA_SEQ, p.n);
    const int32_t* add = plan + plan_array(CA_NEW, p.n);
    const int32_t* base = plan + plan_array(CA_ROW, p.n);
    const int32_t* few = plan + plan_array(CA_FEW, p.n);
    const int g = p.hq / p.hkv, gs = __ffs(g) - 1;   // g divides 128
    const bool fits = plan_fits(plan, p.n, p.max_pages, p.max_rows, p.hq, p.hkv, p.blocks * kFewWarps);
    const int worker = blockIdx.x * kFewWarps + warp;
    const int4 start = reinterpret_cast<const int4*>(plan + plan_starts(p.n))[2 * worker];
    const int4 first = reinterpret_cast<const int4*>(plan + plan_starts(p.n))[2 * worker + 1];
    const int n_units = fits ? start.w : 0;

    // ---------------- the copies: unit i of the worker into slot i % NS
    FewCursor is{start.x, start.y, start.z, first.x};
    int32_t win_req = -1, win_page = 0;            // the 32 table entries the lanes hold
    int32_t e_ph = 0, e_pos = 0;
    uint32_t e_ex = 0;
    auto issue = [&](int i) {
        if (is.req != win_req || is.page < win_page || is.page >= win_page + 32) {
            win_req = is.req;
            win_page = is.page;
            const int32_t pg = is.page + lane;
            e_ph = e_pos = 0;
            e_ex = 0;
            if (pg < is.pages) {
                const int64_t e = (int64_t)is.req * p.max_pages + pg;
                e_ph = p.block_table[e];
                e_pos = p.page_pos[e];
                if (p.excl) e_ex = p.excl[e];
                if (e_ph < 0 || e_ph >= p.n_phys || e_pos < 0 || e_pos > p.max_pos - kPage) {
                    set_dev_error(kDevErrBounds);
                    e_ph = e_pos = 0;
                    e_ex = 0xFFFFu;                // nothing of it takes part
                }
            }
        }
        const int src = is.page - win_page, s = i % NS;
        const int32_t ph = __shfl_sync(0xffffffffu, e_ph, src), pos = __shfl_sync(0xffffffffu, e_pos, src);
        const uint32_t ex = __shfl_sync(0xffffffffu, e_ex, src);
        if (lane == 0) {
            meta[s] = ex;
            mbar_arrive_expect_tx(&bars[s], SM::kSlot + SM::kCs);
            const int32_t y = (ph * p.hkv + is.kvh) * kPage;
#pragma unroll
            for (int hb = 0; hb < D / 64; ++hb)
                tma_load_2d(ring + s * SM::kSlot + hb * SM::kHalf, &tm_k, &bars[s], hb * 64, y);
            bulk_load(ring_cs + s * SM::kCs, p.rope + (int64_t)pos * D, SM::kCs, &bars[s]);
#pragma unroll
            for (int hb = 0; hb < D / 64; ++hb)
                tma_load_2d(ring + s * SM::kSlot + SM::kK + hb * SM::kHalf, &tm_v, &bars[s], hb * 64, y);
        }
        is.step(few, seq, add, p.hkv, p.n);
    };
    int issued = 0;
    for (; issued < NS && issued < n_units; ++issued) issue(issued);

    // cos/sin of 0..15 steps, for everyone
    for (int i = tid; i < kPage * D / 4; i += kFewThreads) {
        const int r = i / (D / 4), f = i % (D / 4);
        *reinterpret_cast<float4*>(smem + SM::oTab + r * SM::kTabRow + f * 16) =
            reinterpret_cast<const float4*>(p.rope)[i];
    }
    __syncthreads();

    // ---------------- the units
    const float scale = 1.4426950408889634f * (D == 128 ? 0.08838834764831845f : 0.125f);   // log2(e) / sqrt(d)
    FewCursor cu{start.x, start.y, start.z, first.x};
    float o[MT][NT][4], m_run[MT][2], l_run[MT][2];
    uint32_t qf[MT == 1 ? KS : 1][4];
    uint4* s_q = reinterpret_cast<uint4*>(smem + SM::oQ + warp * SM::kQ);   // MT == 2: [mt][ks][lane]
    float big = 0.f;
    int32_t seg_page = 0, s_len = 0, t_len = 0, r_base = 0, n_rows = 0;
    bool open = false, ok = true;
    int done = 0;

    for (int i = 0; i < n_units; ++i) {
        if (!open) {
            // a run of one (request, kv head) begins: its rows' queries, rotated and scaled, as A
            // fragments (rows behind the last one zero)
            open = true;
            seg_page = cu.page;
            s_len = i == 0 ? first.y : seq[cu.req];
            t_len = i == 0 ? first.z : add[cu.req];
            r_base = i == 0 ? first.w : base[cu.req];
            n_rows = t_len * g;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                uint32_t lo[2][J], hi[2][J];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = mt * 16 + e * 8 + row;
#pragma unroll
                    for (int j = 0; j < J; ++j) lo[e][j] = hi[e][j] = 0;
                    if (r < n_rows) {
                        const int t = r >> gs, h = cu.kvh * g + (r & (g - 1));
                        const int32_t pos = p.row_pos[r_base + t];
                        if (pos < 0 || pos >= p.max_pos) {
                            set_dev_error(kDevErrBounds);
                        } else {
                            const __nv_bfloat16* q = p.q + (r_base + t) * p.q_stride + h * D + 2 * c;
                            const float* cs = p.rope + (int64_t)pos * D + 4 * c;
#pragma unroll
                            for (int j = 0; j < J; ++j) {
                                const uint32_t a = *reinterpret_cast<const uint32_t*>(q + 8 * j);
                                const uint32_t b = *reinterpret_cast<const uint32_t*>(q + D / 2 + 8 * j);
                                const float4 w = *reinterpret_cast<const float4*>(cs + 16 * j);
                                const float a0 = bf16_lo(a) * scale, a1 = bf16_hi(a) * scale;
                                const float b0 = bf16_lo(b) * scale, b1 = bf16_hi(b) * scale;
                                lo[e][j] = pack_f16x2_track(fmaf(a0, w.x, -b0 * w.y), fmaf(a1, w.z, -b1 * w.w), big);
                                hi[e][j] = pack_f16x2_track(fmaf(b0, w.x, a0 * w.y), fmaf(b1, w.z, a1 * w.w), big);
                            }
                        }
                    }
                }
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    // dimensions 16 ks ..: chunks 2 ks and 2 ks + 1, from the lower or the upper half
                    const int j0 = (2 * ks) % J, j1 = (2 * ks + 1) % J;
                    const bool up = 2 * ks >= J;
                    const uint32_t f0 = up ? hi[0][j0] : lo[0][j0], f1 = up ? hi[1][j0] : lo[1][j0];
                    const uint32_t f2 = up ? hi[0][j1] : lo[0][j1], f3 = up ? hi[1][j1] : lo[1][j1];
                    if constexpr (MT == 1) {
                        qf[ks][0] = f0;
                        qf[ks][1] = f1;
                        qf[ks][2] = f2;
                        qf[ks][3] = f3;
                    } else {
                        s_q[(mt * KS + ks) * 32 + lane] = make_uint4(f0, f1, f2, f3);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
                m_run[mt][0] = m_run[mt][1] = -INFINITY;
                l_run[mt][0] = l_run[mt][1] = 0.f;
            }
        }
        const int s = i % NS;
        ok = mbar_wait(&bars[s], (i / NS) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        ++done;
        const uint32_t ex = meta[s];
        const int32_t j0 = cu.page * kPage;                        // the page's first slot
        uint8_t* sk = ring + s * SM::kSlot;
        uint8_t* sv = sk + SM::kK;
        // every row sees every key of the page: nothing excluded and the page ends at or before the
        // first row's own slot
        const bool clean = ex == 0u && j0 + kPage - 1 <= s_len;
        // keys that no row may see: excluded, or behind the last token (the slot may hold anything)
        uint32_t gone = ex;
        if (!clean) {
            const int left = s_len + t_len - j0;                   // slots of the page that hold tokens
            if (left < kPage) gone |= 0xFFFFu & ~((1u << left) - 1u);
            // their values must not meet a weight of zero
            for (int q = lane; q < kPage * (D / 8); q += 32) {
                const int r = q / (D / 8), ch = q % (D / 8);
                if (gone >> r & 1u)
                    *reinterpret_cast<uint4*>(sv + (ch >> 3) * SM::kHalf + sw128_off(r, ch & 7)) = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
        }
        // S = Q K^T, keys 0-7 and 8-15: a thread turns pairs of key row (+ 8)
        float sc[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[mt][nt][e] = 0.f;
        const uint32_t sk_u = smem_u32(sk), sv_u = smem_u32(sv);
        const float4* cs0 = reinterpret_cast<const float4*>(ring_cs + s * SM::kCs) + c;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            uint32_t kf[2 * J];                                    // chunk j: dimensions 8 j + 2 c, + 1
            {
                const int kr = nt * 8 + (lane & 7), ch = lane >> 3;
#pragma unroll
                for (int q = 0; q < 2 * J; q += 4) {
                    const int cc = q + ch;
                    ldsm4(sk_u + (cc >> 3) * SM::kHalf + sw128_off(kr, cc & 7), kf[q], kf[q + 1], kf[q + 2], kf[q + 3]);
                }
            }
            if (!clean && (gone >> (nt * 8 + row) & 1u)) {
#pragma unroll
                for (int q = 0; q < 2 * J; ++q) kf[q] = 0;
            }
            const float4* csr = reinterpret_cast<const float4*>(smem + SM::oTab + (nt * 8 + row) * SM::kTabRow) + c;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float4 u = cs0[4 * j], w = csr[4 * j];
                const float c0 = fmaf(u.x, w.x, -u.y * w.y), s0 = fmaf(u.y, w.x, u.x * w.y);
                const float c1 = fmaf(u.z, w.z, -u.w * w.w), s1 = fmaf(u.w, w.z, u.z * w.w);
                const float a0 = bf16_lo(kf[j]), a1 = bf16_hi(kf[j]);
                const float b0 = bf16_lo(kf[j + J]), b1 = bf16_hi(kf[j + J]);
                kf[j] = pack_f16x2_track(fmaf(a0, c0, -b0 * s0), fmaf(a1, c1, -b1 * s1), big);
                kf[j + J] = pack_f16x2_track(fmaf(b0, c0, a0 * s0), fmaf(b1, c1, a1 * s1), big);
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                if constexpr (MT == 1) {
                    mma_f16_16816(sc[0][nt], qf[ks], kf[2 * ks], kf[2 * ks + 1]);
                } else {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        if (mt > 0 && n_rows <= 16) continue;
                        const uint4 a = s_q[(mt * KS + ks) * 32 + lane];
                        const uint32_t af[4] = {a.x, a.y, a.z, a.w};
                        mma_f16_16816(sc[mt][nt], af, kf[2 * ks], kf[2 * ks + 1]);
                    }
                }
            }
        }
        // softmax of the unit's 16 keys
        uint32_t pf[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if (mt > 0 && n_rows <= 16) continue;
            if (!clean) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int last = s_len + ((mt * 16 + e * 8 + row) >> gs) - j0;   // last slot of the page the row sees
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int key = nt * 8 + 2 * c + x;
                            if (key > last || (gone >> key & 1u)) sc[mt][nt][2 * e + x] = -INFINITY;
                        }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(fmaxf(sc[mt][0][2 * e], sc[mt][0][2 * e + 1]), fmaxf(sc[mt][1][2 * e], sc[mt][1][2 * e + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const bool need = mx > m_run[mt][e] + 8.0f;
                if (__any_sync(0xffffffffu, need)) {
                    const float al = need ? ex2(m_run[mt][e] - mx) : 1.0f;
                    if (need) m_run[mt][e] = mx;
                    l_run[mt][e] *= al;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        o[mt][nt][2 * e] *= al;
                        o[mt][nt][2 * e + 1] *= al;
                    }
                }
                const float ms = m_run[mt][e] == -INFINITY ? 0.f : m_run[mt][e];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const uint32_t w = pack_bf16x2(ex2(sc[mt][nt][2 * e] - ms), ex2(sc[mt][nt][2 * e + 1] - ms));
                    l_run[mt][e] += bf16_lo(w) + bf16_hi(w);
                    pf[mt][2 * nt + e] = w;
                }
            }
        }
        // O += P V: column tiles two at a time
        {
            const int kr = lane & 15, up = lane >> 4;
#pragma unroll
            for (int nt = 0; nt < NT; nt += 2) {
                const int ch = nt + up;
                uint32_t v0, v1, v2, v3;
                ldsm4_t(sv_u + (ch >> 3) * SM::kHalf + sw128_off(kr, ch & 7), v0, v1, v2, v3);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if (mt > 0 && n_rows <= 16) continue;
                    mma_bf16_16816(o[mt][nt], pf[mt], v0, v1);
                    mma_bf16_16816(o[mt][nt + 1], pf[mt], v2, v3);
                }
            }
        }
        if (!clean) fence_proxy_async_smem();      // zeros written above, before the slot's next copy
        __syncwarp();
        if (issued < n_units) issue(issued++);

        // ---------------- the end of a run, or of the worker
        const bool last = i + 1 == n_units, ended = cu.page + 1 == cu.pages;
        if (ended || last) {
            const bool whole = ended && seg_page == 0;
            const int kind = seg_page > 0 ? 0 : 1;      // begun by a worker before, or here
            // a worker's last partial result takes its ring, an earlier one (its first run) the workspace
            float* part = last ? reinterpret_cast<float*>(ring) : p.worker_o + (int64_t)worker * ROWS * D;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float l = l_run[mt][e];
                    l += __shfl_xor_sync(0xffffffffu, l, 1);
                    l += __shfl_xor_sync(0xffffffffu, l, 2);
                    const int r = mt * 16 + e * 8 + row;
                    if (r < n_rows) {
                        if (whole) {
                            const float inv = l > 0.f ? 1.0f / l : 0.f;
                            uint32_t* dst = reinterpret_cast<uint32_t*>(
                                p.out + ((int64_t)(r_base + (r >> gs)) * p.hq + cu.kvh * g + (r & (g - 1))) * D + 2 * c);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                dst[4 * nt] = pack_bf16x2(o[mt][nt][2 * e] * inv, o[mt][nt][2 * e + 1] * inv);
                        } else {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                *reinterpret_cast<float2*>(part + r * D + nt * 8 + 2 * c) =
                                    make_float2(o[mt][nt][2 * e], o[mt][nt][2 * e + 1]);
                            if (c == 0) s_ml[(warp * 2 + kind) * ROWS + r] = make_float2(m_run[mt][e], l);
                        }
                    }
                }
            if (!whole && lane == 0) {
                volatile int32_t* d = s_desc + (warp * 2 + kind) * 4;
                d[0] = 1 | (ended ? 2 : 0) | (last ? 4 : 0);
                d[1] = cu.req;
                d[2] = cu.kvh;
                d[3] = r_base << 8 | n_rows;         // (rows of a chunk: below 2^22)
            }
            open = false;
        }
        cu.step(few, seq, add, p.hkv, p.n);
    }
    if (!(big < kF16Limit)) set_dev_error(kDevErrRange);
    if (!ok && lane == 0)        // an abort: the copies in flight land before the block exits
        for (int i = done; i < issued; ++i) mbar_drain(&bars[i % NS], (i / NS) & 1);
    __syncthreads();
    // ---------------- join the warps' partial results, run by run
    const bool aborted = *abort_flag != 0;
    int4 desc = make_int4(0, 0, 0, 0);
    // bit 2 w: what warp w ends of a run begun before it; bit 2 w + 1: what it leaves open
    const int32_t state = lane < 2 * kFewWarps ? s_desc[lane * 4] : 0;
    const uint32_t present = __ballot_sync(0xffffffffu, state & 1), closing = __ballot_sync(0xffffffffu, state & 2);
    const uint32_t in_ring = __ballot_sync(0xffffffffu, state & 4);
    // a run's first part here: one left open, or the block's very first part where that is an end
    const uint32_t lowest = present & (0u - present);
    const uint32_t before = lowest & 0x5555u;
    for (uint32_t todo = aborted ? 0u : (present & 0xAAAAu) | before; todo != 0u; todo &= todo - 1u) {
        const int sb = __ffs(todo) - 1;
        const bool from_before = (before >> sb & 1u) != 0u;
        uint32_t parts = 1u << sb;
        bool ended = (closing >> sb & 1u) != 0u;
        for (uint32_t rest = present & 0x5555u & ~((2u << sb) - 1u); rest != 0u && !ended; rest &= rest - 1u) {
            parts |= rest & (0u - rest);
            ended = (closing & rest & (0u - rest)) != 0u;
        }
        const int32_t req = s_desc[sb * 4 + 1], kvh = s_desc[sb * 4 + 2];
        const int rows_run = s_desc[sb * 4 + 3] & 0xFF, rb = s_desc[sb * 4 + 3] >> 8;
        const int slot = blockIdx.x * 2 + (from_before ? 0 : 1);
        for (int idx = tid; idx < rows_run * (D / 4); idx += kFewThreads) {
            const int r = idx / (D / 4), f = idx % (D / 4);
            float top = -INFINITY;
            for (uint32_t m = parts; m != 0u; m &= m - 1u) top = fmaxf(top, s_ml[(__ffs(m) - 1) * ROWS + r].x);
            const float ref = top == -INFINITY ? 0.f : top;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float l = 0.f;
            for (uint32_t m = parts; m != 0u; m &= m - 1u) {
                const int x = __ffs(m) - 1;
                const float2 ml = s_ml[x * ROWS + r];
                const float a = ex2(ml.x - ref);
                const float* src = (in_ring >> x & 1u)
                                       ? reinterpret_cast<const float*>(smem + (x >> 1) * NS * SM::kSlot)
                                       : p.worker_o + (int64_t)(blockIdx.x * kFewWarps + (x >> 1)) * ROWS * D;
                const float4 v = *reinterpret_cast<const float4*>(src + r * D + 4 * f);
                acc.x += a * v.x;
                acc.y += a * v.y;
                acc.z += a * v.z;
                acc.w += a * v.w;
                l += a * ml.y;
            }
            if (!from_before && ended) {
                const float inv = l > 0.f ? 1.0f / l : 0.f;
                *reinterpret_cast<uint2*>(p.out + ((int64_t)(rb + (r >> gs)) * p.hq + kvh * g + (r & (g - 1))) * D + 4 * f) =
                    make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            } else {
                *reinterpret_cast<float4*>(p.block_o + ((int64_t)slot * ROWS + r) * D + 4 * f) = acc;
                if (f == 0) p.block_ml[slot * ROWS + r] = make_float2(top, l);
            }
        }
        if (!from_before && !ended) {
            // the block that holds the run's last unit u: u's owner is the last worker whose first unit
            // is not behind it
            const int64_t units = few[p.n], active = few_active(units, p.blocks * kFewWarps);
            const int64_t u = few[req] + (int64_t)(kvh + 1) * pages_of(seq[req] + add[req]) - 1;
            desc = make_int4(((int)(((u + 1) * active - 1) / units) / kFewWarps) << 8 | 0xFF, rows_run, kvh, rb);
        }
    }
    if (tid == 0) p.block_desc[blockIdx.x] = desc;
}

// Block j adds up the run that block j of few_rows_kernel began and left open: its part, then those of
// the blocks behind up to the one that holds the run's last unit.  A run of a single long request has
// a part in every eighth block or so and few rows, so the parts are taken by groups of threads side by
// side, four loads in flight a thread, and the groups joined in shared memory in their order.
constexpr int kJoinThreads = 512;
template <int D, int MT>
__global__ void __launch_bounds__(kJoinThreads) few_join_kernel(const FewParams p) {
    constexpr int ROWS = 16 * MT;
    __shared__ float4 s_acc[kJoinThreads];
    __shared__ float2 s_w[kJoinThreads];
    grid_dep_wait();
    grid_dep_launch();
    const int j = blockIdx.x;
    const int4 d = p.block_desc[j];
    if (d.x == 0) return;
    const int last = d.x >> 8, rows = d.y, kvh = d.z, rb = d.w;
    const int g = p.hq / p.hkv, gs = __ffs(g) - 1;
    const int cols = rows * (D / 4);
    const int groups = max(1, min(kJoinThreads / cols, last - j + 1));
    for (int c0 = 0; c0 < cols; c0 += kJoinThreads) {
        const int grp = threadIdx.x / min(cols, kJoinThreads), idx = c0 + threadIdx.x - grp * min(cols, kJoinThreads);
        const int r = idx / (D / 4), f = idx % (D / 4);
        const bool mine = grp < groups && idx < cols;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float top = -INFINITY, l = 0.f;
        if (mine)
            for (int b0 = j + grp; b0 <= last; b0 += 4 * groups) {
                float2 ml[4];
                float4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int b = b0 + i * groups, slot = min(b, last) * 2 + (b == j ? 1 : 0);
                    ml[i] = p.block_ml[slot * ROWS + r];
                    v[i] = *reinterpret_cast<const float4*>(p.block_o + ((int64_t)slot * ROWS + r) * D + 4 * f);
                    if (b > last) ml[i].x = -INFINITY;
                }
                const float now = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), top);
                const float ref = now == -INFINITY ? 0.f : now, old = ex2(top - ref);
                top = now;
                l *= old;
                acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = ex2(ml[i].x - ref);
                    acc.x += a * v[i].x;
                    acc.y += a * v[i].y;
                    acc.z += a * v[i].z;
                    acc.w += a * v[i].w;
                    l += a * ml[i].y;
                }
            }
        s_acc[threadIdx.x] = acc;
        s_w[threadIdx.x] = make_float2(top, l);
        __syncthreads();
        if (mine && grp == 0) {
            float all = top;
            for (int q = 1; q < groups; ++q) all = fmaxf(all, s_w[q * cols + threadIdx.x].x);
            const float ref = all == -INFINITY ? 0.f : all, a0 = ex2(top - ref);
            acc = make_float4(acc.x * a0, acc.y * a0, acc.z * a0, acc.w * a0);
            l *= a0;
            for (int q = 1; q < groups; ++q) {
                const float2 w = s_w[q * cols + threadIdx.x];
                const float4 v = s_acc[q * cols + threadIdx.x];
                const float a = ex2(w.x - ref);
                acc.x += a * v.x;
                acc.y += a * v.y;
                acc.z += a * v.z;
                acc.w += a * v.w;
                l += a * w.y;
            }
            const float inv = l > 0.f ? 1.0f / l : 0.f;
            *reinterpret_cast<uint2*>(p.out + ((int64_t)(rb + (r >> gs)) * p.hq + kvh * g + (r & (g - 1))) * D + 4 * f) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        }
        __syncthreads();
    }
}

}  // namespace pcf
