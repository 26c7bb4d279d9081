// Attention of requests with few new rows (single tokens, drafts) over their pages.
//
// Row i is token s + t of request b (s tokens held before the chunk): for query head h of kv head
// h / g, over the slots j <= s + t of b whose page does not exclude them,
//   out = sum_j softmax_j((R_pos(i) q) . (R_(page_pos + r) k_j) / sqrt(d)) v_j,
// a row with no slot left giving zeros.
//
// What bounds it: every (page, kv head) -- 16 keys and values, 4 d bytes a token -- is read once and
// meets at most 16 rows, so HBM bounds it and the arithmetic only has to keep out of the way.  One block
// an SM, twelve warps, each a worker of its own: the units of all requests, in (request, kv head, page)
// order, are dealt to the workers in contiguous shares of equal weight by pcf_chunk_tables, whatever the lengths.
// Lane l of a worker holds the table entry of the l-th page ahead and copies it by TMA (128-byte
// swizzled) with the cos/sin row of the page's first position, into a ring of the worker's own, so no
// warp waits for another and an SM has more than 100 KB on the way.
//
// The keys are rotated in registers: the fragments of mma.m16n8k16's A operand (m = the page's 16 keys,
// k = d) that ldmatrix gives a thread hold dimensions i and i + d/2 of the same key, so a pair turns
// inside one thread.  The angle of slot r is that of the page's first position plus r steps:
// (C + iS)(c_r + i s_r) with the table row copied beside the page and rows 0..15 kept in shared
// memory -- four more multiply-adds a pair instead of sixteen table rows (8 KB at d = 128, as much as
// the unit itself) a page.  S^T = K Q^T (fp16) takes the rows as its 8-wide side, so 8 or 16 rows cost
// one or two products a step (rotated operands are fp16, 11 bits instead of bf16's 8: a score's error then
// stays below that of the inputs; out of its range is reported); the running maximum and sum of the softmax
// stay in registers (rescaled only when the maximum grows by more than 2^8), P^T in bf16 becomes the B operand of O^T +=
// V^T P^T by an 8 x 8 transpose in registers (movmatrix).  The sum takes the rounded weights, so here a
// row with one dominant key is exact.  A tcgen05 tile of 128 rows would be nine tenths padding here.
//
// A run of a (request, kv head) that lies within one worker is written out directly.  Otherwise the
// block joins its warps' partial results through shared memory and passes on at most two (the run
// it shares with the block before and with the block behind); the block that brings a run's last part
// adds them up.  Every sum has a fixed order, so results do not depend on timing.
//
// Measured (32/8 heads, d 128, graph replay): one token behind 33 k: 32 us for 135 MB, 20 of them at the copy
// rate, the others the way to the first page (2.6), the ramp and the joins (a block's and, behind a fence and
// a counter, the run's: some 5).  Behind 4 k: 11.7 us for 17 MB, all latency.  64 requests of 17 k tokens on
// shared spans (64/8 heads): 665 us for 4.8 GB of pages, a third of it found in L2; the copies alone take 609.
// 48 drafts of up to four tokens behind 100 to 9000 (two row tiles): 134 us for 737 MB, 109 at the copy rate;
// 32 requests behind 16 k: 91 % of the copy rate with one row tile and 92 % with two; 64 requests at d 64: 90 %
// and 78 % (half the bytes a key, the same instructions for its softmax).
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
    float* worker_o;            // [workers][8 NQ][D]
    float* block_o;             // [blocks][2][8 NQ][D]
    float2* block_ml;           // [blocks][2][8 NQ]
    int32_t* count;             // [blocks] parts brought of the run that begins in a block and goes on
    int64_t q_stride;
    int32_t n, max_pages, hq, hkv, n_phys, max_pos, tag;
};


template <int D, int NQ>
struct FewSmem {
    static constexpr int kWarps = kFewWarps;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kHalf = kPage * 128;                       // 16 rows of 64 elements
    static constexpr int kK = kPage * D * 2;
    static constexpr int kCs = D * 4;                               // cos/sin row
    // B fragments of a warp's rows: in registers with one tile of 8 rows, here with more
    static constexpr int kQ = NQ > 1 ? NQ * (D / 32) * 512 : 0;
    static constexpr int kTabRow = D * 4 + 64;                      // rows 64 bytes apart modulo 128
    static constexpr int kMl = 2 * 8 * NQ * 8;
    static constexpr int kFixed = kPage * kTabRow + kWarps * (kQ + kMl + 2 * 16) + 1024 + 64;
    // stages of the ring: whole units while they fit, then one more key than values
    static constexpr int kKeyStage = kK + kCs + 16, kValueStage = kK + 8;
    static constexpr int kRoom = (232448 - kFixed) / kWarps;
    static constexpr int kUnits = kRoom / (kKeyStage + kValueStage);
    static constexpr int kStagesV = kUnits >= 4 ? 4 : kUnits >= 2 ? 2 : 1;    // powers of two: slots are masks
    static constexpr int kStagesK = kStagesV > 1 ? kStagesV : 2;
    static_assert(kStagesK * kKeyStage + kStagesV * kValueStage <= kRoom, "the ring needs two keys and a value");
    static constexpr int kRing = (kStagesK + kStagesV) * kK;        // a warp's keys, then its values
    static_assert(kRing >= 8 * NQ * D * 4, "a worker's partial result fits its ring");
    static constexpr int oCs = kWarps * kRing;
    static constexpr int oTab = oCs + kWarps * kStagesK * kCs;
    static constexpr int oQ = oTab + kPage * kTabRow;
    static constexpr int oMl = oQ + kWarps * kQ;
    static constexpr int oDesc = oMl + kWarps * kMl;
    static constexpr int oBar = oDesc + kWarps * 2 * 16;
    static constexpr int oMeta = oBar + kWarps * (kStagesK + kStagesV) * 8;
    static constexpr int oAbort = oMeta + kWarps * kStagesK * 8;
    static constexpr int kBytes = oAbort + 16;                      // the abort flag, two flags of the join
    static constexpr int kAlloc = kBytes + 1024;
    static_assert(kAlloc <= 232448, "more dynamic shared memory than a GB300 block can have");
    static_assert(kThreads * 24 <= kWarps * kRing, "the join's shared memory is the ring's");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
// two packed fp32 pairs, 16 bytes
__device__ __forceinline__ void lds_pair(uint32_t addr, uint64_t& a, uint64_t& b) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint64_t f2_neg(uint64_t v) {
    float a, b;
    f2_unpack(v, a, b);
    return f2_pack(-a, -b);
}
// to fp16 with infinities kept (a key beyond the range shows in its scores)
__device__ __forceinline__ uint32_t pack_f16x2_inf(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// 8 x 8 matrix of 16-bit elements, a fragment's row lane / 4 and columns 2 (lane % 4), + 1: transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
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

// Partial results of a row (maximum and sum; weighted values) joined onto a running one, in their order; a
// part without a maximum adds nothing.
template <int N>
__device__ __forceinline__ void add_parts(const float2 (&ml)[N], const float4 (&v)[N], float& top, float& l, float4& acc) {
    float now = top;
#pragma unroll
    for (int i = 0; i < N; ++i) now = fmaxf(now, ml[i].x);
    const float ref = now == -INFINITY ? 0.f : now, old = ex2(top - ref);
    top = now;
    l *= old;
    acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float a = ex2(ml[i].x - ref);
        acc.x += a * v[i].x;
        acc.y += a * v[i].y;
        acc.z += a * v[i].z;
        acc.w += a * v[i].w;
        l += a * ml[i].y;
    }
}

// `nan`, or NaN where one of the sums is not finite.
__device__ __forceinline__ float not_finite(const float4& v, float nan) {
    return fmaf(v.x, 0.f, fmaf(v.y, 0.f, fmaf(v.z, 0.f, fmaf(v.w, 0.f, nan))));
}

// The ring's barriers and copies by shared-memory address: the loop keeps those in registers, where a
// generic pointer would take two and a conversion at every use.
__device__ __forceinline__ void ring_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void ring_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void ring_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ bool ring_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.b32 %0, 1, 0, p;\n\t}\n"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// Bounded like mbar_wait (which says what happens when the limit runs out); the same answer in every lane.
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    if (__all_sync(0xffffffffu, ring_try(bar, parity))) return true;
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, ring_try(bar, parity))) {
        const bool late = clock64() - t0 > kWaitLimitCycles;
        if (__any_sync(0xffffffffu, late || *abort_flag)) {
            if (late) {
                *abort_flag = 1;
                set_dev_error(kDevErrTimeout);
            }
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ void sts_2(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ uint32_t lds_1(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// (cos, sin, cos', sin') of two frequencies rewritten as (cos, cos', sin, sin')
__device__ __forceinline__ void pair_cs(uint32_t addr) {
    asm volatile("{\n\t.reg .b32 a, b, c, d;\n\tld.shared.v4.b32 {a, b, c, d}, [%0];\n\t"
                 "st.shared.v4.b32 [%0], {a, c, b, d};\n\t}\n" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void sts_zero4(uint32_t addr) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}

// Where a worker stands in the units: page `page` of `pages` of kv head `kvh` of request `req`.
struct FewCursor {
    int32_t req, kvh, page, pages;
    // the run behind this one; the next request is the next one with few rows (units left say there is one)
    __device__ __forceinline__ void next_run(const int32_t* few, const int32_t* seq, const int32_t* add, int32_t hkv, int32_t n) {
        page = 0;
        if (++kvh < hkv) return;
        kvh = 0;
        do { ++req; } while (req < n && few[req + 1] == few[req]);
        if (req < n) pages = pages_of(seq[req] + add[req]);
    }
};

template <int D, int NQ>
__global__ void __launch_bounds__(FewSmem<D, NQ>::kThreads, 1)
few_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const FewParams p) {
    using SM = FewSmem<D, NQ>;
    constexpr int NK = SM::kStagesK, NV = SM::kStagesV, WARPS = SM::kWarps, THREADS = SM::kThreads;
    constexpr int KS = D / 16;       // k steps of K Q^T
    constexpr int MT = D / 16;       // 16-dimension tiles of O^T
    constexpr int J = D / 16;        // 8-frequency chunks: chunk j turns with chunk j + J
    constexpr int ROWS = 8 * NQ;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = lane >> 2, c = lane & 3;     // fragment coordinates
    uint64_t* bar_k = reinterpret_cast<uint64_t*>(smem + SM::oBar) + warp * (NK + NV);
    uint64_t* bar_v = bar_k + NK;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM::oAbort);
    uint8_t* ring = smem + warp * SM::kRing;
    const uint32_t a_bar_k = smem_u32(bar_k), a_bar_v = smem_u32(bar_v);
    const uint32_t a_ring = smem_u32(ring), a_ring_v = a_ring + NK * SM::kK;
    const uint32_t a_cs = smem_u32(smem + SM::oCs + warp * NK * SM::kCs);
    // per key slot: exclusion bits, and the pool row its value will be copied from
    const uint32_t a_meta = smem_u32(smem + SM::oMeta + warp * NK * 8);
    float2* s_ml = reinterpret_cast<float2*>(smem + SM::oMl);       // [warp][first, last][row]
    volatile int32_t* s_desc = reinterpret_cast<volatile int32_t*>(smem + SM::oDesc);   // [warp][2][4]
    if (lane == 0) {
        for (int s = 0; s < NK + NV; ++s) mbar_init(&bar_k[s], 1);
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
    const int worker = blockIdx.x * WARPS + warp;
    const int4* entry = reinterpret_cast<const int4*>(plan + plan_starts(p.n)) + 3 * worker;
    const int4 start = entry[0], first = entry[1];
    const int32_t end = entry[3].w;                 // units before the next worker
    // {tag; first and last block of the run this block's first unit belongs to, last of its last unit's}
    const int32_t tag = entry[2].x;
    const int4 share = reinterpret_cast<const int4*>(plan + plan_starts(p.n))[3 * blockIdx.x * WARPS + 2];
    if (tag != p.tag) set_dev_error(kDevErrBounds);
    const int n_units = tag == p.tag ? end - start.w : 0;
    // cos/sin of 0..15 steps, for everyone, as pairs: (cos, cos', sin, sin') of two frequencies
    for (int i = tid; i < kPage * D / 4; i += THREADS) {
        const int r = i / (D / 4), f = i % (D / 4);
        const float4 v = reinterpret_cast<const float4*>(p.rope)[i];
        *reinterpret_cast<float4*>(smem + SM::oTab + r * SM::kTabRow + f * 16) = make_float4(v.x, v.z, v.y, v.w);
    }

    // ---------------- the copies: unit i's key into slot i % NK, its value into slot i % NV (a key's slot
    // is free again a whole softmax and P V earlier)
    FewCursor is{start.x, start.y, start.z, first.x};
    // lane l holds the table entry of page is.page + l of the run: pool row of its head, cos/sin row, bits
    int32_t win_n = 0, win_at = 0;
    int32_t e_y = 0;
    const float* e_cs = p.rope;
    uint32_t e_ex = 0;
    auto look_up = [&]() {
        win_n = min(32, is.pages - is.page);
        win_at = 0;
        if (lane < win_n) {
            const int64_t e = (int64_t)is.req * p.max_pages + is.page + lane;
            int32_t ph = p.block_table[e], pos = p.page_pos[e];
            e_ex = p.excl ? p.excl[e] : 0u;
            if (ph < 0 || ph >= p.n_phys || pos < 0 || pos > p.max_pos - kPage) {
                set_dev_error(kDevErrBounds);
                ph = pos = 0;
                e_ex = 0xFFFFu;                    // nothing of it takes part
            }
            e_y = (ph * p.hkv + is.kvh) * kPage;
            e_cs = p.rope + (int64_t)pos * D;
        }
    };
    int issued_k = 0, issued_v = 0;
    auto issue_k = [&]() {
        if (lane == win_at) {
            const uint32_t s = (uint32_t)issued_k % NK, bar = a_bar_k + s * 8;
            sts_2(a_meta + s * 8, e_ex, (uint32_t)e_y);
            ring_expect(bar, SM::kK + SM::kCs);
#pragma unroll
            for (int hb = 0; hb < D / 64; ++hb) ring_load_2d(a_ring + s * SM::kK + hb * SM::kHalf, &tm_k, bar, hb * 64, e_y);
            ring_load(a_cs + s * SM::kCs, e_cs, SM::kCs, bar);
        }
        __syncwarp();
        ++issued_k;
        if (++win_at == win_n && issued_k < n_units) {
            is.page += win_n;
            if (is.page == is.pages) is.next_run(few, seq, add, p.hkv, p.n);
            look_up();
        }
    };
    auto issue_v = [&]() {
        if (lane == 0) {
            const uint32_t s = (uint32_t)issued_v % NV, bar = a_bar_v + s * 8;
            const int32_t y = (int32_t)lds_1(a_meta + (uint32_t)issued_v % NK * 8 + 4);
            ring_expect(bar, SM::kK);
#pragma unroll
            for (int hb = 0; hb < D / 64; ++hb) ring_load_2d(a_ring_v + s * SM::kK + hb * SM::kHalf, &tm_v, bar, hb * 64, y);
        }
        ++issued_v;
    };
    if (n_units > 0) look_up();
    // positions of the rows of a run (row 8 q + lane / 4); a row behind the last one, or one whose
    // position is out of range, has none and scores 0 everywhere
    int32_t s_len = first.y, t_len = first.z, r_base = first.w, n_rows = t_len * g;
    int32_t row_at[NQ];
    auto load_positions = [&]() {
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const int r = q * 8 + row;
            row_at[q] = r < n_rows ? p.row_pos[r_base + (r >> gs)] : -1;
            if (r < n_rows && (row_at[q] < 0 || row_at[q] >= p.max_pos)) {
                set_dev_error(kDevErrBounds);
                row_at[q] = -1;
            }
        }
    };
    if (n_units > 0) load_positions();
    if (!__syncthreads_or(n_units > 0)) return;        // nothing to do for the whole block

    // ---------------- the units
    const float scale = 1.4426950408889634f * (D == 128 ? 0.08838834764831845f : 0.125f);   // log2(e) / sqrt(d)
    FewCursor cu{start.x, start.y, start.z, first.x};
    // O^T, columns 2 c and 2 c + 1 of every row tile; the softmax of those two rows over this lane's keys
    float o[NQ][MT][4], m_run[NQ][2], l_run[NQ][2];
    uint32_t qf[2 * J];                                                     // NQ == 1: chunks of row lane / 4
    uint4* s_q = reinterpret_cast<uint4*>(smem + SM::oQ + warp * SM::kQ);   // NQ > 1, see below
    // where ldmatrix finds a lane's row: K matrices (low chunk, its neighbour, their partners) of keys
    // 0-7, V matrices (keys 0-7, 8-15 of two neighbouring chunks); 16-byte chunk x of a row sits at
    // x ^ (row & 7), so the chunk of a step is one exclusive or away
    const uint32_t k_off = (D == 128 ? (uint32_t)(lane >> 4) * SM::kHalf : 0u) + (lane & 7) * 128u +
                           ((((lane >> 3) & 1u) ^ (D == 128 ? 0u : (uint32_t)(lane >> 4) * 4u) ^ (lane & 7u)) << 4);
    const uint32_t v_off = (lane & 15) * 128u + (((uint32_t)(lane >> 4) ^ (lane & 7u)) << 4);
    float big = 0.f;                 // largest rotated query
    // sum of all scores (not finite where a key left fp16's range), and of 0 times all results (NaN where
    // a value that takes part is not finite)
    uint64_t seen = 0;
    int32_t seg_page = 0;
    bool open = false, ok = true;
    int done_k = 0, done_v = 0;
    int32_t clean_pages = 0;                                 // pages of the run that every row sees whole

    for (int i = 0; i < n_units; ++i) {
        if (!open) {
            // a run of one (request, kv head) begins: its rows' queries, rotated and scaled, as B
            // fragments (rows behind the last one zero)
            open = true;
            seg_page = cu.page;
            if (i > 0) {
                s_len = seq[cu.req];
                t_len = add[cu.req];
                r_base = base[cu.req];
                n_rows = t_len * g;
                load_positions();
            }
            clean_pages = (s_len + 1) / kPage;
            uint32_t x[NQ][2 * J];
            float4 w[NQ][J];
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const int r = q * 8 + row;
                const __nv_bfloat16* src = p.q + (r_base + (r >> gs)) * p.q_stride + (cu.kvh * g + (r & (g - 1))) * D + 2 * c;
                const float* cs = p.rope + (int64_t)row_at[q] * D + 4 * c;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    x[q][j] = x[q][j + J] = 0;
                    w[q][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (row_at[q] >= 0) {
                        x[q][j] = *reinterpret_cast<const uint32_t*>(src + 8 * j);
                        x[q][j + J] = *reinterpret_cast<const uint32_t*>(src + D / 2 + 8 * j);
                        w[q][j] = *reinterpret_cast<const float4*>(cs + 16 * j);
                    }
                }
            }
            // the first copies go out behind the first rows' loads, not before: 30 MB of them over the
            // whole device would make those wait
            if (i == 0)
                while (issued_k < NK && issued_k < n_units) {
                    issue_k();
                    if (issued_v < NV) issue_v();
                }
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const float a0 = bf16_lo(x[q][j]) * scale, a1 = bf16_hi(x[q][j]) * scale;
                    const float b0 = bf16_lo(x[q][j + J]) * scale, b1 = bf16_hi(x[q][j + J]) * scale;
                    const float4 v = w[q][j];
                    x[q][j] = pack_f16x2_track(fmaf(a0, v.x, -b0 * v.y), fmaf(a1, v.z, -b1 * v.w), big);
                    x[q][j + J] = pack_f16x2_track(fmaf(b0, v.x, a0 * v.y), fmaf(b1, v.z, a1 * v.w), big);
                }
                if constexpr (NQ > 1) {
                    // [pair of tiles][k step][lane]: both chunks of the k step, both tiles
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
                        reinterpret_cast<uint2*>(s_q + ((q >> 1) * KS + ks) * 32 + lane)[q & 1] =
                            make_uint2(x[q][2 * ks], x[q][2 * ks + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 2 * J; ++j) qf[j] = x[q][j];
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[q][mt][e] = 0.f;
                m_run[q][0] = m_run[q][1] = -INFINITY;
                l_run[q][0] = l_run[q][1] = 0.f;
            }
        }
        const uint32_t s_k = (uint32_t)i % NK, s_v = (uint32_t)i % NV;
        if (!(ok = ring_wait(a_bar_k + s_k * 8, (uint32_t)i / NK & 1u, abort_flag))) break;
        ++done_k;
        const uint32_t sk_a = a_ring + s_k * SM::kK, cs_a = a_cs + s_k * SM::kCs;
        if (lane < D / 4) pair_cs(cs_a + lane * 16);               // the page's cos/sin row, as pairs
        const uint32_t ex = lds_1(a_meta + s_k * 8);
        // every row sees every key of the page: nothing excluded and the page ends at or before the
        // first row's own slot
        const bool clean = ex == 0u && cu.page < clean_pages;
        // keys that no row may see: excluded, or behind the last token (the slot may hold anything)
        uint32_t gone = ex;
        const int32_t j0 = cu.page * kPage;                        // the page's first slot
        if (!clean) {
            const int left = s_len + t_len - j0;                   // slots of the page that hold tokens
            if (left < kPage) gone |= 0xFFFFu & ~((1u << left) - 1u);
        }
        if (gone != 0u) {
            // keys that take no part score 0 (whatever they hold) until the softmax drops them
            for (int q = lane; q < kPage * (D / 8); q += 32) {
                const int r = q / (D / 8), ch = q % (D / 8);
                if (gone >> r & 1u)
                    sts_zero4(sk_a + (ch >> 3) * SM::kHalf + sw128_off(r, ch & 7));
            }
        }
        __syncwarp();
        // S^T = K Q^T, keys 0-7 and 8-15 of the page: a k step of the lower half and its partner at a
        // time, in two chains of products
        float sc[NQ][2][4];
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[q][0][e] = sc[q][1][e] = 0.f;
        const uint32_t sk_u = sk_a + k_off;
        const uint32_t tab = smem_u32(smem + SM::oTab) + row * SM::kTabRow + c * 16, cs_u = cs_a + c * 16;
#pragma unroll
        for (int jj = 0; jj < J / 2; ++jj) {
            uint32_t kf[2][4];                                     // chunks 2 jj, 2 jj + 1, and theirs + J
            ldsm4(sk_u ^ (jj * 32), kf[0][0], kf[0][1], kf[0][2], kf[0][3]);
            ldsm4((sk_u + 1024) ^ (jj * 32), kf[1][0], kf[1][1], kf[1][2], kf[1][3]);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint64_t C0, S0;
                lds_pair(cs_u + (2 * jj + q) * 64, C0, S0);
                const uint64_t NS0 = f2_neg(S0);
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    uint64_t Cr, Sr;
                    lds_pair(tab + nt * 8 * SM::kTabRow + (2 * jj + q) * 64, Cr, Sr);
                    const uint64_t C = f2_fma(NS0, Sr, f2_mul(C0, Cr)), S = f2_fma(C0, Sr, f2_mul(S0, Cr));
                    const uint64_t A = bf16x2_to_f2(kf[nt][q]), B = bf16x2_to_f2(kf[nt][q + 2]);
                    float y0, y1, z0, z1;
                    f2_unpack(f2_fma(f2_mul(B, S), f2_pack(-1.f, -1.f), f2_mul(A, C)), y0, y1);   // a cos - b sin
                    f2_unpack(f2_fma(A, S, f2_mul(B, C)), z0, z1);           // a sin + b cos
                    kf[nt][q] = pack_f16x2_inf(y0, y1);
                    kf[nt][q + 2] = pack_f16x2_inf(z0, z1);
                }
            }
#pragma unroll
            for (int up = 0; up < 2; ++up) {
                const uint32_t a[4] = {kf[0][2 * up], kf[1][2 * up], kf[0][2 * up + 1], kf[1][2 * up + 1]};
                const int ks = jj + up * (KS / 2);
                if constexpr (NQ == 1) {
                    mma_f16_16816(sc[0][up], a, qf[2 * ks], qf[2 * ks + 1]);
                } else {
#pragma unroll
                    for (int q = 0; q < NQ; q += 2) {
                        const uint4 b = s_q[((q >> 1) * KS + ks) * 32 + lane];
                        mma_f16_16816(sc[q][up], a, b.x, b.y);
                        mma_f16_16816(sc[q + 1][up], a, b.z, b.w);
                    }
                }
            }
        }
        // K has been read (and the cos/sin row rewritten in place): the next key for its slot
        fence_proxy_async_smem();
        __syncwarp();
        if (issued_k < n_units) issue_k();
        // softmax of the unit's 16 keys: this lane has keys lane / 4 and + 8 of rows 2 c and 2 c + 1
        // The reference of a row's exponentials is any number near its running maximum: it moves only
        // when some score passes it by more than 2^8, so most units need no maximum over the lanes.
        uint32_t pf[NQ][2];
        float x[NQ][4];
        bool over = false;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[q][e] = sc[q][0][e] + sc[q][1][e];
            seen = f2_add(seen, f2_add(f2_pack(x[q][0], x[q][1]), f2_pack(x[q][2], x[q][3])));
            if (!clean) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = row + 8 * (e >> 1);
                    const int last = s_len + ((q * 8 + 2 * c + (e & 1)) >> gs) - j0;   // last slot of the page the row sees
                    if (key > last || (gone >> key & 1u)) x[q][e] = -INFINITY;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) over |= x[q][e] > m_run[q][e & 1] + 8.0f;
        }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(x[q][e], x[q][2 + e]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    if (mx > m_run[q][e] + 8.0f) {     // (the same for all lanes of a row)
                        const float al = ex2(m_run[q][e] - mx);
                        m_run[q][e] = mx;
                        l_run[q][e] *= al;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            o[q][mt][e] *= al;
                            o[q][mt][2 + e] *= al;
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float ms = m_run[q][e] == -INFINITY ? 0.f : m_run[q][e];
                x[q][e] = ex2(x[q][e] - ms);
                x[q][2 + e] = ex2(x[q][2 + e] - ms);
            }
            // bf16 like the values they meet (an MMA's operands share a type); summed as rounded
            const uint32_t w0 = pack_bf16x2(x[q][0], x[q][1]), w1 = pack_bf16x2(x[q][2], x[q][3]);
            l_run[q][0] += bf16_lo(w0) + bf16_lo(w1);
            l_run[q][1] += bf16_hi(w0) + bf16_hi(w1);
            pf[q][0] = transpose8(w0);
            pf[q][1] = transpose8(w1);
        }
        if (!(ok = ring_wait(a_bar_v + s_v * 8, (uint32_t)i / NV & 1u, abort_flag))) break;
        ++done_v;
        const uint32_t sv_a = a_ring_v + s_v * SM::kK;
        if (gone != 0u) {
            // values of keys that take no part must not meet a weight of zero
            for (int q = lane; q < kPage * (D / 8); q += 32) {
                const int r = q / (D / 8), ch = q % (D / 8);
                if (gone >> r & 1u)
                    sts_zero4(sv_a + (ch >> 3) * SM::kHalf + sw128_off(r, ch & 7));
            }
            fence_proxy_async_smem();              // before the slot's next copy
            __syncwarp();
        }
        // O^T += V^T P^T
        const uint32_t sv_u = sv_a + v_off;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            uint32_t a[4];                                         // (dims, keys): low/high dims, then high keys
            ldsm4_t((sv_u ^ ((2 * mt & 7) * 16)) + (mt >> 2) * SM::kHalf, a[0], a[2], a[1], a[3]);
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                mma_bf16_16816(o[q][mt], a, pf[q][0], pf[q][1]);
            }
        }
        __syncwarp();
        if (issued_v < issued_k) issue_v();

    // ---------------- the end of a run, or of the worker
        const bool last = i + 1 == n_units, ended = cu.page + 1 == cu.pages;
        if (ended || last) {
            const bool whole = ended && seg_page == 0;
            const int kind = seg_page > 0 ? 0 : 1;      // begun by a worker before, or here
            // a worker's last partial result takes its ring, an earlier one (its first run) the workspace
            float* part = last ? reinterpret_cast<float*>(ring) : p.worker_o + (int64_t)worker * ROWS * D;
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                float l[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l[e] = l_run[q][e];
                    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
                    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
                    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
                }
                if (whole) {
                    const float i0 = l[0] > 0.f ? 1.0f / l[0] : 0.f, i1 = l[1] > 0.f ? 1.0f / l[1] : 0.f;
                    const int r = q * 8 + row;                     // after the transpose: row, dimensions 2 c, + 1
                    uint32_t* dst = reinterpret_cast<uint32_t*>(
                        p.out + ((int64_t)(r_base + (r >> gs)) * p.hq + cu.kvh * g + (r & (g - 1))) * D + 2 * c);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const uint32_t w0 = transpose8(pack_bf16x2(o[q][mt][0] * i0, o[q][mt][1] * i1));
                        const uint32_t w1 = transpose8(pack_bf16x2(o[q][mt][2] * i0, o[q][mt][3] * i1));
                        seen = f2_fma(f2_pack(o[q][mt][0], o[q][mt][1]), f2_pack(0.f, 0.f), seen);
                        seen = f2_fma(f2_pack(o[q][mt][2], o[q][mt][3]), f2_pack(0.f, 0.f), seen);
                        if (r < n_rows) {
                            dst[8 * mt] = w0;
                            dst[8 * mt + 4] = w1;
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = q * 8 + 2 * c + e;
                        if (r < n_rows) {
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                part[r * D + 16 * mt + row] = o[q][mt][e];
                                part[r * D + 16 * mt + 8 + row] = o[q][mt][2 + e];
                            }
                            if (row == 0) s_ml[(warp * 2 + kind) * ROWS + r] = make_float2(m_run[q][e], l[e]);
                        }
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
        ++cu.page;
        if (ended && !last) cu.next_run(few, seq, add, p.hkv, p.n);
    }
    {
        float a, b;
        f2_unpack(seen, a, b);
        if (!(big < kF16Limit) || !(fabsf(a) + fabsf(b) < INFINITY)) set_dev_error(kDevErrRange);
    }
    if (!ok && lane == 0)        // an abort: the copies in flight land before the block exits
    {
        for (int i = done_k; i < issued_k; ++i) mbar_drain(&bar_k[i % NK], (i / NK) & 1);
        for (int i = done_v; i < issued_v; ++i) mbar_drain(&bar_v[i % NV], (i / NV) & 1);
    }
    __syncthreads();
    // ---------------- join the warps' partial results, run by run
    const bool aborted = *abort_flag != 0;
    float nan = 0.f;                                   // NaN where a result is not finite
    int rows_of[2] = {0, 0}, kvh_of[2] = {0, 0}, base_of[2] = {0, 0};   // of the runs other blocks hold parts of
    // bit 2 w: what warp w ends of a run begun before it; bit 2 w + 1: what it leaves open
    const int32_t state = lane < 2 * WARPS ? s_desc[lane * 4] : 0;
    const uint32_t present = __ballot_sync(0xffffffffu, state & 1), closing = __ballot_sync(0xffffffffu, state & 2);
    const uint32_t in_ring = __ballot_sync(0xffffffffu, state & 4);
    // a run's first part here: one left open, or the block's very first part where that is an end
    const uint32_t lowest = present & (0u - present);
    const uint32_t before = lowest & 0x55555555u;
    for (uint32_t todo = (present & 0xAAAAAAAAu) | before; todo != 0u; todo &= todo - 1u) {
        const int sb = __ffs(todo) - 1;
        const bool from_before = (before >> sb & 1u) != 0u;
        // its parts: this one, then what the warps behind (each has units, up to the last that does) end
        int np = 1;
        bool ended = (closing >> sb & 1u) != 0u;
        for (int w = (sb >> 1) + 1; w < WARPS && !ended && (present >> 2 * w & 1u); ++w, ++np)
            ended = (closing >> 2 * w & 1u) != 0u;
        const int32_t req = s_desc[sb * 4 + 1], kvh = s_desc[sb * 4 + 2];
        const int rows_run = s_desc[sb * 4 + 3] & 0xFF, rb = s_desc[sb * 4 + 3] >> 8;
        const int slot = blockIdx.x * 2 + (from_before ? 0 : 1);
        for (int idx = tid; idx < rows_run * (D / 4); idx += THREADS) {
            const int r = idx / (D / 4), f = idx % (D / 4);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float top = -INFINITY, l = 0.f;
            for (int x0 = 0; x0 < np; x0 += 4) {           // four parts' loads in flight
                float2 ml[4];
                float4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // (behind the last part: that part again, without weight -- other memory may hold NaN)
                    const int at = min(x0 + i, np - 1), w = (sb >> 1) + at, x = at == 0 ? sb : 2 * w;
                    const float* src = (in_ring >> x & 1u) ? reinterpret_cast<const float*>(smem + w * SM::kRing)
                                                           : p.worker_o + (int64_t)(blockIdx.x * WARPS + w) * ROWS * D;
                    ml[i] = s_ml[x * ROWS + r];
                    v[i] = *reinterpret_cast<const float4*>(src + r * D + 4 * f);
                    if (x0 + i >= np) ml[i].x = -INFINITY;
                }
                add_parts(ml, v, top, l, acc);
            }
            nan = not_finite(acc, nan);
            if (!from_before && ended) {
                const float inv = l > 0.f ? 1.0f / l : 0.f;
                *reinterpret_cast<uint2*>(p.out + ((int64_t)(rb + (r >> gs)) * p.hq + kvh * g + (r & (g - 1))) * D + 4 * f) =
                    make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            } else {
                *reinterpret_cast<float4*>(p.block_o + ((int64_t)slot * ROWS + r) * D + 4 * f) = acc;
                if (f == 0) p.block_ml[slot * ROWS + r] = make_float2(top, l);
            }
        }
        if (from_before || !ended) {
            const int which = from_before ? 0 : 1;
            rows_of[which] = rows_run;
            kvh_of[which] = kvh;
            base_of[which] = rb;
        }
    }
    // ---------------- runs that several blocks share: whoever brings the last part adds them up.  The
    // parts lie in the order of the blocks whoever adds them, so the sum does not depend on timing.
    // The counters are the plan's: cleared with it, and zero again behind every call.
    if (nan != nan) set_dev_error(kDevErrRange);       // (parts of other blocks are theirs to report)
    int* s_last = reinterpret_cast<int*>(smem + SM::oAbort) + 1;
    if (rows_of[0] + rows_of[1] == 0) return;         // (uniform over the block)
    __syncthreads();
    if (tid < 2 && rows_of[tid] > 0) {
        const int from = tid == 0 ? share.y : (int)blockIdx.x, n = (tid == 0 ? share.z : share.w) - from + 1;
        s_last[tid] = atomic_inc_acq_rel_gpu(p.count + from, n - 1) == n - 1 ? 1 : 0;
    }
    __syncthreads();
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const int rows = which ? rows_of[1] : rows_of[0];
        if (rows == 0 || s_last[which] == 0 || aborted) continue;
        const int from = which ? (int)blockIdx.x : share.y, to = which ? share.w : share.z;
        const int kvh = which ? kvh_of[1] : kvh_of[0], rb = which ? base_of[1] : base_of[0];
        // groups of threads take the parts side by side, four loads in flight a thread, and are joined in
        // shared memory in their order
        float4* s_acc = reinterpret_cast<float4*>(smem);
        float2* s_w = reinterpret_cast<float2*>(smem + THREADS * 16);
        const int cols = rows * (D / 4), width = min(cols, THREADS);
        const int groups = max(1, min(THREADS / cols, to - from + 1));
        for (int c0 = 0; c0 < cols; c0 += THREADS) {
            const int grp = tid / width, idx = c0 + tid - grp * width;
            const int r = idx / (D / 4), f = idx % (D / 4);
            const bool mine = grp < groups && idx < cols;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float top = -INFINITY, l = 0.f;
            if (mine)
                for (int b0 = from + grp; b0 <= to; b0 += 4 * groups) {
                    float2 ml[4];
                    float4 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int b = b0 + i * groups;
                        const int64_t at = (int64_t)(min(b, to) * 2 + (b == from ? 1 : 0)) * ROWS + r;
                        ml[i] = __ldcg(p.block_ml + at);
                        v[i] = __ldcg(reinterpret_cast<const float4*>(p.block_o + at * D) + f);
                        if (b > to) ml[i].x = -INFINITY;
                    }
                    add_parts(ml, v, top, l, acc);
                }
            s_acc[tid] = acc;
            s_w[tid] = make_float2(top, l);
            __syncthreads();
            if (mine && grp == 0) {
                float all = top;
                for (int q = 1; q < groups; ++q) all = fmaxf(all, s_w[q * cols + tid].x);
                const float ref = all == -INFINITY ? 0.f : all, a0 = ex2(top - ref);
                acc = make_float4(acc.x * a0, acc.y * a0, acc.z * a0, acc.w * a0);
                l *= a0;
                for (int q = 1; q < groups; ++q) {
                    const float2 w = s_w[q * cols + tid];
                    const float4 v = s_acc[q * cols + tid];
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
}

}  // namespace pcf
