// Attention of a tree of drafted tokens over the pages of its request and its own branches.
//
// Row i is node t of request b: for query head h of kv head h / g, over the slots j < seq and the slots
// seq + u of the nodes u that t goes on from (itself among them), without those the pages exclude,
//   out = sum_j softmax_j((R_pos(i) q) . (R_pos(j) k_j) / sqrt(d)) v_j,
// pos(j) = page_pos + r for a held slot and the node's own position for a node's; a row with no slot left
// gives zeros.
//
// A tree has a few to a few hundred rows a kv head, so a key meets 8 to 256 of them: HBM and the tensor
// cores bound it about alike at 256 rows (a unit of 64 keys and values, 32 KB at d = 128, takes an SM 1400
// cycles at the copy rate and its four products of two row tiles 1280), HBM alone below.  So the keys are
// rotated where they are used, in shared memory: no copy of them is written or read again.  One block an SM,
// twenty warps; a run is one (request, kv head, row pair) or the part of one that a block has, dealt by
// pcf_tree_tables in contiguous parts of equal weight.
//   warps  0-7   softmax of chain 0 (warps 0-3) and 1: S row from TMEM, excluded slots and other branches
//                hidden, online softmax (lazy rescale), P -> TMEM over the S columns, O epilogue
//   warps  8-15  two groups of four, units in turn: keys, bf16 in, rotated fp16 out; values of hidden slots
//                become zeros
//   warp  16     runs in order; a unit's four pages of keys (TMA), its hidden slots
//   warp  19     the same pages of values
//   warp  17     a run's queries (TMA, rotated by a kernel before), Q K^T issue (and the TMEM allocation)
//   warp  18     P V issue
// With more than 128 rows the chains are the pair's two row tiles and both take every unit.  With up to 128
// there is one tile, and the chains take its units in turn, each with sums of its own that meet in the
// epilogue: eight softmax warps share what four would do, and a unit's way through the chain
// (S -> softmax -> P -> P V -> next Q K^T) overlaps the other chain's.
// TMEM: chain t's two S buffers at columns t*128 + {0, 64}, O of chain 0 at 256, of chain 1 at 384; P (bf16
// pairs) overwrites the S it came from and is the A operand of O += P V.
//
// Measured (32/8 heads, d 128, graph replay): 24 requests behind 16 k tokens: 16 nodes 291 us, 5.4 TB/s or 80 % of a
// plain copy; 64 nodes (two row tiles) 393 us, 1024 TFLOP/s.  48 trees of 1 to 64 nodes behind 100 to 9000 tokens:
// 232 us for 872 MB.  64 requests of 16 nodes on shared spans (64/8 heads, 10 % of the slots excluded): 833 us for
// 4.75 GB, a third of it found in L2.  12 trees of 200 to 256 nodes (64/8 heads): 303 us, 738 TFLOP/s.
// What bounds it: with one row tile the copies and, next, the rotation (24 requests of 16 nodes: 276 us without its
// arithmetic); with two the chain of hand-offs through two S buffers (issue slots 52 % used, tensor pipe 40 %; 24
// requests of 64 nodes, 391 us in that run: 398 without the rotation's arithmetic, 385 without the softmax's, 368 with
// one product of each kind a unit).  The five roles' loops also compete for the
// instruction cache: unrolled further here and there they took 1316 us instead of 1149 on the shared requests, with
// 3.2 cycles an instruction waited for the next one instead of 0.7.  So loops are rolled where latency allows it.
#pragma once
#include "kernel_few_rows.cuh"
#include "kernel_many_rows.cuh"
#include "kernel_tree_tables.cuh"
#include "ptx.cuh"
#include "tree_format.h"

namespace pcf {

struct TreeParams {
    const int32_t* plan;
    const __nv_bfloat16* q;
    __half* q_rot;              // [Hkv][max_rows][g][D], scaled by log2(e) / sqrt(d)
    const int32_t* block_table;
    const int32_t* page_pos;
    const uint16_t* excl;       // or null
    const int32_t* row_pos;     // [max_rows] the nodes' positions
    const uint32_t* seen;       // [max_rows][words]
    const float* rope;
    __nv_bfloat16* out;
    float4* part_o;             // [blocks][2][D / 4][256]: a warp's rows side by side
    float2* part_ml;            // [blocks][2][256]
    int4* desc;                 // [blocks][2]: a run begun here that goes on: {last block << 8 | 255, first node, kv head, 0},
                                //   {nodes, first row, row pairs of its request, 0}
    int64_t q_stride;
    int32_t n, max_pages, max_rows, words, hq, hkv, n_phys, max_pos, blocks, tag;
};

constexpr int kTreeAttnThreads = 640;
constexpr int kTreeReaders = 18;    // warps that read a run: softmax, rotation, issuers

// One run, or the part of one this block has, as warp 16 hands it to the others.
struct TreeItem {
    int32_t req;                // < 0: no more
    int32_t kvh, pair;
    int32_t jb, n_loc;          // its units
    int32_t seq, add, row_base;
    int32_t slot;               // partial result, or -1: the whole run
    int32_t single;             // its rows fit one tile
    int32_t code;               // n_loc * 2 + single, -1: no more
    int32_t qy;                 // its first row among the rotated queries
};

template <int D>
struct TreeSmem {
    static constexpr int kQ = kTileRows * D * 2;
    static constexpr int kUnit = kTreeUnit * D * 2;
    // A page lands as one box of eight-row groups, a group's halves (64 dimensions, 128-byte rows) one behind the
    // other: half the copies of boxes of half a page, and groups kGroup bytes apart from page to page too, as the
    // products' operands want them.
    static constexpr int kPageBytes = kPage * D * 2, kGroup = 8 * D * 2, kHalf = 1024;
    // (both even: a stage then belongs to units of one parity)
    static constexpr int NK = D == 128 ? 6 : 12, NV = D == 128 ? 4 : 8;
    // Hidden slots of the units whose keys are here or on the way, read by the rotation and the softmax: unit u
    // enters its own behind Q K^T of unit u - NK, which came behind P V, and so the softmax, of unit
    // u - NK - 4 (a chain's two S buffers, units in turn) and before.
    static constexpr int kMeta = 2 * NK;
    static_assert(kMeta >= NK + 4, "a unit's entry lasts until its softmax is done");
    static constexpr int oK = 2 * kQ;
    static constexpr int oV = oK + NK * kUnit;
    static constexpr int oMl = oV + NV * kUnit;                // [128] chain 1's maximum and sum
    static constexpr int oMeta = oMl + kTileRows * 8;          // [kMeta] a unit's 64 hidden bits
    static constexpr int oItem = oMeta + kMeta * 8;
    static constexpr int oBar = oItem + 2 * (int)sizeof(TreeItem);
    // barriers
    static constexpr int B_ITEM_FULL = 0, B_ITEM_EMPTY = 2, B_Q_FULL = 4, B_Q_EMPTY = 5, B_S_FULL = 6, B_P_FULL = 10,
                         B_PV_DONE = 14, B_O_DONE = 18, B_O_FREE = 20, B_ML = 22, B_DRAIN = 23, B_K_RAW = 25,
                         B_K_ROT = B_K_RAW + NK, B_K_EMPTY = B_K_ROT + NK, B_V_RAW = B_K_EMPTY + NK,
                         B_V_FULL = B_V_RAW + NV, B_V_EMPTY = B_V_FULL + NV,
                         kNumBars = B_V_EMPTY + NV;
    static constexpr int oMisc = oBar + kNumBars * 8;          // TMEM address, abort flag
    static constexpr int kBytes = oMisc + 16;
    static constexpr int kAlloc = kBytes + 1024;
    static_assert(oBar % 8 == 0 && kAlloc <= 232448, "more dynamic shared memory than a GB300 block can have");
};

// A wait sees the parity of a phase only, so a phase may end at most once before each of its waiters has
// passed it.  What keeps each barrier to that:
//   ITEM, K_ROT, V_FULL   every waiter passes every phase;
//   K_RAW, V_RAW    a stage belongs to one rotating group (NK and NV are even), which passes every phase of it;
//   Q, S, P, PV_DONE, O_DONE, O_FREE   as in the many-row kernel: counted by the units and runs that a chain
//                   takes part in; in a run of one tile the warps of chain 0 arrive on both O_FREE;
//   ML              chain 1's sums of a run of one tile: written again only behind chain 1's next result, whose
//                   first P V waited for O_FREE, on which chain 0's warps arrive when they have read them.

// 16 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ uint4 lds_128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts_128(uint32_t addr, const uint4& v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y, int32_t z,
                                            int32_t u) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(u)
        : "memory");
}
// high word of a 128-byte-swizzled descriptor whose eight-row groups are `group` bytes apart
__device__ __forceinline__ constexpr uint32_t desc_sw128_hi(uint32_t group) {
    return (group >> 4) | (1u << (46 - 32)) | (2u << (61 - 32));
}
// One lane of the (whole) warp, the same one every time.  Copies and products are issued in its branch: the
// compiler then knows that one thread is there, and their operands go to uniform registers without a loop over
// the lanes (eight products of 64 keys took 1300 cycles with a predicate on lane 0, 600 so).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}\n" : "=r"(r)::"memory");
    return r != 0;
}
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; }
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// odd + 0 x: NaN in a half of `odd` once that half of an x was not finite
__device__ __forceinline__ uint32_t odd_f16x2(uint32_t x, uint32_t odd) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0), "r"(odd));
    return r;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void prefetch_l1(const void* src) { asm volatile("prefetch.global.L1 [%0];" ::"l"(src)); }

// Eight frequencies' cos and sin as packed pairs.
struct Angles {
    uint64_t C[4], S[4];
    __device__ __forceinline__ void set(const float4 (&cs)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            C[e] = f2_pack(cs[e].x, cs[e].z);
            S[e] = f2_pack(cs[e].y, cs[e].w);
        }
    }
    // further by the angles of `by`, whose negated sines are `ns`
    __device__ __forceinline__ void advance(const Angles& by, const uint64_t (&ns)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t c = f2_fma(S[e], ns[e], f2_mul(C[e], by.C[e]));
            S[e] = f2_fma(C[e], by.S[e], f2_mul(S[e], by.C[e]));
            C[e] = c;
        }
    }
    // 16-byte chunks a and b (dimensions i.. and i + d/2 ..) turned, to fp16; `odd` tells whether they are finite
    __device__ __forceinline__ void turn(uint4& a, uint4& b, uint32_t& odd) const {
        const uint64_t minus = f2_pack(-1.f, -1.f);
        const uint32_t ia[4] = {a.x, a.y, a.z, a.w}, ib[4] = {b.x, b.y, b.z, b.w};
        uint32_t oa[4], ob[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t A = bf16x2_to_f2(ia[e]), B = bf16x2_to_f2(ib[e]);
            float y0, y1, z0, z1;
            f2_unpack(f2_fma(f2_mul(B, S[e]), minus, f2_mul(A, C[e])), y0, y1);   // a cos - b sin
            f2_unpack(f2_fma(A, S[e], f2_mul(B, C[e])), z0, z1);                   // b cos + a sin
            oa[e] = pack_f16x2_inf(y0, y1);
            ob[e] = pack_f16x2_inf(z0, z1);
            odd = odd_f16x2(ob[e], odd_f16x2(oa[e], odd));
        }
        a = make_uint4(oa[0], oa[1], oa[2], oa[3]);
        b = make_uint4(ob[0], ob[1], ob[2], ob[3]);
    }
};

// What a node sees of the 64 slots from slot `first` on, the held ones and those behind the tree included:
// its bits (`words` of them at `seen`) from node u = first - seq on.
__device__ __forceinline__ uint64_t tree_window(const uint32_t* seen, int words, int u) {
    auto word = [&](int w) { return w >= 0 && w < words ? __ldcg(seen + w) : 0u; };
    if (u >= 0) {
        const int w = u >> 5, s = u & 31;
        const uint32_t x = word(w), y = word(w + 1), z = word(w + 2);
        return (uint64_t)__funnelshift_r(y, z, s) << 32 | __funnelshift_r(x, y, s);
    }
    const uint64_t x = (uint64_t)word(1) << 32 | word(0);      // (-64 < u: the slots before node 0 are held ones)
    return x << -u | ((1ull << -u) - 1);
}

// The nodes' queries rotated, a block 16 rows at a time: thread (r, c) turns the 16-byte chunks c and c + d / 16 of
// row r's heads, at one angle for all of them, two heads' loads in flight.  A kernel of its own, which runs while the
// attention starts and has its first keys copied: there it was a fifth of the code and 4000 to 9000 cycles a run
// (64 shared requests 1006 us so, 965 with this kernel; the largest trees 350 and 347, for 12 us of it).
template <int D>
__global__ void __launch_bounds__(256) tree_rotate_kernel(const TreeParams p) {
    constexpr int CP = D / 16, LANES = 256 / (16 * CP);       // heads side by side
    grid_dep_wait();
    grid_dep_launch();
    if (!tree_fits(p.plan, p.tag)) return;
    const int32_t rows = p.plan[T_ROWS];
    const int c = threadIdx.x % CP, r = threadIdx.x / CP % 16, h0 = threadIdx.x / (CP * 16);
    const int g = p.hq / p.hkv, gs = __ffs(g) - 1;
    const float scale = 1.4426950408889634f * (D == 128 ? 0.08838834764831845f : 0.125f);   // log2(e) / sqrt(d)
    uint32_t odd = 0;
    // (blockIdx.y: a share of the heads)
    const int per = (p.hq + gridDim.y - 1) / gridDim.y, head0 = blockIdx.y * per, head1 = min(p.hq, head0 + per);
    for (int32_t row = blockIdx.x * 16 + r; row < rows; row += gridDim.x * 16) {
        const int32_t pos = p.row_pos[row];
        const bool in_table = pos >= 0 && pos < p.max_pos;
        if (!in_table) set_dev_error(kDevErrBounds);
        const float4* src = reinterpret_cast<const float4*>(p.rope + (int64_t)(in_table ? pos : 0) * D + 16 * c);
        float4 f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[e] = src[e];
            f[e] = make_float4(f[e].x * scale, f[e].y * scale, f[e].z * scale, f[e].w * scale);
        }
        Angles a;
        a.set(f);
#pragma unroll 2
        for (int h = head0 + h0; h < head1; h += LANES) {
            const __nv_bfloat16* x = p.q + row * p.q_stride + (int64_t)h * D;
            uint4 lo = *reinterpret_cast<const uint4*>(x + 8 * c), hi = *reinterpret_cast<const uint4*>(x + D / 2 + 8 * c);
            a.turn(lo, hi, odd);
            __half* dst = p.q_rot + (((int64_t)(h >> gs) * p.max_rows + row) * g + (h & (g - 1))) * D;
            *reinterpret_cast<uint4*>(dst + 8 * c) = lo;
            *reinterpret_cast<uint4*>(dst + D / 2 + 8 * c) = hi;
        }
    }
    if (odd != 0u) set_dev_error(kDevErrRange);
}

template <int D>
__global__ void __launch_bounds__(kTreeAttnThreads, 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const TreeParams p) {
    using SM = TreeSmem<D>;
    constexpr int NK = SM::NK, NV = SM::NV, CP = D / 16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM::oBar);
    int32_t* misc = reinterpret_cast<int32_t*>(smem + SM::oMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
    TreeItem* slots = reinterpret_cast<TreeItem*>(smem + SM::oItem);
    uint2* s_meta = reinterpret_cast<uint2*>(smem + SM::oMeta);
    float2* s_ml = reinterpret_cast<float2*>(smem + SM::oMl);
    auto sK = [&](int st) { return smem + SM::oK + st * SM::kUnit; };
    auto sV = [&](int st) { return smem + SM::oV + st * SM::kUnit; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars[SM::B_ITEM_FULL + s], 1);
            mbar_init(&bars[SM::B_ITEM_EMPTY + s], kTreeReaders);
            mbar_init(&bars[SM::B_O_DONE + s], 1);
            mbar_init(&bars[SM::B_O_FREE + s], 4);
        }
        mbar_init(&bars[SM::B_Q_FULL], 1);
        mbar_init(&bars[SM::B_Q_EMPTY], 1);
        mbar_init(&bars[SM::B_ML], 4);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars[SM::B_S_FULL + i], 1);
            mbar_init(&bars[SM::B_P_FULL + i], 4);
            mbar_init(&bars[SM::B_PV_DONE + i], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&bars[SM::B_DRAIN + i], 1);
        for (int s = 0; s < NK; ++s) {
            mbar_init(&bars[SM::B_K_RAW + s], 1);
            mbar_init(&bars[SM::B_K_ROT + s], 4);
            mbar_init(&bars[SM::B_K_EMPTY + s], 1);
        }
        for (int s = 0; s < NV; ++s) {
            mbar_init(&bars[SM::B_V_RAW + s], 1);
            mbar_init(&bars[SM::B_V_FULL + s], 4);
            mbar_init(&bars[SM::B_V_EMPTY + s], 1);
        }
        fence_mbar_init();
        misc[1] = 0;
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    // The kernel before this one in the stream is tree_rotate_kernel, which lets this one start when everything
    // before it is done: only its own results, the rotated queries, have to be waited for (by warp 17, and below
    // where there is nothing to do, so that whatever waits for this kernel has waited for that one).  What earlier
    // kernels wrote is read past L1, which may hold it as it was before them, or behind a wait (the rotation).
    const int4* entry = reinterpret_cast<const int4*>(p.plan + tree_shares(p.n)) + 3 * blockIdx.x;
    const bool fits = __ldcg(p.plan + T_TAG) == p.tag;
    // (all of the share at once: where its first run begins, its weight, the first run's lengths)
    const int4 start = fits ? __ldcg(entry) : make_int4(0, 0, 0, 0), share = fits ? __ldcg(entry + 1) : start;
    const int4 lens = fits ? __ldcg(entry + 2) : start;
    const int weight = share.y == p.tag ? share.x : 0;
    if (weight == 0) {             // nothing to do for the whole block
        if (tid == 0) p.desc[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
        grid_dep_wait();
        grid_dep_launch();
        return;
    }
    grid_dep_launch();
    if (warp == 17) {
        tmem_alloc(reinterpret_cast<uint32_t*>(misc), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(misc[0]);
    const int g = p.hq / p.hkv, gs = __ffs(g) - 1;
    const int tpt = kTileRows >> gs, tpp = 2 * tpt;      // nodes of a row tile, of a pair

    auto take_item = [&](int it, TreeItem& w) -> bool {
        const bool ok = mbar_wait(&bars[SM::B_ITEM_FULL + (it & 1)], (it >> 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) return false;
        w = slots[it & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[SM::B_ITEM_EMPTY + (it & 1)]);
        return true;
    };
    // What an issuer needs of it: n_loc * 2 + single, -1 behind the last one.  (A reduction's result is known to be
    // the same in all lanes, and so is what follows from it: operands of an MMA that are not go through a loop
    // over the lanes.)
    auto take_code = [&](int it, int32_t& qy) -> int {
        const bool ok = mbar_wait(&bars[SM::B_ITEM_FULL + (it & 1)], (it >> 1) & 1, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) return -1;
        const int code = __reduce_max_sync(0xffffffffu, slots[it & 1].code);
        qy = __reduce_max_sync(0xffffffffu, slots[it & 1].qy);
        if (lane == 0) mbar_arrive(&bars[SM::B_ITEM_EMPTY + (it & 1)]);
        return code;
    };
    // An arrival for the whole warp, behind what its lanes did (one a thread would be 384 operations on shared memory
    // a unit).
    auto arrive_warp = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // units of a run that a chain takes, unit kc its first one
    auto chain_units = [&](const TreeItem& w, int kc, int t) { return !w.single ? w.n_loc : (w.n_loc + ((kc & 1) == t ? 1 : 0)) >> 1; };

    // Lane l holds page l of a window of eight units, and of the window behind it: its place in the pool, its
    // slots that no row sees.
    struct Window {
        int32_t y = 0, y_n = 0;
        uint32_t gone = 0, gone_n = 0;
    };
    auto look_up = [&](Window& v, const TreeItem& w, int u0) {
        const int pg = u0 * kTreePagesPerUnit + lane, n_slots = w.seq + w.add;
        v.gone_n = 0xFFFFu;
        v.y_n = 0;
        if (pg < pages_of(n_slots)) {
            const int64_t e = (int64_t)w.req * p.max_pages + pg;
            const int32_t x = __ldcg(p.block_table + e), pos = __ldcg(p.page_pos + e);
            const uint32_t ex = p.excl ? __ldcg(p.excl + e) : 0u;
            const int have = min(n_slots - pg * kPage, kPage);
            v.gone_n = ex | (0xFFFFu & ~((1u << have) - 1u));
            v.y_n = x;
            // (a page of nodes alone has positions of its own)
            if (x < 0 || x >= p.n_phys || (pg * kPage < w.seq && (pos < 0 || pos > p.max_pos - kPage))) {
                set_dev_error(kDevErrBounds);
                v.y_n = 0;
                v.gone_n = 0xFFFFu;                      // nothing of it takes part
            }
        }
        v.y_n = (v.y_n * p.hkv + w.kvh) * (D == 128 ? 2 : kPage);      // in the map's rows: groups of eight, or single ones
    };
    // unit jj of the run: the window moves on; the unit's pages and hidden bits (a reduction's result is known to be
    // the same in all lanes)
    auto next_unit = [&](Window& v, const TreeItem& w, int jj, int32_t (&y)[kTreePagesPerUnit]) {
        if ((jj & 7) == 0) {
            v.y = v.y_n;
            v.gone = v.gone_n;
            if (jj + 8 < w.n_loc) look_up(v, w, w.jb + jj + 8);
        }
        const int at = (jj & 7) * kTreePagesPerUnit;
#pragma unroll
        for (int m = 0; m < kTreePagesPerUnit; ++m) y[m] = __reduce_max_sync(0xffffffffu, lane == at + m ? v.y : 0);
        const uint32_t g0 = __shfl_sync(0xffffffffu, v.gone, at), g1 = __shfl_sync(0xffffffffu, v.gone, at + 1),
                       g2 = __shfl_sync(0xffffffffu, v.gone, at + 2), g3 = __shfl_sync(0xffffffffu, v.gone, at + 3);
        return make_uint2(g0 | g1 << 16, g2 | g3 << 16);
    };
    if (warp == 16 || warp == 19) {
        // ------------------------------------------------------------ runs, K copies (warp 16), V copies (warp 19)
        const bool val = warp == 19;
        const int stages = val ? NV : NK;
        uint8_t* ring = val ? sV(0) : sK(0);
        const CUtensorMap* map = val ? &tm_v : &tm_k;
        uint64_t* raw = &bars[val ? SM::B_V_RAW : SM::B_K_RAW];
        uint64_t* empty = &bars[val ? SM::B_V_EMPTY : SM::B_K_EMPTY];
        const int32_t* seq = p.plan + tree_array(TA_SEQ, p.n);
        const int32_t* add = p.plan + tree_array(TA_NEW, p.n);
        const int32_t* row = p.plan + tree_array(TA_ROW, p.n);
        const int32_t* work = p.plan + tree_array(TA_WORK, p.n);
        int left = weight, begins = share.z;             // weight of the run's beginning, where that is in this share
        int32_t req = start.x, kvh = start.y, pair = start.z, unit = start.w;
        int kc = 0, st = 0, turn = 0;                    // units, place in the ring, its turns
        bool ok = true;
        int4 open_run = make_int4(-1, 0, 0, 0), open_rows = open_run;    // the run begun here that goes on
        for (int it = 0; ok; ++it) {
            TreeItem w;
            left -= begins;
            w.req = left > 0 ? req : -1;
            w.kvh = kvh;
            w.pair = pair;
            w.jb = unit;
            w.n_loc = w.seq = w.add = w.row_base = 0;
            w.slot = -1;
            w.single = 0;
            int pairs = 1;
            if (left > 0) {
                const bool first = it == 0;              // (its lengths came with the share)
                w.seq = first ? lens.x : __ldcg(seq + req);
                w.add = first ? lens.y : __ldcg(add + req);
                w.row_base = first ? lens.z : __ldcg(row + req);
                w.single = min(tpp, w.add - pair * tpp) << gs <= kTileRows;
                pairs = tree_pairs(w.add, g);
                const int all = tree_units(w.seq + w.add);
                w.n_loc = min(all - unit, left);
                left -= w.n_loc;
                if (w.n_loc < all) w.slot = 2 * blockIdx.x + (unit == 0 ? 1 : 0);
                if (unit == 0 && w.n_loc < all) {
                    open_run = make_int4(req, kvh, pair, all);
                    open_rows = make_int4(w.add, w.row_base, pairs, 0);
                }
            }
            w.code = w.req < 0 ? -1 : 2 * w.n_loc + w.single;
            w.qy = (w.kvh * p.max_rows + w.row_base + w.pair * tpp) << gs;
            if (lane == 0 && !val) {
                ok = it < 2 || mbar_wait(&bars[SM::B_ITEM_EMPTY + (it & 1)], ((it >> 1) - 1) & 1, abort_flag);
                if (ok) {
                    slots[it & 1] = w;
                    mbar_arrive(&bars[SM::B_ITEM_FULL + (it & 1)]);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok || w.req < 0) break;
            Window v;
            look_up(v, w, w.jb);
            for (int jj = 0; jj < w.n_loc; ++jj, ++kc) {
                int32_t y[kTreePagesPerUnit];
                const uint2 gone = next_unit(v, w, jj, y);
                ok = turn == 0 || mbar_wait(empty + st, (turn - 1) & 1, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                if (elect_one()) {
                    if (!val) s_meta[kc % SM::kMeta] = gone;
                    mbar_arrive_expect_tx(raw + st, SM::kUnit);
#pragma unroll
                    for (int m = 0; m < kTreePagesPerUnit; ++m) {
                        uint8_t* dst = ring + st * SM::kUnit + m * SM::kPageBytes;
                        if constexpr (D == 128) tma_load_4d(dst, map, raw + st, 0, 0, 0, y[m]);
                        else tma_load_2d(dst, map, raw + st, 0, y[m]);
                    }
                }
                __syncwarp();
                if (++st == stages) st = 0, ++turn;
            }
            // the next run
            unit = 0;
            begins = kTreeRunWeight;
            if (++pair == pairs) {
                pair = 0;
                if (++kvh == p.hkv) {
                    kvh = 0;
                    do { ++req; } while (req < p.n && __ldcg(work + req + 1) == __ldcg(work + req));
                }
            }
        }
        if (lane == 0) {
            if (!val) {
                int4 desc = make_int4(0, 0, 0, 0);
                if (ok && open_run.x >= 0) {               // with the block that holds its last unit
                    const int32_t run = open_run.y * open_rows.z + open_run.z;
                    const int32_t u = __ldcg(work + open_run.x) + (run + 1) * (open_run.w + kTreeRunWeight) - 1;
                    desc = make_int4(Deal(__ldcg(work + p.n), p.blocks).owner(u) << 8 | 0xFF, open_run.z * tpp, open_run.y, 0);
                }
                p.desc[2 * blockIdx.x] = desc;
                p.desc[2 * blockIdx.x + 1] = open_rows;
            }
            // every copy lands before the block exits: each stage's last turn
            for (int s = 0; s < stages; ++s) {
                const int turns = turn + (s < st ? 1 : 0);
                if (turns > 0) mbar_drain(raw + s, (turns - 1) & 1);
            }
        }
    } else if (warp == 17) {
        // ------------------------------------------------------------ Q K^T
        constexpr uint32_t idesc_qk = idesc_f16(128, kTreeUnit);
        int kc = 0, hg0 = 0, hg1 = 0, q_turns = 0;
        bool ok = true;
        grid_dep_wait();
        for (int it = 0; ok; ++it) {
            int32_t qy;
            const int code = take_code(it, qy), n_loc = code >> 1;
            const bool single = code & 1;
            if (code < 0) break;
            // the run's queries, when those of the run before have been read
            if (it > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars[SM::B_Q_EMPTY], (it - 1) & 1, abort_flag));
            if (!ok) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&bars[SM::B_Q_FULL], (single ? 1 : 2) * SM::kQ);
                for (int x = 0; x < (single ? 1 : 2) * (D / 64); ++x)
                    tma_load_2d(smem + x * (kTileRows * 128), &tm_q, &bars[SM::B_Q_FULL], x % (D / 64) * 64, qy + x / (D / 64) * kTileRows);
            }
            __syncwarp();
            q_turns = it + 1;
            ok = __all_sync(0xffffffffu, mbar_wait(&bars[SM::B_Q_FULL], it & 1, abort_flag));
            for (int jj = 0; ok && jj < n_loc; ++jj, ++kc) {
                const int ks = kc % NK;
                ok = __all_sync(0xffffffffu, mbar_wait(&bars[SM::B_K_ROT + ks], (kc / NK) & 1, abort_flag));
                const int t0 = single ? kc & 1 : 0, t1 = single ? t0 : 1;
#pragma unroll 1
                for (int t = t0; ok && t <= t1; ++t) {
                    const int hg = t ? hg1 : hg0;
                    ok = __all_sync(0xffffffffu, hg < 2 || mbar_wait(&bars[SM::B_PV_DONE + 2 * t + (hg & 1)],
                                                                     ((hg - 2) >> 1) & 1, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t aQ = desc_sw128_lo(smem_u32(smem + (single ? 0 : t) * SM::kQ), 16);
                    const uint32_t aK = desc_sw128_lo(smem_u32(sK(ks)), 16);
                    const uint32_t tS = tmem + t * 128 + (hg & 1) * 64;
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_ss(tS, desc_of(aQ + (k >> 2) * 1024 + (k & 3) * 2, kDescSw128Hi),
                                   desc_of(aK + (k >> 2) * (SM::kHalf >> 4) + (k & 3) * 2, desc_sw128_hi(SM::kGroup)), idesc_qk, k);
                        mma_commit(&bars[SM::B_S_FULL + 2 * t + (hg & 1)]);
                        if (t == t1) mma_commit(&bars[SM::B_K_EMPTY + ks]);
                    }
                    __syncwarp();
                    if (t) ++hg1; else ++hg0;
                }
            }
            if (ok && elect_one()) mma_commit(&bars[SM::B_Q_EMPTY]);
            __syncwarp();
        }
        if (elect_one()) {
            mma_commit(&bars[SM::B_DRAIN]);
            mbar_drain(&bars[SM::B_DRAIN], 0);
            if (q_turns > 0) mbar_drain(&bars[SM::B_Q_FULL], (q_turns - 1) & 1);
        }
        __syncwarp();
    } else if (warp == 18) {
        // ------------------------------------------------------------ P V
        constexpr uint32_t idesc_pv = idesc_bf16(128, D, true);
        int kc = 0, vs = 0, vn = 0, hg0 = 0, hg1 = 0, own0 = 0, own1 = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            int32_t qy;
            const int code = take_code(it, qy), n_loc = code >> 1;
            const bool single = code & 1;
            if (code < 0) break;
            bool begun0 = false, begun1 = false;
            for (int jj = 0; ok && jj < n_loc; ++jj, ++kc) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bars[SM::B_V_FULL + vs], vn & 1, abort_flag));
                const int t0 = single ? kc & 1 : 0, t1 = single ? t0 : 1;
#pragma unroll 1
                for (int t = t0; ok && t <= t1; ++t) {
                    const int hg = t ? hg1 : hg0, own = t ? own1 : own0;
                    const bool begun = t ? begun1 : begun0;
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(&bars[SM::B_P_FULL + 2 * t + (hg & 1)], (hg >> 1) & 1, abort_flag) &&
                                        (begun || own == 0 || mbar_wait(&bars[SM::B_O_FREE + t], (own - 1) & 1, abort_flag)));
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kTreePagesPerUnit; ++k)
                            mma_ts(tmem + kTmemO + t * 128, tmem + t * 128 + (hg & 1) * 64 + 8 * k,
                                   desc_of(desc_sw128_lo(smem_u32(sV(vs)), SM::kHalf) + k * (SM::kPageBytes >> 4), desc_sw128_hi(SM::kGroup)),
                                   idesc_pv, k > 0 ? 1u : begun ? 1u : 0u);
                        mma_commit(&bars[SM::B_PV_DONE + 2 * t + (hg & 1)]);
                        if (t == t1) mma_commit(&bars[SM::B_V_EMPTY + vs]);
                    }
                    __syncwarp();
                    if (t) begun1 = true, ++hg1;
                    else begun0 = true, ++hg0;
                }
                if (++vs == NV) vs = 0, ++vn;
            }
            if (!ok) break;
            if (elect_one()) {
                if (begun0) mma_commit(&bars[SM::B_O_DONE]);
                if (begun1) mma_commit(&bars[SM::B_O_DONE + 1]);
            }
            __syncwarp();
            own0 += begun0;
            own1 += begun1;
        }
        if (elect_one()) {
            mma_commit(&bars[SM::B_DRAIN + 1]);
            mbar_drain(&bars[SM::B_DRAIN + 1], 0);
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ------------------------------------------------------------ rotation
        // Thread rt of group r: 16-byte chunk pair c (dimensions 8 c .. and d/2 + 8 c ..) of N consecutive
        // keys, a warp a page; their angles start from the cos/sin row of the first one's position and
        // advance by one position, a rotation by table row 1.  Keys of nodes have positions of their own.
        constexpr int N = 64 * CP / 128;                 // keys a thread
        const int r = warp >> 2 & 1, rt = tid & 127, c = rt % CP, k0 = rt / CP * N, page = rt >> 5;
        const int c_hi = D == 128 ? c : c + 4;
        auto load_row = [&](int32_t pos, float4 (&cs)[4]) {
            const float4* src = reinterpret_cast<const float4*>(p.rope + (int64_t)pos * D + 16 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) cs[e] = src[e];
        };
        // key k0 + i: 16-byte chunk c of a row sits at c ^ (row & 7), and k0 is a multiple of N
        const uint32_t a_k = smem_u32(smem + SM::oK) + (k0 >> 3) * SM::kGroup + sw128_off(k0 & 7, c);
        auto turn_key = [&](uint32_t at, int i, bool have, const Angles& a, uint32_t& odd) {
            const uint32_t lo_at = (at ^ (i << 4)) + i * 128, hi_at = D == 128 ? lo_at + SM::kHalf : lo_at ^ 64u;
            uint4 lo = lds_128(lo_at), hi = lds_128(hi_at);
            if (!have) lo = hi = make_uint4(0, 0, 0, 0);                      // (may hold anything)
            a.turn(lo, hi, odd);
            sts_128(lo_at, lo);
            sts_128(hi_at, hi);
        };
        grid_dep_wait();
        float4 cs[4];
        load_row(1, cs);
        Angles step;
        uint64_t minus_step[4];
        step.set(cs);
#pragma unroll
        for (int e = 0; e < 4; ++e) minus_step[e] = f2_neg(step.S[e]);
        uint32_t odd = 0;                                // NaN where a rotated value is not finite
        int kc = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            TreeItem w;
            ok = take_item(it, w);
            if (!ok || w.req < 0) break;
            // a unit's cos/sin row, and the position of the unit behind it, are loaded as soon as the keys before
            // are handed on: the fence that makes those visible to the tensor cores waits for loads in flight
            const int n_pages = pages_of(w.seq + w.add);
            const int32_t* pos_row = p.page_pos + (int64_t)w.req * p.max_pages;
            auto position = [&](int jj) { return pos_row[min((w.jb + jj) * kTreePagesPerUnit + page, n_pages - 1)] + (k0 & 15); };
            auto row_of = [&](int32_t pos) { return pos >= 0 && pos < p.max_pos ? pos : 0; };
            const int j0 = (kc & 1) == r ? 0 : 1;
            int32_t pos_n = position(j0);
            load_row(row_of(pos_n), cs);
            pos_n = position(j0 + 2);
            for (int jj = j0; jj < w.n_loc; jj += 2) {
                const int u = kc + jj, ks = u % NK;
                const int slot0 = (w.jb + jj) * kTreeUnit;
                ok = mbar_wait(&bars[SM::B_K_RAW + ks], (u / NK) & 1, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                const uint2 meta = s_meta[u % SM::kMeta];
                const uint32_t gone = ((page & 2 ? meta.y : meta.x) >> (page & 1) * 16) & 0xFFFFu;
                const uint32_t at = a_k + ks * SM::kUnit;
                Angles a;
                a.set(cs);
                // (the next unit's row comes nearer meanwhile; two threads share a line)
                if (D == 128 && (c & 1) == 0) prefetch_l1(p.rope + (int64_t)row_of(pos_n) * D + 16 * c);
                if (slot0 + (page + 1) * kPage <= w.seq) {                    // (the same for the warp)
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        turn_key(at, i, !(gone >> ((k0 & 15) + i) & 1u), a, odd);
                        a.advance(step, minus_step);
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < N; ++i) {
                        const int key = k0 + i;
                        const bool have = !(gone >> (key & 15) & 1u);
                        if (have && slot0 + key >= w.seq) {
                            const int32_t pos = p.row_pos[w.row_base + slot0 + key - w.seq];
                            if (pos < 0 || pos >= p.max_pos) set_dev_error(kDevErrBounds);
                            load_row(row_of(pos), cs);
                            a.set(cs);
                        }
                        turn_key(at, i, have, a, odd);
                        a.advance(step, minus_step);
                    }
                }
                fence_proxy_async_smem();
                arrive_warp(&bars[SM::B_K_ROT + ks]);
                load_row(row_of(pos_n), cs);
                pos_n = position(jj + 4);
                // the unit's values: rows of hidden slots become zeros (they may hold anything, and a weight of zero
                // does not silence a NaN)
                const int vs = u % NV;
                ok = mbar_wait(&bars[SM::B_V_RAW + vs], (u / NV) & 1, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                if ((meta.x | meta.y) != 0u) {
                    constexpr int LANES = D / 8, ROWS = 128 / LANES;
                    const int ch = rt % LANES, row0 = rt / LANES;             // (ROWS is a multiple of 8)
                    uint8_t* dst = sV(vs) + (row0 >> 3) * SM::kGroup + (ch >> 3) * SM::kHalf + sw128_off(row0 & 7, ch & 7);
#pragma unroll
                    for (int i = 0; i < kTreeUnit / ROWS; ++i)
                        if ((row0 + i * ROWS < 32 ? meta.x >> (row0 + i * ROWS) : meta.y >> (row0 + i * ROWS - 32)) & 1u)
                            *reinterpret_cast<uint4*>(dst + i * ROWS / 8 * SM::kGroup) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                arrive_warp(&bars[SM::B_V_FULL + vs]);
            }
            kc += w.n_loc;
        }
        if (odd != 0u) set_dev_error(kDevErrRange);
    } else {
        // ------------------------------------------------------------ softmax
        const int t = warp >> 2, m = tid & 127;            // row of the tile = TMEM lane
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tO = tmem + lane_addr + kTmemO;
        int hg = 0, kc = 0, own[2] = {0, 0}, joined = 0;
        float nan = 0.f;                                   // NaN where a result is not finite
        bool ok = true;
        for (int it = 0; ok; ++it) {
            TreeItem w;
            ok = take_item(it, w);
            if (!ok || w.req < 0) break;
            const int tok = w.pair * tpp + (w.single ? 0 : t * tpt) + (m >> gs);
            const bool valid = tok < w.add;
            const bool any = __any_sync(0xffffffffu, valid);   // (a warp without rows has no scores to look at)
            const uint32_t* seen = p.seen + (int64_t)(w.row_base + min(tok, w.add - 1)) * p.words;
            float m_run = -INFINITY, l_run = 0.f;
            const int mine = chain_units(w, kc, t), other = chain_units(w, kc, 1 - t);
            int jj = w.single && (kc & 1) != t ? 1 : 0;
            for (int q = 0; q < mine; ++q, ++hg, jj += w.single ? 2 : 1) {
                const int buf = hg & 1;
                const uint32_t tS = tmem + lane_addr + t * 128 + buf * 64;
                ok = mbar_wait(&bars[SM::B_S_FULL + 2 * t + buf], (hg >> 1) & 1, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                if (any) {
                    const uint2 gone = s_meta[(kc + jj) % SM::kMeta];
                    const int first = (w.jb + jj) * kTreeUnit;
                    uint32_t hide0 = gone.x, hide1 = gone.y;
                    if (first + kTreeUnit > w.seq) {
                        const uint64_t see = tree_window(seen, p.words, first - w.seq);
                        hide0 |= ~(uint32_t)see;
                        hide1 |= ~(uint32_t)(see >> 32);
                    }
                    // Half a unit at a time: 24 requests of 64 nodes behind 16 k tokens 392 us, 516 with a quarter (twice
                    // the votes and branches), 435 to 452 with the whole (more code than the instruction cache holds
                    // beside the other roles', and registers that these have to give).
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t hide = h ? hide1 : hide0;
                        const bool masked = __any_sync(0xffffffffu, hide != 0u);
                        // A row's reference is 16 above the largest of the first scores it sees, and stays while the
                        // weights against it add up to no more than 1 in 32 keys: how small they are costs no precision
                        // (the largest is above 2^-17, and what is lost lies below 2^-126), and most halves need no
                        // maximum.  Weights of 1 at most leave the sums of weights times values the
                        // whole range of fp32: below slots / 32 times the largest value (with the largest score itself as
                        // the reference weights went up to 2^16, and values of 5e33 to infinity).  It moves by whole
                        // numbers: powers of two round nothing.
                        uint32_t pk[16];
                        float sum;
                        for (bool again = false;; again = true) {
                            uint32_t sv[32];
                            tmem_ld32(tS + 32 * h, sv);
                            tmem_ld_wait();
                            if (masked) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (hide >> e & 1u) sv[e] = __float_as_uint(-INFINITY);
                            }
                            const float msub = m_run == -INFINITY ? 0.f : m_run;
                            const uint64_t negm2 = f2_pack(-msub, -msub);
                            uint64_t acc2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float d0, d1;
                                f2_unpack(f2_add(f2_pack(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), negm2), d0, d1);
                                const float p0 = ex2(d0), p1 = ex2(d1);
                                acc2[e & 1] = f2_add(acc2[e & 1], f2_pack(p0, p1));
                                pk[e] = pack_bf16x2(p0, p1);   // bf16 like the values they meet (an MMA's operands share a type)
                            }
                            float a0, a1, b0, b1;
                            f2_unpack(acc2[0], a0, a1);
                            f2_unpack(acc2[1], b0, b1);
                            sum = (a0 + b0) + (a1 + b1);
                            const bool stale = valid && (m_run == -INFINITY || sum > 1.0f);    // (other rows hold anything)
                            if (again || !__any_sync(0xffffffffu, stale)) break;
                            tmem_ld32(tS + 32 * h, sv);
                            tmem_ld_wait();
                            float mx = -INFINITY;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(hide >> e & 1u)) mx = fmaxf(mx, __uint_as_float(sv[e]));
                            const bool need = stale && mx > -INFINITY;
                            const float to = need ? ceilf(mx) + 16.0f : m_run, alpha = need ? ex2(m_run - to) : 1.0f;
                            m_run = to;
                            l_run *= alpha;
                            if (q > 0) {       // every earlier P V of this chain must be done before O is rescaled
                                ok = mbar_wait(&bars[SM::B_PV_DONE + 2 * t + (1 - buf)], ((hg - 1) >> 1) & 1, abort_flag);
                                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                                tc_fence_after();
                            }
#pragma unroll 1
                            for (int cc = q > 0 ? 0 : D / 16; cc < D / 16; ++cc) {
                                uint32_t o[16];
                                tmem_ld16(tO + t * 128 + cc * 16, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st16(tO + t * 128 + cc * 16, o);
                            }
                            // (stored, before O is loaded again: another row's reference may move in the second half)
                            tmem_st_wait();
                            if (h == 1) {      // and the weights of the first half
                                uint32_t o[16];
                                tmem_ld16(tS, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = pack_bf16x2(bf16_lo(o[e]) * alpha, bf16_hi(o[e]) * alpha);
                                tmem_st16(tS, o);
                            }
                        }
                        if (!ok) break;
                        tmem_st16(tS + 16 * h, pk);
                        l_run += sum;
                    }
                    if (!ok) break;
                    tmem_st_wait();
                }
                tc_fence_before();
                arrive_warp(&bars[SM::B_P_FULL + 2 * t + buf]);
            }
            if (!ok) break;
            // ---- epilogue: O / l, or the part's sums as they are
            if (mine > 0) ok = mbar_wait(&bars[SM::B_O_DONE + t], own[t]++ & 1, abort_flag);
            if (w.single && t == 1) {
                // chain 0 has both results' rows
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                if (mine > 0) {
                    tc_fence_after();
                    s_ml[m] = make_float2(m_run, l_run);
                    tc_fence_before();
                    arrive_warp(&bars[SM::B_ML]);
                }
                kc += w.n_loc;
                continue;
            }
            const bool two = w.single && other > 0;
            float2 ml = make_float2(-INFINITY, 0.f);
            if (two) {
                ok = ok && mbar_wait(&bars[SM::B_ML], joined & 1, abort_flag);
                ++joined;
            }
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            tc_fence_after();
            if (two) ml = s_ml[m];
            const float top = fmaxf(m_run, ml.x), ref = top == -INFINITY ? 0.f : top;
            float f0 = mine > 0 ? ex2(m_run - ref) : 0.f, f1 = two ? ex2(ml.x - ref) : 0.f;
            const float l_all = l_run * f0 + ml.y * f1;
            const int part_row = (w.single ? 0 : t * kTileRows) + m;
            if (any) {
                if (w.slot >= 0) {
                    if (valid) p.part_ml[(int64_t)w.slot * (2 * kTileRows) + part_row] = make_float2(top, l_all);
                } else {
                    const float inv = l_all > 0.f ? 1.0f / l_all : 0.f;
                    f0 *= inv;
                    f1 *= inv;
                }
#pragma unroll 1
                for (int cc = 0; cc < D / 16; ++cc) {
                    float o[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = 0.f;
                    uint32_t x[16];
                    if (mine > 0) {
                        tmem_ld16(tO + t * 128 + cc * 16, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(x[e]) * f0;
                    }
                    if (two) {
                        tmem_ld16(tO + 128 + cc * 16, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = fmaf(__uint_as_float(x[e]), f1, o[e]);
                    }
                    if (valid) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) nan = fmaf(o[e], 0.f, nan);
                        if (w.slot >= 0) {
                            float4* dst = p.part_o + ((int64_t)w.slot * (D / 4) + cc * 4) * (2 * kTileRows) + part_row;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                dst[e * (2 * kTileRows)] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        } else {
                            uint4* dst = reinterpret_cast<uint4*>(
                                p.out + ((int64_t)(w.row_base + tok) * p.hq + w.kvh * g + (m & (g - 1))) * D + cc * 16);
                            dst[0] = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                                                pack_bf16x2(o[6], o[7]));
                            dst[1] = make_uint4(pack_bf16x2(o[8], o[9]), pack_bf16x2(o[10], o[11]), pack_bf16x2(o[12], o[13]),
                                                pack_bf16x2(o[14], o[15]));
                        }
                    }
                }
            }
            tc_fence_before();
            if (mine > 0) arrive_warp(&bars[SM::B_O_FREE + t]);
            if (two) arrive_warp(&bars[SM::B_O_FREE + 1]);
            kc += w.n_loc;
        }
        if (nan != nan) set_dev_error(kDevErrRange);       // (a value that takes part is not finite)
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Adds up the runs that a block of tree_attn_kernel began and left open: its part, then those of the blocks behind
// up to the run's last, in their order.  A warp takes 32 rows and 8 dimensions of such a run at a time (the parts lie
// so), four parts' loads in flight, and the warps of one launch go round all of them (a grid with a place for every
// run that a block could begin is nearly all empty blocks).  Where there are warps enough, four share an item, each
// with every fourth part, and meet in shared memory: few runs are long ones of many parts (one long request, 8 runs
// of 20 parts of 128 KB: 8 us so and 14 with a warp an item; 151 runs of two parts: 27 with four and 10 with one).
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeParams p) {
    __shared__ int16_t s_runs[kTreeMaxBlocks];
    __shared__ int s_warp[kJoinWarps];
    __shared__ float s_acc[kJoinWarps][10][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    // the runs, in the same order in every block
    int count = 0;
    for (int b0 = 0; b0 < p.blocks; b0 += kJoinThreads) {
        const int b = b0 + threadIdx.x;
        const bool open = b < p.blocks && p.desc[2 * b].x != 0;
        const uint32_t in_warp = __ballot_sync(0xffffffffu, open);
        if (lane == 0) s_warp[warp] = __popc(in_warp);
        __syncthreads();
        int at = count;
        for (int w = 0; w < kJoinWarps; ++w) {
            if (w < warp) at += s_warp[w];
            count += s_warp[w];
        }
        if (open) s_runs[at + __popc(in_warp & ((1u << lane) - 1))] = (int16_t)b;
        __syncthreads();
    }
    constexpr int COLS = D / 8, ITEMS = 2 * kTileRows / 32 * COLS, SHARE = 4;
    const int g = p.hq / p.hkv, gs = __ffs(g) - 1;
    const bool shared_items = count * ITEMS * SHARE <= (int)gridDim.x * kJoinWarps;
    const int share = shared_items ? SHARE : 1, mine = warp % share;
    float odd = 0.f;
    for (int item = (blockIdx.x * kJoinWarps + warp) / share; item < count * ITEMS || shared_items; item += gridDim.x * kJoinWarps) {
        const bool there = item < count * ITEMS;
        const int j = there ? s_runs[item / ITEMS] : 0, at = item % ITEMS;
        const int4 d = p.desc[2 * j], rows = p.desc[2 * j + 1];
        const int last = d.x >> 8, r = at / COLS * 32 + lane, f = at % COLS;
        const int tok = d.y + (r >> gs);
        const bool valid = there && tok < rows.x;
        float top = -INFINITY, l = 0.f, acc[8] = {};
        constexpr int N = 4;
        for (int b0 = j + mine; valid && b0 <= last; b0 += N * share) {
            float2 ml[N];
            float4 v[N][2];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                // (behind the last part: that part again, without weight -- other memory may hold NaN)
                const int b = min(b0 + i * share, last);
                const int64_t slot = (int64_t)b * 2 + (b == j ? 1 : 0);
                ml[i] = p.part_ml[slot * (2 * kTileRows) + r];
                v[i][0] = p.part_o[(slot * (D / 4) + 2 * f) * (2 * kTileRows) + r];
                v[i][1] = p.part_o[(slot * (D / 4) + 2 * f + 1) * (2 * kTileRows) + r];
                if (b0 + i * share > last) ml[i].x = -INFINITY;
            }
            float now = top;
#pragma unroll
            for (int i = 0; i < N; ++i) now = fmaxf(now, ml[i].x);
            const float ref = now == -INFINITY ? 0.f : now, old = ex2(top - ref);
            top = now;
            l *= old;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] *= old;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float w = ex2(ml[i].x - ref);
                l += w * ml[i].y;
                acc[0] += w * v[i][0].x;
                acc[1] += w * v[i][0].y;
                acc[2] += w * v[i][0].z;
                acc[3] += w * v[i][0].w;
                acc[4] += w * v[i][1].x;
                acc[5] += w * v[i][1].y;
                acc[6] += w * v[i][1].z;
                acc[7] += w * v[i][1].w;
            }
        }
        if (shared_items) {
            s_acc[warp][8][lane] = top;
            s_acc[warp][9][lane] = l;
#pragma unroll
            for (int e = 0; e < 8; ++e) s_acc[warp][e][lane] = acc[e];
            __syncthreads();
            if (mine != 0) break;
            float all = top;
            for (int i = 1; i < SHARE; ++i) all = fmaxf(all, s_acc[warp + i][8][lane]);
            const float ref = all == -INFINITY ? 0.f : all, own = ex2(top - ref);
            l *= own;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] *= own;
            for (int i = 1; i < SHARE; ++i) {
                const float w = ex2(s_acc[warp + i][8][lane] - ref);
                l += w * s_acc[warp + i][9][lane];
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += w * s_acc[warp + i][e][lane];
            }
        }
        if (valid) {
            const float inv = l > 0.f ? 1.0f / l : 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) odd = fmaf(acc[e], 0.f, odd);
            *reinterpret_cast<uint4*>(p.out + ((int64_t)(rows.y + tok) * p.hq + d.z * g + (r & (g - 1))) * D + 8 * f) =
                make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                           pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
        }
        if (shared_items) break;
    }
    if (odd != odd) set_dev_error(kDevErrRange);
}

}  // namespace pcf
