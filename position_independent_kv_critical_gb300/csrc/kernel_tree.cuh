// Attention of a tree of drafted tokens over the pages of its request and its own branches.
//
// Row i is node t of request b: for query head h of kv head h / g, over the slots j < seq and the slots
// seq + u of the nodes u that t goes on from (itself among them), without those the pages exclude,
//   out = sum_j softmax_j((R_pos(i) q) . (R_pos(j) k_j) / sqrt(d)) v_j,
// pos(j) = page_pos + r for a held slot and the node's own position for a node's; a row with no slot left
// gives zeros.
#pragma once
#include "kernel_tree_tables.cuh"
#include "ptx.cuh"
#include "tree_format.h"

namespace pcf {

struct TreeParams {
    const int32_t* plan;
    const __nv_bfloat16* q;
    const __nv_bfloat16* k_pool;
    const __nv_bfloat16* v_pool;
    const int32_t* block_table;
    const int32_t* page_pos;
    const uint16_t* excl;       // or null
    const int32_t* row_pos;     // [max_rows] the nodes' positions
    const uint32_t* seen;       // [max_rows][words]
    const float* rope;
    __nv_bfloat16* out;
    int64_t q_stride;
    int32_t n, max_pages, max_rows, words, hq, hkv, n_phys, max_pos, tag;
};

// One warp a (row, query head), slot by slot: lane l has D / 64 pairs of dimensions that turn together.
template <int D>
__global__ void __launch_bounds__(128) tree_simple_kernel(const TreeParams p) {
    constexpr int N = D / 64;
    grid_dep_wait();
    grid_dep_launch();
    if (!tree_fits(p.plan, p.tag)) return;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t row = item / p.hq;
    const int32_t h = (int32_t)(item % p.hq);
    if (row >= p.plan[T_ROWS]) return;
    const int b = row_request(p.plan + tree_array(TA_ROW, p.n), p.n, (int32_t)row);
    const int32_t seq = p.plan[tree_array(TA_SEQ, p.n) + b], add = p.plan[tree_array(TA_NEW, p.n) + b];
    const int32_t first = p.plan[tree_array(TA_ROW, p.n) + b];
    const int kvh = h / (p.hq / p.hkv);
    const float scale = 1.4426950408889634f * (D == 128 ? 0.08838834764831845f : 0.125f);   // log2(e) / sqrt(d)
    float a[N], c[N], va[N] = {}, vc[N] = {}, top = -INFINITY, l = 0.f, big = 0.f;
    auto turn = [&](const __nv_bfloat16* src, int32_t pos, float (&lo)[N], float (&hi)[N]) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int i = lane * N + e;
            const float x = __bfloat162float(src[i]), y = __bfloat162float(src[i + D / 2]);
            const float2 cs = reinterpret_cast<const float2*>(p.rope)[(int64_t)pos * (D / 2) + i];
            lo[e] = x * cs.x - y * cs.y;
            hi[e] = y * cs.x + x * cs.y;
            if (!(fabsf(lo[e]) < kF16Limit) || !(fabsf(hi[e]) < kF16Limit)) big = INFINITY;
        }
    };
    const int32_t at = p.row_pos[row];
    if (at < 0 || at >= p.max_pos) {
        set_dev_error(kDevErrBounds);
        return;
    }
    turn(p.q + row * p.q_stride + (int64_t)h * D, at, a, c);
    for (int32_t j = 0; j < seq + add; ++j) {
        const int64_t e = (int64_t)b * p.max_pages + j / kPage;
        const int r = j % kPage, u = j - seq;
        if (p.excl && p.excl[e] >> r & 1u) continue;
        if (u >= 0 && !(p.seen[row * p.words + u / 32] >> (u & 31) & 1u)) continue;
        const int32_t ph = p.block_table[e], pos = u >= 0 ? p.row_pos[first + u] : p.page_pos[e] + r;
        if (ph < 0 || ph >= p.n_phys || pos < 0 || pos >= p.max_pos) {
            set_dev_error(kDevErrBounds);
            continue;
        }
        const int64_t src = (((int64_t)ph * p.hkv + kvh) * kPage + r) * D;
        float x[N], y[N], s = 0.f;
        turn(p.k_pool + src, pos, x, y);
#pragma unroll
        for (int i = 0; i < N; ++i) s += a[i] * x[i] + c[i] * y[i];
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= scale;
        const float m = fmaxf(top, s), old = ex2(top - m), w = ex2(s - m);
        top = m;
        l = l * old + w;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float v0 = __bfloat162float(p.v_pool[src + lane * N + i]);
            const float v1 = __bfloat162float(p.v_pool[src + D / 2 + lane * N + i]);
            if (!(fabsf(v0) + fabsf(v1) < INFINITY)) big = INFINITY;
            va[i] = va[i] * old + w * v0;
            vc[i] = vc[i] * old + w * v1;
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    __nv_bfloat16* dst = p.out + item * D;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        dst[lane * N + i] = __float2bfloat16(va[i] * inv);
        dst[D / 2 + lane * N + i] = __float2bfloat16(vc[i] * inv);
    }
    if (!(big < kF16Limit)) set_dev_error(kDevErrRange);
}

}  // namespace pcf
