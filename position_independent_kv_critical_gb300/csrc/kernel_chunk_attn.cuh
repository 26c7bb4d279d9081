// Attention of a chunk of new tokens over the pages of their requests.
//
// Row i is token s + t of request b (s tokens held before the chunk): for query head h of kv head
// h / g, over the slots j <= s + t of b whose page does not exclude them,
//   out = sum_j softmax_j((R_pos(i) q) . (R_(page_pos + r) k_j) / sqrt(d)) v_j,
// a row with no slot left giving zeros.  Keys are stored unrotated and rotated when read.
#pragma once
#include "chunk_format.h"
#include "kernel_chunk_tables.cuh"
#include "ptx.cuh"

namespace pcf {

struct ChunkAttnParams {
    const int32_t* plan;
    const __nv_bfloat16* q;
    const __nv_bfloat16* k_pool;
    const __nv_bfloat16* v_pool;
    const int32_t* block_table;
    const int32_t* page_pos;
    const uint16_t* excl;       // or null
    const int32_t* row_pos;
    const float* rope;
    __nv_bfloat16* out;
    int64_t q_stride;
    int32_t n, max_pages, max_rows, hq, hkv, n_phys, max_pos, workers;
};

// One block per (row, query head), a warp a page at a time: lane l holds the frequencies l (and
// l + 32 for d = 128) of the query, a key's score is a warp sum, the running maximum and sum of the
// softmax are kept per warp and the four warps' results joined in shared memory.
template <int D>
__global__ void __launch_bounds__(128) chunk_attn_simple_kernel(const ChunkAttnParams p) {
    constexpr int F = D / 64;   // frequencies (pairs i, i + D/2) a lane
    __shared__ float s_o[4][D];
    __shared__ float s_m[4], s_l[4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_wait();
    grid_dep_launch();
    const int32_t row = blockIdx.x;
    if (!plan_fits(p.plan, p.n, p.max_pages, p.max_rows, p.hq, p.hkv, p.workers)) return;
    if (row >= p.plan[C_ROWS]) return;
    const int32_t* base = p.plan + plan_array(CA_ROW, p.n);
    const int b = row_request(base, p.n, row);
    if (p.plan[plan_array(CA_NEW, p.n) + b] * (p.hq / p.hkv) <= kFewRows) return;
    const int32_t last = p.plan[plan_array(CA_SEQ, p.n) + b] + row - base[b];
    const int h = blockIdx.y, kvh = h / (p.hq / p.hkv);
    const __nv_bfloat16* q = p.q + row * p.q_stride + h * D;
    const float2* rope = reinterpret_cast<const float2*>(p.rope);
    const int32_t qp = p.row_pos[row];
    float qa[F], qb[F], big = 0.f;   // big: largest rotated magnitude, held to fp16's range like everywhere
    for (int f = 0; f < F; ++f) {
        const int i = lane + 32 * f;
        const float2 cs = rope[(int64_t)qp * (D / 2) + i];
        const float a = __bfloat162float(q[i]), c = __bfloat162float(q[i + D / 2]);
        const float scale = 1.4426950408889634f * rsqrtf((float)D);
        qa[f] = (a * cs.x - c * cs.y) * scale;
        qb[f] = (c * cs.x + a * cs.y) * scale;
        big = max3f(big, fabsf(qa[f]), fabsf(qb[f]));
    }
    float m = -INFINITY, l = 0.f, oa[F], ob[F];
    for (int f = 0; f < F; ++f) oa[f] = ob[f] = 0.f;
    for (int32_t pg = warp; pg * kPage <= last; pg += 4) {
        const int64_t e = (int64_t)b * p.max_pages + pg;
        const int32_t ph = p.block_table[e], pp = p.page_pos[e];
        const uint32_t ex = p.excl ? p.excl[e] : 0u;
        if (ph < 0 || ph >= p.n_phys || pp < 0 || pp > p.max_pos - kPage) {
            set_dev_error(kDevErrBounds);
            continue;
        }
        const int64_t off = ((int64_t)ph * p.hkv + kvh) * kPage * D;
        for (int r = 0; r < kPage && pg * kPage + r <= last; ++r) {
            if (ex >> r & 1u) continue;
            const __nv_bfloat16* k = p.k_pool + off + r * D;
            const __nv_bfloat16* v = p.v_pool + off + r * D;
            float s = 0.f;
            for (int f = 0; f < F; ++f) {
                const int i = lane + 32 * f;
                const float2 cs = rope[(int64_t)(pp + r) * (D / 2) + i];
                const float a = __bfloat162float(k[i]), c = __bfloat162float(k[i + D / 2]);
                const float y = a * cs.x - c * cs.y, z = c * cs.x + a * cs.y;
                big = max3f(big, fabsf(y), fabsf(z));
                s += qa[f] * y + qb[f] * z;
            }
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            const float mn = fmaxf(m, s), al = exp2f(m - mn), pr = exp2f(s - mn);
            l = l * al + pr;
            m = mn;
            for (int f = 0; f < F; ++f) {
                oa[f] = oa[f] * al + pr * __bfloat162float(v[lane + 32 * f]);
                ob[f] = ob[f] * al + pr * __bfloat162float(v[lane + 32 * f + D / 2]);
            }
        }
    }
    for (int f = 0; f < F; ++f) {
        s_o[warp][lane + 32 * f] = oa[f];
        s_o[warp][lane + 32 * f + D / 2] = ob[f];
    }
    if (!(big < kF16Limit)) set_dev_error(kDevErrRange);
    s_m[warp] = m;
    s_l[warp] = l;
    __syncthreads();
    const float top = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    for (int i = threadIdx.x; i < D; i += 128) {
        float o = 0.f, t = 0.f;
        for (int w = 0; w < 4; ++w) {
            const float a = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - top);
            o += a * s_o[w][i];
            t += a * s_l[w];
        }
        p.out[((int64_t)row * p.hq + h) * D + i] = __float2bfloat16(t > 0.f ? o / t : 0.f);
    }
}

}  // namespace pcf
