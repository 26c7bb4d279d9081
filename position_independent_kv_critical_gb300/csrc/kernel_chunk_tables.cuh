// Growing the requests of a batch by a chunk of new tokens: block tables, page positions and slot
// maps from lengths that only the GPU knows, and the write of the chunk's keys and values into the
// pages they name.
#pragma once
#include "chunk_format.h"
#include "ptx.cuh"

namespace pcf {

struct TablesParams {
    const int32_t* seq;        // [n] tokens held
    const int32_t* add;        // [n] new tokens
    const int32_t* next_pos;   // [n] position of the first new token, or null: behind the last one
    const int32_t* free_pages; // [n_free]
    const int32_t* free_head;  // [1]
    int32_t* block_table;      // [n][max_pages], new entries written
    int32_t* page_pos;         // [n][max_pages], likewise
    int32_t* slot_map;         // [max_rows]
    int32_t* row_pos;          // [max_rows]
    int32_t* row_base;         // [n + 1]
    int32_t* seq_out;          // [n], may be seq
    int32_t* head_out;         // [1], may be free_head
    int32_t* plan;
    int32_t n, max_pages, max_rows, max_chunk, max_total_pages, n_phys, max_pos, n_free, hq, hkv, few_rows, workers, blocks, tag;
};

constexpr int kTablesThreads = 512;

// One block reads the lengths, checks them and leaves the plan.  Request b holds s tokens on
// ceil(s / 16) pages and grows by n: the pages behind are taken from the free list in request
// order, so a prefix sum of ceil((s + n) / 16) - ceil(s / 16) gives every request its first one;
// a prefix sum of n gives its first row.  Thread t takes a run of consecutive requests, so one
// block scan of per-thread sums is enough for any batch size.  Everything that is looked up by
// bisection (rows, units, tiles) is kept in shared memory: a probe costs some 30 cycles there and
// several hundred in L2.  What bounds the call is the chain of dependent loads and barriers: where the
// outputs are buffers of their own, every block of one launch reads the lengths and scans them for
// itself and then writes its share of the rows (`alone`); where lengths or list head are updated in
// place, a block must not write them while another still reads, so one block leaves the plan and a
// second launch writes the rows.  Graph replay, 64 requests of one token: 5.0 us apart (4.7 with next_pos),
// 6.2 in place; 512 requests of four: 6.3 and 9.0.
// (Sums of refused lengths may be as large as 4096 x 2^22: they stop at 2^29, above every limit.)
constexpr int kSumLimit = 1 << 29;
constexpr int kSums = 7;   // rows, pages taken, pages held afterwards, few-row units, key tiles and pages of the others, few-row requests
__device__ __forceinline__ int32_t pages_of(int32_t tokens) { return (tokens + kPage - 1) / kPage; }
__device__ __forceinline__ int32_t sat_add(int32_t a, int32_t b) { return min(a + b, kSumLimit); }

// A request's work in the attention: (page, kv head) units with few rows, else the weight of all its row
// pairs (every kv head) and the pages whose keys are rotated beforehand.
struct ChunkWork {
    int32_t few, many, pages;
};
__device__ __forceinline__ ChunkWork chunk_work(const TablesParams& p, int32_t s, int32_t n) {
    const int g = p.hq / p.hkv;
    const int32_t pages = pages_of(s + n);
    if (n == 0) return {0, 0, 0};
    if ((int64_t)n * g <= p.few_rows) return {pages * p.hkv, 0, 0};
    const int tpp = 2 * kTileRows / g, last = many_pairs(n, tpp) - 1;
    const int64_t tiles = (many_weight(s, tpp, last) + kPairWeight + many_tiles(s, n, tpp, last)) * p.hkv;
    // (rows that fit one tile: the kernel rotates the keys itself)
    return {0, (int32_t)min(tiles, (int64_t)kSumLimit), n * g <= kTileRows ? 0 : pages};
}

// Request of row i: the last b with base[b] <= i (requests without rows are passed over).
__device__ __forceinline__ int row_request(const int32_t* __restrict__ base, int n, int32_t i) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (base[mid] <= i) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The plan's per-request arrays, n + 1 words each, in shared memory (order of the CA_ enumeration).
__device__ __forceinline__ int32_t* plan_words_of(int32_t* arrays, int which, int32_t n) {
    return arrays + (int64_t)which * (n + 1);
}

// Everything that follows from the plan, shared out to threads as one range of tasks, so that no thread has
// the chain of one kind behind that of another: the rows, the requests' lengths, the workers' and the blocks'
// shares of the attention's work.  Nothing here reads what the call may overwrite in place (lengths and list
// head come from the plan), and a table entry that is read (a page begun earlier) is never one that is written.
PCF_HOST_DEVICE inline int32_t whole_warps(int32_t n) { return (n + 31) / 32 * 32; }
PCF_HOST_DEVICE inline int32_t rows_tasks(int32_t max_rows, int32_t n, int32_t workers, int32_t blocks) {
    return whole_warps(max_rows) + whole_warps(n + 1) + whole_warps(workers + 1) + 3 * whole_warps(blocks);
}

// Row r: token s + t of a request sits in page (s + t) / 16, at slot (s + t) % 16; the row that starts a page
// enters it.
__device__ __forceinline__ void write_row(const TablesParams& p, int32_t* arrays, int32_t rows, int32_t head, int32_t r) {
    const int32_t* seq = plan_words_of(arrays, CA_SEQ, p.n);
    const int32_t* base = plan_words_of(arrays, CA_ROW, p.n);
    const int32_t* take = plan_words_of(arrays, CA_TAKE, p.n);
    const int32_t* start = plan_words_of(arrays, CA_START, p.n);
    int32_t slot = -1, pos = -1;
    if (r < rows) {
        const int b = row_request(base, p.n, r);
        const int32_t t = r - base[b], s = seq[b] + t, pg = s / kPage, first = pages_of(seq[b]);
        const int64_t e = (int64_t)b * p.max_pages + pg;
        pos = start[b] + t;
        const int32_t ph = pg >= first ? p.free_pages[head + take[b] + pg - first] : p.block_table[e];
        if (pg >= first && s % kPage == 0) {
            p.block_table[e] = ph;
            p.page_pos[e] = pos;
        }
        slot = ph * kPage + s % kPage;
    }
    p.slot_map[r] = slot;
    p.row_pos[r] = pos;
}

// Where a position of the few-row requests' weights lies: request, kv head, page (the run's first one for a
// position in the weight of its beginning), and the units before it.
struct FewPlace {
    int32_t req, kvh, page, pages, units;
};
__device__ __forceinline__ FewPlace few_place(const TablesParams& p, int32_t* arrays, int32_t u) {
    const int32_t weight = plan_words_of(arrays, CA_START, p.n)[p.n];
    const int32_t* few = plan_words_of(arrays, CA_FEW, p.n);
    FewPlace at;
    at.req = row_request(few, p.n, u);
    at.pages = pages_of(plan_words_of(arrays, CA_SEQ, p.n)[at.req] + plan_words_of(arrays, CA_NEW, p.n)[at.req]);
    const int32_t run = at.pages + weight, local = u - few[at.req];
    at.kvh = local / run;
    at.page = max(0, local - at.kvh * run - weight);
    at.units = few[at.req] - weight * p.hkv * plan_words_of(arrays, CA_FEWN, p.n)[at.req] + at.kvh * at.pages + at.page;
    return at;
}
// Where worker w's share of the few-row requests' units begins, dealt by weight in equal runs (it ends where
// the next one's begins).
__device__ __forceinline__ void write_worker(const TablesParams& p, int32_t* arrays, int32_t w) {
    const int32_t* few = plan_words_of(arrays, CA_FEW, p.n);
    const Deal deal(few[p.n], p.workers);
    const int32_t u0 = deal.first(w);
    const int32_t all = few[p.n] - plan_words_of(arrays, CA_START, p.n)[p.n] * p.hkv * plan_words_of(arrays, CA_FEWN, p.n)[p.n];
    int4 e = make_int4(0, 0, 0, all), f = make_int4(1, 0, 0, 0);
    if (u0 < few[p.n]) {
        const FewPlace at = few_place(p, arrays, u0);
        e = make_int4(at.req, at.kvh, at.page, at.units);
        f = make_int4(at.pages, plan_words_of(arrays, CA_SEQ, p.n)[at.req], plan_words_of(arrays, CA_NEW, p.n)[at.req],
                      plan_words_of(arrays, CA_ROW, p.n)[at.req]);
    }
    int4* dst = reinterpret_cast<int4*>(p.plan + plan_starts(p.n)) + 3 * w;
    dst[0] = e;
    dst[1] = f;
    dst[2].x = p.tag;
}

// The blocks that the run of block w's first unit reaches (first, last), or that of its last unit (last).
__device__ __forceinline__ void write_share(const TablesParams& p, int32_t* arrays, int32_t w, bool of_last) {
    const int32_t* few = plan_words_of(arrays, CA_FEW, p.n);
    const int32_t weight = plan_words_of(arrays, CA_START, p.n)[p.n];
    const Deal deal(few[p.n], p.workers);
    const int per = p.workers / p.blocks;
    const int32_t u0 = deal.first(w * per), u1 = deal.first((w + 1) * per);
    if (u0 == u1) return;
    const FewPlace at = few_place(p, arrays, of_last ? u1 - 1 : u0);
    const int32_t first = few[at.req] + at.kvh * (at.pages + weight) + weight;     // its first page
    int4* dst = reinterpret_cast<int4*>(p.plan + plan_starts(p.n)) + 3 * w * per + 2;
    if (of_last) {
        dst->w = deal.owner(first + at.pages - 1) / per;
    } else {
        dst->y = deal.owner(first) / per;
        dst->z = deal.owner(first + at.pages - 1) / per;
    }
}

// Block w's share of the others' key tiles, in (request, kv head, row pair, tile) order, by weight.
__device__ __forceinline__ void write_block(const TablesParams& p, int32_t* arrays, int32_t w) {
    const int32_t* seq = plan_words_of(arrays, CA_SEQ, p.n);
    const int32_t* add = plan_words_of(arrays, CA_NEW, p.n);
    const int32_t* many = plan_words_of(arrays, CA_MANY, p.n);
    const Deal tiles(many[p.n], p.blocks);
    const int g = p.hq / p.hkv, tpp = 2 * kTileRows / g;
    p.plan[plan_count(p.n, p.workers, p.blocks) + w] = 0;
    const int32_t u0 = tiles.first(w);
    int4 e = make_int4(0, 0, 0, 0), f = make_int4(tiles.first(w + 1) - u0, p.tag, 0, 0);
    if (f.x > 0) {
        const int b = row_request(many, p.n, u0);
        const int32_t per_head = (many[b + 1] - many[b]) / p.hkv;
        int32_t local = u0 - many[b];
        e.x = b;
        e.y = local / per_head;
        local %= per_head;
        int lo = 0, hi = many_pairs(add[b], tpp) - 1;   // the pair the tile falls into
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (many_weight(seq[b], tpp, mid) <= local) lo = mid; else hi = mid - 1;
        }
        local -= (int32_t)many_weight(seq[b], tpp, lo);
        e.z = lo;
        e.w = max(0, local - kPairWeight);
        f.z = max(0, kPairWeight - local);
    }
    int4* dst = reinterpret_cast<int4*>(p.plan + plan_many(p.n, p.workers)) + 2 * w;
    dst[0] = e;
    dst[1] = f;
}

__device__ __forceinline__ void write_rows(const TablesParams& p, int32_t* arrays, int32_t rows, int32_t head,
                                           int32_t taken, int32_t i, int32_t step) {
    const int32_t total = rows_tasks(p.max_rows, p.n, p.workers, p.blocks);
    for (; i < total; i += step) {
        int32_t k = i;
        if (k < p.max_rows) {
            write_row(p, arrays, rows, head, k);
            continue;
        }
        k -= whole_warps(p.max_rows);
        if (k >= 0 && k <= p.n) {
            p.row_base[k] = plan_words_of(arrays, CA_ROW, p.n)[k];
            if (k < p.n) p.seq_out[k] = plan_words_of(arrays, CA_SEQ, p.n)[k] + plan_words_of(arrays, CA_NEW, p.n)[k];
            else p.head_out[0] = head + taken;
        }
        k -= whole_warps(p.n + 1);
        if (k >= 0 && k <= p.workers) write_worker(p, arrays, k);
        k -= whole_warps(p.workers + 1);
        if (k >= 0 && k < p.blocks) write_share(p, arrays, k, false);
        k -= whole_warps(p.blocks);
        if (k >= 0 && k < p.blocks) write_share(p, arrays, k, true);
        k -= whole_warps(p.blocks);
        if (k >= 0 && k < p.blocks) write_block(p, arrays, k);
    }
}

__global__ void __launch_bounds__(kTablesThreads) chunk_plan_kernel(const TablesParams p, int alone) {
    extern __shared__ int32_t s_arrays[];
    constexpr int kWarps = kTablesThreads / 32;
    __shared__ int s_warp[kSums][kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dep_wait();
    grid_dep_launch();
    const int per = (p.n + kTablesThreads - 1) / kTablesThreads;
    const int b0 = min(p.n, tid * per), b1 = min(p.n, b0 + per);
    int32_t* plan = p.plan;
    int32_t* o_seq = plan_words_of(s_arrays, CA_SEQ, p.n);
    int32_t* o_new = plan_words_of(s_arrays, CA_NEW, p.n);
    int32_t* o_row = plan_words_of(s_arrays, CA_ROW, p.n);
    int32_t* o_take = plan_words_of(s_arrays, CA_TAKE, p.n);
    int32_t* o_start = plan_words_of(s_arrays, CA_START, p.n);
    int32_t* o_few = plan_words_of(s_arrays, CA_FEW, p.n);
    int32_t* o_many = plan_words_of(s_arrays, CA_MANY, p.n);
    int32_t* o_kpage = plan_words_of(s_arrays, CA_KPAGE, p.n);
    int32_t* o_fewn = plan_words_of(s_arrays, CA_FEWN, p.n);
    const int32_t head = p.free_head[0];
    bool bad = head < 0 || head > p.n_free;
    int sum[kSums] = {};
    for (int b = b0; b < b1; ++b) {
        const int32_t s = p.seq[b], n = p.add[b];
        const int32_t want = p.next_pos ? p.next_pos[b] : 0;
        o_seq[b] = s;
        o_new[b] = 0;
        o_start[b] = 0;
        if (s < 0 || s > p.max_pages * kPage || n < 0 || n > p.max_chunk || s + n > p.max_pages * kPage) {
            bad = true;
            continue;
        }
        const int32_t before = pages_of(s), after = pages_of(s + n);
        int32_t start = 0;
        if (n > 0) {
            // a page's slots sit at consecutive positions, so a started page fixes the next one; its entries
            // are checked here, as the call goes on from them
            const bool started = s % kPage != 0;
            if (started || (s > 0 && !p.next_pos)) {
                const int64_t e = (int64_t)b * p.max_pages + before - 1;
                const int32_t last = p.page_pos[e], ph = started ? p.block_table[e] : 0;
                if (last < 0 || last > p.max_pos - kPage || ph < 0 || ph >= p.n_phys) bad = true;
                else start = last + (started ? s % kPage : kPage);
            }
            if (p.next_pos) {
                if (started && want != start) bad = true;
                start = want;
            }
            // every slot of the last page has a row in the cos/sin table
            if (start < 0 || start > p.max_pos || start + (after * kPage - s) > p.max_pos) bad = true;
        }
        sum[0] = sat_add(sum[0], n);
        sum[1] = sat_add(sum[1], after - before);
        sum[2] = sat_add(sum[2], after);
        const ChunkWork work = chunk_work(p, s, n);
        sum[3] = sat_add(sum[3], work.few);
        sum[4] = sat_add(sum[4], work.many);
        sum[5] = sat_add(sum[5], work.pages);
        sum[6] += work.few > 0;
        o_new[b] = n;
        o_start[b] = start;
    }
    int pre[kSums], tot[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
        int x = sum[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x = sat_add(x, y);
        }
        pre[i] = x;
        if (lane == 31) s_warp[i][warp] = x;
    }
    bad = __syncthreads_or(bad);
    if (warp < kSums) {
        int x = lane < kWarps ? s_warp[warp][lane] : 0;
#pragma unroll
        for (int o = 1; o < kWarps; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x = sat_add(x, y);
        }
        if (lane < kWarps) s_warp[warp][lane] = x;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
        tot[i] = s_warp[i][kWarps - 1];
        pre[i] += (warp ? s_warp[i][warp - 1] : 0) - sum[i];
    }
    bad = bad || tot[0] > p.max_rows || tot[2] > p.max_total_pages || tot[1] > p.n_free - head || tot[3] >= kSumLimit ||
          tot[4] >= kSumLimit;
    if (!bad) {   // the pages about to be taken exist
        for (int i = tid; i < tot[1]; i += kTablesThreads) {
            const int32_t ph = p.free_pages[head + i];
            bad |= ph < 0 || ph >= p.n_phys;
        }
    }
    bad = __syncthreads_or(bad);
    if (bad) {    // nothing is done: no rows, no work
#pragma unroll
        for (int i = 0; i < kSums; ++i) pre[i] = tot[i] = 0;
        if (tid == 0) set_dev_error(kDevErrBounds);
    }
    const int32_t run = run_weight(tot[3], p.workers), weight = run * p.hkv;      // of a run, of a request's runs
    for (int b = b0; b < b1; ++b) {
        if (bad) o_new[b] = 0;
        o_row[b] = pre[0];
        o_take[b] = pre[1];
        o_few[b] = pre[3] + pre[6] * weight;
        o_fewn[b] = pre[6];
        o_many[b] = pre[4];
        o_kpage[b] = pre[5];
        if (!bad) {
            const ChunkWork work = chunk_work(p, o_seq[b], o_new[b]);
            pre[0] += o_new[b];
            pre[1] += pages_of(o_seq[b] + o_new[b]) - pages_of(o_seq[b]);
            pre[3] += work.few;
            pre[4] += work.many;
            pre[5] += work.pages;
            pre[6] += work.few > 0;
        }
    }
    if (tid == 0) {
        o_seq[p.n] = o_new[p.n] = 0;
        o_start[p.n] = run;
        o_row[p.n] = tot[0];
        o_take[p.n] = tot[1];
        o_few[p.n] = tot[3] + tot[6] * weight;
        o_fewn[p.n] = tot[6];
        o_many[p.n] = tot[4];
        o_kpage[p.n] = tot[5];
        if (blockIdx.x == 0)
            *reinterpret_cast<int4*>(plan) = make_int4(p.tag, tot[0], head, tot[1]);   // C_TAG, C_ROWS, C_HEAD, C_TAKEN
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int i = tid; i < CA_COUNT * (p.n + 1); i += kTablesThreads) plan[C_HEADER + i] = s_arrays[i];
    if (alone)
        write_rows(p, s_arrays, tot[0], head, tot[1], blockIdx.x * kTablesThreads + tid, gridDim.x * kTablesThreads);
}

// A plan made for other dims (or by no pcf_chunk_tables call at all) is refused.
__device__ __forceinline__ bool plan_fits(const int32_t* plan, int32_t tag) {
    const bool ok = plan[C_TAG] == tag;
    if (!ok) set_dev_error(kDevErrBounds);
    return ok;
}

constexpr int kRowsThreads = 256;
__global__ void __launch_bounds__(kRowsThreads) chunk_rows_kernel(const TablesParams p) {
    extern __shared__ int32_t s_arrays[];
    grid_dep_wait();
    grid_dep_launch();
    for (int i = threadIdx.x; i < CA_COUNT * (p.n + 1); i += kRowsThreads) s_arrays[i] = p.plan[C_HEADER + i];
    const int4 h = *reinterpret_cast<const int4*>(p.plan);
    __syncthreads();
    write_rows(p, s_arrays, h.y, h.z, h.w, blockIdx.x * kRowsThreads + threadIdx.x, gridDim.x * kRowsThreads);
}

// ------------------------------------------------------------------ append
// Row i's key and value into slot slot_map[i] of the pools, every kv head.  A slot's position is
// fixed by its page (page_pos + r), and attention rotates a key by it; a row whose own position
// `at` differs (a recomputed token, kept behind its request's shared pages) is stored turned by the
// difference, R_{at - slot} k, so that R_slot of the stored key is R_at k.  Where the two agree the
// key is copied bit for bit.  A thread takes the 16-byte chunks c and c + d/16 of one head's key
// (the pairs i, i + d/2 that turn together) and of its value: 64 bytes in flight a thread.  Bound by HBM,
// with a thread a chunk and no loop to set up: 51 k rows of 8 kv heads, d 128, most of them turned, move
// 421 MB in 69.8 us (6.0 TB/s, 89 % of a plain copy); 64 rows take 2 us.
struct AppendParams {
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    __nv_bfloat16* k_pool;
    __nv_bfloat16* v_pool;
    const int32_t* slot_map;
    const int32_t* slot_pos;   // the slots' positions (row_pos of the tables)
    const int32_t* at;         // the rows' own positions, or null
    const float* rope;         // with `at`
    int64_t k_stride, v_stride;   // elements between rows
    int32_t max_rows, hkv, n_phys, max_pos;
};

template <int D>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
    constexpr int CPR = D / 16;
    grid_dep_wait();
    grid_dep_launch();
    const int64_t total = (int64_t)p.max_rows * p.hkv * CPR;
    for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < total; it += (int64_t)gridDim.x * 256) {
        const int c = (int)(it % CPR);
        const int64_t rh = it / CPR;
        const int h = (int)(rh % p.hkv);
        const int32_t row = (int32_t)(rh / p.hkv);
        const int32_t slot = p.slot_map[row];
        if (slot == -1) continue;
        if (slot < 0 || slot >= p.n_phys * kPage) {
            set_dev_error(kDevErrBounds);
            continue;
        }
        const __nv_bfloat16* ks = p.k + row * p.k_stride + h * D;
        const __nv_bfloat16* vs = p.v + row * p.v_stride + h * D;
        const uint4 v0 = *reinterpret_cast<const uint4*>(vs + 8 * c);
        const uint4 v1 = *reinterpret_cast<const uint4*>(vs + D / 2 + 8 * c);
        uint4 k0 = *reinterpret_cast<const uint4*>(ks + 8 * c);
        uint4 k1 = *reinterpret_cast<const uint4*>(ks + D / 2 + 8 * c);
        if (p.at != nullptr) {
            const int32_t at = p.at[row], from = p.slot_pos[row];
            if (at < 0 || at >= p.max_pos || from < 0 || from >= p.max_pos) {
                set_dev_error(kDevErrBounds);
                continue;
            }
            const int32_t by = at - from;
            if (by != 0) {
                const float sgn = by < 0 ? -1.f : 1.f;   // cos(-a) = cos a, sin(-a) = -sin a
                const float4* cs = reinterpret_cast<const float4*>(p.rope + (int64_t)abs(by) * D + 16 * c);
                const uint32_t ia[4] = {k0.x, k0.y, k0.z, k0.w}, ib[4] = {k1.x, k1.y, k1.z, k1.w};
                uint32_t oa[4], ob[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 q = cs[e];   // cos, sin of two frequencies
                    const float s0 = sgn * q.y, s1 = sgn * q.w;
                    const float a0 = bf16_lo(ia[e]), a1 = bf16_hi(ia[e]), b0 = bf16_lo(ib[e]), b1 = bf16_hi(ib[e]);
                    oa[e] = pack_bf16x2(fmaf(a0, q.x, -b0 * s0), fmaf(a1, q.z, -b1 * s1));
                    ob[e] = pack_bf16x2(fmaf(b0, q.x, a0 * s0), fmaf(b1, q.z, a1 * s1));
                }
                k0 = make_uint4(oa[0], oa[1], oa[2], oa[3]);
                k1 = make_uint4(ob[0], ob[1], ob[2], ob[3]);
            }
        }
        const int64_t dst = (((int64_t)(slot / kPage) * p.hkv + h) * kPage + slot % kPage) * D + 8 * c;
        *reinterpret_cast<uint4*>(p.k_pool + dst) = k0;
        *reinterpret_cast<uint4*>(p.k_pool + dst + D / 2) = k1;
        *reinterpret_cast<uint4*>(p.v_pool + dst) = v0;
        *reinterpret_cast<uint4*>(p.v_pool + dst + D / 2) = v1;
    }
}

}  // namespace pcf
