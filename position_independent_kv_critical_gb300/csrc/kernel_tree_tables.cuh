// Trees of drafted tokens: each node's position and the nodes it goes on from, the branch that the
// model's choices confirm, and the move of that branch's keys and values.
//
// Node t of request b is row row_base[b] + t of the chunk and sits in slot seq + t; parent[t] < t is the
// node it goes on from, -1 the last token held.
#pragma once
#include "kernel_chunk_tables.cuh"
#include "ptx.cuh"
#include "tree_format.h"

namespace pcf {

// ------------------------------------------------------------------ tables
struct TreeTablesParams {
    const int32_t* chunk;      // plan of the chunk
    const int32_t* parent;     // [max_rows]
    int32_t* row_pos;          // [max_rows]
    uint32_t* seen;            // [max_rows][words]
    int32_t* plan;
    int32_t n, max_rows, words, hkv, g, blocks, chunk_tag, tag;
};

constexpr int kTreeWarps = 8;
constexpr int kTreeThreads = kTreeWarps * 32;

// Block 0 copies the lengths, scans the requests' weights and writes every block's share of the
// attention; the others take a request a warp.
// A warp takes its tree 32 nodes at a time.  Inside the 32 a node's line goes back by pointer doubling
// over lanes: after step i it reaches 2^i nodes back, five steps reach any (parents come first).  The
// first node of a line inside the 32 has its parent among the 32s before, whose bits are complete: a
// copy of those and the line's own word make the node's bits, whatever the depth.  Bound by dependent loads and
// barriers: 64 trees of 16 nodes 2.8 us in a replayed graph, 512 of up to 256 nodes 6.2 (9.4 with a tree's parents
// loaded 32 at a time).
__global__ void __launch_bounds__(kTreeThreads) tree_tables_kernel(const TreeTablesParams p) {
    extern __shared__ int32_t s_words[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dep_wait();
    grid_dep_launch();
    const bool fits = p.chunk[C_TAG] == p.chunk_tag;
    const int32_t rows = fits ? p.chunk[C_ROWS] : 0;
    const int32_t* seq = p.chunk + plan_array(CA_SEQ, p.n);
    const int32_t* add = p.chunk + plan_array(CA_NEW, p.n);
    const int32_t* base = p.chunk + plan_array(CA_ROW, p.n);
    if (blockIdx.x == 0) {
        __shared__ int s_warp[kTreeWarps];
        int32_t* s_work = s_words;                     // [n + 1] weight of the requests before
        if (tid == 0 && !fits) set_dev_error(kDevErrBounds);
        const int per = (p.n + kTreeThreads - 1) / kTreeThreads;
        const int b0 = min(p.n, tid * per), b1 = min(p.n, b0 + per);
        auto weight = [&](int b) {
            const int32_t n = fits ? add[b] : 0;
            if (n == 0) return 0;
            const int64_t w = (int64_t)(tree_units(seq[b] + n) + kTreeRunWeight) * tree_pairs(n, p.g) * p.hkv;
            return (int)min(w, (int64_t)kSumLimit);
        };
        int sum = 0;
        for (int b = b0; b < b1; ++b) sum = sat_add(sum, weight(b));
        int x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x = sat_add(x, y);
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        int before = 0, all = 0;
        for (int w = 0; w < kTreeWarps; ++w) {
            if (w < warp) before = sat_add(before, s_warp[w]);
            all = sat_add(all, s_warp[w]);
        }
        // (more work than the shares can number: none of it is done)
        const bool too_much = all >= kSumLimit;
        if (too_much && tid == 0) set_dev_error(kDevErrBounds);
        before += x - sum;
        for (int b = b0; b < b1; ++b) {
            s_work[b] = too_much ? 0 : before;
            before = sat_add(before, weight(b));
        }
        if (too_much) all = 0;
        if (tid == 0) s_work[p.n] = all;
        __syncthreads();
        for (int b = tid; b <= p.n; b += kTreeThreads) {
            p.plan[tree_array(TA_SEQ, p.n) + b] = b < p.n && fits ? seq[b] : 0;
            p.plan[tree_array(TA_NEW, p.n) + b] = b < p.n && fits ? add[b] : 0;
            p.plan[tree_array(TA_ROW, p.n) + b] = fits ? base[b] : 0;
            p.plan[tree_array(TA_WORK, p.n) + b] = s_work[b];
        }
        if (tid == kTreeThreads - 1)
            *reinterpret_cast<int4*>(p.plan) = make_int4(p.tag, too_much ? 0 : rows, 0, fits ? p.chunk[plan_step(p.n)] : 0);   // T_TAG, T_ROWS, T_DONE, T_STEP
        const Deal deal(all, p.blocks);
        for (int w = tid; w < p.blocks; w += kTreeThreads) {
            const int32_t u0 = deal.first(w);
            int4 e = make_int4(0, 0, 0, 0), f = make_int4(deal.first(w + 1) - u0, p.tag, 0, 0), l = e;
            if (f.x > 0) {
                const int b = row_request(s_work, p.n, u0);
                const int32_t pairs = tree_pairs(add[b], p.g), run = tree_units(seq[b] + add[b]) + kTreeRunWeight;
                const int32_t local = u0 - s_work[b], r = local / run, at = local - r * run;
                e = make_int4(b, r / pairs, r % pairs, max(0, at - kTreeRunWeight));
                f.z = max(0, kTreeRunWeight - at);
                l = make_int4(seq[b], add[b], base[b], 0);
            }
            int4* dst = reinterpret_cast<int4*>(p.plan + tree_shares(p.n)) + 3 * w;
            dst[0] = e;
            dst[1] = f;
            dst[2] = l;
        }
        return;
    }
    const int words = p.words;
    uint32_t* s_bits = reinterpret_cast<uint32_t*>(s_words) + warp * 32 * words * (words + 1);   // [node][word]
    int32_t* s_depth = reinterpret_cast<int32_t*>(s_bits + 32 * words * words);                  // [node]
    bool bad = false;
    for (int b = (blockIdx.x - 1) * kTreeWarps + warp; b < p.n && fits; b += (gridDim.x - 1) * kTreeWarps) {
        const int32_t n = add[b], first = base[b], pos0 = p.chunk[plan_array(CA_START, p.n) + b];
        int32_t ups[kTreeMaxWords];                    // (all of a tree's parents on their way at once)
#pragma unroll
        for (int k = 0; k < kTreeMaxWords; ++k) ups[k] = 32 * k + lane < n ? p.parent[first + 32 * k + lane] : -1;
#pragma unroll
        for (int k = 0; k < kTreeMaxWords; ++k) {
            if (32 * k >= n) break;
            const int t = 32 * k + lane;
            int32_t up = ups[k];
            if (t < n && (up < -1 || up >= t)) {
                bad = true;
                up = -1;
            }
            // the line inside these 32: its nodes, the lane it has reached
            uint32_t line = 1u << lane;
            int at = up >= 32 * k ? up - 32 * k : lane;
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                line |= __shfl_sync(0xffffffffu, line, at);
                at = __shfl_sync(0xffffffffu, at, at);
            }
            const int32_t out = __shfl_sync(0xffffffffu, up, at);      // (of the line's first node here)
            const int32_t depth = __popc(line) + (out >= 0 ? s_depth[out] : 0);
            if (t < n) {
                s_depth[t] = depth;
                uint32_t* dst = p.seen + (int64_t)(first + t) * words;
                p.row_pos[first + t] = pos0 + depth - 1;
                for (int w = 0; w < words; ++w) {
                    const uint32_t v = w == k ? line : w < k && out >= 0 ? s_bits[out * words + w] : 0u;
                    s_bits[t * words + w] = v;
                    dst[w] = v;
                }
            }
            __syncwarp();
        }
        __syncwarp();
    }
    if (bad) set_dev_error(kDevErrBounds);
    for (int64_t r = rows + (int64_t)(blockIdx.x - 1) * kTreeThreads + tid; r < p.max_rows; r += (int64_t)(gridDim.x - 1) * kTreeThreads) {
        p.row_pos[r] = -1;
        for (int w = 0; w < words; ++w) p.seen[r * words + w] = 0;
    }
}

// A plan made for other dims (or by no pcf_tree_tables call at all) is refused.
__device__ __forceinline__ bool tree_fits(const int32_t* plan, int32_t tag) {
    const bool ok = plan[T_TAG] == tag;
    if (!ok) set_dev_error(kDevErrBounds);
    return ok;
}

// ------------------------------------------------------------------ accept
struct TreeAcceptParams {
    const int32_t* chunk;
    int32_t* plan;
    const int32_t* parent;     // [max_rows]
    const int32_t* draft;      // [max_rows] the nodes' tokens
    const int32_t* choice;     // [max_rows] the model's token behind each node
    const int32_t* root;       // [n] the model's token behind the held ones, or null: node 0 is kept
    const int32_t* block_table;
    int32_t* free_pages;
    int32_t* path;             // [max_rows]
    int32_t* kept;             // [n]
    int32_t* next;             // [n]
    int32_t* seq_out;          // [n]
    int32_t* head_out;         // [1]
    int32_t n, max_rows, max_pages, n_free, chunk_tag, tag;
};

// A warp takes a request: every node whose token is what the model chose behind its parent offers itself to that
// parent, the lowest one stays (of siblings with the same token the first), and one lane follows the offers from the
// held tokens on.  (512 trees of up to 256 nodes: 9.6 us; 16.5 with a ballot over all nodes a step and pages given
// back one behind the other.)  The block
// that is done last scans the pages that the branches need and gives the others back: taken pages lie in the free
// list in request order, so what is needed stays in front and the rest, in the same order, becomes the list's next
// entries.
__global__ void __launch_bounds__(kTreeThreads) tree_accept_kernel(const TreeAcceptParams p) {
    __shared__ int s_last, s_warp[kTreeWarps];
    __shared__ int s_next[kTreeWarps][kTreeMaxNodes + 1];     // the lowest node that goes on from node t; [0]: from the held tokens
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int* next = s_next[warp] + 1;
    grid_dep_wait();
    grid_dep_launch();
    const int4 of_plan = *reinterpret_cast<const int4*>(p.plan);
    if (p.chunk[C_TAG] != p.chunk_tag || of_plan.x != p.tag) {
        if (tid == 0) set_dev_error(kDevErrBounds);
        return;
    }
    // Trees of an earlier chunk: what was attended over and what tree_keep would move are that chunk's.  Nothing is
    // kept, so that nothing moves.  (Looked at below, behind the requests' own loads.)
    const int32_t rows = p.chunk[C_ROWS], head = p.chunk[C_HEAD], taken = p.chunk[C_TAKEN];
    const bool stale = p.chunk[plan_step(p.n)] != of_plan.w;           // (T_STEP)
    const int32_t* seq = p.chunk + plan_array(CA_SEQ, p.n);
    const int32_t* add = p.chunk + plan_array(CA_NEW, p.n);
    const int32_t* base = p.chunk + plan_array(CA_ROW, p.n);
    const int32_t* take = p.chunk + plan_array(CA_TAKE, p.n);
    bool bad = false;
    for (int b = blockIdx.x * kTreeWarps + warp; b < p.n; b += gridDim.x * kTreeWarps) {
        const int32_t n = add[b], first = base[b];
        const int32_t* choice = p.choice + first;
        const int32_t root = p.root ? p.root[b] : -1;
        constexpr int kNobody = 1 << 30;
        for (int i = lane; i <= n; i += 32) next[i - 1] = kNobody;
        int32_t up[kTreeMaxWords], token[kTreeMaxWords];
#pragma unroll
        for (int k = 0; k < kTreeMaxWords; ++k) {
            const int t = 32 * k + lane;
            up[k] = t < n ? p.parent[first + t] : -2;
            token[k] = t < n ? p.draft[first + t] : 0;
        }
        uint32_t hit = 0;                              // bit k: node 32 k + lane is what was chosen
#pragma unroll
        for (int k = 0; k < kTreeMaxWords; ++k) {
            const int t = 32 * k + lane, at = up[k];
            const bool fine = t < n && at >= -1 && at < t;
            bad |= t < n && !fine;
            const int32_t said = fine && at >= 0 ? choice[at] : root;
            if (fine && (at >= 0 || p.root ? token[k] == said : t == 0)) hit |= 1u << k;
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kTreeMaxWords; ++k)
            if (hit >> k & 1u) atomicMin(next + up[k], 32 * k + lane);
        __syncwarp();
        if (stale) {
            if (lane == 0) p.kept[b] = 0;
            continue;
        }
        int32_t at = -1, count = 0;
        if (lane == 0)
            for (int32_t to; (to = next[at]) != kNobody; ++count) {
                at = to;
                p.path[first + count] = at;
            }
        at = __shfl_sync(0xffffffffu, at, 0);
        count = __shfl_sync(0xffffffffu, count, 0);
        for (int i = count + lane; i < n; i += 32) p.path[first + i] = -1;
        if (lane == 0) {
            p.kept[b] = count;
            p.next[b] = count > 0 ? choice[at] : root;
            p.seq_out[b] = seq[b] + count;
        }
    }
    if (bad || stale) set_dev_error(kDevErrBounds);
    if (stale) return;
    for (int64_t r = rows + (int64_t)blockIdx.x * kTreeThreads + tid; r < p.max_rows; r += (int64_t)gridDim.x * kTreeThreads)
        p.path[r] = -1;
    __syncthreads();
    if (tid == 0) s_last = atomic_inc_acq_rel_gpu(p.plan + T_DONE, gridDim.x - 1) == (int)gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
    // what a request's part of the taken pages begins with and where it goes on, in shared memory for all threads
    __shared__ int32_t s_to[kMaxReqs], s_from[kMaxReqs];
    __shared__ uint8_t s_back[kMaxReqs];               // pages it gives back: a tree starts 16 at most
    const int per = (p.n + kTreeThreads - 1) / kTreeThreads;
    const int b0 = min(p.n, tid * per), b1 = min(p.n, b0 + per);
    int sum = 0;
#pragma unroll 2
    for (int b = b0; b < b1; ++b) {
        const int32_t s = seq[b], held = pages_of(s), enough = add[b] > 0 ? pages_of(s + __ldcg(p.kept + b)) : held;
        s_to[b] = take[b] - sum;
        s_from[b] = enough;
        s_back[b] = (uint8_t)(take[b + 1] - take[b] - (enough - held));
        sum += enough - held;
    }
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int before = x - sum, all = 0;
    for (int w = 0; w < kTreeWarps; ++w) {
        if (w < warp) before += s_warp[w];
        all += s_warp[w];
    }
    for (int b = b0; b < b1; ++b) s_to[b] -= before;
    // (another list than the chunk's: all that was taken stays taken, for the list's order does not change and pages that
    // the branches hold lie behind its first ones)
    const bool refused = head < 0 || taken < 0 || head > p.n_free - taken;
    if (tid == 0) p.head_out[0] = head + (refused ? taken : all);
    if (refused) {
        if (tid == 0) set_dev_error(kDevErrBounds);
        return;
    }
    __syncthreads();
    constexpr int PLACES = kTreeMaxNodes / kPage;
    for (int i0 = tid; i0 < p.n * PLACES; i0 += 8 * kTreeThreads) {      // (eight places in flight a thread)
        int32_t page[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * kTreeThreads, b = i / PLACES;
            if (b < p.n && i % PLACES < s_back[b]) page[k] = p.block_table[(int64_t)b * p.max_pages + s_from[b] + i % PLACES];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * kTreeThreads, b = i / PLACES;
            if (b < p.n && i % PLACES < s_back[b]) p.free_pages[head + all + s_to[b] + i % PLACES] = page[k];
        }
    }
}

// ------------------------------------------------------------------ keep
constexpr int kKeepLayers = 64;     // layers of one launch (their pools' addresses are its arguments)
struct TreeKeepParams {
    const int32_t* plan;
    const int32_t* path;
    const int32_t* kept;
    const int32_t* block_table;
    int32_t n, max_pages, hkv, n_phys, pools_n, per_block, tag;
    uint4* pools[2 * kKeepLayers];  // keys and values of every layer
};

// The i-th node of the branch moves from slot seq + path[i] to slot seq + i.  path[i] >= i, so a slot that is written
// is never one that a later i reads: a thread takes one 16-byte column of a head and goes through the branch in
// order, and needs no other thread.  A block lists a request's moves once, for two to eight pools (as many as leave six
// blocks a SM; 128 requests in 32 layers: 15.5 us, 20.3 with a block a pool; one request: 2.6 with two, 3.7 with
// eight); two pools' next four moves are in flight a thread.
constexpr int kKeepPools = 8, kKeepThreads = 256;   // pools of a block at most
template <int D>
__global__ void __launch_bounds__(kKeepThreads) tree_keep_kernel(const __grid_constant__ TreeKeepParams p) {
    constexpr int CH = D / 8;
    __shared__ int2 s_move[kTreeMaxNodes];             // rows of head 0 in the pool: from, to
    __shared__ int s_warp[kKeepThreads / 32];
    grid_dep_wait();
    grid_dep_launch();
    if (!tree_fits(p.plan, p.tag)) return;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t seq = p.plan[tree_array(TA_SEQ, p.n) + b], add = p.plan[tree_array(TA_NEW, p.n) + b];
    const int32_t first = p.plan[tree_array(TA_ROW, p.n) + b];
    if (add == 0) return;
    int32_t count = p.kept[b];
    if (count < 0 || count > add) {
        set_dev_error(kDevErrBounds);
        return;
    }
    // thread i has the i-th node (a tree has no more nodes than the block threads)
    static_assert(kTreeMaxNodes <= kKeepThreads, "a thread a node");
    bool moves = false;
    int2 move = make_int2(0, 0);
    if (tid < count) {
        const int32_t* table = p.block_table + (int64_t)b * p.max_pages;
        const int32_t t = p.path[first + tid];
        if (t < tid || t >= add) {
            set_dev_error(kDevErrBounds);
        } else if (t > tid) {
            const int32_t from = table[(seq + t) / kPage], to = table[(seq + tid) / kPage];
            moves = from >= 0 && from < p.n_phys && to >= 0 && to < p.n_phys;
            if (!moves) set_dev_error(kDevErrBounds);
            // (pages * heads * 16 is below 2^31)
            move = make_int2(from * p.hkv * kPage + (seq + t) % kPage, to * p.hkv * kPage + (seq + tid) % kPage);
        }
    }
    const uint32_t in_warp = __ballot_sync(0xffffffffu, moves);
    if (lane == 0) s_warp[warp] = __popc(in_warp);
    __syncthreads();
    int at = 0;
    count = 0;
    for (int w = 0; w < kKeepThreads / 32; ++w) {
        if (w < warp) at += s_warp[w];
        count += s_warp[w];
    }
    if (moves) s_move[at + __popc(in_warp & ((1u << lane) - 1))] = move;
    __syncthreads();
    const int p0 = blockIdx.y * p.per_block, pools = min(p.per_block, p.pools_n - p0), columns = p.hkv * CH;
    // (pools in pairs: a pair and a column a thread)
    for (int x = tid; x < (pools + 1) / 2 * columns; x += kKeepThreads) {
        const int c = x % columns, q = p0 + x / columns * 2;
        const int64_t col = (int64_t)(c / CH) * kPage * CH + c % CH;
        uint4* pool[2] = {p.pools[q] + col, q + 1 < p0 + pools ? p.pools[q + 1] + col : nullptr};
        for (int i0 = 0; i0 < count; i0 += 4) {
            uint4 v[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i0 + i < count && pool[k]) v[k][i] = pool[k][(int64_t)s_move[i0 + i].x * CH];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i0 + i < count && pool[k]) pool[k][(int64_t)s_move[i0 + i].y * CH] = v[k][i];
        }
    }
}

}  // namespace pcf
