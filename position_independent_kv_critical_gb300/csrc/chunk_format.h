// Word map of the plan a pcf_chunk_tables call leaves on the device for the calls that append to
// and attend over the same chunk, and the limits both sides check.
//
// The lengths of the requests are known to the GPU only, so the plan holds what a host-built layout
// would: the lengths of this chunk (copied, so that the caller's may move on), the rows of every
// request and prefix sums of its work, from which each block of a persistent kernel finds its own
// share by bisection.
#pragma once
#include <stdint.h>

#include "../../include/pcf.h"
#include "layout_format.h"

#include <initializer_list>

namespace pcf {

constexpr int kMaxReqs = 4096;               // requests of one chunk batch (one block scans them)
constexpr int32_t kMaxChunkRows = 1 << 22;   // rows of one chunk batch
constexpr int32_t kMaxTotalPages = 1 << 26;  // pages of all requests together, repeats counted

enum : int {
    C_TAG = 0,        // of the dims the plan was made for (plan_tag)
    C_ROWS = 1,       // rows of the chunk; 0 also where the lengths were refused
    C_HEAD = 2,       // the free list's first page not taken before this chunk
    C_TAKEN = 3,      // pages taken for the chunk
    C_HEADER = 4
};
// arrays behind the header, n_reqs + 1 words each: tokens held, new tokens, first row, pages taken
// before the request, position of its first row; of the requests before it that have few rows their
// weight (their (page, kv head) units and run_weight for each of their runs) and their number; of those with
// more the weight of their row pairs (many_weight) and the pages they hold.  Behind the first positions: run_weight.
// Behind them the work split of both kinds: kStartWords words a worker, then kManyWords a block.
enum : int { CA_SEQ = 0, CA_NEW = 1, CA_ROW = 2, CA_TAKE = 3, CA_START = 4, CA_FEW = 5, CA_MANY = 6, CA_KPAGE = 7, CA_FEWN = 8, CA_COUNT = 9 };
// {request, kv head, page, units before; its pages, tokens held, new tokens, first row; tag, and for a block's
// first worker the blocks its first and last run reach: first, last; last}, and one entry more with all units
constexpr int kStartWords = 12;

PCF_HOST_DEVICE inline int64_t plan_array(int which, int32_t n_reqs) {
    return C_HEADER + (int64_t)which * (n_reqs + 1);
}
PCF_HOST_DEVICE inline int64_t plan_starts(int32_t n_reqs) {
    return (plan_array(CA_COUNT, n_reqs) + 3) / 4 * 4;
}
constexpr int kManyWords = 8;    // {request, kv head, row pair, key tile; weight, tag, weight of the first run's beginning in it, 0}
PCF_HOST_DEVICE inline int64_t plan_many(int32_t n_reqs, int32_t workers) {
    return plan_starts(n_reqs) + (int64_t)(workers + 1) * kStartWords;
}
// parts brought of runs that blocks share, one counter a block
PCF_HOST_DEVICE inline int64_t plan_count(int32_t n_reqs, int32_t workers, int32_t blocks) {
    return plan_many(n_reqs, workers) + (int64_t)blocks * kManyWords;
}
PCF_HOST_DEVICE inline int64_t plan_words(int32_t n_reqs, int32_t workers, int32_t blocks) {
    return plan_count(n_reqs, workers, blocks) + blocks;
}

// A request with more rows: row pair p holds the tokens [p tpp, (p + 1) tpp) of the chunk, tpp = 256 / g
// of them (two tiles of 128 rows, token by token, the g query heads of a kv head together), which see
// the slots up to seq + min(T, (p + 1) tpp) - 1.
PCF_HOST_DEVICE inline int32_t many_pairs(int32_t add, int32_t tpp) { return (add + tpp - 1) / tpp; }
PCF_HOST_DEVICE inline int32_t many_tiles(int32_t seq, int32_t add, int32_t tpp, int32_t pair) {
    const int32_t end = (pair + 1) * tpp < add ? (pair + 1) * tpp : add;
    return (seq + end + kTileKeys - 1) / kTileKeys;
}
// key tiles of the pairs before `pair` (not behind the last one): sum of floor((a + i tpp) / 128),
// a = seq + tpp + 127.  With m = 128 / tpp pairs to a tile (tpp divides 128, or is 256), i = m u + v
// adds u whole tiles and one more from v = v0 on, the first whose tokens cross a tile.  (tpp and m are
// powers of two; divisions by variables would cost more than all the rest.)
PCF_HOST_DEVICE inline int32_t log2_of(int32_t x) {
#ifdef __CUDA_ARCH__
    return __ffs(x) - 1;
#else
    return __builtin_ctz((unsigned)x);
#endif
}
PCF_HOST_DEVICE inline int64_t many_before(int32_t seq, int32_t tpp, int32_t pair) {
    const uint32_t end = (uint32_t)(seq + tpp + kTileKeys - 1);
    const int64_t a = end / kTileKeys, p = pair;
    if (tpp == 2 * kTileKeys) return p * a + p * (p - 1);
    const int32_t lt = log2_of(tpp), lm = log2_of(kTileKeys) - lt, m = 1 << lm;
    const int32_t r = (int32_t)(end % kTileKeys), u = pair >> lm, w = pair & (m - 1);
    const int32_t v0 = (kTileKeys - r + tpp - 1) >> lt;
    return p * a + (((int64_t)u * (u - 1) / 2) << lm) + (int64_t)u * w + (int64_t)u * (m - v0) + (w > v0 ? w - v0 : 0);
}

// Weight of the pairs of a (request, kv head) before `pair`, by which their tiles are dealt to the blocks: the
// key tiles, and kPairWeight more for each pair's beginning and end (its queries' copy, the first scores, the
// results' way out).  Six chunks of 100 to 700 tokens beside 26 single ones: 284 us without it, 279, 275 and
// 274 with 1, 2 and 3; nine chunks behind 0 to 1500 tokens 23.7, 21.1, 21.8 and 22.0.
constexpr int kPairWeight = 2;
PCF_HOST_DEVICE inline int64_t many_weight(int32_t seq, int32_t tpp, int32_t pair) {
    return many_before(seq, tpp, pair) + (int64_t)pair * kPairWeight;
}

// A request has few rows when its new tokens times the query heads of a kv head are at most this: two
// 8-row tiles a warp.  Reading the pages then bounds the attention (a key and value of 4 d bytes meet 4 d
// flops a row).  24 requests of 6 k tokens, 64/8 heads, d 128: 16 rows take 115 us in the few-row kernel
// and 186 in the other one, 24 rows 206 with four tiles a warp (eight warps of 255 registers) and 185 in
// the other one.
constexpr int kFewRows = 16;
// Warps of a block of the few-row kernel, each a worker: three a sub-partition, of 168 registers.
constexpr int kFewWarps = 12;

// Units go to the workers in contiguous runs as equal as can be, worker w from floor(w units / active) on:
// the longer runs are spread evenly over the blocks, and where the runs of a batch are alike (one request:
// its kv heads) their ends fall on ends of workers, which spares a worker a second run with its queries
// and partial results (one request of 4 k tokens: 14.3 us with the longer runs on the first workers, 11.8
// so).  With fewer units than workers the first ones take one each (a run's parts then sit in few blocks).
// `left` is more / active in units of 2^-32, rounded up (more units left over, active <= 12 * 4096 workers:
// w left / 2^32 is then within 2^-16 of its value, and its floor exact); no division a worker.  units < 2^30.
struct Deal {
    uint32_t units, active, each, left;
    PCF_HOST_DEVICE Deal(int32_t n, int32_t workers) : units(n), active(n < workers ? n : workers), each(0), left(0) {
        if (n <= 0) return;
        each = units / active;
        const uint32_t more = units - each * active, hi = (more << 16) / active, rest = (more << 16) - hi * active;
        left = more ? (hi << 16 | (rest << 16) / active) + 1 : 0;
    }
    PCF_HOST_DEVICE int32_t first(uint32_t w) const {
        return (int32_t)(w < active ? w * each + (uint32_t)((uint64_t)w * left >> 32) : units);
    }
    PCF_HOST_DEVICE int32_t owner(int32_t u) const {   // (0 <= u < units): the last worker that begins at or before u
        int32_t w = (int32_t)((float)u * ((float)active / (float)units));
        w = w < (int32_t)active ? w : (int32_t)active - 1;
        while (first(w) > u) --w;
        while (first(w + 1) <= u) ++w;
        return w;
    }
};

// What beginning and ending a run (queries loaded and rotated, a result written) costs a worker, in units, in
// the dealing of a batch that gives every worker four units or more (so that each has one at least, whatever
// the runs).  48 drafts behind 100 to 9000 tokens: 146 us without it, 134 with 1, 2 or 3.  With fewer units a
// worker latencies count, and a unit is a unit.
constexpr int kRunWeight = 1;
PCF_HOST_DEVICE inline int32_t run_weight(int32_t units, int32_t workers) { return units >= 4 * workers ? kRunWeight : 0; }

PCF_HOST_DEVICE inline int32_t chunk_sms(int32_t n_sms) { return n_sms > 0 ? n_sms : kDefaultSms; }

inline pcf_status check_chunk_dims(const pcf_chunk_dims* c) {
    if (!c) return PCF_ERR_INVALID_ARG;
    if (c->n_reqs < 1 || c->n_reqs > kMaxReqs || c->max_rows < 1 || c->max_rows > kMaxChunkRows || c->max_chunk < 1 ||
        c->max_chunk > c->max_rows || c->max_pages < 1 || c->max_pages > kMaxPosLimit / kPage ||
        c->max_total_pages < 1 || c->max_total_pages > kMaxTotalPages || c->n_q_heads < 1 || c->n_kv_heads < 1 ||
        c->n_q_heads % c->n_kv_heads != 0 || c->n_q_heads > 1024 || c->max_pos < kPage || c->max_pos > kMaxPosLimit ||
        c->n_phys_pages < 1 || c->n_sms > 4096)
        return PCF_ERR_INVALID_ARG;
    // slots and the rows of the pool's tensor maps are 32-bit numbers
    if ((int64_t)c->n_phys_pages * c->n_kv_heads * kPage > INT32_MAX) return PCF_ERR_INVALID_ARG;
    // and so are the rows of the rotated copies that longer chunks use
    if ((int64_t)c->max_chunk * (c->n_q_heads / c->n_kv_heads) > kFewRows &&
        ((int64_t)c->max_rows * c->n_q_heads > INT32_MAX ||
         (int64_t)c->max_total_pages * c->n_kv_heads * kPage > INT32_MAX))
        return PCF_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return PCF_ERR_UNSUPPORTED;
    if (kTileRows % (c->n_q_heads / c->n_kv_heads) != 0) return PCF_ERR_UNSUPPORTED;
    return PCF_OK;
}

// Workspace of pcf_chunk_attention (byte offsets).  Few-row partial results: a worker's first run,
// when the block has more of it to come, and per block the two runs it shares with its neighbours.
struct ChunkWs {
    size_t worker_o, block_o, block_ml;
    // requests with more rows: rotated queries and keys, the two runs a block shares with its neighbours
    size_t q_rot, k_rot, many_o, many_ml, many_desc, total;
};
inline size_t chunk_align(size_t x) { return (x + 255) / 256 * 256; }
inline bool any_many(const pcf_chunk_dims* c) {   // a request may have more than few rows
    return (int64_t)c->max_chunk * (c->n_q_heads / c->n_kv_heads) > kFewRows;
}
// Most rows of a request the few-row kernel takes: 8 or 16, what the dims allow.  Where some request may
// have more, so that the other kernels run anyway, what a single token needs: a second row tile costs
// every request of the batch.
inline int few_limit(const pcf_chunk_dims* c) {
    const int64_t g = c->n_q_heads / c->n_kv_heads;
    return (any_many(c) ? g : c->max_chunk * g) <= 8 ? 8 : kFewRows;
}
inline int few_tiles(const pcf_chunk_dims* c) { return few_limit(c) / 8; }   // tiles of 8 rows a warp
inline int few_workers(const pcf_chunk_dims* c) { return kFewWarps * chunk_sms(c->n_sms); }
// A word the kernels compare with the plan's, so that a plan made for other dims (or by no
// pcf_chunk_tables call at all) is refused instead of read.
inline int32_t plan_tag(const pcf_chunk_dims* c) {
    uint32_t h = 2166136261u;
    for (int32_t v : {c->n_reqs, c->max_pages, c->max_rows, c->max_chunk, c->max_total_pages, c->n_q_heads, c->n_kv_heads,
                      c->head_dim, c->n_phys_pages, c->max_pos, chunk_sms(c->n_sms)})
        h = (h ^ (uint32_t)v) * 16777619u;
    return (int32_t)(h | 1u);   // never 0
}

inline ChunkWs chunk_ws(const pcf_chunk_dims* c) {
    ChunkWs w;
    const size_t rows = 8 * (size_t)few_tiles(c), blocks = chunk_sms(c->n_sms), d = c->head_dim;
    w.worker_o = 0;
    w.block_o = chunk_align(w.worker_o + (size_t)few_workers(c) * rows * d * 4);
    w.block_ml = chunk_align(w.block_o + blocks * 2 * rows * d * 4);
    w.q_rot = chunk_align(w.block_ml + blocks * 2 * rows * 8);
    w.total = w.k_rot = w.many_o = w.many_ml = w.many_desc = w.q_rot;
    if (!any_many(c)) return w;
    w.k_rot = chunk_align(w.q_rot + (size_t)c->max_rows * c->n_q_heads * d * 2);
    w.many_o = chunk_align(w.k_rot + (size_t)c->max_total_pages * kPage * c->n_kv_heads * d * 2);
    w.many_ml = chunk_align(w.many_o + blocks * 2 * 256 * d * 4);
    w.many_desc = chunk_align(w.many_ml + blocks * 2 * 256 * 8);
    w.total = chunk_align(w.many_desc + blocks * 32);
    return w;
}

}  // namespace pcf
