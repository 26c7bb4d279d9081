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

namespace pcf {

constexpr int32_t kPlanMagic = 0x504B4843;   // "CHKP"
constexpr int kMaxReqs = 4096;               // requests of one chunk batch (one block scans them)
constexpr int32_t kMaxChunkRows = 1 << 22;   // rows of one chunk batch
constexpr int32_t kMaxTotalPages = 1 << 26;  // pages of all requests together, repeats counted

enum : int {
    C_MAGIC = 0, C_N_REQS = 1, C_MAX_PAGES = 2, C_MAX_ROWS = 3, C_HQ = 4, C_HKV = 5, C_D = 6, C_N_PHYS = 7,
    C_MAX_POS = 8,
    C_ROWS = 9,       // rows of the chunk; 0 also where the lengths were refused
    C_HEAD = 10,      // the free list's first page not taken before this chunk
    C_TAKEN = 11,     // pages taken for the chunk
    C_BAD = 12,       // 1: the lengths were refused and nothing was done
    C_WORKERS = 13,   // warps the few-row requests' pages are dealt to
    C_HEADER = 16
};
// arrays behind the header, n_reqs + 1 words each: tokens held, new tokens, first row, pages taken
// before the request, position of its first row, and the (page, kv head) units of the requests
// before it that have few rows; then the few-row work split, kStartWords words a worker
enum : int { CA_SEQ = 0, CA_NEW = 1, CA_ROW = 2, CA_TAKE = 3, CA_START = 4, CA_FEW = 5, CA_COUNT = 6 };
constexpr int kStartWords = 8;   // {request, kv head, page, units; its pages, tokens held, new tokens, first row}

PCF_HOST_DEVICE inline int64_t plan_array(int which, int32_t n_reqs) {
    return C_HEADER + (int64_t)which * (n_reqs + 1);
}
PCF_HOST_DEVICE inline int64_t plan_starts(int32_t n_reqs) {
    return (plan_array(CA_COUNT, n_reqs) + 3) / 4 * 4;
}
PCF_HOST_DEVICE inline int64_t plan_words(int32_t n_reqs, int32_t workers) {
    return plan_starts(n_reqs) + (int64_t)workers * kStartWords;
}

// A request has few rows when its new tokens times the query heads of a kv head are at most this:
// two 16-row tiles of mma.sync a warp.  Below, reading the pages bounds the attention (a key and
// value of 4 d bytes meet 4 d flops a row, 32 flops a byte at most).
constexpr int kFewRows = 32;
constexpr int kFewWarps = 8;   // warps of a block of the few-row kernel, each a worker

// Units go to the workers in equal runs, worker w from the w-th of `active` equal parts on; with
// fewer units than workers the first ones take one each, so that a run's parts sit in few blocks.
PCF_HOST_DEVICE inline int64_t few_active(int64_t units, int32_t workers) { return units < workers ? units : workers; }

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
    if (c->head_dim != 64 && c->head_dim != 128) return PCF_ERR_UNSUPPORTED;
    if (kTileRows % (c->n_q_heads / c->n_kv_heads) != 0) return PCF_ERR_UNSUPPORTED;
    return PCF_OK;
}

// Workspace of pcf_chunk_attention (byte offsets).  Few-row partial results: a worker's first run,
// when the block has more of it to come, and per block the two runs it shares with its neighbours.
struct ChunkWs {
    size_t worker_o, block_o, block_ml, block_desc, total;
};
inline size_t chunk_align(size_t x) { return (x + 255) / 256 * 256; }
inline int few_tiles(const pcf_chunk_dims* c) {   // 16-row tiles a warp: 1 when no request can have more
    return (int64_t)c->max_chunk * (c->n_q_heads / c->n_kv_heads) <= 16 ? 1 : 2;
}
inline ChunkWs chunk_ws(const pcf_chunk_dims* c) {
    ChunkWs w;
    const size_t rows = 16 * (size_t)few_tiles(c), blocks = chunk_sms(c->n_sms), d = c->head_dim;
    w.worker_o = 0;
    w.block_o = chunk_align(w.worker_o + blocks * kFewWarps * rows * d * 4);
    w.block_ml = chunk_align(w.block_o + blocks * 2 * rows * d * 4);
    w.block_desc = chunk_align(w.block_ml + blocks * 2 * rows * 8);
    w.total = chunk_align(w.block_desc + blocks * 16);
    return w;
}

}  // namespace pcf
