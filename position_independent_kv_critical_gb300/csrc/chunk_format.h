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
    C_HEADER = 16
};
// arrays behind the header, n_reqs + 1 words each
enum : int { CA_SEQ = 0, CA_NEW = 1, CA_ROW = 2, CA_TAKE = 3, CA_START = 4, CA_COUNT = 5 };

PCF_HOST_DEVICE inline int64_t plan_array(int which, int32_t n_reqs) {
    return C_HEADER + (int64_t)which * (n_reqs + 1);
}
PCF_HOST_DEVICE inline int64_t plan_words(int32_t n_reqs) { return plan_array(CA_COUNT, n_reqs); }

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

}  // namespace pcf
