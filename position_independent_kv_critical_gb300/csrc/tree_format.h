// Word map of the plan a pcf_tree_tables call leaves on the device for the calls that attend over a
// tree of drafted tokens and keep a branch of it, and the limits both sides check.
//
// The tree's nodes are the rows of a chunk (chunk_format.h): the plan repeats that chunk's lengths and
// adds the attention's work split.  A run is one (request, kv head, row pair): a row pair holds 256 / g
// nodes (two tiles of 128 rows, node by node, the g query heads of a kv head together) and meets every
// slot of its request, nodes behind its own among them (hidden by their bits): a request's runs are then
// all alike, and their places follow from two divisions.
#pragma once
#include <stdint.h>

#include "../../include/pcf.h"
#include "chunk_format.h"

namespace pcf {

constexpr int kTreeMaxNodes = PCF_TREE_MAX_NODES;
constexpr int kTreeMaxBlocks = 4096;          // blocks of the attention (pcf_chunk_dims.n_sms)
constexpr int kTreeMaxWords = kTreeMaxNodes / 32;
constexpr int kTreeUnit = 64;                 // keys of a unit of work (four pages)
constexpr int kTreePagesPerUnit = kTreeUnit / kPage;

enum : int {
    T_TAG = 0,       // of the dims the plan was made for (tree_tag)
    T_ROWS = 1,      // nodes of all requests together; 0 also where the chunk's lengths were refused
    T_DONE = 2,      // blocks of pcf_tree_accept that are done (0 between calls)
    T_STEP = 3,      // the chunk plan's step (plan_step)
    T_HEADER = 4
};
// arrays behind the header, n_reqs + 1 words each: tokens held, nodes, first row, weight of the requests
// before; then kTreeShareWords a block
enum : int { TA_SEQ = 0, TA_NEW = 1, TA_ROW = 2, TA_WORK = 3, TA_COUNT = 4 };
// {request, kv head, row pair, unit; weight, tag, weight of the first run's beginning in it, 0; the request's tokens
// held, nodes, first row, 0}
constexpr int kTreeShareWords = 12;

PCF_HOST_DEVICE inline int64_t tree_array(int which, int32_t n_reqs) {
    return T_HEADER + (int64_t)which * (n_reqs + 1);
}
PCF_HOST_DEVICE inline int64_t tree_shares(int32_t n_reqs) { return (tree_array(TA_COUNT, n_reqs) + 3) / 4 * 4; }
PCF_HOST_DEVICE inline int64_t tree_plan_words(int32_t n_reqs, int32_t blocks) {
    return tree_shares(n_reqs) + (int64_t)blocks * kTreeShareWords;
}

// Weight of a run's beginning and end in the dealing, in units (12 requests of 200 to 256 nodes, 64/8 heads, 16 runs a
// head behind 500 to 4000 tokens: 330 us with 2, 314 with 4, 305 with 6 and with 8; 48 ragged trees 235, 233, 234 and 236).
constexpr int kTreeRunWeight = 6;
PCF_HOST_DEVICE inline int32_t tree_pairs(int32_t nodes, int32_t g) { return (nodes * g + 2 * kTileRows - 1) / (2 * kTileRows); }
PCF_HOST_DEVICE inline int32_t tree_units(int32_t slots) { return (slots + kTreeUnit - 1) / kTreeUnit; }

inline int32_t tree_words(const pcf_chunk_dims* c) { return (c->max_chunk + 31) / 32; }   // 32-bit words of a row's bits
inline pcf_status check_tree_dims(const pcf_chunk_dims* c) {
    const pcf_status s = check_chunk_dims(c);
    if (s != PCF_OK) return s;
    if ((int64_t)c->max_rows * c->n_q_heads > INT32_MAX) return PCF_ERR_INVALID_ARG;   // rows of the rotated queries
    return c->max_chunk > kTreeMaxNodes ? PCF_ERR_UNSUPPORTED : PCF_OK;
}
inline int32_t tree_tag(const pcf_chunk_dims* c) { return (int32_t)((uint32_t)plan_tag(c) * 2654435761u | 1u); }

constexpr int kMaxKeepLayers = 4096;     // layers of one pcf_tree_keep

// Workspace of pcf_tree_attention (byte offsets): rotated queries, the two runs a block shares with its neighbours.
struct TreeWs {
    size_t q_rot, part_o, part_ml, desc, total;
};
inline TreeWs tree_ws(const pcf_chunk_dims* c) {
    TreeWs w;
    const size_t blocks = chunk_sms(c->n_sms);
    w.q_rot = 0;
    w.part_o = chunk_align((size_t)c->max_rows * c->n_q_heads * c->head_dim * 2);
    w.part_ml = chunk_align(w.part_o + blocks * 2 * 2 * kTileRows * c->head_dim * 4);
    w.desc = chunk_align(w.part_ml + blocks * 2 * 2 * kTileRows * 8);
    w.total = chunk_align(w.desc + blocks * 32);
    return w;
}

}  // namespace pcf
