// shared_attn.h -- what the C-ABI layer and shared_attn.cu share: the plan's layout in the
// workspace and the launchers (not part of the public interface).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bg_attn.h"

namespace bg {

constexpr int kShKeys = 128;          // keys per K/V tile
constexpr int kShRows = 128;          // query rows (token, head) per tile = TMEM lanes
constexpr int kShTiles = 2;           // query tiles per work item
constexpr int kShMaxCtas = 160;       // CTAs of the attention kernel at most (one per SM: GB300 has 152)
// Cost units per CTA below which fewer CTAs share the work (one request of 8 samples over 4096 keys, last
// token: 21.9 us with 4, 22.3 with 6, 27.3 with 8).
constexpr int kShSplitMin = 4;
// Where no entry has this many key tiles none is cut: the join's launch takes longer than a shorter range
// cut in two saves (one request of 15 samples over 400 keys, 5 tiles: 24.2 us cut, 20.8 not; 2 samples over
// 1034 keys, 9 tiles: 27.5 cut, 33.1 not).
constexpr int kShSplitTiles = 8;

// One work entry: kShTiles tiles of query rows of one request against its keys; an entry for one
// kv head is an item.  Rows are (row, head of the kv head) pairs, row-major; "row" is a token
// (prefill) or a sample (last token).
struct __align__(16) ShEntry {
    int32_t prow0, plen;      // prefix rows of the request
    int32_t row0, nrows;      // first row and number of rows
    int32_t ka0, kb0;         // own (packed) keys that tile 0's rows can see: [ka0, kb0)
    int32_t ka1, kb1;         // the same for tile 1 (empty when the entry has one tile)
    int32_t s0;               // prefill: sample of the first row; last token: 0 or 1 (kv head of a pair) or kShPair
    int32_t tiles;            // key tiles: the prefix's, then those of the own keys
    int64_t pos;              // cost units of all entries before this one
};
static_assert(sizeof(ShEntry) == 48, "three 16-byte loads");

// The first tile of a CTA's share of the work, in the order (kv head or pair of them, entry, key tile).
struct __align__(16) ShStart {
    int32_t kh, entry, tile, pad;
};

// An item whose key tiles are shared by `pieces` CTAs from `cta` on, for the join; pair: of the kv heads
// kh and kh + 1.
struct __align__(16) ShSplit {
    int32_t row0, nrows, kh, cta, pieces, pair, pad[2];
};

// Header words at the start of the workspace; from kShHdrKey on the problem the plan is for, which
// every run that reads the plan compares with its own.
// kShHdrStatus: 0, or why no run may use the plan (bits of BG_DEVSTAT: bad offsets, a wait that ran out).
// kShHdrItems: items that are dealt out whole, or 0 where the CTAs have shares of the line.
// kShHdrEmpty: 1 if an entry has no keys at all.
enum {
    kShHdrStatus = 0, kShHdrCtas = 1, kShHdrSplits = 2, kShHdrEntries = 3, kShHdrKey = 4, kShHdrItems = 16, kShHdrEmpty = 17
};
struct __align__(16) ShKey {
    int32_t w[12];
};

// Workspace layout (byte offsets); every part is 256-byte aligned.
struct ShLayout {
    size_t entries, sorted, starts, splits, part_l, part_o, tree, total;
    int64_t max_entries;
    int64_t items, units;     // items and cost units of the work at most, by single heads
    int64_t slots;            // partial results (two per CTA), or 0: no item can be split
};

constexpr int kShPair = 2;

struct ShProblem {
    const int32_t *cu_seqlens, *cu_prefix, *cu_group;
    int32_t num_seqs, total_tokens, max_seqlen;
    int32_t num_groups, total_prefix, max_prefix_len;
    int32_t Hq, Hkv, head_dim;
    int32_t last;             // 1: one query row per sample, 0: one per token
    int32_t tree;             // 1: a request's nodes are its one sample (cu_group NULL), and each sees its ancestors
    const int32_t *parent;
};

// Words of a node's mask over the nodes of its request: whole key tiles.
__host__ __device__ inline int32_t tree_words(int32_t max_nodes) { return (max_nodes + kShKeys - 1) / kShKeys * (kShKeys / 32); }

// kv heads that the work line takes at once: 2 pairs them.  In the last-token call a request has a row per
// sample, often not enough for two query tiles; then two kv heads fill both, and the softmax of one runs
// beside the products of the other.  Measured, 16 / 8 heads of 128: 32 requests of 15 samples over
// 200-500 keys 53.0 us by single heads, 48.1 paired; 4 of 32 samples over 32768 keys 121 and 115.  Not
// where the key ranges would be cut into more than about ten parts, whose joining takes what is won: one
// request of 8 samples over 4096 keys 23.4 single, 26.4 paired; four of them 29.0 and 29.8.
int shared_heads(const ShProblem &pb);
// Query tiles of an entry: one in a prefill that would leave half of the SMs without an item of two, unless
// its key ranges are long enough to be cut.  One request, 16 / 8 heads of 128: 15 samples over 400 keys 20.3 us
// with two, 16.7 with one; 12 samples over 8000 keys 52.1 and 62.3.
int shared_tiles(const ShProblem &pb);
ShLayout shared_layout(const ShProblem &pb);
ShKey shared_key(const ShProblem &pb, int grid);

struct ShParams {
    int32_t Hq, Hkv, g, bt;   // bt = rows of g heads per query tile
    int32_t heads;            // shared_heads
    int32_t last, num_seqs;
    float scale_log2;         // plain scores: softmax scale * log2(e)
    float cap_in, cap_log2;   // capped scores: 2 log2(e) scale / cap, and cap * log2(e)
    __nv_bfloat16 *out;
    float *lse;
    int32_t *dev_status;
    ShKey key;
    const int32_t *cu_seqlens;
    const uint32_t *tree;     // masks [node][tree_words], or NULL
    int32_t tree_words;
    int32_t *hdr;
    const ShEntry *entries;
    const ShEntry *sorted;    // the same in falling order of tiles, where more items than CTAs are dealt out
    const ShStart *starts;    // [CTAs + 1]
    const ShSplit *splits;
    float *part_o;            // [slot][256 rows][D] partial outputs
    float2 *part_l;           // [slot][256 rows] log2 sums, and what the weights' rounding adds to a sum of 1
};

// How partial results are joined: there are none, an item has a few, or many.
enum : int { kShJoinNone = 0, kShJoinFew = 1, kShJoinMany = 2 };

cudaError_t launch_shared_plan(const ShProblem &pb, const ShLayout &lay, void *workspace, int grid,
                               int32_t *dev_status, cudaStream_t stream);
cudaError_t launch_shared_attn(int head_dim, bool capped, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                               const CUtensorMap &tm_v, const CUtensorMap &tm_pk, const CUtensorMap &tm_pv,
                               const ShParams &p, int grid, int join, cudaStream_t stream);

}  // namespace bg
