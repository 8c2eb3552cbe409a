// shared_attn.cu -- attention of the samples of a request over the request's one prefix.
//
// "SLM 生成式高并发推理引擎：延迟约束下的有效吞吐优化", abstract and section 1.2: a Prefill-Only
// request carries several samples, and what they have in common is kept once per request.  For a
// sample s of request r, a query row i of s and a query head h (kv head kvh = h / g):
//     keys  = [prefix rows of r ; own rows of s that i sees]
//     x_j   = scale * q_i,h . k_j,kvh,  or  cap * tanh(scale * q . k / cap)
//     out   = sum_j softmax_j(x) v_j,kvh
// Prefill has a query row per token, which sees its sample's rows up to itself; the last-token
// form has one per sample, which sees the whole sample.
// A tree of drafted tokens (TREE) is a prefill with one sample per request, of whose rows a query sees its ancestors
// and itself: each has a mask over them, one word per 32, which the plan makes from the parents.
//
// A query tile is dense over the rows of the REQUEST, not of one sample: its 128 rows are
// (row, head of the kv head) pairs of consecutive packed rows, whatever samples they belong to.
// Against the prefix nothing but the prefix's end is masked, so short samples and few heads still
// fill the tensor core's 128 rows; against the own keys every row keeps the interval [lo, hi) of
// its sample (block-diagonal), and key tiles that no row of a query tile sees are skipped.
// kShTiles query tiles share every K/V tile that is loaded; in the last-token form, where few rows often
// fill only one, the two may hold the same rows for two kv heads, each with K/V tiles of its own.
//
// Three launches on the caller's stream:
//   1. shared_plan_kernel (one CTA) checks the offsets on the device, writes the list of entries
//      and cuts the whole work, as one line of (kv head or pair, entry, key tile), into equal shares,
//      one per CTA of the next kernel.  A cut through a long key range leaves two partial results.
//      Where all key ranges are short it deals whole items out instead.
//   2. shared_attn_kernel: one CTA per SM, 12 warps:
//        warp 0      walks the CTA's share, tells the other roles each item (through a ring in
//                    shared memory), and loads K and V tiles of 128 keys by TMA (one ring for both)
//        warp 2      TMA producer of Q
//        warp 1      tcgen05.mma issuer (one thread); warp 3 has no part
//        warps 4-11  softmax and output, one warpgroup per query tile, one thread per row
//      The scores of a query tile (128 fp32 TMEM columns) are overwritten by its weights P (64
//      columns), so a tile alternates between its softmax and its two products; the two tiles of
//      a CTA take turns on the tensor core.
//   3. shared_join_kernel joins the partial results (only where the sizes allow a cut).
// Every wait is bounded (sh_wait); on a time-out every role leaves, copies and MMAs in
// flight are drained, TMEM is freed, BG_DEVSTAT_TIMEOUT is reported and the plan is void, so that
// the join writes nothing.
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>

#include "bg_internal.h"
#include "bg_ptx.cuh"
#include "shared_attn.h"

namespace bg {

namespace {

// ------------------------------------------------------------------------------------ plan
constexpr int kPlanThreads = 512;
constexpr int kPlanPos = 2048;                       // entries whose positions are
constexpr int kPlanSeqs = 4096, kPlanGroups = 512;   // offsets up to these counts are held in shared memory

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Exclusive sum over the block's threads; *total gets the sum.  All threads call it.
__device__ int block_exclusive(int v, int *s_warp, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    __syncthreads();                 // s_warp may still be read from the last call
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    // every warp sums the warps before it
    const int w = lane < kPlanThreads / 32 ? s_warp[lane] : 0;
    *total = __reduce_add_sync(0xffffffffu, w);
    return incl - v + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
}

// The sample among [s, end) that holds packed row `row` (cu[s] <= row < cu[end]).
__device__ int sample_of(const int32_t *cu, int s, int end, int row)
{
    while (end - s > 1) {
        const int mid = (s + end) >> 1;
        if (cu[mid] <= row) s = mid; else end = mid;
    }
    return s;
}

// Cost of an entry in units of one key tile: its tiles, and two for loading Q and storing the rows (one:
// 16 samples over 8000 keys 400 us instead of 397, one request of 8 over 4096 keys 23.3 instead of 21.8; 24
// requests of 31 capped samples, last token, 37.5 instead of 39.4).
constexpr int kItemUnits = 2;
__device__ __forceinline__ int entry_units(const ShEntry &E) { return E.tiles > 0 ? E.tiles + kItemUnits : 0; }

// Masks of a tree's nodes: of each one its own bit and its ancestors'.  One CTA per request, a thread per node, which
// follows the parents through shared memory; they have falling numbers, so that the words come one after the other.
__device__ void tree_masks(const ShProblem &pb, int request, int32_t *s_parent, uint32_t *masks, int32_t *dev_status)
{
    const int a = pb.cu_seqlens[request], b = pb.cu_seqlens[request + 1], n = b - a;
    if (a < 0 || b < a || b > pb.total_tokens || n > pb.max_seqlen) return;      // the plan reports it
    bool bad = false;
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        int up = pb.parent[a + i];
        if (up < -1 || up >= i) {
            bad = true;
            up = -1;
        }
        s_parent[i] = up;
    }
    if (bad && dev_status) atomicOr(dev_status, BG_DEVSTAT_PARENT);
    __syncthreads();
    const int words = tree_words(pb.max_seqlen);
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
        uint32_t *out = masks + static_cast<int64_t>(a + i) * words;
        int at = i;
        for (int w = words - 1; w >= 0; --w) {
            uint32_t bits = 0;
            while (at >= 32 * w) {
                bits |= 1u << (at - 32 * w);
                at = s_parent[at];
            }
            out[w] = bits;
        }
    }
}

// Latency alone bounds it: a few loads of the offsets in a row and about ten barriers of one CTA, 3.3 us for
// one request, 4.5 where ranges are cut, with 512 threads (4.9 with 1024; 256 are 0.1 faster for a few
// requests and 0.7 slower for 500 entries); the sort of 500 entries adds 2.5.
// The offsets are held in shared memory because the searches read them many times.  For trees CTA 1 + r makes the masks of
// request r beside it (in a launch of their own: 1 to 2 us more).  Up to 64 nodes they take no longer than the plan (4.2 to
// 4.8 us together); then the deepest node's way through its parents and the words written count: chains of 256, 512 and
// 1024 nodes 8, 17 and 51 us, drafts whose nodes hang below recent ones 4.4, 5.4 and 18.
__global__ void __launch_bounds__(kPlanThreads)
    shared_plan_kernel(const ShProblem pb, const ShKey key, int bt, int32_t *hdr, ShEntry *entries, ShEntry *sorted,
                       ShStart *__restrict__ starts, ShSplit *__restrict__ splits, int grid, int can_split, int tiles_per, int heads,
                       uint32_t *masks, int32_t *dev_status)
{
    __shared__ int s_err, s_nsplit, s_empty;
    __shared__ int s_warp[32];
    __shared__ int s_base[kPlanThreads];
    __shared__ ShStart s_start[kShMaxCtas + 1];
    __shared__ int32_t s_cu[kPlanSeqs + 1], s_cup[kPlanGroups + 1], s_cug[kPlanGroups + 1];
    __shared__ int64_t s_pos[kPlanPos];
    __shared__ int s_class[kPlanThreads / 32][kShSplitTiles];
    const int tid = threadIdx.x;
    grid_dep_launch();
    if (tid == 0) {
        s_err = 0;
        s_nsplit = 0;
        s_empty = 0;
    }
    grid_dep_wait();
    __syncthreads();
    if (blockIdx.x > 0) {
        static_assert(kPlanSeqs >= BG_MAX_TREE, "a request's parents");
        tree_masks(pb, static_cast<int>(blockIdx.x) - 1, s_cu, masks, dev_status);
        return;
    }
    if (tid < 12) hdr[kShHdrKey + tid] = key.w[tid];
    const int32_t *cu = pb.cu_seqlens, *cup = pb.cu_prefix, *cug = pb.cu_group;
    auto group = [&](int r) { return cug ? cug[r] : r; };      // a tree: request r is sample r
    if (pb.num_seqs <= kPlanSeqs && pb.num_groups <= kPlanGroups) {
        for (int i = tid; i <= pb.num_seqs; i += kPlanThreads) s_cu[i] = cu[i];
        for (int i = tid; i <= pb.num_groups; i += kPlanThreads) {
            s_cup[i] = cup[i];
            s_cug[i] = group(i);
        }
        cu = s_cu;
        cup = s_cup;
        cug = s_cug;
        __syncthreads();
    }

    // ---- the offsets, before anything is read through them
    int err = 0;
    for (int i = tid; i < pb.num_groups; i += kPlanThreads) {
        const int a = group(i), b = group(i + 1);
        if (a < 0 || b < a || b > pb.num_seqs || (i == 0 && a != 0) || (i == pb.num_groups - 1 && b != pb.num_seqs))
            err |= BG_DEVSTAT_GROUP;
        const int c = cup[i], d = cup[i + 1];
        if (c < 0 || d < c || d > pb.total_prefix || d - c > pb.max_prefix_len || (i == 0 && c != 0) ||
            (i == pb.num_groups - 1 && d != pb.total_prefix))
            err |= BG_DEVSTAT_CU_PROMPT;
    }
    for (int i = tid; i < pb.num_seqs; i += kPlanThreads) {
        const int a = cu[i], b = cu[i + 1];
        if (a < 0 || b < a || b > pb.total_tokens || (i == 0 && a != 0) ||
            (i == pb.num_seqs - 1 && b != pb.total_tokens))
            err |= BG_DEVSTAT_CU_SEQLENS;
        else if (b - a > pb.max_seqlen)
            err |= BG_DEVSTAT_SEQ_TOO_LONG;
    }
    if (err) atomicOr(&s_err, err);
    __syncthreads();
    if (s_err) {
        if (tid == 0) {
            hdr[kShHdrStatus] = s_err;
            hdr[kShHdrCtas] = 0;
            hdr[kShHdrSplits] = 0;
            hdr[kShHdrItems] = 0;
            if (dev_status) atomicOr(dev_status, s_err);
        }
        return;
    }

    // ---- the entries, in request order
    const int per = tiles_per * bt;        // rows of an entry
    int n_entries = 0;
    int64_t units = 0;
    for (int r0 = 0; r0 < pb.num_groups; r0 += kPlanThreads) {
        const int r = r0 + tid;
        int items = 0;
        if (r < pb.num_groups) {
            const int a = group(r), b = group(r + 1);
            const int rows = pb.last ? b - a : cu[b] - cu[a];
            items = static_cast<int>(ceil_div(rows, per));
            // paired heads: an entry of one query tile serves both heads, the others come once for each
            if (heads == 2 && items > 0) items = 2 * items - (rows - (items - 1) * per <= bt ? 1 : 0);
        }
        int total;
        s_base[tid] = block_exclusive(items, s_warp, &total);
        __syncthreads();
        for (int e0 = 0; e0 < total; e0 += kPlanThreads) {
            const int e = e0 + tid;
            ShEntry E = {};
            if (e < total) {
                int t = 0, end = kPlanThreads;     // the request whose entries include e
                while (end - t > 1) {
                    const int mid = (t + end) >> 1;
                    if (s_base[mid] <= e) t = mid; else end = mid;
                }
                const int grp = r0 + t, first = ((e - s_base[t]) >> (heads - 1)) * per;
                const int sa = group(grp), sb = group(grp + 1);
                E.prow0 = cup[grp];
                E.plen = cup[grp + 1] - E.prow0;
                const int base = pb.last ? sa : cu[sa];
                const int end_row = pb.last ? sb : cu[sb];
                E.row0 = base + first;
                E.nrows = min(per, end_row - E.row0);
                const int n0 = min(bt, E.nrows);
                if (pb.last) {
                    E.s0 = 0;
                    E.ka0 = cu[E.row0];
                    E.kb0 = cu[E.row0 + n0];
                    E.ka1 = E.kb0;
                    E.kb1 = cu[E.row0 + E.nrows];
                } else {
                    E.s0 = sample_of(cu, sa, sb, E.row0);
                    E.ka0 = cu[E.s0];
                    E.kb0 = E.row0 + n0;
                    E.ka1 = E.nrows > bt ? cu[sample_of(cu, E.s0, sb, E.row0 + bt)] : E.kb0;
                    E.kb1 = E.row0 + E.nrows;
                }
                E.tiles = static_cast<int>(ceil_div(E.plen, kShKeys) + ceil_div(E.kb1 - E.ka0, kShKeys));
                if (heads == 2) {
                    if (E.nrows <= bt) {
                        E.s0 = kShPair;
                        E.ka1 = E.ka0;
                    } else {
                        E.s0 = (e - s_base[t]) & 1;
                    }
                }
                if (E.tiles == 0) s_empty = 1;
            }
            int sum;
            const int excl = block_exclusive(entry_units(E), s_warp, &sum);
            if (e < total) {
                E.pos = units + excl;
                entries[n_entries + e] = E;
                if (n_entries + e < kPlanPos) s_pos[n_entries + e] = E.pos;
            }
            units += sum;
        }
        n_entries += total;
        __syncthreads();
    }
    // the rows of an entry without keys, which no CTA visits: every run of the plan reports them
    if (tid == 0) {
        hdr[kShHdrEmpty] = s_empty;
        if (s_empty && dev_status) atomicOr(dev_status, BG_DEVSTAT_EMPTY_ROW);
    }

    // ---- equal shares of the line; fewer CTAs where a share would be below kShSplitMin (half of it for pairs,
    // whose tiles count twice)
    auto pos_of = [&](int e) { return n_entries <= kPlanPos ? s_pos[e] : entries[e].pos; };
    const int lines = pb.Hkv >> (heads - 1);

    // ---- nothing is cut: whole items, dealt out to the CTAs in falling order of their tiles, one round from
    // the first CTA to the last, the next one back.  (Shares of the line that end at items' ends leave the
    // largest 22% above the mean with seven items to a CTA: 112 samples of 1-300 tokens over 1-500 keys,
    // capped, 102 us instead of 96; 32 requests of 15 samples over 200-500 keys 154.6 instead of 142.5.)
    if (!can_split) {
        const int n_items = n_entries * lines;
        const int ctas = min(grid, n_items);
        if (n_items > ctas) {
            // a counting sort, in order within a number of tiles; class c: kShSplitTiles - 1 - c tiles
            const int lane = tid & 31, warp = tid >> 5;
            int base = 0;                          // of lane's class (lane < kShSplitTiles)
            for (int pass = 0; pass < 2; ++pass) {
                int count = 0;                     // of lane's class, in the chunks so far
                for (int e0 = 0; e0 < n_entries; e0 += kPlanThreads) {
                    const int e = e0 + tid;
                    ShEntry E = {};
                    if (e < n_entries) E = entries[e];
                    const int mine = e < n_entries ? kShSplitTiles - 1 - E.tiles : -1;
                    int before = 0;                // entries of this class in lower lanes
#pragma unroll
                    for (int c = 0; c < kShSplitTiles; ++c) {
                        const unsigned m = __ballot_sync(0xffffffffu, mine == c);
                        if (mine == c) before = __popc(m & ((1u << lane) - 1u));
                        if (lane == c) s_class[warp][c] = __popc(m);
                    }
                    __syncthreads();
                    int lower = 0, all = 0;        // of lane's class, in lower warps and in all
                    if (lane < kShSplitTiles)
                        for (int w = 0; w < kPlanThreads / 32; ++w) {
                            const int k = s_class[w][lane];
                            lower += w < warp ? k : 0;
                            all += k;
                        }
                    const int at = __shfl_sync(0xffffffffu, base + count + lower, max(mine, 0)) + before;
                    if (pass == 1 && mine >= 0) sorted[at] = E;
                    count += all;
                    __syncthreads();
                }
                if (pass == 0) {                   // the classes' first places
                    int incl = count;
                    for (int o = 1; o < kShSplitTiles; o <<= 1) {
                        const int u = __shfl_up_sync(0xffffffffu, incl, o);
                        if (lane >= o) incl += u;
                    }
                    base = incl - count;
                }
            }
        }
        if (tid == 0) {
            hdr[kShHdrStatus] = 0;
            hdr[kShHdrCtas] = ctas;
            hdr[kShHdrSplits] = 0;
            hdr[kShHdrEntries] = n_entries;
            hdr[kShHdrItems] = n_items;
        }
        return;
    }
    const int64_t work = units * lines;
    const int split_min = kShSplitMin >> (heads - 1);
    const int ctas = static_cast<int>(min(static_cast<int64_t>(grid), ceil_div(work, split_min)));
    for (int c = tid; c <= ctas; c += kPlanThreads) {
        ShStart S = {lines, 0, 0, 0};              // the end of the line
        if (c < ctas) {
            const int64_t at = work * c / ctas;
            S.kh = static_cast<int>(at / units);
            const int64_t u = at - S.kh * units;
            int lo = 0, end = n_entries;           // the last entry that begins at or before u
            while (end - lo > 1) {
                const int mid = (lo + end) >> 1;
                if (pos_of(mid) <= u) lo = mid; else end = mid;
            }
            S.entry = lo;
            const int n = entries[lo].tiles;
            const int into = static_cast<int>(u - pos_of(lo));
            // A cut near an end of the item moves to that end, and so does every cut through an item that is
            // short next to a share: its partial results cost more than the lesser balance (32 requests of
            // 15 samples over 200-500 keys, 10 items to a share, before they were dealt out: 159.1 us when cut,
            // 156.4 when not; with a limit of a sixth of a share 7 samples over 1-500 keys lost 2%).
            const int64_t share = work / ctas;
            const int least = n * 10 <= share ? n : max(split_min / 2, static_cast<int>(min(share / 32, static_cast<int64_t>(n))));
            S.tile = into;
            if (into < least || n - into < least) {
                S.tile = 0;
                if (2 * into > n) ++S.entry;
            }
        }
        if (S.kh < lines && S.entry == n_entries) {
            ++S.kh;
            S.entry = 0;
        }
        s_start[c] = S;
        starts[c] = S;
    }
    __syncthreads();
    // ---- the items that a cut goes through: the first CTA of each one writes it down
    for (int c = tid; c < ctas; c += kPlanThreads) {
        const ShStart A = s_start[c], B = s_start[c + 1];
        if (B.tile == 0 || (A.kh == B.kh && A.entry == B.entry && A.tile > 0)) continue;
        int pieces = 2;
        while (c + pieces < ctas && s_start[c + pieces].tile > 0 && s_start[c + pieces].kh == B.kh &&
               s_start[c + pieces].entry == B.entry)
            ++pieces;
        const ShEntry &E = entries[B.entry];
        splits[atomicAdd(&s_nsplit, 1)] =
            ShSplit{E.row0, E.nrows, B.kh * heads + (heads == 2 ? E.s0 & 1 : 0), c, pieces,
                    heads == 2 ? E.s0 & kShPair : 0, {}};
    }
    __syncthreads();
    if (tid == 0) {
        hdr[kShHdrStatus] = 0;
        hdr[kShHdrCtas] = ctas;
        hdr[kShHdrSplits] = s_nsplit;
        hdr[kShHdrEntries] = n_entries;
        hdr[kShHdrItems] = 0;
    }
}

// Whether the workspace holds an accepted plan for this problem.
__device__ bool plan_ready(const ShParams &p, bool *other)
{
    const int4 *k = reinterpret_cast<const int4 *>(p.hdr + kShHdrKey);
    bool same = true;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int4 a = k[i];
        same = same && a.x == p.key.w[4 * i] && a.y == p.key.w[4 * i + 1] && a.z == p.key.w[4 * i + 2] &&
               a.w == p.key.w[4 * i + 3];
    }
    *other = !same;
    return same && p.hdr[kShHdrStatus] == 0;
}

// ------------------------------------------------------------------------------------ attention
constexpr int kShKeysLog = 7;                  // kShKeys as a shift (counts are not negative)
static_assert(1 << kShKeysLog == kShKeys, "a power of two");
constexpr int kShRing = 4;                     // items in the ring that warp 0 fills
constexpr int kShReaders = 1 + 1 + 8;          // Q producer, MMA issuer, softmax warps

// The part of an item (an entry for one kv head) that this CTA computes, as the roles read it.
template <bool LAST>
struct __align__(16) ShItem {
    int32_t prow0, plen, row0, nrows;
    int32_t ka0, kb0, ka1, kb1;
    int32_t s0, tb, te;       // key tiles [tb, te)
    int32_t npt;              // prefix tiles
    int32_t kh;
    int32_t slot;             // partial result this part goes to, or -1
    int32_t act[kShTiles];    // key tiles with keys for each query tile
    int32_t more;             // 0: no further item
    int32_t pair, pad[2];     // 1: query tile 1 holds tile 0's rows for the next kv head

    __device__ bool paired() const { return LAST && pair != 0; }
    __device__ int rows(int h, int bt) const
    {
        return h == 0 || paired() ? min(nrows, bt) : max(nrows - bt, 0);
    }
    __device__ int first_row(int h, int bt) const { return paired() ? row0 : row0 + h * bt; }
    __device__ int head(int h) const { return paired() ? kh + h : kh; }
    __device__ int ka(int h) const { return h == 0 ? ka0 : ka1; }
    __device__ int kb(int h) const { return h == 0 ? kb0 : kb1; }
    // first packed key row of own tile j (j >= npt)
    __device__ int own_base(int j) const { return ka0 + (j - npt) * kShKeys; }
    // keys of tile j that any row of the item sees (1..128)
    __device__ int keys(int j) const { return min(kShKeys, j < npt ? plen - j * kShKeys : kb1 - own_base(j)); }
    // keys of tile j up to the last one that a row of query tile h sees (<= 0: none); act[h] > 0
    __device__ int keys_of(int h, int j) const
    {
        if (j < npt) return min(kShKeys, plen - j * kShKeys);
        const int base = own_base(j);
        return kb(h) <= ka(h) || base + kShKeys <= ka(h) ? 0 : min(kShKeys, kb(h) - base);
    }
    // number of key tiles of this part with keys for query tile h
    __device__ int active(int h, int bt) const
    {
        if (rows(h, bt) == 0) return 0;
        const int pre = max(min(te, npt) - tb, 0);
        if (kb(h) <= ka(h)) return pre;
        const int lo = npt + ((ka(h) - ka0) >> kShKeysLog);
        const int hi = npt + ((kb(h) - ka0 + kShKeys - 1) >> kShKeysLog);
        return pre + max(min(te, hi) - max(tb, lo), 0);
    }
};
static_assert(sizeof(ShItem<false>) == 80, "five 16-byte stores");

template <int D>
struct ShCfg {
    static constexpr int kBox = 128 * 128;                   // 128 rows x one 128-byte column block
    static constexpr int kNB = D / 64;
    static constexpr int kTileBytes = kNB * kBox;            // one Q, K or V tile
    static constexpr int kStages = D == 128 ? 5 : 8;         // K and V tiles in flight
    static constexpr int kOffQ = 0;
    static constexpr int kOffKV = kShTiles * kTileBytes;
    static constexpr int kOffBar = kOffKV + kStages * kTileBytes;
    // q_full[2] q_empty[2] s_full[2] p_full[2][2] o_full[2] mma_final kv_full[kStages] kv_empty[kStages]
    // item_full[kShRing] item_empty[kShRing]
    static constexpr int kNumBars = 13 + 2 * kStages + 2 * kShRing;
    static constexpr int kOffItems = (kOffBar + kNumBars * 8 + 15) / 16 * 16;
    static constexpr int kOffMisc = kOffItems + kShRing * static_cast<int>(sizeof(ShItem<false>));
    static constexpr int kSmemBytes = kOffMisc + 16 + 1024;  // + slack for 1024-byte alignment
    static constexpr int kThreads = 384;
    // Register split, as in the attention kernel of the other modes: compiled for kRegsLaunch,
    // warps 0-3 run with kRegsLight, the 8 softmax warps with kRegsSoftmax.
    static constexpr int kRegsLaunch = 168, kRegsLight = 64, kRegsSoftmax = 216;
    static constexpr int kSplitRegs = 4 * 32 * kRegsLight + 8 * 32 * kRegsSoftmax;
    static_assert(kThreads * kRegsLaunch <= 65536 && kSplitRegs <= kThreads * kRegsLaunch, "register split");
    static constexpr int kColS = 0, kColO = kShTiles * kShKeys;   // S (and P) of tile h at 128 h, O behind them
    static constexpr int kTmemCols = 512;
    static_assert(kColO + kShTiles * D <= kTmemCols, "TMEM overflow");
    static_assert(kSmemBytes <= 232448, "shared memory overflow");
};

// mbar_wait, and its form for a whole warp, in less code: the instruction cache serves the loops of all
// roles, whose waits' slow paths lie between.  The clock is first read when 64 polls have failed (read
// at each poll it held the wake-ups up: 16 MMA-bound samples over 8000 keys took 484 us instead of 408).
__device__ __forceinline__ uint32_t sh_time()
{
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}
__device__ __forceinline__ bool sh_wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    uint32_t t0 = 0;
#pragma unroll 1
    for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
        if ((it & 63u) != 0) continue;
        const uint32_t now = sh_time();
        if (it == 64) t0 = now;
        if (*abort || now - t0 > static_cast<uint32_t>(kWaitTimeoutNs)) {
            *abort = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool sh_warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    uint32_t t0 = 0;
#pragma unroll 1
    for (uint32_t it = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++it) {
        if ((it & 63u) != 0) continue;
        const uint32_t now = sh_time();
        if (it == 64) t0 = now;
        if (__any_sync(0xffffffffu, *abort || now - t0 > static_cast<uint32_t>(kWaitTimeoutNs))) {
            *abort = 1;
            return false;
        }
    }
    return true;
}

// S = Q K^T over D = 64 * NB, then a commit to `full`: one asm statement per tile, so that
// the descriptors' offsets are immediates and the MMAs go out back to back.  Q and K column blocks
// are 16 KB (1024 descriptor units) apart, 16-element steps 32 bytes (2 units).
template <int NB>
__device__ __forceinline__ void sh_mma_qk(uint32_t d, uint64_t dq, uint64_t dk, uint32_t idesc, uint64_t *full)
{
    if constexpr (NB == 2) {
        asm volatile(
            "{\n\t.reg .pred pf, pt;\n\t.reg .b64 a1, a2, a3, a4, a5, a6, a7, b1, b2, b3, b4, b5, b6, b7;\n\t"
            "setp.ne.b32 pf, 0, 0;\n\tsetp.eq.b32 pt, 0, 0;\n\t"
            "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
            "add.s64 a4, %1, 1024;\n\tadd.s64 a5, %1, 1026;\n\tadd.s64 a6, %1, 1028;\n\tadd.s64 a7, %1, 1030;\n\t"
            "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
            "add.s64 b4, %2, 1024;\n\tadd.s64 b5, %2, 1026;\n\tadd.s64 b6, %2, 1028;\n\tadd.s64 b7, %2, 1030;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, pf;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, pt;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, pt;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, pt;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a4, b4, %3, pt;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a5, b5, %3, pt;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a6, b6, %3, pt;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a7, b7, %3, pt;\n\t"
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}" ::"r"(d),
            "l"(dq), "l"(dk), "r"(idesc), "r"(smem_u32(full))
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred pf, pt;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
            "setp.ne.b32 pf, 0, 0;\n\tsetp.eq.b32 pt, 0, 0;\n\t"
            "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
            "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, pf;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, pt;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, pt;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, pt;\n\t"
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}" ::"r"(d),
            "l"(dq), "l"(dk), "r"(idesc), "r"(smem_u32(full))
            : "memory");
    }
}

// O (+)= P V over 64 keys: P in TMEM (8 columns per 16 keys), V's 16-key steps 2 KB (128 units) apart.
__device__ __forceinline__ void sh_mma_pv4(uint32_t d, uint32_t a, uint64_t dv, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p0, pt;\n\t.reg .b64 b1, b2, b3;\n\t.reg .b32 t1, t2, t3;\n\t"
        "setp.ne.b32 p0, %4, 0;\n\tsetp.eq.b32 pt, 0, 0;\n\t"
        "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"
        "add.u32 t1, %1, 8;\n\tadd.u32 t2, %1, 16;\n\tadd.u32 t3, %1, 24;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t1], b1, %3, pt;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t2], b2, %3, pt;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [t3], b3, %3, pt;\n\t}" ::"r"(d),
        "r"(a), "l"(dv), "r"(idesc), "r"(acc)
        : "memory");
}

// 32 bytes to global memory (one whole sector per lane).
__device__ __forceinline__ void st_global_32b(void *dst, const uint32_t *w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// 32 bytes of an output row: one whole sector per lane where the rows are 32-byte aligned.
__device__ __forceinline__ void st_out_32b(void *dst, const uint32_t *w, bool wide)
{
    if (wide) {
        st_global_32b(dst, w);
    } else {
        static_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

__device__ __forceinline__ float min_nan(float a, float b)
{
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// Four scores s to cap_log2 * tanh(y) = cap_log2 - 2 cap_log2 / (1 + e^(2y)), y = s * scale / cap
// (cap_in = 2 log2(e) scale / cap).  One reciprocal serves all four, since the special-function unit
// is what bounds capped scores (16 reciprocals and 32 exponentials per cycle and SM): 1 / a =
// b * cd * (1 / abcd).  e^(2y) is held at 2^30, where tanh is 1 to the last bit, so that abcd stays
// finite; NaN stays, and reaches all four.  Next to 0 the difference leaves an error of about 2^-23
// of the cap.
__device__ __forceinline__ void capped4(float *s, float cap_in, float cap_log2)
{
    const float2 in2 = make_float2(cap_in, cap_in), one2 = make_float2(1.f, 1.f), cap2 = make_float2(cap_log2, cap_log2);
    const float2 x01 = fmul2(make_float2(s[0], s[1]), in2), x23 = fmul2(make_float2(s[2], s[3]), in2);
    const float2 a01 = fadd2(make_float2(ex2(min_nan(x01.x, 30.f)), ex2(min_nan(x01.y, 30.f))), one2);
    const float2 a23 = fadd2(make_float2(ex2(min_nan(x23.x, 30.f)), ex2(min_nan(x23.y, 30.f))), one2);
    const float ab = a01.x * a01.y, cd = a23.x * a23.y;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ab * cd));
    r *= -2.f * cap_log2;
    const float rcd = r * cd, rab = r * ab;
    const float2 t01 = ffma2(make_float2(rcd, rcd), make_float2(a01.y, a01.x), cap2);
    const float2 t23 = ffma2(make_float2(rab, rab), make_float2(a23.y, a23.x), cap2);
    s[0] = t01.x;
    s[1] = t01.y;
    s[2] = t23.x;
    s[3] = t23.y;
}

// The same for caps of any size, where that error could be large next to the scores: below |y| = 0.3
// the series y - y^3 / 3 + 2 y^5 / 15 - 17 y^7 / 315 + 62 y^9 / 2835 (the next term is below 2^-24 of y).
__device__ __forceinline__ void capped4_any(float *s, float cap_in, float cap_log2)
{
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = s[i] * cap_in * 0.34657359027997264f;      // ln(2) / 2
    capped4(s, cap_in, cap_log2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float u = y[i] * y[i];
        float t = fmaf(u, 62.f / 2835.f, -17.f / 315.f);
        t = fmaf(u, t, 2.f / 15.f);
        t = fmaf(u, t, -1.f / 3.f);
        const float small = cap_log2 * fmaf(y[i] * u, t, y[i]);
        s[i] = fabsf(y[i]) < 0.3f ? small : s[i];
    }
}

// How scores become weights: plain; capped, by the same running maximum; or capped by at most
// kShCapFixed (in base 2), where 2^x of any score and any sum of them is an ordinary fp32 number, so
// that no running maximum is needed and the tile goes from S to P 32 columns at a time (a cap of 30, 112 samples of
// 1-300 tokens over 1-500 keys: 114 us, with the running maximum 169).  2^80 of a weight and 2^17 keys leave
// |v| < 2^30 within fp32; 2^-80 of one, where all scores of a row are near the negative cap, leaves
// |v| >= 2^-46 among its normal numbers.
enum : int { kShPlain = 0, kShCapped = 1, kShCappedFixed = 2 };
constexpr float kShCapFixed = 80.f;
// The log-sum of a part of a key range whose keys all have weight 0 (a second number to say so would be read
// by the join's first loop: 116.2 us instead of 114.2 for 128 last tokens over 30000-32768 keys).
constexpr float kShNoWeight = -3.402823466e38f;

// Measured, 16 / 8 heads of 128, device time with plan and join: 16 samples of 257-700 tokens over 8000
// keys 399 us within a graph, 418 among other calls, 1310 TFLOP/s; 32 requests of 15 samples of 16-96 tokens over 200-500 keys 142.5 us (prefill)
// and 45 us, 3.5 TB/s (last token); 128 last tokens over 30000-32768 keys 115 us, 5.4 TB/s.  14 / 2 heads
// of 64, scores capped at 30: 112 samples of 1-300 tokens over 1-500 keys 100 us, 744 last tokens 38 us.
// What bounds it is the chain of one query tile per key tile: about 2250 cycles of softmax (tensor memory
// to registers, maximum, 128 exponentials of a row, weights back), then 1400 of hand-overs and products.
// Two query tiles overlap their chains; tensor memory (S and O of each) has no room for a third at D = 128.
// 128-key tiles against 64: half the hand-overs.  Items of few tiles add the start and the end of an item,
// where nothing overlaps: about 4 us of 12 for five key tiles.
template <int D, int MODE, bool LAST, bool TREE>
__global__ void __maxnreg__((ShCfg<D>::kRegsLaunch))
    shared_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_pk,
                       const __grid_constant__ CUtensorMap tm_pv, const ShParams p)
{
    using C = ShCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *q_full = bars, *q_empty = bars + 2, *s_full = bars + 4, *p_full = bars + 6, *o_full = bars + 10;
    uint64_t *mma_final = bars + 12;
    uint64_t *kv_full = bars + 13, *kv_empty = kv_full + C::kStages;
    uint64_t *item_full = kv_empty + C::kStages, *item_empty = item_full + kShRing;
    using Item = ShItem<LAST>;
    Item *ring = reinterpret_cast<Item *>(smem + C::kOffItems);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_launch();

    if (threadIdx.x == 0) {
        for (int h = 0; h < kShTiles; ++h) {
            mbar_init(&q_full[h], 1);
            mbar_init(&q_empty[h], 1);
            mbar_init(&s_full[h], 1);
            mbar_init(&p_full[2 * h], 4);      // one arrive per softmax warp: keys 0-63 of the tile
            mbar_init(&p_full[2 * h + 1], 4);  // ... and keys 64-127
            mbar_init(&o_full[h], 1);
        }
        mbar_init(mma_final, 1);
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < kShRing; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], kShReaders);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    // Query tiles fill bt * g <= 128 rows; the rows past them stay zero.
    if (p.bt * p.g < kShRows) {
        uint4 *z4 = reinterpret_cast<uint4 *>(smem + C::kOffQ);
        for (int i = threadIdx.x; i < kShTiles * C::kTileBytes / 16; i += blockDim.x) z4[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_pk);
        tma_prefetch_desc(&tm_pv);
    }
    grid_dep_wait();     // the plan is written
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int cta = static_cast<int>(blockIdx.x);

    if (warp < 4) {
        reg_dealloc<C::kRegsLight>();
        if (warp == 0) {
            // ============================================================ items, K and V
            if (lane == 0) {
                bool other;
                const bool ready = plan_ready(p, &other), mine = ready && cta < p.hdr[kShHdrCtas];
                if (cta == 0 && p.dev_status) {
                    if (other) atomicOr(p.dev_status, BG_DEVSTAT_PLAN);
                    if (ready && p.hdr[kShHdrEmpty] != 0) atomicOr(p.dev_status, BG_DEVSTAT_EMPTY_ROW);
                }
                ShStart A = {}, B = {};
                int n_entries = 0, ctas = 0, lines = 1;
                uint32_t n_items = 0, at = 0;              // dealt out: all items, and the place of this one
                if (mine) {
                    n_entries = p.hdr[kShHdrEntries];
                    ctas = p.hdr[kShHdrCtas];
                    n_items = p.hdr[kShHdrItems];
                    if (n_items == 0) {
                        A = p.starts[cta];
                        B = p.starts[cta + 1];
                    }
                }
                const bool dealt = n_items > 0;
                if (dealt) {
                    lines = LAST ? p.Hkv / p.heads : p.Hkv;
                    at = cta;
                    A = ShStart{cta % lines, cta / lines, 0, 0};
                    B.kh = -1;
                }
                const uint64_t pol = l2_policy_evict_last();
                const int4 *list = reinterpret_cast<const int4 *>(dealt && n_items > ctas ? p.sorted : p.entries);
                int kh = A.kh, entry = A.entry, tb = A.tile;
                auto before_end = [&]() {
                    return dealt ? at < n_items
                                 : kh < B.kh || (kh == B.kh && (entry < B.entry || (entry == B.entry && tb < B.tile)));
                };
                uint32_t back = static_cast<uint32_t>(2 * (ctas - 1 - cta) + 1);      // to the next place, and then
                                                                                     // 2 * cta + 1, in turn
                int4 e0 = {}, e1 = {}, e2 = {};
                auto fetch = [&]() {
                    const int4 *q = list + 3 * static_cast<int64_t>(entry);
                    e0 = q[0];
                    e1 = q[1];
                    e2 = q[2];
                };
                if (before_end()) fetch();
                uint32_t st = 0, ph = 1;         // stage, and the parity of its release (1: free at first)
                uint32_t n_told = 0;
                uint32_t used = 0;               // stages that hold or await a copy, counted up to kStages
                bool ok = true;
                for (;;) {
                    const bool more = before_end();
                    const uint32_t slot = n_told % kShRing;
                    if (!sh_wait(&item_empty[slot], ((n_told / kShRing) & 1) ^ 1, abort_flag)) break;
                    Item I;
                    I.prow0 = e0.x; I.plen = e0.y; I.row0 = e0.z; I.nrows = e0.w;
                    I.ka0 = e1.x; I.kb0 = e1.y; I.ka1 = e1.z; I.kb1 = e1.w;
                    I.s0 = e2.x;
                    const int tiles = e2.y;
                    const int code = LAST ? e2.x : 0;
                    I.kh = LAST ? kh * p.heads + (code & 1) : kh;
                    I.pair = code & kShPair;
                    I.npt = (I.plen + kShKeys - 1) >> kShKeysLog;
                    I.tb = tb;
                    I.te = kh == B.kh && entry == B.entry ? B.tile : tiles;
                    I.slot = tb > 0 ? 2 * cta : I.te < tiles ? 2 * cta + 1 : -1;
                    if (more && tiles > 0) {
                        I.act[0] = I.active(0, p.bt);
                        I.act[1] = I.active(1, p.bt);
                    }
                    I.more = more ? 1 : 0;
                    if (!more || tiles > 0) {
                        int4 *dst = reinterpret_cast<int4 *>(&ring[slot]);
                        dst[0] = make_int4(I.prow0, I.plen, I.row0, I.nrows);
                        dst[1] = make_int4(I.ka0, I.kb0, I.ka1, I.kb1);
                        dst[2] = make_int4(I.s0, I.tb, I.te, I.npt);
                        dst[3] = make_int4(I.kh, I.slot, I.act[0], I.act[1]);
                        dst[4] = make_int4(I.more, I.pair, 0, 0);
                        mbar_arrive(&item_full[slot]);
                        ++n_told;
                    }
                    if (!more) break;
                    // the next item, fetched while this one's tiles are loaded
                    tb = 0;
                    if (dealt) {
                        at += back;
                        back = 2 * ctas - back;
                        entry = at / lines;
                        kh = at - entry * lines;
                    } else if (++entry == n_entries) {
                        entry = 0;
                        ++kh;
                    }
                    if (before_end()) fetch();
                    if (tiles == 0) continue;
                    // In the order in which the products take them: K of a tile, then V; paired, K of the first
                    // tile for both heads, then V of a tile and K of the next for one head and for the other.
                    auto load = [&](int j, int kv, int kh_kv) {
                        const bool pre = j < I.npt;
                        const int row = pre ? I.prow0 + j * kShKeys : I.own_base(j);
                        ok = sh_wait(&kv_empty[st], ph, abort_flag);
                        if (!ok) return;
                        uint8_t *dst = smem + C::kOffKV + st * C::kTileBytes;
                        const CUtensorMap *tm = kv == 0 ? (pre ? &tm_pk : &tm_k) : (pre ? &tm_pv : &tm_v);
                        mbar_arrive_expect_tx(&kv_full[st], C::kTileBytes);
#pragma unroll
                        for (int b = 0; b < C::kNB; ++b)
                            tma_load_3d(dst + b * C::kBox, tm, &kv_full[st], b * 64, kh_kv, row, pol);
                        if (used < C::kStages) ++used;
                        if (++st == C::kStages) {
                            st = 0;
                            ph ^= 1u;
                        }
                    };
                    if (I.paired()) {
                        const int loads = 4 * (I.te - I.tb);
#pragma unroll 1
                        for (int i = 0; i < loads && ok; ++i) {
                            const bool ends = i < 2 || i >= loads - 2;
                            const int kv = i >= 2 && (i >= loads - 2 || !(i & 1)) ? 1 : 0;
                            load(I.tb + (i < 2 ? 0 : ((i - 2) >> 2) + 1 - kv), kv, I.kh + ((ends ? i : (i - 2) >> 1) & 1));
                        }
                    } else {
                        for (int j = I.tb; j < I.te && ok; ++j) {
#pragma unroll 1
                            for (int kv = 0; kv < 2 && ok; ++kv) load(j, kv, I.kh);
                        }
                    }
                    if (!ok) break;
                }
                // every copy has landed before the CTA exits: the last use of each stage was in the
                // current round (parity ph ^ 1) below `st`, in the one before from `st` on
                for (uint32_t i = 0; i < used; ++i) mbar_wait_drain(&kv_full[i], i < st ? ph ^ 1u : ph);
            }
            __syncwarp();
        } else if (warp == 2) {
            // ============================================================ Q producer
            if (lane == 0) {
                const uint64_t pol = l2_policy_evict_first();
                uint32_t used = 0, par = 0;        // bit h: the buffer was used; parity of its last use
                const uint32_t bytes = static_cast<uint32_t>(C::kNB * p.bt * p.g * 128);
                for (uint32_t it = 0;; ++it) {
                    const uint32_t slot = it % kShRing;
                    if (!sh_wait(&item_full[slot], (it / kShRing) & 1, abort_flag) || !ring[slot].more) break;
                    const int row0 = ring[slot].row0, kh = ring[slot].kh;
                    const int next_row = ring[slot].paired() ? 0 : p.bt, next_head = ring[slot].paired() ? 1 : 0;
                    const uint32_t have = (ring[slot].act[0] > 0 ? 1u : 0u) | (ring[slot].act[1] > 0 ? 2u : 0u);
                    mbar_arrive(&item_empty[slot]);
                    bool ok = true;
                    // into L2 while the item before still uses the buffers
#pragma unroll 1
                    for (int h = 0; h < kShTiles; ++h)
                        if ((have >> h) & 1u) {
#pragma unroll 1
                            for (int b = 0; b < C::kNB; ++b) tma_prefetch_4d(&tm_q, b * 64, 0, kh + h * next_head, row0 + h * next_row);
                        }
#pragma unroll 1
                    for (int h = 0; h < kShTiles; ++h) {
                        if (!ok || !((have >> h) & 1u)) continue;
                        if (((used >> h) & 1u) && !sh_wait(&q_empty[h], (par >> h) & 1u, abort_flag)) {
                            ok = false;
                            continue;
                        }
                        mbar_arrive_expect_tx(&q_full[h], bytes);
#pragma unroll 1
                        for (int b = 0; b < C::kNB; ++b)
                            tma_load_4d(smem + C::kOffQ + h * C::kTileBytes + b * C::kBox, &tm_q, &q_full[h], b * 64, 0,
                                        kh + h * next_head, row0 + h * next_row, pol);
                        if ((used >> h) & 1u) par ^= 1u << h;
                        used |= 1u << h;
                    }
                    if (!ok) break;
                }
                for (int h = 0; h < kShTiles; ++h)
                    if ((used >> h) & 1u) mbar_wait_drain(&q_full[h], (par >> h) & 1u);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ============================================================ MMA issuer
            // One thread for both query tiles, so that [P.V of a tile, QK of its next] of one query tile
            // runs whole before the other's: that staggers the two softmax warpgroups, and each has the
            // special-function units to itself while the tensor core works for the other.
            if (lane == 0) {
                constexpr uint32_t kIdescQK0 = idesc_bf16_f32(128, 0, 0);      // N is set per tile
                constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, 1);
                const uint64_t dq = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
                const uint64_t dk0 = sdesc_sw128(smem_u32(smem + C::kOffKV), 16, 1024);
                const uint64_t dv0 = sdesc_sw128(smem_u32(smem + C::kOffKV), C::kBox, 1024);
                const uint32_t tS = tmem + C::kColS, tO = tmem + C::kColO;
                uint32_t st = 0, ph = 0;         // stage of the next K or V tile, and its parity
                auto bump = [&]() {
                    if (++st == C::kStages) {
                        st = 0;
                        ph ^= 1u;
                    }
                };
                // Per query tile h, in byte h: the 16-key steps of a tile (0: no keys; S then has 16 * steps
                // columns).  Bit h of the others.
                uint32_t prev = 0;               // steps of the tile whose P.V come next, with V from stage vs
                uint32_t vs = 0, vph = 0;
                uint32_t fresh = 0;              // the item's first P.V is still to come
                uint32_t outs = 0;               // query tiles whose output the previous item completes
                uint32_t p_par = 0, q_par = 0;   // parities of p_full and q_full
                bool ok = true;
                // P.V of the previous tile, then QK of this one with K from stage ks.
                auto turn = [&](int h, uint32_t cur, uint32_t ks) {
                    const int sp = (prev >> (8 * h)) & 0xff, sc = (cur >> (8 * h)) & 0xff;
                    const uint32_t a = tS + kShKeys * h, d = tO + D * h;
                    if (sp > 0) {
                        const uint64_t dv = dv0 + static_cast<uint64_t>((vs * C::kTileBytes) >> 4);
                        const uint32_t par = (p_par >> h) & 1u;
                        uint32_t acc = ((fresh >> h) & 1u) ^ 1u;
                        p_par ^= 1u << h;
                        fresh &= ~(1u << h);
                        if (!sh_wait(&p_full[2 * h], par, abort_flag)) return false;
                        tc_fence_after();
                        if (sp >= 4) {
                            sh_mma_pv4(d, a, dv, kIdescPV, acc);
                        } else {
#pragma unroll 1
                            for (int k = 0; k < sp; ++k, acc = 1u)
                                mma_ts(d, a + 8 * k, dv + static_cast<uint64_t>(128 * k), kIdescPV, acc);
                        }
                        if (!sh_wait(&p_full[2 * h + 1], par, abort_flag)) return false;
                        tc_fence_after();
                        if (sp == 8) {
                            sh_mma_pv4(d, a + 32, dv + 512, kIdescPV, 1u);
                        } else {
#pragma unroll 1
                            for (int k = 4; k < sp; ++k)
                                mma_ts(d, a + 8 * k, dv + static_cast<uint64_t>(128 * k), kIdescPV, 1u);
                        }
                    }
                    // S overwrites the P that the P.V just issued reads: tcgen05.mma operations of one
                    // thread execute in issue order.
                    if (sc > 0)
                        sh_mma_qk<C::kNB>(a, dq + static_cast<uint64_t>((h * C::kTileBytes) >> 4),
                                          dk0 + static_cast<uint64_t>((ks * C::kTileBytes) >> 4),
                                          kIdescQK0 | (static_cast<uint32_t>(2 * sc) << 17), &s_full[h]);
                    return true;
                };
                if constexpr (LAST) {
                    // The stages come in the order of the turns.  A turn is in the code twice only: few rows
                    // leave the tensor core time, and the loops of all roles share the instruction cache.
                    bool was_pair = false;
                    for (uint32_t it = 0; ok; ++it) {
                        const uint32_t slot = it % kShRing;
                        ok = sh_wait(&item_full[slot], (it / kShRing) & 1, abort_flag);
                        if (!ok) break;
                        const Item &I = ring[slot];
                        // ---- the previous item's last P.V, which do not wait for this one's Q
#pragma unroll 1
                        for (int h = 0; h < kShTiles && outs != 0; ++h) {
                            vs = st;
                            ok = (h > 0 && !was_pair) || sh_wait(&kv_full[st], ph, abort_flag);
                            ok = ok && turn(h, 0, 0);
                            if (!ok) break;
                            if ((outs >> h) & 1u) mma_commit(&o_full[h]);
                            if (h == 1 || was_pair) {
                                mma_commit(&kv_empty[st]);
                                bump();
                            }
                        }
                        if (!ok || !I.more) break;
                        const int tb = I.tb, te = I.te, whole_end = I.plen >> kShKeysLog;
                        const uint32_t have = (I.act[0] > 0 ? 1u : 0u) | (I.act[1] > 0 ? 2u : 0u);
                        const bool pair = I.paired();
                        was_pair = pair;
                        prev = 0;
                        fresh = 3u;
                        outs = have;
#pragma unroll 1
                        for (int j = tb; j < te && ok; ++j) {
                            uint32_t cur = 0;
#pragma unroll 1
                            for (int h = 0; h < kShTiles; ++h)
                                if ((have >> h) & 1u)
                                    cur |= (j < whole_end ? 8u : static_cast<uint32_t>((max(I.keys_of(h, j), 0) + 15) >> 4))
                                           << (8 * h);
                            uint32_t ks = 0;
#pragma unroll 1
                            for (int h = 0; h < kShTiles; ++h) {
                                if (pair || h == 0) {
                                    if (j > tb) {
                                        vs = st;
                                        ok = sh_wait(&kv_full[vs], ph, abort_flag);
                                        bump();
                                    }
                                    ks = st;
                                    ok = ok && sh_wait(&kv_full[ks], ph, abort_flag);
                                    bump();
                                }
                                if (j == tb && ok && ((have >> h) & 1u)) {
                                    ok = sh_wait(&q_full[h], (q_par >> h) & 1u, abort_flag);
                                    q_par ^= 1u << h;
                                    tc_fence_after();
                                }
                                ok = ok && turn(h, cur, ks);
                                if (!ok) break;
                                if (pair || h == 1) {
                                    if (j > tb) mma_commit(&kv_empty[vs]);
                                    mma_commit(&kv_empty[ks]);
                                }
                            }
                            prev = cur;
                        }
                        if (!ok) break;
                        if (have & 1u) mma_commit(&q_empty[0]);
                        if (have & 2u) mma_commit(&q_empty[1]);
                        mbar_arrive(&item_empty[slot]);
                    }
                } else {
                    // the P.V of an item's last tile
                    auto finish = [&]() {
                        if (outs == 0) return true;
                        if (!sh_wait(&kv_full[vs], vph, abort_flag)) return false;
#pragma unroll 1
                        for (int h = 0; h < kShTiles; ++h) {
                            if (!turn(h, 0, 0)) return false;
                            if ((outs >> h) & 1u) mma_commit(&o_full[h]);
                        }
                        mma_commit(&kv_empty[vs]);
                        return true;
                    };
                    for (uint32_t it = 0;; ++it) {
                        const uint32_t slot = it % kShRing;
                        if (!sh_wait(&item_full[slot], (it / kShRing) & 1, abort_flag)) { ok = false; break; }
                        const Item &I = ring[slot];
                        // the previous item's last P.V, which do not wait for this one's Q
                        ok = finish();
                        if (!ok || !I.more) break;
                        const int tb = I.tb, te = I.te, whole_end = I.plen >> kShKeysLog;
                        const uint32_t have = (I.act[0] > 0 ? 1u : 0u) | (I.act[1] > 0 ? 2u : 0u);
                        auto steps_of = [&](int j) {
                            if (j < whole_end) return ((have & 1u) ? 8u : 0u) | ((have & 2u) ? 8u << 8 : 0u);
                            uint32_t r = 0;
#pragma unroll 1
                            for (int h = 0; h < kShTiles; ++h)
                                if ((have >> h) & 1u) r |= static_cast<uint32_t>((max(I.keys_of(h, j), 0) + 15) >> 4) << (8 * h);
                            return r;
                        };
                        uint32_t cur = steps_of(tb);
                        uint32_t ks = st;
                        // ---- the first tile
                        ok = sh_wait(&kv_full[ks], ph, abort_flag);
                        prev = 0;
                        fresh = 3u;
                        outs = have;
#pragma unroll 1
                        for (int h = 0; h < kShTiles && ok; ++h) {
                            if (!((have >> h) & 1u)) continue;
                            ok = sh_wait(&q_full[h], (q_par >> h) & 1u, abort_flag);
                            q_par ^= 1u << h;
                            if (ok) {
                                tc_fence_after();
                                turn(h, cur, ks);
                            }
                        }
                        if (!ok) break;
                        mma_commit(&kv_empty[ks]);
                        bump();
                        vs = st;
                        vph = ph;
                        bump();
                        prev = cur;
                        // ---- the others
                        for (int j = tb + 1; j < te; ++j) {
                            cur = steps_of(j);
                            ks = st;
                            ok = sh_wait(&kv_full[vs], vph, abort_flag) && sh_wait(&kv_full[ks], ph, abort_flag) &&
                                 turn(0, cur, ks) && turn(1, cur, ks);
                            if (!ok) break;
                            mma_commit(&kv_empty[vs]);
                            mma_commit(&kv_empty[ks]);
                            bump();
                            vs = st;
                            vph = ph;
                            bump();
                            prev = cur;
                        }
                        if (!ok) break;
                        if (have & 1u) mma_commit(&q_empty[0]);
                        if (have & 2u) mma_commit(&q_empty[1]);
                        mbar_arrive(&item_empty[slot]);
                    }
                }
                mma_commit(mma_final);           // every MMA issued completes before TMEM is released
                mbar_wait_drain(mma_final, 0);
            }
            __syncwarp();
        }
    } else {
        reg_alloc<C::kRegsSoftmax>();
        // ================================================================ softmax + output
        const int h = (warp - 4) >> 2;
        const int quad = warp & 3;
        const int trow = quad * 32 + lane;                 // row of the query tile
        const int lr = trow / p.g;                         // its (token or sample) row within the tile
        const int hh = trow - lr * p.g;                    // and its head of the kv head
        const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t tS = tmem + lane_addr + C::kColS + kShKeys * h;
        const uint32_t tO = tmem + lane_addr + C::kColO + D * h;
        const float sl2 = MODE == kShPlain ? p.scale_log2 : 1.f;
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        uint32_t n = 0, tiles = 0, outs = 0;               // K and V tiles passed; tiles and outputs of h
        bool ok = true;
        for (uint32_t it = 0; ok; ++it) {
            const uint32_t rslot = it % kShRing;
            if (!sh_warp_wait(&item_full[rslot], (it / kShRing) & 1, abort_flag)) break;
            const Item &I = ring[rslot];
            if (!I.more) break;
            const int act = I.act[h];
            const int rows_h = I.rows(h, p.bt);
            const bool live = lr < p.bt && lr < rows_h;
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int row = I.first_row(h, p.bt) + lr;     // packed token, or sample
            float m = MODE == kShCappedFixed ? 0.f : -INFINITY;      // running maximum, base-2 units
            float l = 0.f;             // running sum of 2^(x - m)
            float fix = 0.f;           // what rounding the tiles' largest weights to bf16 adds to l
            bool seen = false;         // this row has a key in one of the tiles
            int done = 0;              // tiles of this item so far

            // P of the first (half 0) or second 64 keys of the tile is stored
            auto hand_over = [&](int half) {
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * h + half]);
            };

            // The running maximum becomes m_new.  O holds the earlier tiles, all complete (the commit
            // behind this tile's S covers every MMA issued before it).
            auto rescale = [&](float m_new) {
                const float alpha = m == -INFINITY ? 0.f : ex2(m - m_new);
                m = m_new;
                l *= alpha;
                fix *= alpha;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    tmem_ld32(tO + 32 * c, o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] *= alpha;
                    tmem_st32f(tO + 32 * c, o);
                }
            };
            // A tile's sum of weights and its largest one.  P.V multiplies weights rounded to bf16, as the matrix
            // instruction takes P and V of one type.  The rounding of the tile's largest weight enters the sum
            // that O is divided by, which makes the dominant term exact; the log-sum-exp keeps the unrounded sum.
            auto add_sums = [&](float pmax, float sum) {
                fix += __uint_as_float(pack_bf16x2(pmax, 0.f) << 16) - pmax;
                l += sum;
            };
            // the weight of the score mx
            auto weight_of = [&](float mx, float2 negm) {
                return ex2(ffma2(make_float2(mx, mx), make_float2(sl2, sl2), negm).x);
            };

            // own keys this row sees: [lo, hi)
            int lo = 0, hi = 0;
            if (act > 0 && I.te > I.npt) {
                if constexpr (LAST) {
                    if (live) {
                        lo = p.cu_seqlens[row];
                        hi = p.cu_seqlens[row + 1];
                    }
                } else if constexpr (TREE) {
                    lo = I.ka0;                // of these, the node's mask keeps its ancestors and itself
                    hi = live ? row + 1 : lo;
                } else {
                    // the last sample start that is not behind the row; 32 sample starts at a time
                    const int last_row = I.row0 + I.nrows - 1;
                    lo = I.ka0;
#pragma unroll 1
                    for (int s0 = I.s0 + 1;; s0 += 32) {
                        const int start = p.cu_seqlens[min(s0 + lane, p.num_seqs)];
                        const unsigned in = __ballot_sync(0xffffffffu, start <= last_row && s0 + lane < p.num_seqs);
#pragma unroll 1
                        for (int i = 0; i < 32 && ((in >> i) & 1u); ++i) {
                            const int b = __shfl_sync(0xffffffffu, start, i);
                            if (b <= row) lo = b;
                        }
                        if (in != 0xffffffffu) break;
                    }
                    hi = live ? row + 1 : lo;
                }
            }
            const int npt = I.npt, tb = I.tb, te = act > 0 ? I.te : I.tb;
            const int whole_end = I.plen >> kShKeysLog;        // tiles below it: every row sees all 128 keys
#pragma unroll 1
            for (int j = tb; j < te; ++j) {
                int nk = kShKeys, c0 = 0, c1 = kShKeys;    // keys of the tile; this row's columns [c0, c1)
                bool some = warp_live, masked = false, zero_v = false;
                uint4 path = make_uint4(~0u, ~0u, ~0u, ~0u);       // tree: the nodes of the tile that this row sees
                if (j >= whole_end) {
                    nk = I.keys_of(h, j);
                    if (nk <= 0) continue;
                    if (j >= npt) {
                        const int base = I.own_base(j);
                        c0 = min(max(lo - base, 0), kShKeys);
                        c1 = min(max(hi - base, 0), nk);
                        if constexpr (TREE) {
                            path = make_uint4(0u, 0u, 0u, 0u);
                            if (live)
                                path = *reinterpret_cast<const uint4 *>(p.tree + static_cast<int64_t>(row) * p.tree_words +
                                                                        (kShKeys / 32) * (j - npt));
                        }
                    } else {
                        c1 = nk;
                    }
                    some = __any_sync(0xffffffffu, live && c1 > c0);
                    masked = (TREE && j >= npt) || __any_sync(0xffffffffu, live && (c0 > 0 || c1 < kShKeys));
                    zero_v = ((nk + 15) & ~15) > I.keys(j);
                }
                seen = seen || (TREE ? c1 > c0 && (path.x | path.y | path.z | path.w) != 0 : c1 > c0);
                if (!sh_warp_wait(&s_full[h], tiles & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                // Keys behind the last one that any row of the item sees (a later token, another
                // request's rows) have weight 0, but 0 * Inf is NaN: their V rows become zeros.
                if (zero_v) {
                    const uint32_t nv = n + (I.paired() ? 4 * (j - tb) + 2 + (j == I.te - 1 ? h : 2 * h) : 2 * (j - tb) + 1);
                    const uint32_t vs = nv % C::kStages;
                    if (!sh_warp_wait(&kv_full[vs], (nv / C::kStages) & 1, abort_flag)) { ok = false; break; }
                    const int nkeys = I.keys(j);
                    uint8_t *vt = smem + C::kOffKV + vs * C::kTileBytes + nkeys * 128;
                    const int bytes = (((nkeys + 15) & ~15) - nkeys) * 128;      // per column block, at most 15 rows
                    for (int i = trow * 16; i < bytes; i += 128 * 16)
#pragma unroll
                        for (int b = 0; b < C::kNB; ++b)
                            *reinterpret_cast<uint4 *>(vt + b * C::kBox + i) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                if (!some) {
                    // no row of this warp has a key in the tile: P = 0 (without rows: whatever it is)
                    if (warp_live) {
                        uint32_t zr[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) zr[i] = 0u;
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_st16(tS + 16 * c, zr);
                    }
                    hand_over(0);
                    hand_over(1);
                } else {
                    // 32-column chunks in which any row of the warp sees a key: [cf, ce)
                    int cf = 0, ce = kShKeys / 32;
                    if (masked) {
                        const bool sees = live && c1 > c0;
                        cf = __reduce_min_sync(0xffffffffu, sees ? c0 : kShKeys) >> 5;
                        ce = (__reduce_max_sync(0xffffffffu, sees ? c1 : 0) + 31) >> 5;
                    }
                    // bit i: column 32 c + i is in [c0, c1)
                    auto columns = [&](int c) {
                        const int a = min(max(c0 - 32 * c, 0), 32), b = min(max(c1 - 32 * c, 0), 32);
                        const uint32_t below_b = b == 32 ? ~0u : (1u << b) - 1u;
                        const uint32_t in = a == 32 ? 0u : below_b & ~((1u << a) - 1u);
                        if constexpr (TREE) return in & (c < 2 ? (c == 0 ? path.x : path.y) : (c == 2 ? path.z : path.w));
                        return in;
                    };
                    if constexpr (MODE == kShCappedFixed) {
                        float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                        float pmax = 0.f;
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t pk[16];
                            if (c < cf || c >= ce) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) pk[i] = 0u;
                            } else {
                                float x[32];
                                const uint32_t keep = masked ? columns(c) : ~0u;
                                tmem_ld32(tS + 32 * c, x);
                                if (masked) {              // may be NaN, which is not to reach its neighbours
#pragma unroll
                                    for (int i = 0; i < 32; ++i)
                                        if (!((keep >> i) & 1u)) x[i] = 0.f;
                                }
#pragma unroll
                                for (int i = 0; i < 32; i += 4) {
                                    capped4(x + i, p.cap_in, p.cap_log2);
#pragma unroll
                                    for (int k = i; k < i + 4; ++k) x[k] = ex2(x[k]);
                                }
                                if (masked) {
#pragma unroll
                                    for (int i = 0; i < 32; ++i)
                                        if (!((keep >> i) & 1u)) x[i] = 0.f;
                                }
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    rs[i & 1] = fadd2(rs[i & 1], make_float2(x[2 * i], x[2 * i + 1]));
                                    pmax = fmax3f(pmax, x[2 * i], x[2 * i + 1]);
                                    pk[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
                                }
                            }
                            tmem_st16(tS + 16 * c, pk);          // over scores that have been read
                            if (c & 1) hand_over(c >> 1);
                        }
                        add_sums(pmax, (rs[0].x + rs[1].x) + (rs[0].y + rs[1].y));
                    } else if (MODE == kShPlain && ce - cf <= 3) {
                        // Few columns count, as in most own tiles of prefill: the maximum over those chunks first,
                        // then their weights, 32 columns at a time in short code.  With four chunks the path
                        // below is the faster one (32 samples of 200 keys, last token: 121 us, 131 by this one);
                        // a limit of two leaves too many prefill tiles to it (32 requests of 15 samples of 16-96
                        // tokens: 184 us, 160 with three).
                        float x[32], mx = -INFINITY;
                        auto load = [&](int c) {
                            const uint32_t keep = columns(c);
                            tmem_ld32(tS + 32 * c, x);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((keep >> i) & 1u)) x[i] = -INFINITY;
                        };
#pragma unroll 1
                        for (int c = cf; c < ce; ++c) {
                            load(c);
#pragma unroll
                            for (int i = 0; i < 32; i += 2) mx = fmax3f(mx, x[i], x[i + 1]);
                        }
                        const float m_new = fmaxf(m, mx * sl2);
                        if (done == 0) m = m_new;
                        if (__any_sync(0xffffffffu, m_new > m + 8.f)) rescale(m_new);
                        const float mu = m == -INFINITY ? 0.f : m;
                        const float2 sl2x2 = make_float2(sl2, sl2), negm = make_float2(-mu, -mu);
                        float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t pk[16];
                            if (c < cf || c >= ce) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) pk[i] = 0u;
                            } else {
                                load(c);
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const float2 t = ffma2(make_float2(x[2 * i], x[2 * i + 1]), sl2x2, negm);
                                    const float2 w = make_float2(ex2(t.x), ex2(t.y));
                                    rs[i & 1] = fadd2(rs[i & 1], w);
                                    pk[i] = pack_bf16x2(w.x, w.y);
                                }
                            }
                            tmem_st16(tS + 16 * c, pk);          // over scores that have been read
                            if (c & 1) hand_over(c >> 1);
                        }
                        add_sums(weight_of(mx, negm), (rs[0].x + rs[1].x) + (rs[0].y + rs[1].y));
                    } else {
                        float s[kShKeys];
                        tmem_ld64(tS, s);
                        tmem_ld64(tS + 64, s + 64);
                        if constexpr (MODE == kShCapped) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                // a masked score may be NaN, and is not to reach its neighbours
                                const uint32_t keep = masked ? columns(c) : ~0u;
#pragma unroll
                                for (int i = 32 * c; i < 32 * c + 32; ++i)
                                    if (!((keep >> (i & 31)) & 1u)) s[i] = 0.f;
#pragma unroll
                                for (int i = 32 * c; i < 32 * c + 32; i += 4) capped4_any(s + i, p.cap_in, p.cap_log2);
                            }
                        }
                        if (masked) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const uint32_t keep = columns(c);
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (!((keep >> i) & 1u)) s[32 * c + i] = -INFINITY;
                            }
                        }
                        float mq[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) mq[q] = fmaxf(s[16 * q], s[16 * q + 1]);
#pragma unroll
                        for (int c = 2; c < 16; c += 2)
#pragma unroll
                            for (int q = 0; q < 8; ++q) mq[q] = fmax3f(mq[q], s[16 * q + c], s[16 * q + c + 1]);
                        const float mx =
                            fmax3f(fmax3f(mq[0], mq[1], mq[2]), fmax3f(mq[3], mq[4], mq[5]), fmaxf(mq[6], mq[7]));
                        const float m_new = fmaxf(m, mx * sl2);
                        if (done == 0) m = m_new;
                        const float2 sl2x2 = make_float2(sl2, sl2);
                        float2 negm, rs[4];
                        uint32_t pk[32];
                        auto weights = [&](int c, uint32_t *w) {       // of columns 32 c .. 32 c + 31, as bf16 pairs
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 x = ffma2(make_float2(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]), sl2x2, negm);
                                const float2 e = make_float2(ex2(x.x), ex2(x.y));
                                rs[i & 3] = fadd2(rs[i & 3], e);
                                w[i] = pack_bf16x2(e.x, e.y);
                            }
                        };
                        // The first half's weights use the maximum so far, so that they need not wait for
                        // this tile's; only when that grows by more than 2^8 is O rescaled and the half redone.
#pragma unroll 1
                        for (;;) {
                            const float mu = m == -INFINITY ? 0.f : m;  // no key yet: p = 0, not NaN
                            negm = make_float2(-mu, -mu);
#pragma unroll
                            for (int q = 0; q < 4; ++q) rs[q] = make_float2(0.f, 0.f);
                            weights(0, pk);
                            weights(1, pk + 16);
                            if (!__any_sync(0xffffffffu, m_new > m + 8.f)) break;
                            rescale(m_new);
                        }
                        tmem_st16(tS, pk);
                        tmem_st16(tS + 16, pk + 16);
                        hand_over(0);
                        weights(2, pk);
                        tmem_st16(tS + 32, pk);
                        weights(3, pk + 16);
                        tmem_st16(tS + 48, pk + 16);
                        hand_over(1);
                        const float2 r01 = fadd2(rs[0], rs[1]), r23 = fadd2(rs[2], rs[3]);
                        add_sums(weight_of(mx, negm), (r01.x + r23.x) + (r01.y + r23.y));
                    }
                }
                ++done;
                ++tiles;
            }
            n += (I.paired() ? 4 : 2) * (I.te - tb);
            if (!ok) break;
            // ------------------------------------------------------------ output of the item
            const int slot = I.slot, kh = I.head(h);
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[rslot]);    // the item has been read
            if (act > 0) {
                if (!sh_warp_wait(&o_full[h], outs & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                ++outs;
            }
            if (!warp_live) continue;
            const int64_t orow = static_cast<int64_t>(row) * p.Hq + kh * p.g + hh;
            const int64_t prow = static_cast<int64_t>(slot) * (kShTiles * kShRows) + h * kShRows + trow;
            const bool whole = slot < 0;                       // the item's only part
            if (live) {
                if (whole) {
                    if (!seen && p.dev_status) atomicOr(p.dev_status, BG_DEVSTAT_EMPTY_ROW);
                    if (seen && p.lse) p.lse[orow] = (m + __log2f(l)) * 0.69314718055994530942f;
                } else {
                    // -inf: no key; kShNoWeight: keys whose scores are all -inf
                    p.part_l[prow] = make_float2(!seen ? -INFINITY : l == 0.f ? kShNoWeight : m + __log2f(l),
                                                 seen ? fix / l : 0.f);
                }
            }
            if (act > 0) {
                const float inv = 1.f / (whole ? l + fix : l);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    tmem_ld32(tO + 32 * c, o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] *= inv;
                    if (live && seen) {
                        if (whole) {
                            uint32_t wv[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) wv[i] = pack_bf16x2(o[2 * i], o[2 * i + 1]);
                            st_out_32b(p.out + orow * D + 32 * c, wv, wide);
                            st_out_32b(p.out + orow * D + 32 * c + 16, wv + 8, wide);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                st_global_32b(p.part_o + prow * D + 32 * c + 8 * i,
                                              reinterpret_cast<const uint32_t *>(o) + 8 * i);
                        }
                    }
                }
            }
            tc_fence_before();         // O is read before the next item's first P.V overwrites it
        }
    }

    // ------------------------------------------------------------------------ teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    if (threadIdx.x == 0 && *abort_flag) {
        p.hdr[kShHdrStatus] = BG_DEVSTAT_TIMEOUT;      // the join would read parts that were never written
        if (p.dev_status) atomicOr(p.dev_status, BG_DEVSTAT_TIMEOUT);
    }
}

// ------------------------------------------------------------------------------------ join
// out = sum_i 2^(L_i - L) O_i / (1 + sum_i 2^(L_i - L) fix_i) with L = log2 sum_i 2^(L_i): the
// pieces' own normalised outputs, in piece order.
constexpr int kJoinThreads = 256;

// LANES of a row, AT_ONCE pieces of it under way.  Many rows of two or three pieces are bound by the
// latencies of the few loads each needs, times the waves of CTAs: few lanes and registers per row.  Few
// rows of many pieces leave the SMs empty: twice the lanes, more pieces at once (4 requests of 32 samples
// over 32768 keys, 10 pieces: 114.4 us, 119.6 by the first form; 32 requests of 15 samples, last token:
// 46.3 by the first, 47.3 by the second).
template <int D, int LANES, int AT_ONCE>
__global__ void __launch_bounds__(kJoinThreads) shared_join_kernel(const ShParams p)
{
    grid_dep_launch();
    grid_dep_wait();
    constexpr int kRows = kJoinThreads / LANES, kParts = kShTiles * kShRows / kRows, N4 = D / (4 * LANES);
    const int split = static_cast<int>(blockIdx.x) / kParts;
    const int sub = threadIdx.x % LANES;
    const int r = (static_cast<int>(blockIdx.x) - split * kParts) * kRows + threadIdx.x / LANES;
    const ShSplit S = p.splits[split];         // (not looked at unless it is one)
    bool other;
    if (!plan_ready(p, &other) || split >= p.hdr[kShHdrSplits]) return;
    const int h = r / kShRows, trow = r - h * kShRows;
    const int lr = trow / p.g, hh = trow - lr * p.g;
    const int row = S.pair ? lr : h * p.bt + lr, kh = S.pair ? S.kh + h : S.kh;
    if (lr >= p.bt || row >= S.nrows) return;
    const unsigned lanes = ((1u << LANES) - 1u) << (threadIdx.x & (32 - LANES));      // of this row
    // piece 0 is in the first CTA's second slot, the others in their CTA's first: slot0 + 2 t - (t > 0)
    const int64_t row0 = static_cast<int64_t>(2 * S.cta + 1) * (kShTiles * kShRows) + r;
    auto row_of = [&](int t) { return row0 + (t > 0 ? 2 * t - 1 : 0) * (kShTiles * kShRows); };
    float2 lf[AT_ONCE];
    float4 o[AT_ONCE][N4];                     // float4 i of a lane is at 4 * (sub + LANES * i)
    auto load = [&](int t0) {
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int64_t at = row_of(min(t0 + k, S.pieces - 1));
            lf[k] = t0 + k < S.pieces ? p.part_l[at] : make_float2(-INFINITY, 0.f);
            const float4 *src = reinterpret_cast<const float4 *>(p.part_o + at * D) + sub;
#pragma unroll
            for (int i = 0; i < N4; ++i) o[k][i] = src[LANES * i];
        }
    };
    load(0);                                   // under way while the maximum is found
    float mx = -INFINITY;
    bool keys = false;
#pragma unroll 1
    for (int t = sub; t < S.pieces; t += LANES) {
        const float lt = p.part_l[row_of(t)].x;
        mx = fmaxf(mx, lt);
        keys = keys || lt != -INFINITY;
    }
#pragma unroll
    for (int w = LANES / 2; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(lanes, mx, w));
    keys = (__ballot_sync(lanes, keys) & lanes) != 0;
    if (!keys) {                               // no piece has a key for this row
        if (sub == 0 && p.dev_status) atomicOr(p.dev_status, BG_DEVSTAT_EMPTY_ROW);
        return;
    }
    float sum = 0.f, fix = 0.f;
    float4 acc[N4];
#pragma unroll
    for (int i = 0; i < N4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int t0 = 0;;) {
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            if (lf[k].x <= kShNoWeight) continue;            // weights of 0, or not written: part_o holds anything
            const float wt = ex2(lf[k].x - mx);
            sum += wt;
            fix = fmaf(wt, lf[k].y, fix);
#pragma unroll
            for (int i = 0; i < N4; ++i) {
                acc[i].x = fmaf(wt, o[k][i].x, acc[i].x);
                acc[i].y = fmaf(wt, o[k][i].y, acc[i].y);
                acc[i].z = fmaf(wt, o[k][i].z, acc[i].z);
                acc[i].w = fmaf(wt, o[k][i].w, acc[i].w);
            }
        }
        t0 += AT_ONCE;
        if (t0 >= S.pieces) break;
        load(t0);
    }
    const float inv = 1.f / (sum + fix);
    const int64_t orow = (static_cast<int64_t>(S.row0) + row) * p.Hq + kh * p.g + hh;
    uint2 *dst = reinterpret_cast<uint2 *>(p.out + orow * D) + sub;
#pragma unroll
    for (int i = 0; i < N4; ++i)
        dst[LANES * i] = make_uint2(pack_bf16x2(acc[i].x * inv, acc[i].y * inv),
                                         pack_bf16x2(acc[i].z * inv, acc[i].w * inv));
    if (p.lse && sub == 0) p.lse[orow] = (mx + __log2f(sum)) * 0.69314718055994530942f;
}

template <int D, int MODE, bool LAST, bool TREE>
cudaError_t launch_one(const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                       const CUtensorMap &tm_pk, const CUtensorMap &tm_pv, const ShParams &p, int grid, int join,
                       cudaStream_t stream)
{
    using C = ShCfg<D>;
    auto kern = shared_attn_kernel<D, MODE, LAST, TREE>;
    static std::atomic<uint64_t> smem_done{0}, split_done{0};
    cudaError_t e = ensure_smem_attribute(kern, C::kSmemBytes, smem_done);
    if (e != cudaSuccess) return e;
    e = check_register_split(kern, C::kThreads, C::kSplitRegs, split_done);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, dim3(grid), dim3(C::kThreads), C::kSmemBytes, stream, tm_q, tm_k, tm_v, tm_pk, tm_pv, p);
    if (e != cudaSuccess || join == kShJoinNone) return e;
    // at most one cut item per CTA
    constexpr int kFew = 8, kMany = 16;
    const bool many = join == kShJoinMany;
    return launch_dependent(many ? shared_join_kernel<D, kMany, 4> : shared_join_kernel<D, kFew, 2>,
                            dim3(grid * (kShTiles * kShRows * (many ? kMany : kFew) / kJoinThreads)),
                            dim3(kJoinThreads), 0, stream, p);
}

}  // namespace

namespace {

// Most key tiles of an entry: its prefix, and the own keys of the rows it holds (prefill: one sample's
// start to the entry's last row; last token: whole samples).
int64_t most_tiles(const ShProblem &pb)
{
    const int64_t bt = kShRows / (pb.Hq / pb.Hkv);
    int64_t own = pb.last ? kShTiles * bt * pb.max_seqlen : pb.max_seqlen + kShTiles * bt;
    if (own > pb.total_tokens) own = pb.total_tokens;
    return ceil_div(pb.max_prefix_len, kShKeys) + ceil_div(own, kShKeys);
}

}  // namespace

int shared_tiles(const ShProblem &pb)
{
    const int bt = kShRows / (pb.Hq / pb.Hkv);
    const int64_t items = (static_cast<int64_t>(pb.total_tokens) / (kShTiles * bt) + pb.num_groups) * pb.Hkv;
    return !pb.last && 2 * items <= kShMaxCtas && most_tiles(pb) < kShSplitTiles ? 1 : kShTiles;
}

int shared_heads(const ShProblem &pb)
{
    if (!pb.last || pb.Hkv % 2 != 0) return 1;
    const int64_t tiles = static_cast<int64_t>(pb.total_prefix) / kShKeys + pb.total_tokens / kShKeys;
    return 10 * tiles * (pb.Hkv / 2) >= kShMaxCtas * ceil_div(pb.max_prefix_len, kShKeys) ? 2 : 1;
}

ShLayout shared_layout(const ShProblem &pb)
{
    ShLayout L;
    const int bt = kShRows / (pb.Hq / pb.Hkv);
    const int64_t rows = pb.last ? pb.num_seqs : pb.total_tokens;
    const int most = pb.last && pb.Hkv % 2 == 0 ? 2 : 1;       // of shared_heads
    L.max_entries = rows / (shared_tiles(pb) * bt) + pb.num_groups + 1;
    const int64_t tiles = most_tiles(pb);
    L.items = L.max_entries * pb.Hkv;
    L.units = L.items * (tiles + kItemUnits);
    L.slots = 0;
    if (tiles >= kShSplitTiles) {
        const int64_t ctas = ceil_div(L.units * most, kShSplitMin);
        L.slots = 2 * (ctas < kShMaxCtas ? ctas : kShMaxCtas);
    }
    L.max_entries *= most;
    auto al = [](size_t b) { return (b + 255) & ~size_t(255); };
    L.entries = 256;
    L.sorted = L.entries + al(L.max_entries * sizeof(ShEntry));
    L.starts = L.sorted + (L.slots == 0 ? al(L.max_entries * sizeof(ShEntry)) : 0);
    L.splits = L.starts + al((kShMaxCtas + 1) * sizeof(ShStart));
    L.part_l = L.splits + al(kShMaxCtas * sizeof(ShSplit));
    L.part_o = L.part_l + al(static_cast<size_t>(L.slots) * kShTiles * kShRows * 2 * sizeof(float));
    L.tree = L.part_o + al(static_cast<size_t>(L.slots) * kShTiles * kShRows * pb.head_dim * sizeof(float));
    L.total = L.tree + (pb.tree ? al(static_cast<size_t>(pb.total_tokens) * tree_words(pb.max_seqlen) * 4) : 0);
    return L;
}

ShKey shared_key(const ShProblem &pb, int grid)
{
    return ShKey{{pb.tree ? 2 : pb.last, pb.num_seqs, pb.total_tokens, pb.max_seqlen, pb.num_groups, pb.total_prefix,
                  pb.max_prefix_len, pb.Hq, pb.Hkv, pb.head_dim, grid, 0x5348}};
}

cudaError_t launch_shared_plan(const ShProblem &pb, const ShLayout &lay, void *workspace, int grid,
                               int32_t *dev_status, cudaStream_t stream)
{
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    return launch_dependent(shared_plan_kernel, dim3(pb.tree ? 1 + pb.num_groups : 1), dim3(kPlanThreads), 0, stream, pb, shared_key(pb, grid),
                            kShRows / (pb.Hq / pb.Hkv), reinterpret_cast<int32_t *>(ws),
                            reinterpret_cast<ShEntry *>(ws + lay.entries), reinterpret_cast<ShEntry *>(ws + lay.sorted),
                            reinterpret_cast<ShStart *>(ws + lay.starts),
                            reinterpret_cast<ShSplit *>(ws + lay.splits), grid, lay.slots > 0 ? 1 : 0, shared_tiles(pb), shared_heads(pb),
                            pb.tree ? reinterpret_cast<uint32_t *>(ws + lay.tree) : nullptr, dev_status);
}

cudaError_t launch_shared_attn(int head_dim, bool is_capped, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                               const CUtensorMap &tm_v, const CUtensorMap &tm_pk, const CUtensorMap &tm_pv,
                               const ShParams &p, int grid, int join, cudaStream_t stream)
{
    const int mode = !is_capped ? kShPlain : p.cap_log2 <= kShCapFixed ? kShCappedFixed : kShCapped;
#define BG_SHARED(DD, MM)                                                                                   \
    if (head_dim == DD && mode == MM)                                                                       \
        return p.tree   ? launch_one<DD, MM, false, true>(tm_q, tm_k, tm_v, tm_pk, tm_pv, p, grid, join, stream)  \
               : p.last ? launch_one<DD, MM, true, false>(tm_q, tm_k, tm_v, tm_pk, tm_pv, p, grid, join, stream)  \
                        : launch_one<DD, MM, false, false>(tm_q, tm_k, tm_v, tm_pk, tm_pv, p, grid, join, stream)
    BG_SHARED(128, kShPlain);
    BG_SHARED(128, kShCapped);
    BG_SHARED(128, kShCappedFixed);
    BG_SHARED(64, kShPlain);
    BG_SHARED(64, kShCapped);
    BG_SHARED(64, kShCappedFixed);
#undef BG_SHARED
    return cudaErrorInvalidValue;
}

}  // namespace bg
