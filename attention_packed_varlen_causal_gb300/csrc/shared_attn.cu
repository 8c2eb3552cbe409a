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
//
// A query tile is dense over the rows of the REQUEST, not of one sample: its 128 rows are
// (row, head of the kv head) pairs of consecutive packed rows, whatever samples they belong to.
// Against the prefix nothing but the prefix's end is masked, so short samples and few heads still
// fill the tensor core's 128 rows; against the own keys every row keeps the interval [lo, hi) of
// its sample (block-diagonal), and key tiles that no row of a query tile sees are skipped.
// kShTiles query tiles share every K/V tile that is loaded.
//
// Three launches on the caller's stream:
//   1. shared_plan_kernel (one CTA) checks the offsets on the device and writes the work list,
//      costliest entries first; entries with long key ranges are split into pieces when there are
//      too few of them to fill the GPU.
//   2. shared_attn_kernel: one persistent CTA per SM, 12 warps:
//        warp 0      TMA producer of K and V tiles of 128 keys (one ring for both)
//        warp 2      TMA producer of Q
//        warps 1, 3  tcgen05.mma issuers, one thread per query tile
//        warps 4-11  softmax and output, one warpgroup per query tile, one thread per row
//      The scores of a query tile (128 fp32 TMEM columns) are overwritten by its weights P (64
//      columns), so a tile alternates between its softmax and its two products; the two tiles of
//      a CTA take turns on the tensor core.
//   3. shared_join_kernel joins the pieces of split entries (only where sizes allow a split).
// Every wait is bounded (bg::mbar_wait); on a time-out every role leaves, copies and MMAs in
// flight are drained, TMEM is freed and BG_DEVSTAT_TIMEOUT is reported.
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "bg_internal.h"
#include "bg_ptx.cuh"
#include "shared_attn.h"

namespace bg {

namespace {

// ------------------------------------------------------------------------------------ plan
constexpr int kPlanThreads = 1024;
constexpr int kPlanBuckets = kPlanThreads;      // cost classes of the work list (the last: and above)

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
    if (warp == 0) {
        int w = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += u;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    *total = s_warp[kPlanThreads / 32 - 1];
    return incl - v + (warp > 0 ? s_warp[warp - 1] : 0);
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

__global__ void __launch_bounds__(kPlanThreads)
    shared_plan_kernel(const ShProblem pb, const ShKey key, int bt, int32_t *hdr, ShEntry *__restrict__ entries,
                       ShEntry *__restrict__ raw, ShSplit *__restrict__ splits, int64_t slots, int32_t *dev_status)
{
    __shared__ int s_err, s_nsplit, s_nslot;
    __shared__ int s_warp[32];
    __shared__ int s_base[kPlanThreads];
    __shared__ int s_hist[kPlanBuckets];
    __shared__ unsigned long long s_work;
    const int tid = threadIdx.x;
    grid_dep_launch();
    if (tid == 0) {
        s_err = 0;
        s_nsplit = 0;
        s_nslot = 0;
        s_work = 0;
    }
    s_hist[tid] = 0;
    grid_dep_wait();
    __syncthreads();

    if (tid < 12) hdr[kShHdrKey + tid] = key.w[tid];

    // ---- the offsets, before anything is read through them
    int err = 0;
    for (int i = tid; i < pb.num_groups; i += kPlanThreads) {
        const int a = pb.cu_group[i], b = pb.cu_group[i + 1];
        if (a < 0 || b < a || b > pb.num_seqs || (i == 0 && a != 0) || (i == pb.num_groups - 1 && b != pb.num_seqs))
            err |= BG_DEVSTAT_GROUP;
        const int c = pb.cu_prefix[i], d = pb.cu_prefix[i + 1];
        if (c < 0 || d < c || d > pb.total_prefix || d - c > pb.max_prefix_len || (i == 0 && c != 0) ||
            (i == pb.num_groups - 1 && d != pb.total_prefix))
            err |= BG_DEVSTAT_CU_PROMPT;
    }
    for (int i = tid; i < pb.num_seqs; i += kPlanThreads) {
        const int a = pb.cu_seqlens[i], b = pb.cu_seqlens[i + 1];
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
            hdr[kShHdrEntries] = 0;
            hdr[kShHdrSplits] = 0;
            if (dev_status) atomicOr(dev_status, s_err);
        }
        return;
    }

    // ---- entries in request order, and their total cost in key tiles
    const int per = kShTiles * bt;         // rows of an entry
    const int32_t *cu = pb.cu_seqlens;
    int n_raw = 0;
    unsigned long long work = 0;
    for (int r0 = 0; r0 < pb.num_groups; r0 += kPlanThreads) {
        const int r = r0 + tid;
        int items = 0;
        if (r < pb.num_groups) {
            const int a = pb.cu_group[r], b = pb.cu_group[r + 1];
            items = static_cast<int>(ceil_div(pb.last ? b - a : cu[b] - cu[a], per));
        }
        int total;
        const int excl = block_exclusive(items, s_warp, &total);
        s_base[tid] = excl;
        __syncthreads();
        for (int e = tid; e < total; e += kPlanThreads) {
            int t = 0, end = kPlanThreads;     // the request whose entries include e
            while (end - t > 1) {
                const int mid = (t + end) >> 1;
                if (s_base[mid] <= e) t = mid; else end = mid;
            }
            const int grp = r0 + t, first = (e - s_base[t]) * per;
            const int sa = pb.cu_group[grp], sb = pb.cu_group[grp + 1];
            ShEntry E;
            E.prow0 = pb.cu_prefix[grp];
            E.plen = pb.cu_prefix[grp + 1] - E.prow0;
            const int base = pb.last ? sa : cu[sa];
            const int end_row = pb.last ? sb : cu[sb];
            E.row0 = base + first;
            E.nrows = min(per, end_row - E.row0);
            const int n0 = min(bt, E.nrows);
            if (pb.last) {
                E.s0 = E.row0;
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
            E.tb = 0;
            E.te = static_cast<int>(ceil_div(E.plen, kShKeys) + ceil_div(E.kb1 - E.ka0, kShKeys));
            E.slot = -1;
            raw[n_raw + e] = E;
            work += E.te;
            if (E.te == 0 && dev_status) atomicOr(dev_status, BG_DEVSTAT_EMPTY_ROW);
        }
        n_raw += total;
        __syncthreads();
    }
    if (work) atomicAdd(&s_work, work);
    __syncthreads();

    // ---- pieces: at most `chunk` key tiles each, such that all pieces of split entries fit the
    // slots (an entry of n > chunk tiles gives ceil(n / chunk) < 2 n / chunk pieces, so together
    // fewer than 2 * work * Hkv / chunk <= 2 * kShSplitTarget)
    long long chunk = 0x7fffffff;
    if (slots > 0) {
        chunk = ceil_div(static_cast<long long>(s_work) * pb.Hkv, kShSplitTarget);
        if (chunk < kShSplitMin) chunk = kShSplitMin;
    }
    auto pieces_of = [&](int n) { return n > chunk ? static_cast<int>(ceil_div(n, chunk)) : 1; };
    auto bucket_of = [&](int n, int pieces) { return min(static_cast<int>(ceil_div(n, pieces)), kPlanBuckets - 1); };
    for (int e = tid; e < n_raw; e += kPlanThreads) {
        const int n = raw[e].te;
        if (n == 0) continue;
        const int pieces = pieces_of(n);
        atomicAdd(&s_hist[bucket_of(n, pieces)], pieces);
    }
    __syncthreads();
    int total;
    const int mine = kPlanBuckets - 1 - tid;       // buckets from the costliest down
    const int off = block_exclusive(s_hist[mine], s_warp, &total);
    __syncthreads();
    s_hist[mine] = off;
    __syncthreads();
    for (int e = tid; e < n_raw; e += kPlanThreads) {
        ShEntry E = raw[e];
        const int n = E.te;
        if (n == 0) continue;
        const int pieces = pieces_of(n);
        const int pos = atomicAdd(&s_hist[bucket_of(n, pieces)], pieces);
        int slot0 = -1;
        if (pieces > 1) {
            slot0 = atomicAdd(&s_nslot, pieces);
            splits[atomicAdd(&s_nsplit, 1)] = ShSplit{E.row0, E.nrows, slot0, pieces};
        }
        for (int i = 0; i < pieces; ++i) {
            E.tb = static_cast<int>(static_cast<long long>(n) * i / pieces);
            E.te = static_cast<int>(static_cast<long long>(n) * (i + 1) / pieces);
            E.slot = pieces > 1 ? slot0 + i : -1;
            entries[pos + i] = E;
        }
    }
    __syncthreads();
    if (tid == 0) {
        hdr[kShHdrStatus] = 0;
        hdr[kShHdrEntries] = total;
        hdr[kShHdrSplits] = s_nsplit;
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
template <int D>
struct ShCfg {
    static constexpr int kBox = 128 * 128;                   // 128 rows x one 128-byte column block
    static constexpr int kNB = D / 64;
    static constexpr int kTileBytes = kNB * kBox;            // one Q, K or V tile
    static constexpr int kStages = D == 128 ? 5 : 8;         // K and V tiles in flight
    static constexpr int kOffQ = 0;
    static constexpr int kOffKV = kShTiles * kTileBytes;
    static constexpr int kOffBar = kOffKV + kStages * kTileBytes;
    // q_full[2] q_empty[2] s_full[2] p_full[2] o_full[2] mma_final kv_full[kStages] kv_empty[kStages]
    static constexpr int kNumBars = 11 + 2 * kStages;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
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

// One work item: an entry for one kv head.
struct ShItem {
    ShEntry e;
    int kh, npt;              // kv head; prefix key tiles

    __device__ int rows(int h, int bt) const { return h == 0 ? min(e.nrows, bt) : max(e.nrows - bt, 0); }
    __device__ int ka(int h) const { return h == 0 ? e.ka0 : e.ka1; }
    __device__ int kb(int h) const { return h == 0 ? e.kb0 : e.kb1; }
    // first packed key row of own tile j (j >= npt)
    __device__ int own_base(int j) const { return e.ka0 + (j - npt) * kShKeys; }
    // keys of tile j that any row of the entry sees (1..128)
    __device__ int keys(int j) const
    {
        return min(kShKeys, j < npt ? e.plen - j * kShKeys : e.kb1 - own_base(j));
    }
    // keys of tile j up to the last one that a row of query tile h sees (<= 0: none)
    __device__ int keys_of(int h, int j, int bt) const
    {
        if (rows(h, bt) == 0) return 0;
        if (j < npt) return min(kShKeys, e.plen - j * kShKeys);
        const int base = own_base(j);
        return kb(h) <= ka(h) || base + kShKeys <= ka(h) ? 0 : min(kShKeys, kb(h) - base);
    }
    // number of key tiles of this piece with keys for query tile h
    __device__ int active(int h, int bt) const
    {
        if (rows(h, bt) == 0) return 0;
        const int pre = max(min(e.te, npt) - e.tb, 0);
        if (kb(h) <= ka(h)) return pre;
        const int lo = npt + (ka(h) - e.ka0) / kShKeys;
        const int hi = npt + (kb(h) - e.ka0 + kShKeys - 1) / kShKeys;
        return pre + max(min(e.te, hi) - max(e.tb, lo), 0);
    }
};

// The items of this CTA, round by round in alternating direction (the list is sorted by cost, so
// the CTA that got the costliest item of one round gets the cheapest of the next).  Every role
// walks the same items; the next entry is fetched while the current item runs.
struct ShWalker {
    int round, n_items, hkv;
    const int4 *entries;
    int4 n0, n1, n2;
    int n_kh;

    __device__ int index(int r) const
    {
        const int64_t i = static_cast<int64_t>(r) * gridDim.x + ((r & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        return i < n_items ? static_cast<int>(i) : -1;
    }
    __device__ void fetch()
    {
        const int i = index(round);
        if (i < 0) return;
        const int4 *p = entries + 3 * static_cast<int64_t>(i / hkv);
        n0 = p[0];
        n1 = p[1];
        n2 = p[2];
        n_kh = i % hkv;
    }
    __device__ void first(const ShParams &p, int n)
    {
        round = 0;
        n_items = n;
        hkv = p.Hkv;
        entries = reinterpret_cast<const int4 *>(p.entries);
        fetch();
    }
    __device__ bool next(ShItem &I)
    {
        if (index(round) < 0) return false;
        I.e.prow0 = n0.x; I.e.plen = n0.y; I.e.row0 = n0.z; I.e.nrows = n0.w;
        I.e.ka0 = n1.x; I.e.kb0 = n1.y; I.e.ka1 = n1.z; I.e.kb1 = n1.w;
        I.e.s0 = n2.x; I.e.tb = n2.y; I.e.te = n2.z; I.e.slot = n2.w;
        I.kh = n_kh;
        I.npt = (I.e.plen + kShKeys - 1) / kShKeys;
        ++round;
        fetch();
        return true;
    }
};

// Lane 0 waits, the result is broadcast: the whole warp leaves together.
__device__ __forceinline__ bool sh_warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    int ok = 0;
    if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort) ? 1 : 0;
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
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

// cap * log2(e) * tanh(y) for y = score * scale / cap, from e^(-2|y|).
__device__ __forceinline__ float capped(float s, float cap_in, float cap_log2)
{
    const float y = s * cap_in;
    const float t = ex2(-2.f * 1.44269504088896f * fabsf(y));
    return copysignf(cap_log2 * __fdividef(1.f - t, 1.f + t), y);
}

template <int D, bool CAP>
__global__ void __maxnreg__((ShCfg<D>::kRegsLaunch))
    shared_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_pk,
                       const __grid_constant__ CUtensorMap tm_pv, const ShParams p)
{
    using C = ShCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *q_full = bars, *q_empty = bars + 2, *s_full = bars + 4, *p_full = bars + 6, *o_full = bars + 8;
    uint64_t *mma_final = bars + 10;
    uint64_t *kv_full = bars + 11, *kv_empty = kv_full + C::kStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_launch();

    if (threadIdx.x == 0) {
        for (int h = 0; h < kShTiles; ++h) {
            mbar_init(&q_full[h], 1);
            mbar_init(&q_empty[h], 1);
            mbar_init(&s_full[h], 1);
            mbar_init(&p_full[h], 4);      // one arrive per softmax warp
            mbar_init(&o_full[h], 1);
        }
        mbar_init(mma_final, kShTiles);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], kShTiles);   // one per MMA issuer
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    // Query tiles fill bt * g <= 128 rows; the rows past them stay zero.
    {
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
    bool other;
    const int n_items = plan_ready(p, &other) ? p.hdr[kShHdrEntries] * p.Hkv : 0;
    if (other && blockIdx.x == 0 && threadIdx.x == 0 && p.dev_status) atomicOr(p.dev_status, BG_DEVSTAT_PLAN);

    if (warp < 4) {
        reg_dealloc<C::kRegsLight>();
        if (warp == 0) {
            // ============================================================ K / V producer
            if (lane == 0) {
                const uint64_t pol = l2_policy_evict_last();
                ShWalker w;
                ShItem I;
                w.first(p, n_items);
                uint32_t n = 0;              // K and V tiles issued
                bool ok = true;
                while (ok && w.next(I)) {
                    for (int j = I.e.tb; j < I.e.te && ok; ++j) {
                        const bool pre = j < I.npt;
                        const int row = pre ? I.e.prow0 + j * kShKeys : I.own_base(j);
#pragma unroll
                        for (int kv = 0; kv < 2; ++kv, ++n) {
                            const int st = n % C::kStages;
                            const uint32_t use = n / C::kStages;
                            if (use > 0 && !mbar_wait(&kv_empty[st], (use - 1) & 1, abort_flag)) {
                                ok = false;
                                break;
                            }
                            uint8_t *dst = smem + C::kOffKV + st * C::kTileBytes;
                            const CUtensorMap *tm = kv == 0 ? (pre ? &tm_pk : &tm_k) : (pre ? &tm_pv : &tm_v);
                            mbar_arrive_expect_tx(&kv_full[st], C::kTileBytes);
#pragma unroll
                            for (int b = 0; b < C::kNB; ++b)
                                tma_load_3d(dst + b * C::kBox, tm, &kv_full[st], b * 64, I.kh, row, pol);
                        }
                    }
                }
                for (int st = 0; st < C::kStages; ++st) {   // every copy has landed before the CTA exits
                    const uint32_t uses = n / C::kStages + (st < static_cast<int>(n % C::kStages) ? 1u : 0u);
                    if (uses > 0) mbar_wait_drain(&kv_full[st], (uses - 1) & 1);
                }
            }
            __syncwarp();
        } else if (warp == 2) {
            // ============================================================ Q producer
            if (lane == 0) {
                const uint64_t pol = l2_policy_evict_first();
                ShWalker w;
                ShItem I;
                w.first(p, n_items);
                uint32_t n[kShTiles] = {0, 0};
                const uint32_t bytes = static_cast<uint32_t>(C::kNB * p.bt * p.g * 128);
                bool ok = true;
                while (ok && w.next(I)) {
#pragma unroll
                    for (int h = 0; h < kShTiles; ++h) {
                        if (!ok || I.active(h, p.bt) == 0) continue;
                        if (n[h] > 0 && !mbar_wait(&q_empty[h], (n[h] - 1) & 1, abort_flag)) {
                            ok = false;
                            continue;
                        }
                        mbar_arrive_expect_tx(&q_full[h], bytes);
#pragma unroll
                        for (int b = 0; b < C::kNB; ++b)
                            tma_load_4d(smem + C::kOffQ + h * C::kTileBytes + b * C::kBox, &tm_q, &q_full[h], b * 64, 0,
                                        I.kh, I.e.row0 + h * p.bt, pol);
                        ++n[h];
                    }
                }
                for (int h = 0; h < kShTiles; ++h)
                    if (n[h] > 0) mbar_wait_drain(&q_full[h], (n[h] - 1) & 1);
            }
            __syncwarp();
        } else {
            // ============================================================ MMA issuers (warps 1, 3)
            if (lane == 0) {
                const int h = warp == 1 ? 0 : 1;
                constexpr uint32_t kIdescQK0 = idesc_bf16_f32(128, 0, 0);      // N is set per tile
                constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, 1);
                const uint64_t dq = sdesc_sw128(smem_u32(smem + C::kOffQ + h * C::kTileBytes), 16, 1024);
                const uint64_t dk0 = sdesc_sw128(smem_u32(smem + C::kOffKV), 16, 1024);
                const uint64_t dv0 = sdesc_sw128(smem_u32(smem + C::kOffKV), C::kBox, 1024);
                const uint32_t tS = tmem + C::kColS + kShKeys * h, tO = tmem + C::kColO + D * h;
                ShWalker w;
                ShItem I;
                w.first(p, n_items);
                uint32_t n = 0;              // K and V tiles passed
                uint32_t items = 0, tiles = 0;
                bool ok = true;
                while (ok && w.next(I)) {
                    const int act = I.active(h, p.bt);
                    int done = 0;
                    for (int j = I.e.tb; j < I.e.te; ++j, n += 2) {
                        const int ks = n % C::kStages, vs = (n + 1) % C::kStages;
                        const uint32_t kp = (n / C::kStages) & 1, vp = ((n + 1) / C::kStages) & 1;
                        const int nk = I.keys_of(h, j, p.bt);
                        if (nk <= 0) {       // nothing for this query tile: only pass the stages on
                            if (!mbar_wait(&kv_full[ks], kp, abort_flag)) { ok = false; break; }
                            mbar_arrive(&kv_empty[ks]);
                            if (!mbar_wait(&kv_full[vs], vp, abort_flag)) { ok = false; break; }
                            mbar_arrive(&kv_empty[vs]);
                            continue;
                        }
                        const int steps = (nk + 15) >> 4;       // 16-key steps of P.V; S has 16 * steps columns
                        if (done == 0 && !mbar_wait(&q_full[h], items & 1, abort_flag)) { ok = false; break; }
                        if (!mbar_wait(&kv_full[ks], kp, abort_flag)) { ok = false; break; }
                        // S overwrites the P of the previous tile, which the P.V issued before it reads:
                        // tcgen05.mma operations of one thread execute in issue order.
                        tc_fence_after();
                        const uint64_t dk = dk0 + static_cast<uint64_t>((ks * C::kTileBytes) >> 4);
                        const uint32_t idesc_qk = kIdescQK0 | (static_cast<uint32_t>(2 * steps) << 17);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint64_t off = static_cast<uint64_t>((k >> 2) * (C::kBox >> 4) + (k & 3) * 2);
                            mma_ss(tS, dq + off, dk + off, idesc_qk, k > 0 ? 1u : 0u);
                        }
                        mma_commit(&s_full[h]);
                        mma_commit(&kv_empty[ks]);
                        if (done == act - 1) mma_commit(&q_empty[h]);
                        if (!mbar_wait(&kv_full[vs], vp, abort_flag)) { ok = false; break; }
                        if (!mbar_wait(&p_full[h], tiles & 1, abort_flag)) { ok = false; break; }
                        tc_fence_after();
                        const uint64_t dv = dv0 + static_cast<uint64_t>((vs * C::kTileBytes) >> 4);
                        for (int k = 0; k < steps; ++k)
                            mma_ts(tO, tS + 8 * k, dv + static_cast<uint64_t>(128 * k), kIdescPV,
                                   (done > 0 || k > 0) ? 1u : 0u);
                        mma_commit(&kv_empty[vs]);
                        if (done == act - 1) mma_commit(&o_full[h]);
                        ++done;
                        ++tiles;
                    }
                    if (act > 0) ++items;
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
        const float sl2 = CAP ? 1.f : p.scale_log2;
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        ShWalker w;
        ShItem I;
        w.first(p, n_items);
        uint32_t n = 0, tiles = 0, items = 0;
        bool ok = true;
        while (ok && w.next(I)) {
            const int rows_h = I.rows(h, p.bt);
            const bool live = lr < p.bt && lr < rows_h;
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int act = I.active(h, p.bt);
            const int row = I.e.row0 + h * p.bt + lr;      // packed token, or sample
            // own keys this row sees: [lo, hi)
            int lo = 0, hi = 0;
            if (act > 0) {
                if (p.last) {
                    if (live) {
                        lo = p.cu_seqlens[row];
                        hi = p.cu_seqlens[row + 1];
                    }
                } else {
                    // the last sample start that is not behind the row; 32 sample starts at a time
                    const int last_row = I.e.row0 + I.e.nrows - 1;
                    lo = I.e.ka0;
                    for (int s = I.e.s0 + 1;; s += 32) {
                        const int start = p.cu_seqlens[min(s + lane, p.num_seqs)];
                        const unsigned in = __ballot_sync(0xffffffffu, start <= last_row && s + lane < p.num_seqs);
                        for (int i = 0; i < 32 && ((in >> i) & 1u); ++i) {
                            const int b = __shfl_sync(0xffffffffu, start, i);
                            if (b <= row) lo = b;
                        }
                        if (in != 0xffffffffu) break;
                    }
                    hi = row + 1;
                    if (!live) hi = lo;
                }
            }
            float m = -INFINITY;       // running maximum, base-2 units
            float l = 0.f;             // running sum of 2^(x - m)
            bool seen = false;         // this row has a key in one of the tiles
            float fix = 0.f;           // what rounding the tiles' largest weights to bf16 adds to l
            int done = 0;
            for (int j = I.e.tb; j < I.e.te; ++j, n += 2) {
                const int nk = I.keys_of(h, j, p.bt);
                if (nk <= 0) continue;
                const bool pre = j < I.npt;
                const int base = pre ? 0 : I.own_base(j);
                // this row's columns of the tile: [c0, c1)
                const int c0 = pre ? 0 : min(max(lo - base, 0), kShKeys);
                const int c1 = pre ? nk : min(max(hi - base, 0), nk);
                if (!sh_warp_wait(&s_full[h], tiles & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                // Keys behind the last one that any row of the entry sees (a later token, another
                // request's rows) have weight 0, but 0 * Inf is NaN: their V rows become zeros.
                const int nkeys = I.keys(j);
                if (((nk + 15) & ~15) > nkeys) {
                    const int vs = (n + 1) % C::kStages;
                    if (!sh_warp_wait(&kv_full[vs], ((n + 1) / C::kStages) & 1, abort_flag)) { ok = false; break; }
                    uint8_t *vt = smem + C::kOffKV + vs * C::kTileBytes;
                    const int chunks = (((nkeys + 15) & ~15) - nkeys) * 8;      // 16-byte chunks per column block
                    for (int i = trow; i < chunks * C::kNB; i += 128) {
                        const int b = i / chunks, c = i - b * chunks;
                        *reinterpret_cast<uint4 *>(vt + b * C::kBox + nkeys * 128 + c * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                if (warp_live) {
                    const bool any = __any_sync(0xffffffffu, live && c1 > c0);
                    if (!any) {
                        // no row of this warp has a key in the tile: P = 0
                        uint32_t zr[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) zr[i] = 0u;
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_st16(tS + 16 * c, zr);
                    } else {
                        const bool masked = __any_sync(0xffffffffu, live && (c0 > 0 || c1 < (nk > 64 ? 128 : 64)));
                        seen = seen || c1 > c0;
                        auto tile = [&](auto ncols) {
                            constexpr int NC = decltype(ncols)::value;
                            float s[NC];
#pragma unroll
                            for (int c = 0; c < NC / 64; ++c) tmem_ld64(tS + 64 * c, s + 64 * c);
                            if constexpr (CAP) {
#pragma unroll
                                for (int c = 0; c < NC; ++c) s[c] = capped(s[c], p.cap_in, p.cap_log2);
                            }
                            if (masked) {
                                const unsigned width = static_cast<unsigned>(max(c1 - c0, 0));
#pragma unroll
                                for (int c = 0; c < NC; ++c)
                                    if (static_cast<unsigned>(c - c0) >= width) s[c] = -INFINITY;
                            }
                            float mq[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) mq[q] = fmaxf(s[(NC / 4) * q], s[(NC / 4) * q + 1]);
#pragma unroll
                            for (int c = 2; c < NC / 4; c += 2)
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    mq[q] = fmax3f(mq[q], s[(NC / 4) * q + c], s[(NC / 4) * q + c + 1]);
                            const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
                            const float m_new = fmaxf(m, mx * sl2);
                            if (done == 0) {
                                m = m_new;
                            } else if (__any_sync(0xffffffffu, m_new > m + 8.f)) {
                                // O holds the earlier tiles, all complete (the commit behind this S covers
                                // every MMA issued before it); rescaled only when the maximum grows by > 2^8
                                const float alpha = m == -INFINITY ? 0.f : ex2(m - m_new);
                                m = m_new;
                                l *= alpha;
                                fix *= alpha;
#pragma unroll
                                for (int c = 0; c < D / 32; ++c) {
                                    float o[32];
                                    tmem_ld32(tO + 32 * c, o);
#pragma unroll
                                    for (int i = 0; i < 32; ++i) o[i] *= alpha;
                                    tmem_st32f(tO + 32 * c, o);
                                }
                            }
                            const float mu = m == -INFINITY ? 0.f : m;      // no key yet: p = 0, not NaN
                            const float2 negm = make_float2(-mu, -mu), sl2x2 = make_float2(sl2, sl2);
                            float2 rs[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) rs[q] = make_float2(0.f, 0.f);
                            // P.V multiplies weights rounded to bf16.  The rounding of the tile's largest
                            // weight enters the sum that O is divided by, which makes the dominant term
                            // exact; the log-sum-exp keeps the unrounded sum.
                            const float pmax = ex2(ffma2(make_float2(mx, mx), sl2x2, negm).x);
                            fix += __uint_as_float(pack_bf16x2(pmax, 0.f) << 16) - pmax;
#pragma unroll
                            for (int c = 0; c < NC / 32; ++c) {
                                uint32_t pk[16];
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const float2 x =
                                        ffma2(make_float2(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]), sl2x2, negm);
                                    const float2 e = make_float2(ex2(x.x), ex2(x.y));
                                    rs[i & 3] = fadd2(rs[i & 3], e);
                                    pk[i] = pack_bf16x2(e.x, e.y);
                                }
                                tmem_st16(tS + 16 * c, pk);
                            }
                            const float2 r01 = fadd2(rs[0], rs[1]), r23 = fadd2(rs[2], rs[3]);
                            l += (r01.x + r23.x) + (r01.y + r23.y);
                        };
                        if (nk > 64)
                            tile(std::integral_constant<int, 128>{});
                        else
                            tile(std::integral_constant<int, 64>{});
                    }
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[h]);
                ++done;
                ++tiles;
            }
            if (!ok) break;
            // ------------------------------------------------------------ output of the item
            if (act > 0) {
                if (!sh_warp_wait(&o_full[h], items & 1, abort_flag)) { ok = false; break; }
                tc_fence_after();
                ++items;
            }
            const int head = I.kh * p.g + hh;
            const bool empty = !seen;              // this row has no key (in this piece)
            if (I.e.slot >= 0) {
                if (warp_live) {
                    const int64_t prow = (static_cast<int64_t>(I.e.slot) * p.Hkv + I.kh) * (kShTiles * kShRows) +
                                         h * kShRows + trow;
                    // -inf marks a row that was not written; a sum of 0 over keys (scores of -inf) is NaN
                    if (live) p.part_l[prow] = empty ? -INFINITY : l == 0.f ? NAN : m + __log2f(l);
                    if (live) p.part_l[p.part_fix + prow] = empty ? 0.f : fix / l;
                    if (act > 0) {
                        const float inv = 1.f / l;
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            float o[32];
                            tmem_ld32(tO + 32 * c, o);
                            if (live && !empty) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    uint32_t wv[8];
#pragma unroll
                                    for (int e = 0; e < 8; ++e) wv[e] = __float_as_uint(o[8 * i + e] * inv);
                                    st_global_32b(p.part_o + prow * D + 32 * c + 8 * i, wv);
                                }
                            }
                        }
                    }
                }
            } else if (warp_live) {
                if (live && empty && p.dev_status) atomicOr(p.dev_status, BG_DEVSTAT_EMPTY_ROW);
                if (act > 0) {
                    const float inv = 1.f / (l + fix);
                    const int64_t orow = static_cast<int64_t>(row) * p.Hq + head;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        tmem_ld32(tO + 32 * c, o);
                        if (live && !empty) {
                            uint32_t wv[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) wv[i] = pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
                            st_out_32b(p.out + orow * D + 32 * c, wv, wide);
                            st_out_32b(p.out + orow * D + 32 * c + 16, wv + 8, wide);
                        }
                    }
                    if (p.lse && live && !empty) p.lse[orow] = (m + __log2f(l)) * 0.69314718055994530942f;
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
    if (threadIdx.x == 0 && *abort_flag && p.dev_status) atomicOr(p.dev_status, BG_DEVSTAT_TIMEOUT);
}

// ------------------------------------------------------------------------------------ join
// out = sum_i 2^(L_i - L) O_i / (1 + sum_i 2^(L_i - L) fix_i) with L = log2 sum_i 2^(L_i): the
// pieces' own normalised outputs, in piece order.  One warp per row.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) shared_join_kernel(const ShParams p)
{
    grid_dep_launch();
    grid_dep_wait();
    bool other;
    if (!plan_ready(p, &other)) return;
    const int n_split = p.hdr[kShHdrSplits];
    const int lane = threadIdx.x & 31;
    const int64_t total = static_cast<int64_t>(n_split) * p.Hkv * kShTiles * kShRows;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kJoinThreads / 32);
    constexpr int E = D / 32;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5); i < total; i += stride) {
        const int r = static_cast<int>(i % (kShTiles * kShRows));
        const int64_t q = i / (kShTiles * kShRows);
        const int kh = static_cast<int>(q % p.Hkv);
        const ShSplit S = p.splits[q / p.Hkv];
        const int h = r / kShRows, trow = r - h * kShRows;
        const int lr = trow / p.g, hh = trow - lr * p.g;
        if (lr >= p.bt || h * p.bt + lr >= S.nrows) continue;
        auto prow = [&](int piece) {
            return (static_cast<int64_t>(S.slot0 + piece) * p.Hkv + kh) * (kShTiles * kShRows) + r;
        };
        float mx = -INFINITY;
        bool nan = false;
        for (int t = lane; t < S.pieces; t += 32) {
            const float lt = p.part_l[prow(t)];
            mx = fmaxf(mx, lt);
            nan = nan || lt != lt;
        }
        nan = __any_sync(0xffffffffu, nan);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (mx == -INFINITY && !nan) {          // no piece has a key for this row
            if (lane == 0 && p.dev_status) atomicOr(p.dev_status, BG_DEVSTAT_EMPTY_ROW);
            continue;
        }
        float sum = 0.f, fix = 0.f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        for (int t = 0; t < S.pieces; ++t) {
            const float lt = p.part_l[prow(t)];
            if (lt == -INFINITY) continue;          // its row of part_o was not written
            const float wt = ex2(lt - mx);
            sum += wt;
            fix = fmaf(wt, p.part_l[p.part_fix + prow(t)], fix);
            float o[E];
            if constexpr (E == 4)
                *reinterpret_cast<float4 *>(o) = *reinterpret_cast<const float4 *>(p.part_o + prow(t) * D + lane * E);
            else
                *reinterpret_cast<float2 *>(o) = *reinterpret_cast<const float2 *>(p.part_o + prow(t) * D + lane * E);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(wt, o[e], acc[e]);
        }
        const float inv = 1.f / (sum + fix);
        const int64_t orow = (static_cast<int64_t>(S.row0) + h * p.bt + lr) * p.Hq + kh * p.g + hh;
        uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + orow * D + lane * E);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) dst[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
        if (p.lse && lane == 0) p.lse[orow] = (mx + __log2f(sum)) * 0.69314718055994530942f;
    }
}

template <int D, bool CAP>
cudaError_t launch_one(const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                       const CUtensorMap &tm_pk, const CUtensorMap &tm_pv, const ShParams &p, int grid, bool join,
                       cudaStream_t stream)
{
    using C = ShCfg<D>;
    auto kern = shared_attn_kernel<D, CAP>;
    static std::atomic<uint64_t> smem_done{0}, split_done{0};
    cudaError_t e = ensure_smem_attribute(kern, C::kSmemBytes, smem_done);
    if (e != cudaSuccess) return e;
    e = check_register_split(kern, C::kThreads, C::kSplitRegs, split_done);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, dim3(grid), dim3(C::kThreads), C::kSmemBytes, stream, tm_q, tm_k, tm_v, tm_pk, tm_pv, p);
    if (e != cudaSuccess || !join) return e;
    return launch_dependent(shared_join_kernel<D>, dim3(2 * grid), dim3(kJoinThreads), 0, stream, p);
}

}  // namespace

ShLayout shared_layout(const ShProblem &pb)
{
    ShLayout L;
    const int bt = kShRows / (pb.Hq / pb.Hkv);
    const int64_t rows = pb.last ? pb.num_seqs : pb.total_tokens;
    L.max_entries = rows / (kShTiles * bt) + pb.num_groups + 1;
    // most key tiles of an entry: its prefix, and the own keys of the rows it holds (prefill: one
    // sample's start to the entry's last row; last token: whole samples)
    int64_t own = pb.last ? static_cast<int64_t>(kShTiles) * bt * pb.max_seqlen : pb.max_seqlen + kShTiles * bt;
    if (own > pb.total_tokens) own = pb.total_tokens;
    const int64_t tiles = ceil_div(pb.max_prefix_len, kShKeys) + ceil_div(own, kShKeys);
    L.slots = 0;
    if (tiles > kShSplitMin) {
        // fewer than 2 * work / kShSplitMin pieces, and never more than the plan makes
        L.slots = kShSlots;
        if (L.max_entries * pb.Hkv < kShSlots) {
            const int64_t most = 2 * ceil_div(L.max_entries * pb.Hkv * tiles, kShSplitMin);
            if (most < L.slots) L.slots = most;
        }
    }
    auto al = [](size_t b) { return (b + 255) & ~size_t(255); };
    L.entries = 256;
    L.raw = L.entries + al((L.max_entries + kShSlots) * sizeof(ShEntry));
    L.splits = L.raw + al(L.max_entries * sizeof(ShEntry));
    L.part_l = L.splits + al(kShSlots * sizeof(ShSplit));
    L.part_o = L.part_l + al(static_cast<size_t>(L.slots) * kShTiles * kShRows * 2 * sizeof(float));
    L.total = L.part_o + al(static_cast<size_t>(L.slots) * kShTiles * kShRows * pb.head_dim * sizeof(float));
    return L;
}

ShKey shared_key(const ShProblem &pb)
{
    return ShKey{{pb.last, pb.num_seqs, pb.total_tokens, pb.max_seqlen, pb.num_groups, pb.total_prefix,
                  pb.max_prefix_len, pb.Hq, pb.Hkv, pb.head_dim, 0x5348, 1}};
}

cudaError_t launch_shared_plan(const ShProblem &pb, const ShLayout &lay, void *workspace, int32_t *dev_status,
                               cudaStream_t stream)
{
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    return launch_dependent(shared_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, pb, shared_key(pb),
                            kShRows / (pb.Hq / pb.Hkv), reinterpret_cast<int32_t *>(ws),
                            reinterpret_cast<ShEntry *>(ws + lay.entries), reinterpret_cast<ShEntry *>(ws + lay.raw),
                            reinterpret_cast<ShSplit *>(ws + lay.splits), lay.slots, dev_status);
}

cudaError_t launch_shared_attn(int head_dim, bool is_capped, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                               const CUtensorMap &tm_v, const CUtensorMap &tm_pk, const CUtensorMap &tm_pv,
                               const ShParams &p, int grid, bool join, cudaStream_t stream)
{
    if (head_dim == 128)
        return is_capped ? launch_one<128, true>(tm_q, tm_k, tm_v, tm_pk, tm_pv, p, grid, join, stream)
                         : launch_one<128, false>(tm_q, tm_k, tm_v, tm_pk, tm_pv, p, grid, join, stream);
    if (head_dim == 64)
        return is_capped ? launch_one<64, true>(tm_q, tm_k, tm_v, tm_pk, tm_pv, p, grid, join, stream)
                         : launch_one<64, false>(tm_q, tm_k, tm_v, tm_pk, tm_pv, p, grid, join, stream);
    return cudaErrorInvalidValue;
}

}  // namespace bg
