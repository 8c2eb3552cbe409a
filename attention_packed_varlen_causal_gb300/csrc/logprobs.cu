// logprobs.cu -- log-probability of a given token, entropy and the best alternatives of rows of
// logits.
//
// "SLM 生成式高并发推理引擎：延迟约束下的有效吞吐优化", section 1.1: a Prefill-Only request is
// answered from the next-token logits at the last valid position (softmax, Top-K).  With m the
// largest logit of a row, d_v = x_v - m and Z = sum_v e^(d_v):
//     logprob(t) = d_t - ln Z
//     entropy    = ln Z - sum_v e^(d_v) d_v / Z          (every term of the sum has one sign)
//     top        = the K largest logits, equal ones by the smaller index, as (v, d_v - ln Z)
// Only the row's bytes bound it, so everything comes out of one pass over them, by a team of 4 or 8 warps
// or of the 16 of a CTA (with fewer rows than CTAs, a cluster of up to 8 CTAs):
//   pass    every lane keeps a running maximum with Z and the entropy's sum relative to it, and in
//           shared memory the maximum of each batch of 64 bytes it read, rounded up to bf16; bulk
//           copies bring the batches into shared memory, over the rows' ends;
//   bound   the 32 / W largest lane maxima of each warp are 32 >= K distinct logits, so the K-th
//           largest of them bounds the row's K-th best from below;
//   gather  only the batches whose maximum reaches the bound are read again (from L2), eight at a
//           time; the few logits at or above it go to a list in shared memory, where each one's
//           rank is the number of larger (logit, index) pairs (of a long list, the K best are
//           found bit by bit first).
// The bound is weak where the largest logits lie in few lanes: a label set of neighbouring tokens with
// all others banned gives few finite lane maxima.  If more logits reach it than the list holds, the
// list's own K-th largest becomes the bound and the logits above that are gathered; with the bound at
// -inf it is the logits above it from the start.  Fewer than K above the bound are followed by the
// first tokens that equal it.
// Two CTAs of 16 warps per SM keep 64 KB of copies in flight; what is left to the bound is issue slots
// (about 9 instructions per logit and lane, the K best among them): 8192 rows of 65,536 bf16 logits take
// 196 us for the 20 best, 5.5 TB/s; 480 rows of 50,001 fp32 logits with an eighth of them banned 21.8 us,
// 4.4 TB/s, and 25.6 with all but 16 neighbours banned.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

#include "bg_internal.h"
#include "bg_ptx.cuh"

namespace cg = cooperative_groups;

namespace bg {
namespace {

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpLoads = 4;              // 16-byte loads per lane and batch
constexpr int kLpStages = 2;             // batches in flight per team (32 KB each over a CTA's teams)
constexpr int kLpSlots = 16;             // stored batch maxima per lane (of one or more batches each)
constexpr int kLpCap = 144;              // gathered logits per warp of the team
constexpr int kLpCount = 128;            // lists up to this long are ranked by counting
constexpr int kLpMaxCluster = 8;
static_assert(BG_MAX_TOP <= 32, "at least K lane maxima");
static_assert(kLpSlots == 16, "a lane's stored maxima are two vectors, one mask");

// A slice's results: what the warps of a team, and the CTAs of a cluster, tell each other.
struct LpPart {
    float m, z, s;        // maximum, sum of 2^t, sum of 2^t t
    float bound;          // at least K logits of the slice reach it (-inf: no such bound)
};

struct LpShared {
    uint4 data[kLpStages * kLpThreads * kLpLoads];      // per team: its stages
    uint64_t full[kLpWarps][kLpStages], empty[kLpWarps][kLpStages];
    int abort;
    uint4 slot[kLpWarps][32][kLpSlots / 8];      // bf16 [kLpSlots] per lane
    int pick[kLpWarps][8];                       // batches that a warp reads again
    unsigned long long key[kLpWarps * kLpCap];   // order-preserving logit << 32 | ~index; per team
    LpPart part[kLpMaxCluster];                  // first CTA: one per CTA
    LpPart all[kLpWarps];                        // per team
    LpPart warp[kLpWarps];                       // (bound: unused)
    uint32_t top[kLpWarps][32];                  // a team's 32 lane maxima, at its first warp
    unsigned long long few[kLpWarps / 4][32];    // per team: the K best of a long list
    int n[2][kLpWarps];                          // per team: logits gathered in this sweep, in the next
    int total[2];                                // ... by the CTAs of the cluster
    int joined[2];                               // first CTA: ... that have a place in its list
};

__device__ __forceinline__ uint32_t order_key(float f)
{
    const uint32_t u = __float_as_uint(f + 0.f);          // -0 and 0 are equal
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
// The next number above f (of -inf, the lowest finite one).
__device__ __forceinline__ float above(float f) { return order_value(order_key(f) + 1u); }
__device__ __forceinline__ unsigned long long pair_key(float x, int v)
{
    return static_cast<unsigned long long>(order_key(x)) << 32 | static_cast<uint32_t>(~v);
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

constexpr float kLog2e = 1.44269504088896f;
// e^d is 0 from here down; differences are held above it, so that 0 meets no infinite factor
// (banned tokens at -inf, or at the type's lowest value).
constexpr float kLpFar = -10000.f;

// The largest logit so far, and with t = (x - m) log2(e) sum 2^t and sum 2^t t.
struct Running {
    float m = -INFINITY, z = 0.f, s = 0.f;

    // moves the reference to m_new >= m
    __device__ void rebase(float m_new)
    {
        if (m != -INFINITY) {
            const float t = max_nan(m - m_new, kLpFar) * kLog2e, f = ex2(t);
            s = f * fmaf(z, t, s);
            z *= f;
        }
        m = m_new;
    }
    // joins sums relative to om (-inf: sums of 0, or of NaN)
    __device__ void join(float om, float oz, float os)
    {
        if (om > m) {
            const float tm = m, tz = z, ts = s;
            m = om; z = oz; s = os;
            om = tm; oz = tz; os = ts;
        }
        const float t = om == -INFINITY ? 0.f : max_nan(om - m, kLpFar) * kLog2e, f = ex2(t);
        s += f * fmaf(oz, t, os);
        z += f * oz;
    }
};

template <typename T>
struct LpVec;
template <>
struct LpVec<float> {
    static constexpr int N = 4;
    static __device__ void unpack(const uint4 &w, float *x)
    {
        x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
    }
    static __device__ float load(const float *p) { return *p; }
    static __device__ float largest(const uint4 *w)      // of kLpLoads vectors
    {
        float h[kLpLoads];
#pragma unroll
        for (int i = 0; i < kLpLoads; ++i) {
            float x[4];
            unpack(w[i], x);
            h[i] = fmaxf(fmax3f(x[0], x[1], x[2]), x[3]);
        }
        return fmaxf(fmax3f(h[0], h[1], h[2]), h[3]);
    }
    static __device__ uint4 nothing() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
};
template <>
struct LpVec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ void unpack(const uint4 &w, float *x)
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ float load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    static __device__ float largest(const uint4 *w)
    {
        auto pair = [](uint32_t u) { return *reinterpret_cast<__nv_bfloat162 *>(&u); };
        __nv_bfloat162 h[kLpLoads];
#pragma unroll
        for (int i = 0; i < kLpLoads; ++i)
            h[i] = __hmax2(__hmax2(pair(w[i].x), pair(w[i].y)), __hmax2(pair(w[i].z), pair(w[i].w)));
        const float2 a = __bfloat1622float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
        return fmaxf(a.x, a.y);
    }
    static __device__ uint4 nothing() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
};

struct LpParams {
    const void *logits;
    int64_t stride;
    int32_t N, V, K;
    const int32_t *tokens;
    float *logprob, *entropy;
    int32_t *top_token;
    float *top_logprob;
    int32_t *dev_status;
    int32_t stalled;      // (self-test) rows from this one on are never loaded
};

// `bytes` (a multiple of 16, from a 16-byte boundary) into shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Bounded wait (as bg::mbar_wait) that lets the barrier unit suspend the warp for up to 20 us at a
// time: the polls of waiting warps would take issue slots from the summing ones.
__device__ __forceinline__ bool lp_wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
            : "memory");
        if (ok) return true;
        if (*abort) return false;
        if ((it & 63u) != 0) continue;
        const uint64_t now = globaltimer_ns();
        if (it == 0) t0 = now;
        if (now - t0 > kWaitTimeoutNs) {
            *abort = 1;
            return false;
        }
    }
}

// The warp's 32 keys, largest first.
__device__ __forceinline__ uint32_t sort_desc(uint32_t k, int lane)
{
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int o = size >> 1; o > 0; o >>= 1) {
            const uint32_t u = __shfl_xor_sync(0xffffffffu, k, o);
            const bool up = ((lane & size) != 0) == ((lane & o) != 0);      // this lane keeps the larger
            k = up ? max(k, u) : min(k, u);
        }
    return k;
}

// A batch maximum as it is stored: not below x (exact for bf16 logits; -inf stays).
__device__ __forceinline__ __nv_bfloat16 slot_value(float x)
{
    const uint32_t u = __float_as_uint(x);
    if ((u & 0xffffu) == 0) return __float2bfloat16_rn(x);
    return __float2bfloat16_ru(x);
}

// STALL: the self-test of a wait that runs out.
template <typename T, int W, bool STALL>
__global__ void __launch_bounds__(kLpThreads, 2) logprobs_kernel(const LpParams p)
{
    extern __shared__ __align__(16) uint8_t lp_smem[];
    LpShared &sh = *reinterpret_cast<LpShared *>(lp_smem);
    using Vec = LpVec<T>;
    constexpr int VN = Vec::N;
    constexpr int kLanes = W * 32;                       // of a team
    constexpr int kBatch = kLanes * kLpLoads;            // vectors of a team's batch
    constexpr int kTeams = kLpWarps / W;
    constexpr int kCap = kLpCap * W;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = W == kLpWarps ? static_cast<int>(cluster.num_blocks()) : 1;      // CTAs per row
    const int c = C == 1 ? 0 : static_cast<int>(cluster.block_rank());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int team = warp / W, tw = warp - team * W;     // team of the CTA, warp of the team
    const int tid = tw * 32 + lane;                      // lane of the team
    unsigned long long *list = sh.key + team * kCap;
    auto team_sync = [&]() {
        if constexpr (W == kLpWarps) __syncthreads();
        else named_bar_sync(1 + team, kLanes);
    };
    grid_dep_launch();
    uint64_t *full = sh.full[team], *empty = sh.empty[team];
    volatile int *abort = &sh.abort;
    if (tid == 0) {
        for (int i = 0; i < kLpStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], W);
        }
        fence_barrier_init();
    }
    if (threadIdx.x == 0) sh.abort = 0;
    // every CTA of the cluster has started before one writes into another's shared memory
    if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    grid_dep_wait();
    __syncthreads();
    uint4 *data = sh.data + team * kLpStages * kBatch;

    // consecutive rows in different CTAs, so that a few rows spread over the SMs; a cluster has one row
    const int64_t rows_at_once = static_cast<int64_t>(gridDim.x / C) * kTeams;
    const int64_t row0 = static_cast<int64_t>(team) * (gridDim.x / C) + blockIdx.x / C;
    // A row in memory: [0, head) before the first 16-byte boundary, whole vectors, [tail, V) behind
    // them; of the vectors, this CTA's [v0, v1).
    struct Slice {
        const T *x;
        int head, tail, v0, v1;
    };
    auto slice_of = [&](int64_t row) {
        Slice S;
        S.x = static_cast<const T *>(p.logits) + row * p.stride;
        S.head = min(static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(S.x) & 15u)) & 15u) / sizeof(T)), p.V);
        const int nv = (p.V - S.head) / VN;
        S.tail = S.head + nv * VN;
        S.v0 = C == 1 ? 0 : static_cast<int>(static_cast<int64_t>(nv) * c / C);
        S.v1 = C == 1 ? nv : static_cast<int>(static_cast<int64_t>(nv) * (c + 1) / C);
        return S;
    };
    // The first lane of the team issues the copies, kLpStages - 1 batches ahead of the one that is
    // summed, over the rows' ends.
    int64_t load_row = row0 - rows_at_once;
    const T *load_x = nullptr;
    int load_v = 0, load_end = 0;
    uint32_t loads = 0;                                  // batches issued
    auto issue = [&]() {
        while (load_v >= load_end) {                     // the next row that has vectors
            load_row += rows_at_once;
            if (load_row >= p.N || (STALL && load_row >= p.stalled)) {
                load_row = p.N;
                return;
            }
            const Slice L = slice_of(load_row);
            load_x = L.x + L.head;
            load_v = L.v0;
            load_end = L.v1;
        }
        const uint32_t st = loads % kLpStages, use = loads / kLpStages;
        if (use > 0 && !lp_wait(&empty[st], (use - 1) & 1, abort)) {
            load_row = p.N;                              // give up: nothing more is issued
            load_v = load_end = 0;
            return;
        }
        const int n = min(kBatch, load_end - load_v);
        mbar_arrive_expect_tx(&full[st], n * 16);
        bulk_load(data + st * kBatch, reinterpret_cast<const uint4 *>(load_x) + load_v, n * 16, &full[st]);
        load_v += n;
        ++loads;
    };
    if (tid == 0)
        for (int i = 0; i < kLpStages - 1; ++i) issue();
    uint32_t sums = 0;                                   // batches summed
    bool lost = false;                                   // this warp gave a wait up: its rows from then on are NaN

    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int64_t row = row0; row < p.N; row += rows_at_once) {
        const Slice S = slice_of(row);
        const T *x = S.x;
        const int head = S.head, tail = S.tail, v0 = S.v0, v1 = S.v1;
        const int nb = (v1 - v0 + kBatch - 1) / kBatch;
        const int per_slot = (nb + kLpSlots - 1) / kLpSlots;
        // the loose logits: the head belongs to the first CTA of the row, the tail to the last
        const int n_head = c == 0 ? head : 0, n_tail = c == C - 1 ? p.V - tail : 0;
        const int loose = lane < n_head ? lane : lane >= 16 && lane - 16 < n_tail ? tail + lane - 16 : -1;
        const float loose_x = tw == 0 && loose >= 0 ? Vec::load(x + loose) : -INFINITY;
        if (tid == 0) sh.n[0][team] = 0;
        if (C > 1 && tid == 0) sh.total[0] = sh.joined[0] = 0;
        // the given token's logit, loaded ahead of its use
        int token = -1;
        float token_x = 0.f;
        if (c == 0 && tid == 0 && p.tokens) {
            token = p.tokens[row];
            if (token >= 0 && token < p.V) token_x = Vec::load(x + token);
        }

        Running a;
        float best = -INFINITY;           // this lane's largest logit
        int in_slot = 0, slot = 0;
        __nv_bfloat16 *slots = reinterpret_cast<__nv_bfloat16 *>(sh.slot[warp][lane]);
        float slot_max = -INFINITY;
        bool far = false;                                 // (of the warp) see below
#pragma unroll 1
        for (int b = 0; b < nb && !lost; ++b, ++sums) {
            if (tid == 0) issue();
            __syncwarp();
            const uint32_t st = sums % kLpStages;
            lost = !__all_sync(0xffffffffu, lp_wait(&full[st], (sums / kLpStages) & 1, abort));
            if (lost) break;
            const int left = v1 - v0 - b * kBatch;
            uint4 g[kLpLoads];
#pragma unroll
            for (int i = 0; i < kLpLoads; ++i) g[i] = data[st * kBatch + i * kLanes + tid];
            if (left < kBatch) {                          // past the slice's end -inf, which adds nothing
#pragma unroll
                for (int i = 0; i < kLpLoads; ++i)
                    if (i * kLanes + tid >= left) g[i] = Vec::nothing();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
            const float bm = Vec::largest(g);
            if (bm > a.m) a.rebase(bm);
            slot_max = fmaxf(slot_max, bm);
            const float2 c2 = make_float2(kLog2e, kLog2e);
            const float nm = a.m == -INFINITY ? 0.f : -a.m;      // -inf only so far: no reference
            const float2 nm2 = make_float2(nm, nm);
            float2 z2 = make_float2(0.f, 0.f), s2 = make_float2(0.f, 0.f);
            if (!far) {
#pragma unroll
                for (int i = 0; i < kLpLoads; ++i) {
                    float f[VN];
                    Vec::unpack(g[i], f);
#pragma unroll
                    for (int e = 0; e < VN; e += 2) {
                        const float2 t = fmul2(fadd2(make_float2(f[e], f[e + 1]), nm2), c2);
                        const float2 q = make_float2(ex2(t.x), ex2(t.y));
                        z2 = fadd2(z2, q);
                        s2 = ffma2(q, t, s2);
                    }
                }
                // NaN: 0 * inf of a logit far below the maximum (banned, or past the end), or a NaN logit.
                // Then this batch, and the row's others at once, with the differences held.
                far = __any_sync(0xffffffffu, s2.x + s2.y != s2.x + s2.y);
            }
            if (far) {
                z2 = s2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kLpLoads; ++i) {
                    float f[VN];
                    Vec::unpack(g[i], f);
#pragma unroll
                    for (int e = 0; e < VN; e += 2) {
                        float2 d = fadd2(make_float2(f[e], f[e + 1]), nm2);
                        d = make_float2(max_nan(d.x, kLpFar), max_nan(d.y, kLpFar));
                        const float2 t = fmul2(d, c2);
                        const float2 q = make_float2(ex2(t.x), ex2(t.y));
                        z2 = fadd2(z2, q);
                        s2 = ffma2(q, t, s2);
                    }
                }
            }
            a.z += z2.x + z2.y;
            a.s += s2.x + s2.y;
            if (++in_slot == per_slot || b == nb - 1) {
                slots[slot++] = slot_value(slot_max);
                best = fmaxf(best, slot_max);
                slot_max = -INFINITY;
                in_slot = 0;
            }
        }
        if (tw == 0 && loose >= 0) {
            if (loose_x > a.m) a.rebase(loose_x);
            const float t = max_nan(loose_x + (a.m == -INFINITY ? 0.f : -a.m), kLpFar) * kLog2e, q = ex2(t);
            a.z += q;
            a.s = fmaf(q, t, a.s);
            best = fmaxf(best, loose_x);
        }

        // ---- the warp's sums and lane maxima, the team's, the row's
        if (lost) a.z = NAN;
        uint32_t mine = 0;
        if (p.K > 0) {
            mine = sort_desc(order_key(best), lane);
            if (lane < 32 / W) sh.top[team * W][tw * (32 / W) + lane] = mine;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, a.m, o), oz = __shfl_xor_sync(0xffffffffu, a.z, o),
                        os = __shfl_xor_sync(0xffffffffu, a.s, o);
            a.join(om, oz, os);
        }
        LpPart A{a.m, a.z, a.s, -INFINITY};
        if (lane == 0) sh.warp[warp] = A;
        team_sync();
        if (tw == 0) {
            const LpPart q = sh.warp[team * W + (lane & (W - 1))];
            Running u;
            u.m = q.m; u.z = q.z; u.s = q.s;
#pragma unroll
            for (int o = W / 2; o > 0; o >>= 1) {
                const float om = __shfl_xor_sync(0xffffffffu, u.m, o), oz = __shfl_xor_sync(0xffffffffu, u.z, o),
                            os = __shfl_xor_sync(0xffffffffu, u.s, o);
                u.join(om, oz, os);
            }
            float bd = -INFINITY;
            if (p.K > 0)
                bd = order_value(__shfl_sync(0xffffffffu, sort_desc(sh.top[team * W][lane], lane), p.K - 1));
            const LpPart part{u.m, u.z, u.s, bd};
            if (C == 1 && lane == 0) sh.all[team] = part;
            if (C > 1 && lane < C) cluster.map_shared_rank(&sh, lane)->part[c] = part;
        }
        if (C > 1) {
            cluster.sync();
            if (warp == 0) {
                // every CTA joins all slices' sums in the same order
                const LpPart q = lane < C ? sh.part[lane] : LpPart{-INFINITY, 0.f, 0.f, -INFINITY};
                Running u;
                float bd = -INFINITY;
                for (int i = 0; i < C; ++i) {
                    u.join(__shfl_sync(0xffffffffu, q.m, i), __shfl_sync(0xffffffffu, q.z, i),
                           __shfl_sync(0xffffffffu, q.s, i));
                    bd = fmaxf(bd, __shfl_sync(0xffffffffu, q.bound, i));
                }
                if (lane == 0) sh.all[0] = LpPart{u.m, u.z, u.s, bd};
            }
        }
        team_sync();
        A = sh.all[team];
        const bool bad = A.z != A.z;                       // a NaN or +inf in the row, or a wait was given up
        const float log2z = log2f(A.z);                    // -inf for a row of -inf
        auto logprob = [&](float f) {
            return A.z == 0.f ? -INFINITY : (f - A.m) - log2z * 0.69314718055994530942f;
        };
        if (c == 0 && tid == 0) {
            if (p.tokens && p.logprob) {
                if (token >= 0 && token < p.V) p.logprob[row] = bad ? NAN : logprob(token_x);
                else if (p.dev_status) atomicOr(p.dev_status, BG_DEVSTAT_TOKEN);
            }
            if (p.entropy) p.entropy[row] = A.z == 0.f ? 0.f : (log2z - A.s / A.z) * 0.69314718055994530942f;
        }
        // ---- the logits at or above the bound
        if (p.K > 0) {
            // At least K logits of the row reach `least`; gathered are those from `bound` on, which is least or,
            // to leave out the logits that equal it, the next number.
            float least = A.bound, bound = least == -INFINITY ? above(least) : least;
            int n = 0;
            unsigned long long *cand = C > 1 ? reinterpret_cast<unsigned long long *>(sh.data) : list;
            // Every sweep but the last raises the bound over kCap - K logits at least, usually over nearly all.
            const int sweeps = bad ? 0 : p.V / (kCap - 32) + 2;
#pragma unroll 1
            for (int sweep = 0; sweep < sweeps; ++sweep) {
                int *count = &sh.n[sweep & 1][team];
                auto put = [&](bool in, float f, int v) {      // whole warps call it
                    const unsigned who = __ballot_sync(0xffffffffu, in);
                    if (who == 0) return;
                    int pos = 0;
                    if (lane == 0) pos = atomicAdd(count, __popc(who));
                    pos = __shfl_sync(0xffffffffu, pos, 0) + __popc(who & ((1u << lane) - 1u));
                    if (in && pos < kCap) list[pos] = pair_key(f, v);
                };
                const uint4 *vecs = reinterpret_cast<const uint4 *>(x + head);
                // bit t: stored maximum t of this lane reaches the bound
                unsigned mask = 0;
#pragma unroll
                for (int i = 0; i < kLpSlots / 8; ++i) {
                    float f[8];
                    LpVec<__nv_bfloat16>::unpack(sh.slot[warp][lane][i], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) mask |= f[e] >= bound ? 1u << (8 * i + e) : 0u;
                }
                mask &= (1u << slot) - 1u;
                if (sizeof(T) == 4 && sweep > 0) {
                    // a bound that many logits equal: their stored maxima were rounded up to it or above
                    unsigned left = mask;
#pragma unroll 1
                    while (__any_sync(0xffffffffu, left != 0)) {
                        const int t = __ffs(left) - 1;
                        bool in = false;
#pragma unroll 1
                        for (int b = 0; b < per_slot; ++b) {
                            const int vec = v0 + (t * per_slot + b) * kBatch + tid;
                            uint4 w[kLpLoads];
#pragma unroll
                            for (int i = 0; i < kLpLoads; ++i)
                                w[i] = t >= 0 && vec + i * kLanes < v1 ? vecs[vec + i * kLanes] : Vec::nothing();
                            in = in || Vec::largest(w) >= bound;
                        }
                        if (t >= 0 && !in) mask &= ~(1u << t);
                        left &= left - 1;
                    }
                }
                // eight such batches at a time, a lane for each of their vectors
                for (;;) {
                    const unsigned who = __ballot_sync(0xffffffffu, mask != 0);
                    if (who == 0) break;
                    // more than the list holds: this sweep only serves to raise the bound
                    if (__any_sync(0xffffffffu, *static_cast<volatile int *>(count) > kCap)) break;
                    const int nth = __popc(who & ((1u << lane) - 1u));
                    if (mask != 0 && nth < 8) {
                        sh.pick[warp][nth] = (__ffs(mask) - 1) << 5 | lane;
                        mask &= mask - 1;
                    }
                    __syncwarp();
                    const int picks = min(__popc(who), 8);
                    const int pick = lane / kLpLoads < picks ? sh.pick[warp][lane / kLpLoads] : -1;
                    __syncwarp();
#pragma unroll 1
                    for (int b = 0; b < per_slot; ++b) {
                        const int vec = v0 + ((pick >> 5) * per_slot + b) * kBatch + tw * 32 + (pick & 31) +
                                        (lane % kLpLoads) * kLanes;
                        const bool there = pick >= 0 && vec < v1;
                        const uint4 w = there ? vecs[vec] : Vec::nothing();
                        float f[VN];
                        Vec::unpack(w, f);
#pragma unroll
                        for (int e = 0; e < VN; ++e) put(there && f[e] >= bound, f[e], head + vec * VN + e);
                    }
                }
                if (tw == 0) put(loose >= 0 && loose_x >= bound, loose_x, loose);
                team_sync();
                n = *count;
                if (C > 1) {
                    // the lists of all CTAs into the first one's stages, which are empty by now
                    if (warp == 0) {
                        LpShared *lead = cluster.map_shared_rank(&sh, 0);
                        int pos = 0;
                        if (lane == 0) pos = atomicAdd(&lead->joined[sweep & 1], n);
                        if (lane < C) atomicAdd(&cluster.map_shared_rank(&sh, lane)->total[sweep & 1], n);
                        pos = __shfl_sync(0xffffffffu, pos, 0);
                        unsigned long long *joined = reinterpret_cast<unsigned long long *>(lead->data);
                        for (int i = lane; i < min(n, kCap) && pos + i < kCap; i += 32) joined[pos + i] = list[i];
                    }
                    cluster.sync();
                    n = sh.total[sweep & 1];
                }
                if (n <= kCap) break;
                // The list is full.  Its K-th largest is a bound too; what exceeds that goes into the next sweep.
                if (tid == 0) {
                    sh.n[(sweep + 1) & 1][team] = 0;
                    if (C > 1) sh.total[(sweep + 1) & 1] = sh.joined[(sweep + 1) & 1] = 0;
                }
                if (c == 0 && tw == 0) {
                    auto reach = [&](uint32_t key) {
                        int some = 0;
#pragma unroll 4
                        for (int i = lane; i < kCap; i += 32) some += static_cast<uint32_t>(cand[i] >> 32) >= key ? 1 : 0;
                        return __reduce_add_sync(0xffffffffu, some) >= p.K;
                    };
                    uint32_t kth = order_key(bound);       // the largest key that K of the list reach, bit by bit
                    if (reach(kth + 1)) {                  // (no: a bound that most of the list equal)
                        kth = 0;
#pragma unroll 1
                        for (uint32_t bit = 0x80000000u; bit != 0; bit >>= 1)
                            if (reach(kth | bit)) kth |= bit;
                    }
                    if (lane < C) (C == 1 ? &sh : cluster.map_shared_rank(&sh, lane))->all[team].bound = order_value(kth);
                }
                if (C > 1) cluster.sync();
                else team_sync();
                least = sh.all[team].bound;
                bound = above(least);
            }
            if (c == 0 && tw == 0) {
                int32_t *tt = p.top_token + row * p.K;
                float *tl = p.top_logprob + row * p.K;
                if (bad) {
                    if (lane < p.K) {
                        tt[lane] = -1;
                        tl[lane] = NAN;
                    }
                } else {
                    n = min(n, kCap);
                    int some = n;
                    if (n > kLpCount) {
                        // the largest pair that K of the list reach, bit by bit: those K are all there is to rank
                        unsigned long long kth = 0;
#pragma unroll 1
                        for (unsigned long long bit = 1ull << 63; bit != 0; bit >>= 1) {
                            int reach = 0;
#pragma unroll 4
                            for (int i = lane; i < n; i += 32) reach += cand[i] >= (kth | bit) ? 1 : 0;
                            if (__reduce_add_sync(0xffffffffu, reach) >= p.K) kth |= bit;
                        }
                        some = 0;
#pragma unroll 1
                        for (int i0 = 0; i0 < n; i0 += 32) {
                            const unsigned long long k = i0 + lane < n ? cand[i0 + lane] : 0;
                            const unsigned who = __ballot_sync(0xffffffffu, k >= kth);
                            if (k >= kth) sh.few[team][some + __popc(who & ((1u << lane) - 1u))] = k;
                            some += __popc(who);
                        }
                        __syncwarp();
                        cand = sh.few[team];
                    }
#pragma unroll 1
                    for (int i = lane; i < some; i += 32) {
                        const unsigned long long k = cand[i];
                        int rank = 0;
#pragma unroll 4
                        for (int j = 0; j < some; ++j) rank += cand[j] > k ? 1 : 0;
                        if (rank < p.K) {
                            tt[rank] = static_cast<int32_t>(~static_cast<uint32_t>(k));
                            tl[rank] = logprob(order_value(static_cast<uint32_t>(k >> 32)));
                        }
                    }
                    // fewer than K are above the bound (banned tokens behind the allowed ones, thousands of equal
                    // logits): the first tokens that equal it
#pragma unroll 1
                    for (int first = 0; n < p.K && first < p.V; first += 32 * 8) {
                        bool eq[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int v = first + 32 * i + lane;
                            eq[i] = v < p.V && Vec::load(x + min(v, p.V - 1)) == least;
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const unsigned who = __ballot_sync(0xffffffffu, eq[i]);
                            const int rank = n + __popc(who & ((1u << lane) - 1u));
                            if (eq[i] && rank < p.K) {
                                tt[rank] = first + 32 * i + lane;
                                tl[rank] = logprob(least);
                            }
                            n += __popc(who);
                        }
                    }
                }
            }
        }
        team_sync();                  // the team's shared memory is written again by its next row
    }
    // every copy has landed before the CTA exits
    if (tid == 0) {
        for (uint32_t k = loads > kLpStages ? loads - kLpStages : 0; k < loads; ++k)
            mbar_wait_drain(&full[k % kLpStages], (k / kLpStages) & 1);
        if (*abort && p.dev_status) atomicOr(p.dev_status, BG_DEVSTAT_TIMEOUT);
    }
}

template <typename T, int W, bool STALL>
cudaError_t launch_lp(const LpParams &p, int nsm, cudaStream_t stream)
{
    auto kern = logprobs_kernel<T, W, STALL>;
    static std::atomic<uint64_t> smem_done{0};
    cudaError_t e = ensure_smem_attribute(kern, static_cast<int>(sizeof(LpShared)), smem_done);
    if (e != cudaSuccess) return e;
    // with fewer rows than SMs, clusters of CTAs per row, but at least 16 KB for each
    int C = 1;
    if (W == kLpWarps)
        while (C < kLpMaxCluster && static_cast<int64_t>(p.N) * C * 2 <= 2 * nsm &&
               static_cast<int64_t>(p.V) * sizeof(T) >= (static_cast<int64_t>(C) << 15))
            C *= 2;
    const int64_t most = 2 * nsm / C, need = p.N;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((need < most ? need : most) * C));
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = sizeof(LpShared);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// Up to two rows per SM the whole CTA takes one row (304 rows of 50,001 fp32 logits: 16.1 us, and 23.0
// with 4 warps per row), up to four rows half of it does (480 rows: 27.4 by whole CTAs, 22.0 by 8 warps, 25.9
// by 4), from then on 4 warps do, eight rows at a time per SM (700 rows: 36.9 by 8 warps, 31.0 by 4; 1200
// rows: 45.0 and 42.7).  Rows under 16 KB are too short for 16 warps, and under 48 KB for 8 (400 rows of
// 20,011 bf16 logits: 11.2 us by 8 warps, 10.9 by 4; of 30,011: 13.0 and 14.4).
template <typename T, bool STALL>
cudaError_t launch_team(const LpParams &p, int nsm, cudaStream_t stream)
{
    const int64_t bytes = static_cast<int64_t>(p.V) * sizeof(T);
    if (p.N <= 2 * nsm && bytes >= 16 << 10) return launch_lp<T, 16, STALL>(p, nsm, stream);
    if (p.N > 2 * nsm && p.N <= 4 * nsm && bytes >= 48 << 10) return launch_lp<T, 8, STALL>(p, nsm, stream);
    return launch_lp<T, 4, STALL>(p, nsm, stream);
}

}  // namespace

cudaError_t launch_token_logprobs(const void *logits, int32_t dtype, int64_t row_stride, int32_t N, int32_t V,
                                  const int32_t *tokens, int32_t K, float *logprob, float *entropy, int32_t *top_token,
                                  float *top_logprob, int32_t *dev_status, int nsm, cudaStream_t stream)
{
    const LpParams p{logits, row_stride, N, V, K, tokens, logprob, entropy, top_token, top_logprob, dev_status, N};
    return dtype == BG_DTYPE_F32 ? launch_team<float, false>(p, nsm, stream)
                                 : launch_team<__nv_bfloat16, false>(p, nsm, stream);
}

cudaError_t launch_logprobs_selftest(const float *logits, int32_t N, int32_t V, const int32_t *tokens, int32_t stalled,
                                     float *logprob, float *entropy, int32_t *top_token, float *top_logprob,
                                     int32_t *dev_status, int nsm, cudaStream_t stream)
{
    const LpParams p{logits, V, N, V, 1, tokens, logprob, entropy, top_token, top_logprob, dev_status, stalled};
    return launch_team<float, true>(p, nsm, stream);
}

}  // namespace bg
