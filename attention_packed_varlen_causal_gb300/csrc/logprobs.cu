// logprobs.cu -- log-probability of a given token, entropy and the best alternatives of rows of
// logits.
//
// "SLM 生成式高并发推理引擎：延迟约束下的有效吞吐优化", section 1.1: a Prefill-Only request is
// answered from the next-token logits at the last valid position (softmax, Top-K).  With m the
// largest logit of a row, d_v = x_v - m and Z = sum_v e^(d_v):
//     logprob(t) = d_t - ln Z
//     entropy    = ln Z - sum_v e^(d_v) d_v / Z          (every term of the sum has one sign)
//     top        = the K largest logits, equal ones by the smaller index, as (v, d_v - ln Z)
// Only the row's bytes bound it, so everything comes out of one pass over them, by a team of W warps
// (a power of two up to the 16 of a CTA; with fewer rows than CTAs, a cluster of up to 8 CTAs):
//   pass    every lane keeps a running maximum with Z and the entropy's sum relative to it, and in
//           shared memory the maximum of each batch of 64 bytes it read, rounded up to bf16;
//   bound   the 32 / W largest lane maxima of each warp are 32 >= K distinct logits, so the K-th
//           largest of them bounds the row's K-th best from below;
//   gather  only the batches whose maximum reaches the bound are read again (from L2), one logit
//           per lane; the few logits at or above it go to a list in shared memory, where each one's
//           rank is the number of larger (logit, index) pairs.
// A row with more such logits than the list holds (thousands of equal ones) is searched K times
// instead.
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
constexpr int kLpSlots = 64;             // stored batch maxima per lane (of one or more batches each)
constexpr int kLpCap = 288;              // gathered logits per warp of the team (a row too short to give
                                         // 32 lane maxima fits)
constexpr int kLpMaxCluster = 8;
static_assert(BG_MAX_TOP <= 32, "at least K lane maxima");

// A slice's results: what the warps of a team, and the CTAs of a cluster, tell each other.
struct LpPart {
    float m, z, s;        // maximum, sum of 2^t, sum of 2^t t
    float bound;          // at least K logits of the slice reach it (-inf: no such bound)
};

struct LpShared {
    __nv_bfloat16 slot[kLpWarps][kLpSlots][32];
    unsigned long long key[kLpWarps * kLpCap];   // order-preserving logit << 32 | ~index; per team
    LpPart part[kLpMaxCluster];                  // first CTA: one per CTA
    LpPart all[kLpWarps];                        // per team
    LpPart warp[kLpWarps];                       // (bound: unused)
    uint32_t top[kLpWarps][32];                  // a team's 32 lane maxima, at its first warp
    unsigned long long best[kLpWarps];
    int n[kLpWarps];                             // per team
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

__device__ __forceinline__ float fmin3f(float a, float b, float c)
{
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

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
    static __device__ void bounds(const uint4 *w, float *hi, float *lo)      // of kLpLoads vectors
    {
        float h[kLpLoads], l[kLpLoads];
#pragma unroll
        for (int i = 0; i < kLpLoads; ++i) {
            float x[4];
            unpack(w[i], x);
            h[i] = fmaxf(fmax3f(x[0], x[1], x[2]), x[3]);
            l[i] = fminf(fmin3f(x[0], x[1], x[2]), x[3]);
        }
        *hi = fmaxf(fmax3f(h[0], h[1], h[2]), h[3]);
        *lo = fminf(fmin3f(l[0], l[1], l[2]), l[3]);
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
    static __device__ void bounds(const uint4 *w, float *hi, float *lo)
    {
        auto pair = [](uint32_t u) { return *reinterpret_cast<__nv_bfloat162 *>(&u); };
        __nv_bfloat162 h[kLpLoads], l[kLpLoads];
#pragma unroll
        for (int i = 0; i < kLpLoads; ++i) {
            h[i] = __hmax2(__hmax2(pair(w[i].x), pair(w[i].y)), __hmax2(pair(w[i].z), pair(w[i].w)));
            l[i] = __hmin2(__hmin2(pair(w[i].x), pair(w[i].y)), __hmin2(pair(w[i].z), pair(w[i].w)));
        }
        const float2 a = __bfloat1622float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
        const float2 b = __bfloat1622float2(__hmin2(__hmin2(l[0], l[1]), __hmin2(l[2], l[3])));
        *hi = fmaxf(a.x, a.y);
        *lo = fminf(b.x, b.y);
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
};

// A batch maximum as it is stored: not below x (exact for bf16 logits; -inf stays).
__device__ __forceinline__ __nv_bfloat16 slot_value(float x)
{
    const uint32_t u = __float_as_uint(x);
    if ((u & 0xffffu) == 0) return __float2bfloat16_rn(x);
    return __float2bfloat16_ru(x);
}

template <typename T, int W>
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
    LpShared *lead = C == 1 ? &sh : cluster.map_shared_rank(&sh, 0);
    unsigned long long *list = lead->key + team * kCap;
    auto team_sync = [&]() {
        if constexpr (W == 1) __syncwarp();
        else if constexpr (W == kLpWarps) __syncthreads();
        else named_bar_sync(1 + team, kLanes);
    };
    grid_dep_launch();
    grid_dep_wait();

    const int64_t rows_at_once = static_cast<int64_t>(gridDim.x / C) * kTeams;
    for (int64_t row = static_cast<int64_t>(blockIdx.x / C) * kTeams + team; row < p.N; row += rows_at_once) {
        const T *x = static_cast<const T *>(p.logits) + row * p.stride;
        // [0, head) before the first 16-byte boundary, nv whole vectors, [tail, V) behind them
        const int head = min(static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(x) & 15u)) & 15u) / sizeof(T)), p.V);
        const int nv = (p.V - head) / VN;
        const int tail = head + nv * VN;
        const uint4 *xv = reinterpret_cast<const uint4 *>(x + head);
        const int v0 = C == 1 ? 0 : static_cast<int>(static_cast<int64_t>(nv) * c / C);
        const int v1 = C == 1 ? nv : static_cast<int>(static_cast<int64_t>(nv) * (c + 1) / C);
        const int nb = (v1 - v0 + kBatch - 1) / kBatch;
        const int per_slot = (nb + kLpSlots - 1) / kLpSlots;
        // the loose logits: the head belongs to the first CTA of the row, the tail to the last
        const int n_head = c == 0 ? head : 0, n_tail = c == C - 1 ? p.V - tail : 0;
        const int loose = lane < n_head ? lane : lane >= 16 && lane - 16 < n_tail ? tail + lane - 16 : -1;
        const float loose_x = tw == 0 && loose >= 0 ? Vec::load(x + loose) : -INFINITY;
        if (tid == 0) sh.n[team] = 0;

        Running a;
        float best = -INFINITY;           // this lane's largest logit
        int in_slot = 0, slot = 0;
        float slot_max = -INFINITY;
        uint4 w[kLpLoads];
        auto fetch = [&](int at) {        // past the slice's end -inf, which adds nothing
#pragma unroll
            for (int i = 0; i < kLpLoads; ++i) {
                w[i] = Vec::nothing();
                if (at + i * kLanes < v1) w[i] = __ldg(xv + at + i * kLanes);
            }
        };
        int at = v0 + tid;
        if (nb > 0) fetch(at);
#pragma unroll 1
        for (int b = 0; b < nb; ++b) {
            uint4 g[kLpLoads];
#pragma unroll
            for (int i = 0; i < kLpLoads; ++i) g[i] = w[i];
            at += kBatch;
            if (b + 1 < nb) fetch(at);    // the next batch while this one is summed
            float bm, bl;
            Vec::bounds(g, &bm, &bl);
            if (bm > a.m) a.rebase(bm);
            slot_max = fmaxf(slot_max, bm);
            const float2 c2 = make_float2(kLog2e, kLog2e);
            float2 z2 = make_float2(0.f, 0.f), s2 = make_float2(0.f, 0.f);
            // Far below the maximum (banned logits, or past the slice's end) differences are held; with
            // -inf only there is no reference.  (NaN takes either way and stays.)
            const bool far = !(bl - a.m > kLpFar);
            const float nm = a.m == -INFINITY ? 0.f : -a.m;
            const float2 nm2 = make_float2(nm, nm);
#pragma unroll
            for (int i = 0; i < kLpLoads; ++i) {
                float f[VN];
                Vec::unpack(g[i], f);
#pragma unroll
                for (int e = 0; e < VN; e += 2) {
                    float2 d = fadd2(make_float2(f[e], f[e + 1]), nm2);
                    if (far) d = make_float2(max_nan(d.x, kLpFar), max_nan(d.y, kLpFar));
                    const float2 t = fmul2(d, c2);
                    const float2 q = make_float2(ex2(t.x), ex2(t.y));
                    z2 = fadd2(z2, q);
                    s2 = ffma2(q, t, s2);
                }
            }
            a.z += z2.x + z2.y;
            a.s += s2.x + s2.y;
            if (++in_slot == per_slot || b == nb - 1) {
                sh.slot[warp][slot++][lane] = slot_value(slot_max);
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
        uint32_t mine = order_key(best);
        if (p.K > 0 && W > 1) {
#pragma unroll 1
            for (int i = 0; i < 32 / W; ++i) {
                const uint32_t top = __reduce_max_sync(0xffffffffu, mine);
                const unsigned who = __ballot_sync(0xffffffffu, mine == top);
                if (lane == __ffs(who) - 1) {
                    sh.top[team * W][tw * (32 / W) + i] = top;
                    mine = 0;
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, a.m, o), oz = __shfl_xor_sync(0xffffffffu, a.z, o),
                        os = __shfl_xor_sync(0xffffffffu, a.s, o);
            a.join(om, oz, os);
        }
        LpPart A{a.m, a.z, a.s, -INFINITY};
        auto kth = [&](uint32_t k) {      // the K-th largest of the warp's 32 keys
            int rank = 0;
#pragma unroll 8
            for (int i = 0; i < 32; ++i) {
                const uint32_t u = __shfl_sync(0xffffffffu, k, i);
                rank += u > k || (u == k && i < lane) ? 1 : 0;
            }
            const unsigned who = __ballot_sync(0xffffffffu, rank == p.K - 1);
            return order_value(__shfl_sync(0xffffffffu, k, __ffs(who) - 1));
        };
        if constexpr (W == 1) {
            if (p.K > 0) A.bound = kth(mine);
        } else {
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
                const float bd = p.K > 0 ? kth(sh.top[team * W][lane]) : -INFINITY;
                if (lane == 0) {
                    const LpPart part{u.m, u.z, u.s, bd};
                    if (C > 1) lead->part[c] = part;
                    else sh.all[team] = part;
                }
            }
            if (C > 1) {
                cluster.sync();
                if (warp == 0) {
                    // every CTA joins all slices' sums in the same order
                    const LpPart q = lane < C ? lead->part[lane] : LpPart{-INFINITY, 0.f, 0.f, -INFINITY};
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
        }
        const bool bad = A.z != A.z;                       // a NaN or +inf in the row
        const float log2z = log2f(A.z);                    // -inf for a row of -inf
        auto logprob = [&](float f) {
            return A.z == 0.f ? -INFINITY : (f - A.m) - log2z * 0.69314718055994530942f;
        };
        if (c == 0 && tid == 0) {
            if (p.tokens && p.logprob) {
                const int t = p.tokens[row];
                if (t >= 0 && t < p.V) p.logprob[row] = bad ? NAN : logprob(Vec::load(x + t));
                else if (p.dev_status) atomicOr(p.dev_status, BG_DEVSTAT_TOKEN);
            }
            if (p.entropy) p.entropy[row] = A.z == 0.f ? 0.f : (log2z - A.s / A.z) * 0.69314718055994530942f;
        }
        // ---- the logits at or above the bound
        if (p.K > 0) {
            auto put = [&](bool in, float f, int v) {      // whole warps call it
                const unsigned who = __ballot_sync(0xffffffffu, in);
                if (who == 0) return;
                int pos = 0;
                if (lane == 0) pos = atomicAdd(&lead->n[team], __popc(who));
                pos = __shfl_sync(0xffffffffu, pos, 0) + __popc(who & ((1u << lane) - 1u));
                if (in && pos < kCap) list[pos] = pair_key(f, v);
            };
            if (!bad) {
#pragma unroll 1
                for (int t = 0; t < slot; ++t) {
                    unsigned who = __ballot_sync(0xffffffffu, __bfloat162float(sh.slot[warp][t][lane]) >= A.bound);
                    while (who != 0) {
                        const int owner = __ffs(who) - 1;
                        who &= who - 1;
#pragma unroll 1
                        for (int b = t * per_slot; b < min((t + 1) * per_slot, nb); ++b) {
                            // element e of the owner's batch: its vector e / VN, place e % VN there
                            const int vec = v0 + b * kBatch + tw * 32 + owner + (lane / VN) * kLanes;
                            const int v = head + vec * VN + lane % VN;
                            const bool there = lane < kLpLoads * VN && vec < v1;
                            const float f = there ? Vec::load(x + v) : -INFINITY;
                            put(there && f >= A.bound, f, v);
                        }
                    }
                }
                if (tw == 0) put(loose >= 0 && loose_x >= A.bound, loose_x, loose);
            }
            if (C > 1) cluster.sync();
            else team_sync();
            if (c == 0 && (tw == 0 || sh.n[team] > kCap)) {
                const int n = sh.n[team];
                int32_t *tt = p.top_token + row * p.K;
                float *tl = p.top_logprob + row * p.K;
                auto store = [&](int i, unsigned long long k) {
                    tt[i] = static_cast<int32_t>(~static_cast<uint32_t>(k));
                    tl[i] = logprob(order_value(static_cast<uint32_t>(k >> 32)));
                };
                if (bad) {
                    if (lane < p.K) {
                        tt[lane] = -1;
                        tl[lane] = NAN;
                    }
                } else if (n <= kCap) {
#pragma unroll 1
                    for (int i = lane; i < n; i += 32) {
                        const unsigned long long k = list[i];
                        int rank = 0;
#pragma unroll 4
                        for (int j = 0; j < n; ++j) rank += list[j] > k ? 1 : 0;
                        if (rank < p.K) store(rank, k);
                    }
                } else {
                    // the largest pair below the last one found, K times
                    unsigned long long found = ~0ull;
#pragma unroll 1
                    for (int i = 0; i < p.K; ++i) {
                        unsigned long long k = 0;
#pragma unroll 1
                        for (int v = tid; v < p.V; v += kLanes) {
                            const unsigned long long u = pair_key(Vec::load(x + v), v);
                            if (u < found && u > k) k = u;
                        }
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) {
                            const unsigned long long u = __shfl_xor_sync(0xffffffffu, k, o);
                            k = u > k ? u : k;
                        }
                        if constexpr (W > 1) {
                            if (lane == 0) sh.best[warp] = k;
                            team_sync();
                            k = sh.best[team * W + (lane & (W - 1))];
#pragma unroll
                            for (int o = W / 2; o > 0; o >>= 1) {
                                const unsigned long long u = __shfl_xor_sync(0xffffffffu, k, o);
                                k = u > k ? u : k;
                            }
                            team_sync();
                        }
                        found = k;
                        if (tid == 0) store(i, found);
                    }
                }
            }
        }
        team_sync();                  // the team's shared memory is written again by its next row
        if (C > 1) cluster.sync();    // ... also by the other CTAs, and no CTA leaves while it is read
    }
}

template <typename T, int W>
cudaError_t launch_lp(const LpParams &p, int nsm, cudaStream_t stream)
{
    auto kern = logprobs_kernel<T, W>;
    static std::atomic<uint64_t> smem_done{0};
    cudaError_t e = ensure_smem_attribute(kern, static_cast<int>(sizeof(LpShared)), smem_done);
    if (e != cudaSuccess) return e;
    // with fewer rows than CTAs (2 per SM), clusters of CTAs per row, but at least 16 KB for each
    int C = 1;
    if (W == kLpWarps)
        while (C < kLpMaxCluster && static_cast<int64_t>(p.N) * C * 2 <= 2 * nsm &&
               static_cast<int64_t>(p.V) * sizeof(T) >= (static_cast<int64_t>(C) << 15))
            C *= 2;
    const int64_t most = 2 * nsm / C, need = (p.N + kLpWarps / W - 1) / (kLpWarps / W);
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

// Warps per row: as few as keep 32 warps per SM busy, and none without a vector for each lane.
template <typename T>
cudaError_t launch_team(const LpParams &p, int nsm, cudaStream_t stream)
{
    const int64_t nv = static_cast<int64_t>(p.V) * sizeof(T) / 16;
    int W = 1;
    while (W < kLpWarps && static_cast<int64_t>(p.N) * W < 32 * nsm && nv >= 64 * W) W *= 2;
    if (W == 16) return launch_lp<T, 16>(p, nsm, stream);
    if (W >= 4) return launch_lp<T, 4>(p, nsm, stream);
    return launch_lp<T, 1>(p, nsm, stream);
}

}  // namespace

cudaError_t launch_token_logprobs(const void *logits, int32_t dtype, int64_t row_stride, int32_t N, int32_t V,
                                  const int32_t *tokens, int32_t K, float *logprob, float *entropy, int32_t *top_token,
                                  float *top_logprob, int32_t *dev_status, int nsm, cudaStream_t stream)
{
    const LpParams p{logits, row_stride, N, V, K, tokens, logprob, entropy, top_token, top_logprob, dev_status};
    return dtype == BG_DTYPE_F32 ? launch_team<float>(p, nsm, stream) : launch_team<__nv_bfloat16>(p, nsm, stream);
}

}  // namespace bg
