// logprobs.cu -- log-probability of a given token, entropy and the best alternatives of rows of
// logits.
//
// "SLM 生成式高并发推理引擎：延迟约束下的有效吞吐优化", section 1.1: a Prefill-Only request is
// answered from the next-token logits at the last valid position (softmax, Top-K).  With m the
// largest logit of a row, d_v = x_v - m and Z = sum_v e^(d_v):
//     logprob(t) = d_t - ln Z
//     entropy    = ln Z - sum_v e^(d_v) d_v / Z          (every term of the sum has one sign)
//     top        = the K largest logits, equal ones by the smaller index, as (v, d_v - ln Z)
// Only the row's bytes bound it, so everything comes out of one pass over them:
//   pass    every thread keeps a running maximum with Z and the entropy's sum relative to it, and
//           the maximum of each batch of 64 bytes it read in shared memory;
//   bound   the 2 largest thread maxima of each of the 16 warps are 32 >= K distinct logits, so
//           the K-th largest of them bounds the row's K-th best from below;
//   gather  a thread re-reads (from L2) only the batches whose maximum reaches the bound; the few
//           logits at or above it go to a list in shared memory, where each one's rank is the
//           number of larger (logit, index) pairs.
// A row with more than kLpCap such logits (thousands of equal ones) is searched K times instead.
// Few rows: a cluster of up to 8 CTAs shares a row, and its leader joins the sums and the lists.
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
constexpr int kLpLoads = 4;              // 16-byte loads per thread and batch
constexpr int kLpSlots = 16;             // stored batch maxima per thread
constexpr int kLpCap = 4096;             // gathered logits (a row this short never overflows)
constexpr int kLpMaxCluster = 8;
static_assert(2 * kLpWarps == 32 && BG_MAX_TOP <= 32, "two thread maxima per warp: one per lane, at least K");

// What a row's CTAs tell each other.
struct LpPart {
    float m, z, s;        // maximum, sum of e^(x - m), sum of e^(x - m) (x - m)
    float bound;          // at least K logits of this CTA's slice reach it (-inf: no such bound)
};

struct LpShared {
    float slot[kLpSlots][kLpThreads];
    unsigned long long key[kLpCap];          // order-preserving logit << 32 | ~index
    LpPart part[kLpMaxCluster];              // leader: one per CTA
    LpPart all;
    LpPart warp[kLpWarps];                   // bound: unused
    uint32_t top[2 * kLpWarps];              // the warps' largest thread maxima, then their second largest
    unsigned long long best[kLpWarps];
    int n;
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

// e^d is 0 from here down; differences are held above it, so that 0 meets no infinite factor
// (banned tokens at -inf, or at the type's lowest value).
constexpr float kLpFar = -10000.f;

// The maximum, and the two sums relative to it.
struct Running {
    float m = -INFINITY, z = 0.f, s = 0.f;

    // moves the reference to m_new >= m
    __device__ void rebase(float m_new)
    {
        if (m != -INFINITY) {
            const float d = max_nan(m - m_new, kLpFar), f = ex2(d * 1.44269504088896f);
            s = f * fmaf(z, d, s);
            z *= f;
        }
        m = m_new;
    }
    // joins sums relative to om (om -inf: sums of 0, or of NaN)
    __device__ void join(float om, float oz, float os)
    {
        if (om > m) {
            const float tm = m, tz = z, ts = s;
            m = om; z = oz; s = os;
            om = tm; oz = tz; os = ts;
        }
        const float d = om == -INFINITY ? 0.f : max_nan(om - m, kLpFar), f = ex2(d * 1.44269504088896f);
        s += f * fmaf(oz, d, os);
        z += f * oz;
    }
};

// e^(x - m) into the sums
__device__ __forceinline__ void add_term(Running &r, float x)
{
    const float d = max_nan(x - r.m, kLpFar), e = ex2(d * 1.44269504088896f);
    r.z += e;
    r.s = fmaf(e, d, r.s);
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

template <typename T>
__global__ void __launch_bounds__(kLpThreads, 2) logprobs_kernel(const LpParams p)
{
    extern __shared__ __align__(16) uint8_t lp_smem[];
    LpShared &sh = *reinterpret_cast<LpShared *>(lp_smem);
    using Vec = LpVec<T>;
    constexpr int VN = Vec::N;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks());
    const int c = static_cast<int>(cluster.block_rank());
    LpShared *lead = cluster.map_shared_rank(&sh, 0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_launch();
    grid_dep_wait();

    for (int64_t row = blockIdx.x / C; row < p.N; row += gridDim.x / C) {
        const T *x = static_cast<const T *>(p.logits) + row * p.stride;
        // [0, head) before the first 16-byte boundary, nv whole vectors, [tail, V) behind them
        const int head = min(static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(x) & 15u)) & 15u) / sizeof(T)), p.V);
        const int nv_row = (p.V - head) / VN;
        const int tail = head + nv_row * VN;
        const uint4 *xv = reinterpret_cast<const uint4 *>(x + head);
        const int v0 = static_cast<int>(static_cast<int64_t>(nv_row) * c / C);
        const int v1 = static_cast<int>(static_cast<int64_t>(nv_row) * (c + 1) / C);
        const int nb = (v1 - v0 + kLpThreads * kLpLoads - 1) / (kLpThreads * kLpLoads);   // batches
        const int per_slot = (nb + kLpSlots - 1) / kLpSlots;
        // the loose logits: the head belongs to the first CTA of the row, the tail to the last
        int loose = -1;
        if (c == 0 && tid < head) loose = tid;
        if (c == C - 1 && tid >= 32 && tid - 32 < p.V - tail) loose = tail + tid - 32;

        if (tid == 0) sh.n = 0;
        Running r;
        float best = -INFINITY;           // this thread's largest logit
        int in_slot = 0, slot = 0;
        float slot_max = -INFINITY;
        for (int b = 0; b < nb; ++b) {
            uint4 w[kLpLoads];
            float bm = -INFINITY;
            const int base = v0 + b * kLpThreads * kLpLoads + tid;
#pragma unroll
            for (int i = 0; i < kLpLoads; ++i)
                if (base + i * kLpThreads < v1) w[i] = __ldcs(xv + base + i * kLpThreads);
#pragma unroll
            for (int i = 0; i < kLpLoads; ++i) {
                if (base + i * kLpThreads < v1) {
                    float f[VN];
                    Vec::unpack(w[i], f);
#pragma unroll
                    for (int e = 0; e < VN; ++e) bm = fmaxf(bm, f[e]);
                }
            }
            if (bm > r.m) r.rebase(bm);
            slot_max = fmaxf(slot_max, bm);
            if (r.m == -INFINITY) {
                // only -inf so far (or NaN): nothing to add but a NaN
#pragma unroll
                for (int i = 0; i < kLpLoads; ++i) {
                    if (base + i * kLpThreads < v1) {
                        float f[VN];
                        Vec::unpack(w[i], f);
#pragma unroll
                        for (int e = 0; e < VN; ++e) r.z += f[e] != f[e] ? f[e] : 0.f;
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < kLpLoads; ++i) {
                    if (base + i * kLpThreads < v1) {
                        float f[VN];
                        Vec::unpack(w[i], f);
#pragma unroll
                        for (int e = 0; e < VN; ++e) add_term(r, f[e]);
                    }
                }
            }
            if (++in_slot == per_slot || b == nb - 1) {
                sh.slot[slot++][tid] = slot_max;
                best = fmaxf(best, slot_max);
                slot_max = -INFINITY;
                in_slot = 0;
            }
        }
        if (loose >= 0) {
            const float f = Vec::load(x + loose);
            if (f > r.m) r.rebase(f);
            if (r.m == -INFINITY) r.z += f != f ? f : 0.f;
            else add_term(r, f);
            best = fmaxf(best, f);
        }

        // ---- the CTA's sums, and its bound
        if (p.K > 0) {
            const uint32_t k1 = order_key(best);
            const uint32_t first = __reduce_max_sync(0xffffffffu, k1);
            const unsigned who = __ballot_sync(0xffffffffu, k1 == first);
            const uint32_t second = __reduce_max_sync(0xffffffffu, lane == __ffs(who) - 1 ? 0u : k1);
            if (lane == 0) {
                sh.top[warp] = first;
                sh.top[kLpWarps + warp] = second;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, r.m, o), oz = __shfl_xor_sync(0xffffffffu, r.z, o),
                        os = __shfl_xor_sync(0xffffffffu, r.s, o);
            r.join(om, oz, os);
        }
        if (lane == 0) sh.warp[warp] = LpPart{r.m, r.z, r.s, 0.f};
        __syncthreads();
        if (warp == 0) {
            LpPart q = sh.warp[lane & (kLpWarps - 1)];
            Running a;
            a.m = q.m; a.z = q.z; a.s = q.s;
            float bd = -INFINITY;
            if (p.K > 0) {
                const uint32_t k = sh.top[lane];
                int rank = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const uint32_t u = __shfl_sync(0xffffffffu, k, i);
                    rank += u > k || (u == k && i < lane) ? 1 : 0;
                }
                const unsigned who = __ballot_sync(0xffffffffu, rank == p.K - 1);
                bd = order_value(__shfl_sync(0xffffffffu, k, __ffs(who) - 1));
            }
#pragma unroll
            for (int o = kLpWarps / 2; o > 0; o >>= 1) {
                const float om = __shfl_xor_sync(0xffffffffu, a.m, o), oz = __shfl_xor_sync(0xffffffffu, a.z, o),
                            os = __shfl_xor_sync(0xffffffffu, a.s, o);
                a.join(om, oz, os);
            }
            if (lane == 0) {
                const LpPart mine{a.m, a.z, a.s, bd};
                if (C > 1) lead->part[c] = mine;
                else sh.all = mine;
            }
        }
        if (C > 1) {
            cluster.sync();
            if (warp == 0) {
                // every CTA joins all slices' sums in the same order
                const LpPart q = lane < C ? lead->part[lane] : LpPart{-INFINITY, 0.f, 0.f, -INFINITY};
                Running a;
                float bd = -INFINITY;
                for (int i = 0; i < C; ++i) {
                    a.join(__shfl_sync(0xffffffffu, q.m, i), __shfl_sync(0xffffffffu, q.z, i),
                           __shfl_sync(0xffffffffu, q.s, i));
                    bd = fmaxf(bd, __shfl_sync(0xffffffffu, q.bound, i));
                }
                if (lane == 0) sh.all = LpPart{a.m, a.z, a.s, bd};
            }
        }
        __syncthreads();
        const LpPart A = sh.all;
        const bool bad = A.z != A.z;                       // a NaN or +inf in the row
        const float lnz = logf(A.z);                       // -inf for a row of -inf
        if (c == 0 && tid == 0) {
            if (p.tokens && p.logprob) {
                const int t = p.tokens[row];
                if (t >= 0 && t < p.V)
                    p.logprob[row] = bad ? NAN : A.z == 0.f ? -INFINITY : Vec::load(x + t) - A.m - lnz;
                else if (p.dev_status)
                    atomicOr(p.dev_status, BG_DEVSTAT_TOKEN);
            }
            if (p.entropy) p.entropy[row] = A.z == 0.f ? 0.f : lnz - A.s / A.z;
        }
        // ---- the logits at or above the bound
        if (p.K > 0) {
            if (!bad) {
                auto put = [&](float f, int v) {
                    if (f >= A.bound) {
                        const int at = atomicAdd(&lead->n, 1);
                        if (at < kLpCap) lead->key[at] = pair_key(f, v);
                    }
                };
                for (int t = 0; t < slot; ++t) {
                    if (sh.slot[t][tid] < A.bound) continue;
                    for (int b = t * per_slot; b < min((t + 1) * per_slot, nb); ++b) {
                        const int base = v0 + b * kLpThreads * kLpLoads + tid;
#pragma unroll
                        for (int i = 0; i < kLpLoads; ++i) {
                            const int at = base + i * kLpThreads;
                            if (at < v1) {
                                const uint4 w = xv[at];
                                float f[VN];
                                Vec::unpack(w, f);
#pragma unroll
                                for (int e = 0; e < VN; ++e) put(f[e], head + at * VN + e);
                            }
                        }
                    }
                }
                if (loose >= 0) put(Vec::load(x + loose), loose);
            }
            if (C > 1) cluster.sync(); else __syncthreads();
            if (c == 0) {
                const int n = sh.n;
                int32_t *tt = p.top_token + row * p.K;
                float *tl = p.top_logprob + row * p.K;
                auto value = [&](unsigned long long k) {
                    return A.z == 0.f ? -INFINITY : order_value(static_cast<uint32_t>(k >> 32)) - A.m - lnz;
                };
                if (bad) {
                    if (tid < p.K) {
                        tt[tid] = -1;
                        tl[tid] = NAN;
                    }
                } else if (n <= kLpCap) {
                    for (int i = tid; i < n; i += kLpThreads) {
                        const unsigned long long k = sh.key[i];
                        int rank = 0;
                        for (int j = 0; j < n; ++j) rank += sh.key[j] > k ? 1 : 0;
                        if (rank < p.K) {
                            tt[rank] = static_cast<int32_t>(~static_cast<uint32_t>(k));
                            tl[rank] = value(k);
                        }
                    }
                } else {
                    // the largest pair below the last one found, K times
                    unsigned long long last = ~0ull;
                    for (int i = 0; i < p.K; ++i) {
                        unsigned long long mine = 0;
                        for (int v = tid; v < p.V; v += kLpThreads) {
                            const unsigned long long k = pair_key(Vec::load(x + v), v);
                            if (k < last && k > mine) mine = k;
                        }
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) {
                            const unsigned long long u = __shfl_xor_sync(0xffffffffu, mine, o);
                            mine = u > mine ? u : mine;
                        }
                        if (lane == 0) sh.best[warp] = mine;
                        __syncthreads();
                        mine = sh.best[lane & (kLpWarps - 1)];
#pragma unroll
                        for (int o = kLpWarps / 2; o > 0; o >>= 1) {
                            const unsigned long long u = __shfl_xor_sync(0xffffffffu, mine, o);
                            mine = u > mine ? u : mine;
                        }
                        __syncthreads();
                        last = mine;
                        if (tid == 0) {
                            tt[i] = static_cast<int32_t>(~static_cast<uint32_t>(last));
                            tl[i] = value(last);
                        }
                    }
                }
            }
        }
        __syncthreads();              // sh is written again by the next row
        if (C > 1) cluster.sync();    // ... also by the other CTAs, and no CTA leaves while it is read
    }
}

template <typename T>
cudaError_t launch_lp(const LpParams &p, int nsm, cudaStream_t stream)
{
    auto kern = logprobs_kernel<T>;
    static std::atomic<uint64_t> smem_done{0};
    cudaError_t e = ensure_smem_attribute(kern, static_cast<int>(sizeof(LpShared)), smem_done);
    if (e != cudaSuccess) return e;
    // as many CTAs per row as keep the GPU's 2 CTAs per SM filled, but at least 16 KB of it each
    int C = 1;
    while (C < kLpMaxCluster && static_cast<int64_t>(p.N) * C * 2 <= 2 * nsm &&
           static_cast<int64_t>(p.V) * sizeof(T) >= (static_cast<int64_t>(C) << 15))
        C *= 2;
    int64_t rows = 2 * nsm / C;
    if (rows > p.N) rows = p.N;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * C));
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

}  // namespace

cudaError_t launch_token_logprobs(const void *logits, int32_t dtype, int64_t row_stride, int32_t N, int32_t V,
                                  const int32_t *tokens, int32_t K, float *logprob, float *entropy, int32_t *top_token,
                                  float *top_logprob, int32_t *dev_status, int nsm, cudaStream_t stream)
{
    const LpParams p{logits, row_stride, N, V, K, tokens, logprob, entropy, top_token, top_logprob, dev_status};
    return dtype == BG_DTYPE_F32 ? launch_lp<float>(p, nsm, stream) : launch_lp<__nv_bfloat16>(p, nsm, stream);
}

}  // namespace bg
