// logits.cu -- penalties for repeated tokens, biases and grammar masks on rows of logits.
//
// "SLM 生成式高并发推理引擎：延迟约束下的有效吞吐优化", section 1.1: a request is answered from the
// next-token logits, whose candidates are selected per step.  Ahead of that selection, with p(v) whether token v
// is in the prompt of the row's group and c(v) how often it is among the row's own tokens:
//     y = x > 0 ? x / rho : x * rho                 if p(v) or c(v) > 0
//     y = y - (alpha c(v) + beta)                   if c(v) > 0
//     y = y + b(v)                                  if the group has a bias for v (the last one listed)
//     y = -inf                                      if the row's mask does not have bit v
// in fp32, rounded once where the output is bf16.
//
// Memory bounds it: a logit is read (unless the mask bans it and its neighbours) and written.  A CTA takes a
// chunk of the vocabulary for some rows of one group.  It keeps one word per token of its chunk in shared memory:
// the bias' number, whether the prompt has the token, and the row's count, which is added before a row and
// taken away after it.  So prompt and biases are looked at once for all rows of the CTA, histories of any
// length cost their own reading, and integer atomics leave no order to depend on.
#include <cuda_bf16.h>

#include "bg_internal.h"
#include "bg_ptx.cuh"

namespace bg {
namespace {

constexpr int kLgThreads = 256;
constexpr int kLgMaxChunk = 8192;
constexpr int kLgMinChunk = 1024;
constexpr int kCountBits = 18;                       // two rows' counts meet for a moment: 2 * 65536 fits
constexpr uint32_t kCountMask = (1u << kCountBits) - 1, kPromptBit = 1u << kCountBits;
constexpr int kBiasShift = kCountBits + 1;
static_assert(2 * BG_MAX_SEQLEN <= static_cast<int>(kCountMask), "count bits");
static_assert(BG_MAX_BIAS < (1 << (32 - kBiasShift)), "bias numbers");

__device__ __forceinline__ float load_one(const float *p) { return *p; }
__device__ __forceinline__ float load_one(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_one(float *p, float x) { *p = x; }
__device__ __forceinline__ void store_one(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

template <int N>
__device__ __forceinline__ void load_vec(const float *p, float *x)
{
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(x + i) = *reinterpret_cast<const float4 *>(p + i);
}
template <int N>
__device__ __forceinline__ void load_vec(const __nv_bfloat16 *p, float *x)
{
    static_assert(N == 8, "16 bytes");
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <int N>
__device__ __forceinline__ void store_vec(float *p, const float *x)
{
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}
template <int N>
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const float *x)
{
    static_assert(N == 8, "16 bytes");
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                               pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Whether offsets [a, b) lie within [0, n]; the first ones start at 0 and the last ones end at n.
__device__ __forceinline__ bool offsets_ok(int a, int b, int n, int g, int groups)
{
    return a >= 0 && b >= a && b <= n && (g > 0 || a == 0) && (g < groups - 1 || b == n);
}

// N logits (1, 4 or 8 side by side) per thread and step.
template <typename TI, typename TO, int N>
__global__ void __launch_bounds__(kLgThreads)
    logits_kernel(const LogitsParams p, int chunk, int chunks, int rows_per_cta, int row_blocks)
{
    extern __shared__ uint32_t table[];              // [chunk], where there are lists
    grid_dep_launch();
    grid_dep_wait();
    const int tid = threadIdx.x;
    const int block = static_cast<int>(blockIdx.x) / chunks, v0 = (static_cast<int>(blockIdx.x) - block * chunks) * chunk;
    const int n = min(chunk, p.V - v0);
    const int g = block / row_blocks, first = (block - g * row_blocks) * rows_per_cta;
    const int last = min(first + rows_per_cta, p.per);
    const bool lists = p.prompt || p.own || p.bias_tokens;
    int pa = 0, pb = 0, ba = 0, bb = 0, bad = 0;
    if (p.prompt) {
        pa = p.cu_prompt[g];
        pb = p.cu_prompt[g + 1];
        if (!offsets_ok(pa, pb, p.total_prompt, g, p.groups)) bad |= BG_DEVSTAT_CU_PROMPT;
    }
    if (p.bias_tokens) {
        ba = p.cu_bias[g];
        bb = p.cu_bias[g + 1];
        if (!offsets_ok(ba, bb, p.total_bias, g, p.groups) || bb - ba > BG_MAX_BIAS) bad |= BG_DEVSTAT_BIAS;
    }
    if (bad) {                                       // the same for all threads
        if (tid == 0 && p.dev_status) atomicOr(p.dev_status, bad);
        return;
    }
    bool outside = false;                            // a token outside the vocabulary
    if (lists) {
        for (int i = tid; i < (n + 3) / 4; i += kLgThreads) reinterpret_cast<uint4 *>(table)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        for (int i = ba + tid; i < bb; i += kLgThreads) {
            const int t = p.bias_tokens[i];
            outside = outside || t < 0 || t >= p.V;
            if (t >= v0 && t < v0 + n) atomicMax(&table[t - v0], static_cast<uint32_t>(i - ba + 1) << kBiasShift);
        }
        if (p.bias_tokens) __syncthreads();
        for (int i = pa + tid; i < pb; i += kLgThreads) {
            const int t = p.prompt[i];
            outside = outside || t < 0 || t >= p.V;
            if (t >= v0 && t < v0 + n) atomicOr(&table[t - v0], kPromptBit);
        }
        __syncthreads();
    }
    const float rho = p.repetition ? p.repetition[g] : 1.f;
    const float alpha = p.frequency ? p.frequency[g] : 0.f, beta = p.presence ? p.presence[g] : 0.f;
    auto edit = [&](float x, uint32_t w) {
        const uint32_t c = w & kCountMask;
        if (p.repetition && (w & (kCountMask | kPromptBit))) x = x > 0.f ? x / rho : x * rho;
        if (c) x -= fmaf(alpha, static_cast<float>(c), beta);
        if (w >> kBiasShift) x += p.bias_values[ba + static_cast<int>(w >> kBiasShift) - 1];
        return x;
    };

    for (int r = first; r < last; ++r) {
        const int64_t row = static_cast<int64_t>(g) * p.per + r;
        const int m = !p.mask ? -1 : p.mask_index ? p.mask_index[row] : static_cast<int>(row);
        int len = 0;
        if (p.own) len = p.own_lens ? p.own_lens[row] : p.own_max;
        const int wrong = (p.mask && (m < -1 || m >= p.num_masks) ? BG_DEVSTAT_MASK : 0) |
                          (len < 0 || len > p.own_max ? BG_DEVSTAT_SEQ_TOO_LONG : 0);
        if (wrong) {                                 // the same for all threads
            if (tid == 0 && p.dev_status) atomicOr(p.dev_status, wrong);
            continue;
        }
        const int32_t *own = p.own ? p.own + row * p.own_stride : nullptr;
        if (p.own) {
            for (int i = tid; i < len; i += kLgThreads) {
                const int t = own[i];
                outside = outside || t < 0 || t >= p.V;
                if (t >= v0 && t < v0 + n) atomicAdd(&table[t - v0], 1u);
            }
            __syncthreads();
        }
        const TI *in = static_cast<const TI *>(p.in) + row * p.in_stride + v0;
        TO *out = static_cast<TO *>(p.out) + row * p.out_stride + v0;
        const uint32_t *mask = m < 0 ? nullptr : p.mask + m * p.mask_stride + v0 / 32;
        constexpr int kSteps = N == 1 ? 8 : 4;
        for (int i0 = tid * N; i0 < n; i0 += kSteps * kLgThreads * N) {
            uint32_t keep[kSteps];
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const int i = i0 + k * kLgThreads * N;
                keep[k] = i < n ? (mask ? mask[i / 32] >> (i % 32) : ~0u) & ((1u << N) - 1u) : 0u;
            }
            float x[kSteps][N];
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const int i = i0 + k * kLgThreads * N;
                if (!keep[k]) continue;
                if (N > 1 && i + N <= n) {
                    if constexpr (N > 1) load_vec<N>(in + i, x[k]);
                } else {
#pragma unroll
                    for (int e = 0; e < N; ++e) x[k][e] = i + e < n ? load_one(in + i + e) : 0.f;
                }
            }
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const int i = i0 + k * kLgThreads * N;
                if (i >= n) break;
                if (lists && keep[k]) {
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const uint32_t w = table[i + e];       // (past n: whatever it is)
                        if (w && i + e < n) x[k][e] = edit(x[k][e], w);
                    }
                }
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (!((keep[k] >> e) & 1u)) x[k][e] = -INFINITY;
                if (N > 1 && i + N <= n) {
                    if constexpr (N > 1) store_vec<N>(out + i, x[k]);
                } else {
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (i + e < n) store_one(out + i + e, x[k][e]);
                }
            }
        }
        if (p.own) {
            __syncthreads();
            for (int i = tid; i < len; i += kLgThreads) {
                const int t = own[i];
                if (t >= v0 && t < v0 + n) atomicSub(&table[t - v0], 1u);
            }
        }
    }
    if (outside && p.dev_status) atomicOr(p.dev_status, BG_DEVSTAT_TOKEN);
}

template <typename TI, typename TO, int N>
cudaError_t launch_typed(const LogitsParams &p, int chunk, int rows_per_cta, cudaStream_t stream)
{
    const int row_blocks = (p.per + rows_per_cta - 1) / rows_per_cta, chunks = (p.V + chunk - 1) / chunk;
    const bool lists = p.prompt || p.own || p.bias_tokens;
    const int64_t ctas = static_cast<int64_t>(p.groups) * row_blocks * chunks;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    return launch_dependent(logits_kernel<TI, TO, N>, dim3(static_cast<unsigned>(ctas)), dim3(kLgThreads),
                            lists ? chunk * sizeof(uint32_t) : 0, stream, p, chunk, chunks, rows_per_cta, row_blocks);
}

}  // namespace

cudaError_t launch_adjust_logits(const LogitsParams &p, int in_dtype, int out_dtype, bool vectors, int nsm, cudaStream_t stream)
{
    // Chunks as large as leaves two CTAs per SM, then rows as many as leave eight.
    int chunk = kLgMaxChunk;
    const int64_t rows = static_cast<int64_t>(p.groups) * p.per;
    auto chunks = [&] { return (p.V + chunk - 1) / chunk; };
    while (chunk > kLgMinChunk && chunks() * rows < 2 * nsm) chunk /= 2;
    int per = p.per;
    while (per > 1 && chunks() * static_cast<int64_t>(p.groups) * ((p.per + per - 1) / per) < 8 * nsm) per = (per + 1) / 2;
    if (in_dtype == BG_DTYPE_F32)
        return vectors ? launch_typed<float, float, 4>(p, chunk, per, stream) : launch_typed<float, float, 1>(p, chunk, per, stream);
    if (out_dtype == BG_DTYPE_F32)
        return vectors ? launch_typed<__nv_bfloat16, float, 8>(p, chunk, per, stream)
                       : launch_typed<__nv_bfloat16, float, 1>(p, chunk, per, stream);
    return vectors ? launch_typed<__nv_bfloat16, __nv_bfloat16, 8>(p, chunk, per, stream)
                   : launch_typed<__nv_bfloat16, __nv_bfloat16, 1>(p, chunk, per, stream);
}

}  // namespace bg
