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
// chunk of the vocabulary for some rows of one group.  In shared memory it keeps two bits per token of its chunk (the
// prompt has it; it has a bias) and one word (the bias' number, and in the LONG form the row's count), so that
// prompt and biases are looked at once for all rows of the CTA.
//   Each warp copies a block of 1024 logits of a row: the mask's words with one load, the logits that they allow,
// then the stores.  What is listed and allowed is few: the warp then reads, changes and writes those again.  (In the
// copying loop the changes leave no registers for what is fetched ahead: 305 and 114 us instead of the first two below.)
// A row's mask, lengths and words are fetched ahead.
//   A row's own tokens are few (at most 32; beams): there is no barrier; the lanes hold the tokens and change them last.
//   They are many (LONG): the warps take a row together.  Its counts are added to the words beside the copy and taken
//   away after it, so that a history costs its reading, once per chunk of the vocabulary, and integer atomics leave no
//   order to depend on.  Room for more tokens than a row has costs nothing (480 rows of 50,001 with at most 20: 46 to
//   47 us with room for 20, 33 or 2048).
// Measured: 3200 rows of 65,536 fp32 logits in groups of 100, 2% allowed, 180 us (the writes alone 138), in place 172; 480
// rows of 50,001 bf16 logits, prompts of 2000-4000 tokens, histories of 350-700, 300 biases, 54 us, a row's chain of counts,
// barrier, logits, changes and barrier (to bf16 55, in place 54; with 50,000, which gives vectors, 50, 44 and 43); one row of
// 65,536 7 us.
#include <cuda_bf16.h>

#include "bg_internal.h"
#include "bg_ptx.cuh"

namespace bg {
namespace {

constexpr int kLgThreads = 128;
constexpr int kLgWarps = kLgThreads / 32;
constexpr int kChunk = 4096;                         // tokens of a CTA: a block per warp
constexpr int kBlock = 1024;                         // logits that a warp takes at once
// CTAs per SM that the rows are cut to (8: 64 groups of 8 rows of 100,000 bf16 logits 81 us instead of 72; 32: the first case
// above 183 instead of 180).
constexpr int kLgShare = 16;
constexpr int kBlocks = kChunk / kBlock;
static_assert(kChunk / 32 == kLgThreads && kBlocks == kLgWarps, "a bit word per thread, a block per warp");
constexpr int kBiasShift = 18;                       // a row's count, at most 2^16, fits below it
constexpr uint32_t kCountMask = (1u << kBiasShift) - 1;
static_assert(BG_MAX_SEQLEN <= static_cast<int>(kCountMask), "count bits");
static_assert(BG_MAX_BIAS < (1 << (32 - kBiasShift)), "bias numbers");

__device__ __forceinline__ void store_one(float *p, float x) { *p = x; }
__device__ __forceinline__ void store_one(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// N logits as they lie in memory, read where `want` is set (0 elsewhere).  The loads of a block carry predicates and are
// converted later: in branches, each one's conversion waits for it.  64 bytes are the least that memory gives; where a mask
// leaves few of them the usual 128 are too many (3200 rows of 65,536 fp32 logits with 2% allowed: 208 us, so 196).
template <typename T, int N>
struct Raw {
    uint32_t w[N * sizeof(T) / 4 > 0 ? N * sizeof(T) / 4 : 1];
    __device__ __forceinline__ void load(const T *p, bool want)
    {
        const int on = want;
        if constexpr (N * sizeof(T) == 16) {
            w[0] = w[1] = w[2] = w[3] = 0;
            asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t@q ld.global.L2::64B.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
                         : "+r"(w[0]), "+r"(w[1]), "+r"(w[2]), "+r"(w[3])
                         : "l"(p), "r"(on)
                         : "memory");
        } else if constexpr (sizeof(T) == 4) {
            w[0] = 0;
            asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q ld.global.b32 %0, [%1];\n\t}"
                         : "+r"(w[0])
                         : "l"(p), "r"(on)
                         : "memory");
        } else {
            uint16_t h = 0;
            asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q ld.global.b16 %0, [%1];\n\t}"
                         : "+h"(h)
                         : "l"(p), "r"(on)
                         : "memory");
            w[0] = h;
        }
    }
    __device__ __forceinline__ float get(int e) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
        else return __uint_as_float((e & 1) ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
};
template <int N>
__device__ __forceinline__ void store_vec(float *p, const float *x)
{
    if (N == 1) *p = x[0];
    else
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}
template <int N>
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const float *x)
{
    if constexpr (N == 1) *p = __float2bfloat16_rn(x[0]);
    else
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                               pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Whether offsets [a, b) lie within [0, n]; the first ones start at 0 and the last ones end at n.
__device__ __forceinline__ bool offsets_ok(int a, int b, int n, int g, int groups)
{
    return a >= 0 && b >= a && b <= n && (g > 0 || a == 0) && (g < groups - 1 || b == n);
}

// kBlock logits (WHOLE), or the first n of them, by one warp, N side by side per lane and step: -inf where the mask has no
// bit; lane l has the word of tokens 32 l .. 32 l + 31.
template <typename TI, typename TO, int N, bool WHOLE>
__device__ __forceinline__ void copy_block(const TI *in, TO *out, uint32_t words, int n, bool in_place)
{
    constexpr int kStep = 32 * N, kSteps = N == 1 ? 16 : kBlock / kStep;      // steps whose loads are under way together
    constexpr uint32_t kFull = (1u << N) - 1u;
    const int lane = threadIdx.x & 31;
    in += lane * N;
    out += lane * N;
#pragma unroll 1
    for (int s0 = 0; s0 < kBlock; s0 += kSteps * kStep) {
        uint32_t keep = 0;                           // N bits per step
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
            keep |= ((__shfl_sync(0xffffffffu, words, s0 / 32 + k * N + lane * N / 32) >> (lane * N % 32)) & kFull) << (k * N);
        Raw<TI, N> raw[kSteps];
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const uint32_t bits = (keep >> (k * N)) & kFull;
            raw[k].load(in + s0 + k * kStep, bits != 0 && !(in_place && bits == kFull) && (WHOLE || s0 + k * kStep + lane < n));
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const uint32_t bits = (keep >> (k * N)) & kFull;
            if ((in_place && bits == kFull) || (!WHOLE && s0 + k * kStep + lane >= n)) continue;      // in place: they stay
            float x[N];
#pragma unroll
            for (int e = 0; e < N; ++e) x[e] = (bits >> e) & 1u ? raw[k].get(e) : -INFINITY;
            store_vec<N>(out + s0 + k * kStep, x);
        }
    }
}

// N logits (1, 4 or 8 side by side) per lane and step of a warp.  As many CTAs per SM as leave the registers for what is
// fetched ahead: spilled, it is waited for at once (eight CTAs: 3200 rows of 65,536 logits 398 us, seven 180; seven leave
// 72 registers, with two words spilled in <float, float, 4, few> and six in <bf16, bf16, 1, few>).
template <typename TI, typename TO, int N, bool LONG>
__global__ void __launch_bounds__(kLgThreads, LONG ? 6 : 7)
    logits_kernel(const LogitsParams p, int chunks, int rows_per_cta, int row_blocks)
{
    extern __shared__ __align__(16) uint32_t table[];      // [kChunk], where there are biases or counts; cleared as uint4
    __shared__ uint32_t s_prompt[kChunk / 32], s_bias[kChunk / 32], s_own[LONG ? kChunk / 32 : 1];
    grid_dep_launch();
    grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the first chunks first: vocabularies begin with the frequent tokens, which have the most to change
    const int all = static_cast<int>(gridDim.x) / chunks, v0 = static_cast<int>(blockIdx.x) / all * kChunk;
    const int block = static_cast<int>(blockIdx.x) % all;
    const int n = min(kChunk, p.V - v0);
    const int g = block / row_blocks, first = (block - g * row_blocks) * rows_per_cta;
    const int last = min(first + rows_per_cta, p.per);
    const int b0 = warp * kBlock, word0 = b0 / 32 + lane;      // this warp's block, this lane's word
    const bool in_place = static_cast<const void *>(p.in) == p.out;
    const bool lists = LONG || p.prompt || p.bias_tokens, words_kept = LONG || p.bias_tokens;

    // what a row needs: its mask, the number of its own tokens, and the first of them
    constexpr int kHeld = LONG ? 4 : 1;
    struct Row {
        int m, len, t[kHeld];
    };
    auto row_at = [&](int r) { return static_cast<int64_t>(g) * p.per + r; };
    auto fetch = [&](int r) {
        Row R = {-1, 0, {}};
        if (r >= last) return R;
        const int64_t row = row_at(r);
        if (p.mask_index) R.m = p.mask_index[row];
        else if (p.mask) R.m = static_cast<int>(row);
        if (p.own) R.len = p.own_lens ? p.own_lens[row] : p.own_max;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
            const int i = (LONG ? tid : lane) + k * kLgThreads;
            if (i < p.own_max) R.t[k] = p.own[row * p.own_stride + i];
        }
        return R;
    };
    auto words_of = [&](const Row &R) {              // of the mask, for tokens b0 + 32 lane ..
        return R.m >= 0 && R.m < p.num_masks && b0 + 32 * lane < n ? p.mask[R.m * p.mask_stride + v0 / 32 + word0] : ~0u;
    };
    Row cur = fetch(first), next = fetch(first + 1);
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
    // the quotient comes by the reciprocal (below), which is a normal number for these factors alone
    if (p.repetition && !(p.repetition[g] >= 0x1p-126f && p.repetition[g] <= 0x1p126f)) bad |= BG_DEVSTAT_PENALTY;
    if (bad) {                                       // the same for all threads
        if (tid == 0 && p.dev_status) atomicOr(p.dev_status, bad);
        return;
    }
    bool outside = false;                            // a token outside the vocabulary
    if (lists) {
        s_prompt[tid] = 0;
        s_bias[tid] = 0;
        if (LONG) s_own[tid] = 0;
        if (words_kept)
            for (int i = tid; i < kChunk / 4; i += kLgThreads) reinterpret_cast<uint4 *>(table)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
#pragma unroll 4
        for (int i = ba + tid; i < bb; i += kLgThreads) {
            int t = p.bias_tokens[i];
            outside = outside || t < 0 || t >= p.V;
            t -= v0;
            if (t >= 0 && t < n) {
                atomicMax(&table[t], static_cast<uint32_t>(i - ba + 1) << kBiasShift);
                atomicOr(&s_bias[t / 32], 1u << t % 32);
            }
        }
#pragma unroll 8
        for (int i = pa + tid; i < pb; i += kLgThreads) {
            int t = p.prompt[i];
            outside = outside || t < 0 || t >= p.V;
            t -= v0;
            if (t >= 0 && t < n) atomicOr(&s_prompt[t / 32], 1u << t % 32);
        }
        __syncthreads();
    }
    // one division for all (the product's second rounding is 2^-24; a division for each logit needs registers: 279 us instead
    // of 180): without penalties both factors are 1
    const float rho = p.repetition ? p.repetition[g] : 1.f, inv = 1.f / rho;
    const float alpha = p.frequency ? p.frequency[g] : 0.f, beta = p.presence ? p.presence[g] : 0.f;
    // The logits of M tokens t[k] >= 0 of the chunk, c times among the row's own (LONG: as their words say): those that
    // `ok` has are changed, and in the LONG form all counts are taken away.  Each kind of load is made for all of them
    // together, before any store, which the next loads would not pass.
    auto edit = [&](const TI *in, TO *out, auto &t, auto &ok, int c_own) {
        constexpr int M = sizeof(t) / sizeof(t[0]);
        Raw<TI, 1> x[M];
        uint32_t w[M], said[M];
        float bias[M];
#pragma unroll
        for (int k = 0; k < M; ++k) x[k].load(in + t[k], ok[k]);
#pragma unroll
        for (int k = 0; k < M; ++k) {
            w[k] = words_kept && t[k] >= 0 ? table[t[k]] : 0u;
            said[k] = lists && t[k] >= 0 ? s_prompt[t[k] / 32] >> t[k] % 32 & 1u : 0u;
        }
#pragma unroll
        for (int k = 0; k < M; ++k) bias[k] = w[k] >> kBiasShift ? p.bias_values[ba + static_cast<int>(w[k] >> kBiasShift) - 1] : 0.f;
#pragma unroll
        for (int k = 0; k < M; ++k) {
            const int c = LONG ? static_cast<int>(w[k] & kCountMask) : c_own;
            float y = x[k].get(0);
            if (c > 0 || said[k] != 0) y *= y > 0.f ? inv : rho;
            if (c > 0) y -= fmaf(alpha, static_cast<float>(c), beta);
            if (w[k] >> kBiasShift) y += bias[k];
            if (ok[k]) store_one(out + t[k], y);
            if (LONG && c > 0) table[t[k]] = w[k] & ~kCountMask;
        }
    };
    // The tokens of the block whose bits are set, bit e of lane l for token b0 + 32 l + e.  Each lane goes through its own
    // where they are few; where some lane has many (the frequent tokens often lie side by side), all lanes go through
    // the words together.
    auto change = [&](const TI *in, TO *out, uint32_t bits, uint32_t allowed) {
        constexpr int kFew = 3, kWords = 4;
        if (__any_sync(0xffffffffu, __popc(bits) > 3 * kFew)) {
#pragma unroll 1
            for (int l0 = 0; l0 < 32; l0 += kWords) {
                int t[kWords];
                bool ok[kWords];
#pragma unroll
                for (int k = 0; k < kWords; ++k) {
                    const uint32_t some = __shfl_sync(0xffffffffu, bits, l0 + k), free = __shfl_sync(0xffffffffu, allowed, l0 + k);
                    t[k] = (some >> lane) & 1u ? b0 + 32 * (l0 + k) + lane : -1;
                    ok[k] = (some & free) >> lane & 1u;
                }
                edit(in, out, t, ok, 0);
            }
        } else {
#pragma unroll 1
            while (__any_sync(0xffffffffu, bits != 0)) {
                int t[kFew];
                bool ok[kFew];
#pragma unroll
                for (int k = 0; k < kFew; ++k) {
                    const int e = __ffs(bits) - 1;
                    bits &= bits - 1;
                    t[k] = e >= 0 ? 32 * word0 + e : -1;
                    ok[k] = e >= 0 && (allowed >> (e & 31)) & 1u;
                }
                edit(in, out, t, ok, 0);
            }
        }
    };
    auto copy = [&](const TI *in, TO *out, uint32_t words) {
        if (b0 + kBlock <= n) copy_block<TI, TO, N, true>(in + b0, out + b0, words, kBlock, in_place);
        else copy_block<TI, TO, 1, false>(in + b0, out + b0, words, n - b0, in_place);
    };
    // whether the row can be written
    auto row_ok = [&](const Row &R, bool tell) {
        const int wrong = (R.m < -1 || R.m >= p.num_masks ? BG_DEVSTAT_MASK : 0) |
                          (R.len < 0 || R.len > p.own_max ? BG_DEVSTAT_SEQ_TOO_LONG : 0);
        if (wrong && tell && p.dev_status) atomicOr(p.dev_status, wrong);
        return wrong == 0;
    };

    auto in_of = [&](int r) { return static_cast<const TI *>(p.in) + row_at(r) * p.in_stride + v0; };
    auto out_of = [&](int r) { return static_cast<TO *>(p.out) + row_at(r) * p.out_stride + v0; };
    uint32_t words = words_of(cur);
    if constexpr (!LONG) {
        for (int r = first; r < last; ++r) {
            const Row R = cur;
            const uint32_t allowed = words;
            cur = next;
            words = words_of(cur);
            next = fetch(r + 2);
            if (!row_ok(R, tid == 0)) continue;                // the same for all threads
            int t = R.t[0];
            if (lane < R.len && (t < 0 || t >= p.V)) outside = true;
            if (b0 >= n) continue;
            const TI *in = in_of(r);
            TO *out = out_of(r);
            copy(in, out, allowed);
            // the lane's token lies in the block: the last lane of those with the same token changes it
            t -= v0;
            const bool mine = lane < R.len && t >= b0 && t < min(b0 + kBlock, n);
            bool leads = false;
            int c = 0;
            uint32_t bits = lists ? allowed & (s_prompt[word0] | s_bias[word0]) : 0u;
            if (__any_sync(0xffffffffu, mine)) {
                const unsigned same = __match_any_sync(0xffffffffu, mine ? t : -1 - lane);
                c = __popc(same);
                const uint32_t w = __shfl_sync(0xffffffffu, allowed, mine ? (t - b0) / 32 : 0);
                leads = mine && (same >> lane) == 1u && (w >> t % 32) & 1u;
                for (unsigned l = __ballot_sync(0xffffffffu, leads); l != 0; l &= l - 1) {
                    const int u = __shfl_sync(0xffffffffu, t, __ffs(l) - 1);
                    if (u / 32 == word0) bits &= ~(1u << u % 32);
                }
            }
            __syncwarp();                                      // what other lanes have copied is there
            change(in, out, bits, allowed);
            if (leads) {
                const int u[1] = {t};
                const bool yes[1] = {true};
                edit(in, out, u, yes, c);
            }
        }
    } else {
        // counts of a row's own tokens into the words of the chunk
        auto add = [&](int r, const Row &R) {
            auto one = [&](int t) {
                outside = outside || t < 0 || t >= p.V;
                t -= v0;
                if (t >= 0 && t < n) {
                    atomicAdd(&table[t], 1u);
                    atomicOr(&s_own[t / 32], 1u << t % 32);
                }
            };
#pragma unroll
            for (int k = 0; k < kHeld; ++k)
                if (tid + k * kLgThreads < R.len) one(R.t[k]);
            for (int i = tid + kHeld * kLgThreads; i < R.len; i += kLgThreads) one(p.own[row_at(r) * p.own_stride + i]);
        };
        bool ok = row_ok(cur, tid == 0);                       // the same for all threads
        if (ok) {
            add(first, cur);
            if (b0 < n) copy(in_of(first), out_of(first), words);
        }
        for (int r = first; r < last; ++r) {
            const uint32_t allowed = words;
            const bool changes = ok && b0 < n;
            cur = next;
            words = words_of(cur);
            next = fetch(r + 2);
            __syncthreads();                                   // row r's counts are there
            if (changes) {
                const uint32_t own = s_own[word0];
                change(in_of(r), out_of(r), (allowed & (s_prompt[word0] | s_bias[word0])) | own, allowed);
                s_own[word0] = 0;
            }
            ok = r + 1 < last && row_ok(cur, tid == 0);
            if (ok && b0 < n) copy(in_of(r + 1), out_of(r + 1), words);
            __syncthreads();                                   // ... and gone
            if (ok) add(r + 1, cur);
        }
    }
    if (outside && p.dev_status) atomicOr(p.dev_status, BG_DEVSTAT_TOKEN);
}

template <typename TI, typename TO, int N>
cudaError_t launch_typed(const LogitsParams &p, int rows_per_cta, cudaStream_t stream)
{
    const int row_blocks = (p.per + rows_per_cta - 1) / rows_per_cta, chunks = (p.V + kChunk - 1) / kChunk;
    const bool many = p.own && p.own_max > 32;
    const size_t smem = many || p.bias_tokens ? kChunk * sizeof(uint32_t) : 0;
    const int64_t ctas = static_cast<int64_t>(p.groups) * row_blocks * chunks;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    return launch_dependent(many ? logits_kernel<TI, TO, N, true> : logits_kernel<TI, TO, N, false>,
                            dim3(static_cast<unsigned>(ctas)), dim3(kLgThreads), smem, stream, p, chunks, rows_per_cta,
                            row_blocks);
}

}  // namespace

cudaError_t launch_adjust_logits(const LogitsParams &p, int in_dtype, int out_dtype, bool vectors, int nsm, cudaStream_t stream)
{
    // The rows of a group are cut to kLgShare CTAs per SM, as long as a CTA has four of them, and four logits for each
    // token of the lists that it has to look at (eight: 480 rows with prompts of 3000 tokens 69 us instead of 54; two: the same
    // 54, and one group of 480 rows of 50,000 with a prompt of 8000 55 instead of 91).
    const int64_t chunks = (p.V + kChunk - 1) / kChunk, listed = p.total_prompt / p.groups + p.total_bias / p.groups;
    int per = p.per;
    while (per >= 8 && per / 2 * static_cast<int64_t>(kChunk) >= 4 * listed && chunks * p.groups * ((p.per + per - 1) / per) < kLgShare * nsm)
        per = (per + 1) / 2;
    if (in_dtype == BG_DTYPE_F32)
        return vectors ? launch_typed<float, float, 4>(p, per, stream) : launch_typed<float, float, 1>(p, per, stream);
    if (out_dtype == BG_DTYPE_F32)
        return vectors ? launch_typed<__nv_bfloat16, float, 8>(p, per, stream)
                       : launch_typed<__nv_bfloat16, float, 1>(p, per, stream);
    return vectors ? launch_typed<__nv_bfloat16, __nv_bfloat16, 8>(p, per, stream)
                   : launch_typed<__nv_bfloat16, __nv_bfloat16, 1>(p, per, stream);
}

}  // namespace bg
