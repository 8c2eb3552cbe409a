// qk_rope.cu -- norm of every head of Q and K and the rotation by the token's position.
//
// "SLM 生成式高并发推理引擎：延迟约束下的有效吞吐优化", section 1.2: the attention calls read packed
// tokens; their Q and K arrive normed and rotated.  For a head x of a token at positions pos[0..A):
//     y      = x / sqrt(mean(x^2) + eps) * (offset + w)                  (with weights; else y = x)
//     angle  = pos[axis(i)] * f_i,  c_i = s cos(angle), s_i = s sin(angle),   i < rot / 2
//     out_a  = y_a c_i - y_b s_i,   out_b = y_b c_i + y_a s_i
// over the pairs (a, b) = (i, i + rot / 2), or (2 i, 2 i + 1) where they are interleaved; dimensions from rot on
// keep y.  V is copied beside them, out of the fused projection's rows.  All in fp32, rounded to bf16 once.
//
// Memory bounds it: every element is read once and written once.  A warp takes a token (or a part of its heads, where
// there are few tokens) in rounds of 1 KB, whole rows one after the other: four tokens at a time, 256 bytes of each, reach
// 0.63 of the copy rate on rows of 12 KB, this 0.96.  Eight lanes (four at d = 64) hold a head, each 16 of its elements
// that make up eight whole pairs in either layout, so that the rotation needs no exchange and the norm a sum over the
// lanes of a head.  The angles of a token are computed once, two (one) per lane, and shuffled to the lanes that need them.
// Each lane's elements come through shared memory by copies of its own, kRopeAhead rounds ahead, without a barrier.
// Measured: 70,375 tokens of 16/8 heads of 128 176 us, 6.5 TB/s; 32,768 of 32/8 heads without a norm 124 us, 6.5 TB/s;
// 23,041 of 14/2 heads of 64 26 us, 4.0 TB/s (the latency of a token's three rounds, the last of which holds two heads).
#include <cuda_bf16.h>

#include "bg_internal.h"
#include "bg_ptx.cuh"

namespace bg {
namespace {

// Warps of a CTA: ten where many tokens are normed, which need issue slots (the first case above 176 us; with eight 183);
// eight where memory alone counts (the second one 124; with ten 134) or few tokens (392 tokens 4.6; with ten 5.4).  Around the
// border, 24,320 tokens, eight and ten take: 16/8 heads of 128 46.6 and 48.1 us for 16,001 tokens, 57.5 and 56.7 for 20,001,
// 68.3 and 66.7 for 24,400, 77.1 and 74.8 for 28,001; 14/2 heads of 64 22.5 and 24.0 for 20,001, 27.2 and 27.8 for 24,400,
// 38.0 and 38.6 for 36,001.
constexpr int kRopeFew = 8, kRopeMany = 10;
constexpr int kRopeCtas = 2;              // per SM (three of eight warps leave 80 registers, with spills: 195 us instead of 183)
// Rounds whose copies are under way, per warp.  Not more: with three the second case takes 134 us, the first 200 (with eight
// warps 192).
constexpr int kRopeAhead = 2;

__device__ __forceinline__ void unpack(const uint4 &v, float *x)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// cos and sin of 2 pi * pos * (hi + lo).  Whole turns are taken from the products with the upper and the lower bits of pos
// before these are rounded (a far position's first one is exact then, and may hold some more).  What is left: the three
// fractions and the last one's sum round by 2^-25 or 2^-26 of a turn, their sum by 2^-25 and 2^-24, 11 * 2^-26 together; lo
// rounds by 2^-52 (times pos); 2 pi and its product by 2^-22.  For frequencies up to 1 the angle is off by less than 2^-19
// for positions up to 2^24 and 2^-17 for all others.
__device__ __forceinline__ float2 cos_sin(int32_t pos, float hi, float lo)
{
    const float up = static_cast<float>(pos & ~0xfff), low = static_cast<float>(pos & 0xfff);
    const float f1 = fmaf(up, hi, -rintf(up * hi)), f2 = fmaf(low, hi, -rintf(low * hi));
    const float f3 = fmaf(up, lo, -rintf(up * lo));
    float r = ((f1 - rintf(f1)) + f2) + fmaf(low, lo, f3);
    r = (r - rintf(r)) * 6.2831853071795864769f;
    // [-pi, pi], where the fast forms are off by at most 2^-21; outputs are rounded to 2^-8 of theirs
    return make_float2(__cosf(r), __sinf(r));
}

// The two runs of 8 elements of a head, at a and b, that lane j of the head's D / 16 lanes holds, whether they turn, and
// the first of the four frequencies of each.  The lanes' runs lie side by side in memory.  Halves: the runs are the two
// sides of pairs i .. i + 7 (where they turn).  Interleaved: each holds four pairs.
template <int D, bool INTERLEAVED>
struct Share {
    int a, b, fa, fb;
    bool ta, tb;
    __device__ Share(int j, int half)
    {
        constexpr int kLanes = D / 16;
        if (INTERLEAVED) {
            a = 8 * j;
            b = 8 * (j + kLanes);
            ta = a < 2 * half;
            tb = b < 2 * half;
            fa = 4 * j;
            fb = 4 * (j + kLanes);
        } else {
            const int n = half / 8;                // lanes that turn
            ta = tb = j < n;
            a = 8 * (j < n ? j : j + n);
            b = 8 * (j < n ? j + n : j + kLanes);
            fa = 8 * j;
            fb = 8 * j + 4;
        }
    }
};

// Norm over the lanes of a head, then the rotation of the pairs that this lane holds.  All lanes of the warp call it.
template <int D, bool INTERLEAVED, bool NORM>
__device__ __forceinline__ void turn_head(uint4 &a, uint4 &b, const float *w, const float *c, const float *s,
                                          const Share<D, INTERLEAVED> &at, float eps)
{
    float x[16];
    unpack(a, x);
    unpack(b, x + 8);
    if (NORM) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
        for (int o = 1; o < D / 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = rsqrtf(fmaf(sum, 1.f / D, eps));
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= inv * w[i];
    }
    if (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = x[2 * i], v = x[2 * i + 1];
            if (i < 4 ? at.ta : at.tb) {
                x[2 * i] = u * c[i] - v * s[i];
                x[2 * i + 1] = v * c[i] + u * s[i];
            }
        }
    } else if (at.ta) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = x[i], v = x[8 + i];
            x[i] = u * c[i] - v * s[i];
            x[8 + i] = v * c[i] + u * s[i];
        }
    }
    a = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    b = make_uint4(pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]), pack_bf16x2(x[12], x[13]), pack_bf16x2(x[14], x[15]));
}

// f / (2 pi) as a sum of two numbers, the lower one at most half a step of the upper one: otherwise its own rounding,
// times a far position, would be four times as large.
__device__ __forceinline__ float2 per_turn(float f)
{
    constexpr double kTurn = 0.15915494309189533577;
    constexpr float kHi = static_cast<float>(kTurn), kLo = static_cast<float>(kTurn - kHi);
    constexpr float kRest = static_cast<float>(kTurn - kHi - kLo);
    const float h = f * kHi, e = fmaf(f, kHi, -h);            // h + e is f * kHi
    const float p = f * kLo, pe = fmaf(f, kRest, fmaf(f, kLo, -p));
    const float s = e + p, b = s - e, se = (e - (s - b)) + (p - b);      // s + se is e + p
    const float hi = h + s;
    return make_float2(hi, (s - (hi - h)) + (se + pe));
}

__device__ __forceinline__ void copy_async(void *smem, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(src) : "memory");
}

template <int D, bool INTERLEAVED, bool NORM, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, kRopeCtas) rope_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int kLanes = D / 16;                 // lanes of a head
    constexpr int kHeads = 32 / kLanes;            // heads of a round
    constexpr int kOwn = D / 64;                   // frequencies whose angle a lane computes
    extern __shared__ uint4 s_ring[];              // [warp][slot][2][lane]: what a lane copies, it alone reads
    const int lane = threadIdx.x & 31, j = lane % kLanes, sub = lane / kLanes;
    uint4 *ring = s_ring + (threadIdx.x >> 5) * (kRopeAhead * 64) + lane;
    const int half = p.rot / 2;
    grid_dep_launch();
    grid_dep_wait();

    const Share<D, INTERLEAVED> share(j, half);
    const int lo = share.a, hi = share.b;
    const int k0 = p.Hq, v0 = p.Hq + p.Hkv, n_heads = v0 + (p.v ? p.Hkv : 0);
    // unit u: token u / parts, and its rounds u % parts, + parts, ...
    const int rounds = (n_heads + kHeads - 1) / kHeads;
    const int64_t units = p.rows * p.parts, stride = static_cast<int64_t>(gridDim.x) * WARPS;
    const int64_t u0 = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);

    // ---- copies, kRopeAhead rounds ahead; a group for each round, also behind the last one
    int64_t u_in = u0;
    int round_in = 0, slot_in = 0;
    const __nv_bfloat16 *src_q = nullptr, *src_k = nullptr, *src_v = nullptr;
    auto start_in = [&] {
        if (u_in >= units) return;
        const int64_t row = u_in / p.parts;
        round_in = static_cast<int>(u_in - row * p.parts);
        src_q = p.q + row * p.q_stride;
        src_k = p.k + row * p.k_stride - k0 * D;
        src_v = p.v + row * p.v_stride - v0 * D;
    };
    auto fetch = [&] {
        if (u_in < units) {
            const int h = round_in * kHeads + sub;
            if (h < n_heads) {
                const __nv_bfloat16 *at = (h < k0 ? src_q : h < v0 ? src_k : src_v) + h * D;
                copy_async(ring + slot_in * 64, at + lo);
                copy_async(ring + slot_in * 64 + 32, at + hi);
            }
            round_in += p.parts;
            if (round_in >= rounds) {
                u_in += stride;
                start_in();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (++slot_in == kRopeAhead) slot_in = 0;
    };
    start_in();
#pragma unroll 1
    for (int i = 0; i < kRopeAhead; ++i) fetch();

    float2 f[kOwn];
    int axis[kOwn];
#pragma unroll
    for (int m = 0; m < kOwn; ++m) {
        const int i = lane * kOwn + m;
        f[m] = per_turn(i < half ? p.inv_freq[i] : 0.f);
        axis[m] = p.axis[i];
    }
    // offset + weight of the elements that lane j of a head holds, four at (part * kLanes + j)
    __shared__ float4 s_weight[NORM ? 2 : 1][NORM ? 4 * kLanes : 1];
    if (NORM) {
        if (threadIdx.x < 2 * kLanes) {
            const int t = threadIdx.x % kLanes, k = threadIdx.x / kLanes;
            const Share<D, INTERLEAVED> of(t, half);
            const __nv_bfloat16 *weight = k == 0 ? p.q_weight : p.k_weight;
            float w[16];
            unpack(*reinterpret_cast<const uint4 *>(weight + of.a), w);
            unpack(*reinterpret_cast<const uint4 *>(weight + of.b), w + 8);
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] += p.weight_offset;
#pragma unroll
            for (int i = 0; i < 4; ++i) s_weight[k][i * kLanes + t] = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
        __syncthreads();
    }
    int32_t next[kOwn];                            // positions, fetched a unit ahead
    auto places = [&](int64_t u) {
        if (u >= units) return;
        const int64_t place = u / p.parts / p.rows_per_pos;
#pragma unroll
        for (int m = 0; m < kOwn; ++m) next[m] = p.positions[axis[m] * p.places + place];
    };
    places(u0);
    int slot = 0;
    for (int64_t u = u0; u < units; u += stride) {
        const int64_t row = u / p.parts;
        float c[8], s[8];
        {
            float2 cs[kOwn];
#pragma unroll
            for (int m = 0; m < kOwn; ++m) cs[m] = cos_sin(static_cast<int32_t>(static_cast<uint32_t>(next[m]) + p.step), f[m].x, f[m].y);
            places(u + stride);
#pragma unroll
            for (int i = 0; i < 8; ++i) {          // frequency e is lane e / kOwn's
                const int src = ((i < 4 ? share.fa : share.fb) + i % 4) / kOwn;
                c[i] = __shfl_sync(0xffffffffu, cs[i % kOwn].x, src) * p.rope_scale;
                s[i] = __shfl_sync(0xffffffffu, cs[i % kOwn].y, src) * p.rope_scale;
            }
        }
        __nv_bfloat16 *dst_q = p.q_out + row * k0 * D, *dst_k = p.k_out + row * p.kv_out_stride - k0 * D;
        __nv_bfloat16 *dst_v = p.v_out + row * p.kv_out_stride - v0 * D;
#pragma unroll 1
        for (int r = static_cast<int>(u - row * p.parts); r < rounds; r += p.parts) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kRopeAhead - 1) : "memory");
            uint4 a = ring[slot * 64], b = ring[slot * 64 + 32];
            if (++slot == kRopeAhead) slot = 0;
            const int h = r * kHeads + sub;
            if (r * kHeads < v0) {                 // (V's heads of this round keep what they are)
                float w[16];
                if (NORM) {
                    const float4 *from = s_weight[h < k0 ? 0 : 1] + j;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 v = from[i * kLanes];
                        w[4 * i] = v.x;
                        w[4 * i + 1] = v.y;
                        w[4 * i + 2] = v.z;
                        w[4 * i + 3] = v.w;
                    }
                }
                uint4 ta = a, tb = b;
                turn_head<D, INTERLEAVED, NORM>(ta, tb, w, c, s, share, p.eps);
                if (h < v0) {
                    a = ta;
                    b = tb;
                }
            }
            if (h < n_heads) {
                __nv_bfloat16 *at = (h < k0 ? dst_q : h < v0 ? dst_k : dst_v) + h * D;
                *reinterpret_cast<uint4 *>(at + lo) = a;
                *reinterpret_cast<uint4 *>(at + hi) = b;
            }
            fetch();                               // into the slot that has been read
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int D, bool INTERLEAVED, bool NORM, int WARPS>
cudaError_t launch_warps(RopeParams &p, int nsm, cudaStream_t stream)
{
    // Few tokens: their heads over several warps, a round to each at least, as long as the card has room for them.
    const int64_t room = static_cast<int64_t>(nsm) * kRopeCtas * WARPS;
    const int heads = p.Hq + p.Hkv + (p.v ? p.Hkv : 0), rounds = (heads * D + 511) / 512;
    p.parts = 1;
    while (2 * p.parts <= rounds && 2 * p.parts * p.rows <= room) p.parts *= 2;
    const int64_t ctas = (p.rows * p.parts + WARPS - 1) / WARPS;
    const int grid = static_cast<int>(ctas < nsm * kRopeCtas ? ctas : nsm * kRopeCtas);
    constexpr int kSmem = WARPS * kRopeAhead * 1024;
    static_assert(kSmem <= 48 * 1024, "no larger limit to be asked for");
    return launch_dependent(rope_kernel<D, INTERLEAVED, NORM, WARPS>, dim3(grid), dim3(32 * WARPS), kSmem, stream, p);
}

template <int D, bool INTERLEAVED, bool NORM>
cudaError_t launch_one(RopeParams &p, int nsm, cudaStream_t stream)
{
    // many: eight tokens and more for each warp
    if (NORM && p.rows >= static_cast<int64_t>(8) * nsm * kRopeCtas * kRopeMany)
        return launch_warps<D, INTERLEAVED, NORM, NORM ? kRopeMany : kRopeFew>(p, nsm, stream);
    return launch_warps<D, INTERLEAVED, NORM, kRopeFew>(p, nsm, stream);
}

}  // namespace

cudaError_t launch_qk_rope(RopeParams p, int head_dim, bool interleaved, int nsm, cudaStream_t stream)
{
    const bool norm = p.q_weight != nullptr;
    if (head_dim == 128)
        return interleaved ? (norm ? launch_one<128, true, true>(p, nsm, stream) : launch_one<128, true, false>(p, nsm, stream))
                           : (norm ? launch_one<128, false, true>(p, nsm, stream) : launch_one<128, false, false>(p, nsm, stream));
    return interleaved ? (norm ? launch_one<64, true, true>(p, nsm, stream) : launch_one<64, true, false>(p, nsm, stream))
                       : (norm ? launch_one<64, false, true>(p, nsm, stream) : launch_one<64, false, false>(p, nsm, stream));
}

}  // namespace bg
