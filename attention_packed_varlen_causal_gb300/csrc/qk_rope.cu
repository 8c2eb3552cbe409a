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
// Memory bounds it: every element is read once and written once.  Eight lanes (four at d = 64) take a token, a warp
// four (eight) of them, and go through the heads.  A lane holds 16 elements of a head that make up eight whole pairs,
// with the frequencies 8 j .. 8 j + 7 in either layout: it computes their angles once for all heads of its token, the
// rotation needs no exchange, and the norm a sum over the lanes of a head.  (A warp for one token, with each angle
// computed once and shuffled to the lanes that need it, and heads left over in the last round: 70,375 tokens of 16/8
// heads of 128 196 us, 23,041 of 14/2 heads of 64 31 us.)  Where there are few tokens, their heads are dealt out to
// several warps.
#include <cuda_bf16.h>

#include "bg_internal.h"
#include "bg_ptx.cuh"

namespace bg {
namespace {

constexpr int kRopeThreads = 256;
#ifndef CTAS
#define CTAS 2
#define BATCH 2
#endif
constexpr int kRopeCtas = CTAS;              // per SM
constexpr int kRopeBatch = BATCH;             // heads whose loads are under way together

__device__ __forceinline__ void unpack(const uint4 &v, float *x)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// cos and sin of 2 pi * pos * (hi + lo).  The products with the upper and the lower bits of pos are held exactly as a
// rounded value and its error (both factors have few enough bits), and whole turns are dropped exactly, so that the
// angle is off by about 2^-20 for positions up to 2^24, and 2^-17 for all others (of frequencies up to 1).
__device__ __forceinline__ float2 cos_sin(int32_t pos, float hi, float lo)
{
    const float up = static_cast<float>(pos & ~0xfff), low = static_cast<float>(pos & 0xfff);
    const float t1 = up * hi, t2 = low * hi, t3 = static_cast<float>(pos) * lo;
    const float e1 = fmaf(up, hi, -t1), e2 = fmaf(low, hi, -t2);
    float r = (t1 - rintf(t1)) + (t2 - rintf(t2));
    r += (e1 - rintf(e1)) + e2 + (t3 - rintf(t3));
    r = (r - rintf(r)) * 6.2831853071795864769f;
    // [-pi, pi], where the fast forms are off by at most 2^-21; outputs are rounded to 2^-9 of theirs
    return make_float2(__cosf(r), __sinf(r));
}

template <int D, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int kLanes = D / 16;                 // lanes of a token
    constexpr int kTokens = 32 / kLanes;           // tokens of a warp
    const int lane = threadIdx.x & 31, j = lane % kLanes, sub = lane / kLanes;
    const int half = p.rot / 2;
    grid_dep_launch();
    grid_dep_wait();

    // elements lo .. lo + 7 and hi .. hi + 7 of a head are this lane's
    const bool turns = 8 * j < half;
    const int lo = INTERLEAVED || !turns ? 16 * j : 8 * j;
    const int hi = INTERLEAVED || !turns ? 16 * j + 8 : 8 * j + half;
    float f[8];
    uint32_t axes = 0;                             // two bits each
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[i] = turns ? p.inv_freq[8 * j + i] : 0.f;
        axes |= static_cast<uint32_t>(p.axis[8 * j + i]) << (2 * i);
    }

    const int n_heads = p.Hq + p.Hkv + (p.v ? p.Hkv : 0);
    const int64_t units = (p.rows + kTokens - 1) / kTokens * p.parts;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kRopeThreads / 32);
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5); u < units; u += stride) {
        const int64_t first = u / p.parts * kTokens;
        const int part = static_cast<int>(u % p.parts);
        const int begin = part * n_heads / p.parts, end = (part + 1) * n_heads / p.parts;
        const bool live = first + sub < p.rows;
        const int64_t row = live ? first + sub : p.rows - 1;
        float c[8], s[8];
        if (begin < p.Hq + p.Hkv) {
            const int64_t place = row / p.rows_per_pos;
            int32_t pos[BG_MAX_AXES];
#pragma unroll
            for (int a = 0; a < BG_MAX_AXES; ++a) pos[a] = a < p.num_axes ? p.positions[a * p.places + place] : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                int32_t at = pos[0];
                if (p.num_axes > 1) {
                    const uint32_t a = (axes >> (2 * i)) & 3u;
                    at = a < 2 ? (a == 0 ? pos[0] : pos[1]) : (a == 2 ? pos[2] : pos[3]);
                }
                // f / (2 pi) as a sum of two numbers
                constexpr double kTurn = 0.15915494309189533577;
                constexpr float kTurnHi = static_cast<float>(kTurn), kTurnLo = static_cast<float>(kTurn - kTurnHi);
                const float f_hi = f[i] * kTurnHi, f_lo = fmaf(f[i], kTurnLo, fmaf(f[i], kTurnHi, -f_hi));
                const float2 cs = cos_sin(at + p.step, f_hi, f_lo);
                c[i] = cs.x * p.rope_scale;
                s[i] = cs.y * p.rope_scale;
            }
        }
        // heads [from, to) of q or k, kRopeBatch at a time; V: copied
        auto heads = [&](const __nv_bfloat16 *src, __nv_bfloat16 *dst, const __nv_bfloat16 *weight, int from, int to, bool copied) {
            float w[NORM ? 16 : 1];
            if (NORM && !copied && from < to) {
                unpack(*reinterpret_cast<const uint4 *>(weight + lo), w);
                unpack(*reinterpret_cast<const uint4 *>(weight + hi), w + (NORM ? 8 : 0));
#pragma unroll
                for (int i = 0; i < (NORM ? 16 : 1); ++i) w[i] += p.weight_offset;
            }
#pragma unroll 1
            for (int h0 = from; h0 < to; h0 += kRopeBatch) {
                uint4 a[kRopeBatch], b[kRopeBatch];
#pragma unroll
                for (int k = 0; k < kRopeBatch; ++k) {
                    const __nv_bfloat16 *at = src + min(h0 + k, to - 1) * D;
                    a[k] = *reinterpret_cast<const uint4 *>(at + lo);
                    b[k] = *reinterpret_cast<const uint4 *>(at + hi);
                }
#pragma unroll
                for (int k = 0; k < kRopeBatch; ++k) {
                    if (h0 + k >= to) break;
                    if (!copied) {
                        float x[16];
                        unpack(a[k], x);
                        unpack(b[k], x + 8);
                        if (NORM) {
                            float sum = 0.f;
#pragma unroll
                            for (int i = 0; i < 16; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
                            for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                            const float inv = rsqrtf(fmaf(sum, 1.f / D, p.eps));
#pragma unroll
                            for (int i = 0; i < 16; ++i) x[i] *= inv * w[NORM ? i : 0];
                        }
                        uint32_t o[8];
                        if (!turns) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
                        } else if (INTERLEAVED) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                o[i] = pack_bf16x2(x[2 * i] * c[i] - x[2 * i + 1] * s[i], x[2 * i + 1] * c[i] + x[2 * i] * s[i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int e = 2 * i, g = 2 * i + 1;
                                o[i] = pack_bf16x2(x[e] * c[e] - x[8 + e] * s[e], x[g] * c[g] - x[8 + g] * s[g]);
                                o[4 + i] = pack_bf16x2(x[8 + e] * c[e] + x[e] * s[e], x[8 + g] * c[g] + x[g] * s[g]);
                            }
                        }
                        a[k] = make_uint4(o[0], o[1], o[2], o[3]);
                        b[k] = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                    if (live) {
                        __nv_bfloat16 *at = dst + (h0 + k) * D;
                        *reinterpret_cast<uint4 *>(at + lo) = a[k];
                        *reinterpret_cast<uint4 *>(at + hi) = b[k];
                    }
                }
            }
        };
        const int k0 = p.Hq, v0 = p.Hq + p.Hkv;
        heads(p.q + row * p.q_stride, p.q_out + row * p.Hq * D, p.q_weight, begin, min(end, k0), false);
        heads(p.k + row * p.k_stride, p.k_out + row * p.kv_out_stride, p.k_weight, max(begin, k0) - k0, min(end, v0) - k0, false);
        heads(p.v + row * p.v_stride, p.v_out + row * p.kv_out_stride, nullptr, max(begin, v0) - v0, end - v0, true);
    }
}

template <int D>
cudaError_t launch_d(const RopeParams &p, bool interleaved, int grid, cudaStream_t stream)
{
    const bool norm = p.q_weight != nullptr;
    auto kern = interleaved ? (norm ? rope_kernel<D, true, true> : rope_kernel<D, true, false>)
                            : (norm ? rope_kernel<D, false, true> : rope_kernel<D, false, false>);
    return launch_dependent(kern, dim3(grid), dim3(kRopeThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_qk_rope(RopeParams p, int head_dim, bool interleaved, int nsm, cudaStream_t stream)
{
    const int heads = p.Hq + p.Hkv + (p.v ? p.Hkv : 0);
    const int64_t tokens = 512 / head_dim, groups = (p.rows + tokens - 1) / tokens;      // of a warp
    // Few tokens: their heads over several warps, two heads to each at least, as long as the card has room for them.
    p.parts = 1;
    while (4 * p.parts <= heads && 2 * p.parts * groups <= nsm * kRopeCtas * (kRopeThreads / 32)) p.parts *= 2;
    const int64_t warps = kRopeThreads / 32, ctas = (groups * p.parts + warps - 1) / warps;
    const int grid = static_cast<int>(ctas < nsm * kRopeCtas ? ctas : nsm * kRopeCtas);
    return head_dim == 128 ? launch_d<128>(p, interleaved, grid, stream) : launch_d<64>(p, interleaved, grid, stream);
}

}  // namespace bg
