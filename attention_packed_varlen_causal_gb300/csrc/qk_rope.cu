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
// Memory bounds it: every element is read once and written once, about 130 instructions of a warp for 2 KB.
// A warp takes a token (or a part of its heads, where there are few tokens), so that its angles are computed
// once for all heads.  Eight lanes (four at d = 64) hold a head, each 16 of its elements that make up eight
// whole pairs with the frequencies 8 j .. 8 j + 7 in either layout: the rotation needs no exchange, the norm
// a sum over the lanes of a head.
#include <cuda_bf16.h>

#include "bg_internal.h"
#include "bg_ptx.cuh"

namespace bg {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeCtas = 3;              // per SM
constexpr int kRopeBatch = 2;             // head rounds whose loads are under way together

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
    constexpr int kLanes = D / 16;                 // lanes of a head
    constexpr int kHeads = 32 / kLanes;            // heads of a round
    constexpr int kOwn = D / 64;                   // frequencies whose angle a lane computes
    const int lane = threadIdx.x & 31, j = lane % kLanes, sub = lane / kLanes;
    const int half = p.rot / 2;
    grid_dep_launch();
    grid_dep_wait();

    // elements lo .. lo + 7 and hi .. hi + 7 of a head are this lane's
    const bool turns = 8 * j < half;
    const int lo = INTERLEAVED || !turns ? 16 * j : 8 * j;
    const int hi = INTERLEAVED || !turns ? 16 * j + 8 : 8 * j + half;
    uint4 wq[2], wk[2];
    if (NORM) {
        wq[0] = *reinterpret_cast<const uint4 *>(p.q_weight + lo);
        wq[1] = *reinterpret_cast<const uint4 *>(p.q_weight + hi);
        wk[0] = *reinterpret_cast<const uint4 *>(p.k_weight + lo);
        wk[1] = *reinterpret_cast<const uint4 *>(p.k_weight + hi);
    }
    // f / (2 pi) as a sum of two numbers
    constexpr double kTurn = 0.15915494309189533577;
    constexpr float kTurnHi = static_cast<float>(kTurn), kTurnLo = static_cast<float>(kTurn - kTurnHi);
    float f_hi[kOwn], f_lo[kOwn];
    int axis[kOwn];
#pragma unroll
    for (int m = 0; m < kOwn; ++m) {
        const int i = lane * kOwn + m;
        const float f = i < half ? p.inv_freq[i] : 0.f;
        axis[m] = p.axis[i];
        f_hi[m] = f * kTurnHi;
        f_lo[m] = fmaf(f, kTurnLo, fmaf(f, kTurnHi, -f_hi[m]));
    }

    const int n_heads = p.Hq + p.Hkv + (p.v ? p.Hkv : 0);
    const int64_t units = p.rows * p.parts, stride = static_cast<int64_t>(gridDim.x) * (kRopeThreads / 32);
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5); u < units; u += stride) {
        const int64_t row = u / p.parts;
        const int part = static_cast<int>(u - row * p.parts);
        const int64_t place = row / p.rows_per_pos;
        float c[8], s[8];
        {
            float2 cs[kOwn];
#pragma unroll
            for (int m = 0; m < kOwn; ++m)
                cs[m] = cos_sin(p.positions[axis[m] * p.places + place] + p.step, f_hi[m], f_lo[m]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {          // frequency 8 j + i is lane (8 j + i) / kOwn's
                const int src = (8 * j + i) / kOwn;
                c[i] = __shfl_sync(0xffffffffu, cs[i % kOwn].x, src) * p.rope_scale;
                s[i] = __shfl_sync(0xffffffffu, cs[i % kOwn].y, src) * p.rope_scale;
            }
        }
        for (int h0 = part * kHeads; h0 < n_heads; h0 += kRopeBatch * p.parts * kHeads) {
            uint4 a[kRopeBatch], b[kRopeBatch];
            __nv_bfloat16 *dst[kRopeBatch];
#pragma unroll
            for (int k = 0; k < kRopeBatch; ++k) {
                const int h = h0 + k * p.parts * kHeads + sub;
                const __nv_bfloat16 *src;
                if (h < p.Hq) {
                    src = p.q + row * p.q_stride + h * D;
                    dst[k] = p.q_out + (row * p.Hq + h) * D;
                } else if (h < p.Hq + p.Hkv) {
                    src = p.k + row * p.k_stride + (h - p.Hq) * D;
                    dst[k] = p.k_out + row * p.kv_out_stride + (h - p.Hq) * D;
                } else {
                    src = p.v + row * p.v_stride + (h - p.Hq - p.Hkv) * D;
                    dst[k] = p.v_out + row * p.kv_out_stride + (h - p.Hq - p.Hkv) * D;
                }
                if (h < n_heads) {
                    a[k] = *reinterpret_cast<const uint4 *>(src + lo);
                    b[k] = *reinterpret_cast<const uint4 *>(src + hi);
                } else {
                    a[k] = b[k] = make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll
            for (int k = 0; k < kRopeBatch; ++k) {
                const int hr = h0 + k * p.parts * kHeads;     // the round's first head
                const int h = hr + sub;
                if (hr < p.Hq + p.Hkv) {
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
                        float w[16];
                        const bool is_q = h < p.Hq;
                        unpack(is_q ? wq[0] : wk[0], w);
                        unpack(is_q ? wq[1] : wk[1], w + 8);
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] *= inv * (w[i] + p.weight_offset);
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
                            const int e = 2 * i, f = 2 * i + 1;
                            o[i] = pack_bf16x2(x[e] * c[e] - x[8 + e] * s[e], x[f] * c[f] - x[8 + f] * s[f]);
                            o[4 + i] = pack_bf16x2(x[8 + e] * c[e] + x[e] * s[e], x[8 + f] * c[f] + x[f] * s[f]);
                        }
                    }
                    if (h < p.Hq + p.Hkv) {
                        a[k] = make_uint4(o[0], o[1], o[2], o[3]);
                        b[k] = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
                if (h < n_heads) {
                    *reinterpret_cast<uint4 *>(dst[k] + lo) = a[k];
                    *reinterpret_cast<uint4 *>(dst[k] + hi) = b[k];
                }
            }
        }
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
    const int rounds = (p.Hq + 2 * p.Hkv) * head_dim / 512;      // of a token; one at least
    // Few tokens: the heads of a token over several warps, as long as a warp per SM sub-partition and more is free.
    p.parts = 1;
    while (2 * p.parts <= rounds && 2 * p.parts * p.rows <= nsm * 32) p.parts *= 2;
    const int64_t warps = kRopeThreads / 32, ctas = (p.rows * p.parts + warps - 1) / warps;
    const int grid = static_cast<int>(ctas < nsm * kRopeCtas ? ctas : nsm * kRopeCtas);
    return head_dim == 128 ? launch_d<128>(p, interleaved, grid, stream) : launch_d<64>(p, interleaved, grid, stream);
}

}  // namespace bg
