// rope.cu -- rotary positions of a step's queries and keys (definition:
// include/dspark.h).
//
// Pair i of a token at position m is turned by theta = 2 pi frac(m F_i / 2^64),
// F_i the turns per position in units of 2^-64.  m F_i is a 64-bit integer
// product that wraps at whole turns, so what is left is exact to 2^-64 m of a
// turn wherever the token stands; its upper 32 bits, as a signed fraction of a half
// turn, are rounded once to fp32 (2^-25 of it) for the sine and cosine.  An fp32
// product m * f would be off by 2^-24 m f radians: 0.06 at position 10^6.
//
// Bytes bound it: a token's rows are read and written once, its sines and
// cosines are formed once for all heads, by the block, and kept in shared memory.
#include <cuda_bf16.h>

#include "pdl.cuh"
#include "serve.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;

struct Vec8 { float x[8]; };

__device__ __forceinline__ Vec8 load8(const float* p) {
    Vec8 r;
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    r.x[0] = a.x; r.x[1] = a.y; r.x[2] = a.z; r.x[3] = a.w; r.x[4] = b.x; r.x[5] = b.y; r.x[6] = b.z; r.x[7] = b.w;
    return r;
}
__device__ __forceinline__ Vec8 load8(const uint16_t* p) {
    Vec8 r;
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        r.x[2 * j] = __uint_as_float(w[j] << 16);
        r.x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
    return r;
}
__device__ __forceinline__ void store8(float* p, const Vec8& v) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v.x[0], v.x[1], v.x[2], v.x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v.x[4], v.x[5], v.x[6], v.x[7]);
}
__device__ __forceinline__ void store8(uint16_t* p, const Vec8& v) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v.x[2 * j + 1]), "f"(v.x[2 * j]));
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) {
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.bf16.f32 h, %1;\n\tmov.b16 %0, h;\n\t}" : "=h"(*p) : "f"(x));
}

// kVector: how an item covers its entries.  kHalves: 8 pairs (i, i + r/2), two
// vectors.  kPairs: 4 neighbouring pairs, one vector.  kSingle: one pair, where
// the halves or the pairs do not fill vectors of 8.
enum class Items { kHalves, kPairs, kSingle };

template <typename T, Items kItems>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
    extern __shared__ float2 turn[];              // [tokens][rotary / 2]: cos, sin
    grid_dependency_wait();
    const int half = p.rotary / 2, heads = p.Hq + p.Hkv;
    for (int t0 = blockIdx.x * p.side; t0 < p.T; t0 += gridDim.x * p.side) {
        const int n = min(p.side, p.T - t0);
        __syncthreads();
        for (int i = threadIdx.x; i < n * half; i += kThreads) {
            const int t = p.by_half(i), pair = i - t * half, pos = __ldg(p.positions + t0 + t);
            const uint64_t frac = (uint64_t)(uint32_t)max(pos, 0) * __ldg(p.turns + pair);
            float s, c;
            sincospif((float)(int32_t)(frac >> 32) * 0x1p-31f, &s, &c);
            turn[i] = make_float2(c * p.mult, s * p.mult);
        }
        __syncthreads();
        const int per = heads * p.items;          // of a token: the turned items of each head, then the copied ones
        for (int i = threadIdx.x; i < n * per; i += kThreads) {
            const int hi = p.by_items(i), it = i - hi * p.items, t = p.by_heads(hi), h = hi - t * heads;
            if (__ldg(p.positions + t0 + t) < 0) continue;
            const bool q = h < p.Hq;
            const int at = (q ? h : h - p.Hq) * p.D;
            const T* in = static_cast<const T*>(q ? p.q : p.k) + (t0 + t) * (q ? p.q_stride : p.k_stride) + at;
            T* out = static_cast<T*>(q ? p.q_out : p.k_out) + (t0 + t) * (q ? p.q_out_stride : p.k_out_stride) + at;
            const float2* cs = turn + t * half;
            if (it >= p.turned) {                 // entries behind the rotated ones
                const int d = p.rotary + (it - p.turned) * (kItems == Items::kSingle ? 1 : 8);
                if (kItems == Items::kSingle) out[d] = in[d];
                else store8(out + d, load8(in + d));
            } else if (kItems == Items::kHalves) {
                Vec8 a = load8(in + 8 * it), b = load8(in + half + 8 * it);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 w = cs[8 * it + j];
                    const float x = a.x[j], y = b.x[j];
                    a.x[j] = fmaf(x, w.x, -(y * w.y));
                    b.x[j] = fmaf(y, w.x, x * w.y);
                }
                store8(out + 8 * it, a);
                store8(out + half + 8 * it, b);
            } else if (kItems == Items::kPairs) {
                Vec8 a = load8(in + 8 * it);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 w = cs[4 * it + j];
                    const float x = a.x[2 * j], y = a.x[2 * j + 1];
                    a.x[2 * j] = fmaf(x, w.x, -(y * w.y));
                    a.x[2 * j + 1] = fmaf(y, w.x, x * w.y);
                }
                store8(out + 8 * it, a);
            } else {
                const int i0 = p.interleaved ? 2 * it : it, i1 = p.interleaved ? 2 * it + 1 : it + half;
                const float2 w = cs[it];
                const float x = load1(in + i0), y = load1(in + i1);
                store1(out + i0, fmaf(x, w.x, -(y * w.y)));
                store1(out + i1, fmaf(y, w.x, x * w.y));
            }
        }
    }
}

template <typename T>
cudaError_t launch(RopeParams& p, cudaStream_t s) {
    const int rest = p.D - p.rotary;
    const bool vectors = p.interleaved ? p.rotary % 8 == 0 : p.rotary % 16 == 0;
    p.turned = !vectors ? p.rotary / 2 : p.interleaved ? p.rotary / 8 : p.rotary / 16;
    p.items = p.turned + (vectors ? rest / 8 : rest);
    p.by_items.set((uint32_t)p.items);
    p.by_half.set((uint32_t)(p.rotary / 2));
    p.by_heads.set((uint32_t)(p.Hq + p.Hkv));
    // several tokens a block where there are many: fewer barriers a row
    p.side = p.T >= 16 * num_sms() ? 4 : 1;
    long long grid = ((long long)p.T + p.side - 1) / p.side;
    if (grid > 64LL * num_sms()) grid = 64LL * num_sms();
    const size_t smem = sizeof(float2) * p.side * (p.rotary / 2);
    auto kernel = !vectors ? rope_kernel<T, Items::kSingle> : p.interleaved ? rope_kernel<T, Items::kPairs> : rope_kernel<T, Items::kHalves>;
    return launch_dependent(kernel, dim3((unsigned)grid), dim3(kThreads), smem, s, p);
}

}  // namespace

cudaError_t launch_rope(RopeParams p, cudaStream_t s) { return p.bf16 ? launch<uint16_t>(p, s) : launch<float>(p, s); }

}  // namespace dspark
