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
// Bytes bound it: a token's rows are read and written once.  32768 tokens of 40
// heads of 128, 671 MB: 102 us (6.6 TB/s; with sines in shared memory, a block to 4
// tokens and two barriers each, 139), 512 tokens 3.9 (4.6 without sharing the sines); in fp32, 1342 MB,
// 230 us in halves and 248 in neighbours (5.8 and 5.4 TB/s, some registers spilled).
#include <cuda_bf16.h>

#include "pdl.cuh"
#include "serve.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;

// 8 entries as they lie in memory, and as numbers.
template <typename T> struct Raw;
template <> struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) { a = __ldcs(reinterpret_cast<const float4*>(p)); b = __ldcs(reinterpret_cast<const float4*>(p) + 1); }
    __device__ __forceinline__ void store(float* p) const { reinterpret_cast<float4*>(p)[0] = a; reinterpret_cast<float4*>(p)[1] = b; }
    __device__ __forceinline__ void get(float (&x)[8]) const { x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w; }
    __device__ __forceinline__ void set(const float (&x)[8]) { a = make_float4(x[0], x[1], x[2], x[3]); b = make_float4(x[4], x[5], x[6], x[7]); }
};
template <> struct Raw<uint16_t> {
    uint4 v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = v; }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) { x[2 * j] = __uint_as_float(w[j] << 16); x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u); }
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(x[2 * j + 1]), "f"(x[2 * j]));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) {
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.bf16.f32 h, %1;\n\tmov.b16 %0, h;\n\t}" : "=h"(*p) : "f"(x));
}

// How an item covers its entries.  kHalves: 8 pairs (i, i + r/2), two
// vectors.  kPairs: 4 neighbouring pairs, one vector.  kSingle: one pair, where
// the halves or the pairs do not fill vectors of 8.
enum class Items { kHalves, kPairs, kSingle };

// A warp takes a token, or a share of its heads where there are few tokens.  A
// lane keeps its place within the head: it forms its pairs' sines and cosines once
// and then turns them in one head after another, p.side heads of the warp at a
// time, kBatch loads ahead of the arithmetic.  No barrier, no table in memory.
template <typename T, Items kItems>
__global__ void __launch_bounds__(kThreads, 5) rope_kernel(const RopeParams p) {
    constexpr int kPairs = kItems == Items::kHalves ? 8 : kItems == Items::kPairs ? 4 : 1;      // of a lane
    constexpr int kBatch = kItems == Items::kHalves ? 2 : 4;
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, half = p.rotary / 2, heads = p.Hq + p.Hkv;
    const long long job = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(job / p.shares), share = (int)(job - (long long)t * p.shares);
    if (t >= p.T) return;
    const int pos = __ldg(p.positions + t);
    if (pos < 0) return;
    // heads [h0, h1) of the warp; items beyond a warp's lanes come in further rounds
    const int h0 = (int)((long long)heads * share / p.shares), h1 = (int)((long long)heads * (share + 1) / p.shares);
    const T *q = static_cast<const T*>(p.q) + t * p.q_stride, *k = static_cast<const T*>(p.k) + t * p.k_stride;
    T *q_out = static_cast<T*>(p.q_out) + t * p.q_out_stride, *k_out = static_cast<T*>(p.k_out) + t * p.k_out_stride;
    for (int it0 = 0; it0 < p.items; it0 += 32) {
        const int mine = p.side > 1 ? lane / p.items : 0, it = p.side > 1 ? lane - mine * p.items : it0 + lane;
        const bool turned = it < p.turned;
        // lanes at the same place of different heads share the work on their sines and cosines
        float c[kPairs], s[kPairs];
#pragma unroll 1
        for (int j0 = 0; j0 < kPairs; j0 += p.side) {
            float sj = 0.f, cj = 0.f;
            if (turned && mine < p.side && j0 + mine < kPairs) {
                const uint64_t frac = (uint64_t)(uint32_t)pos * __ldg(p.turns + it * kPairs + j0 + mine);
                sincospif((float)(int32_t)(frac >> 32) * 0x1p-31f, &sj, &cj);
                sj *= p.mult;
                cj *= p.mult;
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j)
                if (j >= j0 && j < j0 + p.side) {
                    const int from = p.side > 1 ? (j - j0) * p.items + it : lane;
                    c[j] = __shfl_sync(~0u, cj, from);
                    s[j] = __shfl_sync(~0u, sj, from);
                }
        }
        if (mine >= p.side || it >= p.items) continue;
        if constexpr (kItems == Items::kSingle) {
            const int i0 = !turned ? p.rotary + it - p.turned : p.interleaved ? 2 * it : it, i1 = p.interleaved ? i0 + 1 : i0 + half;
            for (int h = h0 + mine; h < h1; h += p.side) {
                const T* in = h < p.Hq ? q + h * p.D : k + (h - p.Hq) * p.D;
                T* out = h < p.Hq ? q_out + h * p.D : k_out + (h - p.Hq) * p.D;
                if (!turned) { out[i0] = in[i0]; continue; }
                const float x = load1(in + i0), y = load1(in + i1);
                store1(out + i0, fmaf(x, c[0], -(y * s[0])));
                store1(out + i1, fmaf(y, c[0], x * s[0]));
            }
        } else {
            const int d = turned ? 8 * it : p.rotary + (it - p.turned) * 8;
            for (int h = h0 + mine; h < h1; h += kBatch * p.side) {
                Raw<T> a[kBatch], b[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int hu = h + u * p.side;
                    if (hu >= h1) continue;
                    const T* in = (hu < p.Hq ? q + hu * p.D : k + (hu - p.Hq) * p.D) + d;
                    a[u].load(in);
                    if (kItems == Items::kHalves && turned) b[u].load(in + half);
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int hu = h + u * p.side;
                    if (hu >= h1) continue;
                    T* out = (hu < p.Hq ? q_out + hu * p.D : k_out + (hu - p.Hq) * p.D) + d;
                    if (turned) {
                        float x[8], y[8];
                        a[u].get(x);
                        if (kItems == Items::kHalves) b[u].get(y);
#pragma unroll
                        for (int j = 0; j < kPairs; ++j) {
                            float& v = kItems == Items::kHalves ? x[j] : x[2 * j];
                            float& w = kItems == Items::kHalves ? y[j] : x[2 * j + 1];
                            const float v0 = v, w0 = w;
                            v = fmaf(v0, c[j], -(w0 * s[j]));
                            w = fmaf(w0, c[j], v0 * s[j]);
                        }
                        a[u].set(x);
                        if (kItems == Items::kHalves) {
                            b[u].set(y);
                            b[u].store(out + half);
                        }
                    }
                    a[u].store(out);
                }
            }
        }
    }
}

template <typename T>
cudaError_t launch(RopeParams& p, cudaStream_t s) {
    const int rest = p.D - p.rotary, heads = p.Hq + p.Hkv;
    const bool vectors = p.interleaved ? p.rotary % 8 == 0 : p.rotary % 16 == 0;
    p.turned = !vectors ? p.rotary / 2 : p.interleaved ? p.rotary / 8 : p.rotary / 16;
    p.items = p.turned + (vectors ? rest / 8 : rest);
    p.side = p.items <= 32 ? 32 / p.items : 1;
    // few tokens: several warps to each, down to one round of heads
    const long long want = 16LL * num_sms();
    int most = (heads + p.side - 1) / p.side;
    p.shares = p.T >= want ? 1 : (int)((want + p.T - 1) / p.T);
    if (p.shares > most) p.shares = most;
    const long long warps = (long long)p.T * p.shares;
    const long long grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
    auto kernel = !vectors ? rope_kernel<T, Items::kSingle> : p.interleaved ? rope_kernel<T, Items::kPairs> : rope_kernel<T, Items::kHalves>;
    return launch_dependent(kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_rope(RopeParams p, cudaStream_t s) { return p.bf16 ? launch<uint16_t>(p, s) : launch<float>(p, s); }

}  // namespace dspark
