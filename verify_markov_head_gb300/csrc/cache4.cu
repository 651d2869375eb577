// cache4.cu -- the paged cache held in 4 bits: rows quantised as they are
// written, and read back (formats: fp4.cuh; definitions: include/dspark.h).
//
// For a group of 16 entries y = x * 2^-exp:
//     scale = e4m3(max |y| / 6),   code_i = e2m1(y_i / scale).
// Both roundings are decided exactly: a number next to a border between two
// codes would otherwise go the wrong way, and bf16 entries meet borders often
// (a border is a level's midpoint, 3 bits, times a scale, 4 bits: a short number
// that inputs take).  The quotient is therefore rounded correctly: r = 1 / scale
// to nearest, q = y r, q + (y - q scale) r with fused multiply-adds (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// theorem 1), three operations an entry.  It cannot fall on a border that y / scale
// is not on: neighbours of (border * scale), a number of 7 bits, are 2^-23 of it
// away or more, the quotient's rounding moves it by 2^-24 at most.
#include "fp4.cuh"
#include "pdl.cuh"
#include "serve.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;

// 16 entries from p, times `by` (a power of two).
__device__ __forceinline__ void load_group(const float* p, float by, float (&y)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(p) + i);
        y[4 * i] = v.x * by; y[4 * i + 1] = v.y * by; y[4 * i + 2] = v.z * by; y[4 * i + 3] = v.w * by;
    }
}
__device__ __forceinline__ void load_group(const uint16_t* p, float by, float (&y)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[8 * i + 2 * j] = __uint_as_float(w[j] << 16) * by;
            y[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u) * by;
        }
    }
}

__device__ __forceinline__ void store_group(float* p, const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) __stcs(reinterpret_cast<float4*>(p) + i, make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
}
__device__ __forceinline__ void store_group(uint16_t* p, const float (&x)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    __stcs(reinterpret_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
}

// Where item `i` of the launch lies: its token, its group in the token's rows
// (keys first, then values), and in the cache.
struct Place {
    int t, slot, values, group;
    long long codes, scales;         // bytes from the caches' starts
    bool ok;
    __device__ __forceinline__ Place(const Cache4Params& p, long long i) {
        const int per = p.heads * p.groups;                  // groups of a token's keys
        // (i < 2^31 * 2: tokens by division of the pair of rows)
        t = (int)(i / (2 * per));
        int g = (int)(i - (long long)t * (2 * per));
        values = g >= per;
        group = values ? g - per : g;
        slot = __ldg(p.slot_map + t);
        ok = slot >= 0;
        if (!ok) return;
        const int page = p.by_page(slot), row = slot - page * p.page_size;
        if (page >= p.pages) { raise_status(p.status, kBadPage); ok = false; return; }
        const int h = p.by_groups(group), c = group - h * p.groups;
        const long long at = ((long long)h * p.page_size + row) * p.groups + c;      // group within the page
        codes = page * p.page_bytes + at * (fp4::kGroup / 2);
        scales = page * p.scale_bytes + at;
    }
};

// A thread takes a group: 32 or 64 bytes in, 8 of codes and a scale out.
template <typename T>
__global__ void __launch_bounds__(kThreads) cache_append4_kernel(const Cache4Params p) {
    grid_dependency_wait();
    const long long items = 2LL * p.T * p.heads * p.groups;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < items; i += (long long)gridDim.x * kThreads) {
        const Place at(p, i);
        if (!at.ok) continue;
        const T* src = static_cast<const T*>(at.values ? p.v : p.k) + at.t * (at.values ? p.v_stride : p.k_stride) + at.group * fp4::kGroup;
        float y[16];
        load_group(src, at.values ? p.v_by : p.k_by, y);
        uint32_t top = 0u;                                   // as integers: a NaN is above infinity
#pragma unroll
        for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(y[j]) & 0x7fffffffu);
        const uint32_t sc = fp4::scale_code(__fdiv_rn(__uint_as_float(top), 6.f));
        const float s = fp4::scale_value(sc), r = s > 0.f ? __frcp_rn(s) : 0.f;
        uint32_t w[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            float q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // (beyond 6 * 448 the level is 6 in any case; infinities do not reach the products)
                const float x = copysignf(fminf(fabsf(y[8 * hf + j]), 4096.f), y[8 * hf + j]);
                const float a = x * r;
                q[j] = fmaf(fmaf(-a, s, x), r, a);
            }
            w[hf] = fp4::pack(q);
        }
        *reinterpret_cast<uint2*>((at.values ? p.v_cache : p.k_cache) + at.codes) = make_uint2(w[0], w[1]);
        (at.values ? p.v_scale : p.k_scale)[at.scales] = (uint8_t)sc;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) cache_read4_kernel(const Cache4Params p) {
    grid_dependency_wait();
    const long long items = 2LL * p.T * p.heads * p.groups;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < items; i += (long long)gridDim.x * kThreads) {
        const Place at(p, i);
        if (!at.ok) continue;
        const uint2 w = *reinterpret_cast<const uint2*>((at.values ? p.v_cache : p.k_cache) + at.codes);
        const float s = fp4::scale_value((at.values ? p.v_scale : p.k_scale)[at.scales]) * (at.values ? p.v_by : p.k_by);
        uint32_t h[4];
        float x[16];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            fp4::unpack(hf ? w.y : w.x, h);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = fp4::floats(h[j]);
                x[8 * hf + 2 * j] = f.x * s;
                x[8 * hf + 2 * j + 1] = f.y * s;
            }
        }
        store_group(static_cast<T*>(const_cast<void*>(at.values ? p.v : p.k)) + at.t * (at.values ? p.v_stride : p.k_stride) + at.group * fp4::kGroup, x);
    }
}

cudaError_t launch(void (*kernel)(const Cache4Params), const Cache4Params& p, cudaStream_t s) {
    const long long items = 2LL * p.T * p.heads * p.groups;
    long long grid = (items + kThreads - 1) / kThreads;
    if (grid > 1024LL * num_sms()) grid = 1024LL * num_sms();
    return launch_dependent(kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_cache_append4(const Cache4Params& p, cudaStream_t s) {
    return launch(p.bf16 ? cache_append4_kernel<uint16_t> : cache_append4_kernel<float>, p, s);
}
cudaError_t launch_cache_read4(const Cache4Params& p, cudaStream_t s) {
    return launch(p.bf16 ? cache_read4_kernel<uint16_t> : cache_read4_kernel<float>, p, s);
}

}  // namespace dspark
