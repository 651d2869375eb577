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
// away or more, the quotient's rounding moves it by 2^-24 at most.  (That is what fp32
// entries need; a bf16 entry's quotient is on a border or 2^-8 of it away, and would do with
// two operations.  Both types share these three.)
//
// The work on a group bounds both as much as HBM does: of 32768 tokens of 4 KB the
// append takes 33 us and the read 33, 172 MB each (5.2 TB/s), of fp32 rows 50 and 52 (306 MB, 6.0 TB/s).  On the way, both
// together: a division of 64 bits and two loads of 16 bytes a group 78 us, a block to
// two tokens and no more 91 (the places of a group are formed anew), 8 blocks an
// SM with one operation an entry 70, with two entries 68, 6 blocks 67.
#include "fp4.cuh"
#include "pdl.cuh"
#include "serve.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256, kBlocks = 6;       // and blocks of an SM

// 32 bytes at once: with two loads or stores of 16 a warp would pass each sector twice.
__device__ __forceinline__ void load_sector(const void* p, uint32_t (&w)[8]) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p));
}
__device__ __forceinline__ void store_sector(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}

// A group as it lies in memory (`wide`: at a multiple of 32 bytes), and as numbers.
template <typename T>
struct RawGroup {
    static constexpr int kWords = sizeof(T) * fp4::kGroup / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* p, bool wide) {
#pragma unroll
        for (int i = 0; i < kWords / 8; ++i) {
            uint32_t x[8];
            if (wide) load_sector(reinterpret_cast<const uint32_t*>(p) + 8 * i, x);
            else {
                *reinterpret_cast<uint4*>(x) = __ldg(reinterpret_cast<const uint4*>(p) + 2 * i);
                *reinterpret_cast<uint4*>(x + 4) = __ldg(reinterpret_cast<const uint4*>(p) + 2 * i + 1);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) w[8 * i + j] = x[j];
        }
    }
    // the largest magnitude: magnitudes are ordered as integers, a NaN above infinity
    __device__ __forceinline__ float top() const {
        uint32_t m = 0u;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < kWords; ++j) m = max(m, w[j] & 0x7fffffffu);
        } else {
#pragma unroll
            for (int j = 0; j < kWords; ++j) m = __vmaxu2(m, w[j] & 0x7fff7fffu);
            m = max(m << 16, m & 0xffff0000u);
        }
        return __uint_as_float(m);
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};

__device__ __forceinline__ void store_words(void* p, bool wide, const uint32_t (&w)[8]) {
    if (wide) store_sector(p, w);
    else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
__device__ __forceinline__ void store_group(float* p, bool wide, const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(x[8 * i + j]);
        store_words(p + 8 * i, wide, w);
    }
}
__device__ __forceinline__ void store_group(uint16_t* p, bool wide, const float (&x)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    store_words(p, wide, w);
}

// Two numbers at a time.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// y / s to nearest, r = 1 / s to nearest (infinite y stay infinite).
__device__ __forceinline__ float quotient(float y, float s, float r) {
    const float a = y * r;
    return a < INFINITY ? fmaf(fmaf(-a, s, y), r, a) : a;
}
// 1 / s to nearest, s a scale above 0: a Newton step from the approximation, which
// is off by 1 place at most, leaves 2^-46.  1 / s, one of 8 fractions n / 8 .. n / 15
// times a power of two, is a multiple of 1 / 15 of 2^-25 away from every midpoint.
__device__ __forceinline__ float inverse_of(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return fmaf(fmaf(-s, r, 1.f), r, r);
}

// A thread keeps one group of a token's rows (keys first, then values) through
// all tokens that it takes: head, group and places follow once.
struct Group {
    const uint8_t* rows;             // of token 0 (bytes)
    long long row_bytes;             // from token to token
    uint8_t *codes, *scales;         // in page 0, row 0
    float by, inverse;               // what entries are multiplied by, and its inverse
    bool wide;                       // rows at multiples of 32 bytes
    __device__ __forceinline__ Group(const Cache4Params& p, int e, int entry_bytes) {
        const int per = p.heads * p.groups;
        const bool v = e >= per;
        const int g = v ? e - per : e, h = p.by_groups(g), c = g - h * p.groups;
        const long long at = (long long)h * p.page_size * p.groups + c;
        rows = static_cast<const uint8_t*>(v ? p.v : p.k) + (long long)g * fp4::kGroup * entry_bytes;
        row_bytes = (v ? p.v_stride : p.k_stride) * entry_bytes;
        codes = (v ? p.v_cache : p.k_cache) + at * (fp4::kGroup / 2);
        scales = (v ? p.v_scale : p.k_scale) + at;
        by = v ? p.v_by : p.k_by;
        inverse = 1.f / by;
        wide = ((reinterpret_cast<uintptr_t>(rows) | (uintptr_t)row_bytes) & 31) == 0;
    }
};
// The place of a slot from a group's own, in groups from the page's start; false: not to be touched.
__device__ __forceinline__ bool place(const Cache4Params& p, int slot, int& page, int& row) {
    if (slot < 0) return false;
    page = p.by_page(slot);
    row = (slot - page * p.page_size) * p.groups;
    if (page < p.pages) return true;
    raise_status(p.status, kBadPage);
    return false;
}

// Runs body(Group, token) over the launch's groups and tokens; `lanes` threads to a token.
template <typename Body>
__device__ __forceinline__ void each_group(const Cache4Params& p, int lanes, int entry_bytes, Body&& body) {
    const int per = 2 * p.heads * p.groups, side = kThreads / lanes, lt = threadIdx.x / lanes;
    if (lt >= side) return;
    for (int e = threadIdx.x - lt * lanes; e < per; e += lanes) {
        const Group g(p, e, entry_bytes);
        for (long long t = (long long)blockIdx.x * side + lt; t < p.T; t += (long long)gridDim.x * side) body(g, t);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kBlocks) cache_append4_kernel(const Cache4Params p, int lanes) {
    grid_dependency_wait();
    each_group(p, lanes, (int)sizeof(T), [&](const Group& g, long long t) {
        RawGroup<T> x;
        x.load(reinterpret_cast<const T*>(g.rows + t * g.row_bytes), g.wide);     // (does not wait for the slot)
        int page, row;
        if (!place(p, __ldg(p.slot_map + t), page, row)) return;
        const float top = x.top() * g.by;
        const uint32_t sc = fp4::scale_code(quotient(top, 6.f, 0x1.555556p-3f));
        // the quotient of x * 2^-exp by s, with the power of two in s and 1 / s
        const float s0 = fp4::scale_value(sc), s = s0 * g.inverse, r = s0 > 0.f ? inverse_of(s0) * g.by : 0.f;
        // (beyond 6 * 448 the level is 6 in any case; infinities do not reach the products)
        const bool clamped = top > 4096.f;
        const float most = 4096.f * g.inverse;
        const uint64_t rr = pair(r, r), ss = pair(-s, -s);
        uint32_t w[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            float q[8];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float v0 = x.get(8 * hf + j), v1 = x.get(8 * hf + j + 1);
                if (clamped) {
                    v0 = fminf(fmaxf(v0, -most), most);
                    v1 = fminf(fmaxf(v1, -most), most);
                }
                const uint64_t v = pair(v0, v1), a = mul_pair(v, rr);
                unpair(fma_pair(fma_pair(a, ss, v), rr, a), q[j], q[j + 1]);
            }
            w[hf] = fp4::pack(q);
        }
        *reinterpret_cast<uint2*>(g.codes + page * p.page_bytes + (long long)row * (fp4::kGroup / 2)) = make_uint2(w[0], w[1]);
        g.scales[page * p.scale_bytes + row] = (uint8_t)sc;
    });
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kBlocks) cache_read4_kernel(const Cache4Params p, int lanes) {
    grid_dependency_wait();
    each_group(p, lanes, (int)sizeof(T), [&](const Group& g, long long t) {
        int page, row;
        if (!place(p, __ldg(p.slot_map + t), page, row)) return;
        const uint2 w = *reinterpret_cast<const uint2*>(g.codes + page * p.page_bytes + (long long)row * (fp4::kGroup / 2));
        const float s = fp4::scale_value(g.scales[page * p.scale_bytes + row]) * g.by;
        uint32_t h[4];
        float x[16];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            fp4::unpack(hf ? w.y : w.x, h);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = fp4::floats(h[j]);
                unpair(mul_pair(pair(f.x, f.y), pair(s, s)), x[8 * hf + 2 * j], x[8 * hf + 2 * j + 1]);
            }
        }
        store_group(reinterpret_cast<T*>(const_cast<uint8_t*>(g.rows) + t * g.row_bytes), g.wide, x);
    });
}

cudaError_t launch(void (*kernel)(const Cache4Params, int), const Cache4Params& p, cudaStream_t s) {
    const int per = 2 * p.heads * p.groups, lanes = per < kThreads ? per : kThreads, side = kThreads / lanes;
    long long grid = ((long long)p.T + side - 1) / side;
    if (grid > (long long)kBlocks * num_sms()) grid = (long long)kBlocks * num_sms();
    return launch_dependent(kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, p, lanes);
}

}  // namespace

cudaError_t launch_cache_append4(const Cache4Params& p, cudaStream_t s) {
    return launch(p.bf16 ? cache_append4_kernel<uint16_t> : cache_append4_kernel<float>, p, s);
}
cudaError_t launch_cache_read4(const Cache4Params& p, cudaStream_t s) {
    return launch(p.bf16 ? cache_read4_kernel<uint16_t> : cache_read4_kernel<float>, p, s);
}

}  // namespace dspark
