// sample.cu -- a token of each row of logits, with temperature, top-k, top-p and
// min-p, from a given random number (definition: include/dspark.h).
//
// A cluster of CTAs takes a row, in a few passes: the first from HBM, which finds the
// largest entry, the others from L2 or L1.  With weights w_v = e^((x_v - max) / T):
//   few      top-k up to 512: of the threads' own maxima, the 1/32 power of 2 of the weight in
//            which the k-th largest lies is a bound that k entries reach; the entries that
//            reach it, hardly more than k, go to one CTA, which ranks, cuts and draws.
//   many     top-k beyond, and top-p: a histogram of counts, or of weights, over such
//            steps, the step in which the wanted count or sum is reached, and its entries (of a
//            model's row a hundredth, up to 4096) to one CTA, which finds the last one kept, 9
//            bits at a time.  No sort.  A step of more entries (rows of few different values,
//            and flat ones: of 151936 normal entries of deviation 0.3 a step holds up to 4500) is
//            searched over the slices, a bit of the key and then of the id to a pass.
//   the draw sums of the weights left, by warp and CTA in the order of the ids (formed on
//            the way to the list, where there is one), and a walk through the one warp's
//            share that holds u times the total.
//
// 512 rows of 151936 fp32 entries, 311 MB that HBM reads in 46 us: the largest entry 88 us,
// nothing cut 170, top-k 50 106, top-k 200 134, top-k 2000 290, top-p 0.9 378; one row 7 to
// 30, of 34 to 53 passes over its slices 144 to 177 (64 rows 500 to 650).  No unit bounds it: 1.5 to 1.9 of 4
// instructions a cycle are issued (20 an entry where weights are formed, 35 with the histogram), and warps
// wait at the barriers between a row's phases first, which the other row on an SM covers in part.
//
// A token's boundaries are sums over up to 2^19 entries, and a sum that is off by
// 2^-24 moves the draw across one in a row of some thousand (the boundaries of a
// flat row are 10^-5 apart).  So weights are integers: sums are exact, and the same in
// any order, atomics among them.  Their unit is 2^-50 of the largest, or what keeps the sum
// of a row below 2^63: the maxima of 512 groups of entries, each times the n = V / 512 entries of a group,
// are a sum S that no row's exceeds, and a row's is S / n at least.  So what V entries lose
// by the cut to integers is V 2^-50 of the largest or V n 2^-60 of the sum, 2^-31 at most.  (With
// 2^-42 for all rows 130000 light entries lost up to 2^-25 of the sum.)  A weight is
//     2^(y - ref),  y = x log2(e) / T = k / 256 + r,  |r| <= 2^-9,
// y by fused multiply-adds with log2(e) / T in two floats, 2^(k mod 256 / 256) from a
// table of integers, and 2^r - 1 by its series to r^3, as an integer: off by 2^-31 of
// the weight, in 15 operations (floats two at a time).  In double precision it would be
// the FP64 units' two operations a cycle that bound the kernel.
#include <cooperative_groups.h>

#include "pdl.cuh"
#include "serve.cuh"

namespace dspark {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32, kBins = 2048;
constexpr int kUnit = 50;                        // a weight of 1 is 2^kUnit at most
constexpr int kFine = 8;                         // log2 of the table's entries
constexpr int kCoarse = 3;                       // log2 of the table's steps to a bin
constexpr float kDeep = 52.f;                    // entries that many powers of 2 below the largest weigh nothing
constexpr uint32_t kNothing = (uint32_t)(kDeep - 1.f) << (kFine - kCoarse);      // the bins from which on entries weigh nothing
constexpr int kFew = 512, kCandidates = 1024;    // top_k that is looked for among candidates, and their most
constexpr int kListed = 4096;                    // entries of a step that one CTA takes
constexpr int kDigit = 9;                        // bits of a key that a list is searched by at a time
constexpr uint32_t kAll = 0xffffffffu;

using u64 = unsigned long long;

// 2^(31 + j / 256), from the 256th root of 2 (square roots by Newton's method).
struct Powers {
    uint32_t v[1 << kFine];
    constexpr Powers() : v{} {
        double root = 2.0;
        for (int i = 0; i < kFine; ++i) {
            double x = 1.5;
            for (int n = 0; n < 30; ++n) x = 0.5 * (x + root / x);
            root = x;
        }
        for (int j = 0; j < 1 << kFine; ++j) {
            double x = 1.0, f = root;            // root^j by squares: few roundings
            for (int n = j; n; n >>= 1, f *= f)
                if (n & 1) x *= f;
            v[j] = (uint32_t)(x * 2147483648.0 + 0.5);
        }
    }
};
__constant__ Powers c_powers = Powers();

// Integers in the order of the numbers they stand for (no NaN; -0 is 0).
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
// Two numbers at a time.
__device__ __forceinline__ u64 two(float a, float b) {
    u64 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void apart(u64 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
    u64 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ u64 shift_right(u64 x, uint32_t n) {   // (0 from 64 on)
    u64 r;
    asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"(x), "r"(n));
    return r;
}

// log2(e) / temperature in two floats, and what entries are taken from.
struct Scale {
    float base, low, c_hi, c_lo;
    static __device__ __forceinline__ float within(float T) { return fminf(fmaxf(T, 1e-30f), 1e36f); }
    static __device__ __forceinline__ float per(float T) { return 1.44269502f / within(T); }
    __device__ __forceinline__ Scale(float top, float T) {
        // (Temperatures are taken into 10^-30 .. 10^36: below only the largest entries weigh
        // anything, above -inf would.)
        T = within(T);
        constexpr float e_hi = 1.44269502f, e_lo = 1.92596303e-8f;
        c_hi = e_hi / T;
        c_lo = (fmaf(-c_hi, T, e_hi) + e_lo) / T;
        // Where y itself is so large that its fraction is lost, entries are taken from
        // the largest one: exactly, since what still weighs something is that near to it.
        base = fabsf(top * c_hi) > 4096.f ? top : 0.f;
        low = fmaxf((top - base) - kDeep / c_hi, -3.4e38f);      // (behind the base)
    }
};

// x (0 <= x < 1) times n, in units of 2^-64: the whole part, and whether a rest is left.
__device__ __forceinline__ u64 part_of(float x, u64 n, bool& rest) {
    const u64 f = __float2ull_rz(x * 0x1p64f);
    rest = f * n != 0ull;
    return __umul64hi(f, n);
}

// Weights of a row's entries.
struct Weigher {
    u64 base, c_hi, c_lo;                        // (the negative base)
    float low;
    uint32_t ref;                                // the step of the largest entry, rounded down to a power of 2
    uint32_t down;                               // what a product at ref is shifted by to be a weight
    const uint32_t* powers;
    static constexpr float kMagic = 1.5f * (1 << (23 - kFine));      // a sum's last place is a step
    static constexpr float kRound = 12582912.f;                      // 1.5 * 2^23: a sum's last place is 1
    // z = x less the base, not below `low`, and k (as the bits of a float) of two entries
    __device__ __forceinline__ u64 steps(float x0, float x1, uint32_t& k0, uint32_t& k1, u64& m) const {
        float a, b, s, t;
        apart(add2(two(x0, x1), base), a, b);
        const u64 z = two(fmaxf(a, low), fmaxf(b, low));
        m = fma2(z, c_hi, two(kMagic, kMagic));
        apart(m, s, t);
        k0 = __float_as_uint(s);
        k1 = __float_as_uint(t);
        return z;
    }
    // most: a bound on the sum of the weights, the largest entry's being 1
    __device__ __forceinline__ void set(const Scale& c, float top, const uint32_t* table, float most) {
        base = two(-c.base, -c.base); c_hi = two(c.c_hi, c.c_hi); c_lo = two(c.c_lo, c.c_lo);
        low = c.low;
        powers = table;
        uint32_t k, same;
        u64 m;
        steps(top, top, k, same, m);
        ref = k >> kFine;
        // (a weight is below 2^(unit + 1), the sum below 2^(unit + 1) most)
        const int log2_most = (int)(__float_as_uint(most) >> 23) - 127;
        down = ref + 62u - (uint32_t)min(kUnit, 61 - log2_most);
    }
    __device__ __forceinline__ void operator()(float x0, float x1, u64& w0, u64& w1, uint32_t& k0, uint32_t& k1) const {
        u64 m;
        const u64 z = steps(x0, x1, k0, k1, m);
        u64 r = fma2(z, c_hi, fma2(m, two(-1.f, -1.f), two(kMagic, kMagic)));
        r = fma2(z, c_lo, r);
        // (2^r - 1) 2^31 = 2^31 (r ln 2 + (r ln 2)^2 / 2 + (r ln 2)^3 / 6 ..), to an integer
        constexpr float a1 = 1488522236.f, a2 = 515882496.f, a3 = 119194166.f;
        const u64 e = fma2(r, fma2(r, fma2(r, two(a3, a3), two(a2, a2)), two(a1, a1)), two(kRound, kRound));
        float f0, f1;
        apart(e, f0, f1);
        constexpr uint32_t kOne = 0x80000000u - 0x4b400000u;       // 2^31, less the bits of kRound
        w0 = shift_right((u64)powers[k0 & ((1 << kFine) - 1)] * (__float_as_uint(f0) + kOne), down - (k0 >> kFine));
        w1 = shift_right((u64)powers[k1 & ((1 << kFine) - 1)] * (__float_as_uint(f1) + kOne), down - (k1 >> kFine));
    }
    __device__ __forceinline__ u64 of(float x) const {
        u64 w, same;
        uint32_t k0, k1;
        (*this)(x, x, w, same, k0, k1);
        return w;
    }
    // the bin of a step, from the largest entry's down
    __device__ __forceinline__ uint32_t top_bin() const { return (ref << kFine | ((1 << kFine) - 1)) >> kCoarse; }
    __device__ __forceinline__ uint32_t bin(uint32_t k) const { return top_bin() - (k >> kCoarse); }
    // numbers that no entry of a bin is below, or above: its ends and a little more
    // (the last bins also hold what lies below them)
    __device__ __forceinline__ float least(uint32_t b, const Scale& c) const {
        if (b >= kNothing) return -INFINITY;
        const int at = (int)(top_bin() - (__float_as_uint(kMagic) >> kCoarse) - b) << kCoarse;
        const float x = c.base + ((float)at * (1.f / (1 << kFine)) - 0.01f) / c.c_hi;
        return x - 1e-5f * fabsf(x);
    }
    __device__ __forceinline__ float most(uint32_t b, const Scale& c) const {
        const int at = (int)(top_bin() - (__float_as_uint(kMagic) >> kCoarse) - b + 1) << kCoarse;
        const float x = c.base + ((float)at * (1.f / (1 << kFine)) + 0.01f) / c.c_hi;
        return x + 1e-5f * fabsf(x);
    }
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <typename T> struct Row;
template <> struct Row<float> {
    static constexpr int kVec = 4;
    static __device__ __forceinline__ void get(uint4 w, float (&x)[4]) {
        x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y); x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    static __device__ __forceinline__ float one(const float* p) { return *p; }
    static __device__ __forceinline__ float top(uint4 w) {
        return max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y)), max_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
};
template <> struct Row<uint16_t> {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ void get(uint4 w, float (&x)[8]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { x[2 * i] = __uint_as_float(u[i] << 16); x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u); }
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = __byte_perm(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]), 0x7632);
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    static __device__ __forceinline__ float one(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
    static __device__ __forceinline__ float top(uint4 w) {
        uint32_t m;
        asm("{\n\t.reg .b32 a, b;\n\tmax.NaN.bf16x2 a, %1, %2;\n\tmax.NaN.bf16x2 b, %3, %4;\n\tmax.NaN.bf16x2 %0, a, b;\n\t}"
            : "=r"(m) : "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w));
        return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
};

struct Shared {
    uint32_t powers[1 << kFine];
    union {
        struct { uint32_t lo[kBins], hi[kBins]; u64 merged[kBins]; } hist;       // counts, or weights in two words; this CTA's share of the bins, over the cluster
        struct { uint2 entry[kCandidates]; u64 w[kCandidates]; } cand;      // an entry and its id
        struct { float x[kListed]; uint32_t id[kListed]; u64 w[kListed]; } list;
    };
    float tops[kThreads];                        // the threads' maxima
    float warp_top[kWarps], warp_mass[kWarps];   // of warps of groups: the largest entry, and the sum of the groups' weights against it
    uint32_t digit_lo[1 << kDigit], digit_hi[1 << kDigit];
    u64 warp_sum[kWarps], block;
    u64 total, sums[2];                          // read by the other CTAs
    u64 share_above, share_all;
    u64 warp_kept[kWarps];                       // the weight that is kept of a warp's share
    u64 found_above;
    uint32_t found_bin, found_share;
    u64 top_w;                                   // the largest entry's weight,
    float top, T;                                // the entry itself, and the temperature
    uint32_t best;
    uint32_t gathered;                           // candidates, or entries listed, of CTA 0
    float last_x; uint32_t last_id;              // the last entry kept, of CTA 0
    float bound;
    uint32_t warp_word[kWarps];
};

// Adds a weight to a bin of Shared::hist, by its two words and without a branch.
__device__ __forceinline__ void add_weight(uint32_t bin, u64 w) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b32 lo, hi, old;\n\tmov.b64 {lo, hi}, %1;\n\tmov.u32 old, 0;\n\tsetp.ne.u64 p, %1, 0;\n\t"
                 "@p atom.shared.add.u32 old, [%0], lo;\n\tadd.cc.u32 lo, lo, old;\n\taddc.u32 hi, hi, 0;\n\tsetp.ne.u32 p, hi, 0;\n\t"
                 "@p red.shared.add.u32 [%0 + %2], hi;\n\t}" ::"r"(bin), "l"(w), "n"(4 * kBins) : "memory");
}
__device__ __forceinline__ float warp_add(float x) {         // (the same in every lane)
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    return x;
}
__device__ __forceinline__ u64 warp_add(u64 x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    return x;
}
__device__ __forceinline__ u64 warp_scan(u64 x) {            // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// The sum over the CTA, in every thread.
__device__ __forceinline__ u64 block_add(u64 x, Shared& s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    x = warp_add(x);
    if (lane == 0) s.warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
        x = warp_add(lane < kWarps ? s.warp_sum[lane] : 0ull);
        if (lane == 0) s.block = x;
    }
    __syncthreads();
    return s.block;
}

// ln(w / total), a share near 1 by what it lacks.  The quotient q is off by r / total,
// which its logarithm takes up: the numbers are in two floats.
__device__ __forceinline__ float log_share(u64 w, u64 total) {
    const bool near = total - w < w;
    const u64 n = near ? total - w : w;
    const float n_hi = __ull2float_rn(n), t_hi = __ull2float_rn(total);
    const float n_lo = (float)(long long)(n - __float2ull_rn(n_hi)), t_lo = (float)(long long)(total - __float2ull_rn(t_hi));
    const float q = n_hi / t_hi, r = (fmaf(-q, t_hi, n_hi) + fmaf(-q, t_lo, n_lo)) / t_hi;
    return near ? log1pf(-q) - r / (1.f - q) : logf(q) + r / q;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
    using R = Row<T>;
    constexpr int kVec = R::kVec;
    extern __shared__ __align__(16) uint8_t raw[];
    Shared& s = *reinterpret_cast<Shared*>(raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = p.ctas, rank = (int)(blockIdx.x % ctas), row = (int)(blockIdx.x / ctas);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < 1 << kFine) s.powers[tid] = c_powers.v[tid];
    if (tid == 0) s.gathered = 0u;
    __syncthreads();
    grid_dependency_wait();

    // this CTA's slice of the row.  Every pass reads it again, from L1 or L2
    const int first = min(p.V, rank * p.slice), count = min(p.V - first, p.slice), vecs = (count + kVec - 1) / kVec;
    const T* const src = static_cast<const T*>(p.logits) + row * p.row_stride + first;
    bool dirty = false;                          // some entries are no numbers: they are taken as -inf
    // body(v, x) for the vectors begin, begin + step, .. below end, kAhead loads ahead
    constexpr int kAhead = 4;
    auto load = [&](int v) {
        if ((v + 1) * kVec <= count) return __ldg(reinterpret_cast<const uint4*>(src) + v);
        float x[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) x[j] = v * kVec + j < count ? R::one(src + v * kVec + j) : -INFINITY;
        return R::put(x);
    };
    auto each_vec = [&](int begin, int end, int step, auto&& body) {
        for (int v = begin; v < end; v += kAhead * step) {
            uint4 w[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (v + i * step < end) w[i] = load(v + i * step);
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (v + i * step < end) {
                    float x[kVec];
                    R::get(w[i], x);
                    if (dirty)
#pragma unroll
                        for (int j = 0; j < kVec; ++j)
                            if (!(x[j] < INFINITY)) x[j] = -INFINITY;
                    body(v + i * step, x);
                }
        }
    };
    float top = -INFINITY;                       // NaN once an entry is, +inf once one is
    for (int v = tid; v < vecs; v += 8 * kThreads) {
        uint4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (v + i * kThreads < vecs) w[i] = load(v + i * kThreads);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (v + i * kThreads < vecs) top = max_nan(top, R::top(w[i]));
    }
    dirty = __syncthreads_or(!(top < INFINITY));
    if (dirty) {
        top = -INFINITY;
        each_vec(tid, vecs, kThreads, [&](int, float (&x)[kVec]) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) top = fmaxf(top, x[j]);
        });
    }
    s.tops[tid] = top;
    if (tid == 0 && dirty) raise_status(p.status, kBadInput);
    const float T_ = p.temperature ? p.temperature[row] : 1.f;
    const bool T_ok = T_ >= 0.f && T_ < INFINITY;
    cluster.sync();
    // The largest entry, and the sum over the row's groups (the vectors that thread tid took of every
    // slice: slices are whole numbers of them, so a group is the same however many CTAs there are)
    // of the weights of their largest.
    float mass;
    {
        float group = top;
        for (int r = 0; r < ctas; ++r) group = fmaxf(group, cluster.map_shared_rank(s.tops, r)[tid]);
        const float c = Scale::per(T_), most = value_of(__reduce_max_sync(~0u, key_of(group)));
        const float sum = warp_add(group > -INFINITY ? fast_exp2((group - most) * c) : 0.f);
        if (lane == 0) { s.warp_top[warp] = most; s.warp_mass[warp] = sum; }
        __syncthreads();
        const float w = lane < kWarps ? s.warp_top[lane] : -INFINITY;
        top = value_of(__reduce_max_sync(~0u, key_of(w)));
        mass = warp_add(w > -INFINITY ? s.warp_mass[lane] * fast_exp2((w - top) * c) : 0.f);
    }

    // a warp's share of the slice, in the order of the ids
    const int share = (vecs + kWarps - 1) / kWarps, v0 = min(vecs, warp * share), v1 = min(vecs, v0 + share);
    float top_p = p.top_p ? p.top_p[row] : 1.f, min_p = p.min_p ? p.min_p[row] : 0.f;
    int top_k = p.top_k ? p.top_k[row] : 0;
    if (top_k <= 0 || top_k >= p.V) top_k = 0;   // all
    const float u_ = p.u[row], u = u_ > 0.f ? fminf(u_, 0x1.fffffep-1f) : 0.f;
    if (rank == 0 && tid == 0 && (!T_ok || top_p != top_p || min_p != min_p)) raise_status(p.status, kBadInput);
    if (top_p != top_p) top_p = 1.f;
    if (min_p != min_p) min_p = 0.f;

    if (top == -INFINITY) {                      // nothing to draw
        if (rank == 0 && tid == 0) {
            raise_status(p.status, kDeadRow);
            p.tok[row] = -1;
            if (p.logprob) p.logprob[row] = -INFINITY;
        }
        cluster.sync();                          // (shared memory stays until all have read it)
        return;
    }
    if (!T_ok || T_ == 0.f) {                    // the lowest id of the largest
        uint32_t best = kAll;
        each_vec(tid, vecs, kThreads, [&](int v, float (&x)[kVec]) {
#pragma unroll
            for (int j = kVec - 1; j >= 0; --j)
                if (x[j] == top) best = min(best, (uint32_t)(first + v * kVec + j));
        });
        best = __reduce_min_sync(~0u, best);
        if (lane == 0) s.warp_word[warp] = best;
        __syncthreads();
        if (tid == 0) {
            for (int w = 0; w < kWarps; ++w) best = min(best, s.warp_word[w]);
            s.best = best;
        }
        cluster.sync();
        if (rank == 0 && tid == 0) {
            for (int r = 0; r < ctas; ++r) best = min(best, *cluster.map_shared_rank(&s.best, r));
            p.tok[row] = (int)best;
            if (p.logprob) p.logprob[row] = 0.f;
        }
        cluster.sync();
        return;
    }
    const Scale scale(top, T_);
    Weigher weight;
    weight.set(scale, top, s.powers, mass * (float)(((p.V + kVec - 1) / kVec + kThreads - 1) / kThreads * kVec));
    // the logarithm of an entry's share: the largest one's, less the distance to it (a light
    // entry's own weight is an integer of few digits)
    if (tid == 0) { s.top_w = weight.of(top); s.top = top; s.T = Scale::within(T_); }      // (barriers lie between)
    auto log_of = [&](float x, u64 total) { return log_share(s.top_w, total) + (x - s.top) / s.T; };
    // min_p, of the largest entry's weight
    u64 least_w = 0ull;
    if (min_p > 0.f) {
        least_w = weight.of(top);
        if (min_p < 1.f) {
            bool rest;
            const u64 part = part_of(min_p, least_w, rest);
            least_w = part + (rest ? 1ull : 0ull);
        }
    }

    // ------------------------------------------------------------------- few
    if (top_k && top_k <= kFew) {
        if (rank == 0) {
            // the bin of the threads' maxima in which the top_k-th lies
            for (int i = tid; i < kBins; i += kThreads) s.hist.lo[i] = 0u;
            __syncthreads();
            for (int r = 0; r < ctas; r += 2) {
                const float a = cluster.map_shared_rank(s.tops, r)[tid], b = r + 1 < ctas ? cluster.map_shared_rank(s.tops, r + 1)[tid] : -INFINITY;
                uint32_t ka, kb;
                u64 m;
                weight.steps(a, b, ka, kb, m);
                if (a > -INFINITY) atomicAdd(&s.hist.lo[weight.bin(ka)], 1u);
                if (b > -INFINITY) atomicAdd(&s.hist.lo[weight.bin(kb)], 1u);
            }
            if (tid == 0) s.bound = -INFINITY;
            __syncthreads();
            constexpr int kBinsEach = kBins / kThreads;
            uint32_t own[kBinsEach], all = 0u;
#pragma unroll
            for (int e = 0; e < kBinsEach; ++e) all += own[e] = s.hist.lo[kBinsEach * tid + e];
            const u64 scan = warp_scan(all);
            if (lane == 31) s.warp_word[warp] = (uint32_t)scan;
            __syncthreads();
            uint32_t before = (uint32_t)scan - all;
            for (int w = 0; w < warp; ++w) before += s.warp_word[w];
#pragma unroll
            for (int e = 0; e < kBinsEach; ++e) {
                if (before < (uint32_t)top_k && before + own[e] >= (uint32_t)top_k) s.bound = weight.least(kBinsEach * tid + e, scale);
                before += own[e];
            }
        }
        cluster.sync();
        Shared* const to = cluster.map_shared_rank(&s, 0);
        const float least = to->bound;
        if (least > -INFINITY) {                 // (else fewer than top_k maxima weigh something)
            each_vec(tid, vecs, kThreads, [&](int v, float (&x)[kVec]) {
                bool any = false;
#pragma unroll
                for (int j = 0; j < kVec; ++j) any |= x[j] >= least;
                if (!any) return;
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (x[j] >= least) {
                        const uint32_t at = atomicAdd(&to->gathered, 1u);
                        if (at < kCandidates) to->cand.entry[at] = make_uint2(__float_as_uint(x[j]), (uint32_t)(first + v * kVec + j));
                    }
            });
            cluster.sync();
            const int n = (int)to->gathered;
            cluster.sync();
            if (n <= kCandidates) {
                if (rank) return;                // (CTA 0 reads its own memory alone from here on)
                constexpr int kEach = kCandidates / kThreads;
                // `lanes` neighbouring threads to a candidate, or kEach candidates to a thread
                int lanes = 1;
                while (lanes < 32 && 2 * lanes * n <= kThreads) lanes *= 2;
                const int part = tid % lanes, rounds = n > kThreads ? kEach : 1;
                float x[kEach];
                uint32_t id[kEach], before[kEach], lower[kEach];
                u64 w[kEach];
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const int i = tid / lanes + e * kThreads;
                    const uint2 c = i < n ? s.cand.entry[i] : make_uint2(0xff800000u, kAll);
                    x[e] = __uint_as_float(c.x);
                    id[e] = c.y;
                    w[e] = i < n ? weight.of(x[e]) : 0ull;
                    before[e] = lower[e] = 0u;
                }
                // the numbers of those that come before: in descending order, and in the order of the ids
#pragma unroll 2
                for (int j = part; j < n; j += lanes) {
                    const uint2 c = s.cand.entry[j];
                    const float xj = __uint_as_float(c.x);
#pragma unroll
                    for (int e = 0; e < kEach; ++e)
                        if (e < rounds) {
                            const bool less = c.y < id[e];
                            lower[e] += less ? 1u : 0u;
                            before[e] += xj > x[e] || (xj == x[e] && less) ? 1u : 0u;
                        }
                }
                auto over_lanes = [&](uint32_t y) {
                    for (int o = 1; o < lanes; o <<= 1) y += __shfl_xor_sync(~0u, y, o);
                    return y;
                };
                // sums over the places before each (kEach neighbouring ones to a thread), and over all
                auto scan_places = [&]() {
                    u64 own[kEach], all = 0ull;
#pragma unroll
                    for (int e = 0; e < kEach; ++e) all += own[e] = s.cand.w[kEach * tid + e];
                    const u64 scan = warp_scan(all);
                    if (lane == 31) s.warp_sum[warp] = scan;
                    __syncthreads();
                    u64 sum = scan - all, total = 0ull;
#pragma unroll
                    for (int i = 0; i < kWarps; ++i) {
                        sum += i < warp ? s.warp_sum[i] : 0ull;
                        total += s.warp_sum[i];
                    }
#pragma unroll
                    for (int e = 0; e < kEach; ++e) {
                        s.cand.w[kEach * tid + e] = sum;
                        sum += own[e];
                    }
                    __syncthreads();
                    return total;
                };
                auto clear_places = [&]() {
                    for (int i = tid; i < kCandidates; i += kThreads) s.cand.w[i] = 0ull;
                    __syncthreads();
                };
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    before[e] = over_lanes(before[e]);
                    lower[e] = over_lanes(lower[e]);
                    if (before[e] >= (uint32_t)top_k) w[e] = 0ull;
                }
                if (top_p < 1.f) {
                    clear_places();
#pragma unroll
                    for (int e = 0; e < kEach; ++e)
                        if (part == 0 && w[e]) s.cand.w[before[e]] = w[e];
                    __syncthreads();
                    bool rest;
                    u64 want = part_of(fmaxf(top_p, 0.f), scan_places(), rest);
                    want = max(1ull, want + (rest ? 1ull : 0ull));
#pragma unroll
                    for (int e = 0; e < kEach; ++e)
                        if (w[e] && s.cand.w[before[e]] >= want) w[e] = 0ull;
                    __syncthreads();
                }
                clear_places();
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    if (w[e] < least_w) w[e] = 0ull;
                    if (part == 0 && w[e]) s.cand.w[lower[e]] = w[e];
                }
                __syncthreads();
                const u64 total = scan_places();
                bool rest;
                const u64 target = part_of(u, total, rest);       // (below the total)
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    if (part || w[e] == 0ull) continue;
                    const u64 at = s.cand.w[lower[e]];
                    if (at <= target && target < at + w[e]) {
                        p.tok[row] = (int)id[e];
                        if (p.logprob) p.logprob[row] = log_of(x[e], total);
                    }
                }
                return;
            }
        }
    }

    // ------------------------------------------------------------------ many
    // what is kept: entries above `last`, and those at it up to id `last_id`
    float last = -INFINITY;
    uint32_t last_id = 0u;
    auto kept = [&](float x, uint32_t id) { return x > last || (x == last && id <= last_id && x > -INFINITY); };
    const int chunk = kBins / ctas;
    int turn = 0;
    // a sum over the cluster of what each thread counted (places in turn: another CTA
    // may still read the one before), and what the CTAs before this one counted
    auto sum_all = [&](u64 mine) {
        mine = block_add(mine, s);
        if (tid == 0) s.sums[turn] = mine;
        cluster.sync();
        if (warp == 0) {
            const u64 x = lane < ctas ? *cluster.map_shared_rank(&s.sums[turn], lane) : 0ull, all = warp_add(x), less = warp_add(lane < rank ? x : 0ull);
            if (lane == 0) { s.share_all = all; s.share_above = less; }
        }
        __syncthreads();
        turn ^= 1;
        return s.share_all;
    };
    // Keeps, of what is kept, the entries in descending order (ties: the lower id first)
    // until they reach a wanted amount: `want` of them, or `part` of their weight.
    bool summed = false;                         // s.warp_kept holds the sums of what is kept
    auto keep = [&](const bool mass, u64 want, float part) {
        summed = false;
        for (int i = tid; i < kBins / 4; i += kThreads) {
            reinterpret_cast<uint4*>(s.hist.lo)[i] = make_uint4(0u, 0u, 0u, 0u);
            reinterpret_cast<uint4*>(s.hist.hi)[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncthreads();
        const uint32_t bins = (uint32_t)__cvta_generic_to_shared(s.hist.lo);
        each_vec(tid, vecs, kThreads, [&](int v, float (&x)[kVec]) {
            if (last > -INFINITY)
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (!kept(x[j], (uint32_t)(first + v * kVec + j))) x[j] = -INFINITY;
#pragma unroll
            for (int j = 0; j < kVec; j += 2) {
                u64 w[2], m;
                uint32_t k[2];
                if (mass) {
                    weight(x[j], x[j + 1], w[0], w[1], k[0], k[1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        add_weight(bins + 4 * weight.bin(k[e]), w[e]);
                    }
                } else {
                    // (Entries that weigh nothing are not counted: where the wanted number ends among them,
                    // keeping all is the same.  At low temperatures nearly all of a row lies there, in one bin.)
                    weight.steps(x[j], x[j + 1], k[0], k[1], m);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (weight.bin(k[e]) < kNothing) atomicAdd(&s.hist.lo[weight.bin(k[e])], 1u);
                }
            }
        });
        if (tid == 0) s.gathered = 0u;
        cluster.sync();
        // the cluster's sums of this CTA's share of the bins
        u64 mine = 0ull;
        for (int i = tid; i < chunk; i += kThreads) {
            u64 sum = 0ull;
#pragma unroll 4
            for (int r = 0; r < ctas; ++r) {
                const Shared* o = cluster.map_shared_rank(&s, r);
                sum += ((u64)o->hist.hi[rank * chunk + i] << 32) + o->hist.lo[rank * chunk + i];
            }
            s.hist.merged[i] = sum;
            mine += sum;
        }
        mine = block_add(mine, s);
        if (tid == 0) s.total = mine;
        cluster.sync();
        // the share of the bins that the wanted sum is reached in
        if (warp == 0) {
            const u64 x = lane < ctas ? *cluster.map_shared_rank(&s.total, lane) : 0ull, scan = warp_scan(x), all = __shfl_sync(~0u, scan, 31);
            if (mass) {
                bool rest;
                want = part_of(part, all, rest);
                want = max(1ull, want + (rest ? 1ull : 0ull));
            }
            if (lane == 0) s.share_all = want <= all ? want : 0ull;
            if (scan - x < want && scan >= want) { s.share_above = scan - x; s.found_share = (uint32_t)lane; }
        }
        __syncthreads();
        want = s.share_all;
        if (want == 0ull) { cluster.sync(); return; }        // all that weigh something are kept (counts)
        // and the bin, `each` of them to a thread
        {
            const u64* bins = cluster.map_shared_rank(s.hist.merged, s.found_share);
            const int each = (chunk + kThreads - 1) / kThreads;
            u64 own[kBins / kThreads], all = 0ull;
#pragma unroll
            for (int e = 0; e < kBins / kThreads; ++e) {
                const int i = tid * each + e;
                own[e] = e < each && i < chunk ? bins[i] : 0ull;
                all += own[e];
            }
            const u64 scan = warp_scan(all);
            if (lane == 31) s.warp_sum[warp] = scan;
            __syncthreads();
            u64 before = s.share_above + scan - all;
            for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
#pragma unroll
            for (int e = 0; e < kBins / kThreads; ++e) {
                if (before < want && before + own[e] >= want) {
                    s.found_bin = s.found_share * chunk + (uint32_t)(tid * each + e);
                    s.found_above = before;
                }
                before += own[e];
            }
        }
        cluster.sync();                          // (the bins' sums were read: their place takes the list)
        const uint32_t found = s.found_bin;
        const u64 above = s.found_above;
        const float from = weight.least(found, scale), to = weight.most(found, scale);
        Shared* const list = cluster.map_shared_rank(&s, 0);
        // body(x, id) for the entries of the bin in this CTA's slice
        auto each_entry = [&](auto&& body) {
            each_vec(tid, vecs, kThreads, [&](int v, float (&x)[kVec]) {
                bool any = false;
#pragma unroll
                for (int j = 0; j < kVec; ++j) any |= x[j] >= from && x[j] <= to;
                if (!any) return;
#pragma unroll
                for (int j = 0; j < kVec; j += 2) {
                    uint32_t k[2];
                    u64 m;
                    weight.steps(x[j], x[j + 1], k[0], k[1], m);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t id = (uint32_t)(first + v * kVec + j + e);
                        if (weight.bin(k[e]) == found && kept(x[j + e], id)) body(x[j + e], id);
                    }
                }
            });
        };
        // the entries of the bin to CTA 0, the sums of those above it by warp's share
        u64 over = 0ull;
        each_vec(v0 + lane, v1, 32, [&](int v, float (&x)[kVec]) {
            bool any = false;
#pragma unroll
            for (int j = 0; j < kVec; ++j) any |= x[j] >= from;
            if (!any) return;
            if (last > -INFINITY)
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (!kept(x[j], (uint32_t)(first + v * kVec + j))) x[j] = -INFINITY;
#pragma unroll
            for (int j = 0; j < kVec; j += 2) {
                u64 w[2];
                uint32_t k[2];
                weight(x[j], x[j + 1], w[0], w[1], k[0], k[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t bin = weight.bin(k[e]);
                    if (bin < found) over += w[e];
                    if (bin == found && x[j + e] > -INFINITY) {
                        const uint32_t at = atomicAdd(&list->gathered, 1u);
                        if (at < kListed) { list->list.x[at] = x[j + e]; list->list.id[at] = (uint32_t)(first + v * kVec + j + e); }
                    }
                }
            }
        });
        over = warp_add(over);
        if (lane == 0) s.warp_kept[warp] = over;
        cluster.sync();
        const uint32_t n = list->gathered;
        // The last entry: the largest key at which the sum over the keys from it up
        // reaches what is wanted, and among the entries at it the number of ids that are needed.
        // sum(body): the sum of body(key, id, weight or 1) over the entries, in every thread that is here.
        // (over: the sum above the key)
        auto finish = [&](uint32_t key, u64 over, auto&& sum, auto&& nth_id) {
            const u64 at = sum([&](uint32_t k, uint32_t, u64) { return k == key ? 1ull : 0ull; });
            const u64 w = mass ? max(weight.of(value_of(key)), 1ull) : 1ull, needed = (want - over + w - 1ull) / w;
            uint32_t id = value_of(key) == last ? last_id : 0x7fffffffu;      // (where the cut before lies among the same entries, it stays)
            if (needed < at) id = nth_id(needed);        // the id that has needed - 1 others below it
            if (tid == 0) { s.last_x = value_of(key); s.last_id = id; }
        };
        if (n <= kListed) {
            if (rank == 0) {
                constexpr int kEach = kListed / kThreads;
                uint32_t k[kEach], most = 0u, least = kAll;
                const int rounds = ((int)n + kThreads - 1) / kThreads;
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const int i = tid + e * kThreads;
                    k[e] = i < (int)n ? key_of(s.list.x[i]) : 0u;          // (no entry's key)
                    most = max(most, k[e]);
                    if (i < (int)n) {
                        least = min(least, k[e]);
                        s.list.w[i] = mass ? weight.of(s.list.x[i]) : 1ull;
                    }
                }
                most = __reduce_max_sync(~0u, most);
                least = __reduce_min_sync(~0u, least);
                if (tid == 0) { s.best = 0u; s.found_bin = kAll; }
                __syncthreads();
                if (lane == 0) { atomicMax(&s.best, most); atomicMin(&s.found_bin, least); }
                __syncthreads();
                most = s.best;
                // the digits that all keys share are known
                const int bits = 32 - __clz(most ^ s.found_bin);
                const uint32_t known = bits == 32 ? 0u : most >> bits << bits;
                // the largest number at which the amounts of the entries from it up reach `goal` (over: of those above
                // it), 9 bits at a time; number(e): of the thread's entry e, 0: none; `value` holds the bits above `left`
                auto by_digits = [&](uint32_t value, int left, u64& over, const u64 goal, auto&& number, auto&& amount) {
                    while (left > 0) {
                        static_assert(1 << kDigit == kThreads, "a digit to a thread");
                        const int d = min(left, kDigit), shift = left - d;
                        s.digit_lo[tid] = s.digit_hi[tid] = 0u;
                        __syncthreads();
#pragma unroll
                        for (int e = 0; e < kEach; ++e) {
                            const uint32_t x = e < rounds ? number(e) : 0u;
                            if (x && (u64)(x ^ value) >> left == 0ull) {
                                const u64 w = amount(e);
                                const uint32_t at = (x >> shift) & ((1u << d) - 1u), lo = (uint32_t)w, old = atomicAdd(&s.digit_lo[at], lo);
                                const uint32_t hi = (uint32_t)(w >> 32) + (old > ~lo ? 1u : 0u);
                                if (hi) atomicAdd(&s.digit_hi[at], hi);
                            }
                        }
                        __syncthreads();
                        // the largest digit first
                        const int mine = kThreads - 1 - tid;
                        const u64 own = ((u64)s.digit_hi[mine] << 32) + s.digit_lo[mine], scan = warp_scan(own);
                        if (lane == 31) s.warp_sum[warp] = scan;
                        __syncthreads();
                        u64 before = over + scan - own;
                        for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
                        if (before < goal && before + own >= goal) { s.best = (uint32_t)mine; s.found_above = before; }
                        __syncthreads();
                        over = s.found_above;
                        value |= s.best << shift;
                        left = shift;
                    }
                    return value;
                };
                u64 over = above;
                const uint32_t key = by_digits(known, bits, over, want, [&](int e) { return k[e]; }, [&](int e) { return s.list.w[tid + e * kThreads]; });
                finish(key, over, [&](auto&& body) {
                    u64 sum = 0ull;
#pragma unroll
                    for (int e = 0; e < kEach; ++e)
                        if (e < rounds && k[e]) sum += body(k[e], s.list.id[tid + e * kThreads], s.list.w[tid + e * kThreads]);
                    return block_add(sum, s);
                }, [&](u64 needed) {
                    constexpr uint32_t kIds = DSPARK_MAX_SAMPLE_VOCAB - 1;     // (lower ids as larger numbers, above 0)
                    u64 none = 0ull;
                    return kIds & ~by_digits(kIds + 1u, 19, none, needed, [&](int e) { return k[e] == key ? kIds + 1u + (kIds ^ s.list.id[tid + e * kThreads]) : 0u; },
                                             [](int) { return 1ull; });
                });
                __syncthreads();
                // what is kept of the list, to the warps whose shares hold it
                const uint32_t last_key = key_of(s.last_x), end_id = s.last_id;
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    if (e >= rounds || !k[e]) continue;
                    const int i = tid + e * kThreads, id = (int)s.list.id[i];
                    if (k[e] < last_key || (k[e] == last_key && (uint32_t)id > end_id)) continue;
                    const int r = id / p.slice, at = r * p.slice, all = (min(p.V - at, p.slice) + kVec - 1) / kVec;
                    atomicAdd(&cluster.map_shared_rank(&s, r)->warp_kept[(id - at) / kVec / ((all + kWarps - 1) / kWarps)],
                              mass ? s.list.w[i] : weight.of(s.list.x[i]));
                }
            }
            summed = true;
        } else {                                 // many equal entries, or a flat row: over the slices
            auto sum = [&](auto&& body) {
                u64 mine = 0ull;
                each_entry([&](float x, uint32_t id) { mine += body(key_of(x), id, mass ? weight.of(x) : 1ull); });
                return sum_all(mine);
            };
            uint32_t key = 0u;
            for (int b = 31; b >= 0; --b) {
                const uint32_t tried = key | 1u << b;
                if (above + sum([&](uint32_t k, uint32_t, u64 w) { return k < tried ? 0ull : w; }) >= want) key = tried;
            }
            finish(key, above + sum([&](uint32_t k, uint32_t, u64 w) { return k <= key ? 0ull : w; }), sum, [&](u64 needed) {
                uint32_t id = 0u;
                for (int b = 18; b >= 0; --b) {
                    const uint32_t tried = id | 1u << b;
                    if (sum([&](uint32_t k, uint32_t i, u64) { return k == key && i < tried ? 1ull : 0ull; }) < needed) id = tried;
                }
                return id;
            });
        }
        cluster.sync();
        const float new_x = list->last_x;
        const uint32_t new_id = list->last_id;
        cluster.sync();                          // (before the next call writes them)
        last = new_x;
        last_id = new_id;
    };
    if (top_k) keep(false, (u64)top_k, 0.f);
    if (top_p < 1.f) keep(true, 0ull, fmaxf(top_p, 0.f));

    // ------------------------------------------------------------------ draw
    // the weights of a vector's entries (0: left out); warps walk their shares in the order of the ids
    auto weigh = [&](int v, float (&x)[kVec], u64 (&w)[kVec]) {
        if (last > -INFINITY) {
            bool any = false;
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const bool in = x[j] >= last;
                any |= in;
                if (!in) x[j] = -INFINITY;
            }
            if (!any) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) w[j] = 0ull;
                return;
            }
            if (last_id < 0x7fffffffu)
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (x[j] == last && (uint32_t)(first + v * kVec + j) > last_id) x[j] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < kVec; j += 2) {
            uint32_t k0, k1;
            weight(x[j], x[j + 1], w[j], w[j + 1], k0, k1);
        }
        if (least_w)
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (w[j] < least_w) w[j] = 0ull;
    };
    u64 mine = 0ull;
    if (summed && least_w == 0ull) mine = lane == 0 ? s.warp_kept[warp] : 0ull;
    else
        each_vec(v0 + lane, v1, 32, [&](int v, float (&x)[kVec]) {
            u64 w[kVec];
            weigh(v, x, w);
#pragma unroll
            for (int j = 0; j < kVec; ++j) mine += w[j];
        });
    const u64 total = sum_all(mine);
    bool rest;
    const u64 target = part_of(u, total, rest);           // (below the total)
    u64 before = s.share_above;
    for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
    if (before <= target && target < before + s.warp_sum[warp]) {
        for (int v = v0; v < v1; v += 32) {
            u64 w[kVec], own = 0ull;
#pragma unroll
            for (int j = 0; j < kVec; ++j) w[j] = 0ull;
            each_vec(v + lane, min(v1, v + 32), 32, [&](int at, float (&x)[kVec]) { weigh(at, x, w); });
#pragma unroll
            for (int j = 0; j < kVec; ++j) own += w[j];
            const u64 scan = warp_scan(own);
            u64 at = before + scan - own;
            const bool here = at <= target && target < at + own;
            before += __shfl_sync(~0u, scan, 31);
            if (here) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    if (at <= target && target < at + w[j]) {
                        const int at_v = (v + lane) * kVec + j;
                        p.tok[row] = first + at_v;
                        if (p.logprob) p.logprob[row] = log_of(R::one(src + at_v), total);
                    }
                    at += w[j];
                }
            }
            if (__any_sync(~0u, here)) break;
        }
    }
    cluster.sync();                              // shared memory stays until all have read it
}

template <typename T>
cudaError_t launch(SampleParams p, cudaStream_t s) {
    constexpr int kVec = Row<T>::kVec;
    // two CTAs to a row, and on an SM: the phases of two rows overlap, and the rows at
    // work fit the L2 for their later passes (512 rows of 151936, settings mixed: 240 us; one CTA 299,
    // four 244, eight that keep the row in shared memory, at an earlier stage, 323 for 265).  Up to 16
    // while that leaves no more CTAs than run at once, and twice
    // as many where slices stay long, since rows that are cut take several times as long
    // as others (64 rows of 151936, settings mixed: two CTAs 92 us, four 62; nothing cut
    // 44 and 31; 128 rows 98 and 77, 52 and 53).
    int ctas = p.V > 16384 ? 2 : 1;
    while (ctas < 16 && (long long)p.N * ctas * 2 <= (p.V >= ctas * 2 * 24576 ? 4 : 2) * num_sms() && p.V > ctas * 4096) ctas *= 2;
    p.ctas = ctas;
    constexpr int kRound = kVec * kThreads;      // (whole rounds of the threads: a thread takes the same group in every slice)
    p.slice = ctas == 1 ? (p.V + kVec - 1) / kVec * kVec : ((p.V + ctas - 1) / ctas + kRound - 1) / kRound * kRound;
    cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
    if (e == cudaSuccess && ctas > 8) e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.N * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T>, p);
}

}  // namespace

cudaError_t launch_sample(const SampleParams& p, cudaStream_t s) { return p.bf16 ? launch<uint16_t>(p, s) : launch<float>(p, s); }

}  // namespace dspark
