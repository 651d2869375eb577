// sample.cu -- a token of each row of logits, with temperature, top-k, top-p and
// min-p, from a given random number (definition: include/dspark.h).
//
// A cluster of CTAs takes a row and keeps it in shared memory: it is read from
// HBM once, whatever is asked of it.  With weights w_v = e^((x_v - max) / T):
//   thresholds  the k-th largest entry, and the entry at which the descending sum of
//               weights reaches top_p of the total, by digits of the entries' bits
//               taken as ordered integers (11, 11 and 10 bits, 11 and 5 of bf16):
//               a histogram of counts, or of weights, over the row, the digit in
//               which the wanted count or sum is reached, then the next digit of
//               the entries that share it.  No sort.
//   the draw    sums of the weights left, by warp and CTA in the order of the ids, and a
//               walk through the one warp's share that holds u times the total.
//
// A token's boundaries are sums over up to 2^19 entries, and a sum that is off by
// 2^-24 moves the draw across one in a row of some thousand (the boundaries of a
// flat row are 10^-5 apart).  So weights are integers of 2^-42 of the largest:
// sums are exact, and the same in any order, atomics among them.  A weight is
//     2^(y - M),  y = x log2(e) / T = k / 64 + r,  |r| <= 2^-7,
// the product y in two floats, 2^(k mod 64 / 64) from a table of integers, and
// 2^r - 1 by its series to r^4: off by 2^-31 of the weight.  In double precision it
// would be the FP64 units' two operations a cycle that bound the kernel.
#include <cooperative_groups.h>

#include "pdl.cuh"
#include "serve.cuh"

namespace dspark {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32, kBins = 2048;
constexpr int kUnit = 42;                        // a weight of 1 is 2^kUnit
constexpr uint32_t kLowest = 0x007fffffu;        // the key of -inf
constexpr uint32_t kAll = 0xffffffffu;

using u64 = unsigned long long;

// 2^(j / 64) * 2^kUnit, from the 64th root of 2 (by Newton's method).
struct Powers {
    u64 v[64];
    constexpr Powers() : v{} {
        double root = 2.0;
        for (int i = 0; i < 6; ++i) {            // six square roots
            double x = 1.5;
            for (int n = 0; n < 30; ++n) x = 0.5 * (x + root / x);
            root = x;
        }
        for (int j = 0; j < 64; ++j) {
            double x = 1.0, f = root;            // root^j by squares: few roundings
            for (int n = j; n; n >>= 1, f *= f)
                if (n & 1) x *= f;
            v[j] = (u64)(x * (double)(1ull << kUnit) + 0.5);
        }
    }
};
__constant__ Powers c_powers = Powers();

// Integers in the order of the numbers they stand for (no NaN, no -0).
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// log2(e) / temperature in two floats, and what entries are taken from.  In
// double precision, by one thread of a CTA: the FP64 units do two operations a
// cycle, 512 threads would take 4 us.
struct Scale {
    float base, low, c_hi, c_lo;
    __device__ __forceinline__ void set(float top, float T) {
        // entries 50 powers of 2 below the largest weigh nothing.  Where y itself
        // is so large that its fraction is lost, entries are taken from the
        // largest one: exactly, since what still weighs something is that near to it
        const double c = fmin(fmax(1.4426950408889634 / (double)T, 1e-37), 1e30);
        c_hi = (float)c;
        c_lo = (float)(c - (double)c_hi);
        base = fabs(top * c) > 16384.0 ? top : 0.f;
        low = fmaxf((float)((double)(top - base) - 50.0 / c), -3.4e38f);      // (behind the base)
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
    float base, low, c_hi, c_lo;
    int ref;
    const u64* powers;
    // (k, r) of y = k / 64 + r
    __device__ __forceinline__ int split(float x, float& r) const {
        constexpr float kMagic = 196608.f;       // 1.5 * 2^17: a sum's last place is 1 / 64
        const float z = fmaxf(x - base, low), y = z * c_hi;
        const float rest = fmaf(z, c_lo, fmaf(z, c_hi, -y)), m = y + kMagic;
        r = (y - (m - kMagic)) + rest;
        return __float_as_int(m) - __float_as_int(kMagic);
    }
    __device__ __forceinline__ void set(const Scale& c, float top, const u64* table) {
        base = c.base; low = c.low; c_hi = c.c_hi; c_lo = c.c_lo;
        powers = table;
        ref = 0;
        float r;
        ref = split(top, r) >> 6;
    }
    __device__ __forceinline__ u64 operator()(float x) const {
        float r;
        const int k = split(x, r);
        // 2^r - 1 = r ln 2 + (r ln 2)^2 / 2 + ..
        const float p = r * fmaf(r, fmaf(r, fmaf(r, 0.00961812911f, 0.0555041087f), 0.240226507f), 0.693147181f);
        const u64 t = powers[k & 63];
        const int more = __float2int_rn(p * __uint2float_rn((uint32_t)(t >> (kUnit - 30))) * 128.f);      // of 2^-37
        const int down = min(ref - (k >> 6), 63);
        return x == -INFINITY ? 0ull : (t + (u64)((long long)more << (kUnit - 37))) >> down;
    }
};

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
};

struct Shared {
    u64 powers[64];
    uint32_t lo[kBins], hi[kBins];               // counts, or weights in two words
    u64 merged[kBins];                           // this CTA's share of the bins, over the cluster
    u64 warp_sum[kWarps];
    u64 total, sums[2];                          // read by the other CTAs
    u64 found_above, found_at;
    uint32_t found_bin, best;
    Scale scale;
    float floor;                                 // the least entry that min_p keeps
    float top;
    uint32_t bad;
    uint32_t warp_ties[kWarps], ties;
};

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

struct Found { uint32_t key; u64 above, at, want; };   // a key, the sum above it and at it, the sum that was wanted

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p) {
    using R = Row<T>;
    constexpr int kVec = R::kVec;
    extern __shared__ __align__(16) uint8_t raw[];
    Shared& s = *reinterpret_cast<Shared*>(raw);
    uint4* slice = reinterpret_cast<uint4*>(raw + ((sizeof(Shared) + 15) & ~(size_t)15));
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = p.ctas, rank = (int)(blockIdx.x % ctas), row = (int)(blockIdx.x / ctas);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < 64) s.powers[tid] = c_powers.v[tid];
    if (tid == 0) s.bad = 0u;
    __syncthreads();
    grid_dependency_wait();

    // the row's slice, into shared memory; entries that are no numbers become -inf
    const int first = min(p.V, rank * p.slice), count = min(p.V - first, p.slice), vecs = (count + kVec - 1) / kVec;
    const T* src = static_cast<const T*>(p.logits) + row * p.row_stride + first;
    float top = -INFINITY;
    bool bad = false;
#pragma unroll 4
    for (int i = tid; i < vecs; i += kThreads) {
        float x[kVec];
        if ((i + 1) * kVec <= count) R::get(__ldcs(reinterpret_cast<const uint4*>(src) + i), x);
        else
#pragma unroll
            for (int j = 0; j < kVec; ++j) x[j] = i * kVec + j < count ? R::one(src + i * kVec + j) : -INFINITY;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            if (!(x[j] < INFINITY)) { x[j] = -INFINITY; bad = true; }
            x[j] += 0.f;                         // -0 is 0
            top = fmaxf(top, x[j]);
        }
        slice[i] = R::put(x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane == 0) s.warp_sum[warp] = key_of(top);
    if (bad) s.bad = 1u;
    __syncthreads();
    if (tid == 0) {
        uint32_t k = 0u;
        for (int w = 0; w < kWarps; ++w) k = max(k, (uint32_t)s.warp_sum[w]);
        s.top = value_of(k);
        if (s.bad) raise_status(p.status, kBadInput);
    }
    cluster.sync();
    for (int r = 0; r < ctas; ++r) top = fmaxf(top, *cluster.map_shared_rank(&s.top, r));

    // a warp's share of the slice, in the order of the ids
    const int share = (vecs + kWarps - 1) / kWarps, v0 = min(vecs, warp * share), v1 = min(vecs, v0 + share);
    const float T_ = p.temperature ? p.temperature[row] : 1.f;
    const bool T_ok = T_ >= 0.f && T_ < INFINITY;
    float top_p = p.top_p ? p.top_p[row] : 1.f, min_p = p.min_p ? p.min_p[row] : 0.f;
    const int top_k = p.top_k ? p.top_k[row] : 0;
    if (rank == 0 && tid == 0 && (!T_ok || top_p != top_p || min_p != min_p)) raise_status(p.status, kBadInput);
    if (top_p != top_p) top_p = 1.f;
    if (min_p != min_p) min_p = 0.f;

    if (top == -INFINITY) {                      // nothing to draw
        if (rank == 0 && tid == 0) {
            raise_status(p.status, kDeadRow);
            p.tok[row] = -1;
            if (p.logprob) p.logprob[row] = -INFINITY;
        }
    } else if (!T_ok || T_ == 0.f) {             // the lowest id of the largest
        uint32_t best = kAll;
        for (int v = v0 + lane; v < v1; v += 32) {
            float x[kVec];
            R::get(slice[v], x);
#pragma unroll
            for (int j = kVec - 1; j >= 0; --j)
                if (x[j] == top) best = min(best, (uint32_t)(first + v * kVec + j));
        }
        best = __reduce_min_sync(~0u, best);
        if (lane == 0) s.warp_ties[warp] = best;
        __syncthreads();
        if (tid == 0) {
            for (int w = 0; w < kWarps; ++w) best = min(best, s.warp_ties[w]);
            s.best = best;
        }
        cluster.sync();
        if (rank == 0 && tid == 0) {
            for (int r = 0; r < ctas; ++r) best = min(best, *cluster.map_shared_rank(&s.best, r));
            p.tok[row] = (int)best;
            if (p.logprob) p.logprob[row] = 0.f;
        }
    } else {
        if (tid == 0) {
            s.scale.set(top, T_);
            // (rounded up: an entry is kept where it is not below the exact border)
            s.floor = min_p > 0.f ? __double2float_ru((double)top + (double)T_ * log((double)fminf(min_p, 1.f))) : -INFINITY;
        }
        __syncthreads();
        Weigher weight;
        weight.set(s.scale, top, s.powers);
        const int chunk = kBins / ctas;

        // The key above `floor` at which the sum from the largest key down reaches a
        // wanted amount: `want` entries, or weights of `part` of all of them and
        // `beside` together (then the key is `floor` where they do not reach it).
        auto select = [&](bool mass, u64 want, float part, u64 beside, uint32_t floor) {
            Found f{0u, 0ull, 0ull, want};
            int shift = 32;
#pragma unroll 1
            for (int level = 0; level < (sizeof(T) == 2 ? 2 : 3); ++level) {
                const int bits = level == 0 ? 11 : sizeof(T) == 2 ? 5 : level == 1 ? 11 : 10, above = shift;
                shift -= bits;
                for (int i = tid; i < kBins; i += kThreads) s.lo[i] = s.hi[i] = 0u;
                __syncthreads();
                for (int v = tid; v < vecs; v += kThreads) {
                    float x[kVec];
                    R::get(slice[v], x);
#pragma unroll
                    for (int j = 0; j < kVec; ++j) {
                        const uint32_t k = key_of(x[j]);
                        if (k <= floor || (level && k >> above != f.key >> above)) continue;
                        const uint32_t bin = (k >> shift) & ((1u << bits) - 1u);
                        if (mass) {
                            const u64 w = weight(x[j]);
                            const uint32_t lo = (uint32_t)w, old = atomicAdd(&s.lo[bin], lo);
                            const uint32_t hi = (uint32_t)(w >> 32) + (old + lo < old ? 1u : 0u);
                            if (hi) atomicAdd(&s.hi[bin], hi);
                        } else {
                            atomicAdd(&s.lo[bin], 1u);
                        }
                    }
                }
                cluster.sync();
                // the cluster's sums of this CTA's share of the bins
                u64 mine = 0ull;
                for (int i = tid; i < chunk; i += kThreads) {
                    u64 sum = 0ull;
                    for (int r = 0; r < ctas; ++r) {
                        const Shared* o = cluster.map_shared_rank(&s, r);
                        sum += ((u64)o->hi[rank * chunk + i] << 32) + o->lo[rank * chunk + i];
                    }
                    s.merged[i] = sum;
                    mine += sum;
                }
                mine = warp_add(mine);
                if (lane == 0) s.warp_sum[warp] = mine;
                __syncthreads();
                if (tid == 0) {
                    u64 sum = 0ull;
                    for (int w = 0; w < kWarps; ++w) sum += s.warp_sum[w];
                    s.total = sum;
                }
                cluster.sync();
                if (level == 0 && mass) {
                    u64 all = 0ull;
                    for (int r = 0; r < ctas; ++r) all += *cluster.map_shared_rank(&s.total, r);
                    bool rest;
                    const u64 goal = part_of(part, all + beside, rest);
                    f.want = max(1ull, goal + (rest ? 1ull : 0ull));
                    if (f.want > all) { f.key = floor; f.above = all; break; }
                }
                // the share of the bins that the wanted sum is reached in, from the top
                u64 sum = f.above;
                int r = ctas - 1;
                for (; r > 0; --r) {
                    const u64 t = *cluster.map_shared_rank(&s.total, r);
                    if (sum + t >= f.want) break;
                    sum += t;
                }
                // and the bin: the share's bins in descending order, `each` to a thread
                const u64* bins = cluster.map_shared_rank(s.merged, r);
                const int each = (chunk + kThreads - 1) / kThreads;
                u64 own[4], all = 0ull;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = tid * each + e;
                    own[e] = e < each && i < chunk ? bins[chunk - 1 - i] : 0ull;
                    all += own[e];
                }
                const u64 scan = warp_scan(all);
                if (lane == 31) s.warp_sum[warp] = scan;
                __syncthreads();
                u64 before = sum + scan - all;
                for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (before < f.want && before + own[e] >= f.want) {
                        s.found_bin = (uint32_t)(r * chunk + chunk - 1 - (tid * each + e));
                        s.found_above = before;
                        s.found_at = own[e];
                    }
                    before += own[e];
                }
                __syncthreads();
                f.key |= s.found_bin << shift;
                f.above = s.found_above;
                f.at = s.found_at;
            }
            __syncthreads();
            if (sizeof(T) == 2 && f.key != floor && !(f.key & 0x80000000u)) f.key |= 0xffffu;     // (negative: the low bits are set)
            return f;
        };
        // a sum over the cluster of what each thread counted (a place of its own: another
        // CTA may still read the one before)
        auto sum_all = [&](u64 mine, int which) {
            mine = warp_add(mine);
            __syncthreads();
            if (lane == 0) s.warp_sum[warp] = mine;
            __syncthreads();
            if (tid == 0) {
                u64 sum = 0ull;
                for (int w = 0; w < kWarps; ++w) sum += s.warp_sum[w];
                s.sums[which] = sum;
            }
            cluster.sync();
            u64 all = 0ull;
            for (int r = 0; r < ctas; ++r) all += *cluster.map_shared_rank(&s.sums[which], r);
            return all;
        };

        // what is kept: the keys above `cut`, and the first `ties` entries at it
        uint32_t cut = kLowest, ties = 0u;
        if (top_k > 0 && top_k < p.V) {
            u64 mine = 0ull;
            for (int v = tid; v < vecs; v += kThreads) {
                float x[kVec];
                R::get(slice[v], x);
#pragma unroll
                for (int j = 0; j < kVec; ++j) mine += x[j] > -INFINITY ? 1ull : 0ull;
            }
            if ((u64)top_k < sum_all(mine, 0)) {
                const Found f = select(false, (u64)top_k, 0.f, 0ull, kLowest);
                const u64 n = f.want - f.above;
                cut = n < f.at ? f.key : f.key - 1u;
                ties = n < f.at ? (uint32_t)n : 0u;
            }
        }
        if (top_p < 1.f) {
            const u64 at_cut = ties ? weight(value_of(cut)) : 0ull;
            const Found f = select(true, 0ull, fmaxf(top_p, 0.f), at_cut * ties, cut);
            const bool above = f.key != cut;             // reached above the cut
            const u64 w = max(above ? weight(value_of(f.key)) : at_cut, 1ull), n = (f.want - f.above + w - 1ull) / w;
            if (above) {
                const bool all = n * w >= f.at;
                cut = all ? f.key - 1u : f.key;
                ties = all ? 0u : (uint32_t)n;
            } else {
                ties = (uint32_t)min((u64)ties, n);
            }
        }
        if (min_p > 0.f) {
            const uint32_t k = key_of(s.floor + 0.f);
            if (k > cut) { cut = k - 1u; ties = 0u; }
        }

        // entries at the cut in the shares before this warp's
        uint32_t ties_before = 0u;
        if (ties) {
            uint32_t n = 0u;
            for (int v = v0 + lane; v < v1; v += 32) {
                float x[kVec];
                R::get(slice[v], x);
#pragma unroll
                for (int j = 0; j < kVec; ++j) n += key_of(x[j]) == cut ? 1u : 0u;
            }
            n = __reduce_add_sync(~0u, n);
            if (lane == 0) s.warp_ties[warp] = n;
            __syncthreads();
            if (tid == 0) {
                uint32_t sum = 0u;
                for (int w = 0; w < kWarps; ++w) sum += s.warp_ties[w];
                s.ties = sum;
            }
            cluster.sync();
            for (int r = 0; r < rank; ++r) ties_before += *cluster.map_shared_rank(&s.ties, r);
            for (int w = 0; w < warp; ++w) ties_before += s.warp_ties[w];
        }
        // the weights of a vector's entries (0: left out); warps walk their shares in the order of the ids
        uint32_t ties_seen = ties_before;
        auto weigh = [&](int v, u64 (&w)[kVec]) {
            float x[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) x[j] = -INFINITY;
            if (v < v1) R::get(slice[v], x);
            uint32_t mine = 0u, order = 0u;
            if (ties) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) mine += key_of(x[j]) == cut ? 1u : 0u;
                if (__any_sync(~0u, mine)) {
                    uint32_t scan = mine;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t y = __shfl_up_sync(~0u, scan, o);
                        if (lane >= o) scan += y;
                    }
                    order = ties_seen + scan - mine;
                    ties_seen += __shfl_sync(~0u, scan, 31);
                }
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const uint32_t k = key_of(x[j]);
                const bool tie = mine && k == cut;
                w[j] = k > cut || (tie && order < ties) ? weight(x[j]) : 0ull;
                order += tie ? 1u : 0u;
            }
        };
        u64 mine = 0ull;
        for (int v = v0; v < v1; v += 32) {
            u64 w[kVec];
            weigh(v + lane, w);
#pragma unroll
            for (int j = 0; j < kVec; ++j) mine += w[j];
        }
        const u64 total = sum_all(mine, 1);
        bool rest;
        const float u = p.u[row];
        const u64 target = part_of(u > 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f, total, rest);    // (below the total)
        u64 before = 0ull;
        for (int r = 0; r < rank; ++r) before += *cluster.map_shared_rank(&s.sums[1], r);
        for (int w = 0; w < warp; ++w) before += s.warp_sum[w];
        if (before <= target && target < before + s.warp_sum[warp]) {
            ties_seen = ties_before;
            for (int v = v0; v < v1; v += 32) {
                u64 w[kVec], own = 0ull;
                weigh(v + lane, w);
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
                            p.tok[row] = first + (v + lane) * kVec + j;
                            if (p.logprob) {
                                // (a share near 1 by what it lacks)
                                const double lack = (double)(total - w[j]) / (double)total;
                                p.logprob[row] = lack < 0.5 ? log1pf(-(float)lack) : logf((float)((double)w[j] / (double)total));
                            }
                        }
                        at += w[j];
                    }
                }
                if (__any_sync(~0u, here)) break;
            }
        }
    }
    cluster.sync();                              // shared memory stays until all have read it
}

template <typename T>
cudaError_t launch(SampleParams p, cudaStream_t s) {
    constexpr int kVec = Row<T>::kVec;
    const size_t fixed = (sizeof(Shared) + 15) & ~(size_t)15;
    auto bytes = [&](int ctas) { return fixed + (size_t)(((p.V + ctas - 1) / ctas + kVec - 1) / kVec) * 16; };
    // as many CTAs to a row as leave two rows' slices on an SM, more where SMs would be idle
    int ctas = 1;
    while (ctas < 16 && (bytes(ctas) > 112 * 1024 || ((long long)p.N * ctas * 2 <= num_sms() && p.V > ctas * 2048))) ctas *= 2;
    p.ctas = ctas;
    p.slice = ((p.V + ctas - 1) / ctas + kVec - 1) / kVec * kVec;
    const size_t smem = bytes(ctas);
    cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && ctas > 8) e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.N * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
