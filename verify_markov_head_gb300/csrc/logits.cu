// logits.cu -- penalties for repeated tokens, biases and grammar masks on the
// rows of logits a verification (or a draft) draws from.
//
// Row i of request b follows the request's history and the first i tokens of
// its drafted block, so a token's count differs from row to row:
//     c_i(v)  = #{output tokens of the history equal v} + #{j < i : draft_j = v},
//     seen_i(v) = v in the prompt, or c_i(v) > 0,
//     x' = seen ? (x > 0 ? x / rep : x * rep) : x,
//     y  = x' - freq * c_i(v) - pres * [c_i(v) > 0] + bias(v),
//     out = allowed_i(v) ? y : fill              (fill = -inf unless the caller names another).
// With these rows as the target, the verification stays lossless for the
// constrained distribution: row i is the law after exactly those i drafts.
#include "pdl.cuh"
#include "serve.cuh"
#include "sm100_ptx.cuh"

namespace dspark {
namespace {

// The word a vocabulary entry has in shared memory; 0 = nothing to do but the mask.
// (kOdd beside kBias: the request's bias ids are not all valid and ascending.)
constexpr uint32_t kPrompt = 1u << 31, kBias = 1u << 30, kDraft = 1u << 29, kOdd = 1u << 28, kCount = kOdd - 1;

// The bias of token v where the entries [l, end) are not all valid and ascending: that of
// an entry with v and no larger valid id before it.  (Called, not inlined: 256 requests of
// bf16 rows 181.5 us, with this loop in the rows' 184.7.)
__device__ __noinline__ float bias_among(const int32_t* tok, const float* val, int l, int end, int V, int v) {
    for (int top = -1; l < end && top < v; ++l) {
        const int t = tok[l];
        if (t == v) return val[l];
        if (t < V) top = max(top, t);
    }
    return -0.f;                             // none
}

template <typename T> struct Row;
template <> struct Row<float> {
    static constexpr int kVec = 4;
    __device__ __forceinline__ static float round(float x) { return x; }
    // r with `low` where a bit is clear
    __device__ __forceinline__ static uint4 masked(const uint4& r, uint32_t bits, uint32_t low) {
        return make_uint4(bits & 1u ? r.x : low, bits & 2u ? r.y : low, bits & 4u ? r.z : low, bits & 8u ? r.w : low);
    }
    // entries above -inf among those whose bit is set: all of them where the
    // least entry is (NaN carries through the minimum)
    __device__ __forceinline__ static int live(const uint4& r, uint32_t bits) {
        const float a = __uint_as_float(r.x), b = __uint_as_float(r.y), c = __uint_as_float(r.z), d = __uint_as_float(r.w);
        float m, n;
        asm("min.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
        asm("min.NaN.f32 %0, %1, %2;" : "=f"(n) : "f"(c), "f"(d));
        asm("min.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(n));
        if (!(m > -INFINITY))
            bits &= (a > -INFINITY ? 1u : 0u) | (b > -INFINITY ? 2u : 0u) | (c > -INFINITY ? 4u : 0u) | (d > -INFINITY ? 8u : 0u);
        return __popc(bits);
    }
};
template <> struct Row<uint16_t> {
    static constexpr int kVec = 8;
    // r with `low` (twice in the word) where a bit is clear.  (4 bits) * 0x10204080 has them in the
    // tops of the four bytes; the byte permutation spreads a top over a half word.
    __device__ __forceinline__ static uint4 masked(const uint4& r, uint32_t bits, uint32_t low) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t keep;
            const uint32_t tops = (i < 2 ? bits & 15u : bits >> 4) * 0x10204080u;
            if (i & 1) asm("prmt.b32 %0, %1, 0, 0xbbaa;" : "=r"(keep) : "r"(tops));
            else asm("prmt.b32 %0, %1, 0, 0x9988;" : "=r"(keep) : "r"(tops));
            o[i] = (w[i] & keep) | (low & ~keep);
        }
        return make_uint4(o[0], o[1], o[2], o[3]);
    }
    // the one rounding of the result (nearest even)
    __device__ __forceinline__ static uint16_t round(float x) {
        uint32_t w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(0.f), "f"(x));
        return (uint16_t)w;
    }
    // entries above -inf among those whose bit is set: all of them where the
    // least entry is (NaN carries through the minimum)
    __device__ __forceinline__ static int live(const uint4& r, uint32_t bits) {
        uint32_t m, n;
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(r.x), "r"(r.y));
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(n) : "r"(r.z), "r"(r.w));
        asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(n));
        uint32_t both;
        asm("set.gt.u32.bf16x2 %0, %1, %2;" : "=r"(both) : "r"(m), "r"(0xff80ff80u));
        if (both != 0xffffffffu) {
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
            uint32_t above = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                above |= __uint_as_float(w[i] << 16) > -INFINITY ? 1u << 2 * i : 0u;
                above |= __uint_as_float(w[i] & 0xffff0000u) > -INFINITY ? 2u << 2 * i : 0u;
            }
            bits &= above;
        }
        return __popc(bits);
    }
};

// CTA (range, b, z): entries [lo, lo + n) of rows [z part, (z + 1) part) of request b.
//
// Every logit is read once and written once, so HBM bounds the large calls.  A
// producer thread copies the rows' slices into a ring in shared memory (bulk
// copies, kStages ahead; a slice that the mask empties is not read, and of one
// that keeps little only the 16-byte vectors with an allowed entry), so the
// reads go on while the other warps prepare: what a row needs of the history
// is found once per CTA for all its rows, a word in shared memory per
// vocabulary entry with the output count and flags (prompt, bias, in the
// drafted block), from a scan of the request's history.  The entries with a
// word, few beside the vocabulary, are listed; in each row they are corrected
// in the ring, before the row leaves with the mask applied.
// Measured on one GB300: 64 requests of 8 fp32 rows of 151936, a quarter of
// them under a tight mask, 556 MB: 100 us (5.5 TB/s); 256 requests of 8 bf16
// rows of 129280, half of them under a loose mask, 1067 MB: 182 us (5.9 TB/s; a
// plain copy of these rows takes 156); one request 7.3 us.  On the way, the
// first of them: rows through registers with the formula inlined in the stream
// 283 us, with the listed entries corrected in the output afterwards 119, with
// mask words read by every thread (the first-level cache is small beside this
// much shared memory) 116, whole slices read under tight masks 106.
template <typename T> struct Ring;
template <> struct Ring<float> { static constexpr int kStages = 3, kCtas = 3; };       // 16 KB slices
template <> struct Ring<uint16_t> { static constexpr int kStages = 2, kCtas = 5; };    // 8 KB slices
constexpr long long kDrainCycles = 200000000LL;

// Arrive on an mbarrier once this thread's cp.async so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <typename T, int kPer, int kThreads>
struct Smem {
    static constexpr int kRange = kPer * kThreads * Row<T>::kVec;
    static constexpr int kStages = kPer == 1 ? 4 : Ring<T>::kStages;
    static constexpr int kSlice = kRange * (int)sizeof(T);
    static constexpr int kWord = kStages * kSlice;
    static constexpr int kList = kWord + kRange * 4;
    static constexpr int kMaskWords = kRange / 32;               // of a slice
    static constexpr int kMask = kList + kRange * 2;
    static constexpr int kBar = kMask + kStages * kMaskWords * 4;
    static constexpr int kTotal = kBar + 16 * kStages;
};

template <typename T, bool kMask, int kPer, int kThreads>
__global__ void __launch_bounds__(kThreads + 32, kThreads == 256 ? Ring<T>::kCtas : 2) logits_kernel(const LogitsParams p, const int part) {
    using L = Smem<T, kPer, kThreads>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_listed;
    __shared__ int s_unsorted;                 // the request's bias ids are not all in range and ascending
    __shared__ int s_live[DSPARK_MAX_GAMMA + 1];
    __shared__ int s_tok[DSPARK_MAX_GAMMA + 1];
    __shared__ uint32_t s_abort;
    __shared__ uint32_t s_skip[L::kStages];    // the slice in this stage was not read: nothing of it is allowed
    constexpr int kPast = 8;                     // history tokens a thread has on their way
    constexpr int kVec = Row<T>::kVec, kAll = (1 << kVec) - 1, kStages = L::kStages, range = L::kRange;
    uint32_t* s_word = reinterpret_cast<uint32_t*>(smem + L::kWord);
    uint16_t* s_list = reinterpret_cast<uint16_t*>(smem + L::kList);
    uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem + L::kMask);
    const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.y, lo = blockIdx.x * range, n = min(range, p.V - lo);
    const int words = (p.V + 31) / 32, row0 = blockIdx.z * part, rows = min(part, p.R - row0);
    const uint32_t ring = ptx::smem_addr(smem), bar = ring + L::kBar;
    auto full = [&](int s) { return bar + 8u * s; };
    auto empty = [&](int s) { return bar + 8u * (kStages + s); };
    volatile uint32_t* abort_flag = &s_abort;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) { ptx::mbar_init(full(i), 33); ptx::mbar_init(empty(i), kThreads / 32); }
        s_abort = 0u;
        s_listed = 0;
        s_unsorted = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    grid_dependency_wait();
    const long long wl = wait_limit_of(reinterpret_cast<const unsigned long long*>(p.status) + 1);

    if (tid >= kThreads) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = ptx::policy_evict_first();
        const uint32_t bytes = (uint32_t)n * sizeof(T);
        const T* in = static_cast<const T*>(p.logits) + ((size_t)b * p.R + row0) * p.row_stride + lo;
        const uint32_t* mask = kMask ? p.mask + ((size_t)b * p.R + row0) * words + lo / 32 : nullptr;
        // mask words of a slice, kLane a lane, two rows ahead
        constexpr int kLane = L::kMaskWords / 32, kAhead = 2;
        const int mine = (n + 31) / 32, vecs = n / kVec;
        auto groups_of = [](uint32_t w) {            // vectors of a mask word with an allowed entry
            uint32_t x = w | w >> 1;
            x |= x >> 2;
            if (kVec == 8) x |= x >> 4;
            return __popc(x & (kVec == 8 ? 0x01010101u : 0x11111111u));
        };
        uint32_t ahead[kAhead][kLane];
        auto fetch = [&](int i, uint32_t (&w)[kLane]) {
#pragma unroll
            for (int k = 0; k < kLane; ++k)
                w[k] = i < rows && lane + 32 * k < mine ? __ldg(mask + (size_t)i * words + lane + 32 * k) : 0u;
        };
        if (kMask)
#pragma unroll
            for (int r = 0; r < kAhead; ++r) fetch(r, ahead[r]);
        int filled = 0;
        bool ok = true;
        for (int i0 = 0; i0 < rows && ok; i0 += kAhead) {
#pragma unroll
            for (int r = 0; r < kAhead; ++r) {
                const int i = i0 + r, s = i % kStages;
                if (i >= rows || !ok) break;
                if (i >= kStages) ok = __all_sync(~0u, ptx::mbar_wait_strict(empty(s), (i / kStages - 1) & 1, abort_flag, wl));
                if (!ok) break;
                // how the slice is read: 0 not at all, 1 the vectors that keep an entry, 2 whole
                int how = 2;
                const T* row = in + i * p.row_stride;
                if (kMask) {
                    int groups = 0;              // vectors with an allowed entry
#pragma unroll
                    for (int k = 0; k < kLane; ++k) {
                        groups += groups_of(ahead[r][k]);
                        s_mask[s * L::kMaskWords + lane + 32 * k] = ahead[r][k];
                    }
                    groups = __reduce_add_sync(~0u, groups);
                    how = groups == 0 ? 0 : groups <= vecs / 4 ? 1 : 2;
                    if (how == 1)
#pragma unroll
                        for (int k = 0; k < kLane; ++k)
#pragma unroll
                            for (int g = 0; g < 32 / kVec; ++g)
                                if (ahead[r][k] >> (g * kVec) & (uint32_t)kAll) {
                                    const int c = (lane + 32 * k) * (32 / kVec) + g;
                                    if (c < vecs) ptx::cp_async_16(ring + s * L::kSlice + 16 * c, row + c * kVec, 16u);
                                }
                    fetch(i + kAhead, ahead[r]);
                    __syncwarp();
                }
                // each lane arrives once, or its copies do, and lane 0 once more
                // behind the words that the warp wrote
                if (how == 1) cp_async_arrive(full(s));
                else ptx::mbar_arrive(full(s));
                if (lane == 0) {
                    s_skip[s] = how == 0;
                    if (how == 2) {
                        // (the stage may have been written by copies of the other kind)
                        if (kMask) ptx::fence_proxy_async_smem();
                        ptx::mbar_arrive_expect_tx(full(s), bytes);
                        ptx::bulk_load(ring + s * L::kSlice, row, bytes, full(s), pol);
                    } else ptx::mbar_arrive(full(s));
                }
                filled = i + 1;
            }
        }
        if (!ok && lane == 0) { raise_timeout(p.status, 0); *abort_flag = 1u; }
        // every copy issued lands before the CTA leaves: the last fill of each stage
        if (lane == 0)
            for (int f = max(0, filled - kStages); f < filled; ++f)
                ptx::mbar_wait_drain(full(f % kStages), (f / kStages) & 1, kDrainCycles);
    } else {
        // ----------------------------------------------------------- consumers
        // the request's parameters and the first of its history: on their way first
        const int len_in = p.hist ? p.hist_len[b] : 0, prompt = p.hist && p.prompt_len ? p.prompt_len[b] : 0;
        int bias0 = p.bias_tok ? p.bias_off[b] : 0, bias1 = p.bias_tok ? p.bias_off[b + 1] : 0;
        const float rep = p.rep ? p.rep[b] : 1.f, freq = p.freq ? p.freq[b] : 0.f, pres = p.pres ? p.pres[b] : 0.f;
        const int draft = p.draft_tok && tid < p.R - 1 ? p.draft_tok[(size_t)b * p.draft_stride + tid] : -1;
        const int32_t* h = p.hist + (size_t)b * p.hist_stride;
        int past[kPast];
        auto load_past = [&](int i0) {               // within the row of hist (of no tokens without one); judged by the length later
#pragma unroll
            for (int u = 0; u < kPast; ++u) past[u] = i0 + u * kThreads < p.hist_stride ? __ldg(h + i0 + u * kThreads) : -1;
        };
        load_past(tid);
        for (int i = tid; i < (n + 3) / 4; i += kThreads) reinterpret_cast<uint4*>(s_word)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (tid <= DSPARK_MAX_GAMMA) {
            s_live[tid] = 0;
            s_tok[tid] = -1;
        }
        ptx::named_barrier(1, kThreads);
        if (p.bias_tok) {
            if (bias0 < 0 || bias1 > p.bias_n || bias0 > bias1) {
                if (tid == 0) raise_status(p.status, kBadLength);
                bias0 = bias1 = 0;
            }
            for (int i = bias0 + tid; i < bias1; i += kThreads) {
                const int v = p.bias_tok[i], before = i > bias0 ? p.bias_tok[i - 1] : -1, e = v - lo;
                // ascending ids: one entry a token, found again by halving; else by going through them
                if (v < 0 || v >= p.V || before >= v) {
                    raise_status(p.status, kBadToken);
                    s_unsorted = 1;
                }
                if (e >= 0 && e < n) atomicOr(&s_word[e], kBias);
            }
        }
        if (p.draft_tok && tid < p.R - 1) {
            const int e = draft - lo;
            if (draft < 0 || draft >= p.V) raise_status(p.status, kBadToken);
            else if (e >= 0 && e < n) {
                s_tok[tid] = e;
                atomicOr(&s_word[e], kDraft);
            }
        }
        if (p.hist) {
            int len = len_in;
            if (len < 0 || len > p.hist_stride) {
                if (tid == 0) raise_status(p.status, kBadLength);
                len = max(0, min(len, p.hist_stride));
            }
            for (int i0 = tid; i0 < len; i0 += kThreads * kPast) {
                int cur[kPast];
#pragma unroll
                for (int u = 0; u < kPast; ++u) cur[u] = past[u];
                load_past(i0 + kThreads * kPast);    // the next ones meanwhile
#pragma unroll
                for (int u = 0; u < kPast; ++u) {
                    const int i = i0 + u * kThreads;
                    if (i >= len) break;
                    const unsigned e = (unsigned)(cur[u] - lo);
                    if (e < (unsigned)n) {
                        if (i < prompt) atomicOr(&s_word[e], kPrompt);
                        else atomicAdd(&s_word[e], 1u);
                    } else if ((unsigned)cur[u] >= (unsigned)p.V) raise_status(p.status, kBadToken);
                }
            }
        }
        if (tid == 0 && !(rep > 0.f && rep < INFINITY)) raise_status(p.status, kBadInput);
        ptx::named_barrier(1, kThreads);
        // the list (in any order: entries are corrected one by one)
        for (int i = tid; i < (n + 3) / 4; i += kThreads) {
            const uint4 w = reinterpret_cast<const uint4*>(s_word)[i];
            const int mine = (w.x != 0u) + (w.y != 0u) + (w.z != 0u) + (w.w != 0u);
            if (mine) {
                int at = atomicAdd(&s_listed, mine);
                if (w.x) s_list[at++] = (uint16_t)(4 * i);
                if (w.y) s_list[at++] = (uint16_t)(4 * i + 1);
                if (w.z) s_list[at++] = (uint16_t)(4 * i + 2);
                if (w.w) s_list[at++] = (uint16_t)(4 * i + 3);
                if (s_unsorted)
                    for (int j = 4 * i; j < 4 * i + 4; ++j)
                        if (s_word[j] & kBias) s_word[j] |= kOdd;
            }
        }
        ptx::named_barrier(1, kThreads);
        const int listed = s_listed, vecs = n / kVec;

        uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + ((size_t)b * p.R + row0) * p.V + lo) + tid;
        const size_t out_step = p.V / kVec;
        const int shift = (tid * kVec) & 7;
        bool ok = true;
        for (int i = 0; i < rows; ++i, out += out_step) {
            const int s = i % kStages;
            T* slice = reinterpret_cast<T*>(smem + s * L::kSlice);
            ok = ptx::mbar_wait_strict(full(s), (i / kStages) & 1, abort_flag, wl);
            const bool read = !kMask || !s_skip[s];
            if (read)
                for (int k = tid; k < listed; k += kThreads) {
                    const int e = s_list[k];
                    const uint32_t w = s_word[e];
                    float x = to_f32(slice[e]);
                    int c = (int)(w & kCount);
                    if (w & kDraft)
                        for (int j = 0; j < row0 + i; ++j) c += s_tok[j] == e ? 1 : 0;
                    if ((w & kPrompt) || c > 0) x = x > 0.f ? x / rep : x * rep;
                    x -= freq * (float)c;
                    if (c > 0) x -= pres;
                    if (w & kBias) {
                        int l = bias0, r = bias1;
                        if (w & kOdd) x += bias_among(p.bias_tok, p.bias_val, l, r, p.V, lo + e);
                        else {
                            while (r - l > 1) {
                                const int m = (l + r) >> 1;
                                if (p.bias_tok[m] <= lo + e) l = m; else r = m;
                            }
                            x += p.bias_val[l];
                        }
                    }
                    slice[e] = Row<T>::round(x);
                }
            if (i + kStages < rows && read && tid < listed) ptx::fence_proxy_async_smem();   // before the next copy into this stage
            if (ptx::bar_red_or(1, kThreads, !ok)) { ok = false; break; }
            int live = 0;                            // entries left of this row, this thread's
            uint4 raw[kPer];
            uint32_t bits[kPer];
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                bits[j] = (uint32_t)kAll;
                // a byte of the mask: the bits of one vector of 8, or of two of 4
                if (kMask) bits[j] &= reinterpret_cast<const uint8_t*>(s_mask)[s * L::kMaskWords * 4 + tid * kVec / 8 + j * (kThreads * kVec / 8)] >> shift;
                raw[j] = make_uint4(p.low, p.low, p.low, p.low);
                if (read && tid + j * kThreads < vecs) raw[j] = reinterpret_cast<const uint4*>(slice)[tid + j * kThreads];
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(empty(s));
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if (tid + j * kThreads >= vecs) continue;
                live += Row<T>::live(raw[j], bits[j]);
                if (kMask && bits[j] != (uint32_t)kAll) raw[j] = Row<T>::masked(raw[j], bits[j], p.low);
                out[j * kThreads] = raw[j];
            }
            live = __reduce_add_sync(~0u, live);
            if (lane == 0 && live) atomicAdd(&s_live[i], live);
        }
        if (!ok && tid == 0) { raise_timeout(p.status, 1); *abort_flag = 1u; }
        // the entries left in each row: one 64-bit addition per CTA and row, arrivals
        // above, entries below, so the last CTA to arrive has the sum (of integers:
        // any order gives the same) and clears it for the next call
        ptx::named_barrier(1, kThreads);
        if (tid < rows) {
            unsigned long long* at = p.counts + (size_t)b * p.R + row0 + tid;
            const unsigned long long add = 1ull << 32 | (unsigned)s_live[tid], sum = atomicAdd(at, add) + add;
            if ((sum >> 32) == gridDim.x) {
                *at = 0ull;
                if (p.live) p.live[(size_t)b * p.R + row0 + tid] = (int)(uint32_t)sum;
                if ((uint32_t)sum == 0u) raise_status(p.status, kDeadRow);
            }
        }
    }
}

template <typename T, bool kMask, int kPer, int kThreads>
cudaError_t launch(const LogitsParams& p, cudaStream_t s) {
    using L = Smem<T, kPer, kThreads>;
    const cudaError_t e = cudaFuncSetAttribute(logits_kernel<T, kMask, kPer, kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
    if (e != cudaSuccess) return e;
    // few CTAs: the rows of a request split over several, which saves the rows' turn
    const int ranges = (p.V + L::kRange - 1) / L::kRange;
    int parts = 1;
    while (2 * parts <= p.R && 2LL * parts * ranges * p.B <= 3LL * num_sms()) parts *= 2;
    const int part = (p.R + parts - 1) / parts;
    return launch_dependent(logits_kernel<T, kMask, kPer, kThreads>, dim3(ranges, p.B, (p.R + part - 1) / part), dim3(kThreads + 32),
                            (size_t)L::kTotal, s, p, part);
}

// Entries of a CTA: 4096 (8192: b64 146 us, not 100; 512 threads: 108), or 2048
// where that leaves SMs idle, and then, where it still does, 512 threads, which
// read a history in half the turns (one request: 7.3 us, 8.1 with 256 threads).
template <typename T, bool kMask>
cudaError_t launch_range(const LogitsParams& p, cudaStream_t s) {
    constexpr int kUnit = 256 * Row<T>::kVec;
    auto fills = [&](int range) { return (long long)p.B * ((p.V + range - 1) / range) >= 2LL * num_sms(); };
    if constexpr (kUnit == 1024) {
        if (fills(4096)) return launch<T, kMask, 4, 256>(p, s);
        if (fills(2048)) return launch<T, kMask, 2, 256>(p, s);
    } else {
        if (fills(4096)) return launch<T, kMask, 2, 256>(p, s);
        if (fills(2048)) return launch<T, kMask, 1, 256>(p, s);
    }
    return launch<T, kMask, 1, 512>(p, s);
}

}  // namespace

cudaError_t launch_logits(const LogitsParams& p, cudaStream_t s) {
    if (p.mask) return p.bf16 ? launch_range<uint16_t, true>(p, s) : launch_range<float, true>(p, s);
    return p.bf16 ? launch_range<uint16_t, false>(p, s) : launch_range<float, false>(p, s);
}

}  // namespace dspark
