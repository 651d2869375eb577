// logits.cu -- penalties for repeated tokens, biases and grammar masks on the
// rows of logits a verification (or a draft) draws from.
//
// Row i of request b follows the request's history and the first i tokens of
// its drafted block, so a token's count differs from row to row:
//     c_i(v)  = #{output tokens of the history equal v} + #{j < i : draft_j = v},
//     seen_i(v) = v in the prompt, or c_i(v) > 0,
//     x' = seen ? (x > 0 ? x / rep : x * rep) : x,
//     y  = x' - freq * c_i(v) - pres * [c_i(v) > 0] + bias(v),
//     out = allowed_i(v) ? y : -inf.
// With these rows as the target, the verification stays lossless for the
// constrained distribution: row i is the law after exactly those i drafts.
#include "serve.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;

// The word a vocabulary entry has in shared memory; 0 = nothing to do but the mask.
constexpr uint32_t kPrompt = 1u << 31, kBias = 1u << 30, kDraft = 1u << 29, kCount = kDraft - 1;

template <typename T> struct Row;
template <> struct Row<float> {
    static constexpr int kVec = 4;
    __device__ __forceinline__ static void unpack(const uint4& r, float (&x)[4]) {
        x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
        x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
    }
    __device__ __forceinline__ static uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <> struct Row<uint16_t> {
    static constexpr int kVec = 8;
    __device__ __forceinline__ static void unpack(const uint4& r, float (&x)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ static uint4 pack(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)     // the one rounding of the result (nearest even)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// CTA (range, b): entries [lo, lo + n) of every row of request b.
template <typename T>
__global__ void __launch_bounds__(kThreads) logits_kernel(const LogitsParams p, int range) {
    extern __shared__ __align__(16) uint32_t s_word[];
    __shared__ int s_live[DSPARK_MAX_GAMMA + 1];
    __shared__ int s_tok[DSPARK_MAX_GAMMA + 1];
    __shared__ unsigned s_last;
    constexpr int kVec = Row<T>::kVec;
    const int tid = threadIdx.x, b = blockIdx.y, lo = blockIdx.x * range, n = min(range, p.V - lo);
    for (int i = tid; i < n; i += kThreads) s_word[i] = 0u;
    if (tid <= DSPARK_MAX_GAMMA) {
        s_live[tid] = 0;
        s_tok[tid] = -1;
    }
    __syncthreads();
    if (p.hist) {
        int len = p.hist_len[b], prompt = p.prompt_len ? p.prompt_len[b] : 0;
        if (len < 0 || len > p.hist_stride) {
            if (tid == 0) raise_status(p.status, kBadLength);
            len = max(0, min(len, p.hist_stride));
        }
        const int32_t* h = p.hist + (size_t)b * p.hist_stride;
        for (int i = tid; i < len; i += kThreads) {
            const int v = h[i];
            if (v < 0 || v >= p.V) { raise_status(p.status, kBadToken); continue; }
            const int e = v - lo;
            if (e < 0 || e >= n) continue;
            if (i < prompt) atomicOr(&s_word[e], kPrompt);
            else atomicAdd(&s_word[e], 1u);
        }
    }
    if (p.draft_tok && tid < p.R - 1) {
        const int v = p.draft_tok[(size_t)b * p.draft_stride + tid], e = v - lo;
        if (v < 0 || v >= p.V) raise_status(p.status, kBadToken);
        else if (e >= 0 && e < n) {
            s_tok[tid] = e;
            atomicOr(&s_word[e], kDraft);
        }
    }
    int bias0 = 0, bias1 = 0;
    if (p.bias_tok) {
        bias0 = p.bias_off[b];
        bias1 = p.bias_off[b + 1];
        if (bias0 < 0 || bias1 > p.bias_n || bias0 > bias1) {
            if (tid == 0) raise_status(p.status, kBadLength);
            bias0 = bias1 = 0;
        }
        for (int i = bias0 + tid; i < bias1; i += kThreads) {
            const int v = p.bias_tok[i], e = v - lo;
            // ascending ids: one entry a token, found again by halving
            if (v < 0 || v >= p.V || (i > bias0 && p.bias_tok[i - 1] >= v)) raise_status(p.status, kBadToken);
            else if (e >= 0 && e < n) atomicOr(&s_word[e], kBias);
        }
    }
    __syncthreads();
    const float rep = p.rep ? p.rep[b] : 1.f, freq = p.freq ? p.freq[b] : 0.f, pres = p.pres ? p.pres[b] : 0.f;
    if (tid == 0 && !(rep > 0.f && rep < INFINITY)) raise_status(p.status, kBadInput);

    auto changed = [&](float x, uint32_t w, int e, int i) {
        int c = (int)(w & kCount);
        if (w & kDraft)
            for (int j = 0; j < i; ++j) c += s_tok[j] == e ? 1 : 0;
        if ((w & kPrompt) || c > 0) x = x > 0.f ? x / rep : x * rep;
        x -= freq * (float)c;
        if (c > 0) x -= pres;
        if (w & kBias) {
            int l = bias0, r = bias1;
            while (r - l > 1) {
                const int m = (l + r) >> 1;
                if (p.bias_tok[m] <= lo + e) l = m; else r = m;
            }
            x += p.bias_val[l];
        }
        return x;
    };
    const int vecs = n / kVec, words = (p.V + 31) / 32;
    for (int i = 0; i < p.R; ++i) {
        const size_t row = (size_t)b * p.R + i;
        const T* in = static_cast<const T*>(p.logits) + row * p.row_stride + lo;
        T* out = static_cast<T*>(p.out) + row * p.V + lo;
        const uint32_t* mask = p.mask ? p.mask + row * words : nullptr;
        int live = 0;
        for (int c = tid; c < vecs; c += kThreads) {
            const int e0 = c * kVec;
            uint32_t bits = (1u << kVec) - 1u;
            if (mask) bits &= mask[(lo + e0) >> 5] >> ((lo + e0) & 31);
            float x[kVec];
            uint4 raw = make_uint4(0u, 0u, 0u, 0u);
            if (bits) raw = __ldcs(reinterpret_cast<const uint4*>(in + e0));   // nothing allowed: nothing to read
            Row<T>::unpack(raw, x);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const uint32_t w = s_word[e0 + e];
                if (w) x[e] = changed(x[e], w, e0 + e, i);
                if (!(bits >> e & 1u)) x[e] = -INFINITY;
            }
            raw = Row<T>::pack(x);
            __stcs(reinterpret_cast<uint4*>(out + e0), raw);
            Row<T>::unpack(raw, x);                      // as rounded
#pragma unroll
            for (int e = 0; e < kVec; ++e) live += x[e] > -INFINITY ? 1 : 0;
        }
        live = __reduce_add_sync(~0u, live);
        if ((tid & 31) == 0 && live) atomicAdd(&s_live[i], live);
    }
    // the entries left in each row: integer sums over the CTAs of the request;
    // the last CTA (an arrival ticket) reports them and clears the counters
    __syncthreads();
    if (tid < p.R && s_live[tid]) atomicAdd(&p.counts[(size_t)b * p.R + tid], (unsigned)s_live[tid]);
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(&p.tickets[b], 1u) == gridDim.x - 1 ? 1u : 0u;
    __syncthreads();
    if (s_last) {
        __threadfence();
        if (tid < p.R) {
            const unsigned c = atomicExch(&p.counts[(size_t)b * p.R + tid], 0u);
            if (p.live) p.live[(size_t)b * p.R + tid] = (int)c;
            if (c == 0) raise_status(p.status, kDeadRow);
        }
        if (tid == 0) p.tickets[b] = 0u;
    }
}

template <typename T>
cudaError_t launch(const LogitsParams& p, cudaStream_t s) {
    int range = 8192;
    while (range > 1024 && (long long)p.B * ((p.V + range - 1) / range) < 2LL * num_sms()) range >>= 1;
    logits_kernel<T><<<dim3((p.V + range - 1) / range, p.B), kThreads, range * sizeof(uint32_t), s>>>(p, range);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logits(const LogitsParams& p, cudaStream_t s) {
    return p.bf16 ? launch<uint16_t>(p, s) : launch<float>(p, s);
}

}  // namespace dspark
