// attn_rows.cuh -- the rows of an attention over the cache as its kernels see
// them: a request's tokens and length, checked, and the places of results.
#pragma once

#include "serve.cuh"

namespace dspark {

// Start of the partial maxima and sums behind the partial outputs.
__device__ __forceinline__ float* part_stats(const AttnParams& p) {
    return p.part + (size_t)2 * p.ctas * p.row_tile * p.D;
}

// Query row `rr` of request b: token rr / G, head h * G + rr % G.
struct RowMap {
    int q0, n, len;       // first token of the request in q, its tokens, its cache length
    // `reports`: the thread that raises the status
    __device__ __forceinline__ RowMap(const AttnParams& p, int b, bool reports) {
        q0 = p.q_off[b];
        n = p.q_off[b + 1] - q0;
        len = p.kv_len[b];
        // (n is right modulo 2^32; with q0 in range and n in [0, max_new], q0 + n is compared without a sum)
        if (n > p.max_new || n < 0 || q0 < 0 || q0 > p.N - n || (long long)len > (long long)p.width * p.page_size || len < 0) {
            if (reports) raise_status(p.status, kBadLength);
            n = q0 < 0 ? 0 : max(0, min(n, min(p.max_new, p.N - q0)));
            len = max(0, min(len, p.width * p.page_size));
        }
    }
};

template <typename T>
__device__ __forceinline__ void store_out(T* out, float x);
template <>
__device__ __forceinline__ void store_out<float>(float* out, float x) { *out = x; }
template <>
__device__ __forceinline__ void store_out<uint16_t>(uint16_t* out, float x) {
    // the one rounding of the result (nearest even)
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.bf16.f32 h, %1;\n\tmov.b16 %0, h;\n\t}" : "=h"(*out) : "f"(x));
}

// Requests that own no cache position have no tile: their rows are zero.  The
// offsets of every request are compared with its length here.
// (the first `threads` threads of the CTA)
template <typename T>
__device__ __forceinline__ void empty_rows(const AttnParams& p, int cta, int ctas, int threads) {
    for (int b = cta; b < p.B; b += ctas) {
        const int off = p.tile_off[b], next = p.tile_off[b + 1];
        if (threadIdx.x == 0 && !attn_offsets_fit(p, b, off, next)) raise_status(p.status, kBadLength);
        if (next > off) continue;
        const RowMap r(p, b, threadIdx.x == 0);
        const size_t o0 = (size_t)r.q0 * p.Hq * p.D, n = (size_t)r.n * p.Hq * p.D;
        for (size_t i = threadIdx.x; i < n; i += threads) static_cast<T*>(p.out)[o0 + i] = T(0);
        if (p.lse)
            for (int i = threadIdx.x; i < r.n * p.Hq; i += threads) p.lse[(size_t)r.q0 * p.Hq + i] = -INFINITY;
    }
}

}  // namespace dspark
