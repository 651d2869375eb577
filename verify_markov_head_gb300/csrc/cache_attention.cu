// cache_attention.cu -- attention of a block's new tokens over the paged
// key-value cache.
//
// For token i of request b (position p_i = kv_len_b - n_b + i, n_b new tokens)
// and query head h, key-value head h / G:
//     s_j = scale * q . k_j  for the cache positions j <= p_i,
//     o   = sum_j e^(s_j - m) v_j / l,   m = max_j s_j,   l = sum_j e^(s_j - m),
//     lse = m + ln l.
// The G * n_b query rows that share a key-value head are taken together, so
// every key and value is read from HBM once for all of them.  One pass over
// the cache keeps the running maximum and sum of every row; partial results
// (m, l, unnormalised o) of disjoint ranges of positions join exactly:
//     m = max_c m_c,   l = sum_c l_c e^(m_c - m),   o = sum_c o_c e^(m_c - m) / l.
#include "pdl.cuh"
#include "serve.cuh"

namespace dspark {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Start of the partial maxima and sums behind the partial outputs.
__device__ __forceinline__ float* part_stats(const AttnParams& p) {
    return p.part + (size_t)2 * p.ctas * p.row_tile * p.D;
}

// Query row `rr` of request b: token rr / G, head h * G + rr % G.
struct RowMap {
    int q0, n, len;       // first token of the request in q, its tokens, its cache length
    __device__ __forceinline__ RowMap(const AttnParams& p, int b) {
        q0 = p.q_off[b];
        n = p.q_off[b + 1] - q0;
        len = p.kv_len[b];
        if (n > p.max_new || n < 0 || q0 < 0 || q0 + n > p.N || (long long)len > (long long)p.width * p.page_size || len < 0) {
            if (threadIdx.x == 0) raise_status(p.status, kBadLength);
            n = max(0, min(n, min(p.max_new, p.N - q0)));
            if (q0 < 0) n = 0;
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

// Requests that own no cache position have no tile: their rows are zero.
template <typename T>
__device__ __forceinline__ void empty_rows(const AttnParams& p, int cta, int ctas) {
    for (int b = cta; b < p.B; b += ctas) {
        if (p.tile_off[b + 1] > p.tile_off[b]) continue;
        const RowMap r(p, b);
        const size_t o0 = (size_t)r.q0 * p.Hq * p.D, n = (size_t)r.n * p.Hq * p.D;
        for (size_t i = threadIdx.x; i < n; i += blockDim.x) store_out(static_cast<T*>(p.out) + o0 + i, 0.f);
        if (p.lse)
            for (int i = threadIdx.x; i < r.n * p.Hq; i += blockDim.x) p.lse[(size_t)r.q0 * p.Hq + i] = -INFINITY;
    }
}

// --------------------------------------------------- on CUDA cores, any type
// fp32 caches, and bf16 ones with a head size the tensor-core kernel does not
// take.  128 threads; a tile of 64 keys and values in shared memory as fp32.
// Scores: thread t takes position t % 64 and half of the rows.  Outputs: warp
// w takes MR / 4 rows, lane the dimensions 4 lane .. 4 lane + 3 (and + 128).
constexpr int kSimtThreads = 128;

template <typename T, int MR>
__global__ void __launch_bounds__(kSimtThreads) attn_simt_kernel(const AttnParams p) {
    extern __shared__ __align__(16) float smem[];
    const int D = p.D, ldk = D + 4;
    float* sk = smem;                       // [64][D + 4]
    float* sv = sk + kTile * ldk;           // [64][D]
    float* sq = sv + kTile * D;             // [MR][D]
    float* ss = sq + MR * D;                // [MR][64 + 4] scores, then weights
    constexpr int lds = kTile + 4;
    __shared__ float s_m[MR], s_l[MR], s_a[MR];
    __shared__ long long s_base[kTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) grid_launch_dependents();   // the join is scheduled now and waits for this grid
    const int cta = blockIdx.x;
    empty_rows<T>(p, cta, gridDim.x);
    const AttnSplit sp(p, p.tile_off[p.B], p.tile_off[0]);
    if (cta >= sp.n) return;
    const T* kc = static_cast<const T*>(p.k);
    const T* vc = static_cast<const T*>(p.v);
    const float scale2 = p.scale * kLog2e;
    constexpr int RW = MR / 4;              // rows of a warp
    const int end = sp.first(cta + 1);
    for (int t = sp.first(cta); t < end;) {
        const AttnSegment g = attn_segment(p, sp, t, attn_first_round(p));
        const RowMap rm(p, g.b);
        const int r0 = g.rt * p.row_tile;
        const int rows = max(0, min(p.row_tile, rm.n * p.G - r0));
        const int j0 = g.tile(sp, t), j1 = g.tile(sp, end);
        t = g.t0 + sp.pad + g.tiles;             // the next segment
        if (j0 == j1) continue;
        __syncthreads();
        for (int i = tid; i < MR * D; i += kSimtThreads) {
            const int r = i / D, d = i - r * D;
            float x = 0.f;
            if (r < rows) {
                const int rr = r0 + r, tok = rr / p.G;
                x = to_f32(static_cast<const T*>(p.q)[(rm.q0 + tok) * p.q_stride + (size_t)(g.h * p.G + rr - tok * p.G) * D + d]);
            }
            sq[i] = x;
        }
        if (tid < MR) { s_m[tid] = -INFINITY; s_l[tid] = 0.f; }
        float acc[RW][8];
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[r][e] = 0.f;
        for (int j = j0; j < j1; ++j) {
            const int pos0 = j * kTile;
            __syncthreads();
            if (tid < kTile) {
                const int pos = pos0 + tid;
                long long base = -1;
                if (pos < rm.len) {
                    const int pg = pos / p.page_size;
                    const int page = p.table[(size_t)g.b * p.width + pg];
                    if (page >= 0 && page < p.pages)
                        base = page * p.page_stride + ((long long)g.h * p.page_size + (pos - pg * p.page_size)) * D;
                    else raise_status(p.status, kBadPage);
                }
                s_base[tid] = base;
            }
            __syncthreads();
            const int quads = D / 4;
            for (int i = tid; i < kTile * quads; i += kSimtThreads) {
                const int r = i / quads, c = i - r * quads;
                const long long base = s_base[r];
                float4 k4 = make_float4(0.f, 0.f, 0.f, 0.f), v4 = k4;
                if (base >= 0) { k4 = Vec4<T>::load(kc + base + 4 * c); v4 = Vec4<T>::load(vc + base + 4 * c); }
                *reinterpret_cast<float4*>(sk + r * ldk + 4 * c) = k4;
                *reinterpret_cast<float4*>(sv + r * D + 4 * c) = v4;
            }
            __syncthreads();
            {   // scores
                const int tk = tid & (kTile - 1), half = tid / kTile;
                constexpr int RH = MR / 2;
                float s[RH];
#pragma unroll
                for (int r = 0; r < RH; ++r) s[r] = 0.f;
                for (int c = 0; c < D; c += 4) {
                    const float4 k4 = *reinterpret_cast<const float4*>(sk + tk * ldk + c);
#pragma unroll
                    for (int r = 0; r < RH; ++r) {
                        const float4 q4 = *reinterpret_cast<const float4*>(sq + (half * RH + r) * D + c);
                        s[r] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, s[r]))));
                    }
                }
                const bool there = s_base[tk] >= 0;
#pragma unroll
                for (int r = 0; r < RH; ++r) {
                    const int rr = r0 + half * RH + r;
                    const int last = rm.len - rm.n + rr / p.G;     // the row's own position
                    ss[(half * RH + r) * lds + tk] = (there && pos0 + tk <= last) ? s[r] * scale2 : -INFINITY;
                }
            }
            __syncthreads();
            for (int r = warp; r < MR; r += 4) {   // running maximum and sum, base 2
                const float a = ss[r * lds + lane], b = ss[r * lds + 32 + lane];
                float m = fmaxf(a, b);
#pragma unroll
                for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
                const float old = s_m[r];
                m = fmaxf(m, old);
                const float ref = m == -INFINITY ? 0.f : m;
                const float pa = fast_exp2(a - ref), pb = fast_exp2(b - ref);
                ss[r * lds + lane] = pa;
                ss[r * lds + 32 + lane] = pb;
                float sum = pa + pb;
#pragma unroll
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
                if (lane == 0) {
                    const float al = fast_exp2(old - ref);
                    s_a[r] = al;
                    s_l[r] = s_l[r] * al + sum;
                    s_m[r] = m;
                }
            }
            __syncthreads();
            float al[RW];
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                al[r] = s_a[warp * RW + r];
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[r][e] *= al[r];
            }
            const bool d0 = 4 * lane < D, d1 = 4 * lane + 128 < D;
            for (int tk = 0; tk < kTile; ++tk) {
                float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f), v1 = v0;
                if (d0) v0 = *reinterpret_cast<const float4*>(sv + tk * D + 4 * lane);
                if (d1) v1 = *reinterpret_cast<const float4*>(sv + tk * D + 4 * lane + 128);
#pragma unroll
                for (int r = 0; r < RW; ++r) {
                    const float w = ss[(warp * RW + r) * lds + tk];
                    if (w != 0.f) {     // a hidden position adds nothing, whatever its value holds
                        acc[r][0] = fmaf(w, v0.x, acc[r][0]); acc[r][1] = fmaf(w, v0.y, acc[r][1]);
                        acc[r][2] = fmaf(w, v0.z, acc[r][2]); acc[r][3] = fmaf(w, v0.w, acc[r][3]);
                        acc[r][4] = fmaf(w, v1.x, acc[r][4]); acc[r][5] = fmaf(w, v1.y, acc[r][5]);
                        acc[r][6] = fmaf(w, v1.z, acc[r][6]); acc[r][7] = fmaf(w, v1.w, acc[r][7]);
                    }
                }
            }
        }
        __syncthreads();
        const bool whole = j0 == 0 && j1 == g.tiles;
        const int slot = 2 * cta + (j0 == 0 ? 1 : 0);
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const int row = warp * RW + r;
            if (row >= rows) continue;
            const float l = s_l[row], inv = l != 0.f ? 1.f / l : 0.f;
            const int rr = r0 + row, tok = rr / p.G, head = g.h * p.G + rr - tok * p.G;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int d = 4 * lane + 128 * hf;
                if (d >= D) continue;
                if (whole) {
                    T* o = static_cast<T*>(p.out) + ((size_t)(rm.q0 + tok) * p.Hq + head) * D + d;
#pragma unroll
                    for (int e = 0; e < 4; ++e) store_out(o + e, acc[r][4 * hf + e] * inv);
                } else {
                    float* o = p.part + ((size_t)slot * p.row_tile + row) * D + d;
                    *reinterpret_cast<float4*>(o) = make_float4(acc[r][4 * hf], acc[r][4 * hf + 1], acc[r][4 * hf + 2], acc[r][4 * hf + 3]);
                }
            }
            if (lane == 0) {
                if (whole) {
                    if (p.lse) p.lse[(size_t)(rm.q0 + tok) * p.Hq + head] = l != 0.f ? s_m[row] * kLn2 + logf(l) : -INFINITY;
                } else {
                    float* st = part_stats(p) + ((size_t)slot * p.row_tile + row) * 2;
                    st[0] = s_m[row];
                    st[1] = l;
                }
            }
        }
    }
}

// ------------------------------------------------------------------- join
// Block (c, y): the segment that CTA c continues from CTA c - 1, if it began
// there; one warp per row of rows 8 y .. 8 y + 7.  The partial results are
// added in CTA order, so the result does not depend on which CTA ended first.
template <typename T>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnParams p) {
    grid_dependency_wait();
    const int mine = attn_first_round(p);
    const AttnSplit sp(p, p.tile_off[p.B], p.tile_off[0]);
    const int c = blockIdx.x + 1;
    if (c >= sp.n) return;
    const int t = sp.first(c);
    const AttnSegment g = attn_segment(p, sp, t, mine);
    const int t1 = g.t0 + sp.pad;                // the place of its first tile
    if (g.tiles == 0 || t1 >= t || sp.cta_of(t1) != c - 1) return;
    const int last = sp.cta_of(t1 + g.tiles - 1);
    const RowMap rm(p, g.b);
    const int row = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int rr = g.rt * p.row_tile + row;
    if (row >= p.row_tile || rr >= rm.n * p.G) return;
    const float2* stats = reinterpret_cast<const float2*>(part_stats(p));
    auto place = [&](int i) { return (size_t)(i == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + i)) * p.row_tile + row; };
    const int parts = last - c + 2;
    float m = -INFINITY;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, stats[place(i)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    const bool d0 = 4 * lane < p.D, d1 = 4 * lane + 128 < p.D;
    for (int i0 = 0; i0 < parts; i0 += 32) {
        // lane i weighs part i0 + i; the parts' rows are then read 8 at a time
        float w = 0.f, s = 0.f;
        if (i0 + lane < parts) {
            const float2 st = stats[place(i0 + lane)];
            w = fast_exp2(st.x - ref);
            s = w * st.y;
        }
        const int n = min(32, parts - i0);
        for (int j0 = 0; j0 < n; j0 += 8) {
            float4 x[8], y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j0 + j < n) {
                    const float4* at = reinterpret_cast<const float4*>(p.part + place(i0 + j0 + j) * p.D) + lane;
                    if (d0) x[j] = at[0];
                    if (d1) y[j] = at[32];
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float wj = __shfl_sync(~0u, w, j0 + j);
                l += __shfl_sync(~0u, s, j0 + j);
                if (wj != 0.f) {
                    acc[0] = fmaf(wj, x[j].x, acc[0]); acc[1] = fmaf(wj, x[j].y, acc[1]);
                    acc[2] = fmaf(wj, x[j].z, acc[2]); acc[3] = fmaf(wj, x[j].w, acc[3]);
                    acc[4] = fmaf(wj, y[j].x, acc[4]); acc[5] = fmaf(wj, y[j].y, acc[5]);
                    acc[6] = fmaf(wj, y[j].z, acc[6]); acc[7] = fmaf(wj, y[j].w, acc[7]);
                }
            }
        }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int tok = rr / p.G, head = g.h * p.G + rr - tok * p.G;
    const size_t o0 = (size_t)(rm.q0 + tok) * p.Hq + head;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        const int d = 4 * lane + 128 * hf;
        if (d < p.D)
#pragma unroll
            for (int e = 0; e < 4; ++e) store_out(static_cast<T*>(p.out) + o0 * p.D + d + e, acc[4 * hf + e] * inv);
    }
    if (lane == 0 && p.lse) p.lse[o0] = l != 0.f ? m * kLn2 + logf(l) : -INFINITY;
}

template <typename T, int MR>
cudaError_t launch_simt(const AttnParams& p, cudaStream_t s) {
    const size_t smem = sizeof(float) * ((size_t)kTile * (2 * p.D + 4) + (size_t)MR * p.D + (size_t)MR * (kTile + 4));
    cudaError_t e = cudaFuncSetAttribute(attn_simt_kernel<T, MR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    attn_simt_kernel<T, MR><<<p.ctas, kSimtThreads, smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_join(const AttnParams& p, cudaStream_t s) {
    if (p.ctas < 2) return cudaSuccess;
    return launch_dependent(attn_join_kernel<T>, dim3(p.ctas - 1, (p.row_tile + 7) / 8), dim3(256), 0, s, p);
}

}  // namespace

cudaError_t launch_cache_attention(const AttnParams& p, cudaStream_t s) {
    cudaError_t e;
    if (attn_mma_supported(p)) e = launch_attn_mma(p, s);
    else if (p.row_tile == 8) e = p.bf16 ? launch_simt<uint16_t, 8>(p, s) : launch_simt<float, 8>(p, s);
    else e = p.bf16 ? launch_simt<uint16_t, 32>(p, s) : launch_simt<float, 32>(p, s);
    if (e != cudaSuccess) return e;
    return p.bf16 ? launch_join<uint16_t>(p, s) : launch_join<float>(p, s);
}

}  // namespace dspark
