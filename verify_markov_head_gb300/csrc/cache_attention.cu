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
#include "attn_rows.cuh"
#include "fp4.cuh"
#include "pdl.cuh"
#include "serve.cuh"
#include "sm100_ptx.cuh"

namespace dspark {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// --------------------------------------------------- on CUDA cores: fp32
// fp32 arithmetic throughout, so the FMA rate and the shared-memory reads that
// feed it bound a block's many rows, HBM a single row.  256 threads, MR = 8 or 32 rows, TT positions at a time: two
// stages of keys and values by cp.async, 16-byte chunks swizzled so that eight
// positions' chunks lie in different banks.
// Measured on one GB300: 16 requests of 2730-8192 positions, 8 fp32 heads of
// 128, 0.72 GB, 32 rows: 629 us (18 TFLOP/s; 1075 us without the register tiles),
// 4 rows: 245 us (2.9 TB/s), of 8192 positions each 808 and 305; a call of 4
// short requests 12.3 us (14.3 us a call without its programmatic launch, now
// 12.8).  Issue slots are used to 53 %, a warp waits for shared memory and for
// its own products.
//   scores   8 rows x TPT positions a thread over a quarter of the head
//            (lane = position group + 8 * quarter), the quarters summed by
//            shuffles, which leave each thread NR rows of one position;
//   weights  maxima by shuffles and an exchange over the warps, weights to
//            shared memory [position][row];
//   output   8 rows x ND dimensions a thread over 1 / TS of the
//            positions; the TS parts are added at the segment's end.
constexpr int kSimtThreads = 256;

template <int MR, int TT>
struct Simt {
    static constexpr int TPT = MR == 32 ? 4 : 1;            // positions of a thread
    static constexpr int NR = MR == 32 ? 8 : 2;             // rows of a thread after the sum over the quarters
    static constexpr int kRowGroups = MR / 8;
    static constexpr int kTokWarps = TT / (8 * TPT);        // warps that share the positions of a row group
    static constexpr int kScoreWarps = kRowGroups * kTokWarps;
    static constexpr int TS = 8 / kRowGroups;
    static constexpr int ND = TT == 64 ? 4 : 8;             // dimensions of a thread: 4 lane .., and 128 + 4 lane ..
    static size_t bytes(int D) {
        return (size_t)4 * TT * D * sizeof(float) + sizeof(float) * ((size_t)MR * D + TT * MR + (size_t)(TS - 1) * MR * D);
    }
};

// k4: a cache in 4 bits, made fp32 on its way to shared memory by the threads,
// which wait for its codes before a step's arithmetic.
template <int MR, int TT, bool k4>
__global__ void __launch_bounds__(kSimtThreads, 1) attn_simt_kernel(const AttnParams p) {
    using S = Simt<MR, TT>;
    constexpr int E = 4, TPT = S::TPT, NR = S::NR, ND = S::ND;
    extern __shared__ __align__(16) uint8_t raw[];
    const int D = p.D, chunks = D / E, tile_elems = TT * D;
    float* ring = reinterpret_cast<float*>(raw);                     // [2 stages][keys, values][TT][D]
    float* sq = reinterpret_cast<float*>(ring + 4 * tile_elems);   // [MR][D]
    float* sp_ = sq + MR * D;                                // weights [TT][MR]
    float* merge = sp_ + TT * MR;                            // [TS - 1][MR][D]
    __shared__ float s_max[S::kTokWarps][MR], s_sum[S::kTokWarps][MR], s_alpha[MR], s_ref[MR];
    __shared__ long long s_base[2][TT], s_scale[k4 ? 2 : 1][k4 ? TT : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) grid_launch_dependents();   // the join is scheduled now and waits for this grid
    grid_dependency_wait();
    const int cta = blockIdx.x;
    empty_rows<float>(p, cta, gridDim.x, blockDim.x);
    const AttnSplit sp(p, p.tile_off[p.B], p.tile_off[0]);
    if (tid == 0) p.split[cta].parts = 0;
    if (cta >= sp.n) return;
    const float* kc = static_cast<const float*>(p.k);
    const float* vc = static_cast<const float*>(p.v);
    const float scale2 = p.scale * kLog2e;
    // scores: position group and quarter of the head
    const int tg = lane & 7, quarter = lane >> 3, rg = warp / S::kTokWarps, tw = warp % S::kTokWarps;
    const bool scores = warp < S::kScoreWarps;
    const int tok0 = tw * 8 * TPT + tg * TPT;                // the thread's first position
    const int my_tok = MR == 32 ? tok0 + quarter : tok0;     // the position it keeps
    const int my_row = MR == 32 ? rg * 8 : 2 * quarter;      // and its first row
    // output: row group, part of the positions, dimensions
    const int org = warp / S::TS, part = warp % S::TS;
    const int end = sp.first(cta + 1);
    for (int t = sp.first(cta); t < end;) {
        const AttnSegment g = attn_segment(p, sp, t, attn_first_round(p));
        const RowMap rm(p, g.b, tid == 0);
        const int r0 = g.rt * p.row_tile;
        const int rows = max(0, min(p.row_tile, rm.n * p.G - r0));
        const int j0 = g.tile(sp, t), j1 = g.tile(sp, end), next = g.t0 + sp.pad + g.tiles;
        if (next <= t) break;                    // (offsets that do not ascend)
        t = next;                                // the next segment
        if (j0 == j1 || rows == 0 || g.tiles != attn_tiles(rm.len)) continue;
        const int steps = (j1 - j0) * (kTile / TT), first_new = rm.len - rm.n;
        // where position `tid` of a step lies, -1 beyond the end or in a bad page
        auto base_of = [&](int s) {
            const int pos = j0 * kTile + s * TT + tid;
            if (pos >= rm.len) return -1LL;
            const int pg = p.by_page(pos), page = p.table[(size_t)g.b * p.width + pg];
            if (page < 0 || page >= p.pages) { raise_status(p.status, kBadPage); return -1LL; }
            const long long row = (long long)g.h * p.page_size + (pos - pg * p.page_size);
            if constexpr (k4) s_scale[s & 1][tid] = page * p.scale_stride + row * (D / fp4::kGroup);
            return page * p.page_stride + row * (k4 ? D / 2 : D);
        };
        // chunk c of position r (whole groups of 8 chunks are swizzled)
        auto place = [&](int r, int c) { return r * chunks + ((c | 7) < chunks ? c ^ ((r / TPT) & 7) : c); };
        auto issue = [&](int s) {
            const int st = s & 1;
            if constexpr (k4) {
                for (int i = tid; i < TT * (D / 8); i += kSimtThreads) {
                    const int r = i / (D / 8), c = i - r * (D / 8);
                    const long long base = s_base[st][r], scale = s_scale[st][r] + c / 2;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        uint32_t w = 0u, h[4];
                        float by = 0.f;
                        if (base >= 0) {
                            w = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(kv ? p.v : p.k) + base + 4 * c);
                            by = fp4::scale_value((kv ? p.vs : p.ks)[scale]);
                        }
                        fp4::unpack(w, h);
                        float4* to = reinterpret_cast<float4*>(ring + (2 * st + kv) * tile_elems);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 a = fp4::floats(h[2 * e]), b = fp4::floats(h[2 * e + 1]);
                            to[place(r, 2 * c + e)] = make_float4(a.x * by, a.y * by, b.x * by, b.y * by);
                        }
                    }
                }
                return;
            }
            const uint32_t k0 = ptx::smem_addr(ring + 2 * st * tile_elems), v0 = k0 + tile_elems * (uint32_t)sizeof(float);
            for (int i = tid; i < TT * chunks; i += kSimtThreads) {
                const int r = i / chunks, c = i - r * chunks;
                const long long base = s_base[st][r];
                const long long o = base < 0 ? 0 : base + c * E;
                const uint32_t at = (uint32_t)place(r, c) * 16u;
                ptx::cp_async_16(k0 + at, kc + o, base < 0 ? 0u : 16u);
                ptx::cp_async_16(v0 + at, vc + o, base < 0 ? 0u : 16u);
            }
            ptx::cp_async_commit();
        };
        __syncthreads();
        if (tid < TT) s_base[0][tid] = base_of(0);
        for (int i = tid; i < MR * D; i += kSimtThreads) {
            const int r = i / D, d = i - r * D;
            float x = 0.f;
            if (r < rows) {
                const int rr = r0 + r, tok = p.by_group(rr);
                x = static_cast<const float*>(p.q)[(rm.q0 + tok) * p.q_stride + (size_t)(g.h * p.G + rr - tok * p.G) * D + d];
            }
            sq[i] = x;
        }
        __syncthreads();
        issue(0);
        if (tid < TT && steps > 1) s_base[1][tid] = base_of(1);
        float m[NR], l[NR], acc[8][ND];
#pragma unroll
        for (int r = 0; r < NR; ++r) { m[r] = -INFINITY; l[r] = 0.f; }
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int e = 0; e < ND; ++e) acc[r][e] = 0.f;
        for (int s = 0; s < steps; ++s) {
            const int st = s & 1, pos0 = j0 * kTile + s * TT;
            ptx::cp_async_wait_group<0>();
            __syncthreads();                     // the step's tiles are there, the other stage is free
            if (s + 1 < steps) issue(s + 1);
            const long long later = tid < TT && s + 2 < steps ? base_of(s + 2) : -1LL;
            const float4* kt = reinterpret_cast<const float4*>(ring + 2 * st * tile_elems);
            float z[NR];
            if (scores) {
                float a[8][TPT];
#pragma unroll
                for (int r = 0; r < 8; ++r)
#pragma unroll
                    for (int i = 0; i < TPT; ++i) a[r][i] = 0.f;
                for (int c = quarter; c < chunks; c += 4) {
                    float4 k[TPT];
#pragma unroll
                    for (int i = 0; i < TPT; ++i) k[i] = kt[place(tok0 + i, c)];
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float4 q = *reinterpret_cast<const float4*>(sq + (rg * 8 + r) * D + c * E);
#pragma unroll
                        for (int i = 0; i < TPT; ++i)
                            a[r][i] = fmaf(q.x, k[i].x, fmaf(q.y, k[i].y, fmaf(q.z, k[i].z, fmaf(q.w, k[i].w, a[r][i]))));
                    }
                }
                // the sum over the quarters, split on the way
                const bool up2 = quarter & 2, up1 = quarter & 1;
                if constexpr (MR == 32) {
                    float b2[8][2];
#pragma unroll
                    for (int r = 0; r < 8; ++r)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            b2[r][i] = (up2 ? a[r][i + 2] : a[r][i]) + __shfl_xor_sync(~0u, up2 ? a[r][i] : a[r][i + 2], 16);
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        z[r] = (up1 ? b2[r][1] : b2[r][0]) + __shfl_xor_sync(~0u, up1 ? b2[r][0] : b2[r][1], 8);
                } else {
                    float b4[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        b4[r] = (up2 ? a[r + 4][0] : a[r][0]) + __shfl_xor_sync(~0u, up2 ? a[r][0] : a[r + 4][0], 16);
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        z[r] = (up1 ? b4[r + 2] : b4[r]) + __shfl_xor_sync(~0u, up1 ? b4[r] : b4[r + 2], 8);
                }
                const bool there = s_base[st][my_tok] >= 0;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const int last = first_new + p.by_group(r0 + my_row + r);     // the row's own position
                    z[r] = there && pos0 + my_tok <= last ? z[r] * scale2 : -INFINITY;
                }
                // maxima over the warp's positions
                float w[NR];
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    w[r] = z[r];
#pragma unroll
                    for (int o = 1; o < (MR == 32 ? 32 : 8); o <<= 1) w[r] = fmaxf(w[r], __shfl_xor_sync(~0u, w[r], o));
                    if ((MR == 32 ? lane : tg) == 0) s_max[tw][my_row + r] = w[r];
                }
            }
            __syncthreads();
            if (tid < TT && s + 2 < steps) s_base[st][tid] = later;
            if (scores) {
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    float to = m[r];
#pragma unroll
                    for (int w = 0; w < S::kTokWarps; ++w) to = fmaxf(to, s_max[w][my_row + r]);
                    const float ref = to == -INFINITY ? 0.f : to, al = fast_exp2(m[r] - ref), x = fast_exp2(z[r] - ref);
                    m[r] = to;
                    l[r] = fmaf(l[r], al, x);
                    sp_[my_tok * MR + my_row + r] = x;
                    if (tw == 0 && (MR == 32 ? lane : tg) == 0) s_alpha[my_row + r] = al;
                }
            }
            __syncthreads();
            const float* vt = ring + (2 * st + 1) * tile_elems;
            // a hidden position adds nothing, whatever its value holds
            const bool guard = pos0 + TT > first_new + 1;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float al = s_alpha[org * 8 + r];
#pragma unroll
                for (int e = 0; e < ND; ++e) acc[r][e] *= al;
            }
            constexpr int kPart = TT / S::TS;
#pragma unroll 4
            for (int i = 0; i < kPart; ++i) {
                const int tk = part * kPart + i;
                float w[8], v[ND];
                *reinterpret_cast<float4*>(w) = *reinterpret_cast<const float4*>(sp_ + tk * MR + org * 8);
                *reinterpret_cast<float4*>(w + 4) = *reinterpret_cast<const float4*>(sp_ + tk * MR + org * 8 + 4);
#pragma unroll
                for (int hf = 0; hf < ND / 4; ++hf) {
                    const int d = 4 * lane + 128 * hf;
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (d < D) y = *reinterpret_cast<const float4*>(vt + place(tk, d / E) * E);
                    v[4 * hf] = y.x; v[4 * hf + 1] = y.y; v[4 * hf + 2] = y.z; v[4 * hf + 3] = y.w;
                }
                if (guard) {
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        if (w[r] != 0.f)
#pragma unroll
                            for (int e = 0; e < ND; ++e) acc[r][e] = fmaf(w[r], v[e], acc[r][e]);
                } else {
#pragma unroll
                    for (int r = 0; r < 8; ++r)
#pragma unroll
                        for (int e = 0; e < ND; ++e) acc[r][e] = fmaf(w[r], v[e], acc[r][e]);
                }
            }
        }
        // the segment's end: sums over the threads, parts of the output together
        if (scores) {
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                float x = l[r];
#pragma unroll
                for (int o = 1; o < (MR == 32 ? 32 : 8); o <<= 1) x += __shfl_xor_sync(~0u, x, o);
                if ((MR == 32 ? lane : tg) == 0) {
                    s_sum[tw][my_row + r] = x;
                    if (tw == 0) s_ref[my_row + r] = m[r];
                }
            }
        }
        if (part > 0) {
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int e = 0; e < ND; ++e) {
                    const int d = 4 * lane + 128 * (e / 4) + e % 4;
                    if (d < D) merge[((part - 1) * MR + org * 8 + r) * D + d] = acc[r][e];
                }
        }
        __syncthreads();
        if (part > 0) continue;
        const bool whole = j0 == 0 && j1 == g.tiles;
        const int slot = 2 * cta + (j0 == 0 ? 1 : 0);
        if (tid == 0 && j0 == 0 && !whole) p.split[cta] = attn_split_row(sp, g, cta, rm.q0, r0, rows);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int row = org * 8 + r;
            if (row >= rows) continue;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < S::kTokWarps; ++w) sum += s_sum[w][row];
            const float inv = sum != 0.f ? 1.f / sum : 0.f;
            const int rr = r0 + row, tok = p.by_group(rr), head = g.h * p.G + rr - tok * p.G;
            const size_t at = (size_t)(rm.q0 + tok) * p.Hq + head;
#pragma unroll
            for (int e = 0; e < ND; ++e) {
                const int d = 4 * lane + 128 * (e / 4) + e % 4;
                if (d >= D) continue;
                float x = acc[r][e];
#pragma unroll
                for (int w = 0; w < S::TS - 1; ++w) x += merge[(w * MR + row) * D + d];
                if constexpr (k4) x *= p.out_by;
                if (whole) static_cast<float*>(p.out)[at * D + d] = x * inv;
                else p.part[((size_t)slot * p.row_tile + row) * D + d] = x;
            }
            if (lane == 0) {
                if (whole) {
                    if (p.lse) p.lse[at] = sum != 0.f ? s_ref[row] * kLn2 + logf(sum) : -INFINITY;
                } else {
                    float* stats = part_stats(p) + ((size_t)slot * p.row_tile + row) * 2;
                    stats[0] = s_ref[row];
                    stats[1] = sum;
                }
            }
        }
    }
}

// ------------------------------------------------------------------- join
// Block (c, y): the segment that begins in CTA c and ends in another; one warp
// per row of rows 8 y .. 8 y + 7.  The partial results are added in CTA order,
// so the result does not depend on which CTA ended first.  Latency bounds it:
// three dependent loads (what CTA c left, the parts' maxima and sums, the parts
// eight at a time).
// kWide: heads above 128, two vectors a lane.  Without the second one the registers leave
// room for four blocks an SM, of which there are many where every warp of the attention
// leaves parts (a cache in 4 bits, 64 requests of 32 rows: 1216 of them, 23 us with two an SM).
template <typename T, bool kWide>
__global__ void __launch_bounds__(256, kWide ? 2 : 4) attn_join_kernel(const AttnParams p) {
    if (threadIdx.x == 0) grid_launch_dependents();
    grid_dependency_wait();
    const int c = blockIdx.x, row = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int4 w0 = __ldcg(reinterpret_cast<const int4*>(p.split + c));
    const int parts = w0.x, rows = __ldcg(&p.split[c].rows);
    if (row >= rows || parts < 2) return;
    const int rr = w0.w + row;
    const float2* stats = reinterpret_cast<const float2*>(part_stats(p));
    auto place = [&](int i) { return (size_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * p.row_tile + row; };
    float m = -INFINITY;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, stats[place(i)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    const bool d0 = 4 * lane < p.D, d1 = kWide && 4 * lane + 128 < p.D;
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
            float4 x[8], y[kWide ? 8 : 1];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = y[kWide ? j : 0] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j0 + j < n) {
                    const float4* at = reinterpret_cast<const float4*>(p.part + place(i0 + j0 + j) * p.D) + lane;
                    if (d0) x[j] = at[0];
                    if (d1) y[kWide ? j : 0] = at[32];
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float wj = __shfl_sync(~0u, w, j0 + j);
                l += __shfl_sync(~0u, s, j0 + j);
                if (wj != 0.f) {
                    acc[0] = fmaf(wj, x[j].x, acc[0]); acc[1] = fmaf(wj, x[j].y, acc[1]);
                    acc[2] = fmaf(wj, x[j].z, acc[2]); acc[3] = fmaf(wj, x[j].w, acc[3]);
                    if (kWide) {
                        const float4 z = y[kWide ? j : 0];
                        acc[4] = fmaf(wj, z.x, acc[4]); acc[5] = fmaf(wj, z.y, acc[5]);
                        acc[6] = fmaf(wj, z.z, acc[6]); acc[7] = fmaf(wj, z.w, acc[7]);
                    }
                }
            }
        }
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int tok = p.by_group(rr), head = w0.z * p.G + rr - tok * p.G;
    const size_t o0 = (size_t)(w0.y + tok) * p.Hq + head;
#pragma unroll
    for (int hf = 0; hf < (kWide ? 2 : 1); ++hf) {
        const int d = 4 * lane + 128 * hf;
        if (d < p.D)
#pragma unroll
            for (int e = 0; e < 4; ++e) store_out(static_cast<T*>(p.out) + o0 * p.D + d + e, acc[4 * hf + e] * inv);
    }
    if (lane == 0 && p.lse) p.lse[o0] = l != 0.f ? m * kLn2 + logf(l) : -INFINITY;
}

template <int MR, int TT, bool k4>
cudaError_t launch_simt_tile(const AttnParams& p, cudaStream_t s) {
    const size_t smem = Simt<MR, TT>::bytes(p.D);
    cudaError_t e = cudaFuncSetAttribute(attn_simt_kernel<MR, TT, k4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(attn_simt_kernel<MR, TT, k4>, dim3(p.ctas), dim3(kSimtThreads), smem, s, p);
}
template <int MR, bool k4>
cudaError_t launch_simt(const AttnParams& p, cudaStream_t s) {
    // 64 positions at a time as far as shared memory holds two stages of them
    return p.D <= 128 ? launch_simt_tile<MR, 64, k4>(p, s) : launch_simt_tile<MR, 32, k4>(p, s);
}

cudaError_t launch_join(const AttnParams& p, cudaStream_t s) {
    auto kernel = p.D > 128 ? (p.bf16 ? attn_join_kernel<uint16_t, true> : attn_join_kernel<float, true>)
                            : (p.bf16 ? attn_join_kernel<uint16_t, false> : attn_join_kernel<float, false>);
    return launch_dependent(kernel, dim3(p.ctas, (p.row_tile + 7) / 8), dim3(256), 0, s, p);
}

}  // namespace

cudaError_t launch_cache_attention(const AttnParams& p, cudaStream_t s) {
    cudaError_t e;
    if (p.bf16) e = launch_attn_mma(p, s);
    else e = p.row_tile == 8 ? launch_simt<8, false>(p, s) : launch_simt<32, false>(p, s);
    return e == cudaSuccess ? launch_join(p, s) : e;
}

cudaError_t launch_cache_attention4(const AttnParams& p, bool tensor, cudaStream_t s) {
    cudaError_t e;
    if (tensor) e = launch_attn4_tensor(p, s);
    else if (p.bf16) e = launch_attn4_mma(p, s);
    else e = p.row_tile == 8 ? launch_simt<8, true>(p, s) : launch_simt<32, true>(p, s);
    return e == cudaSuccess ? launch_join(p, s) : e;
}

}  // namespace dspark
