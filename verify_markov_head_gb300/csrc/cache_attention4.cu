// cache_attention4.cu -- attention over a paged cache held in 4 bits, bf16
// queries (formulas: cache_attention.cu; formats: fp4.cuh; fp32 queries run on
// CUDA cores, cache_attention.cu).
//
// A key-value head's position is 144 bytes at head size 128 (512 in bf16), so HBM
// asks for 3.6 times the positions a second, and what is left to do for each is
// the work: 256 codes become fp16 numbers (two conversions and products to a
// register of two), one 2^x and two products for each row.  Codes that became
// fp16 in shared memory, for tcgen05 to read, would cross it three more times
// (written, and read by two products: 64 KB for 128 positions, where the codes
// are 18 KB); so they are converted in registers, in the layout of mma.sync's A
// operand, and never stored:
//     S^T [16 positions x 8 rows] = K [16 x D] . Q^T       A: keys, B: queries
//     O^T [D x 8 rows]          += V^T [D x 16] . P^T      A: values, B: weights
// The sum over D may take its terms in any order: thread t of a quad reads D/4
// neighbouring entries of a key (16 bytes at head size 128), scales included, and
// the queries are laid out to match.  Of the values a thread reads 8 bytes of
// four positions and pairs the positions' nibbles before they are converted (4
// operations for 16 entries), since A wants two positions in a register.  P^T is
// S^T transposed 8 x 8 (movmatrix).  Which position is which row of S^T is free
// too: rows 2t and 2t + 1 are positions t and t + 4, so that a warp's reads of
// the values meet every bank once.
//
// Each warp is on its own: it takes every W-th unit of 16 positions, copies it by
// cp.async into a ring of its own, some units ahead and into the next segment, and
// keeps its own maxima, sums and O^T in registers; the W results of a segment are
// joined at its end, in the order of the warps.  One more warp prepares the next
// segment (its place in the list, its queries) meanwhile.  No waits but barriers.
//
// Precision: q is scaled by a power of two to below 1 a row and held in fp16, keys and
// values are exact in fp16, products are exact and summed in fp32.  Weights are
// fp16, 2^(s - ref + 7): the reference of a row moves when a score exceeds it by
// more than 8, so the largest lies between 2^7 and 2^15, and one of 2^-21 of the
// largest still has 10 bits.  Their sum l is taken of the fp32 weights.
#include "attn_rows.cuh"
#include "fp4.cuh"
#include "pdl.cuh"
#include "serve.cuh"
#include "sm100_ptx.cuh"

namespace dspark {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kUnit = 16;                // positions of a unit
constexpr float kLift = 7.f;             // log2 of a weight at the reference
constexpr float kSlack = 8.f;            // log2 of the growth of a maximum that is let pass

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {       // an 8 x 8 tile of 16-bit entries over the warp
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Copies of 4, 8 or 16 bytes; `bytes` 0 writes zeros.
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, bool there) {
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(kBytes), "r"(there ? kBytes : 0) : "memory");
}

struct Seg {
    int b, h, q0, r0, rows;   // request, key-value head, first token in q, first query row and their number
    int len, pos0, units;     // cache length, first position, units; -1: no more segments
    int slot;                 // -1: the whole segment, else the partial result's slot
    int seen;                 // positions below it are seen by every row
};

// NT: groups of 8 query rows.  DP: the head size rounded up to 64, 128 or 256.
template <int NT, int DP>
struct Layout {
    static constexpr int kRows = 8 * NT;
    static constexpr int kWarps = NT == 1 && DP <= 128 ? 15 : 7;
    static constexpr int kSteps = DP / 16;                        // of 16 entries
    static constexpr int kStage = 2 * kUnit * (DP / 2 + DP / 16);    // bytes of a unit, and room for every head size below
    static constexpr int kStages = DP == 256 ? (NT == 1 ? 4 : 3) : kWarps == 15 ? 4 : 6;
    static constexpr int kQ = kSteps * NT * 32 * 8;               // bytes of a Q tile
    // the join of the warps, kJoin groups of 8 rows at a time
    static constexpr int kPitch = DP + 2;
    static constexpr int kJoin = NT * kWarps * 8 * DP * 4 <= 65536 ? NT : 65536 / (kWarps * 8 * DP * 4);
    static constexpr int kRing = 0;
    static constexpr int kQs = kRing + kWarps * kStages * kStage;
    static constexpr int kMerge = kQs + 2 * kQ;
    static constexpr int kMergeBytes = kWarps * kJoin * 8 * kPitch * 4;
    static constexpr int kTotal = kMerge + kMergeBytes;
    static_assert(kJoin >= 1 && kTotal <= 220 * 1024, "shared memory");
};

// kExact: the head fills DP, and rows of scales are whole words.
template <int NT, int DP, bool kExact>
__global__ void __launch_bounds__((Layout<NT, DP>::kWarps + 1) * 32, 1) attn4_kernel(const AttnParams p) {
    using L = Layout<NT, DP>;
    constexpr int W = L::kWarps, kRows = L::kRows, kStages = L::kStages, kSteps = L::kSteps;
    constexpr int kKeyWords = DP / 32;       // words of a key that a thread reads, and of a value
    constexpr int kValWords = DP / 64;
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ Seg s_seg[4];
    __shared__ volatile int s_ready;         // segments that are described
    __shared__ float s_by[2][kRows];         // what a row's products are multiplied by: log2(e) * scale * 2^its exponent
    __shared__ int s_last[2][kRows];         // the last position that it sees
    __shared__ float s_ref[W][kRows], s_sum[W][kRows];
    __shared__ uint32_t s_there[W][kStages];   // positions of a unit in the ring that are in the cache
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int D = kExact ? DP : p.D;
    if (tid == 0) {
        grid_launch_dependents();            // the join is scheduled now and waits for this grid
        s_ready = 0;
    }
    grid_dependency_wait();
    const int cta = blockIdx.x;
    empty_rows<uint16_t>(p, cta, gridDim.x);
    const AttnSplit sp(p, p.tile_off[p.B], p.tile_off[0]);
    if (tid == 0) p.split[cta].parts = 0;
    if (cta >= sp.n) return;
    __syncthreads();

    if (warp == W) {
        // ------------------------------------------- segments and their queries
        int place = sp.first(cta);
        const int end = sp.first(cta + 1);
        for (int n = 0;; ++n) {
            Seg d;
            d.units = -1;
            while (place < end) {
                const AttnSegment s = attn_segment(p, sp, place, attn_first_round(p));
                const RowMap rm(p, s.b, lane == 0);
                d.r0 = s.rt * p.row_tile;
                d.rows = max(0, min(p.row_tile, rm.n * p.G - d.r0));
                const int j0 = s.tile(sp, place), j1 = s.tile(sp, end), next = s.t0 + sp.pad + s.tiles;
                if (next <= place) { place = end; break; }         // (offsets that do not ascend)
                place = next;
                if (j0 == j1 || d.rows == 0 || s.tiles != attn_tiles(rm.len)) continue;
                d.b = s.b; d.h = s.h; d.q0 = rm.q0; d.len = rm.len;
                d.pos0 = j0 * kTile;
                d.units = (min(j1 * kTile, rm.len) - d.pos0 + kUnit - 1) / kUnit;
                const bool whole = j0 == 0 && j1 == s.tiles;
                d.slot = whole ? -1 : 2 * cta + (j0 == 0 ? 1 : 0);
                d.seen = rm.len - rm.n + 1;
                if (lane == 0 && j0 == 0 && !whole) p.split[cta] = attn_split_row(sp, s, cta, rm.q0, d.r0, d.rows);
                break;
            }
            if (lane == 0) {
                s_seg[n & 3] = d;
                __threadfence_block();
                s_ready = n + 1;
            }
            if (d.units >= 0) {
                uint2* qs = reinterpret_cast<uint2*>(raw + L::kQs + (n & 1) * L::kQ);
#pragma unroll 1
                for (int nt = 0; nt < NT; ++nt) {
                    const int row = 8 * nt + g, rr = d.r0 + row, tok = p.by_group(rr);
                    const uint16_t* src = static_cast<const uint16_t*>(p.q) + (d.q0 + tok) * p.q_stride + (size_t)(d.h * p.G + rr - tok * p.G) * D;
                    uint2 x[kSteps];
                    uint32_t top = 0u;
#pragma unroll
                    for (int j = 0; j < kSteps; ++j) {
                        const int at = t * (DP / 4) + 4 * j;
                        x[j] = row < d.rows && (kExact || at < D) ? __ldg(reinterpret_cast<const uint2*>(src + at)) : make_uint2(0u, 0u);
                    }
#pragma unroll
                    for (int j = 0; j < kSteps; ++j)
                        top = max(max(max(top, x[j].x << 16 & 0x7fffffffu), x[j].x & 0x7fff0000u), max(x[j].y << 16 & 0x7fffffffu, x[j].y & 0x7fff0000u));
                    top = max(top, __shfl_xor_sync(~0u, top, 1));
                    top = max(top, __shfl_xor_sync(~0u, top, 2));
                    const int e = min(max((int)(top >> 23) - 126, -100), 100);
                    const float by = __int_as_float((127 - e) << 23);
#pragma unroll
                    for (int j = 0; j < kSteps; ++j)
                        qs[(j * NT + nt) * 32 + lane] = make_uint2(
                            pack_half(__uint_as_float(x[j].x << 16) * by, __uint_as_float(x[j].x & 0xffff0000u) * by),
                            pack_half(__uint_as_float(x[j].y << 16) * by, __uint_as_float(x[j].y & 0xffff0000u) * by));
                    if (t == 0) {
                        s_by[n & 1][row] = p.scale * kLog2e * __int_as_float((127 + e) << 23);
                        s_last[n & 1][row] = row < d.rows ? d.seen - 1 + tok : 0x7fffffff;
                    }
                }
            }
            __syncthreads();                 // segment n is ready, segment n - 1 done
            if (d.units < 0) return;
        }
    }

    // ------------------------------------------------------ copies into the ring
    const uint32_t ring = ptx::smem_addr(raw) + L::kRing + warp * (kStages * L::kStage);
    const int code_row = D / 2, scale_row = D / fp4::kGroup;
    // a stage: codes of the keys, of the values, scales of the keys, of the values
    constexpr int kVals = kUnit * (DP / 2), kKeyScales = 2 * kVals, kValScales = kKeyScales + kUnit * (DP / 16);
    int issued = 0, used = 0;                // units so far
    int iseg = 0, iunit = warp;              // the next unit to be copied
    int page_of = -1;                        // of the position that this lane looks up, -1: none
    bool known = false;                      // page_of is that of (iseg, iunit)
    // where a lane's position of the next unit lies
    auto look_up = [&]() {
        known = false;
        const int ready = __shfl_sync(~0u, s_ready, 0);
        __threadfence_block();
        while (iseg < ready) {
            const volatile Seg& d = s_seg[iseg & 3];
            if (d.units < 0) return;
            if (iunit >= d.units) { ++iseg; iunit = warp; continue; }
            const int pos = d.pos0 + iunit * kUnit + (lane & 15);
            page_of = -1;
            if (pos < d.len) {
                page_of = __ldg(p.table + (size_t)d.b * p.width + p.by_page(pos));
                if (page_of < 0 || page_of >= p.pages) { raise_status(p.status, kBadPage); page_of = -1; }
            }
            known = true;
            return;
        }
    };
    auto issue = [&]() {
        const volatile Seg& d = s_seg[iseg & 3];
        const int pos = d.pos0 + iunit * kUnit + (lane & 15), pg = p.by_page(pos), stage = issued % kStages;
        const long long row = (long long)d.h * p.page_size + (pos - pg * p.page_size);
        const bool there = page_of >= 0;
        const long long codes = there ? page_of * p.page_stride + row * code_row : 0, scales = there ? page_of * p.scale_stride + row * scale_row : 0;
        const uint32_t mask = __ballot_sync(~0u, there) & 0xffffu;
        const uint32_t to = ring + stage * L::kStage;
        if (lane == 0) s_there[warp][stage] = mask;
        const uint8_t *k = static_cast<const uint8_t*>(p.k), *v = static_cast<const uint8_t*>(p.v);
        if constexpr (kExact) {
            constexpr int kChunks = DP / 32;                     // of a row's codes
#pragma unroll
            for (int i = 0; i < kUnit * kChunks / 32; ++i) {
                const int c = i * 32 + lane, r = c / kChunks, at = (c % kChunks) * 16;
                const long long o = __shfl_sync(~0u, codes, r) + at;
                const bool ok = mask >> r & 1u;
                copy_async<16>(to + r * (DP / 2) + at, k + (ok ? o : 0), ok);
                copy_async<16>(to + kVals + r * (DP / 2) + at, v + (ok ? o : 0), ok);
            }
            // a row of scales: a lane of the lower half takes the key's, one of the upper the value's
            const uint32_t st = to + (lane < 16 ? kKeyScales : kValScales) + (lane & 15) * (DP / 16);
            copy_async<DP / 16>(st, (lane < 16 ? p.ks : p.vs) + scales, there);
        } else {
            const int chunks = code_row / 8;
            for (int i = 0; i < kUnit * chunks; i += 32) {
                const int c = i + lane, r = min(c / chunks, kUnit - 1), at = (c - r * chunks) * 8;
                const long long o = __shfl_sync(~0u, codes, r) + at;
                const bool ok = mask >> r & 1u;
                if (c < kUnit * chunks) {
                    copy_async<8>(to + r * code_row + at, k + (ok ? o : 0), ok);
                    copy_async<8>(to + kVals + r * code_row + at, v + (ok ? o : 0), ok);
                }
            }
            uint8_t* st = raw + L::kRing + warp * (kStages * L::kStage) + stage * L::kStage + (lane < 16 ? kKeyScales : kValScales) + (lane & 15) * scale_row;
            const uint8_t* from = (lane < 16 ? p.ks : p.vs) + scales;
            for (int i = 0; i < scale_row; ++i) st[i] = there ? __ldg(from + i) : (uint8_t)0;
        }
        ptx::cp_async_commit();
        ++issued;
        iunit += W;
        look_up();
    };

    look_up();
    for (int n = 0;; ++n) {
        __syncthreads();
        const Seg d = s_seg[n & 3];
        if (d.units < 0) return;
        if (!known) look_up();
        // -------------------------------------------------------- a segment
        const uint2* qs = reinterpret_cast<const uint2*>(raw + L::kQs + (n & 1) * L::kQ) + lane;
        float by[NT][2], neg[NT][2], sum[NT][2], o[kSteps][NT][4];   // neg: kLift - reference, +inf: none yet
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                by[nt][c] = s_by[n & 1][8 * nt + 2 * t + c];
                neg[nt][c] = INFINITY;
                sum[nt][c] = 0.f;
            }
#pragma unroll
        for (int m = 0; m < kSteps; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[m][nt][c] = 0.f;
        uint2 q[NT <= 2 ? kSteps * NT : 1];
        if constexpr (NT <= 2)
#pragma unroll
            for (int j = 0; j < kSteps * NT; ++j) q[j] = qs[j * 32];

#pragma unroll 1
        for (int u = warp; u < d.units; u += W) {
            __syncwarp();                                    // the unit before is done, its stage free
            while (issued - used < kStages && known) issue();
            if (issued - used == kStages) ptx::cp_async_wait_group<kStages - 1>();
            else ptx::cp_async_wait_group<0>();
            __syncwarp();                                    // this unit has landed
            const int stage = used % kStages;
            const uint8_t* st = raw + L::kRing + warp * (kStages * L::kStage) + stage * L::kStage;
            const uint32_t there = s_there[warp][stage];
            const int pos0 = d.pos0 + u * kUnit;
            // ---------------------------------------------------- S^T = K Q^T
            const int row0 = (g >> 1) + 4 * (g & 1);         // the position of row g; row g + 8 is 8 further
            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[nt][c] = 0.f;
            {
                uint32_t k0[kKeyWords], k1[kKeyWords];
                const uint8_t* a0 = st + row0 * code_row + t * (DP / 8);
                const uint8_t* a1 = a0 + 8 * code_row;
                if constexpr (kExact && DP >= 128) {
#pragma unroll
                    for (int i = 0; i < kKeyWords / 4; ++i) {
                        *reinterpret_cast<uint4*>(k0 + 4 * i) = reinterpret_cast<const uint4*>(a0)[i];
                        *reinterpret_cast<uint4*>(k1 + 4 * i) = reinterpret_cast<const uint4*>(a1)[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kKeyWords / 2; ++i) {
                        const bool in = kExact || t * (DP / 4) + 16 * i < D;
                        *reinterpret_cast<uint2*>(k0 + 2 * i) = in ? reinterpret_cast<const uint2*>(a0)[i] : make_uint2(0u, 0u);
                        *reinterpret_cast<uint2*>(k1 + 2 * i) = in ? reinterpret_cast<const uint2*>(a1)[i] : make_uint2(0u, 0u);
                    }
                }
                const uint8_t* ks = st + kKeyScales + row0 * scale_row + t * (DP / 64);
                uint32_t sc0 = 0u, sc1 = 0u;
#pragma unroll
                for (int w = 0; w < kKeyWords; ++w) {
                    if (w % 2 == 0) {                        // the next group of 16
                        const bool in = kExact || t * (DP / 4) + 8 * w < D;
                        const uint32_t b0 = in ? ks[w / 2] : 0u, b1 = in ? ks[w / 2 + 8 * scale_row] : 0u;
                        const uint32_t both = fp4::scale_pair(b0 | b1 << 8);
                        sc0 = __byte_perm(both, both, 0x1010);
                        sc1 = __byte_perm(both, both, 0x3232);
                    }
                    uint32_t x[4], y[4];
                    fp4::unpack(k0[w], x);
                    fp4::unpack(k1[w], y);
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint32_t a[4] = {fp4::mul2(x[2 * hf], sc0), fp4::mul2(y[2 * hf], sc1),
                                               fp4::mul2(x[2 * hf + 1], sc0), fp4::mul2(y[2 * hf + 1], sc1)};
                        const int j = 2 * w + hf;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint2 b = NT <= 2 ? q[j * NT + nt] : qs[(j * NT + nt) * 32];
                            mma_16816(s[nt], a, b.x, b.y);
                        }
                    }
                }
            }
            // ----------------------------------------------------- weights
            // in units of log2; positions that a row does not see get -inf
            const bool masked = there != 0xffffu || pos0 + kUnit > d.seen;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[nt][c] *= by[nt][c & 1];
            if (masked) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int r = row0 + (c >= 2 ? 8 : 0);
                        if (!(there >> r & 1u) || pos0 + r > s_last[n & 1][8 * nt + 2 * t + (c & 1)]) s[nt][c] = -INFINITY;
                    }
            }
            bool grown = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) grown |= s[nt][c] + neg[nt][c & 1] > kLift + kSlack;
            if (__any_sync(~0u, grown)) {
                // the references move to the maxima so far
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float top = fmaxf(s[nt][c], s[nt][c + 2]);
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
                        const float to = fminf(neg[nt][c], kLift - top);       // (+inf while nothing is seen)
                        const float al = neg[nt][c] == INFINITY ? 0.f : fast_exp2(to - neg[nt][c]);
                        if (to != neg[nt][c]) {
                            neg[nt][c] = to;
                            sum[nt][c] *= al;
#pragma unroll
                            for (int m = 0; m < kSteps; ++m) {
                                o[m][nt][c] *= al;
                                o[m][nt][c + 2] *= al;
                            }
                        }
                    }
            }
            uint32_t pt[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    // (a row that sees nothing yet: -inf + inf)
                    const float x = s[nt][c] + neg[nt][c & 1];
                    w[c] = fast_exp2(masked && s[nt][c] == -INFINITY ? -INFINITY : x);
                    sum[nt][c & 1] += w[c];
                }
                pt[nt][0] = transposed(pack_half(w[0], w[1]));
                pt[nt][1] = transposed(pack_half(w[2], w[3]));
            }
            // -------------------------------------------------- O^T += V^T P^T
            uint32_t vs[4][(kValWords + 1) / 2];             // scale bytes of this thread's groups at its four positions
            const int word0 = g * kValWords;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int w = 0; w < (kValWords + 1) / 2; ++w) {
                    const int gr = word0 / 2 + w;
                    vs[i][w] = kExact || gr < scale_row ? st[kValScales + (t + 4 * i) * scale_row + gr] : 0u;
                }
            // a NaN among the values of later tokens of the block must not reach the
            // rows that do not see it (0 * NaN): it is left out here and added below
            uint32_t later = 0u;
            if (masked) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int w = 0; w < (kValWords + 1) / 2; ++w)
                        if ((vs[i][w] & 0x7fu) == 0x7fu) { vs[i][w] = 0u; later = 1u; }
                later = __any_sync(~0u, later);
            }
            uint32_t words[4][kValWords];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t* at = st + kVals + (t + 4 * i) * code_row + 4 * word0;
                if constexpr (kValWords == 1) words[i][0] = kExact || 8 * word0 < D ? *reinterpret_cast<const uint32_t*>(at) : 0u;
                else if constexpr (kValWords == 4 && kExact) *reinterpret_cast<uint4*>(words[i]) = *reinterpret_cast<const uint4*>(at);
                else
#pragma unroll
                    for (int w = 0; w < kValWords; w += 2)
                        *reinterpret_cast<uint2*>(words[i] + w) = kExact || 8 * (word0 + w) < D ? *reinterpret_cast<const uint2*>(at + 4 * w) : make_uint2(0u, 0u);
            }
#pragma unroll
            for (int w = 0; w < kValWords; ++w) {
                const uint32_t v[4] = {words[0][w], words[1][w], words[2][w], words[3][w]};
                const uint32_t sa = fp4::scale_pair(vs[0][w / 2] | vs[1][w / 2] << 8), sb = fp4::scale_pair(vs[2][w / 2] | vs[3][w / 2] << 8);
                // even and odd entries of two positions side by side
                uint32_t x[4], y[4], z[4], r[4];
                fp4::unpack((v[0] & 0x0f0f0f0fu) | (v[1] & 0x0f0f0f0fu) << 4, x);
                fp4::unpack((v[0] >> 4 & 0x0f0f0f0fu) | (v[1] & 0xf0f0f0f0u), y);
                fp4::unpack((v[2] & 0x0f0f0f0fu) | (v[3] & 0x0f0f0f0fu) << 4, z);
                fp4::unpack((v[2] >> 4 & 0x0f0f0f0fu) | (v[3] & 0xf0f0f0f0u), r);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint32_t a[4] = {fp4::mul2(x[b], sa), fp4::mul2(y[b], sa), fp4::mul2(z[b], sb), fp4::mul2(r[b], sb)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_16816(o[4 * w + b][nt], a, pt[nt][0], pt[nt][1]);
                }
            }
            if (later) {
#pragma unroll 1
                for (int r = 0; r < kUnit; ++r) {
                    if (!(there >> r & 1u)) continue;
#pragma unroll
                    for (int w = 0; w < kValWords; ++w) {
                        const int gr = (word0 + w) / 2;
                        const bool bad = gr < scale_row && (st[kValScales + r * scale_row + gr] & 0x7fu) == 0x7fu;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                if (bad && pos0 + r <= s_last[n & 1][8 * nt + 2 * t + c])
#pragma unroll
                                    for (int b = 0; b < 4; ++b) o[4 * w + b][nt][c] = o[4 * w + b][nt][c + 2] = NAN;
                    }
                }
            }
            ++used;
        }
        // ------------------------------------------------ the warps' results together
        // (a reference as kLift - neg, -inf where nothing was seen)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x = sum[nt][c];
#pragma unroll
                for (int y = 4; y < 32; y <<= 1) x += __shfl_xor_sync(~0u, x, y);
                if (g == 0) {
                    s_ref[warp][8 * nt + 2 * t + c] = kLift - neg[nt][c];
                    s_sum[warp][8 * nt + 2 * t + c] = x;
                }
            }
        ptx::named_barrier(1, W * 32);
        float* merge = reinterpret_cast<float*>(raw + L::kMerge);
        // entries 2 b, 2 b + 1 of word w (8 entries) of a row lie where eight words' reads and writes meet every bank
        auto at = [&](int row, int w, int b) { return row * L::kPitch + 8 * w + 2 * ((b + (w >> 2)) & 3); };
#pragma unroll
        for (int n0 = 0; n0 < NT; n0 += L::kJoin) {
            if (n0) ptx::named_barrier(1, W * 32);
#pragma unroll
            for (int nt = n0; nt < n0 + L::kJoin; ++nt) {
                float f[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float top = -INFINITY;
#pragma unroll
                    for (int w = 0; w < W; ++w) top = fmaxf(top, s_ref[w][8 * nt + 2 * t + c]);
                    const float mine = s_ref[warp][8 * nt + 2 * t + c];
                    f[c] = mine == -INFINITY ? 0.f : fast_exp2(mine - top);
                }
                float* to = merge + (size_t)(warp * L::kJoin + nt - n0) * 8 * L::kPitch;
#pragma unroll
                for (int m = 0; m < kSteps; ++m)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        *reinterpret_cast<float2*>(to + at(2 * t + c, g * kValWords + m / 4, m % 4)) = make_float2(o[m][nt][c] * f[c], o[m][nt][c + 2] * f[c]);
            }
            ptx::named_barrier(1, W * 32);
            for (int i = tid; i < L::kJoin * 8 * (DP / 2); i += W * 32) {
                const int row = i / (DP / 2), pair = i % (DP / 2), out_row = 8 * n0 + row;
                if (out_row >= d.rows || (!kExact && 2 * pair >= D)) continue;
                float2 x = make_float2(0.f, 0.f);
                float top = -INFINITY, l = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) top = fmaxf(top, s_ref[w][out_row]);
                const int from = (row / 8) * 8 * L::kPitch + at(row % 8, pair / 4, pair % 4);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float2 y = *reinterpret_cast<const float2*>(merge + (size_t)w * L::kJoin * 8 * L::kPitch + from);
                    const float ref = s_ref[w][out_row];
                    x.x += y.x;
                    x.y += y.y;
                    l += ref == -INFINITY ? 0.f : s_sum[w][out_row] * fast_exp2(ref - top);
                }
                x.x *= p.out_by;
                x.y *= p.out_by;
                if (d.slot < 0) {
                    const int rr = d.r0 + out_row, tok = p.by_group(rr);
                    const size_t o0 = (size_t)(d.q0 + tok) * p.Hq + d.h * p.G + rr - tok * p.G;
                    const float inv = l != 0.f ? 1.f / l : 0.f;
                    uint32_t r;
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x.y * inv), "f"(x.x * inv));
                    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + o0 * D + 2 * pair) = r;
                    if (pair == 0 && p.lse) p.lse[o0] = l != 0.f ? (top - kLift) * kLn2 + logf(l) : -INFINITY;
                } else {
                    const size_t o0 = (size_t)d.slot * p.row_tile + out_row;
                    *reinterpret_cast<float2*>(p.part + o0 * D + 2 * pair) = x;
                    if (pair == 0) {
                        float* stats = part_stats(p) + o0 * 2;
                        stats[0] = top == -INFINITY ? -INFINITY : top - kLift;
                        stats[1] = l;
                    }
                }
            }
        }
    }
}

template <int NT, int DP, bool kExact>
cudaError_t launch(const AttnParams& p, cudaStream_t s) {
    using L = Layout<NT, DP>;
    auto kernel = attn4_kernel<NT, DP, kExact>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(p.ctas), dim3((L::kWarps + 1) * 32), L::kTotal, s, p);
}
template <int NT>
cudaError_t launch_rows(const AttnParams& p, cudaStream_t s) {
    if constexpr (NT <= 2) {
        if (p.D > 128) return p.D == 256 ? launch<NT, 256, true>(p, s) : launch<NT, 256, false>(p, s);
    }
    if (p.D > 64) return p.D == 128 ? launch<NT, 128, true>(p, s) : launch<NT, 128, false>(p, s);
    return p.D == 64 ? launch<NT, 64, true>(p, s) : launch<NT, 64, false>(p, s);
}

}  // namespace

int attn4_row_tile(int rows, int D) { return rows <= 8 ? 8 : rows <= 16 || D > 128 ? 16 : 32; }

cudaError_t launch_attn4_mma(const AttnParams& p, cudaStream_t s) {
    return p.row_tile == 8 ? launch_rows<1>(p, s) : p.row_tile == 16 ? launch_rows<2>(p, s) : launch_rows<4>(p, s);
}

}  // namespace dspark
