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
// Each warp is a worker of its own, with its own share of the list of segments
// (AttnSplit), a ring of units of 32 positions that it fills by cp.async some units
// ahead and into its next segment, and its own maxima, sums and O^T in registers.
// Nothing waits for another warp.  (Warps that share a segment and join at its end,
// with one more warp to prepare the next: 236 us for 64 requests of 2000 positions, 8
// heads of 32 rows, now 172; 225 us for 256 requests of 8 rows, now 159.)  HBM would take
// 51 and 93.  Of 8 rows 56 of 100 issue slots are taken, most by conversions; of 32 rows 41,
// and what is left is latency, since 255 registers a thread leave 8 warps to an SM.
//
// Precision: each row of q is scaled by a power of two to below 1 and held in fp16, keys and
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
constexpr int kUnit = 32;                // positions of a unit
constexpr float kLift = 7.f;             // log2 of a weight at the reference
constexpr float kSlack = 8.f;            // log2 of the growth of a maximum that is let pass
constexpr float kUnset = -3.4e38f;       // a reference before the first score: -inf less it is -inf, and any score is above

// (x - r) * s + n, and l + w, of two columns.  (The difference first: of large scores a
// product that is rounded by itself and one that is not would differ by whole units.)
__device__ __forceinline__ void exponent_pair(float& x0, float& x1, float r0, float r1, float s0, float s1, float n) {
    asm("{\n\t.reg .b64 x, r, s, n;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 r, {%2, %3};\n\tmov.b64 s, {%4, %5};\n\tmov.b64 n, {%6, %6};\n\t"
        "sub.rn.f32x2 x, x, r;\n\tfma.rn.f32x2 x, x, s, n;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(x0), "+f"(x1) : "f"(r0), "f"(r1), "f"(s0), "f"(s1), "f"(n));
}
__device__ __forceinline__ void add_pair(float& l0, float& l1, float w0, float w1) {
    asm("{\n\t.reg .b64 l, w;\n\tmov.b64 l, {%0, %1};\n\tmov.b64 w, {%2, %3};\n\tadd.rn.f32x2 l, l, w;\n\tmov.b64 {%0, %1}, l;\n\t}"
        : "+f"(l0), "+f"(l1) : "f"(w0), "f"(w1));
}
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
    int len, pos0, units;     // cache length, first position, units; 0: no more segments
    int slot;                 // -1: the whole segment, else the partial result's slot
    int seen;                 // positions below it are seen by every row
};

// NT: groups of 8 query rows.  DP: the head size rounded up to 64, 128 or 256.
template <int NT, int DP>
struct Layout {
    static constexpr int kWarps = attn4_warps(NT, DP);
    static constexpr int kSteps = DP / 16;                        // of 16 entries
    static constexpr bool kQRegs = NT * kSteps <= 16;             // Q in registers
    static constexpr int kStage = 2 * kUnit * (DP / 2 + DP / 16);    // bytes of a unit, and room for every head size below
    static constexpr int kStages = DP == 256 ? (NT == 1 ? 3 : 2) : NT == 1 ? 4 : 3;
    static constexpr int kQ = kQRegs ? 0 : kSteps * NT * 32 * 8;  // bytes of a Q tile
    static constexpr int kWarpBytes = kStages * kStage + kQ;
    static constexpr int kTotal = kWarps * kWarpBytes;
    static_assert(kTotal <= 222 * 1024, "shared memory");
};

// kExact: the head fills DP, and rows of scales are whole words.
template <int NT, int DP, bool kExact>
__global__ void __launch_bounds__(Layout<NT, DP>::kWarps * 32, 1) attn4_kernel(const AttnParams p) {
    using L = Layout<NT, DP>;
    constexpr int W = L::kWarps, kStages = L::kStages, kSteps = L::kSteps;
    constexpr int kKeyWords = DP / 32;       // words of a key that a thread reads, and of a value
    constexpr int kValWords = DP / 64;
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ Seg s_seg[W][2];              // the segment being copied, and the one being worked on
    __shared__ uint32_t s_there[W][kStages]; // positions of a unit in the ring that are in the cache
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int D = kExact ? DP : p.D;
    if (tid == 0) grid_launch_dependents();  // the join is scheduled now and waits for this grid
    grid_dependency_wait();
    empty_rows<uint16_t>(p, blockIdx.x, gridDim.x, blockDim.x);
    // workers with neighbouring shares on different SMs: a short list reaches them all
    const int worker = warp * gridDim.x + blockIdx.x;
    const AttnSplit sp(p, p.tile_off[p.B], p.tile_off[0]);
    if (lane == 0) p.split[worker].parts = 0;
    if (worker >= sp.n) return;
    uint8_t* const mine = raw + warp * L::kWarpBytes;

    // ------------------------------------------------------ copies into the ring
    const uint32_t ring = ptx::smem_addr(mine);
    const int code_row = D / 2, scale_row = D / fp4::kGroup;
    // a stage: codes of the keys, of the values, scales of the keys, of the values
    constexpr int kVals = kUnit * (DP / 2), kKeyScales = 2 * kVals, kValScales = kKeyScales + kUnit * (DP / 16);
    int place = sp.first(worker);
    const int end = sp.first(worker + 1);
    int issued = 0, used = 0;                // units so far
    int segs = 0, iunit = 0;                 // segments found, and the next unit of the last one to be copied
    int page_of = -1;                        // of the position that this lane looks up, -1: none
    // the next segment of this worker's share that has positions, into s_seg[segs & 1]
    auto find = [&]() {
        Seg d;
        d.units = 0;
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
            d.slot = whole ? -1 : 2 * worker + (j0 == 0 ? 1 : 0);
            d.seen = rm.len - rm.n + 1;
            if (lane == 0 && j0 == 0 && !whole) p.split[worker] = attn_split_row(sp, s, worker, rm.q0, d.r0, d.rows);
            break;
        }
        if (lane == 0) s_seg[warp][segs & 1] = d;
        __syncwarp();
        ++segs;
        iunit = 0;
    };
    // where a lane's position of the next unit lies
    auto look_up = [&]() {
        const Seg& d = s_seg[warp][(segs - 1) & 1];
        const int pos = d.pos0 + iunit * kUnit + lane;
        page_of = -1;
        if (iunit < d.units && pos < d.len) {
            page_of = __ldg(p.table + (size_t)d.b * p.width + p.by_page(pos));
            if (page_of < 0 || page_of >= p.pages) { raise_status(p.status, kBadPage); page_of = -1; }
        }
    };
    auto issue = [&]() {
        const Seg& d = s_seg[warp][(segs - 1) & 1];
        const int pos = d.pos0 + iunit * kUnit + lane, pg = p.by_page(pos), stage = issued % kStages;
        const long long row = (long long)d.h * p.page_size + (pos - pg * p.page_size);
        const bool there = page_of >= 0;
        const long long codes = there ? page_of * p.page_stride + row * code_row : 0, scales = there ? page_of * p.scale_stride + row * scale_row : 0;
        const uint32_t mask = __ballot_sync(~0u, there);
        const uint32_t to = ring + stage * L::kStage;
        if (lane == 0) s_there[warp][stage] = mask;
        const uint8_t *k = static_cast<const uint8_t*>(p.k), *v = static_cast<const uint8_t*>(p.v);
        if constexpr (kExact) {
            constexpr int kChunks = DP / 32;                     // of a row's codes
#pragma unroll
            for (int i = 0; i < kUnit * kChunks / 32; ++i) {
                const int r = i * (32 / kChunks) + lane / kChunks, at = (lane % kChunks) * 16;
                const long long o = __shfl_sync(~0u, codes, r) + at;      // (of row 0 where there is none)
                const bool ok = mask >> r & 1u;
                copy_async<16>(to + r * (DP / 2) + at, k + o, ok);
                copy_async<16>(to + kVals + r * (DP / 2) + at, v + o, ok);
            }
            copy_async<DP / 16>(to + kKeyScales + lane * (DP / 16), p.ks + scales, there);
            copy_async<DP / 16>(to + kValScales + lane * (DP / 16), p.vs + scales, there);
        } else {
            const int chunks = code_row / 8;
            for (int i = 0; i < kUnit * chunks; i += 32) {
                const int c = i + lane, r = c / chunks, at = (c - r * chunks) * 8;
                const long long o = __shfl_sync(~0u, codes, r) + at;
                const bool ok = mask >> r & 1u;
                copy_async<8>(to + r * code_row + at, k + o, ok);
                copy_async<8>(to + kVals + r * code_row + at, v + o, ok);
            }
            uint8_t* st = mine + stage * L::kStage + lane * scale_row;
            for (int i = 0; i < scale_row; ++i) {
                st[kKeyScales + i] = there ? __ldg(p.ks + scales + i) : (uint8_t)0;
                st[kValScales + i] = there ? __ldg(p.vs + scales + i) : (uint8_t)0;
            }
        }
        ptx::cp_async_commit();
        ++issued;
        ++iunit;
        look_up();
    };

    find();
    look_up();
    for (int n = 0;; ++n) {
        if (n == segs) {                     // (nothing of it is copied yet)
            find();
            look_up();
        }
        const Seg d = s_seg[warp][n & 1];
        if (d.units == 0) return;
        // -------------------------------------------------------- a segment
        // the queries: rows scaled below 1 by a power of two, in the order in which the keys' entries are read
        uint2* const qs = reinterpret_cast<uint2*>(mine + kStages * L::kStage) + lane;
        uint2 q[L::kQRegs ? kSteps * NT : 1];
        float by[NT][2], ref[NT][2], sum[NT][2], o[kSteps][NT][4];
#pragma unroll
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
            for (int j = 0; j < kSteps; ++j) top = __vmaxu2(top, __vmaxu2(x[j].x & 0x7fff7fffu, x[j].y & 0x7fff7fffu));
            top = max(top << 16, top & 0xffff0000u);
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            const int e = min(max((int)(top >> 23) - 126, -126), 126);
            const float down = __int_as_float((127 - e) << 23), 
                        up = fminf(fmaxf(p.scale * kLog2e * __int_as_float((127 + e) << 23), 1e-37f), 3e38f);      // (neither 0 nor inf, which -inf and 0 would make NaN)
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                const uint2 y = make_uint2(pack_half(__uint_as_float(x[j].x << 16) * down, __uint_as_float(x[j].x & 0xffff0000u) * down),
                                           pack_half(__uint_as_float(x[j].y << 16) * down, __uint_as_float(x[j].y & 0xffff0000u) * down));
                if constexpr (L::kQRegs) q[j * NT + nt] = y;
                else qs[(j * NT + nt) * 32] = y;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                by[nt][c] = __shfl_sync(~0u, up, (2 * t + c) * 4);
                ref[nt][c] = kUnset;
                sum[nt][c] = 0.f;
            }
        }
        // the last position that a column's row sees
        auto last_of = [&](int col) { return col < d.rows ? d.seen - 1 + p.by_group(d.r0 + col) : 0x7fffffff; };
#pragma unroll
        for (int m = 0; m < kSteps; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[m][nt][c] = 0.f;

#pragma unroll 1
        for (int u = 0; u < d.units; ++u) {
            __syncwarp();                                    // the unit before is done, its stage free
            while (issued - used < kStages) {
                const int units = s_seg[warp][(segs - 1) & 1].units;
                if (iunit < units) { issue(); continue; }
                if (units == 0 || segs > n + 1) break;       // no more, or the next segment is all here
                find();
                look_up();
            }
            if (issued - used == kStages) ptx::cp_async_wait_group<kStages - 1>();
            else ptx::cp_async_wait_group<0>();
            __syncwarp();                                    // this unit has landed
            const int stage = used % kStages;
            const uint8_t* st = mine + stage * L::kStage;
            const uint32_t there = s_there[warp][stage];
            const int pos0 = d.pos0 + u * kUnit;
            // ---------------------------------------------------- S^T = K Q^T
            const int row0 = (g >> 1) + 4 * (g & 1);         // the position of row g; row g + 8 is 8 further, the other tile 16
            float s[2][NT][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[x][nt][c] = 0.f;
            {
                // this thread's entries of four positions, 8 apart, four words (32 entries) at a time
                constexpr int kWords = kKeyWords < 4 ? kKeyWords : 4;
#pragma unroll
                for (int w0 = 0; w0 < kKeyWords; w0 += kWords) {
                    uint32_t k[4][kWords], sc[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint8_t* at = st + (row0 + 8 * i) * code_row + t * (DP / 8) + 4 * w0;
                        if constexpr (kExact && kWords == 4) *reinterpret_cast<uint4*>(k[i]) = *reinterpret_cast<const uint4*>(at);
                        else
#pragma unroll
                            for (int j = 0; j < kWords; j += 2)
                                *reinterpret_cast<uint2*>(k[i] + j) = kExact || t * (DP / 4) + 8 * (w0 + j) < D ? *reinterpret_cast<const uint2*>(at + 4 * j) : make_uint2(0u, 0u);
                    }
                    const uint8_t* ks = st + kKeyScales + row0 * scale_row + t * (DP / 64) + w0 / 2;
#pragma unroll
                    for (int w = 0; w < kWords; ++w) {
                        if (w % 2 == 0) {                    // the next group of 16
                            const bool in = kExact || t * (DP / 4) + 8 * (w0 + w) < D;
                            uint32_t b[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) b[i] = in ? ks[w / 2 + 8 * i * scale_row] : 0u;
#pragma unroll
                            for (int i = 0; i < 4; i += 2) {
                                const uint32_t both = fp4::scale_pair(b[i] | b[i + 1] << 8);
                                sc[i] = __byte_perm(both, both, 0x1010);
                                sc[i + 1] = __byte_perm(both, both, 0x3232);
                            }
                        }
                        uint32_t h[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) fp4::unpack(k[i][w], h[i]);
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const int j = 2 * (w0 + w) + hf;
                            uint32_t a[2][4];
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                a[x][0] = fp4::mul2(h[2 * x][2 * hf], sc[2 * x]);
                                a[x][1] = fp4::mul2(h[2 * x + 1][2 * hf], sc[2 * x + 1]);
                                a[x][2] = fp4::mul2(h[2 * x][2 * hf + 1], sc[2 * x]);
                                a[x][3] = fp4::mul2(h[2 * x + 1][2 * hf + 1], sc[2 * x + 1]);
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint2 b = L::kQRegs ? q[j * NT + nt] : qs[(j * NT + nt) * 32];
                                mma_16816(s[0][nt], a[0], b.x, b.y);
                                mma_16816(s[1][nt], a[1], b.x, b.y);
                            }
                        }
                    }
                }
            }
            // ----------------------------------------------------- weights
            // in units of log2; positions that a row does not see get -inf
            const bool masked = there != ~0u || pos0 + kUnit > d.seen;
            if (masked) {
                int last[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) last[nt][c] = last_of(8 * nt + 2 * t + c);
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int r = row0 + 16 * x + (c >= 2 ? 8 : 0);
                            if (!(there >> r & 1u) || pos0 + r > last[nt][c & 1]) s[x][nt][c] = -INFINITY;
                        }
            }
            // does an exponent exceed its row's reference by more than the slack?
            float high = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float y0 = fmaxf(fmaxf(s[0][nt][0], s[0][nt][2]), fmaxf(s[1][nt][0], s[1][nt][2]));
                float y1 = fmaxf(fmaxf(s[0][nt][1], s[0][nt][3]), fmaxf(s[1][nt][1], s[1][nt][3]));
                exponent_pair(y0, y1, ref[nt][0], ref[nt][1], by[nt][0], by[nt][1], 0.f);
                high = fmaxf(high, fmaxf(y0, y1));
            }
            if (__any_sync(~0u, high > kSlack)) {
                // the references move to the maxima so far
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float top = fmaxf(fmaxf(s[0][nt][c], s[0][nt][c + 2]), fmaxf(s[1][nt][c], s[1][nt][c + 2]));
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
                        const float to = fmaxf(ref[nt][c], top);
                        const float al = ref[nt][c] == kUnset ? 0.f : fast_exp2((ref[nt][c] - to) * by[nt][c]);
                        if (to != ref[nt][c]) {
                            ref[nt][c] = to;
                            sum[nt][c] *= al;
#pragma unroll
                            for (int m = 0; m < kSteps; ++m) {
                                o[m][nt][c] *= al;
                                o[m][nt][c + 2] *= al;
                            }
                        }
                    }
            }
            uint32_t pt[2][NT][2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; c += 2) {
                        float w0 = s[x][nt][c], w1 = s[x][nt][c + 1];
                        exponent_pair(w0, w1, ref[nt][0], ref[nt][1], by[nt][0], by[nt][1], kLift);
                        w0 = fast_exp2(w0);
                        w1 = fast_exp2(w1);
                        add_pair(sum[nt][0], sum[nt][1], w0, w1);
                        pt[x][nt][c / 2] = transposed(pack_half(w0, w1));
                    }
            // -------------------------------------------------- O^T += V^T P^T
            const int word0 = g * kValWords;
            bool later = false;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t vs[4][(kValWords + 1) / 2];         // scale bytes of this thread's groups at its four positions
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int w = 0; w < (kValWords + 1) / 2; ++w) {
                        const int gr = word0 / 2 + w;
                        vs[i][w] = kExact || gr < scale_row ? st[kValScales + (16 * x + t + 4 * i) * scale_row + gr] : 0u;
                    }
                // a NaN among the values of later tokens of the block must not reach the
                // rows that do not see it (0 * NaN): it is left out here and added below
                if (masked) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int w = 0; w < (kValWords + 1) / 2; ++w)
                            if ((vs[i][w] & 0x7fu) == 0x7fu) { vs[i][w] = 0u; later = true; }
                }
                uint32_t words[4][kValWords];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint8_t* at = st + kVals + (16 * x + t + 4 * i) * code_row + 4 * word0;
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
                    uint32_t e0[4], o0[4], e1[4], o1[4];
                    fp4::unpack((v[0] & 0x0f0f0f0fu) | (v[1] << 4 & 0xf0f0f0f0u), e0);
                    fp4::unpack((v[0] >> 4 & 0x0f0f0f0fu) | (v[1] & 0xf0f0f0f0u), o0);
                    fp4::unpack((v[2] & 0x0f0f0f0fu) | (v[3] << 4 & 0xf0f0f0f0u), e1);
                    fp4::unpack((v[2] >> 4 & 0x0f0f0f0fu) | (v[3] & 0xf0f0f0f0u), o1);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint32_t a[4] = {fp4::mul2(e0[b], sa), fp4::mul2(o0[b], sa), fp4::mul2(e1[b], sb), fp4::mul2(o1[b], sb)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_16816(o[4 * w + b][nt], a, pt[x][nt][0], pt[x][nt][1]);
                    }
                }
            }
            if (masked) later = __any_sync(~0u, later);
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
                                if (bad && pos0 + r <= last_of(8 * nt + 2 * t + c))
#pragma unroll
                                    for (int b = 0; b < 4; ++b) o[4 * w + b][nt][c] = o[4 * w + b][nt][c + 2] = NAN;
                    }
                }
            }
            ++used;
        }
        // ------------------------------------------------------- the segment's end
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = sum[nt][c];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(~0u, l, x);
                const int row = 8 * nt + 2 * t + c;
                if (row >= d.rows) continue;
                const int rr = d.r0 + row, tok = p.by_group(rr);
                const bool whole = d.slot < 0;
                // (weights are relative to the reference less kLift; of a row that saw nothing -inf)
                const float base = ref[nt][c] == kUnset ? -INFINITY : fmaf(ref[nt][c], by[nt][c], -kLift);
                const size_t at = whole ? (size_t)(d.q0 + tok) * p.Hq + d.h * p.G + rr - tok * p.G : (size_t)d.slot * p.row_tile + row;
                const float f = whole ? (l != 0.f ? p.out_by / l : 0.f) : p.out_by;
#pragma unroll
                for (int w = 0; w < kValWords; ++w) {
                    const int d0 = 8 * (g * kValWords + w);
                    if (!kExact && d0 >= D) continue;
                    float x[8];
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        x[2 * b] = o[4 * w + b][nt][c] * f;
                        x[2 * b + 1] = o[4 * w + b][nt][c + 2] * f;
                    }
                    if (whole) {
                        uint32_t r[4];
#pragma unroll
                        for (int b = 0; b < 4; ++b) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r[b]) : "f"(x[2 * b + 1]), "f"(x[2 * b]));
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * D + d0) = make_uint4(r[0], r[1], r[2], r[3]);
                    } else {
                        float4* to = reinterpret_cast<float4*>(p.part + at * D + d0);
                        to[0] = make_float4(x[0], x[1], x[2], x[3]);
                        to[1] = make_float4(x[4], x[5], x[6], x[7]);
                    }
                }
                if (g == 0) {
                    if (!whole) *reinterpret_cast<float2*>(part_stats(p) + at * 2) = make_float2(base, l);
                    else if (p.lse) p.lse[at] = l != 0.f ? fmaf(base, kLn2, logf(l)) : -INFINITY;
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
    return launch_dependent(kernel, dim3(p.ctas / L::kWarps), dim3(L::kWarps * 32), L::kTotal, s, p);
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

cudaError_t launch_attn4_mma(const AttnParams& p, cudaStream_t s) {
    return p.row_tile == 8 ? launch_rows<1>(p, s) : p.row_tile == 16 ? launch_rows<2>(p, s) : launch_rows<4>(p, s);
}

}  // namespace dspark
