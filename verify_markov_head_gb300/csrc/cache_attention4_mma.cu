// cache_attention4_mma.cu -- attention over a paged cache held in 4 bits on the
// tensor cores: bf16 queries, head size 128, more than 32 query rows a key-value head, or
// more than 16 of few requests (formulas: cache_attention.cu; formats: fp4.cuh; fewer rows
// and other head sizes: cache_attention4.cu).
//
// Both products are taken transposed, 128 cache positions at a time:
//     S^T [128 positions x 64] = K [128 x 128] . Q^T       (A: K, B: Q)
//     O^T [128 entries x 64]  += V^T [128 x 128] . P^T     (A: V^T, B: P)
// with A in tensor memory.  The codes (18 KB for 128 positions) come to shared memory
// by TMA; eight warps turn them into fp16 in registers, exactly, and write
// them straight into tensor memory, as the rows of A: 64 KB that do not cross shared
// memory, where the products would read them at 64 bytes a cycle (cache_attention_mma.cu).
//   keys     a lane of A is a position: a thread takes its 64 bytes of codes and 8
//            scales; TMA's 64-byte swizzle keeps the threads' reads apart
//   values   a lane of A is an entry of the head: a thread takes 4 entries of four
//            positions at a time, pairs the positions' nibbles (4 operations for 16
//            entries) and writes fragments of 16 lanes.  Position r of 16 is the
//            product's step 2r mod 8 + ..: P's rows are written in that order.
// The products are issued in a fixed order, S of a step and O of the step before, with two
// buffers of P, so that the softmax of a step runs beside them.
// The softmax, the segments and the split over CTAs are cache_attention_mma.cu's; weights
// are fp16, 2^(s - ref + 7), as in cache_attention4.cu, whose notes on precision hold
// here too, except that a row of q is scaled to below 2^15, so that fp16 keeps all of a
// bf16 entry down to 2^-29 of the row's largest.  (Each row by its own power of two: of one
// for 16 rows a NaN, an infinity or a large row took the others' entries below fp16's range.)
//
// One request of 131072 positions, 8 heads of 64 rows: 91 us, of them 9 the join (with
// registers dequantising for mma.sync 153; with one scale to 16 rows of queries 89; on the
// way one buffer of P 145, queries brought by one warp 121, one more wait in a step 115).
// HBM would take 22 and the products 15: the issue slots bind it, 65 of 100 taken by 28 warps
// that wait on one another, with 72 registers a thread (160 bytes spilled).
//
// Roles (28 warps, one CTA per SM):
//   first 16         softmax: groups of 4 warps, 16 columns each; thread = position
//   then 8           four keys, four values: codes to tensor memory (warp & 3 = its 32 lanes); the keys' also Q
//   then two         copies of the keys' and of the values' codes and scales
//   one              MMA issuer, one more the segments
#include <cudaTypedefs.h>

#include "attn_rows.cuh"
#include "fp4.cuh"
#include "pdl.cuh"
#include "serve.cuh"
#include "sm100_ptx.cuh"

namespace dspark {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSteps = 128;              // positions per step
constexpr int kDim = 128;                // head size
constexpr int N = 64;                    // query rows of a tile: columns of the products
constexpr int kSegs = 8;                 // segment descriptors in flight
constexpr int kBadRing = 16;             // steps the copies may be ahead of the softmax, and more
constexpr int kQTop = 15;                // queries are scaled to below 2^kQTop
constexpr float kLift = 7.f;             // log2 of a weight at the reference
constexpr float kSlack = 8.f;            // log2 of the growth of a maximum that is let pass
constexpr long long kDrainCycles = 200000000LL;
constexpr int kRow = 64;                 // bytes of a position's codes, chunks of 16 swizzled as TMA's 64-byte mode does
constexpr int kCodes = kSteps * kRow;    // of a stage, then the scales
constexpr int kStageBytes = kCodes + kSteps * (kDim / fp4::kGroup);
constexpr int kStages = 6;               // of keys, and of values
constexpr int kTiles = 4;                // A tiles in tensor memory: keys 0 and 2, values 1 and 3
constexpr int kTileCols = kDim / 2;      // columns of one

struct Roles {
    static constexpr int HC = 16;                 // columns of a softmax group
    static constexpr int kSoftWarps = 4 * (N / HC), kValWarps = 4;
    static constexpr int kKeyWarp = kSoftWarps, kValWarp = kKeyWarp + 4, kCopyWarp = kValWarp + kValWarps;
    static constexpr int kMmaWarp = kCopyWarp + 2, kSegWarp = kCopyWarp + 3, kWarps = kCopyWarp + 4;
};

struct Seg {
    int b, h, q0, n, len;     // request, key-value head, first token in q, tokens, cache length
    int r0, rows;             // query rows of this tile
    int pos0, pos1;           // cache positions [pos0, pos1)
    int steps;                // -1: no more segments
    int slot;                 // -1: the whole segment, else the partial result's slot
};

struct Smem {
    static constexpr int kQBytes = N * kDim * 2, kQBufs = 2;
    static constexpr int kCols = 4 * N + kTiles * kTileCols;      // tensor memory: two S, two O, the A tiles
    static constexpr int kTmem = 512;
    static constexpr int kQ = 0;
    static constexpr int kPBytes = kSteps * 128;
    static constexpr int kP = kQ + kQBufs * kQBytes;              // two of [128][64] fp16, 128-byte rows
    static constexpr int kRing = kP + 2 * kPBytes;                // [keys, values][stage]
    static constexpr int kMax = kRing + 2 * kStages * kStageBytes;    // [2][N][4], by the step's parity
    static constexpr int kSum = kMax + 2 * N * 16;                // [2][N][4], by the segment's parity
    static constexpr int kScale = kSum + 2 * N * 16;              // [kSegs][N] what the scores of a Q tile's rows are multiplied by
    static constexpr int kSeg = kScale + kSegs * N * 4;
    static constexpr int kBar = (kSeg + kSegs * (int)sizeof(Seg) + 7) / 8 * 8;
    static constexpr int kBars = 4 * kStages + 2 * kTiles + 2 * kSegs + 2 * kQBufs + 2 + 2 + 2 + 2 + 2 + 1;
    static constexpr int kFlags = kBar + 8 * kBars;               // TMEM address, abort, NaN flag, -, the limit of waits
    static constexpr int kLater = kFlags + 24;                    // [kStages] first of a step's positions that not every row sees
    static constexpr int kBad = kLater + 4 * kStages;             // [kBadRing] boxes whose page is out of range, and a bit where not every row sees every position
    static constexpr int kThere = kBad + 4 * kBadRing;            // [kStages] boxes of a step's values that were copied, and its positions before the end
    static constexpr int kTotal = kThere + 8 * kStages;
};

__device__ __forceinline__ float warp_max(float x) {     // over the warp, NaN left out
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// Nonzero in one lane of the (converged) warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

// A wait that a test did not end; `flags`: Smem::kFlags.  (Not inlined, and what it reads in
// shared memory: the roles' loops share the SM's instruction cache, and registers are few.)
__device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, uint32_t flags) {
    const uint8_t* at = static_cast<const uint8_t*>(__cvta_shared_to_generic(flags));
    return ptx::mbar_wait_strict(bar, parity, reinterpret_cast<const volatile uint32_t*>(at) + 1, *reinterpret_cast<const volatile long long*>(at + 16));
}

// 16 columns of 32 lanes, waited for.
__device__ __forceinline__ void tmem_get(uint32_t a, float (&v)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 "\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
                   "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(a) : "memory");
}
__device__ __forceinline__ void tmem_put(uint32_t a, const float (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 "\n\ttcgen05.wait::st.sync.aligned;"
                 ::"r"(a), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
                   "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]) : "memory");
}

// (x - r) * s + n, and l + w, of two columns.  (The difference first: of large scores a
// product that is rounded by itself and one that is not would differ by whole units.)
__device__ __forceinline__ void exponent_pair(float& x0, float& x1, float r0, float r1, float s0, float s1, float n) {
    asm("{\n\t.reg .b64 x, r, s, n;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 r, {%2, %3};\n\tmov.b64 s, {%4, %5};\n\tmov.b64 n, {%6, %6};\n\t"
        "sub.rn.f32x2 x, x, r;\n\tfma.rn.f32x2 x, x, s, n;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(x0), "+f"(x1) : "f"(r0), "f"(r1), "f"(s0), "f"(s1), "f"(n));
}
// (volatile: read where it is used, the registers are few)
__device__ __forceinline__ float4 load_four(uint32_t from) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(from));
    return v;
}
__device__ __forceinline__ void add_pair(float& l0, float& l1, float w0, float w1) {
    asm("{\n\t.reg .b64 l, w;\n\tmov.b64 l, {%0, %1};\n\tmov.b64 w, {%2, %3};\n\tadd.rn.f32x2 l, l, w;\n\tmov.b64 {%0, %1}, l;\n\t}"
        : "+f"(l0), "+f"(l1) : "f"(w0), "f"(w1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store_chunk(uint32_t to, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// The box of codes from position `pos` of (page, head) `z`.
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* m, int pos, int z, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(pos), "r"(z), "r"(bar), "l"(policy)
        : "memory");
}
// 16 lanes x 8 columns of tensor memory, as fragments: thread t holds columns t % 4 and
// 4 + t % 4 of lanes t / 4 (v0, v2) and t / 4 + 8 (v1, v3).
__device__ __forceinline__ void tmem_put_16x128b(uint32_t a, uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v0), "r"(v1), "r"(v2), "r"(v3) : "memory");
}
// 32 lanes x 16 columns: thread t holds lane t.
__device__ __forceinline__ void tmem_put_32x32b(uint32_t a, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                   "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]) : "memory");
}
// kind::f16 with both operands fp16 (format 0), A K-major.
constexpr uint32_t idesc_half(int N, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__global__ void __launch_bounds__(Roles::kWarps * 32, 1) attn4_mma_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const int bx, const int page_heads) {
    using L = Smem;
    using R = Roles;
    constexpr int kSoftWarps = R::kSoftWarps, HC = R::HC;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile uint32_t* s_flags = reinterpret_cast<volatile uint32_t*>(gbase + L::kFlags);   // [0] TMEM, [1] abort, [2] NaN
    volatile uint32_t* s_bad = reinterpret_cast<volatile uint32_t*>(gbase + L::kBad);
    volatile float* s_scale = reinterpret_cast<volatile float*>(gbase + L::kScale);
    volatile int* s_later = reinterpret_cast<volatile int*>(gbase + L::kLater);
    volatile int* s_there = reinterpret_cast<volatile int*>(gbase + L::kThere);
    volatile Seg* s_seg = reinterpret_cast<volatile Seg*>(gbase + L::kSeg);
    volatile uint32_t* abort_flag = s_flags + 1;
    uint32_t bar = base + L::kBar;
    auto take = [&](int n) { const uint32_t b = bar; bar += 8u * n; return b; };
    const uint32_t b_cfull = take(2 * kStages), b_cempty = take(2 * kStages);       // codes: keys' stages, then values'
    const uint32_t b_full = take(kTiles), b_empty = take(kTiles);                   // A tiles
    const uint32_t b_seg_full = take(kSegs), b_seg_empty = take(kSegs);
    const uint32_t b_q_full = take(L::kQBufs), b_q_empty = take(L::kQBufs), b_s_full = take(2), b_s_empty = take(2);
    const uint32_t b_o_empty = take(2), b_p_full = take(2), b_pv = take(2), b_end = take(1);

    if (tid == 0) {
        grid_launch_dependents();       // the join is scheduled now and waits for this grid
        for (int i = 0; i < 2 * kStages; ++i) { ptx::mbar_init(b_cfull + 8 * i, 1); ptx::mbar_init(b_cempty + 8 * i, i < kStages ? 4 : R::kValWarps); }
        for (int i = 0; i < kTiles; ++i) { ptx::mbar_init(b_full + 8 * i, i & 1 ? R::kValWarps : 4); ptx::mbar_init(b_empty + 8 * i, 1); }
        for (int i = 0; i < kSegs; ++i) { ptx::mbar_init(b_seg_full + 8 * i, 1); ptx::mbar_init(b_seg_empty + 8 * i, 1 + 2 + 4 + R::kValWarps + kSoftWarps); }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(b_s_full + 8 * i, 1); ptx::mbar_init(b_s_empty + 8 * i, kSoftWarps);
            ptx::mbar_init(b_o_empty + 8 * i, kSoftWarps);
            ptx::mbar_init(b_p_full + 8 * i, kSoftWarps); ptx::mbar_init(b_pv + 8 * i, 1);
        }
        for (int i = 0; i < L::kQBufs; ++i) { ptx::mbar_init(b_q_full + 8 * i, 4); ptx::mbar_init(b_q_empty + 8 * i, 1); }
        ptx::mbar_init(b_end, 1);
        s_flags[1] = 0u;
        s_flags[2] = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == R::kMmaWarp) {
        ptx::tmem_alloc(base + L::kFlags, L::kTmem);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = s_flags[0], tiles = tmem + 4 * N;
    grid_dependency_wait();             // the set-up above overlaps the launch before this one
    // (every warp writes the limit, the same, for its own waits)
    if (lane == 0) *reinterpret_cast<volatile long long*>(gbase + L::kFlags + 16) = wait_limit_of(reinterpret_cast<const unsigned long long*>(p.status) + 1);
    __syncwarp();
    auto wait = [&](uint32_t b, uint32_t parity) { return ptx::mbar_test_wait(b, parity & 1u) || wait_longer(b, parity & 1u, base + L::kFlags); };
    auto wait_all = [&](uint32_t b, uint32_t parity) { return (bool)__all_sync(~0u, wait(b, parity)); };
    auto give_up = [&](int site) {
        raise_timeout(p.status, site);
        *abort_flag = 1u;
    };

    if (warp == R::kSegWarp) {
        // ----------------------------------------------------------- segments
        const AttnSplit sp(p, p.tile_off[p.B], p.tile_off[0]);
        const int cta = blockIdx.x;
        int place = 0, end = 0;
        if (cta < sp.n) { place = sp.first(cta); end = sp.first(cta + 1); }
        AttnSplitRow split{};                    // the segment that begins here and goes on in the next CTA
        bool ok = true;
        for (int si = 0; ok; ++si) {
            Seg d;
            d.steps = -1;
            while (place < end) {
                const AttnSegment g = attn_segment(p, sp, place, attn_first_round(p));
                const RowMap rm(p, g.b, lane == 0);
                d.r0 = g.rt * p.row_tile;
                d.rows = max(0, min(p.row_tile, rm.n * p.G - d.r0));
                const int j0 = g.tile(sp, place), j1 = g.tile(sp, end), next = g.t0 + sp.pad + g.tiles;
                if (next <= place) { place = end; break; }         // (offsets that do not ascend)
                place = next;
                if (j0 == j1 || d.rows == 0 || g.tiles != attn_tiles(rm.len)) continue;
                d.b = g.b; d.h = g.h; d.q0 = rm.q0; d.n = rm.n; d.len = rm.len;
                d.pos0 = j0 * kTile;
                d.pos1 = min(j1 * kTile, rm.len);
                d.steps = (d.pos1 - d.pos0 + kSteps - 1) / kSteps;
                const bool whole = j0 == 0 && j1 == g.tiles;
                d.slot = whole ? -1 : 2 * cta + (j0 == 0 ? 1 : 0);
                if (j0 == 0 && !whole) split = attn_split_row(sp, g, cta, rm.q0, d.r0, d.rows);
                break;
            }
            const int slot = si % kSegs;
            if (si >= kSegs) ok = wait_all(b_seg_empty + 8 * slot, (si / kSegs) - 1);
            if (!ok) { if (lane == 0) give_up(0); break; }
            if (lane == 0) {
                const_cast<Seg&>(s_seg[slot]) = d;
                ptx::mbar_arrive(b_seg_full + 8 * slot);
            }
            __syncwarp();
            if (d.steps < 0) break;
        }
        if (lane == 0) p.split[cta] = split;
    } else if (warp == R::kCopyWarp || warp == R::kCopyWarp + 1) {
        // --------------------------------------------------------------- copies
        // lanes 0 .. : a box of bx positions' codes each; lanes 16 .. : their scales
        const int kv = warp - R::kCopyWarp, mine = lane & 15, nbox = kSteps / bx;
        const CUtensorMap* map = kv ? &vmap : &kmap;
        const uint8_t* scales = kv ? p.vs : p.ks;
        const uint64_t pol = p.row_tiles == 1 ? ptx::policy_evict_first() : ptx::policy_evict_last();
        uint32_t step = 0;
        bool ok = true;
        for (int si = 0; ok; ++si) {
            const int slot = si % kSegs;
            ok = wait_all(b_seg_full + 8 * slot, si / kSegs);
            if (!ok) { if (lane == 0) give_up(2); break; }
            const Seg& sg = const_cast<Seg&>(s_seg[slot]);
            struct { int b, h, pos0, pos1, steps, seen; } d = {sg.b, sg.h, sg.pos0, sg.pos1, sg.steps, sg.len - sg.n + 1};
            __syncwarp();
            if (d.steps < 0) break;
            if (lane == 0) ptx::mbar_arrive(b_seg_empty + 8 * slot);
            const int32_t* row = p.table + (size_t)d.b * p.width;
            auto page_of = [&](int pos) { return mine < nbox && pos < d.pos1 ? __ldg(row + p.by_page(pos)) : -1; };
            int next = page_of(d.pos0 + mine * bx);
            for (int s = 0; s < d.steps; ++s, ++step) {
                const int stage = step % kStages, pos0 = d.pos0 + s * kSteps, pos = pos0 + mine * bx, page = next;
                const bool in = mine < nbox && pos < d.pos1, have = in && page >= 0 && page < p.pages;
                const uint32_t there = __ballot_sync(~0u, have) & 0xffffu, bad = __ballot_sync(~0u, in && !have) & 0xffffu;
                next = page_of(pos + kSteps);
                if (bad && lane == 0) raise_status(p.status, kBadPage);
                if (step >= (uint32_t)kStages) ok = wait_all(b_cempty + 8 * (kv * kStages + stage), step / kStages - 1);
                if (!ok) { if (lane == 0) give_up(3); break; }
                const uint32_t full = b_cfull + 8 * (kv * kStages + stage), to = base + L::kRing + (kv * kStages + stage) * kStageBytes;
                if (lane == 0) {
                    if (!kv) s_bad[step % kBadRing] = bad | (d.seen - pos0 < kSteps || d.pos1 - pos0 < kSteps ? 1u << 16 : 0u);
                    else {
                        s_later[stage] = d.seen - pos0;
                        s_there[2 * stage] = (int)there;
                        s_there[2 * stage + 1] = d.pos1 - pos0;
                    }
                    if (there) ptx::mbar_arrive_expect_tx(full, __popc(there) * bx * (kRow + kDim / fp4::kGroup));
                    else ptx::mbar_arrive(full);
                }
                __syncwarp();
                if (have) {
                    const int r = pos - p.by_page(pos) * p.page_size;
                    if (lane < 16) tma_load_rows(to + mine * bx * kRow, map, r, page * page_heads + d.h, full, pol);
                    else ptx::bulk_load(to + kCodes + mine * bx * (kDim / fp4::kGroup),
                                        scales + page * p.scale_stride + ((long long)d.h * p.page_size + r) * (kDim / fp4::kGroup),
                                        bx * (kDim / fp4::kGroup), full, pol);
                }
                __syncwarp();
            }
        }
        // every copy lands before the CTA leaves: the last fill of each stage
        if (lane == 0)
            for (uint32_t f = step; f-- > 0 && f + kStages >= step;)
                ptx::mbar_wait_drain(b_cfull + 8 * (kv * kStages + f % kStages), (f / kStages) & 1u, kDrainCycles);
        __syncwarp();
    } else if (warp >= R::kKeyWarp && warp < R::kCopyWarp) {
        // ------------------------------------------------ codes to tensor memory
        const int kv = warp >= R::kValWarp, quarter = warp & 3, g = lane >> 2, t = lane & 3;
        uint32_t step = 0;
        bool ok = true;
        for (int si = 0; ok; ++si) {
            const int slot = si % kSegs;
            ok = wait_all(b_seg_full + 8 * slot, si / kSegs);
            if (!ok) { if (lane == 0) give_up(6); break; }
            const Seg& sg = const_cast<Seg&>(s_seg[slot]);
            struct { int h, q0, r0, rows, steps; } d = {sg.h, sg.q0, sg.r0, sg.rows, sg.steps};
            __syncwarp();
            if (d.steps < 0) break;
            if (lane == 0) ptx::mbar_arrive(b_seg_empty + 8 * slot);
            if (!kv) {
                // 16 rows of the Q tile, each scaled by a power of two to below 2^kQTop, those beyond the
                // request's as zeros.  (One warp for the whole tile took 27000 cycles a segment, ahead of the first product)
                const int c = lane & 15, first = 16 * quarter + (lane >> 4);         // a 16-byte chunk of rows first, first + 2, ..
                uint4 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int rr = d.r0 + min(first + 2 * i, d.rows - 1), tok = p.by_group(rr);
                    x[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + (d.q0 + tok) * p.q_stride +
                                                                (size_t)(d.h * p.G + rr - tok * p.G) * kDim) + c);
                }
                const int qb = si % L::kQBufs;
                if (si >= L::kQBufs) ok = wait_all(b_q_empty + 8 * qb, si / L::kQBufs - 1);
                if (!ok) { if (lane == 0) give_up(1); break; }
                const uint32_t to = base + L::kQ + qb * L::kQBytes + (c / 8) * (N * 128);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = first + 2 * i;
                    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    // (magnitudes are ordered as integers; the 16 lanes of a row)
                    uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
                    top = max(top << 16, top & 0xffff0000u);
#pragma unroll
                    for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
                    const int e = min(max((int)(top >> 23) - 126 - kQTop, -126), 126);
                    const float by = r < d.rows ? __int_as_float((127 - e) << 23) : 0.f;
                    uint32_t y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = pack_half(__uint_as_float(w[j] << 16) * by, __uint_as_float(w[j] & 0xffff0000u) * by);
                    store_chunk(to + r * 128 + (((c & 7) ^ (r & 7)) << 4), y[0], y[1], y[2], y[3]);
                    // (neither 0 nor inf, which -inf and 0 would make NaN)
                    if (c == 0) s_scale[N * slot + r] = fminf(fmaxf(p.scale * kLog2e * __int_as_float((127 + e) << 23), 1e-37f), 3e38f);
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(b_q_full + 8 * qb);
            }
            for (int s = 0; s < d.steps; ++s, ++step) {
                const int stage = step % kStages;
                const uint32_t fill = 2 * step + kv, tile = fill % kTiles, at = tiles + tile * kTileCols + ((uint32_t)quarter << 21);
                ok = wait_all(b_cfull + 8 * (kv * kStages + stage), step / kStages);
                if (fill >= (uint32_t)kTiles) ok = wait_all(b_empty + 8 * tile, fill / kTiles - 1) && ok;
                if (!ok) { if (lane == 0) give_up(7); break; }
                ptx::tc_fence_after();
                const uint8_t* st = gbase + L::kRing + (kv * kStages + stage) * kStageBytes;
                // (loops that stay small: twenty warps of six roles share an SM's instruction cache)
                if (!kv) {
                    // position 32 * quarter + lane: its entries in order
                    const uint4* mine = reinterpret_cast<const uint4*>(st + (32 * quarter + lane) * kRow);
                    const uint8_t* sc = st + kCodes + (32 * quarter + lane) * 8;
                    const int turn = lane >> 1 & 3;          // of the chunks
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        const uint4 w = mine[i ^ turn];
                        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
                        const uint32_t both = fp4::scale_pair(reinterpret_cast<const uint16_t*>(sc)[i]);
                        const uint32_t by[2] = {__byte_perm(both, both, 0x1010), __byte_perm(both, both, 0x3232)};
                        uint32_t v[16];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t h[4];
                            fp4::unpack(words[j], h);
#pragma unroll
                            for (int x = 0; x < 4; ++x) v[4 * j + x] = fp4::mul2(h[x], by[j / 2]);
                        }
                        tmem_put_32x32b(at + 16 * i, v);
                    }
                } else {
                    // entries 32 * quarter + 4 g .. + 3 of positions t, t + 4, t + 8, t + 12 of each 16
                    constexpr int kMine = kSteps / 16;                   // sixteens
                    // (rows t and t + 8 swap their chunks alike, t + 4 and t + 12 the other way)
                    const uint8_t* mine = st + t * kRow + 2 * g;
                    const int even_at = 16 * (quarter ^ (t >> 1)), odd_at = 16 * (quarter ^ (t >> 1) ^ 2);
                    const uint8_t* sc = st + kCodes + t * 8 + 2 * quarter + (g >> 2);
                    const int later = s_later[stage], there = s_there[2 * stage], stop = s_there[2 * stage + 1];
                    const bool edge = later < kSteps || stop < kSteps || there != (1 << kSteps / bx) - 1;
#pragma unroll 2
                    for (int k = 0; k < kMine; ++k, mine += 16 * kRow, sc += 16 * 8) {
                        uint32_t v[4], b[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            v[i] = *reinterpret_cast<const uint16_t*>(mine + 4 * i * kRow + (i & 1 ? odd_at : even_at));
                            b[i] = sc[4 * i * 8];
                        }
                        if (edge) {
                            // what no row may use counts as 0, and a NaN among the values of later tokens of the
                            // block, which must not reach the rows that do not see it (0 * NaN), is left out
                            // here and added at the segment's end
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int r = t + 16 * k + 4 * i;
                                if (r >= stop || !(there >> r / bx & 1)) b[i] = 0u;
                                else if (r >= later && (b[i] & 0x7fu) == 0x7fu) { b[i] = 0u; s_flags[2] = 1u; }
                            }
                        }
                        // positions t, t + 4 in the lower half of a word, t + 8, t + 12 in the upper
                        const uint32_t a = __byte_perm(v[0], v[2], 0x5410), c = __byte_perm(v[1], v[3], 0x5410);
                        const uint32_t s0 = fp4::scale_pair(b[0] | b[1] << 8), s1 = fp4::scale_pair(b[2] | b[3] << 8);
                        uint32_t even[4], odd[4];            // [entry / 2 + 2 * half of the 16 positions]
                        fp4::unpack((a & 0x0f0f0f0fu) | (c << 4 & 0xf0f0f0f0u), even);
                        fp4::unpack((a >> 4 & 0x0f0f0f0fu) | (c & 0xf0f0f0f0u), odd);
                        const uint32_t to = at + 8 * k;
                        tmem_put_16x128b(to, fp4::mul2(even[0], s0), fp4::mul2(odd[0], s0), fp4::mul2(even[2], s1), fp4::mul2(odd[2], s1));
                        tmem_put_16x128b(to + (16u << 16), fp4::mul2(even[1], s0), fp4::mul2(odd[1], s0), fp4::mul2(even[3], s1), fp4::mul2(odd[3], s1));
                    }
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(b_cempty + 8 * (kv * kStages + stage));
                    ptx::mbar_arrive(b_full + 8 * tile);
                }
            }
        }
    } else if (warp == R::kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        // the whole warp runs the loop, so that descriptors are uniform values;
        // one elected lane issues
        constexpr uint32_t id_s = idesc_half(N, false), id_o = idesc_half(N, true);
        const uint32_t one = elect_one();
        const uint64_t q_desc = ptx::smem_desc_sw128(base + L::kQ, 16, 1024);
        const uint64_t p_desc = ptx::smem_desc_sw128(base + L::kP, 16, 1024);
        // S of a step, then O of the step before
        uint32_t step = 0, o_seg = 0;
        bool ok = true, o_first = true;
        auto product_o = [&](uint32_t of) {      // O^T (+)= V^T P^T of step `of`, of segment o_seg
            const uint32_t vi = 2 * of + 1, ob = o_seg & 1u;
            ok = wait_all(b_full + 8 * (vi % kTiles), vi / kTiles) && ok;
            if (o_first && o_seg >= 2) ok = wait_all(b_o_empty + 8 * ob, o_seg / 2 - 1) && ok;
            ok = wait_all(b_p_full + 8 * (of & 1u), of / 2) && ok;
            if (!ok) return;
            ptx::tc_fence_after();
            if (one) {
#pragma unroll
                for (int k = 0; k < kSteps / 16; ++k)
                    ptx::mma_f16_ts(tmem + (2 + ob) * N, tiles + vi % kTiles * kTileCols + 8 * k, p_desc + (of & 1u) * (L::kPBytes / 16) + k * (2048 / 16),
                                    id_o, o_first && k == 0 ? 0u : 1u);
                ptx::mma_commit(b_empty + 8 * (vi % kTiles));
                ptx::mma_commit(b_pv + 8 * (of & 1u));
            }
            __syncwarp();
            o_first = false;
        };
        for (uint32_t si = 0; ok; ++si) {
            ok = wait_all(b_seg_full + 8 * (si % kSegs), si / kSegs);
            if (!ok) break;
            const int steps = s_seg[si % kSegs].steps;
            __syncwarp();
            if (steps < 0) break;
            if (lane == 0) ptx::mbar_arrive(b_seg_empty + 8 * (si % kSegs));
            const uint32_t qb = si % L::kQBufs;
            ok = wait_all(b_q_full + 8 * qb, si / L::kQBufs);
            for (int s = 0; s < steps && ok; ++s, ++step) {
                const uint32_t ki = 2 * step, sb = step & 1u;
                ok = wait_all(b_full + 8 * (ki % kTiles), ki / kTiles) && ok;
                if (step >= 2) ok = wait_all(b_s_empty + 8 * sb, step / 2 - 1) && ok;
                if (!ok) break;
                ptx::tc_fence_after();
                if (one) {
                    const uint64_t qa = q_desc + qb * (L::kQBytes / 16);
#pragma unroll
                    for (int k = 0; k < kDim / 16; ++k)
                        ptx::mma_f16_ts(tmem + sb * N, tiles + ki % kTiles * kTileCols + 8 * k, qa + (k / 4) * (N * 128 / 16) + (k % 4) * 2, id_s, k ? 1u : 0u);
                    ptx::mma_commit(b_empty + 8 * (ki % kTiles));
                    ptx::mma_commit(b_s_full + 8 * sb);
                    if (s == steps - 1) ptx::mma_commit(b_q_empty + 8 * qb);
                }
                __syncwarp();
                if (step > 0) product_o(step - 1);
                if (s == 0) { o_seg = si; o_first = true; }
            }
        }
        if (ok && step > 0) product_o(step - 1);
        if (!ok && lane == 0) give_up(4);
        // nothing is in flight in the tensor core when the CTA leaves
        if (one) ptx::mma_commit(b_end);
        __syncwarp();
        ptx::mbar_wait_drain(b_end, 0, kDrainCycles);
        __syncwarp();
    } else {
        // ------------------------------------------------------------- softmax
        const int group = warp >> 2, quarter = warp & 3, row = tid & 127;
        const uint32_t lanes = (uint32_t)quarter << 21;             // TMEM lane offset of this warp
        float4* s_max = reinterpret_cast<float4*>(gbase + L::kMax);
        float4* s_sum = reinterpret_cast<float4*>(gbase + L::kSum);
        // the product's step that this position is: of 16, r is (r & 8) + 2 (r & 3) + (r >> 2 & 1)
        const int prow = (row & ~7) | (row & 3) << 1 | (row >> 2 & 1);
        // the entry of the head that this lane of O^T holds
        const int dim = (row & ~31) | (row & 7) << 2 | (row >> 4 & 1) << 1 | (row >> 3 & 1);
        uint32_t step = 0;
        bool ok = true;
        // A segment's rows are written after the first step of the next segment
        // (its O^T is in the other half of tensor memory), so the tensor core
        // and the producers go on meanwhile.  What is kept of it until then:
        bool pend = false;
        float pend_ref = 0.f;                                      // lane c: column c's reference, in units of log2
        for (uint32_t si = 0;; ++si) {
            const int slot = si % kSegs;
            ok = wait(b_seg_full + 8 * slot, si / kSegs) && ok;
            if (ptx::bar_red_or(1 + group, 128, !ok)) { ok = false; break; }
            const Seg& sg = const_cast<Seg&>(s_seg[slot]);
            const int steps = sg.steps;
            const bool none = steps < 0;                           // no more segments
            if (none && !pend) break;
            // no row of the tile in this group's columns: what the products make of them is not read
            const bool idle = !none && group * HC >= sg.rows;
            const uint32_t o_at = tmem + lanes + (2 + (si & 1u)) * N + group * HC;
            float ref[HC], l[HC];                                  // the references (of scores before the scale), this thread's sum of the weights
            const uint32_t scales = base + L::kScale + 4 * (N * slot + group * HC);      // (a segment's first scores follow its Q tile)
#pragma unroll
            for (int c = 0; c < HC; ++c) ref[c] = l[c] = 0.f;
            float my_ref = -INFINITY;                              // lane c: column c's reference, -inf before the first score
            bool unset = true;                                     // a column of the group has no reference yet
            bool stop = false;
            for (int s = 0; s < steps || s == 0; ++s) {
                if (idle) {
                    ok = wait(b_s_full + 8 * (step & 1u), step / 2) && ok;
                    ok = __all_sync(~0u, ok);
                    if (lane == 0) {
                        if (!ok) give_up(5);                       // (the group leaves where it meets next)
                        ptx::mbar_arrive(b_s_empty + 8 * (step & 1u));
                        ptx::mbar_arrive(b_p_full + 8 * (step & 1u));
                    }
                    __syncwarp();
                    ++step;
                } else if (!none) {
                ok = wait(b_s_full + 8 * (step & 1u), step / 2) && ok;
                ok = __all_sync(~0u, ok);
                const uint32_t s_at = tmem + lanes + (step & 1u) * N + group * HC;
                const uint32_t marks = ok ? s_bad[step % kBadRing] : 0u;
                float x[HC];
                // the scores, -inf where the column does not see the position (read
                // again where a reference moves)
                auto scores = [&]() {
                    if (ok) tmem_get(s_at, x);
                    else {
#pragma unroll
                        for (int c = 0; c < HC; ++c) x[c] = 0.f;
                    }
                    if (marks) {
                        // positions beyond the end or in a bad page, and the block's later tokens
                        const int pos = sg.pos0 + s * kSteps + row;
                        const bool gone = pos >= sg.pos1 || (marks >> (row / bx) & 1u);
                        // lane c: the last position that column c of this group sees
                        const int my_last = sg.len - sg.n + p.by_group(sg.r0 + group * HC + (lane & (HC - 1)));
#pragma unroll
                        for (int c = 0; c < HC; ++c) {
                            const int last = __shfl_sync(~0u, my_last, c);
                            if (gone || pos > last) x[c] = -INFINITY;
                        }
                    }
                };
                // .. as exponents
                auto exponents = [&]() {
#pragma unroll
                    for (int c = 0; c < HC; c += 4) {
                        const float4 by = load_four(scales + 4 * c);
                        exponent_pair(x[c], x[c + 1], ref[c], ref[c + 1], by.x, by.y, kLift);
                        exponent_pair(x[c + 2], x[c + 3], ref[c + 2], ref[c + 3], by.z, by.w, kLift);
                    }
                };
                ptx::tc_fence_after();
                float high = -INFINITY;
                if (!unset) {
                    scores();
                    exponents();
#pragma unroll
                    for (int c = 0; c < HC; ++c) high = fmaxf(high, x[c]);
                }
                // (unset is the same in the whole group)
                const bool move = unset || ptx::bar_red_or(1 + group, 128, high > kLift + kSlack || !ok);
                // (O of the step before the last is done, and its P may be overwritten: that product was issued
                // before this step's S, by the same thread, and what a commit signals is all that was issued before it)
                if (move) {                     // the same in every thread of the group
                    // the last one too: O may be rescaled
                    if (step > 0) ok = wait(b_pv + 8 * ((step - 1) & 1u), (step - 1) / 2) && ok;
                    float mine = -INFINITY;
                    scores();
#pragma unroll
                    for (int c = 0; c < HC; ++c) {
                        const float w = warp_max(x[c]);
                        if (lane == c) mine = w;
                    }
                    float* mx = reinterpret_cast<float*>(s_max + (step & 1u) * N + group * HC);
                    if (lane < HC) mx[lane * 4 + quarter] = mine;
                    if (ptx::bar_red_or(1 + group, 128, !ok)) { stop = true; break; }
                    const float4 w4 = reinterpret_cast<const float4*>(mx)[lane & (HC - 1)];
                    const float top = fmaxf(fmaxf(w4.x, w4.y), fmaxf(w4.z, w4.w));
                    const float to = fmaxf(my_ref, top);
                    const float my_a = to > my_ref ? fast_exp2((my_ref - to) * s_scale[N * slot + group * HC + (lane & (HC - 1))]) : 1.f;
                    my_ref = to;
                    unset = __any_sync(~0u, to == -INFINITY);
                    if (s > 0) ptx::tc_fence_after();
                    float a[HC];
#pragma unroll
                    for (int c = 0; c < HC; ++c) {
                        a[c] = __shfl_sync(~0u, my_a, c);
                        const float r = __shfl_sync(~0u, to, c);
                        ref[c] = r == -INFINITY ? 0.f : r;
                        l[c] *= a[c];
                    }
                    if (s > 0) {
                        float o[HC];
                        tmem_get(o_at, o);
#pragma unroll
                        for (int c = 0; c < HC; ++c) o[c] *= a[c];
                        tmem_put(o_at, o);
                    }
                    exponents();
                }
                ptx::tc_fence_before();          // the scores were read
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(b_s_empty + 8 * (step & 1u));
                // weights: row `prow` of P, columns group * HC ..
                const uint32_t at = base + L::kP + (step & 1u) * L::kPBytes + prow * 128;
#pragma unroll
                for (int c0 = 0; c0 < HC; c0 += 8) {
                    float w[8];
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        w[e] = fast_exp2(x[c0 + e]);
                        w[e + 1] = fast_exp2(x[c0 + e + 1]);
                        add_pair(l[c0 + e], l[c0 + e + 1], w[e], w[e + 1]);
                    }
                    store_chunk(at + ((((group * HC + c0) / 8) ^ (prow & 7)) << 4), pack_half(w[0], w[1]), pack_half(w[2], w[3]),
                                pack_half(w[4], w[5]), pack_half(w[6], w[7]));
                }
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(b_p_full + 8 * (step & 1u));
                ++step;
                }
                if (s > 0 || !pend) continue;
                // ------------------------------- the rows of the segment before
                pend = false;
                {
                    const uint32_t its = step - (none ? 1u : 2u);          // its last step
                    ok = wait(b_pv + 8 * (its & 1u), its / 2) && ok;
                }
                ok = __all_sync(~0u, ok);
                const uint32_t pi = si - 1;
                const Seg& e = const_cast<Seg&>(s_seg[pi % kSegs]);
                const int e_row = group * HC + (lane & (HC - 1)), e_tok = p.by_group(e.r0 + e_row);
                const int e_at = (e.q0 + e_tok) * p.Hq + e.h * p.G + (e.r0 + e_row - e_tok * p.G);   // below N * Hq < 2^31
                const int cols = min(HC, e.rows - group * HC);
                const int part_slot = e.slot, e_new = e.len - e.n;
                // (written before the barrier that began this segment)
                const float4 s4 = s_sum[(pi & 1u) * N + e_row];
                const float pend_sum = (s4.x + s4.y) + (s4.z + s4.w), e_inv = pend_sum != 0.f ? 1.f / pend_sum : 0.f;
                ptx::tc_fence_after();
                float o[HC];
                if (ok && cols > 0) tmem_get(tmem + lanes + (2 + (pi & 1u)) * N + group * HC, o);
                else {
#pragma unroll
                    for (int c = 0; c < HC; ++c) o[c] = 0.f;
                }
                if (s_flags[2] && cols > 0) {
                    // the NaN of the block's later tokens (this CTA's positions)
                    for (int pos = max(e_new + 1, e.pos0); pos < e.pos1; ++pos) {
                        const int pg = p.by_page(pos), page = p.table[(size_t)e.b * p.width + pg];
                        if (page < 0 || page >= p.pages) continue;
                        const uint32_t by = p.vs[page * p.scale_stride + ((long long)e.h * p.page_size + (pos - pg * p.page_size)) * (kDim / fp4::kGroup) + dim / fp4::kGroup];
#pragma unroll
                        for (int c = 0; c < HC; ++c) {
                            const int last = e_new + __shfl_sync(~0u, e_tok, c);
                            if ((by & 0x7fu) == 0x7fu && pos <= last) o[c] = NAN;
                        }
                    }
                }
                if (part_slot < 0) {
                    uint16_t* out = static_cast<uint16_t*>(p.out) + dim;
#pragma unroll
                    for (int c = 0; c < HC; ++c) {
                        const float inv = __shfl_sync(~0u, e_inv, c) * p.out_by;
                        const int to = __shfl_sync(~0u, e_at, c);
                        if (c < cols) out[(size_t)to * kDim] = (uint16_t)pack_bf16(o[c] * inv, 0.f);
                    }
                } else {
                    float* part = p.part + ((size_t)part_slot * p.row_tile + group * HC) * kDim + dim;
#pragma unroll
                    for (int c = 0; c < HC; ++c)
                        if (c < cols) part[c * kDim] = o[c] * p.out_by;
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(b_o_empty + 8 * (pi & 1u));
                if (quarter == 0 && lane < cols) {
                    if (part_slot >= 0) {
                        float2* stats = reinterpret_cast<float2*>(part_stats(p));
                        stats[(size_t)part_slot * p.row_tile + e_row] = make_float2(pend_ref - kLift, pend_sum);
                    } else if (p.lse) p.lse[e_at] = pend_sum != 0.f ? (pend_ref - kLift) * kLn2 + logf(pend_sum) : -INFINITY;
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(b_seg_empty + 8 * (pi % kSegs));
            }
            if (stop) { ok = false; break; }
            if (none) break;
            // column sums: after the exchanges of 16, 8, .. lanes lane c holds
            // column c % HC of this warp's positions, then the 4 warps' are added
            float* sm = reinterpret_cast<float*>(s_sum + (si & 1u) * N + group * HC);
            {
#pragma unroll
                for (int w = HC / 2; w; w >>= 1) {
                    const bool up = lane & w;
#pragma unroll
                    for (int c = 0; c < HC / 2; ++c)
                        if (c < w) {
                            const float give = up ? l[c] : l[c + w], keep = up ? l[c + w] : l[c];
                            l[c] = keep + __shfl_xor_sync(~0u, give, w);
                        }
                }
#pragma unroll
                for (int w = HC; w < 32; w <<= 1) l[0] += __shfl_xor_sync(~0u, l[0], w);
            }
            if (lane < HC) sm[lane * 4 + quarter] = l[0];
            pend = true;
            pend_ref = my_ref * s_scale[N * slot + group * HC + (lane & (HC - 1))];
        }
        if (!ok && lane == 0) give_up(5);
    }
    // requests that own no cache position have no tile: their rows are zero
    if (warp < kSoftWarps) empty_rows<uint16_t>(p, blockIdx.x, gridDim.x, kSoftWarps * 32);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == R::kMmaWarp) ptx::tmem_dealloc(tmem, L::kTmem);
}

}  // namespace

bool attn4_tensor(const AttnParams& p, int rows) {
    // pages a whole number of heads apart, all of them within a tensor map's last dimension, scales that bulk copies reach
    const long long per_head = (long long)p.page_size * kRow;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.ks) | reinterpret_cast<uintptr_t>(p.vs) | (uintptr_t)p.scale_stride;
    return attn4_tensor_rows(rows, p.D, p.B * p.Hkv <= num_sms()) && p.page_size % 8 == 0 && p.page_stride % per_head == 0 && p.page_stride / per_head < (1LL << 31) &&
           p.pages * (p.page_stride / per_head) < (1LL << 31) && at % 16 == 0 && tma_encoder() != nullptr;
}

cudaError_t launch_attn4_tensor(const AttnParams& p, cudaStream_t s) {
    using L = Smem;
    static_assert(L::kTotal + 1024 <= 232448 && L::kCols <= 512, "shared and tensor memory of a CTA");
    int bx = kTile;                              // positions of a box: a power of two that divides a page and a tile, where steps begin
    while (p.page_size % bx) bx >>= 1;
    const long long per_head = (long long)p.page_size * kRow;
    const int page_heads = (int)(p.page_stride / per_head);
    CUtensorMap maps[2];
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tma_encoder());
    const cuuint64_t dims[3] = {kRow, (cuuint64_t)p.page_size, (cuuint64_t)(p.pages - 1) * page_heads + p.Hkv};
    const cuuint64_t strides[2] = {kRow, (cuuint64_t)per_head};
    const cuuint32_t box[3] = {kRow, (cuuint32_t)bx, 1}, es[3] = {1, 1, 1};
    for (int i = 0; i < 2; ++i)
        if (enc(&maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(i ? p.v : p.k), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(attn4_mma_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal + 1024);
    if (e != cudaSuccess) return e;
    return launch_dependent(attn4_mma_kernel, dim3(p.ctas), dim3(Roles::kWarps * 32), L::kTotal + 1024, s, p, maps[0], maps[1], bx, page_heads);
}

}  // namespace dspark
