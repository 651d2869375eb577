// cache_attention_mma.cu -- attention over the paged cache on the tensor
// cores: bf16 (fp32 runs on CUDA cores, cache_attention.cu, where the formulas
// stand).
//
// Both products are taken transposed, so that 128 cache positions fill the
// 128 lanes of the accumulator and the few query rows of a key-value head are
// its columns (N = 16, 32, 64 or 128 of them):
//     S^T [128 positions x N] = K [128 x D] . Q^T       (K, Q: K-major)
//     O^T [D x N]            += V^T [D x 128] . P^T      (V, P: MN-major)
// K and V tiles go from the pages to shared memory by TMA exactly as they lie
// there, each is read once by the tensor core whatever N is, and no lane is
// spent on padding rows.  What is left per position and row is one 2^x.
//
// Head sizes: a row of a tile has D = 64, 128 or 256 entries.  Sizes below 128
// other than 64 come in two boxes of 64 entries, what lies beyond the head
// read as zeros; sizes above 128 in two stages of 128 entries, whose products
// go to the same S^T and to two O^T.  Pages that are no boxes (not a multiple
// of 8 positions, not a whole number of heads apart, or heads above 128 that
// are no multiple of 64) are copied row by row, by cp.async of four warps.
// 64 requests of 32 rows, and on CUDA cores before: head size 96 154 us (1900),
// 192 284 (3230), 256 350 (3460); 128 in pages of 1 position 206 (1869).
//
// Roles (12 or 20 warps, 2 more row by row, one CTA per SM, a ring of 5 stages of 32 KB, 4 with 64 or 128 columns):
//   first 8 or 16    softmax, 2 or 4 groups of 4 warps, each with its share of the
//                    columns: thread = position; weights to shared memory
//   then two         producers of the keys and of the values (lane = box of a page:
//                    a multiple of 8 positions, up to 64); four, row by row
//   one              MMA issuer: whichever of the two products is ready
//   one              walks the CTA's segments: descriptors and Q tiles
// The reference of a column's weights, 2^(s - ref), moves only when a score
// exceeds it by more than 8 (weights stay below 2^8, their relative precision
// is the same).  So an ordinary step needs no maximum: each thread forms the
// exponents it needs anyway, a barrier ORs "one of mine is above 8" over the
// group, and only then are the column maxima found (a warp reduction and an
// exchange over the 4 warps), and the sums and O^T in tensor memory rescaled.
//
// What bounds it: HBM.  A key-value head's position is 512 bytes (head size
// 128) and 4 N multiply-adds per byte pair; at 6.8 TB/s an SM has 2800 cycles
// for a step of 128 positions, of which the tensor core is busy 1024 (it reads
// the 128 x 16 operand at 64 bytes a cycle, whatever N is up to 64; with 64
// columns 1536) and a softmax warp 600-1600 (with weights of one part).  So the
// work is to keep copies in flight: two producer warps (one issued a tile in
// 1200 cycles with pages of 16 positions, too slow),
// segment ends off the way (the rows are written behind the next segment's
// first step), the split over CTAs weighted by segments (AttnSplit).
// Measured on one GB300 (another card reads up to 5 % more): 64 requests of
// 1024-8192 positions, 1.22 GB: 32 rows 182 us (6.7 TB/s), 64 rows 195, 128 rows
// 237 (32 columns a thread: the softmax bounds it); 256 requests of 128-4096, 8
// rows, 2.22 GB: 318 us (7.0 TB/s); one of 131072, 64 rows, 0.54 GB: 90 us (6.0
// TB/s, 6 us of it before the ring is full and the join); 256 of 16-300
// positions, 32 rows: 68 us (43 % of the rate: a segment takes the softmax 9000
// cycles, of which its beginning and end are half).
// Steps on the way, with weights of one part, the first of these cases: column
// maxima in every step 263 us, one producer warp and serial segment ends 203,
// MMAs issued from a diverged lane 203, an unweighted split 197, products in
// fixed order 188, a barrier more in a segment's first step and at its end 184
// (64 rows 197), then 182 (190).  Exponents formed twice and column by column:
// head size 256 with 64 rows 418 us, 384 in pairs and kept.  A second buffer for
// P gained nothing (64 rows 202, short ones 74).
//
// Weights go into the second product as two bf16 parts, the leading 8 bits and
// the rest (what is left is 2^-15 of a weight): with one part, rounded, the
// outputs' error against 64 bits is 2.3e-3 of their norm, with two 1.7e-3, the
// rounding of the outputs themselves.  Up to 32 columns the parts are columns of
// one product, whose time does not grow with them, and the halves of O^T are
// added at a segment's end; of 64 columns the second part is a product of its
// own.  One part / two, us: 64 requests of 32 rows 182.1 / 183.1 (the second part
// as its own product 184.6), of 64 rows 190 / 196, 131072 positions of 64 rows
// 88.6 / 90.4, 256 requests of 8 rows 322.4 / 323.2, head size 64 with 32 rows 107
// / 114, with 64 148 / 185.  128 columns keep one part, rounded to nearest: 237
// us for 64 requests, where two take 318 with the second one in the stage of the
// keys, the only place left (64 columns 201 so, head size 64 167), and 390 as
// two tiles of 64 columns, which read the cache twice.  So more than 64 rows of a
// key head have the larger error.  The sum l is taken in fp32 of the whole weights.
#include <cudaTypedefs.h>

#include "pdl.cuh"
#include "serve.cuh"
#include "sm100_ptx.cuh"

namespace dspark {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSteps = 128;              // positions per step (one tile of K and one of V)
// How a tile comes to shared memory: a box of a page with whole rows; two boxes
// of 64 entries, where the head does not fill the row; row by row, where pages
// are no boxes.
enum class Copy { kBoxes, kHalves, kRows };

// The columns are shared by kParts groups of 4 softmax warps: 8, 16 or (of 128
// columns) 32 a thread.  64 columns over two groups, 32 a thread in registers,
// took 209 us for 64 requests of 64 rows, over four 195; 32 columns over four 70
// us for 256 requests of 16-300 positions, over two 82, and the same for long
// ones (head size 64: two, 111 us against 114).
template <int N, int D, Copy kCopy>
struct Roles {
    static constexpr int kParts = N >= 64 || (N == 32 && D == 128) ? 4 : 2, kSoftWarps = 4 * kParts;
    static constexpr int kKeyWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1, kSegWarp = kSoftWarps + 2, kValWarp = kSoftWarps + 3;
    // row by row two warps copy keys and two values, half of a tile's positions each
    // (one of each: 64 requests of 32 rows in pages of 1 position 239 us, 8 rows 207)
    static constexpr int kWarps = kSoftWarps + (kCopy == Copy::kRows ? 6 : 4), kProducers = kWarps - kSoftWarps - 2;
};
constexpr int kSegs = 8;                 // segment descriptors in flight
constexpr int kBadRing = 8;              // steps the producer may be ahead of the softmax, and more
constexpr float kSlack = 8.f;            // log2 of the growth of a maximum that is let pass
constexpr long long kDrainCycles = 200000000LL;

struct Seg {
    int b, h, q0, n, len;     // request, key-value head, first token in q, tokens, cache length
    int r0, rows;             // query rows of this tile
    int pos0, pos1;           // cache positions [pos0, pos1)
    int steps;                // -1: no more segments
    int slot;                 // -1: the whole segment, else the partial result's slot
    int page[16];             // the pages of the first step's boxes
};

// The weights' parts in P: one, two side by side, or two blocks (and products).
enum class Weights { kOne, kBeside, kBlocks };

// D: entries of a tile's row, the head size p.D rounded up to 64, 128 or 256.
template <int N, int D, Copy kCopy>
struct Smem {
    static constexpr int kUnits = D == 256 ? 2 : 1;               // a tile in parts of 128 entries, each a stage
    static constexpr int kUnit = D / kUnits;                      // entries of a part
    static constexpr int kTileBytes = kSteps * kUnit * 2;         // a stage
    // a stage is [8 positions][64-entry half][position][64] as one box brings it,
    // or [half][position][64] where the halves come apart
    static constexpr int kGroup = kCopy == Copy::kHalves ? 1024 : 8 * kUnit * 2;  // from 8 positions to the next 8
    static constexpr int kHalf = kCopy == Copy::kHalves ? kSteps * 128 : kUnit == 128 ? 1024 : 0;
    static constexpr Weights kWeights = N <= 32 ? Weights::kBeside : N == 64 ? Weights::kBlocks : Weights::kOne;
    static constexpr int kStages = (N == 128 || (N == 64 && D >= 128) ? 4 : 5) * 128 / kUnit;
    static constexpr int kQBytes = N * D * 2;
    // Q tiles: segments may be a step long
    static constexpr int kQBufs = N <= 32 && N * D <= 32 * 128 ? 4 : N == 128 || N * D == 64 * 256 ? 1 : 2;
    static constexpr int kO = kWeights == Weights::kBeside ? 2 * N : N;      // columns of an O^T
    static constexpr int kCols = 2 * N + 2 * kUnits * kO;         // tensor memory: two S, two O of kUnits parts
    static constexpr int kTmem = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static constexpr int kRing = 0;
    static constexpr int kQ = kRing + kStages * kTileBytes;
    static constexpr int kP = kQ + kQBufs * kQBytes;                   // [128][64] bf16, 128-byte rows (columns 64 .., or the second part: another)
    static constexpr int kPBytes = kSteps * 128 * (N >= 64 ? 2 : 1);
    static constexpr int kMax = kP + kPBytes;                     // [2][N][4], by the step's parity
    static constexpr int kSum = kMax + 2 * N * 16;                    // [2][N][4], by the segment's parity
    static constexpr int kNeg = kSum + 2 * N * 16;                    // [N], where 32 columns a thread leave no registers for it
    static constexpr int kSeg = kNeg + (N == 128 ? N * 4 : 0);
    static constexpr int kBar = kSeg + kSegs * (int)sizeof(Seg);
    static constexpr int kBars = 2 * kStages + 2 * kSegs + 2 * kQBufs + 2 + 2 + 2 + 3;
    static constexpr int kFlags = kBar + 8 * kBars;               // TMEM address, abort, non-finite flag, -, the producers' counts, bad boxes
    static constexpr int kTotal = kFlags + 24 + 16 * kBadRing;
};

// The box at half `h` and group `g` of 8 positions of (page, head) `z`.
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* m, int h, int g, int z, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %2, %3, %4, %5}], [%6], %7;"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(h), "r"(g), "r"(z), "r"(bar), "l"(policy)
        : "memory");
}

// The box from entry `x` of position `pos` of (page, head) `z`; entries beyond the head are zeros.
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* m, int x, int pos, int z, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(pos), "r"(z), "r"(bar), "l"(policy)
        : "memory");
}

__device__ __forceinline__ float warp_max(float x) {     // over the warp, NaN left out
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// Arrive on an mbarrier once this thread's cp.async so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Nonzero in one lane of the (converged) warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

// N columns of 32 lanes, waited for.
template <int C> __device__ __forceinline__ void tmem_get(uint32_t a, float (&v)[C]);
template <> __device__ __forceinline__ void tmem_get<8>(uint32_t a, float (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(a) : "memory");
}
template <> __device__ __forceinline__ void tmem_get<16>(uint32_t a, float (&v)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 "\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
                   "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(a) : "memory");
}
template <int C> __device__ __forceinline__ void tmem_put(uint32_t a, const float (&v)[C]);
template <> __device__ __forceinline__ void tmem_put<8>(uint32_t a, const float (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\ttcgen05.wait::st.sync.aligned;"
                 ::"r"(a), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]) : "memory");
}
template <> __device__ __forceinline__ void tmem_put<16>(uint32_t a, const float (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 "\n\ttcgen05.wait::st.sync.aligned;"
                 ::"r"(a), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
                   "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]) : "memory");
}

// x * s + n, and l + w, of two columns in one instruction each.
__device__ __forceinline__ void fma_pair(float& x0, float& x1, float s, float n0, float n1) {
    asm("{\n\t.reg .b64 x, s, n;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 s, {%2, %2};\n\tmov.b64 n, {%3, %4};\n\t"
        "fma.rn.f32x2 x, x, s, n;\n\tmov.b64 {%0, %1}, x;\n\t}" : "+f"(x0), "+f"(x1) : "f"(s), "f"(n0), "f"(n1));
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

// Weights x, y >= 0 as a leading part, cut off, and the rest.  The rest is made of
// (1 + 2^-20) times the weight, so that it is above zero wherever the weight is:
// an infinite value then gives the same infinity with both parts.
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t& high, uint32_t& low) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    high = __byte_perm(a, b, 0x7632);
    constexpr float kUp = 1.f + 0x1p-20f;
    low = pack_bf16(fmaf(x, kUp, -__uint_as_float(a & 0xffff0000u)), fmaf(y, kUp, -__uint_as_float(b & 0xffff0000u)));
}

__device__ __forceinline__ void store_chunk(uint32_t to, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Two 16-bit halves of w with the non-finite bf16 ones cleared.
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
    return w;
}

template <int N, int D, Copy kCopy>
__global__ void __launch_bounds__(Roles<N, D, kCopy>::kWarps * 32, 1)
attn_mma_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                const int bx, const int page_heads) {
    using L = Smem<N, D, kCopy>;
    using R = Roles<N, D, kCopy>;
    constexpr int kParts = R::kParts, kSoftWarps = R::kSoftWarps, kKeyWarp = R::kKeyWarp, kMmaWarp = R::kMmaWarp, kSegWarp = R::kSegWarp, kValWarp = R::kValWarp;
    constexpr int HC = N / kParts;           // columns of a softmax group
    constexpr int kStages = L::kStages, kUnits = L::kUnits;
    constexpr bool kExact = kCopy == Copy::kBoxes && kUnits == 1;     // the head fills the row
    const int hd = kExact ? D : p.D;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile uint32_t* s_flags = reinterpret_cast<volatile uint32_t*>(gbase + L::kFlags);   // [0] TMEM, [1] abort, [2] fix
    volatile uint32_t* s_bad = s_flags + 6;     // [kBadRing][4] boxes (one word), or positions, of a step whose page is out of range
    volatile Seg* s_seg = reinterpret_cast<volatile Seg*>(gbase + L::kSeg);
    volatile uint32_t* abort_flag = s_flags + 1;
    uint32_t bar = base + L::kBar;
    auto take = [&](int n) { const uint32_t b = bar; bar += 8u * n; return b; };
    const uint32_t b_full = take(kStages), b_empty = take(kStages);
    const uint32_t b_seg_full = take(kSegs), b_seg_empty = take(kSegs);
    const uint32_t b_q_full = take(L::kQBufs), b_q_empty = take(L::kQBufs), b_s_full = take(2), b_s_empty = take(2);
    const uint32_t b_o_empty = take(2), b_p_full = take(1), b_pv = take(1), b_end = take(1);

    if (tid == 0) {
        grid_launch_dependents();       // the join is scheduled now and waits for this grid
        for (int i = 0; i < kStages; ++i) { ptx::mbar_init(b_full + 8 * i, kCopy == Copy::kRows ? 2 * 33 : 1); ptx::mbar_init(b_empty + 8 * i, 1); }
        for (int i = 0; i < kSegs; ++i) { ptx::mbar_init(b_seg_full + 8 * i, 1); ptx::mbar_init(b_seg_empty + 8 * i, 1 + R::kProducers + kSoftWarps); }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(b_s_full + 8 * i, 1); ptx::mbar_init(b_s_empty + 8 * i, kSoftWarps);
            ptx::mbar_init(b_o_empty + 8 * i, kSoftWarps);
        }
        for (int i = 0; i < L::kQBufs; ++i) { ptx::mbar_init(b_q_full + 8 * i, 32); ptx::mbar_init(b_q_empty + 8 * i, 1); }
        ptx::mbar_init(b_p_full, kSoftWarps); ptx::mbar_init(b_pv, 1); ptx::mbar_init(b_end, 1);
        s_flags[1] = 0u;
        s_flags[2] = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(base + L::kFlags, L::kTmem);
        ptx::tmem_relinquish();
    }
    if (kCopy != Copy::kRows && warp == kKeyWarp && lane == 0) ptx::prefetch_tmap(&kmap);
    if (kCopy != Copy::kRows && warp == kValWarp && lane == 0) ptx::prefetch_tmap(&vmap);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = s_flags[0];
    grid_dependency_wait();             // the set-up above overlaps the launch before this one
    const long long wl = wait_limit_of(reinterpret_cast<const unsigned long long*>(p.status) + 1);
    auto wait = [&](uint32_t b, uint32_t parity) { return ptx::mbar_wait_strict(b, parity & 1u, abort_flag, wl); };
    auto give_up = [&](int site) {
        raise_timeout(p.status, site);
        *abort_flag = 1u;
    };

    if (warp == kSegWarp) {
        // ------------------------------------------------ segments and Q tiles
        const int first_round = attn_first_round(p);
        const AttnSplit sp(p, p.tile_off[p.B], p.tile_off[0]);
        const int cta = blockIdx.x, nbox = kCopy == Copy::kRows ? 0 : kSteps / bx;
        bool ok = true;
        int t = 0, end = 0;
        AttnSegment g{};
        AttnSplitRow split{};                    // the segment that begins here and goes on in the next CTA
        if (cta < sp.n) {
            t = sp.first(cta);
            end = sp.first(cta + 1);
            g = attn_segment(p, sp, t, first_round);
        }
        // to the next segment of this CTA that has tiles: the next head or row
        // tile, or the next request
        auto skip = [&]() {
            while (t < end && g.tile(sp, t) == g.tile(sp, end)) {
                const int to = g.tiles > 0 ? g.t0 + sp.pad + g.tiles : attn_request_at(p, sp, g.b + 1) * sp.heads;
                // offsets that do not ascend: nothing more (the places, or the requests at
                // one place, ascend from here on, so the walk ends)
                t = to > t || (to == t && g.tiles > 0) ? to : end;
                if (t >= end) break;
                if (g.tiles > 0 && ++g.rt == p.row_tiles) { g.rt = 0; ++g.h; }
                g.t0 = t;
                if (g.tiles == 0 || g.h == p.Hkv) {
                    // the next request, or (after one without tiles) looked up
                    if (g.tiles > 0) g = attn_segment_of(p, sp, t, g.b + 1, attn_request_at(p, sp, g.b + 1), attn_request_at(p, sp, min(p.B, g.b + 2)));
                    else g = attn_segment(p, sp, t, attn_first_round(p));
                }
            }
        };
        skip();
        // descriptor si, then the Q tile of segment si - 1: the producers learn of
        // a segment while the Q buffers are still taken by the two before it
        int q0 = 0, qh = 0, qr0 = 0, qrows = 0;
        for (int si = 0; ok; ++si) {
            const int slot = si % kSegs;
            if (si >= kSegs) ok = __all_sync(~0u, wait(b_seg_empty + 8 * slot, (si / kSegs) - 1));
            if (!ok) { if (lane == 0) give_up(0); break; }
            const bool more = t < end;
            volatile Seg& d = s_seg[slot];
            int n0 = 0, nrows = 0, nr0 = 0;
            if (more) {
                // four loads on their way together: the page of this lane's box as if
                // the request were as long as its tiles say
                const int j0 = g.tile(sp, t), j1 = g.tile(sp, end);
                const unsigned pos_in = (unsigned)j0 * kTile + lane * bx;
                const int cap = p.width * p.page_size;
                const int len_in = p.kv_len[g.b], qa = p.q_off[g.b], qe = p.q_off[g.b + 1];
                const int page_in = lane < nbox && pos_in < (unsigned)cap ? __ldg(p.table + (size_t)g.b * p.width + p.by_page((int)pos_in)) : -1;
                int n = qe - qa, len = len_in;
                n0 = qa;
                if (n > p.max_new || n < 0 || qa < 0 || qa > p.N - n || len < 0 || len > cap) {
                    if (lane == 0) raise_status(p.status, kBadLength);
                    n = qa < 0 ? 0 : max(0, min(n, min(p.max_new, p.N - qa)));
                    len = max(0, min(len, cap));
                }
                nr0 = g.rt * p.row_tile;
                nrows = max(0, min(p.row_tile, n * p.G - nr0));
                // no row of the request here, or offsets that do not fit its length: nothing to publish
                if (nrows == 0 || g.tiles != attn_tiles(len)) {
                    t = g.t0 + sp.pad + j1;
                    skip();
                    --si;
                    continue;
                }
                const int pos0 = min(j0 * kTile, len), pos1 = min(j1 * kTile, len);
                if (lane < nbox) d.page[lane] = (int)pos_in < pos1 ? page_in : -1;
                if (j0 == 0 && j1 < g.tiles) split = attn_split_row(sp, g, cta, qa, nr0, nrows);
                if (lane == 0) {
                    d.b = g.b; d.h = g.h; d.q0 = qa; d.n = n; d.len = len; d.r0 = nr0; d.rows = nrows;
                    d.pos0 = pos0; d.pos1 = pos1;
                    d.steps = max(1, (pos1 - pos0 + kSteps - 1) / kSteps);
                    d.slot = j0 == 0 && j1 == g.tiles ? -1 : 2 * cta + (j0 == 0 ? 1 : 0);
                }
            } else if (lane == 0) d.steps = -1;
            const int nh = g.h;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(b_seg_full + 8 * slot);
            if (si > 0) {
                // the Q tile, rows beyond the request's as zeros
                const int qi = si - 1, qb = qi % L::kQBufs;
                if (qi >= L::kQBufs) ok = __all_sync(~0u, wait(b_q_empty + 8 * qb, (qi / L::kQBufs) - 1));
                if (!ok) { if (lane == 0) give_up(1); break; }
                // lane: a 16-byte chunk c of rows r, r + kRows, ...
                constexpr int kChunks = D / 8, kRows = 32 / kChunks;
                const int c = lane % kChunks;
                int r = lane / kChunks, tok = p.by_group(qr0 + r), head = qr0 + r - tok * p.G;
                const uint16_t* q = static_cast<const uint16_t*>(p.q);
                const uint16_t* src = q + (q0 + tok) * p.q_stride + (size_t)(qh * p.G + head) * hd + 8 * c;
                const bool in_head = kExact || 8 * c < hd;
                const uint32_t qs = base + L::kQ + qb * L::kQBytes + (c / 8) * (N * 128);
#pragma unroll 4
                for (int i = 0; i < N / kRows; ++i) {
                    const bool have = r < qrows && in_head;
                    ptx::cp_async_16(qs + r * 128 + (((c & 7) ^ (r & 7)) << 4), have ? src : q, have ? 16u : 0u);
                    r += kRows;
                    head += kRows;
                    src += kRows * hd;
                    while (head >= p.G) { head -= p.G; src += p.q_stride - (long long)p.G * hd; }
                }
                cp_async_arrive(b_q_full + 8 * qb);  // when this lane's copies have landed
            }
            if (!more) break;
            q0 = n0; qh = nh; qr0 = nr0; qrows = nrows;
            t = g.t0 + sp.pad + g.tile(sp, end);     // the place behind the tiles just taken
            skip();
        }
        if (lane == 0) p.split[cta] = split;
    } else if (warp == kKeyWarp || warp >= kValWarp) {
        // ------------------------------------------------------------ producers
        const int kv = (warp - kKeyWarp) & 1, part = warp > kValWarp;     // (part: row by row, the second half)
        const CUtensorMap* map = kv ? &vmap : &kmap;
        const uint64_t pol = p.row_tiles == 1 ? ptx::policy_evict_first() : ptx::policy_evict_last();
        const int nbox = kSteps / bx;
        uint32_t fill = kv * kUnits;             // this warp's next stage: keys tiles 0, 2, .., values tiles 1, 3, ..
        static_assert(kStages / 2 + 1 < kBadRing, "the producer stays within the ring of bad boxes");
        bool ok = true;
        for (int si = 0; ok; ++si) {
            const int slot = si % kSegs;
            ok = __all_sync(~0u, wait(b_seg_full + 8 * slot, si / kSegs));
            if (!ok) { if (lane == 0) give_up(2); break; }
            const Seg& sg = const_cast<Seg&>(s_seg[slot]);
            struct { int b, h, pos0, pos1, steps; } d = {sg.b, sg.h, sg.pos0, sg.pos1, sg.steps};
            int page = sg.page[lane & 15];
            __syncwarp();
            if (d.steps < 0) break;
            if (lane == 0) ptx::mbar_arrive(b_seg_empty + 8 * slot);
            const int32_t* row = p.table + (size_t)d.b * p.width;
            if constexpr (kCopy == Copy::kRows) {
                const uint16_t* from = static_cast<const uint16_t*>(kv ? p.v : p.k) + (long long)d.h * p.page_size * hd;
                constexpr int kChunks = L::kUnit / 8, kAt = 32 / kChunks;      // 16-byte chunks of a row, rows of an instruction
                const int c = lane % kChunks, sub = lane / kChunks;
                int pages[2];                    // of this lane's positions 64 part + lane, + 32
                auto look_up = [&](int pos0) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int pos = pos0 + 64 * part + 32 * i + lane;
                        pages[i] = pos < d.pos1 ? __ldg(row + p.by_page(pos)) : -1;
                    }
                };
                look_up(d.pos0);
                for (int s = 0; s < d.steps && ok; ++s, fill += kUnits) {
                    long long at[2];             // where they lie, -1: nowhere, their rows are zeros
                    uint32_t bad[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int pos = d.pos0 + s * kSteps + 64 * part + 32 * i + lane;
                        const bool have = pos < d.pos1 && pages[i] >= 0 && pages[i] < p.pages;
                        at[i] = have ? pages[i] * p.page_stride + (long long)(pos - p.by_page(pos) * p.page_size) * hd : -1;
                        bad[i] = __ballot_sync(~0u, pos < d.pos1 && !have);
                    }
                    if ((bad[0] | bad[1]) && lane == 0) raise_status(p.status, kBadPage);
                    look_up(d.pos0 + (s + 1) * kSteps);
#pragma unroll
                    for (int u = 0; u < kUnits; ++u, ++fill) {
                        const int stage = fill % kStages;
                        if (fill >= (uint32_t)kStages) ok = __all_sync(~0u, wait(b_empty + 8 * stage, fill / kStages - 1));
                        if (!ok) { if (lane == 0) give_up(3); break; }
                        if (lane == 0) {
                            if (!kv) {
                                s_bad[(fill / (2 * kUnits)) % kBadRing * 4 + 2 * part] = bad[0];
                                s_bad[(fill / (2 * kUnits)) % kBadRing * 4 + 2 * part + 1] = bad[1];
                            }
                            ptx::mbar_arrive(b_full + 8 * stage);
                        }
                        const uint32_t to = base + L::kRing + stage * L::kTileBytes + 8 * part * L::kGroup + (c / 8) * L::kHalf;
                        const uint16_t* mine = from + u * 128 + 8 * c;
                        const bool in_head = u * 128 + 8 * c < hd;
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int j = 0; j < 32; j += kAt) {
                                const int r = j + sub;                         // row 64 part + 32 i + r of the tile
                                const long long o = __shfl_sync(~0u, at[i], r);
                                const bool have = in_head && o >= 0;
                                ptx::cp_async_16(to + (4 * i + j / 8) * L::kGroup + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4),
                                                 have ? mine + o : from, have ? 16u : 0u);
                            }
                        cp_async_arrive(b_full + 8 * stage);       // when this lane's copies have landed
                    }
                }
            } else for (int s = 0; s < d.steps; ++s, fill += kUnits) {
                const int pos = d.pos0 + s * kSteps + lane * bx;
                const bool want = lane < nbox && pos < d.pos1;
                const bool have = want && page >= 0 && page < p.pages;
                const uint32_t bad = __ballot_sync(~0u, want && !have);
                const int boxes = __popc(__ballot_sync(~0u, have));
                if (bad && lane == 0) raise_status(p.status, kBadPage);
                const int group = (pos - p.by_page(pos) * p.page_size) >> 3, z = page * page_heads + d.h;
                // the next step's page
                page = lane < nbox && pos + kSteps < d.pos1 ? __ldg(row + p.by_page(pos + kSteps)) : -1;
#pragma unroll
                for (int u = 0; u < kUnits; ++u, ++fill) {
                    const int stage = fill % kStages;
                    if (fill >= (uint32_t)kStages) ok = __all_sync(~0u, wait(b_empty + 8 * stage, fill / kStages - 1));
                    if (!ok) { if (lane == 0) give_up(3); break; }
                    const uint32_t full = b_full + 8 * stage;
                    if (lane == 0) {
                        if (!kv) s_bad[(fill / (2 * kUnits)) % kBadRing * 4] = bad;
                        if (boxes) ptx::mbar_arrive_expect_tx(full, boxes * bx * L::kUnit * 2);
                        else ptx::mbar_arrive(full);
                    }
                    __syncwarp();
                    const uint32_t to = base + L::kRing + stage * L::kTileBytes + lane * (bx / 8) * L::kGroup;
                    if (have) {
                        if constexpr (kCopy == Copy::kHalves) {
                            tma_load_rows(to, map, 0, 8 * group, z, full, pol);
                            tma_load_rows(to + L::kHalf, map, 64, 8 * group, z, full, pol);
                        } else tma_load_box(to, map, 2 * u, group, z, full, pol);
                    }
                }
                if (!ok) break;
            }
        }
        // every copy issued lands before the CTA leaves: the last fill of each stage
        if constexpr (kCopy == Copy::kRows) ptx::cp_async_wait_all();
        else {
            if (lane == 0) s_flags[4 + kv] = fill;
            ptx::named_barrier(1 + kParts, 64);
        }
        if (kCopy != Copy::kRows && lane == 0 && !kv) {
            const uint32_t keys = s_flags[4], vals = s_flags[5];      // stages of tiles 0, 2, .. < keys and of 1, 3, .. < vals
            for (uint32_t i = 0; i < (uint32_t)kStages; ++i) {
                // the last fill of stage i
                const uint32_t top = max(keys, vals);
                for (uint32_t f = top; f-- > 0 && f + 4 * kStages >= top;)
                    if (f % kStages == i && f < (f / kUnits & 1u ? vals : keys)) {
                        ptx::mbar_wait_drain(b_full + 8 * i, (f / kStages) & 1u, kDrainCycles);
                        break;
                    }
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        // the whole warp runs the loop, so that descriptors are uniform values;
        // one elected lane issues
        constexpr uint32_t id_s = ptx::idesc_bf16_f32(128, N, false, false);
        constexpr uint32_t id_o = ptx::idesc_bf16_f32(128, L::kO, true, true);
        const uint32_t one = elect_one();
        const uint64_t k_desc = ptx::smem_desc_sw128(base + L::kRing, 16, L::kGroup);
        // V^T: entries of a position lie along M, the 64-entry halves kHalf
        // apart (head size 64: the second half of the lanes repeats the
        // first and is not used); 16 positions = 2 groups
        const uint64_t v_desc = ptx::smem_desc_sw128(base + L::kRing, L::kHalf, L::kGroup);
        const uint64_t q_desc = ptx::smem_desc_sw128(base + L::kQ, 16, 1024);
        const uint64_t p_desc = ptx::smem_desc_sw128(base + L::kP, N == 128 ? kSteps * 128 : 16, 1024);
        // Whatever is ready goes first: the O product of the oldest step whose S
        // product was issued, or the next S product (of the next segment, too), at
        // most one step ahead: further, a producer could be two phases ahead of a
        // stage's barrier, whose parity tells only one.  Short segments keep both going.
        struct Step { uint32_t step, seg; bool first; } old{}, young{};   // S issued, O not: the oldest, and one behind it
        bool has_old = false, has_young = false, in_seg = false, q_ready = false, done = false, ok = true;
        uint32_t step = 0, si = 0;
        int s = 0, steps = 0, idle = 0;
        long long since = clock64();
        auto ready = [&](uint32_t b, uint32_t phase) { return __all_sync(~0u, ptx::mbar_test_wait(b, phase & 1u)); };
        auto landed = [&](uint32_t fill) {       // the tile that begins at this fill
            return ready(b_full + 8 * (fill % kStages), fill / kStages) &&
                   (kUnits == 1 || ready(b_full + 8 * ((fill + 1) % kStages), (fill + 1) / kStages));
        };
        while (!(done && !has_old)) {
            bool moved = false;
            if (has_old) {                       // O^T (+)= V^T P^T
                const uint32_t vi = (2 * old.step + 1) * kUnits, ob = old.seg & 1u;
                if (ready(b_p_full, old.step) && landed(vi) &&
                    (!old.first || old.seg < 2 || ready(b_o_empty + 8 * ob, old.seg / 2 - 1))) {
                    ptx::tc_fence_after();
                    if (kCopy == Copy::kRows) ptx::fence_proxy_async_smem();
                    if (one) {
#pragma unroll
                        for (int u = 0; u < kUnits; ++u) {
                            const uint32_t st = (vi + u) % kStages;
                            const uint64_t va = v_desc + st * (L::kTileBytes / 16);
#pragma unroll
                            for (int w = 0; w < (L::kWeights == Weights::kBlocks ? 2 : 1); ++w)
#pragma unroll
                                for (int k = 0; k < kSteps / 16; ++k)
                                    ptx::mma_f16(tmem + 2 * N + (ob * kUnits + u) * L::kO, va + k * (2 * L::kGroup / 16),
                                                 p_desc + w * (kSteps * 128 / 16) + k * (2048 / 16), id_o, old.first && w + k == 0 ? 0u : 1u);
                            ptx::mma_commit(b_empty + 8 * st);
                        }
                        ptx::mma_commit(b_pv);
                    }
                    __syncwarp();
                    old = young;
                    has_old = has_young;
                    has_young = false;
                    moved = true;
                }
            }
            if (!done && !in_seg && ready(b_seg_full + 8 * (si % kSegs), si / kSegs)) {
                steps = s_seg[si % kSegs].steps;
                __syncwarp();
                if (steps < 0) done = true;
                else {
                    if (lane == 0) ptx::mbar_arrive(b_seg_empty + 8 * (si % kSegs));
                    in_seg = true;
                    q_ready = false;
                    s = 0;
                }
                moved = true;
            }
            if (in_seg && !has_young) {          // S^T = K Q^T
                const uint32_t qb = si % L::kQBufs, ki = 2 * step * kUnits, sb = step & 1u;
                if (!q_ready && ready(b_q_full + 8 * qb, si / L::kQBufs)) {
                    ptx::fence_proxy_async_smem();       // the Q tile came by the generic proxy
                    q_ready = true;
                }
                if (q_ready && landed(ki) && (step < 2 || ready(b_s_empty + 8 * sb, step / 2 - 1))) {
                    ptx::tc_fence_after();
                    if (kCopy == Copy::kRows) ptx::fence_proxy_async_smem();   // the rows came by the generic proxy
                    if (one) {
#pragma unroll
                        for (int u = 0; u < kUnits; ++u) {
                            const uint32_t st = (ki + u) % kStages;
                            const uint64_t ka = k_desc + st * (L::kTileBytes / 16);
                            const uint64_t qa = q_desc + qb * (L::kQBytes / 16) + u * (2 * N * 128 / 16);
#pragma unroll
                            for (int k = 0; k < L::kUnit / 16; ++k)
                                ptx::mma_f16(tmem + sb * N, ka + (k / 4) * (L::kHalf / 16) + (k % 4) * 2,
                                             qa + (k / 4) * (N * 128 / 16) + (k % 4) * 2, id_s, u || k ? 1u : 0u);
                            ptx::mma_commit(b_empty + 8 * st);
                        }
                        ptx::mma_commit(b_s_full + 8 * sb);
                        if (s == steps - 1) ptx::mma_commit(b_q_empty + 8 * qb);
                    }
                    __syncwarp();
                    const Step now{step, si, s == 0};
                    if (has_old) { young = now; has_young = true; }
                    else { old = now; has_old = true; }
                    ++step;
                    if (++s == steps) { in_seg = false; ++si; }
                    moved = true;
                }
            }
            if (moved) idle = 0;
            else {
                if (idle == 0) since = clock64();
                __nanosleep(20);
                if ((++idle & 15) == 0 || wl < (1LL << 20))
                    if (__any_sync(~0u, *abort_flag != 0u || clock64() - since > wl)) { ok = false; break; }
            }
        }
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
        const float scale2 = p.scale * kLog2e;
        const int my_box = kCopy == Copy::kRows ? lane : row / bx, bad_word = kCopy == Copy::kRows ? quarter : 0;
        float4* s_max = reinterpret_cast<float4*>(gbase + L::kMax);
        float4* s_sum = reinterpret_cast<float4*>(gbase + L::kSum);
        // columns in chunks of CH; with more than one, scores are read from tensor
        // memory twice and the references from shared memory
        constexpr int CH = HC > 16 ? 16 : HC, NCH = HC / CH;
        float* s_neg = reinterpret_cast<float*>(gbase + L::kNeg) + group * HC;
        uint32_t step = 0;
        bool ok = true;
        // A segment's rows are written after the first step of the next segment
        // (its O^T is in the other half of tensor memory), so the tensor core
        // and the producers go on meanwhile.  What is kept of it until then:
        bool pend = false;
        float pend_ref = 0.f;                                      // lane c: column c's reference
        for (uint32_t si = 0;; ++si) {
            const int slot = si % kSegs;
            ok = wait(b_seg_full + 8 * slot, si / kSegs) && ok;
            if (ptx::bar_red_or(1 + group, 128, !ok)) { ok = false; break; }
            const Seg& sg = const_cast<Seg&>(s_seg[slot]);
            struct { int n, len, r0, pos0, pos1, steps; } d = {sg.n, sg.len, sg.r0, sg.pos0, sg.pos1, sg.steps};
            const bool none = d.steps < 0;                         // no more segments
            if (none && !pend) break;
            const uint32_t o_at = tmem + lanes + 2 * N + (si & 1u) * (kUnits * L::kO) + group * HC;
            const int first_new = d.len - d.n;                     // position of the block's first token
            // lane c: the last position that column c of this group sees
            const int my_last = first_new + p.by_group(d.r0 + group * HC + (lane & (HC - 1)));
            float neg[CH], l[HC];                                  // minus the reference, this thread's sum of the weights
#pragma unroll
            for (int c = 0; c < CH; ++c) neg[c] = 0.f;
#pragma unroll
            for (int c = 0; c < HC; ++c) l[c] = 0.f;
            float my_ref = -INFINITY;                              // lane c: column c's reference, -inf before the first score
            bool unset = true;                                     // a column of the group has no reference yet
            bool stop = false;
            for (int s = 0; s < d.steps || s == 0; ++s) {
                if (!none) {
                const int pos0 = d.pos0 + s * kSteps, pos = pos0 + row, there = d.pos1 - pos0;
                ok = wait(b_s_full + 8 * (step & 1u), step / 2) && ok;
                ok = __all_sync(~0u, ok);
                const uint32_t s_at = tmem + lanes + (step & 1u) * N + group * HC;
                const uint32_t bad = ok ? s_bad[step % kBadRing * 4 + bad_word] : 0u;
                // positions beyond the end or in a bad page, and the block's later tokens
                const bool edge = there < kSteps || bad || pos0 + kSteps > first_new + 1;
                const bool gone = row >= there || (bad >> my_box & 1u);
                float x[CH];
                // the scores of chunk k, -inf where the column does not see the position
                // (read again where a reference moves)
                auto scores = [&](int k) {
                    if (ok) tmem_get<CH>(s_at + k * CH, x);
                    else {
#pragma unroll
                        for (int c = 0; c < CH; ++c) x[c] = 0.f;
                    }
                    if (edge) {
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            const int last = __shfl_sync(~0u, my_last, k * CH + c);
                            if (gone || pos > last) x[c] = -INFINITY;
                        }
                    }
                };
                auto refs = [&](int k) {
                    if constexpr (NCH > 1) {
#pragma unroll
                        for (int c = 0; c < CH; c += 4)
                            *reinterpret_cast<float4*>(neg + c) = *reinterpret_cast<const float4*>(s_neg + k * CH + c);
                    }
                };
                // .. as exponents
                auto exponents = [&]() {
#pragma unroll
                    for (int c = 0; c < CH; c += 2) fma_pair(x[c], x[c + 1], scale2, neg[c], neg[c + 1]);
                };
                auto read_done = [&]() {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(b_s_empty + 8 * (step & 1u));
                };
                ptx::tc_fence_after();
                float high = -INFINITY;
                if (NCH == 1 || !unset) {
#pragma unroll
                    for (int k = 0; k < NCH; ++k) {
                        scores(k);
                        refs(k);
                        exponents();
#pragma unroll
                        for (int c = 0; c < CH; ++c) high = fmaxf(high, x[c]);
                    }
                }
                // (unset is the same in the whole group)
                const bool move = unset || ptx::bar_red_or(1 + group, 128, high > kSlack || !ok);
                // the product before this one is done: P may be overwritten, O rescaled
                if (step > 0) ok = wait(b_pv, step - 1) && ok;
                if (move) {                     // the same in every thread of the group
                    float mine = -INFINITY;
#pragma unroll
                    for (int k = 0; k < NCH; ++k) {
                        scores(k);
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            const float w = warp_max(x[c]);
                            if (lane == k * CH + c) mine = w;
                        }
                    }
                    float* mx = reinterpret_cast<float*>(s_max + (step & 1u) * N + group * HC);
                    if (lane < HC) mx[lane * 4 + quarter] = mine;
                    if (ptx::bar_red_or(1 + group, 128, !ok)) { stop = true; break; }
                    const float4 w4 = reinterpret_cast<const float4*>(mx)[lane & (HC - 1)];
                    const float top = fmaxf(fmaxf(w4.x, w4.y), fmaxf(w4.z, w4.w)) * scale2;
                    const float to = fmaxf(my_ref, top);
                    const float my_a = to > my_ref ? fast_exp2(my_ref - to) : 1.f;
                    my_ref = to;
                    unset = __any_sync(~0u, to == -INFINITY);
                    // (the next write here, two steps on, comes after another barrier)
                    if (NCH > 1) {
                        if (quarter == 0) s_neg[lane] = to == -INFINITY ? 0.f : -to;
                        ptx::named_barrier(1 + group, 128);
                    }
                    if (s > 0) ptx::tc_fence_after();
#pragma unroll
                    for (int k = 0; k < NCH; ++k) {
                        float a[CH];
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            a[c] = __shfl_sync(~0u, my_a, k * CH + c);
                            if (NCH == 1) {
                                const float r = __shfl_sync(~0u, to, c);
                                neg[c] = r == -INFINITY ? 0.f : -r;
                            }
                            l[k * CH + c] *= a[c];
                        }
                        if (s > 0)
#pragma unroll
                            for (int u = 0; u < kUnits * L::kO / N; ++u) {
                                float o[CH];
                                tmem_get<CH>(o_at + u * N + k * CH, o);
#pragma unroll
                                for (int c = 0; c < CH; ++c) o[c] *= a[c];
                                tmem_put<CH>(o_at + u * N + k * CH, o);
                            }
                    }
                }
                if (NCH == 1) {
                    if (move) exponents();
                    read_done();
                }
                // weights: row `row` of P, columns group * HC ..
#pragma unroll
                for (int k = 0; k < NCH; ++k) {
                    if (NCH > 1) { scores(k); refs(k); exponents(); }
                    const int col0 = group * HC + k * CH;
                    const uint32_t prow = base + L::kP + (col0 / 64) * (kSteps * 128) + row * 128;
#pragma unroll
                    for (int c0 = 0; c0 < CH; c0 += 8) {
                        float w[8];
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            w[e] = fast_exp2(x[c0 + e]);
                            w[e + 1] = fast_exp2(x[c0 + e + 1]);
                            add_pair(l[k * CH + c0 + e], l[k * CH + c0 + e + 1], w[e], w[e + 1]);
                        }
                        const int chunk = (col0 + c0) / 8;
                        if constexpr (L::kWeights == Weights::kOne) {
                            store_chunk(prow + (((chunk & 7) ^ (row & 7)) << 4), pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]),
                                        pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7]));
                        } else {
                            uint32_t high[4], low[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) split_bf16(w[2 * e], w[2 * e + 1], high[e], low[e]);
                            constexpr int kBlock = L::kWeights == Weights::kBlocks ? kSteps * 128 : 0;
                            store_chunk(prow + ((chunk ^ (row & 7)) << 4), high[0], high[1], high[2], high[3]);
                            store_chunk(prow + kBlock + (((kBlock ? chunk : chunk + N / 8) ^ (row & 7)) << 4), low[0], low[1], low[2], low[3]);
                        }
                    }
                }
                if (NCH > 1) read_done();
                if (edge) {
                    // a value that no row may use is zero in shared memory: the
                    // product would turn 0 * NaN into NaN.  Of the block's later
                    // tokens, whose values some rows use, the non-finite entries
                    // are cleared and added again below to the rows that see them.
                    const uint32_t vi = (2 * step + 1) * kUnits;
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) ok = wait(b_full + 8 * ((vi + u) % kStages), (vi + u) / kStages) && ok;
                    const bool later = !gone && pos > first_new;
                    if (gone || later) {
                        // the groups share a row's chunks,
                        // each row begins at another one (other banks)
#pragma unroll
                        for (int c = group; c < D / 8; c += kParts) {
                            uint4* at = reinterpret_cast<uint4*>(gbase + L::kRing + ((vi + c / 16) % kStages) * L::kTileBytes +
                                                                 (row >> 3) * L::kGroup + (c / 8 % 2) * L::kHalf) + (row & 7) * 8 + ((c + row) & 7);
                            if (gone) *at = make_uint4(0u, 0u, 0u, 0u);
                            else {
                                const uint4 y = *at;
                                const uint4 z = make_uint4(finite_only(y.x), finite_only(y.y), finite_only(y.z), finite_only(y.w));
                                if (z.x != y.x || z.y != y.y || z.z != y.z || z.w != y.w) { *at = z; s_flags[2] = 1u; }
                            }
                        }
                    }
                }
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(b_p_full);
                ++step;
                }
                if (s > 0 || !pend) continue;
                // ------------------------------- the rows of the segment before
                // (its last product was waited for in the step above)
                pend = false;
                if (none) ok = wait(b_pv, step - 1) && ok;
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
#pragma unroll
                for (int i = 0; i < NCH * kUnits; ++i) {
                    const int k = i % NCH, u = i / NCH, dim = u * 128 + row;
                    float o[CH];
                    if (ok) {
                        const uint32_t at = tmem + lanes + 2 * N + ((pi & 1u) * kUnits + u) * L::kO + group * HC + k * CH;
                        tmem_get<CH>(at, o);
                        if constexpr (L::kWeights == Weights::kBeside) {
                            float y[CH];
                            tmem_get<CH>(at + N, y);
#pragma unroll
                            for (int c = 0; c < CH; ++c) o[c] += y[c];
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < CH; ++c) o[c] = 0.f;
                    }
                    if (s_flags[2]) {
                        // non-finite values of the block's later tokens (this CTA's positions)
                        for (int pos = max(e_new + 1, e.pos0); pos < e.pos1; ++pos) {
                            const int pg = p.by_page(pos), page = p.table[(size_t)e.b * p.width + pg];
                            if (page < 0 || page >= p.pages) continue;
                            float v = 0.f;
                            if (dim < hd)
                                v = to_f32(static_cast<const uint16_t*>(p.v)[page * p.page_stride +
                                           ((long long)e.h * p.page_size + (pos - pg * p.page_size)) * hd + dim]);
                            const bool odd = !(fabsf(v) < INFINITY);
#pragma unroll
                            for (int c = 0; c < CH; ++c) {
                                const int last = e_new + __shfl_sync(~0u, e_tok, k * CH + c);
                                if (odd && pos <= last) o[c] += v;
                            }
                        }
                    }
                    if (part_slot < 0) {
                        uint16_t* out = static_cast<uint16_t*>(p.out) + dim;
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            const float inv = __shfl_sync(~0u, e_inv, k * CH + c);
                            const int at = __shfl_sync(~0u, e_at, k * CH + c);
                            if (k * CH + c < cols && dim < hd) out[(size_t)at * hd] = (uint16_t)pack_bf16(o[c] * inv, 0.f);
                        }
                    } else {
                        float* part = p.part + ((size_t)part_slot * p.row_tile + group * HC + k * CH) * hd + dim;
#pragma unroll
                        for (int c = 0; c < CH; ++c)
                            if (k * CH + c < cols && dim < hd) part[c * hd] = o[c];
                    }
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(b_o_empty + 8 * (pi & 1u));
                if (quarter == 0 && lane < cols) {
                    if (part_slot >= 0) {
                        float2* stats = reinterpret_cast<float2*>(p.part + (size_t)2 * p.ctas * p.row_tile * hd);
                        stats[(size_t)part_slot * p.row_tile + e_row] = make_float2(pend_ref, pend_sum);
                    } else if (p.lse) p.lse[e_at] = pend_sum != 0.f ? pend_ref * kLn2 + logf(pend_sum) : -INFINITY;
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
            pend_ref = my_ref;
        }
        if (!ok && lane == 0) give_up(5);
    }
    // requests that own no cache position have no tile: their rows are zero; the
    // offsets of every request are compared with its length
    if (warp < kSoftWarps) {
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            const int off = p.tile_off[b], next = p.tile_off[b + 1];
            if (tid == 0 && !attn_offsets_fit(p, b, off, next)) raise_status(p.status, kBadLength);
            if (next > off) continue;
            int q0 = p.q_off[b], n = p.q_off[b + 1] - q0;
            if (tid == 0 && (n > p.max_new || n < 0 || q0 < 0 || q0 > p.N - n)) raise_status(p.status, kBadLength);
            n = q0 < 0 ? 0 : max(0, min(n, min(p.max_new, p.N - q0)));
            for (int i = tid; i < n * p.Hq * hd; i += kSoftWarps * 32) static_cast<uint16_t*>(p.out)[(size_t)q0 * p.Hq * hd + i] = 0;
            if (p.lse)
                for (int i = tid; i < n * p.Hq; i += kSoftWarps * 32) p.lse[(size_t)q0 * p.Hq + i] = -INFINITY;
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, L::kTmem);
}

template <int N, int D, Copy kCopy>
cudaError_t launch(const AttnParams& p, cudaStream_t s) {
    using L = Smem<N, D, kCopy>;
    constexpr bool kHalves = kCopy == Copy::kHalves;
    int bx = 64;                                 // positions of a box: a power of two that divides a page
    while (p.page_size % bx) bx >>= 1;
    const long long per_head = (long long)p.page_size * p.D;
    const int page_heads = (int)(p.page_stride / per_head);
    CUtensorMap maps[2] = {};
    if constexpr (kCopy != Copy::kRows) {
        auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tma_encoder());
        const cuuint64_t heads = (cuuint64_t)(p.pages - 1) * page_heads + p.Hkv, row = (cuuint64_t)p.D * 2, page = (cuuint64_t)per_head * 2;
        // a cache as [page and head][group of 8 positions][64-entry half][position][64 entries], or
        // [page and head][position][entry], what lies beyond the last entry read as zeros
        const cuuint64_t dims5[5] = {64, 8, (cuuint64_t)p.D / 64, (cuuint64_t)p.page_size / 8, heads}, strides5[4] = {row, 128, 8 * row, page};
        const cuuint32_t box5[5] = {64, 8, L::kUnit / 64, (cuuint32_t)bx / 8, 1};
        const cuuint64_t dims3[3] = {(cuuint64_t)p.D, (cuuint64_t)p.page_size, heads}, strides3[2] = {row, page};
        const cuuint32_t box3[3] = {64, (cuuint32_t)bx, 1};
        const cuuint32_t es[5] = {1, 1, 1, 1, 1};
        for (int i = 0; i < 2; ++i)
            if (enc(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kHalves ? 3 : 5, const_cast<void*>(i ? p.v : p.k), kHalves ? dims3 : dims5,
                    kHalves ? strides3 : strides5, kHalves ? box3 : box5, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return cudaErrorInvalidValue;
    }
    const size_t smem = L::kTotal + 1024;
    static_assert(L::kTotal + 1024 <= 232448 && L::kCols <= 512, "shared and tensor memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(attn_mma_kernel<N, D, kCopy>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(attn_mma_kernel<N, D, kCopy>, dim3(p.ctas), dim3(Roles<N, D, kCopy>::kWarps * 32), smem, s, p, maps[0], maps[1], bx, page_heads);
}

template <int D, Copy kCopy>
cudaError_t launch_head(const AttnParams& p, cudaStream_t s) {
    switch (p.row_tile) {
        case 16: return launch<16, D, kCopy>(p, s);
        case 32: return launch<32, D, kCopy>(p, s);
        case 64: return launch<64, D, kCopy>(p, s);
    }
    if constexpr (D <= 128 && kCopy != Copy::kRows) return launch<128, D, kCopy>(p, s);
    return cudaErrorInvalidValue;
}

}  // namespace

bool attn_pages_are_boxes(const AttnParams& p) {
    // pages a whole number of heads apart, all of them within a tensor map's last dimension
    const long long per_head = (long long)p.page_size * p.D;
    return (p.D <= 128 || p.D % 64 == 0) && p.page_size % 8 == 0 && p.page_stride % per_head == 0 &&
           p.page_stride / per_head < (1LL << 31) && p.pages * (p.page_stride / per_head) < (1LL << 31) &&
           tma_encoder() != nullptr;
}

cudaError_t launch_attn_mma(const AttnParams& p, cudaStream_t s) {
    if (!attn_pages_are_boxes(p)) {
        if (p.D > 128) return launch_head<256, Copy::kRows>(p, s);
        return p.D > 64 ? launch_head<128, Copy::kRows>(p, s) : launch_head<64, Copy::kRows>(p, s);
    }
    if (p.D > 128) return launch_head<256, Copy::kBoxes>(p, s);
    if (p.D == 128) return launch_head<128, Copy::kBoxes>(p, s);
    return p.D == 64 ? launch_head<64, Copy::kBoxes>(p, s) : launch_head<128, Copy::kHalves>(p, s);
}

}  // namespace dspark
