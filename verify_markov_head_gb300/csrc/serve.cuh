// serve.cuh -- parameter blocks, work partition and launchers of the serving
// operators around the draft + verify step: the paged key-value cache (plan,
// append, attention) and the controls on logits.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dspark {

// Status bits of the serving operators (beside those of common.cuh).
enum ServeStatusBits : uint32_t {
    kDeadRow = 1u << 4,      // a processed row of logits has no token left
    kBadPage = 1u << 5,      // a page or slot out of range, a block table too narrow, or no free page left
};

constexpr int kTile = DSPARK_CACHE_TILE;   // cache positions per attention tile
constexpr int kMaxAttnCtas = 160;          // CTAs of an attention launch (bounds its partial results)

// ---------------------------------------------------------------- cache plan
struct PlanParams {
    const int32_t* seq_len; const int32_t* n_new; const int32_t* owned;
    int32_t* ring; const int32_t* ring_state; int pages;
    int32_t* table; int width; int page_size;
    int B, T;
    int32_t* owned_out; int32_t* ring_state_out; int32_t* kv_len; int32_t* q_off; int32_t* tile_off;
    int32_t* slot_map; int32_t* positions;
    uint32_t* status;   // may be null
};
cudaError_t launch_cache_plan(const PlanParams& p, cudaStream_t s);

// -------------------------------------------------------------- cache append
struct AppendParams {
    const char* k; const char* v; long long k_stride, v_stride;   // bytes between tokens
    const int32_t* slot_map; int T;
    char* k_cache; char* v_cache; long long page_bytes;           // bytes between pages
    int pages, page_size, heads, row_bytes;                       // row_bytes: one head's vector
    uint32_t* status;   // may be null
};
cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t s);

// ----------------------------------------------------------- cache attention
// Division of 0 <= x < 2^31 by a number fixed on the host (Granlund and
// Montgomery, "Division by invariant integers using multiplication").
struct FastDiv {
    uint32_t d = 1, mul = 1, shift = 0;
    void set(uint32_t div) {
        d = div;
        shift = 0;
        while ((1ull << shift) < div) ++shift;
        mul = (uint32_t)((((1ull << shift) - div) << 32) / div + 1);
    }
    __device__ __forceinline__ int operator()(int x) const { return (int)((__umulhi((uint32_t)x, mul) + (uint32_t)x) >> shift); }
};

// What a CTA leaves for the join of a segment that begins in it.
struct __align__(16) AttnSplitRow {
    int parts;           // CTAs that hold a part of it, 0: no such segment
    int q0, h, r0;       // first token in q, key-value head, first query row
    int rows, pad[3];
};

struct AttnParams {
    const void* q; long long q_stride;                 // elements between tokens
    const void* k; const void* v; long long page_stride;   // elements between pages
    int bf16;
    const int32_t* table; int width;
    const int32_t* kv_len; const int32_t* q_off; const int32_t* tile_off;
    int B, N, Hq, Hkv, G, D, pages, page_size, max_new;
    float scale;
    void* out; float* lse;
    FastDiv by_page, by_group;  // by page_size, by G
    int row_tile, row_tiles;    // query rows of a key-value head per tile of rows, and such tiles
    int ctas;                   // CTAs the work is split over
    int pad;                    // what a segment costs beside its tiles, in tiles (at least 1)
    int spare;                  // few tiles: fewer CTAs, rather than a place for each
    AttnSplitRow* split;        // [ctas] the segment that begins in each CTA and ends in another
    float* part;                // [2 ctas][row_tile][D] sums, then [2 ctas][row_tile][2] (max, sum)
    uint32_t* status;
};
cudaError_t launch_cache_attention(const AttnParams& p, cudaStream_t s);
bool attn_pages_are_boxes(const AttnParams& p);   // bf16 pages that TMA can copy
cudaError_t launch_attn_mma(const AttnParams& p, cudaStream_t s);
// Rows of a row tile where a key-value head has `rows` query rows.
inline int attn_row_tile(int rows, bool mma) {
    return mma ? (rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128) : (rows <= 8 ? 8 : 32);
}

// The split of an attention launch.  A segment is the run of tiles of kTile
// cache positions of one (request, key-value head, row tile); the work is the
// list of all segments, ordered by request, head and row tile.  Beginning and
// ending a segment costs a CTA about as much as `pad` tiles, so each segment
// enters the list with `pad` places before its tiles, and CTA c takes the
// places [first(c), first(c + 1)), a contiguous share that differs by one at
// most.  A segment whose tiles lie in several CTAs leaves one partial result
// in each (slot 2c + 1 where its first tile is in c, else 2c), which the join
// kernel adds up in CTA order.
struct AttnSplit {
    int total;         // places, below 2^30
    int n;             // CTAs that have places
    int heads;         // key-value heads * row tiles
    int pad;
    int tiles;         // of one head and row tile
    int each, more;    // places of a CTA; the first `more` CTAs take one more
    // tiles_all = tile_off[B], first_off = tile_off[0]
    __device__ __forceinline__ AttnSplit(const AttnParams& p, int tiles_all, int first_off) {
        heads = p.Hkv * p.row_tiles;
        pad = p.pad;
        const long long most = (long long)p.B * (((long long)p.width * p.page_size + kTile - 1) / kTile);
        const long long all = ((long long)tiles_all + (long long)p.pad * p.B) * heads;
        const bool ok = tiles_all >= 0 && tiles_all <= most && first_off == 0 && all < (1LL << 30);
        if (!ok && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x % 32 == 0) raise_status(p.status, kBadLength);
        total = ok ? (int)all : 0;
        tiles = ok ? tiles_all : 0;
        n = total < p.ctas ? total : p.ctas;
        if (p.spare && n) {
            // few places: a place more is half a step, a part more a read of the join
            // behind the others', so shares grow as the root of a segment's length
            // (1000 positions, 8 heads: one place a CTA 11.0 us, two 9.5, five 10.2;
            // 8000, one head: one 30.2, two 21.4, five 17.6)
            int least = 2;                           // half the root of the mean length
            for (const float segments = 4.f * (float)(p.B * heads); segments * (float)((least + 1) * (least + 1)) <= (float)total;) ++least;
            n = min(n, (total + least - 1) / least);
        }
        each = n ? total / n : 0;
        more = n ? total - each * n : 0;
    }
    // Place of request b's first segment, in units of `heads` places, from the
    // entry tile_off[b].  An entry out of range is taken as the nearest one
    // within, so no place leaves the list whatever tile_off holds.
    __device__ __forceinline__ int at(int entry, int b) const { return min(max(entry, 0), tiles) + pad * b; }
    __device__ __forceinline__ int first(int c) const { return c * each + min(c, more); }
    __device__ __forceinline__ int cta_of(int t) const {
        const int longer = more * (each + 1);
        return t < longer ? t / (each + 1) : more + (t - longer) / each;
    }
};

struct AttnSegment {
    int b, h, rt;        // request, key-value head, row tile
    int t0;              // its first place in the list
    int tiles;           // its tiles (may be none), in the places t0 + pad ..
    // the tile at place t, or the first one after it
    __device__ __forceinline__ int tile(const AttnSplit& sp, int t) const { return min(max(0, t - t0 - sp.pad), tiles); }
};

// Tiles of a request of `len` positions.  What tile_off says of a request is
// compared with it: attn_offsets_fit for the status, and before a segment is
// worked on, since positions and table entries follow from its tiles.
__device__ __forceinline__ int attn_tiles(int len) { return len > 0 ? (len - 1) / kTile + 1 : 0; }
__device__ __forceinline__ bool attn_offsets_fit(const AttnParams& p, int b, int off, int next) {
    const int len = p.kv_len[b];
    return len >= 0 && len <= p.width * p.page_size && (unsigned)next - (unsigned)off == (unsigned)attn_tiles(len);
}

// What CTA c leaves of a segment that begins in it and goes on in the next.
__device__ __forceinline__ AttnSplitRow attn_split_row(const AttnSplit& sp, const AttnSegment& g, int c, int q0, int r0, int rows) {
    return AttnSplitRow{sp.cta_of(g.t0 + sp.pad + g.tiles - 1) - c + 1, q0, g.h, r0, rows, {0, 0, 0}};
}

// Place of request b's first segment, in units of `heads` places.
__device__ __forceinline__ int attn_request_at(const AttnParams& p, const AttnSplit& sp, int b) { return sp.at(p.tile_off[b], b); }

// The segment at place t of request b, whose places begin at off * heads and
// end at next * heads.
__device__ __forceinline__ AttnSegment attn_segment_of(const AttnParams& p, const AttnSplit& sp, int t, int b, int off, int next) {
    AttnSegment g;
    g.b = b;
    const int len = max(sp.pad, next - off), local = t - off * sp.heads;
    int hr = local / len;
    hr = hr < 0 ? 0 : (hr >= sp.heads ? sp.heads - 1 : hr);
    g.tiles = len - sp.pad;
    g.t0 = off * sp.heads + hr * len;
    g.h = hr / p.row_tiles;
    g.rt = hr - g.h * p.row_tiles;
    return g;
}

// The segment at place t, looked up by a whole warp: the request whose places
// enclose t, 32 requests at a time (`entry`: this lane's entry of the first
// round, attn_first_round).
__device__ __forceinline__ AttnSegment attn_segment(const AttnParams& p, const AttnSplit& sp, int t, int entry) {
    const int lane = threadIdx.x & 31, tt = t / sp.heads;
    int lo = 0, stride = (p.B + 31) / 32, mine = sp.at(entry, min(p.B, lane * stride));
    for (;;) {
        const unsigned le = __ballot_sync(~0u, mine <= tt && lo + lane * stride < p.B);
        const int k = le ? 31 - __clz(le) : 0;
        lo += k * stride;
        if (stride == 1) {
            const int off = __shfl_sync(~0u, mine, k);
            int next = __shfl_sync(~0u, mine, (k + 1) & 31);
            if (k == 31) next = attn_request_at(p, sp, min(p.B, lo + 1));
            return attn_segment_of(p, sp, t, lo, off, next);
        }
        stride = (stride + 31) / 32;
        mine = attn_request_at(p, sp, min(p.B, lo + lane * stride));
    }
}
__device__ __forceinline__ int attn_first_round(const AttnParams& p) {
    return p.tile_off[min(p.B, (int)(threadIdx.x & 31) * ((p.B + 31) / 32))];
}

// ------------------------------------------------------------------- logits
struct LogitsParams {
    const void* logits; long long row_stride; int bf16;   // elements between rows
    void* out;
    int B, R, V;
    const int32_t* hist; int hist_stride; const int32_t* hist_len; const int32_t* prompt_len;
    const int32_t* draft_tok; int draft_stride;
    const float* rep; const float* freq; const float* pres;
    const int32_t* bias_tok; const float* bias_val; const int32_t* bias_off; int bias_n;
    const uint32_t* mask;
    uint32_t low;                 // what a masked entry becomes: an fp32 word, or a bf16 one twice
    int32_t* live;
    uint32_t* status;
    unsigned long long* counts;   // [B][R] arrivals and entries left, zero between launches
};
cudaError_t launch_logits(const LogitsParams& p, cudaStream_t s);

}  // namespace dspark
