// serve_api.cu -- the C ABI of the serving operators (include/dspark.h):
// host-side argument checks, workspace layout and launches.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <string.h>

#include "serve.cuh"

namespace dspark {
namespace {

struct CallRange {
    explicit CallRange(const char* name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
};

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// a device pointer aligned to `a` bytes
bool dev(const void* p, size_t a = 4) { return aligned(p, a) && is_device_ptr(p); }
bool dev_or_null(const void* p, size_t a = 4) { return !p || dev(p, a); }
bool dtype_ok(dspark_dtype t) { return t == DSPARK_F32 || t == DSPARK_BF16; }
int bytes_of(dspark_dtype t) { return t == DSPARK_BF16 ? 2 : 4; }

bool head_ok(int D) { return D >= 8 && D <= DSPARK_MAX_HEAD_DIM && D % 8 == 0; }
bool pages_ok(int pages, int page_size) {
    return pages >= 1 && page_size >= 1 && page_size <= DSPARK_MAX_PAGE_SIZE && (long long)pages * page_size < (1LL << 31);
}

// A run of n 32-bit words.
struct Words {
    const int32_t* p;
    long long n;
    bool meets(const Words& o) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
        return n > 0 && o.n > 0 && a < b + 4 * o.n && b < a + 4 * n;
    }
};

// Workspaces: the status word in the first 256 bytes, then the regions.
constexpr size_t kHead = 256;

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

dspark_status dspark_cache_plan(const int32_t* seq_len, const int32_t* n_new, const int32_t* owned, int B,
                                int32_t* ring, const int32_t* ring_state, int pages, int32_t* block_table, int width,
                                int page_size, int32_t* owned_out, int32_t* ring_state_out, int32_t* kv_len,
                                int32_t* q_off, int32_t* tile_off, int32_t* slot_map, int32_t* positions,
                                int max_tokens, void* ws, void* stream) {
    const CallRange range_(__func__);
    if (B < 1 || B > DSPARK_MAX_CACHE_REQUESTS || width < 1 || max_tokens < 0 || max_tokens >= (1 << 30) ||
        !pages_ok(pages, page_size) || (long long)width * page_size >= (1LL << 31))
        return DSPARK_ERR_INVALID;
    if (!dev(seq_len) || !dev(n_new) || !dev(owned) || !dev(ring) || !dev(ring_state) || !dev(block_table) ||
        !dev(owned_out) || !dev(ring_state_out) || !dev(kv_len) || !dev(q_off) || !dev(tile_off) ||
        (max_tokens > 0 && (!dev(slot_map) || !dev(positions))) || !dev_or_null(ws, 256))
        return DSPARK_ERR_INVALID;
    // the inputs are read again while the outputs are written
    const Words in[] = {{seq_len, B}, {n_new, B}, {owned, B}, {ring_state, 2}};
    const Words out[] = {{owned_out, B}, {ring_state_out, 2}, {kv_len, B}, {q_off, B + 1}, {tile_off, B + 1}, {slot_map, max_tokens},
                         {positions, max_tokens}, {block_table, (long long)B * width}, {ring, pages}};
    for (const Words& o : out) {
        for (const Words& i : in)
            if (o.meets(i)) return DSPARK_ERR_INVALID;
        for (const Words* q = out; q != &o; ++q)
            if (o.meets(*q)) return DSPARK_ERR_INVALID;
    }
    PlanParams p;
    p.seq_len = seq_len; p.n_new = n_new; p.owned = owned;
    p.ring = ring; p.ring_state = ring_state; p.pages = pages;
    p.table = block_table; p.width = width; p.page_size = page_size;
    p.B = B; p.T = max_tokens;
    p.owned_out = owned_out; p.ring_state_out = ring_state_out; p.kv_len = kv_len;
    p.q_off = q_off; p.tile_off = tile_off; p.slot_map = slot_map; p.positions = positions;
    p.status = static_cast<uint32_t*>(ws);
    return launch_status(launch_cache_plan(p, static_cast<cudaStream_t>(stream)));
}

dspark_status dspark_cache_append(const void* k, const void* v, dspark_dtype kv_t, long long k_stride,
                                  long long v_stride, const int32_t* slot_map, int T, void* k_cache, void* v_cache,
                                  long long page_stride, int pages, int page_size, int kv_heads, int head_dim,
                                  void* ws, void* stream) {
    const CallRange range_(__func__);
    if (!dtype_ok(kv_t)) return DSPARK_ERR_UNSUPPORTED;
    if (T < 0 || kv_heads < 1 || kv_heads > 4096 || !head_ok(head_dim) || !pages_ok(pages, page_size))
        return DSPARK_ERR_INVALID;
    const int es = bytes_of(kv_t);
    const long long row = (long long)kv_heads * head_dim;
    if (k_stride < row || v_stride < row || page_stride < row * page_size || (k_stride * es) % 16 ||
        (v_stride * es) % 16 || (page_stride * es) % 16)
        return DSPARK_ERR_INVALID;
    if (T == 0) return DSPARK_OK;
    if (!dev(k, 16) || !dev(v, 16) || !dev(slot_map) || !dev(k_cache, 16) || !dev(v_cache, 16) || !dev_or_null(ws, 256))
        return DSPARK_ERR_INVALID;
    AppendParams p;
    p.k = static_cast<const char*>(k); p.v = static_cast<const char*>(v);
    p.k_stride = k_stride * es; p.v_stride = v_stride * es;
    p.slot_map = slot_map; p.T = T;
    p.k_cache = static_cast<char*>(k_cache); p.v_cache = static_cast<char*>(v_cache);
    p.page_bytes = page_stride * es;
    p.pages = pages; p.page_size = page_size; p.heads = kv_heads; p.row_bytes = head_dim * es;
    p.status = static_cast<uint32_t*>(ws);
    return launch_status(launch_cache_append(p, static_cast<cudaStream_t>(stream)));
}

static bool attn_sizes_ok(int B, int q_heads, int kv_heads, int head_dim, int max_new) {
    return B >= 1 && B <= DSPARK_MAX_CACHE_REQUESTS && kv_heads >= 1 && q_heads >= kv_heads && q_heads <= 4096 &&
           q_heads % kv_heads == 0 && head_ok(head_dim) && max_new >= 1 && max_new <= DSPARK_MAX_GAMMA + 1;
}

size_t dspark_cache_workspace_bytes(int B, int q_heads, int kv_heads, int head_dim, int max_new) {
    if (!attn_sizes_ok(B, q_heads, kv_heads, head_dim, max_new)) return 0;
    // the larger of the two kernels' tiles (of 9 to 16 rows 32 on CUDA cores, 16 on tensor cores)
    const int all = q_heads / kv_heads * max_new, mma = attn_row_tile(all, true), simt = attn_row_tile(all, false);
    const size_t rows = mma > simt ? mma : simt;
    return kHead + ws_align256(sizeof(AttnSplitRow) * kMaxAttnCtas) + ws_align256((size_t)2 * kMaxAttnCtas * rows * (head_dim + 2) * sizeof(float));
}

dspark_status dspark_cache_attention(const void* q, long long q_stride, const void* k_cache, const void* v_cache,
                                     dspark_dtype kv_t, long long page_stride, int pages, int page_size,
                                     const int32_t* block_table, int width, const int32_t* kv_len,
                                     const int32_t* q_off, const int32_t* tile_off, int B, int N, int q_heads,
                                     int kv_heads, int head_dim, int max_new, float scale, void* out, float* lse,
                                     void* ws, size_t ws_bytes, void* stream) {
    const CallRange range_(__func__);
    if (!dtype_ok(kv_t)) return DSPARK_ERR_UNSUPPORTED;
    // (the kernels look up to two steps of 128 positions beyond a length)
    if (!attn_sizes_ok(B, q_heads, kv_heads, head_dim, max_new) || N < 0 || width < 1 || !pages_ok(pages, page_size) ||
        (long long)width * page_size > (1LL << 31) - 256 || (long long)N * q_heads >= (1LL << 31))
        return DSPARK_ERR_INVALID;
    if (!(scale > 0.f && scale < 3e38f)) return DSPARK_ERR_INVALID;
    const int es = bytes_of(kv_t);
    if (page_stride < (long long)kv_heads * page_size * head_dim || (page_stride * es) % 16 ||
        q_stride < (long long)q_heads * head_dim || (q_stride * es) % 16)
        return DSPARK_ERR_INVALID;
    if (N == 0) return DSPARK_OK;
    if (!dev(q, 16) || !dev(k_cache, 16) || !dev(v_cache, 16) || !dev(block_table) || !dev(kv_len) || !dev(q_off) ||
        !dev(tile_off) || !dev(out, 16) || !dev_or_null(lse) || !dev(ws, 256))
        return DSPARK_ERR_INVALID;
    if (ws_bytes < dspark_cache_workspace_bytes(B, q_heads, kv_heads, head_dim, max_new)) return DSPARK_ERR_INVALID;
    AttnParams p;
    p.q = q; p.q_stride = q_stride; p.k = k_cache; p.v = v_cache; p.page_stride = page_stride;
    p.bf16 = kv_t == DSPARK_BF16;
    p.table = block_table; p.width = width;
    p.kv_len = kv_len; p.q_off = q_off; p.tile_off = tile_off;
    p.B = B; p.N = N; p.Hq = q_heads; p.Hkv = kv_heads; p.G = q_heads / kv_heads; p.D = head_dim;
    p.pages = pages; p.page_size = page_size; p.max_new = max_new;
    p.scale = scale; p.out = out; p.lse = lse;
    p.by_page.set((uint32_t)page_size);
    p.by_group.set((uint32_t)p.G);
    const int rows = p.G * max_new;
    const bool mma = p.bf16;                       // tensor cores
    p.row_tile = attn_row_tile(rows, mma);
    // tiles the block tables can hold (the lengths are on the device): few of
    // them, fewer rows at a time.  On CUDA cores where SMs would be idle
    // otherwise; 128 rows in two tiles of 64 below 32 tiles an SM and for heads
    // above 128, whose O^T of 128 columns tensor memory does not hold, and row
    // by row, where the copies bound it.  In two tiles / at once: 64 requests of
    // 1024-8192 positions, 8 heads 390 / 237 us (the cache read once); 8 of 8192,
    // 2 heads 32.3 / 32.3.  Tables far wider than the contexts go by the tables:
    // of 131072 positions, 64 requests of 1000 111 / 84, 8 of 1000 28.3 / 30.4, 8
    // of 100-300 19.8 / 24.4
    const long long tiles = ((long long)width * page_size + kTile - 1) / kTile * B * kv_heads;
    if (mma && p.row_tile == 128 && (head_dim > 128 || tiles < 32LL * num_sms() || !attn_pages_are_boxes(p))) p.row_tile = 64;
    if (!mma && tiles * ((rows + p.row_tile - 1) / p.row_tile) < 2LL * num_sms()) p.row_tile = 8;
    p.row_tiles = (rows + p.row_tile - 1) / p.row_tile;
    p.ctas = num_sms() < kMaxAttnCtas ? num_sms() : kMaxAttnCtas;      // one resident CTA per SM
    // (tensor cores: 64 requests of 64 rows, head size 128: 3 places 203 us, 4 196; 256 of 16-300
    // positions 72, 68; head size 96, the same: 4 places 73.4, 6 72.2, 32 rows 152.7 with 3, 150.5 with 6)
    p.pad = mma ? (head_dim < 128 ? 6 : 4) : 1;
    p.spare = mma;              // (on CUDA cores a tile costs more than its part: 4 short requests 13.4 us, two places a CTA 14.0)
    p.split = reinterpret_cast<AttnSplitRow*>(static_cast<char*>(ws) + kHead);
    p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kHead + ws_align256(sizeof(AttnSplitRow) * kMaxAttnCtas));
    p.status = static_cast<uint32_t*>(ws);
    return launch_status(launch_cache_attention(p, static_cast<cudaStream_t>(stream)));
}

size_t dspark_logits_workspace_bytes(int B, int R) {
    if (B < 1 || B > 65535 || R < 1 || R > DSPARK_MAX_GAMMA + 1) return 0;
    return kHead + ws_align256(sizeof(unsigned long long) * (size_t)B * R);
}

dspark_status dspark_logits_process(const void* logits, dspark_dtype t, long long row_stride, void* out, int B, int R,
                                    int V, const int32_t* hist, int hist_stride, const int32_t* hist_len,
                                    const int32_t* prompt_len, const int32_t* draft_tok, int draft_stride,
                                    const float* rep, const float* freq, const float* pres, const int32_t* bias_tok,
                                    const float* bias_val, const int32_t* bias_off, int bias_n, const uint32_t* mask,
                                    float fill, int32_t* live, void* ws, size_t ws_bytes, void* stream) {
    const CallRange range_(__func__);
    if (!dtype_ok(t)) return DSPARK_ERR_UNSUPPORTED;
    const size_t need = dspark_logits_workspace_bytes(B, R);
    if (need == 0 || V < 8 || V % 8 || V >= (1 << 30) || row_stride < V || (row_stride * bytes_of(t)) % 16)
        return DSPARK_ERR_INVALID;
    if (!dev(logits, 16) || !dev(out, 16) || !dev(ws, 256) || ws_bytes < need) return DSPARK_ERR_INVALID;
    if (out == logits && row_stride != V) return DSPARK_ERR_INVALID;      // in place: the same rows
    if (hist && (!dev(hist) || !dev(hist_len) || !dev_or_null(prompt_len) || hist_stride < 0 || hist_stride >= (1 << 28))) return DSPARK_ERR_INVALID;
    if (!hist && (hist_len || prompt_len)) return DSPARK_ERR_INVALID;
    if (draft_tok && (!dev(draft_tok) || draft_stride < R - 1)) return DSPARK_ERR_INVALID;
    if (!dev_or_null(rep) || !dev_or_null(freq) || !dev_or_null(pres) || !dev_or_null(mask) || !dev_or_null(live))
        return DSPARK_ERR_INVALID;
    if (fill != fill) return DSPARK_ERR_INVALID;
    if (bias_off && (bias_n < 0 || !dev(bias_off))) return DSPARK_ERR_INVALID;
    if (bias_off && bias_n > 0 && (!dev(bias_tok) || !dev(bias_val))) return DSPARK_ERR_INVALID;
    LogitsParams p;
    p.logits = logits; p.row_stride = row_stride; p.bf16 = t == DSPARK_BF16;
    p.out = out; p.B = B; p.R = R; p.V = V;
    p.hist = hist; p.hist_stride = hist ? hist_stride : 0;     // (tokens a row of hist holds)
    p.hist_len = hist_len; p.prompt_len = prompt_len;
    p.draft_tok = draft_tok; p.draft_stride = draft_stride;
    p.rep = rep; p.freq = freq; p.pres = pres;
    p.bias_tok = bias_off && bias_n > 0 ? bias_tok : nullptr;
    p.bias_val = bias_val; p.bias_off = bias_off; p.bias_n = bias_n;
    p.mask = mask; p.live = live;
    uint32_t word;
    memcpy(&word, &fill, sizeof(word));
    if (p.bf16) {                                  // nearest even
        word = (word + 0x7fffu + (word >> 16 & 1u)) >> 16;
        word |= word << 16;
    }
    p.low = word;
    char* base = static_cast<char*>(ws);
    p.status = reinterpret_cast<uint32_t*>(base);
    p.counts = reinterpret_cast<unsigned long long*>(base + kHead);
    return launch_status(launch_logits(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
