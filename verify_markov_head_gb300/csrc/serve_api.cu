// serve_api.cu -- the C ABI of the serving operators (include/dspark.h):
// host-side argument checks, workspace layout and launches.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <math.h>
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

// Addresses and page strides as whole rows allow: the largest power of two that divides a row, 16 at most.
int row_align(int row) { return (row | 16) & -(row | 16); }
bool exp_ok(int e) { return e >= -DSPARK_CACHE4_MAX_EXP && e <= DSPARK_CACHE4_MAX_EXP; }
float power(int e) { return ldexpf(1.f, e); }

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

struct Bytes {
    const char* p;
    long long n;
    bool meets(const Bytes& o) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
        return n > 0 && o.n > 0 && a < b + o.n && b < a + n;
    }
};
// Whether rows of `width` bytes, `stride` apart, share a byte with others.  Slices
// of one projection's rows (the same stride) interleave without sharing any.
bool rows_meet(const Bytes& a, long long a_stride, long long a_width, const Bytes& b, long long b_stride, long long b_width) {
    if (!a.meets(b)) return false;
    if (a_stride != b_stride) return true;
    long long gap = (reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p)) % a_stride;
    if (gap < 0) gap += a_stride;                // b's rows begin `gap` behind a's
    return gap < a_width || gap + b_width > a_stride;
}

// Rows of `width` bytes, `stride` apart: tokens of a projection, or pages of a cache.
struct Strided {
    Bytes all;
    long long stride, width;
    Strided(const void* p, long long n, long long stride_, long long width_)
        : all{static_cast<const char*>(p), p && n > 0 ? (n - 1) * stride_ + width_ : 0}, stride(stride_), width(width_) {}
    bool meets(const Strided& o) const { return rows_meet(all, stride, width, o.all, o.stride, o.width); }
    bool meets(const Bytes& o) const { return all.meets(o); }
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

// What the two calls over a cache in 4 bits share; false: an argument is refused.
static bool cache4_params(Cache4Params& p, const void* k_cache, const void* v_cache, const void* k_scale, const void* v_scale,
                          long long page_stride, long long scale_stride, int pages, int page_size, int kv_heads, int head_dim,
                          int k_exp, int v_exp, const int32_t* slot_map, int T, const void* k, const void* v, dspark_dtype kv_t,
                          long long k_stride, long long v_stride, void* ws, bool reads) {
    if (T < 0 || kv_heads < 1 || kv_heads > 4096 || !head_ok(head_dim) || head_dim % DSPARK_CACHE4_GROUP || !pages_ok(pages, page_size) ||
        !exp_ok(k_exp) || !exp_ok(v_exp))
        return false;
    const int es = bytes_of(kv_t), groups = head_dim / DSPARK_CACHE4_GROUP;
    const long long row = (long long)kv_heads * head_dim, rows = (long long)kv_heads * page_size;
    if (k_stride < row || v_stride < row || (k_stride * es) % 16 || (v_stride * es) % 16) return false;
    if (page_stride < rows * (head_dim / 2) || page_stride % 8 || scale_stride < rows * groups) return false;
    if (T > 0 && (!dev(k, 16) || !dev(v, 16) || !dev(slot_map) || !dev(k_cache, 8) || !dev(v_cache, 8) || !dev(k_scale, 1) ||
                  !dev(v_scale, 1) || !dev_or_null(ws, 256)))
        return false;
    // what is written shares no byte with what is read, nor with another result
    const Strided tokens[] = {{k, T, k_stride * es, row * es}, {v, T, v_stride * es, row * es}};
    const Strided cache[] = {{k_cache, pages, page_stride, rows * (head_dim / 2)}, {v_cache, pages, page_stride, rows * (head_dim / 2)},
                             {k_scale, pages, scale_stride, rows * groups}, {v_scale, pages, scale_stride, rows * groups}};
    const Bytes slots{reinterpret_cast<const char*>(slot_map), 4LL * T};
    if (T > 0) {
        for (const Strided& t : tokens)
            for (const Strided& c : cache)
                if (t.meets(c)) return false;
        if (reads && tokens[0].meets(tokens[1])) return false;
        for (int i = 0; !reads && i < 4; ++i)
            for (int j = 0; j < i; ++j)
                if (cache[i].meets(cache[j])) return false;
        for (int i = 0; i < (reads ? 2 : 4); ++i)
            if ((reads ? tokens[i] : cache[i]).meets(slots)) return false;
    }
    p.k = k; p.v = v; p.k_stride = k_stride; p.v_stride = v_stride;
    p.bf16 = kv_t == DSPARK_BF16;
    p.slot_map = slot_map; p.T = T;
    p.k_cache = static_cast<uint8_t*>(const_cast<void*>(k_cache)); p.v_cache = static_cast<uint8_t*>(const_cast<void*>(v_cache));
    p.k_scale = static_cast<uint8_t*>(const_cast<void*>(k_scale)); p.v_scale = static_cast<uint8_t*>(const_cast<void*>(v_scale));
    p.page_bytes = page_stride; p.scale_bytes = scale_stride;
    p.pages = pages; p.page_size = page_size; p.heads = kv_heads; p.groups = groups;
    p.by_page.set((uint32_t)page_size);
    p.by_groups.set((uint32_t)groups);
    p.status = static_cast<uint32_t*>(ws);
    return true;
}

dspark_status dspark_cache_append4(const void* k, const void* v, dspark_dtype kv_t, long long k_stride, long long v_stride,
                                   const int32_t* slot_map, int T, void* k_cache, void* v_cache, void* k_scale,
                                   void* v_scale, long long page_stride, long long scale_stride, int pages, int page_size,
                                   int kv_heads, int head_dim, int k_exp, int v_exp, void* ws, void* stream) {
    const CallRange range_(__func__);
    if (!dtype_ok(kv_t)) return DSPARK_ERR_UNSUPPORTED;
    Cache4Params p;
    if (!cache4_params(p, k_cache, v_cache, k_scale, v_scale, page_stride, scale_stride, pages, page_size, kv_heads, head_dim,
                       k_exp, v_exp, slot_map, T, k, v, kv_t, k_stride, v_stride, ws, false))
        return DSPARK_ERR_INVALID;
    if (T == 0) return DSPARK_OK;
    p.k_by = power(-k_exp);
    p.v_by = power(-v_exp);
    return launch_status(launch_cache_append4(p, static_cast<cudaStream_t>(stream)));
}

dspark_status dspark_cache_read4(const void* k_cache, const void* v_cache, const void* k_scale, const void* v_scale,
                                 long long page_stride, long long scale_stride, int pages, int page_size, int kv_heads,
                                 int head_dim, int k_exp, int v_exp, const int32_t* slot_map, int T, void* k, void* v,
                                 dspark_dtype kv_t, long long k_stride, long long v_stride, void* ws, void* stream) {
    const CallRange range_(__func__);
    if (!dtype_ok(kv_t)) return DSPARK_ERR_UNSUPPORTED;
    Cache4Params p;
    if (!cache4_params(p, k_cache, v_cache, k_scale, v_scale, page_stride, scale_stride, pages, page_size, kv_heads, head_dim,
                       k_exp, v_exp, slot_map, T, k, v, kv_t, k_stride, v_stride, ws, true))
        return DSPARK_ERR_INVALID;
    if (T == 0) return DSPARK_OK;
    p.k_by = power(k_exp);
    p.v_by = power(v_exp);
    return launch_status(launch_cache_read4(p, static_cast<cudaStream_t>(stream)));
}

dspark_status dspark_rope(const void* q, long long q_stride, const void* k, long long k_stride, dspark_dtype t,
                          const int32_t* positions, const uint64_t* turns, int rotary_dim, int interleaved, float mult,
                          void* q_out, long long q_out_stride, void* k_out, long long k_out_stride, int T, int q_heads,
                          int kv_heads, int head_dim, void* stream) {
    const CallRange range_(__func__);
    if (!dtype_ok(t)) return DSPARK_ERR_UNSUPPORTED;
    if (T < 0 || q_heads < 1 || kv_heads < 0 || q_heads > 8192 || kv_heads > 8192 || q_heads + kv_heads > 8192 || !head_ok(head_dim) ||
        rotary_dim < 2 || rotary_dim % 2 || rotary_dim > head_dim || !(fabsf(mult) < INFINITY))
        return DSPARK_ERR_INVALID;
    const int es = bytes_of(t);
    const long long strides[] = {q_stride, q_out_stride, k_stride, k_out_stride};
    for (int i = 0; i < (kv_heads ? 4 : 2); ++i)
        if (strides[i] < (long long)(i < 2 ? q_heads : kv_heads) * head_dim || (strides[i] * es) % 16) return DSPARK_ERR_INVALID;
    if (T == 0) return DSPARK_OK;
    if (!dev(q, 16) || !dev(q_out, 16) || !dev(positions) || !dev(turns, 8)) return DSPARK_ERR_INVALID;
    if (kv_heads && (!dev(k, 16) || !dev(k_out, 16))) return DSPARK_ERR_INVALID;
    // an output is its input (the same rows), or apart from all the others
    auto rows = [&](const void* a, long long stride, int heads) {
        return Bytes{static_cast<const char*>(a), ((T - 1) * stride + (long long)heads * head_dim) * es};
    };
    const int sides = kv_heads ? 2 : 1;
    const void* in[] = {q, k};
    void* out[] = {q_out, k_out};
    const long long in_stride[] = {q_stride, k_stride}, out_stride[] = {q_out_stride, k_out_stride};
    const int heads[] = {q_heads, kv_heads};
    for (int o = 0; o < sides; ++o) {
        const Bytes to = rows(out[o], out_stride[o], heads[o]);
        for (int i = 0; i < sides; ++i) {
            const bool same = i == o && in[i] == out[o] && in_stride[i] == out_stride[o];
            if (!same && rows_meet(to, out_stride[o] * es, heads[o] * head_dim * es, rows(in[i], in_stride[i], heads[i]), in_stride[i] * es,
                                   heads[i] * head_dim * es))
                return DSPARK_ERR_INVALID;
        }
        const Bytes fixed[] = {{reinterpret_cast<const char*>(positions), 4LL * T}, {reinterpret_cast<const char*>(turns), 4LL * rotary_dim}};
        for (const Bytes& f : fixed)
            if (to.meets(f)) return DSPARK_ERR_INVALID;
    }
    if (sides == 2 && rows_meet(rows(q_out, q_out_stride, q_heads), q_out_stride * es, q_heads * head_dim * es,
                                rows(k_out, k_out_stride, kv_heads), k_out_stride * es, kv_heads * head_dim * es))
        return DSPARK_ERR_INVALID;
    RopeParams p;
    p.q = q; p.k = k; p.q_out = q_out; p.k_out = k_out;
    p.q_stride = q_stride; p.k_stride = k_stride; p.q_out_stride = q_out_stride; p.k_out_stride = k_out_stride;
    p.bf16 = t == DSPARK_BF16;
    p.positions = positions; p.turns = reinterpret_cast<const unsigned long long*>(turns);
    p.T = T; p.Hq = q_heads; p.Hkv = kv_heads; p.D = head_dim; p.rotary = rotary_dim; p.interleaved = interleaved != 0;
    p.mult = mult;
    return launch_status(launch_rope(p, static_cast<cudaStream_t>(stream)));
}

size_t dspark_sample_workspace_bytes(int N) { return N < 0 || N > DSPARK_MAX_SAMPLE_ROWS ? 0 : kHead; }

dspark_status dspark_sample(const void* logits, dspark_dtype t, long long row_stride, int N, int V, const float* u,
                            const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                            int32_t* tok, float* logprob, void* ws, size_t ws_bytes, void* stream) {
    const CallRange range_(__func__);
    if (!dtype_ok(t)) return DSPARK_ERR_UNSUPPORTED;
    const size_t need = dspark_sample_workspace_bytes(N);
    if (need == 0 || V < 1 || V > DSPARK_MAX_SAMPLE_VOCAB) return DSPARK_ERR_INVALID;
    if (N > 1 && (row_stride < V || (row_stride * bytes_of(t)) % 16)) return DSPARK_ERR_INVALID;
    if (N == 0) return DSPARK_OK;
    if (!dev(logits, 16) || !dev(u) || !dev_or_null(temperature) || !dev_or_null(top_k) || !dev_or_null(top_p) ||
        !dev_or_null(min_p) || !dev(tok) || !dev_or_null(logprob) || !dev(ws, 256) || ws_bytes < need)
        return DSPARK_ERR_INVALID;
    // rows read their inputs while others write their results
    const long long rows = 4LL * N, all = ((N - 1) * row_stride + V) * bytes_of(t);
    auto bytes = [](const void* a, long long n) { return Bytes{static_cast<const char*>(a), a ? n : 0}; };
    const Bytes out[] = {bytes(tok, rows), bytes(logprob, rows)};
    const Bytes in[] = {bytes(logits, all), bytes(u, rows), bytes(temperature, rows), bytes(top_k, rows), bytes(top_p, rows), bytes(min_p, rows)};
    for (const Bytes& i : in)
        if (i.meets(out[0]) || i.meets(out[1])) return DSPARK_ERR_INVALID;
    if (out[0].meets(out[1])) return DSPARK_ERR_INVALID;
    SampleParams p;
    p.logits = logits; p.row_stride = row_stride; p.bf16 = t == DSPARK_BF16;
    p.N = N; p.V = V;
    p.u = u; p.temperature = temperature; p.top_k = top_k; p.top_p = top_p; p.min_p = min_p;
    p.tok = tok; p.logprob = logprob;
    p.status = static_cast<uint32_t*>(ws);
    return launch_status(launch_sample(p, static_cast<cudaStream_t>(stream)));
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

size_t dspark_cache4_workspace_bytes(int B, int q_heads, int kv_heads, int head_dim, int max_new) {
    const size_t least = dspark_cache_workspace_bytes(B, q_heads, kv_heads, head_dim, max_new);
    if (least == 0 || head_dim % DSPARK_CACHE4_GROUP) return 0;
    // a warp is a worker where registers dequantise; the other kernels' parts are as those of dspark_cache_attention
    const size_t tile = attn4_row_tile(q_heads / kv_heads * max_new, head_dim), workers = (size_t)kMaxAttnCtas * attn4_warps((int)tile / 8, head_dim);
    const size_t need = kHead + ws_align256(sizeof(AttnSplitRow) * workers) + ws_align256(2 * workers * tile * (head_dim + 2) * sizeof(float));
    return need > least ? need : least;
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

dspark_status dspark_cache_attention4(const void* q, long long q_stride, dspark_dtype q_t, const void* k_cache,
                                      const void* v_cache, const void* k_scale, const void* v_scale, long long page_stride,
                                      long long scale_stride, int pages, int page_size, int k_exp, int v_exp,
                                      const int32_t* block_table, int width, const int32_t* kv_len, const int32_t* q_off,
                                      const int32_t* tile_off, int B, int N, int q_heads, int kv_heads, int head_dim,
                                      int max_new, float scale, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    const CallRange range_(__func__);
    if (!dtype_ok(q_t)) return DSPARK_ERR_UNSUPPORTED;
    if (!attn_sizes_ok(B, q_heads, kv_heads, head_dim, max_new) || head_dim % DSPARK_CACHE4_GROUP || N < 0 || width < 1 ||
        !pages_ok(pages, page_size) || (long long)width * page_size > (1LL << 31) - 256 || (long long)N * q_heads >= (1LL << 31) ||
        !exp_ok(k_exp) || !exp_ok(v_exp))
        return DSPARK_ERR_INVALID;
    if (!(scale > 0.f && scale < 3e38f) || !(scale * power(k_exp) > 0.f && scale * power(k_exp) < 3e38f)) return DSPARK_ERR_INVALID;
    const int code_row = head_dim / 2, scale_row = head_dim / DSPARK_CACHE4_GROUP;
    const long long rows_a_page = (long long)kv_heads * page_size;
    if (page_stride < rows_a_page * code_row || page_stride % row_align(code_row) || scale_stride < rows_a_page * scale_row ||
        scale_stride % row_align(scale_row) || q_stride < (long long)q_heads * head_dim || (q_stride * bytes_of(q_t)) % 16)
        return DSPARK_ERR_INVALID;
    if (N == 0) return DSPARK_OK;
    if (!dev(q, 16) || !dev(k_cache, row_align(code_row)) || !dev(v_cache, row_align(code_row)) || !dev(k_scale, row_align(scale_row)) ||
        !dev(v_scale, row_align(scale_row)) || !dev(block_table) || !dev(kv_len) || !dev(q_off) || !dev(tile_off) || !dev(out, 16) ||
        !dev_or_null(lse) || !dev(ws, 256))
        return DSPARK_ERR_INVALID;
    const size_t need = dspark_cache4_workspace_bytes(B, q_heads, kv_heads, head_dim, max_new);
    if (ws_bytes < need) return DSPARK_ERR_INVALID;
    // CTAs write their rows while others read theirs
    const long long es = bytes_of(q_t), q_row = (long long)q_heads * head_dim * es;
    const Strided in[] = {{q, N, q_stride * es, q_row}, {k_cache, pages, page_stride, rows_a_page * code_row}, {v_cache, pages, page_stride, rows_a_page * code_row},
                          {k_scale, pages, scale_stride, rows_a_page * scale_row}, {v_scale, pages, scale_stride, rows_a_page * scale_row}};
    auto bytes = [](const void* a, long long n) { return Bytes{static_cast<const char*>(a), a ? n : 0}; };
    const Bytes lists[] = {bytes(block_table, 4LL * B * width), bytes(kv_len, 4LL * B), bytes(q_off, 4LL * (B + 1)), bytes(tile_off, 4LL * (B + 1)), bytes(ws, (long long)need)};
    const Bytes results[] = {bytes(out, N * q_row), bytes(lse, 4LL * N * q_heads)};
    if (results[0].meets(results[1])) return DSPARK_ERR_INVALID;
    for (const Bytes& r : results) {
        for (const Strided& i : in)
            if (i.meets(r)) return DSPARK_ERR_INVALID;
        for (const Bytes& i : lists)
            if (i.meets(r)) return DSPARK_ERR_INVALID;
    }
    AttnParams p;
    p.q = q; p.q_stride = q_stride; p.k = k_cache; p.v = v_cache; p.page_stride = page_stride;
    p.ks = static_cast<const uint8_t*>(k_scale); p.vs = static_cast<const uint8_t*>(v_scale); p.scale_stride = scale_stride;
    p.out_by = power(v_exp);
    p.bf16 = q_t == DSPARK_BF16;
    p.table = block_table; p.width = width;
    p.kv_len = kv_len; p.q_off = q_off; p.tile_off = tile_off;
    p.B = B; p.N = N; p.Hq = q_heads; p.Hkv = kv_heads; p.G = q_heads / kv_heads; p.D = head_dim;
    p.pages = pages; p.page_size = page_size; p.max_new = max_new;
    p.scale = scale * power(k_exp); p.out = out; p.lse = lse;
    p.by_page.set((uint32_t)page_size);
    p.by_group.set((uint32_t)p.G);
    const int rows = p.G * max_new;
    const bool tensor = p.bf16 && attn4_tensor(p, rows);
    p.row_tile = tensor ? 64 : p.bf16 ? attn4_row_tile(rows, head_dim) : attn_row_tile(rows, false);
    const long long tiles = ((long long)width * page_size + kTile - 1) / kTile * B * kv_heads;
    if (!p.bf16 && tiles * ((rows + p.row_tile - 1) / p.row_tile) < 2LL * num_sms()) p.row_tile = 8;
    p.row_tiles = (rows + p.row_tile - 1) / p.row_tile;
    p.ctas = num_sms() < kMaxAttnCtas ? num_sms() : kMaxAttnCtas;      // one resident CTA per SM
    if (p.bf16 && !tensor) p.ctas *= attn4_warps(p.row_tile / 8, head_dim);
    p.pad = tensor ? 4 : 1;
    p.spare = p.bf16;
    p.split = reinterpret_cast<AttnSplitRow*>(static_cast<char*>(ws) + kHead);
    p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kHead + ws_align256(sizeof(AttnSplitRow) * p.ctas));
    p.status = static_cast<uint32_t*>(ws);
    return launch_status(launch_cache_attention4(p, tensor, static_cast<cudaStream_t>(stream)));
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
