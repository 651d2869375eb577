// cache.cu -- the paged key-value cache beside the verification: the plan of
// a step (which pages each request owns, where its new tokens go) and the
// append of new keys and values.
#include "pdl.cuh"
#include "serve.cuh"

namespace dspark {
namespace {

// ------------------------------------------------------------------- plan
// For request b with len_b positions in the cache and new_b tokens to come:
//     goal_b = ceil((len_b + new_b) / P)    pages it needs,
//     need_b = max(0, goal_b - owned_b)     taken from the front of the ring,
//     give_b = max(0, owned_b - goal_b)     put back at its end,
// and every place follows from exclusive sums over b of new_b, need_b, give_b
// and the attention tiles.  The pages taken are ring[head + i], the pages
// returned go to ring[head + free + i]: the two ranges never meet, since the
// ring has room for every page, so one launch does both and the same inputs
// always give the same outputs.
//
// A few kilobytes are read and written, so latency bounds it.  Each CTA forms
// the sums over all requests itself (B <= 4096 lengths, a few loads a thread)
// instead of waiting for another launch, and then fills its share of the slot
// map, the table entries and the ring entries.  64 requests 4.8 us, 512
// requests with 135168 slots 6.2 us (0.9 and 1.1 more with a second scan, for the
// rare case that the ring runs out, in every call; 0.5 more with sums that
// notice a carry instead of stopping by a minimum).
constexpr int kPlanThreads = 1024;

struct Sum4 { unsigned tok, need, give, tiles; };

// Terms and sums stop at 2^31 - 1 (two of them do not wrap 32 bits).  A sum that
// stops is still the same in any order of its terms, but its terms cannot be
// taken off again: exclusive sums are formed without subtracting.
__device__ __forceinline__ unsigned add_sat(unsigned a, unsigned b) { return min(a + b, 0x7fffffffu); }
__device__ __forceinline__ Sum4 operator+(const Sum4& a, const Sum4& b) {
    return Sum4{add_sat(a.tok, b.tok), add_sat(a.need, b.need), add_sat(a.give, b.give), add_sat(a.tiles, b.tiles)};
}
__device__ __forceinline__ Sum4 shfl_up(const Sum4& a, int d) {
    return Sum4{__shfl_up_sync(~0u, a.tok, d), __shfl_up_sync(~0u, a.need, d), __shfl_up_sync(~0u, a.give, d),
                __shfl_up_sync(~0u, a.tiles, d)};
}

struct PlanItem {
    int fresh;     // new tokens, none where their number is out of [0, width * page_size]
    int need;      // pages it asks for (0 where it cannot be served)
    int goal;
    int owned;
    int seq;
    bool ok;       // lengths in range and table wide enough
};

__device__ __forceinline__ PlanItem plan_item(const PlanParams& p, int b) {
    PlanItem it;
    it.seq = p.seq_len[b];
    it.fresh = p.n_new[b];
    it.owned = p.owned[b];
    const bool fresh_ok = it.fresh >= 0 && it.fresh <= p.width * p.page_size;     // (below 2^31)
    if (!fresh_ok) it.fresh = 0;
    it.ok = fresh_ok && it.seq >= 0 && it.owned >= 0 && it.owned <= p.width;
    const long long goal = ((long long)it.seq + it.fresh + p.page_size - 1) / p.page_size;
    it.ok = it.ok && goal <= p.width;
    it.goal = it.ok ? (int)goal : it.owned;
    it.need = it.ok ? max(0, it.goal - it.owned) : 0;
    return it;
}

// the b in [0, B) with off[b] <= x < off[b + 1], where off[0] = 0 and x < off[B]
__device__ __forceinline__ int owner_of(const unsigned* off, int B, unsigned x) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const PlanParams p) {
    extern __shared__ unsigned sm[];
    unsigned* s_q = sm;                      // [B + 1] exclusive sums of the new tokens
    unsigned* s_need = s_q + p.B + 1;        // [B + 1] of the pages asked for
    unsigned* s_give = s_need + p.B + 1;     // [B + 1] of the pages returned
    __shared__ Sum4 s_warp[32];
    __shared__ unsigned s_popped;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = p.B;
    grid_dependency_wait();
    int head = p.ring_state[0], avail = p.ring_state[1];
    bool bad = false;
    bool state_ok = head >= 0 && head < p.pages && avail >= 0 && avail <= p.pages;
    if (!state_ok) { head = 0; avail = 0; }

    const int per = (B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    auto block_scan = [&](Sum4 v) {     // exclusive over the threads
        Sum4 x = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Sum4 y = shfl_up(x, d);
            if (lane >= d) x = x + y;
        }
        if (lane == 31) s_warp[warp] = x;
        Sum4 before = shfl_up(x, 1);
        if (lane == 0) before = Sum4{0u, 0u, 0u, 0u};
        __syncthreads();
        if (warp == 0) {
            Sum4 z = s_warp[lane];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const Sum4 y = shfl_up(z, d);
                if (lane >= d) z = z + y;
            }
            z = shfl_up(z, 1);
            s_warp[lane] = lane == 0 ? Sum4{0u, 0u, 0u, 0u} : z;
        }
        __syncthreads();
        before = s_warp[warp] + before;
        __syncthreads();
        return before;
    };
    // a thread's requests; up to 1024 of them stay in registers
    PlanItem one{};
    if (b0 < b1) one = plan_item(p, b0);
    auto item = [&](int b) { return b == b0 ? one : plan_item(p, b); };
    auto give_of = [](const PlanItem& it) { return (unsigned)max(0, it.owned - it.goal); };
    auto tiles_of = [](const PlanItem& it) { return ((unsigned)it.seq + it.fresh + kTile - 1) / kTile; };
    auto served_at = [&](const PlanItem& it, unsigned need) {     // `need` pages asked for before it
        return it.ok && (it.need == 0 || need + it.need <= (unsigned)avail);
    };
    // sums as if every request could be served (usually so)
    Sum4 mine{0u, 0u, 0u, 0u};
    for (int b = b0; b < b1; ++b) {
        const PlanItem it = item(b);
        mine = mine + Sum4{(unsigned)it.fresh, (unsigned)it.need, it.ok ? give_of(it) : 0u, it.ok ? tiles_of(it) : 0u};
    }
    Sum4 at = block_scan(mine);
    if (tid == kPlanThreads - 1) s_popped = add_sat(at.need, mine.need);
    __syncthreads();
    Sum4 at2 = at;
    if (s_popped > (unsigned)avail) {
        // requests are served in order while the ring has pages for them
        __syncthreads();
        if (tid == 0) s_popped = 0;
        __syncthreads();
        Sum4 second{0u, 0u, 0u, 0u};
        unsigned need = at.need;
        for (int b = b0; b < b1; ++b) {
            const PlanItem it = item(b);
            const bool served = served_at(it, need);
            need = add_sat(need, it.need);
            if (served) {
                second = second + Sum4{0u, 0u, give_of(it), tiles_of(it)};
                if (it.need) atomicAdd(&s_popped, (unsigned)it.need);     // an integer sum: any order gives the same
            }
        }
        at2 = block_scan(second);
    }
    {
        unsigned tok = at.tok, need = at.need, give = at2.give, tiles = at2.tiles;
        for (int b = b0; b < b1; ++b) {
            const PlanItem it = item(b);
            const bool served = served_at(it, need);
            bad |= !served;
            s_q[b] = tok; s_need[b] = need; s_give[b] = give;
            if (blockIdx.x == 0) {
                p.owned_out[b] = served ? it.goal : it.owned;
                p.kv_len[b] = served ? it.seq + it.fresh : 0;
                p.q_off[b] = (int)tok;
                p.tile_off[b] = (int)tiles;
            }
            tok = add_sat(tok, it.fresh);
            need = add_sat(need, it.need);
            if (served) {
                give = add_sat(give, give_of(it));
                tiles = add_sat(tiles, tiles_of(it));
            }
            if (b == B - 1) {
                s_q[B] = tok; s_need[B] = need; s_give[B] = give;
                if (blockIdx.x == 0) { p.q_off[B] = (int)tok; p.tile_off[B] = (int)tiles; }
            }
        }
    }
    __syncthreads();
    const unsigned popped = s_popped, given = s_give[B], tokens = s_q[B];
    if (blockIdx.x == 0) {
        if (bad) raise_status(p.status, kBadPage);
        if (tid == 0) {
            p.ring_state_out[0] = (int)(((long long)head + popped) % p.pages);
            p.ring_state_out[1] = (int)add_sat((unsigned)avail - popped, given);
            if (!state_ok) raise_status(p.status, kBadPage);
            if (tokens > (unsigned)p.T) raise_status(p.status, kBadLength);
        }
    }
    auto ring_at = [&](long long i) { return (int)(((long long)head + i) % p.pages); };
    const unsigned g0 = blockIdx.x * kPlanThreads + tid, gs = gridDim.x * kPlanThreads;
    // the pages that change hands
    for (unsigned g = g0; g < popped; g += gs) {
        const int b = owner_of(s_need, B, g);
        const int j = (int)(p.owned[b] + (g - s_need[b]));
        if (j >= 0 && j < p.width) p.table[(size_t)b * p.width + j] = p.ring[ring_at(g)];
    }
    for (unsigned g = g0; g < given; g += gs) {
        const int b = owner_of(s_give, B, g);
        const PlanItem it = plan_item(p, b);
        const int j = (int)(it.goal + (g - s_give[b]));
        if (j >= 0 && j < it.owned) p.ring[ring_at((long long)avail + g)] = p.table[(size_t)b * p.width + j];
    }
    // the slot of every new token; a page taken in this call is read from the
    // ring, since another CTA may not have written the table yet
    for (unsigned t = g0; t < (unsigned)p.T; t += gs) {
        int slot = -1, pos = -1;
        if (t < tokens) {
            const int b = owner_of(s_q, B, t);
            const PlanItem it = plan_item(p, b);
            const unsigned i = t - s_q[b];           // below it.fresh
            pos = (int)(it.seq + i);                 // (of a served request below 2^31)
            if (i < (unsigned)it.fresh && served_at(it, s_need[b])) {
                const int j = pos / p.page_size;
                const int page = j < it.owned ? p.table[(size_t)b * p.width + j]
                                              : p.ring[ring_at((long long)s_need[b] + j - it.owned)];
                if (page >= 0 && page < p.pages) slot = page * p.page_size + (pos - j * p.page_size);
                else raise_status(p.status, kBadPage);
            }
        }
        p.slot_map[t] = slot;
        p.positions[t] = pos;
    }
}

// ----------------------------------------------------------------- append
// cache[slot] = row: a copy, bound by HBM for prompts and by latency for a
// block.  A thread keeps one 16-byte place of a token's row (its head and
// place follow once) and moves it for kAppend tokens at a time, keys and
// values: the loads do not wait for the slots.  512 tokens of 4 KB 1.8 us, 32768
// 42.2 us (6.4 TB/s, read and written).
constexpr int kAppendThreads = 256, kAppend = 2;

__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendParams p, int group) {
    // `group` threads to a token, several tokens to a block
    grid_dependency_wait();
    const int vecs = p.row_bytes / 16, per = p.heads * vecs;
    const int side = kAppendThreads / group, lt = threadIdx.x / group, e0 = threadIdx.x - lt * group;
    if (lt >= side) return;
    for (int e = e0; e < per; e += group) {
        const int h = e / vecs;
        const long long in_page = (long long)h * p.page_size * p.row_bytes + 16 * (e - h * vecs);
        const long long step = (long long)gridDim.x * side;
        for (long long t0 = (long long)blockIdx.x * side + lt; t0 < p.T; t0 += step * kAppend) {
            int slot[kAppend];
            uint4 k[kAppend], v[kAppend];
#pragma unroll
            for (int u = 0; u < kAppend; ++u) {
                const long long t = t0 + u * step;
                slot[u] = -1;
                if (t < p.T) {
                    slot[u] = __ldg(p.slot_map + t);
                    k[u] = __ldcs(reinterpret_cast<const uint4*>(p.k + t * p.k_stride) + e);
                    v[u] = __ldcs(reinterpret_cast<const uint4*>(p.v + t * p.v_stride) + e);
                }
            }
#pragma unroll
            for (int u = 0; u < kAppend; ++u) {
                if (slot[u] < 0) continue;
                const int page = slot[u] / p.page_size, row = slot[u] - page * p.page_size;
                if (page >= p.pages) { raise_status(p.status, kBadPage); continue; }
                const long long o = page * p.page_bytes + in_page + (long long)row * p.row_bytes;
                *reinterpret_cast<uint4*>(p.k_cache + o) = k[u];
                *reinterpret_cast<uint4*>(p.v_cache + o) = v[u];
            }
        }
    }
}

}  // namespace

cudaError_t launch_cache_plan(const PlanParams& p, cudaStream_t s) {
    const size_t smem = sizeof(int) * 3 * ((size_t)p.B + 1);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(cache_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const int items = p.T > p.B ? p.T : p.B;
    int grid = (items + kPlanThreads - 1) / kPlanThreads;
    if (grid > num_sms()) grid = num_sms();
    return launch_dependent(cache_plan_kernel, dim3(grid), dim3(kPlanThreads), smem, s, p);
}

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    const int per = p.heads * (p.row_bytes / 16), group = per < kAppendThreads ? per : kAppendThreads;
    const int side = kAppendThreads / group;
    // one pass of the tokens, kAppend to a thread, over as many blocks as there are
    // (up to 64 per SM: 42.0 us for 32768 tokens of 4 KB, 43.9 with 8)
    const long long blocks = ((long long)p.T + side - 1) / side;
    long long grid = (blocks + kAppend - 1) / kAppend;
    if (grid < num_sms()) grid = blocks < num_sms() ? blocks : num_sms();
    if (grid > 64LL * num_sms()) grid = 64LL * num_sms();
    return launch_dependent(cache_append_kernel, dim3((unsigned)grid), dim3(kAppendThreads), 0, s, p, group);
}

}  // namespace dspark
