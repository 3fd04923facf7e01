// chunk_common.cuh -- the work list of the chunk attention over a paged cache, shared by
// its kernels and their merge.
//
// A group is up to kTok new tokens of one sequence (12 kTok rows of a KV head's queries), an
// item a group with one KV head.  Sequence s owns the group slots from
// floor(cu_q[s] / kTok) + s on: one more than its whole groups, so the slot of a group
// follows from cu_q alone, without a prefix sum, and total_q / kTok + batch slots hold
// every batch (those without tokens are empty).
//
// A group's visible keys are [0, min(sinks, w0)) and [w0, t_last], w0 = the first position
// inside its first token's window, cut into tiles of kKeys aligned at multiples of kKeys.
// The tiles of all items, in item order, are cut into equal shares, one per worker (a
// CTA or a CTA pair), from the lengths on the device alone: a batch of any mix of lengths is
// balanced and a captured launch stays valid as the caches grow.  An item inside one share
// is finished there.  A cut item is attended in pieces whose normalised outputs and
// log-sum-exps (base 2) the merge kernel adds up: the piece that begins the item goes to
// slot 2 c + 1 of its share c, any later piece to slot 2 c (a share has at most one of
// each).
#pragma once
#include "kernels.cuh"

namespace qsa {

namespace {

constexpr int kHQ = 24, kHKV = 2, kD = 256, kGrp = kHQ / kHKV;

struct ChunkGroup {
    int s;            // sequence
    int nq;           // tokens, 0: an empty slot
    int64_t row0;     // first packed query row
    int64_t t0;       // position of the first token (may be negative: no visible key)
    int nt;           // key tiles
    int ns;           // leading tiles that hold the first tokens (sinks)
    int64_t w_tile;   // tile index (of kKeys) of the first window tile
};

// first key tile after the sinks, etc.: tile i of the group starts at position
__device__ __forceinline__ int64_t tile_start(const ChunkGroup &g, int i, int keys)
{
    return (i < g.ns ? (int64_t)i : g.w_tile + (i - g.ns)) * keys;
}

template <int kTok, int kKeys>
__device__ __forceinline__ ChunkGroup chunk_group(const ChunkArgs &a, int64_t slot)
{
    ChunkGroup g;
    g.nt = g.ns = g.nq = 0;
    g.w_tile = g.row0 = g.t0 = 0;
    int lo = 0, hi = a.batch;  // the last s whose first slot is <= slot
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)(__ldg(a.cu_q + mid) / kTok) + mid <= slot) lo = mid; else hi = mid;
    }
    g.s = lo;
    const int64_t q0 = __ldg(a.cu_q + lo), q1 = __ldg(a.cu_q + lo + 1);
    const int64_t first = (slot - (q0 / kTok + lo)) * kTok, Lq = q1 - q0;
    if (q0 < 0 || first < 0 || first >= Lq) return g;
    if (q1 > a.total_q) {  // lengths that the query tensor does not hold
        set_device_status(QSA_ERR_DEVICE_CHECK);
        return g;
    }
    const int64_t Lk = (int64_t)__ldg(a.cu_k + lo + 1) - __ldg(a.cu_k + lo);
    g.nq = (int)(Lq - first < kTok ? Lq - first : kTok);
    g.row0 = q0 + first;
    g.t0 = Lk - Lq + first;
    const int64_t last = g.t0 + g.nq - 1;
    if (last < 0) return g;
    const int64_t t_first = g.t0 > 0 ? g.t0 : 0;
    const int64_t w0 = a.window > 0 && t_first - a.window + 1 > 0 ? t_first - a.window + 1 : 0;
    const int64_t sinks = a.sinks < w0 ? a.sinks : w0;
    const int64_t end = last / kKeys + 1;
    int64_t ns = (sinks + kKeys - 1) / kKeys, w = w0 / kKeys;
    if (ns >= w) ns = w = 0;  // the sinks reach the window's first tile: one range from 0
    g.ns = (int)ns;
    g.w_tile = w;
    g.nt = (int)(ns + end - w);
    return g;
}

// the group slots of a call (a host bound and the device's range)
template <int kTok>
__host__ __device__ __forceinline__ int64_t chunk_slots(int64_t total_q, int batch)
{
    return total_q / kTok + batch;
}

struct ChunkShare {
    int64_t ts, te;       // this worker's tiles [ts, te) of the call's
    int64_t slot, first;  // the group slot that holds ts and that slot's first tile
};

// first tile of share c
__device__ __forceinline__ int64_t share_start(int64_t c, int64_t total, int64_t workers) { return c * total / workers; }

// This worker's share, by the whole CTA (threads a power of two of whole warps); `scan`: a
// shared array of one entry per warp.  `prefix` (worker 0's CTA, or null): the first tile
// of every slot and, behind them, the total, for the merge.
template <int kTok, int kKeys, int kThreads>
__device__ __forceinline__ void chunk_share(const ChunkArgs &a, int64_t worker, int64_t workers, ChunkShare *out,
                                            int64_t *scan, int64_t *prefix)
{
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t slots = chunk_slots<kTok>(a.total_q, a.batch);
    const int64_t per = (slots + kThreads - 1) / kThreads;  // consecutive slots of a thread
    const int64_t u0 = tid * per < slots ? tid * per : slots, u1 = u0 + per < slots ? u0 + per : slots;
    int64_t mine = 0;
    for (int64_t u = u0; u < u1; ++u) mine += kHKV * (int64_t)chunk_group<kTok, kKeys>(a, u).nt;
    int64_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    const int64_t ts = share_start(worker, total, workers), te = share_start(worker + 1, total, workers);
    if (tid == 0) {
        out->ts = ts;
        out->te = te;
        out->slot = slots;
        out->first = total;
    }
    __syncthreads();
    const bool holds = ts < te && before <= ts && ts < before + mine;
    if (holds || prefix != nullptr) {
        int64_t at = before;
        for (int64_t u = u0; u < u1; ++u) {
            const int64_t n = kHKV * (int64_t)chunk_group<kTok, kKeys>(a, u).nt;
            if (prefix != nullptr) prefix[u] = at;
            if (holds && at <= ts && ts < at + n) {
                out->slot = u;
                out->first = at;
            }
            at += n;
        }
    }
    if (prefix != nullptr && tid == 0) prefix[slots] = total;
    __syncthreads();
}

// does position t see key j <= t
__device__ __forceinline__ bool chunk_sees(int64_t t, int64_t j, int64_t window, int64_t sinks)
{
    return j <= t && (window <= 0 || t - j < window || j < sinks);
}

// the pool row of position j of sequence s, -1 (flagged) when the table has no valid page
__device__ __forceinline__ int64_t chunk_pool_row(const CachePool &c, int64_t s, int64_t j)
{
    const int64_t p = j / c.page_size;
    const int32_t page = p < c.max_pages ? __ldg(c.table + s * c.max_pages + p) : -1;
    if (page < 0 || page >= c.num_pages) {
        set_device_status(QSA_ERR_DEVICE_CHECK);
        return -1;
    }
    return (int64_t)page * c.page_size + j % c.page_size;
}

}  // namespace

}  // namespace qsa
