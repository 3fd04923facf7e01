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

// A batch's lengths in shared memory (up to kCuBatch sequences), for the searches of every role and item.
constexpr int kCuBatch = 128;
struct ChunkLengths {
    int32_t q[kCuBatch + 1], k[kCuBatch + 1];

    __device__ __forceinline__ void fill(const ChunkArgs &a)  // by the whole CTA
    {
        if (a.batch <= kCuBatch)
            for (int i = threadIdx.x; i <= a.batch; i += blockDim.x) {
                q[i] = __ldg(a.cu_q + i);
                k[i] = __ldg(a.cu_k + i);
            }
        __syncthreads();
    }
};

template <int kTok, int kKeys>
__device__ __forceinline__ ChunkGroup chunk_group(const ChunkArgs &a, int64_t slot, const ChunkLengths *sh = nullptr)
{
    const bool local = sh != nullptr && a.batch <= kCuBatch;
    auto cu_q = [&](int i) -> int32_t { return local ? sh->q[i] : __ldg(a.cu_q + i); };
    auto cu_k = [&](int i) -> int32_t { return local ? sh->k[i] : __ldg(a.cu_k + i); };
    ChunkGroup g;
    g.nt = g.ns = g.nq = 0;
    g.w_tile = g.row0 = g.t0 = 0;
    int lo = 0, hi = a.batch;  // the last s whose first slot is <= slot
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)(cu_q(mid) / kTok) + mid <= slot) lo = mid; else hi = mid;
    }
    g.s = lo;
    const int64_t q0 = cu_q(lo), q1 = cu_q(lo + 1);
    const int64_t first = (slot - (q0 / kTok + lo)) * kTok, Lq = q1 - q0;
    if (q0 < 0 || first < 0 || first >= Lq) return g;
    if (q1 > a.total_q) {  // lengths that the query tensor does not hold
        set_device_status(QSA_ERR_DEVICE_CHECK);
        return g;
    }
    const int64_t Lk = (int64_t)cu_k(lo + 1) - cu_k(lo);
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
__device__ __forceinline__ int64_t share_start(int64_t c, int64_t total, int64_t workers)
{
    const int64_t x = c * total;
    return x < ((int64_t)1 << 32) ? (int64_t)((uint32_t)x / (uint32_t)workers) : x / workers;
}

// This worker's share, by the whole CTA (threads a power of two of whole warps); `scan`: a
// shared array of one entry per warp.  `prefix` (worker 0's CTA, or null): the first tile
// of every slot and, behind them, the total, for the merge.
template <int kTok, int kKeys, int kThreads>
__device__ __forceinline__ void chunk_share(const ChunkArgs &a, int64_t worker, int64_t workers, ChunkShare *out,
                                            int64_t *scan, int64_t *prefix, const ChunkLengths *sh)
{
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t slots = chunk_slots<kTok>(a.total_q, a.batch);
    const int64_t per = (slots + kThreads - 1) / kThreads;  // consecutive slots of a thread
    const int64_t u0 = tid * per < slots ? tid * per : slots, u1 = u0 + per < slots ? u0 + per : slots;
    int64_t mine = 0;
    for (int64_t u = u0; u < u1; ++u) mine += kHKV * (int64_t)chunk_group<kTok, kKeys>(a, u, sh).nt;
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
            const int64_t n = kHKV * (int64_t)chunk_group<kTok, kKeys>(a, u, sh).nt;
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
    uint32_t off;
    const uint32_t p = c.page_of((uint32_t)j, &off);
    const int32_t page = p < (uint32_t)c.max_pages ? __ldg(c.table + s * c.max_pages + p) : -1;
    if (page < 0 || page >= c.num_pages) {
        set_device_status(QSA_ERR_DEVICE_CHECK);
        return -1;
    }
    return (int64_t)page * c.page_size + off;
}

constexpr int kMergeWarps = 8, kMergeThreads = kMergeWarps * 32;
static_assert(kMergeThreads == kD, "a thread per dim");

// Merge of the pieces of the cut items, and the rows of items without any visible key.  For few
// rows: a CTA per row, its eight warps over the row's pieces.  Where the item's tiles lie is worked out
// from the lengths while the attention kernel still runs (that one was scheduled after everything
// before it had completed); only then the CTA waits for it.
template <int kTok, int kKeys>
__global__ void __launch_bounds__(kMergeThreads)
chunk_merge_kernel(const ChunkArgs a, int64_t workers)
{
    constexpr int kRows = kTok * kGrp, kAhead = 4;
    __shared__ float part[kMergeWarps][kD + 2];
    __shared__ int64_t sums[2][kMergeWarps];
    const int slot = blockIdx.x >> 1, slots = (int)chunk_slots<kTok>(a.total_q, a.batch);
    const int hd = blockIdx.x & 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t before = 0, all = 0;
    for (int u = threadIdx.x; u < slots; u += kMergeThreads) {
        const int64_t n = 2 * (int64_t)chunk_group<kTok, kKeys>(a, u).nt;
        all += n;
        if (u < slot) before += n;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, off);
        before += __shfl_xor_sync(0xffffffffu, before, off);
    }
    if (lane == 0) {
        sums[0][warp] = all;
        sums[1][warp] = before;
    }
    const ChunkGroup g = chunk_group<kTok, kKeys>(a, slot);
    __syncthreads();
    int64_t total = 0, p0 = 0;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
        total += sums[0][w];
        p0 += sums[1][w];
    }
    const int64_t rs = p0 + hd * (int64_t)g.nt, re = rs + g.nt;
    int64_t c0 = 0, last = -1;
    const int rows = g.nq * kGrp;
    bool mine = blockIdx.y < rows;
    if (g.nt > 0) {
        c0 = ((rs + 1) * workers - 1) / total;                                // the share that holds the item's first tile
        if (share_start(c0 + 1, total, workers) >= re) mine = false;          // finished by one worker
        last = (re * workers - 1) / total;                                    // and its last one
    }
    pdl_enter();
    if (!mine) return;  // uniform for the CTA
    const float *lse = a.ws + 2 * workers * kRows * kD;
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        float mx = -INFINITY, sum = 0.f, acc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
        // pieces: slot 2 c0 + 1, then slot 2 c of every share c > c0 that holds tiles of the item
        for (int64_t cb = c0 + warp; cb <= last; cb += kMergeWarps * kAhead) {
            float w[kAhead], x[kAhead][8];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int64_t c = cb + u * kMergeWarps;
                const bool have = c <= last && (c == c0 || share_start(c + 1, total, workers) > share_start(c, total, workers));
                const int64_t p = c == c0 ? 2 * c0 + 1 : 2 * c;
                w[u] = -INFINITY;
#pragma unroll
                for (int j = 0; j < 8; ++j) x[u][j] = 0.f;
                if (have) {
                    w[u] = lse[p * kRows + r];
                    const float4 *src = reinterpret_cast<const float4 *>(a.ws + (p * kRows + r) * kD + lane * 8);
                    *reinterpret_cast<float4 *>(&x[u][0]) = __ldcs(src);
                    *reinterpret_cast<float4 *>(&x[u][4]) = __ldcs(src + 1);
                }
            }
            float m = mx;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) m = fmaxf(m, w[u]);
            const float base = m == -INFINITY ? 0.f : m;  // nothing visible (or only NaNs, which stay)
            const float f = exp2f(mx - base);
            mx = m;
            sum *= f;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] *= f;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const float e = exp2f(w[u] - base);
                sum += e;
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] = fmaf(e, x[u][j], acc[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) part[warp][lane * 8 + j] = acc[j];
        if (lane == 0) {
            part[warp][kD] = sum;
            part[warp][kD + 1] = mx;
        }
        __syncthreads();
        const int d = threadIdx.x;  // kMergeThreads = kD: a dim each
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) top = fmaxf(top, part[w][kD + 1]);
        const float base = top == -INFINITY ? 0.f : top;
        float L = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
            const float f = exp2f(part[w][kD + 1] - base);
            L = fmaf(f, part[w][kD], L);
            o = fmaf(f, part[w][d], o);
        }
        const bool none = L == 0.f;
        const int64_t row = (g.row0 + r / kGrp) * kHQ + hd * kGrp + r % kGrp;
        a.o[row * kD + d] = __float2bfloat16_rn(none ? 0.f : o / L);
        if (a.lse != nullptr && d == 0) a.lse[row] = none ? -INFINITY : (top + log2f(L)) * 0.6931471805599453f;
        __syncthreads();  // the next row overwrites the parts
    }
}

// The same for many rows and few pieces each: a warp per kPer rows, with the tiles' prefix that the
// attention kernel leaves.
template <int kTok, int kKeys, int kPer>
__global__ void __launch_bounds__(kMergeThreads)
chunk_merge_many_kernel(const ChunkArgs a, const int64_t *__restrict__ prefix, int64_t workers)
{
    constexpr int kRows = kTok * kGrp;
    pdl_enter();
    const int64_t slot = blockIdx.x >> 1;
    const int hd = blockIdx.x & 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t slots = chunk_slots<kTok>(a.total_q, a.batch);
    const int64_t total = prefix[slots], p0 = prefix[slot], p1 = prefix[slot + 1];
    const int64_t nt = (p1 - p0) >> 1, rs = p0 + hd * nt, re = rs + nt;
    int64_t c0 = 0, last = -1;
    if (nt > 0) {
        c0 = ((rs + 1) * workers - 1) / total;  // the share that holds the item's first tile
        if (share_start(c0 + 1, total, workers) >= re) return;  // finished by one worker
        last = (re * workers - 1) / total;      // and its last one
    }
    const ChunkGroup g = chunk_group<kTok, kKeys>(a, slot);
    const int rows = g.nq * kGrp, r0 = (blockIdx.y * kMergeWarps + warp) * kPer;
    if (r0 >= rows) return;
    const float *lse = a.ws + 2 * workers * kRows * kD;
    float mx[kPer], sum[kPer], acc[kPer][8];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        mx[u] = -INFINITY;
        sum[u] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[u][j] = 0.f;
    }
    for (int64_t c = c0; c <= last; ++c) {
        if (c != c0 && share_start(c + 1, total, workers) == share_start(c, total, workers)) continue;  // an empty share
        const int64_t p = c == c0 ? 2 * c0 + 1 : 2 * c;
        float w[kPer], x[kPer][8];
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int64_t at = p * kRows + (r0 + u < rows ? r0 + u : r0);
            w[u] = lse[at];
            const float4 *src = reinterpret_cast<const float4 *>(a.ws + at * kD + lane * 8);
            *reinterpret_cast<float4 *>(&x[u][0]) = __ldcs(src);
            *reinterpret_cast<float4 *>(&x[u][4]) = __ldcs(src + 1);
        }
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const float m = fmaxf(mx[u], w[u]), base = m == -INFINITY ? 0.f : m;
            const float f = exp2f(mx[u] - base), e = exp2f(w[u] - base);
            mx[u] = m;
            sum[u] = fmaf(sum[u], f, e);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[u][j] = fmaf(acc[u][j], f, e * x[u][j]);
        }
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int r = r0 + u;
        if (r >= rows) break;
        const bool none = sum[u] == 0.f;
        const float inv = none ? 0.f : 1.f / sum[u];
        const int64_t row = (g.row0 + r / kGrp) * kHQ + hd * kGrp + r % kGrp;
        __nv_bfloat162 h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            h[j] = __floats2bfloat162_rn(none ? 0.f : acc[u][2 * j] * inv, none ? 0.f : acc[u][2 * j + 1] * inv);
        *reinterpret_cast<uint4 *>(a.o + row * kD + lane * 8) = *reinterpret_cast<const uint4 *>(h);
        if (a.lse != nullptr && lane == 0) a.lse[row] = none ? -INFINITY : (mx[u] + log2f(sum[u])) * 0.6931471805599453f;
    }
}

template <int kTok, int kKeys>
cudaError_t launch_chunk_merge(const ChunkArgs &a, const int64_t *prefix, int64_t workers, cudaStream_t stream)
{
    constexpr int kRows = kTok * kGrp;
    const int64_t items = 2 * chunk_slots<kTok>(a.total_q, a.batch);
    if (items > 0x7FFFFFFF) return cudaErrorInvalidValue;
    // Items that are cut into eight pieces or more: a CTA per row, its eight warps over the row's pieces
    // (one sequence of 8191 cached tokens: 4 us less); otherwise a warp per four rows, whose lookups
    // cost less (batch 64 of decoded tokens: 20 us less).
    const int64_t groups = a.total_q / kTok, some = a.batch < a.total_q ? a.batch : a.total_q;
    if (16 * (groups > some ? groups : some) <= workers) {
        const int64_t most = a.max_len_q < kTok ? (a.max_len_q > 0 ? a.max_len_q : 1) : kTok;
        return launch_pdl(chunk_merge_kernel<kTok, kKeys>, dim3((unsigned)items, (unsigned)(most * kGrp)),
                          dim3(kMergeThreads), 0, stream, a, workers);
    }
    constexpr int kPer = 4, kBlock = kMergeWarps * kPer;
    return launch_pdl(chunk_merge_many_kernel<kTok, kKeys, kPer>, dim3((unsigned)items, (kRows + kBlock - 1) / kBlock),
                      dim3(kMergeThreads), 0, stream, a, prefix, workers);
}

}  // namespace

}  // namespace qsa
