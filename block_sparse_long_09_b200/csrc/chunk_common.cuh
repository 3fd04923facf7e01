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
// The tiles are shared out to the workers (a CTA or a CTA pair) from the lengths on the device
// alone: a batch of any mix of lengths is balanced and a captured launch stays valid as
// the caches grow.  Two ways:
//   even    the tiles of all items, in item order, in equal shares; a share may end one item and
//           begin another (a restart costs as much as kRestart tiles: its loads, Q and the epilogue)
//   apart   no more than one item per worker, workers dealt to the items by their tiles: less even, for
//           batches whose shares are a few tiles
// An item that one worker has whole is finished there.  A cut item is attended in pieces whose
// normalised outputs and log-sum-exps (base 2) the merge kernel adds up: the piece that begins the
// item goes to slot 2 c + 1 of its worker c, any later piece to slot 2 c (a worker has at
// most one of each).
#pragma once
#include "kernels.cuh"

namespace qsa {

namespace {

constexpr int kHQ = 24, kHKV = 2, kD = 256, kGrp = kHQ / kHKV;

struct ChunkGroup {
    int s;            // sequence
    int nq;           // tokens, 0: an empty slot
    int row0;         // first packed query row
    int t0;           // position of the first token (may be negative: no visible key)
    int nt;           // key tiles
    int ns;           // leading tiles that hold the first tokens (sinks)
    int w_tile;       // tile index (of kKeys) of the first window tile
};

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

// what a group follows from
struct ChunkDims {
    const int32_t *q, *k;
    int batch, total_q, window, sinks;

    __device__ __forceinline__ explicit ChunkDims(const ChunkArgs &a, const ChunkLengths *sh = nullptr)
        : q(a.cu_q), k(a.cu_k), batch(a.batch), total_q((int)a.total_q), window((int)a.window), sinks((int)a.sinks)
    {
        if (sh != nullptr && batch <= kCuBatch) {
            q = sh->q;
            k = sh->k;
        }
    }
};

// (lengths and positions are int32, rows fewer than 2^28, sequences fewer than 2^28)
template <int kTok, int kKeys>
__device__ __forceinline__ ChunkGroup chunk_group_inline(const ChunkDims &a, int slot)
{
    ChunkGroup g;
    g.nt = g.ns = g.nq = 0;
    g.w_tile = g.row0 = g.t0 = 0;
    int lo = 0, hi = a.batch;  // the last s whose first slot is <= slot
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.q[mid] / kTok + mid <= slot) lo = mid; else hi = mid;
    }
    g.s = lo;
    const int q0 = a.q[lo], q1 = a.q[lo + 1];
    const int first = (slot - (q0 / kTok + lo)) * kTok, Lq = q1 - q0;
    if (q0 < 0 || first < 0 || first >= Lq) return g;
    if (q1 > a.total_q) {  // lengths that the query tensor does not hold
        set_device_status(QSA_ERR_DEVICE_CHECK);
        return g;
    }
    g.nq = Lq - first < kTok ? Lq - first : kTok;
    g.row0 = q0 + first;
    g.t0 = a.k[lo + 1] - a.k[lo] - Lq + first;
    const int last = g.t0 + g.nq - 1;
    if (last < 0) return g;
    const int t_first = g.t0 > 0 ? g.t0 : 0;
    const int w0 = a.window > 0 && t_first >= a.window ? t_first - a.window + 1 : 0;
    const int sinks = a.sinks < w0 ? a.sinks : w0;
    const int end = last / kKeys + 1;
    int ns = sinks / kKeys + (sinks % kKeys != 0 ? 1 : 0), w = w0 / kKeys;
    if (ns >= w) ns = w = 0;  // the sinks reach the window's first tile: one range from 0
    g.ns = ns;
    g.w_tile = w;
    g.nt = ns + end - w;
    return g;
}

// One copy for the work list's several passes: the first fetches of their instructions took 1 us of a
// small call.
template <int kTok, int kKeys>
static __device__ __noinline__ ChunkGroup chunk_group(ChunkDims a, int slot)
{
    return chunk_group_inline<kTok, kKeys>(a, slot);
}

// the group slots of a call (a host bound and the device's range)
template <int kTok>
__host__ __device__ __forceinline__ int64_t chunk_slots(int64_t total_q, int batch)
{
    return total_q / kTok + batch;
}

struct ChunkShare {
    int64_t ts, te;       // this worker's tiles [ts, te) of the call's
    int64_t first;        // first tile of the group slot that holds ts
    int slot;             // that slot
    ChunkGroup g;         // and its group
};

// x / y of numbers that mostly fit 32 bits
__device__ __forceinline__ int64_t divide(int64_t x, int64_t y)
{
    return (x | y) < ((int64_t)1 << 32) ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

// first tile of share c (even)
__device__ __forceinline__ int64_t share_start(int64_t c, int64_t total, int64_t workers) { return divide(c * total, workers); }

struct ChunkTotals {
    int64_t tiles, items;
    bool apart;
};
template <int kRestart>
__device__ __forceinline__ ChunkTotals chunk_totals(int64_t tiles, int64_t items, int64_t workers)
{
    return ChunkTotals{tiles, items, items <= workers && (tiles <= workers ||
                       tiles * items < kRestart * workers * (workers - items))};
}

// workers of an item of nt tiles (apart): at most one per tile, all items' together at most `workers`
__device__ __forceinline__ int item_workers(int nt, const ChunkTotals &t, int64_t workers)
{
    if (nt == 0) return 0;
    const int64_t n = 1 + divide(nt * (workers - t.items), t.tiles);
    return n < nt ? (int)n : nt;
}

// sums over the CTA's threads of x and y; before: over the threads before this one.  `scan`: two entries per warp
template <int kThreads>
__device__ __forceinline__ void block_scan(int64_t x, int64_t y, int64_t *scan, int64_t &x_before, int64_t &y_before,
                                           int64_t &x_all, int64_t &y_all)
{
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t xi = x, yi = y;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, xi, off), v = __shfl_up_sync(0xffffffffu, yi, off);
        if (lane >= off) {
            xi += u;
            yi += v;
        }
    }
    __syncthreads();  // an earlier scan has been read
    if (lane == 31) {
        scan[warp] = xi;
        scan[kWarps + warp] = yi;
    }
    __syncthreads();
    x_before = xi - x;
    y_before = yi - y;
    x_all = y_all = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            x_before += scan[w];
            y_before += scan[kWarps + w];
        }
        x_all += scan[w];
        y_all += scan[kWarps + w];
    }
}

// an item's share of worker j of its n
__device__ __forceinline__ void share_apart(ChunkShare *out, int slot, int64_t first, int64_t nt, int hd, int64_t j, int n)
{
    out->slot = slot;
    out->first = first;
    out->ts = first + hd * nt + divide(j * nt, n);
    out->te = first + hd * nt + divide((j + 1) * nt, n);
}

// the shares that hold an item's first and last tile (even)
__device__ __forceinline__ int2 even_pieces(int64_t at, int64_t nt, int64_t total, int64_t workers)
{
    if (nt == 0) return make_int2(0, -1);
    return make_int2((int)divide((at + 1) * workers - 1, total), (int)divide((at + nt) * workers - 1, total));
}

// The same for up to 32 slots, by the first warp alone, without barriers between the steps (these and the
// scans over the CTA took 3 us of a small call).
template <int kTok, int kKeys, int kRestart>
__device__ __forceinline__ void chunk_share_warp(const ChunkArgs &a, int64_t worker, int64_t workers, ChunkShare *out,
                                                 int2 *pieces, const ChunkDims &dims, int slots)
{
    const int u = threadIdx.x;
    const int64_t nt = u < slots ? chunk_group<kTok, kKeys>(dims, u).nt : 0;
    int64_t incl = kHKV * nt;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
        if (u >= off) incl += x;
    }
    const int64_t total = __shfl_sync(0xffffffffu, incl, 31), before = incl - kHKV * nt;
    const int items = kHKV * __popc(__ballot_sync(0xffffffffu, nt > 0));
    if (u == 0) out->ts = out->te = out->first = out->slot = 0;
    __syncwarp();
    int2 p0 = make_int2(0, -1), p1 = p0;
    bool holds = false;
    if (total > 0) {  // uniform
        const ChunkTotals t = chunk_totals<kRestart>(total, items, workers);
        if (t.apart) {
            const int n = item_workers((int)nt, t, workers);
            int at = kHKV * n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, at, off);
                if (u >= off) at += x;
            }
            at -= kHKV * n;
            p0 = make_int2(at, at + n - 1);
            p1 = make_int2(at + n, at + 2 * n - 1);
            holds = at <= worker && worker < at + kHKV * n;
            if (holds) {
                const int hd = worker - at >= n ? 1 : 0;
                share_apart(out, u, before, nt, hd, worker - at - hd * n, n);
            }
        } else {
            const int64_t ts = share_start(worker, total, workers), te = share_start(worker + 1, total, workers);
            p0 = even_pieces(before, nt, total, workers);
            p1 = even_pieces(before + nt, nt, total, workers);
            holds = ts < te && before <= ts && ts < incl;
            if (holds) {
                out->slot = u;
                out->first = before;
                out->ts = ts;
                out->te = te;
            }
        }
    }
    if (pieces != nullptr && u < slots) {
        pieces[2 * u] = p0;
        pieces[2 * u + 1] = p1;
    }
    if (holds) out->g = chunk_group<kTok, kKeys>(dims, u);
}

// This worker's share, by the whole CTA (whole warps); `scan`: two shared entries per warp.  `pieces`
// (worker 0's CTA, or null): every item's first and last worker, for the merge; none: 0, -1.
template <int kTok, int kKeys, int kThreads, int kRestart>
__device__ __forceinline__ void chunk_share(const ChunkArgs &a, int64_t worker, int64_t workers, ChunkShare *out,
                                            int64_t *scan, int2 *pieces, const ChunkLengths *sh)
{
    const int slots = (int)chunk_slots<kTok>(a.total_q, a.batch);
    const ChunkDims dims(a, sh);
    if (slots <= 32) {
        if (threadIdx.x < 32) chunk_share_warp<kTok, kKeys, kRestart>(a, worker, workers, out, pieces, dims, slots);
        __syncthreads();
        return;
    }
    const int per = (slots + kThreads - 1) / kThreads;  // consecutive slots of a thread
    const int u0 = (int)threadIdx.x * per < slots ? (int)threadIdx.x * per : slots, u1 = u0 + per < slots ? u0 + per : slots;
    int64_t mine = 0, items = 0;
    int one = 0;  // the tiles of a thread's only slot
    auto tiles_of = [&](int u) -> int { return per == 1 ? one : chunk_group<kTok, kKeys>(dims, u).nt; };
    for (int u = u0; u < u1; ++u) {
        const int nt = chunk_group<kTok, kKeys>(dims, u).nt;
        one = nt;
        mine += kHKV * (int64_t)nt;
        items += nt > 0 ? kHKV : 0;
    }
    if (threadIdx.x == 0) out->ts = out->te = out->first = out->slot = 0;
    int64_t before, items_before, total, all;
    block_scan<kThreads>(mine, items, scan, before, items_before, total, all);
    if (total == 0) {
        if (pieces != nullptr)
            for (int u = u0; u < u1; ++u) pieces[2 * u] = pieces[2 * u + 1] = make_int2(0, -1);
        __syncthreads();
        return;
    }
    const ChunkTotals t = chunk_totals<kRestart>(total, all, workers);
    if (t.apart) {
        int64_t wanted = 0, at_w, unused, all_w, unused_all;
        for (int u = u0; u < u1; ++u) wanted += kHKV * item_workers(tiles_of(u), t, workers);
        block_scan<kThreads>(wanted, 0, scan, at_w, unused, all_w, unused_all);
        const bool holds = at_w <= worker && worker < at_w + wanted;
        if (holds || pieces != nullptr) {
            int64_t at = before;
            for (int u = u0; u < u1; ++u) {
                const int nt = tiles_of(u), n = item_workers(nt, t, workers);
                if (pieces != nullptr) {
                    pieces[2 * u] = make_int2((int)at_w, (int)at_w + n - 1);
                    pieces[2 * u + 1] = make_int2((int)at_w + n, (int)at_w + 2 * n - 1);
                }
                if (at_w <= worker && worker < at_w + kHKV * n) {
                    const int hd = worker - at_w >= n ? 1 : 0;
                    const int64_t j = worker - at_w - hd * n;
                    share_apart(out, u, at, nt, hd, j, n);
                    out->g = chunk_group<kTok, kKeys>(dims, u);
                }
                at += kHKV * (int64_t)nt;
                at_w += kHKV * n;
            }
        }
    } else {
        const int64_t ts = share_start(worker, total, workers), te = share_start(worker + 1, total, workers);
        const bool holds = ts < te && before <= ts && ts < before + mine;
        if (holds || pieces != nullptr) {
            int64_t at = before;
            for (int u = u0; u < u1; ++u) {
                const int64_t nt = tiles_of(u);
                if (pieces != nullptr)
                    for (int hd = 0; hd < kHKV; ++hd) pieces[2 * u + hd] = even_pieces(at + hd * nt, nt, total, workers);
                if (holds && at <= ts && ts < at + kHKV * nt) {
                    out->slot = u;
                    out->first = at;
                    out->ts = ts;
                    out->te = te;
                    out->g = chunk_group<kTok, kKeys>(dims, u);
                }
                at += kHKV * nt;
            }
        }
    }
    __syncthreads();
}

constexpr int kMergeScan = 32;  // group slots that the first merge's CTAs scan, at most
constexpr int kMergeWarps = 8, kMergeThreads = kMergeWarps * 32;
static_assert(kMergeThreads == kD, "a thread per dim");

// Merge of the pieces of the cut items, and the rows of items without any visible key.  For few
// rows: a CTA per row, its eight warps over the row's pieces.  Where the item's tiles lie is worked out
// from the lengths while the attention kernel still runs (that one was scheduled after everything
// before it had completed); only then the CTA waits for it.
template <int kTok, int kKeys, int kRestart>
__global__ void __launch_bounds__(kMergeThreads)
chunk_merge_kernel(const ChunkArgs a, int64_t workers)
{
    constexpr int kRows = kTok * kGrp, kAhead = 4;
    __shared__ float part[kMergeWarps][kD + 2];
    __shared__ int64_t scan[2 * kMergeWarps];
    const int slot = blockIdx.x >> 1, slots = (int)chunk_slots<kTok>(a.total_q, a.batch);
    const int hd = blockIdx.x & 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t tiles = 0, items = 0, p0 = 0, unused, total, all, before;
    const ChunkDims dims(a);
    const ChunkGroup g = chunk_group<kTok, kKeys>(dims, slot);
    if (blockIdx.y >= g.nq * kGrp) {  // uniform for the CTA: no such row, before the scan over all slots
        pdl_enter();
        return;
    }
    for (int u = threadIdx.x; u < slots; u += kMergeThreads) {
        const int64_t nt = chunk_group<kTok, kKeys>(dims, u).nt;
        tiles += kHKV * nt;
        items += nt > 0 ? kHKV : 0;
        if (u < slot) p0 += kHKV * nt;
    }
    block_scan<kMergeThreads>(tiles, items, scan, unused, unused, total, all);
    block_scan<kMergeThreads>(p0, 0, scan, unused, unused, before, unused);
    int64_t c0 = 0, last = -1;
    if (g.nt > 0) {
        const ChunkTotals t = chunk_totals<kRestart>(total, all, workers);
        if (t.apart) {
            int64_t wanted = 0, at_w;
            for (int u = threadIdx.x; u < slot; u += kMergeThreads)
                wanted += kHKV * item_workers(chunk_group<kTok, kKeys>(dims, u).nt, t, workers);
            block_scan<kMergeThreads>(wanted, 0, scan, unused, unused, at_w, unused);
            const int n = item_workers(g.nt, t, workers);
            c0 = at_w + hd * n;
            last = c0 + n - 1;
        } else {
            const int64_t rs = before + hd * (int64_t)g.nt;
            c0 = divide((rs + 1) * workers - 1, total);
            last = divide((rs + g.nt) * workers - 1, total);
        }
    }
    const int rows = g.nq * kGrp;
    pdl_enter();
    if (g.nt > 0 && last == c0) return;  // uniform for the CTA: finished by one worker
    const float *lse = a.ws + 2 * workers * kRows * kD;
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        float mx = -INFINITY, sum = 0.f, acc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
        // pieces: slot 2 c0 + 1, then slot 2 c of every worker c > c0 that holds tiles of the item
        for (int64_t cb = c0 + warp; cb <= last; cb += kMergeWarps * kAhead) {
            float w[kAhead], x[kAhead][8];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int64_t c = cb + u * kMergeWarps;
                const bool have = c <= last;
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

// The same for many rows and few pieces each: a warp per kPer rows, with the items' workers as the
// attention kernel leaves them.
template <int kTok, int kKeys, int kPer>
__global__ void __launch_bounds__(kMergeThreads)
chunk_merge_many_kernel(const ChunkArgs a, const int2 *__restrict__ pieces, int64_t workers)
{
    constexpr int kRows = kTok * kGrp;
    pdl_enter();
    const int slot = blockIdx.x >> 1;
    const int hd = blockIdx.x & 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int2 range = pieces[blockIdx.x];
    const int64_t c0 = range.x, last = range.y;
    if (c0 == last) return;  // finished by one worker
    const ChunkGroup g = chunk_group<kTok, kKeys>(ChunkDims(a), slot);
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

template <int kTok, int kKeys, int kRestart>
cudaError_t launch_chunk_merge(const ChunkArgs &a, const int2 *pieces, int64_t workers, cudaStream_t stream)
{
    constexpr int kRows = kTok * kGrp;
    const int64_t items = 2 * chunk_slots<kTok>(a.total_q, a.batch);
    if (items > 0x7FFFFFFF) return cudaErrorInvalidValue;
    // Items that are cut into eight pieces or more: a CTA per row, its eight warps over the row's pieces
    // (one sequence of 8191 cached tokens: 4 us less); otherwise a warp per four rows, whose lookups
    // cost less (batch 64 of decoded tokens: 20 us less).  A few tokens in a batch that is mostly empty go the
    // second way too: the CTAs of the first each scan all group slots (four tokens, e4m3, 1000 cached
    // ones each, 22 and 22 us among 16 sequences, 27 and 25 us among 64, 103 and 47 us among 1024).
    const int64_t groups = a.total_q / kTok, some = a.batch < a.total_q ? a.batch : a.total_q;
    if (16 * (groups > some ? groups : some) <= workers && items <= 2 * kMergeScan) {
        const int64_t most = a.max_len_q < kTok ? (a.max_len_q > 0 ? a.max_len_q : 1) : kTok;
        return launch_pdl(chunk_merge_kernel<kTok, kKeys, kRestart>, dim3((unsigned)items, (unsigned)(most * kGrp)),
                          dim3(kMergeThreads), 0, stream, a, workers);
    }
    constexpr int kPer = 4, kBlock = kMergeWarps * kPer;
    return launch_pdl(chunk_merge_many_kernel<kTok, kKeys, kPer>, dim3((unsigned)items, (kRows + kBlock - 1) / kBlock),
                      dim3(kMergeThreads), 0, stream, a, pieces, workers);
}

}  // namespace

}  // namespace qsa
