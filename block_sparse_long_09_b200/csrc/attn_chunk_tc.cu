// attn_chunk_tc.cu -- attention of the new tokens of every sequence over its paged cache,
// tensor-core kernel: up to 21 new tokens (252 rows of a KV head's queries) per item, or up to 10.
//
//   S = Q K^T,  P = exp2(c2 S - m),  O = P V,  o = O / rowsum(P)       c2 = scale log2(e)
//
// A pair of CTAs (cta_group::2) works on an item: 256 rows, 128 per CTA, against tiles of 128 keys.
// The twelve heads of a KV head fill the rows, so that every key read serves 252 rows and the
// causal edge of a chunk wastes 21 keys at most; each CTA holds half of every K tile (64 keys)
// and of every V tile (128 of the 256 dims), so that a pair reads each key once.
//   S: M 256 N 128 K 256, Q and K from shared memory, two buffers of 128 TMEM columns
//   O: M 256 N 256 K 128, P from TMEM (the first half of its S buffer, as bf16), V from shared
//      memory; 256 TMEM columns, so the 512 columns of an SM are full
// S(i + 1) is issued before O += P(i) V(i), and overwrites P(i - 1) behind the product that reads it (one
// thread's products run in order): the tensor cores run it while the softmax of tile i is done, whose 128 exponentials per row (1024 cycles of an SM's exp2 units)
// take half of the 2048 cycles of the tile's two products.
// With at most 10 new tokens per sequence a CTA works alone (kCtas = 1): 128 rows, tiles of 64 keys.
// The rows are mostly empty then and what counts is how fast keys are read: 148 CTAs that read
// different keys instead of 74 pairs (four tokens each over 32 caches of 32768, bf16: 342 us, 6.3 TB/s,
// 97 % of the copy rate; e4m3 394 us against a pair's 515).  A single CTA is the faster one up to its ten tokens in
// every case measured: 2, 4, 8 and 10 tokens over 1, 4, 16 and 32 caches of 1000, 8192 and 32768, by 7 to 26 % in
// bf16 and 10 to 35 % in e4m3.
// Measured: 1024 new tokens over 16384, 1.38 PFLOP/s bf16, 1.10 e4m3; 2048 over 65536, bf16, 2.8 ms,
// 1.17 PFLOP/s under the power cap (84 % of the sustained product rate).  A tile takes 2450 cycles in
// bf16, bound by the chain S -> softmax -> O of 2300; 2900 in e4m3, where the softmax shares its
// schedulers with the conversion (ten operations per four codes).
//   warp 0       Q, once per item (TMA)
//   warp 1       CTA 0: issues the products of both CTAs; CTA 1: passes on to CTA 0 that its Q and
//                slots are full.  The fence between the slots' writers and the tensor cores stands
//                here: in a writer it would wait for the copies that are still on their way
//   warps 2, 3   bf16 pools: K and V half tiles into a ring of five 32 KB slots, by 16-byte
//                asynchronous copies: pages of any size, and zeros for keys that no row of the
//                item sees.  (TMA gathers of four rows by index took 75 cycles per 512 bytes.)
//                e4m3 pools: the pool rows and scales of the tiles' keys, into a ring of tables
//   warps 4..7   softmax, a thread per row; running maxima move (and O is rescaled) only when a
//                row's maximum grows by more than 2^8
//   warps 8..15  (e4m3 pools) codes to bf16 in registers, exactly, times the row's scale; then to one of
//                four slots
// Work is shared out and cut items are merged as chunk_common.cuh describes.  Every wait is bounded.
#include <cuda_fp16.h>

#include <mutex>

#include "chunk_common.cuh"

namespace qsa {

namespace {

constexpr int kTcSlot = 32768, kTcMaxStages = 5, kTcTables = 4;
constexpr int kTcQ = 128 * kD * 2;
constexpr int kTcQChunk = 128 * 128, kTcKChunk = 64 * 128;
constexpr uint32_t kTcO = 256, kTcCols = 512;
constexpr float kTcRescale = 8.f;
constexpr int64_t kTcMaxPairs = 80, kTcMaxSingles = 160;

struct TcShared {
    uint64_t kv_full[kTcMaxStages], kv_peer[kTcMaxStages], kv_empty[kTcMaxStages];
    uint64_t q_full, q_peer, q_empty;
    uint64_t s_full[2], p_full[2];
    uint64_t pv_done, o_full, o_empty, drained;
    uint64_t tab_full[kTcTables], tab_empty[kTcTables];
    uint32_t tmem_base;
    int abort_flag;
    int64_t scan[32], walk[16][3];
    ChunkShare share;
    ChunkLengths lengths;
};

template <int kCtas>
struct TcTable {  // e4m3: pool rows (of the KV head, -1: none) and scale bytes of a tile's keys
    int32_t row[kTcTables][64 * kCtas];
    uint8_t ks[kTcTables][64 * kCtas], vs[kTcTables][64 * kCtas];
};

template <bool kFp8, int kCtas>
struct TcCfg {
    static constexpr int kTok = kCtas == 2 ? 21 : 10, kRows = kTok * kGrp, kKeys = 64 * kCtas;
    static constexpr int kRestart = kCtas == 2 ? 8 : 16;  // tiles that another item on a worker costs (11 us)
    static constexpr int kVChunks = 4 / kCtas, kVChunk = kKeys * 128;  // 64 dims of a V tile
    static constexpr int kThreads = kFp8 ? 512 : 256;
    static constexpr int kStages = kFp8 ? 4 : 5;
    static constexpr int kFills = kFp8 ? 8 : 64;  // arrivals that fill a slot: warps that convert, threads that copy
    static constexpr int kOffRing = kTcQ;
    static constexpr int kOffTable = kOffRing + kStages * kTcSlot;
    static constexpr int kOffShared = kOffTable + (kFp8 ? (int)sizeof(TcTable<kCtas>) : 0);
    static constexpr int kSmem = kOffShared + (int)sizeof(TcShared) + 1024;
    static_assert(kSmem <= 232448, "shared memory of one CTA");
};

__device__ __forceinline__ uint32_t cta_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// arrive on the barrier at the same place in CTA 0 of the pair
__device__ __forceinline__ void arrive_leader(uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .b32 r;\n\t"
        "mapa.shared::cluster.u32 r, %0, 0;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [r];\n\t}"
        ::"r"(smem_u32(bar)) : "memory");
}

// the same without a release: for what tcgen05 fences order (a release at the cluster's scope waits for
// the thread's global stores)
__device__ __forceinline__ void arrive_leader_relaxed(uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .b32 r;\n\t"
        "mapa.shared::cluster.u32 r, %0, 0;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [r];\n\t}"
        ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
        : "memory");
    return ok != 0;
}

// bounded wait for arrivals from either CTA of the pair
static __device__ __noinline__ bool wait_pair_slow(uint64_t *bar, uint32_t parity, volatile int *abort_flag)
{
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (try_wait_cluster(bar, parity)) return true;
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > QSA_WAIT_LIMIT_NS) {
            set_device_status(QSA_ERR_TIMEOUT);
            *abort_flag = 1;
            return false;
        }
    }
}

__device__ __forceinline__ bool wait_pair(uint64_t *bar, uint32_t parity, volatile int *abort_flag)
{
    if (try_wait_cluster(bar, parity)) return true;
    return wait_pair_slow(bar, parity, abort_flag);
}

// 16 bytes global -> shared, zeros unless `have`
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool have)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}

// D (+)= A B^T over the item's CTAs, A from shared memory or from TMEM
template <int kCtas>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if (kCtas == 1) {
        mma_bf16_ss(d, a, b, idesc, accumulate);
        return;
    }
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

template <int kCtas>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if (kCtas == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
            ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
            ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

// arrive on the barrier of the item's CTAs once this thread's tcgen05 operations have completed
template <int kCtas>
__device__ __forceinline__ void commit_all(uint64_t *bar)
{
    if (kCtas == 1) {
        mma_commit(bar);
        return;
    }
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
        " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
          "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// 16 columns times f
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float *v, float f)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
        " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "f"(v[0] * f), "f"(v[1] * f), "f"(v[2] * f), "f"(v[3] * f), "f"(v[4] * f), "f"(v[5] * f),
          "f"(v[6] * f), "f"(v[7] * f), "f"(v[8] * f), "f"(v[9] * f), "f"(v[10] * f), "f"(v[11] * f),
          "f"(v[12] * f), "f"(v[13] * f), "f"(v[14] * f), "f"(v[15] * f)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// two fp32 values at a time
__device__ __forceinline__ uint64_t pack2(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// lane 4 x + q of every four lanes gives its v[j] to lane 4 x + j, which holds it as v[q]
__device__ __forceinline__ void transpose4(uint4 (&v)[4], int lane)
{
    auto swap = [&](uint4 &a, uint4 &b, int bit) {  // the lane with the bit sends a, the other b
        const bool up = (lane & bit) != 0;
        uint4 s = up ? a : b, r;
        r.x = __shfl_xor_sync(0xffffffffu, s.x, bit);
        r.y = __shfl_xor_sync(0xffffffffu, s.y, bit);
        r.z = __shfl_xor_sync(0xffffffffu, s.z, bit);
        r.w = __shfl_xor_sync(0xffffffffu, s.w, bit);
        if (up) a = r; else b = r;
    };
    swap(v[0], v[1], 1);
    swap(v[2], v[3], 1);
    swap(v[0], v[2], 2);
    swap(v[1], v[3], 2);
}

// The items of a share, in order: every role walks the same list.
// kCached: the first item's group as the share has it (e4m3: computed anew, the kernel's 128 registers fall
// in a better order then, 3 % of a chunk).
template <int kTok, int kKeys, bool kCached>
struct TcWalk {
    const TcShared *sh;
    int64_t *state;  // shared memory, of this warp: next tile, its group's slot and that slot's first tile
    // the current item
    int s, nq, nt, ns, w_tile;  // as in its ChunkGroup
    int row0, t0;
    int hd, i0, i1;
    int t_first, t_last;  // positions of the first (at least 0) and the last token
    int near, sinks;      // some row sees the keys near .. t_last and those below sinks
    const int32_t *table; // the sequence's row of the block table

    __device__ __forceinline__ TcWalk(const TcShared *shared, int64_t *st) : sh(shared), state(st)
    {
        if ((threadIdx.x & 31) == 0) {
            st[0] = sh->share.ts;
            st[1] = sh->share.slot;
            st[2] = sh->share.first;
        }
        __syncwarp();
    }

    // The next item, by all 32 lanes together (kWarp) or by one lane that walks for its warp.  All lanes have
    // read the state before it is written, wherever they came from (a role may leave a divergent branch
    // right before), and it is written before any of them reads it again.
    template <bool kWarp>
    __device__ __forceinline__ bool next(const ChunkArgs &a)
    {
        if (kWarp) __syncwarp();
        int64_t at = state[0], first = state[2];
        int slot = (int)state[1];
        const int64_t te = sh->share.te;
        if (at >= te) return false;
        ChunkGroup g = kCached && slot == sh->share.slot ? sh->share.g
                                                         : chunk_group_inline<kTok, kKeys>(ChunkDims(a, &sh->lengths), slot);
        while (at >= first + 2 * (int64_t)g.nt) {  // empty slots between two groups
            first += 2 * (int64_t)g.nt;
            g = chunk_group_inline<kTok, kKeys>(ChunkDims(a, &sh->lengths), ++slot);
        }
        hd = at >= first + g.nt ? 1 : 0;
        const int64_t item = first + (int64_t)hd * g.nt;
        i0 = (int)(at - item);
        i1 = te - item < g.nt ? (int)(te - item) : g.nt;
        s = g.s;
        nq = g.nq;
        nt = g.nt;
        ns = g.ns;
        w_tile = g.w_tile;
        row0 = g.row0;
        t0 = g.t0;
        t_first = t0 > 0 ? t0 : 0;
        t_last = t0 + nq - 1;
        near = a.window > 0 ? t_first - (int)a.window + 1 : 0;
        sinks = (int)a.sinks;
        table = a.pool.table + (int64_t)s * a.pool.max_pages;
        if (kWarp) __syncwarp();
        if (!kWarp || (threadIdx.x & 31) == 0) {
            state[0] = item + i1;
            state[1] = slot;
            state[2] = first;
        }
        if (kWarp) __syncwarp();
        return true;
    }

    // first key of tile i
    __device__ __forceinline__ int tile(int i) const { return (i < ns ? i : w_tile + (i - ns)) * kKeys; }

    // does any row of the item see key j
    __device__ __forceinline__ bool any_sees(int j) const
    {
        return j <= t_last && (j >= near || j < sinks);
    }

    // A key's place in the pool, in two steps, so that the page's load is not waited for: its page
    // (kUnseen: no row of the item sees the key, kNoPage: not in the table) and its row there.
    static constexpr int32_t kUnseen = -2, kNoPage = -1;
    __device__ __forceinline__ int32_t page_of(const ChunkArgs &a, int i, int key, uint32_t *off) const
    {
        if (i >= i1) return kUnseen;
        const int j = tile(i) + key;
        if (!any_sees(j)) return kUnseen;
        const uint32_t p = a.pool.page_of((uint32_t)j, off);
        return p < (uint32_t)a.pool.max_pages ? __ldg(table + p) : kNoPage;
    }
    // the row of this KV head, -1: none
    __device__ __forceinline__ int32_t row_of(const ChunkArgs &a, int32_t page, uint32_t off) const
    {
        if (page == kUnseen) return -1;
        if ((uint32_t)page >= (uint32_t)a.pool.num_pages) {
            set_device_status(QSA_ERR_DEVICE_CHECK);
            return -1;
        }
        return ((int32_t)page * a.pool.page_size + (int32_t)off) * kHKV + hd;  // (a pool has fewer than 2^31 rows)
    }
};

// 16 e4m3 codes -> 16 bf16 values times their row's scale, in a slot.  By the conversion instructions, which
// give NaN for the type's NaN codes (shifts and masks take them for 480; with a test for them beside the shifts
// the calls below took 12 % longer).  fp16, fp32 and bf16 hold a code exactly, and times a power of two too.  The
// scale goes to the fp32 values in a pair (four prompts' chunks 289 against 297 us as bf16 products), to the bf16
// ones in a single CTA (four tokens over 32 caches 418 against 465 us as fp32 products).
template <int kCtas>
__device__ __forceinline__ void codes_to_slot(const uint4 &codes, float scale, uint32_t row_addr, uint32_t unit, uint32_t sw)
{
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    const uint64_t s2 = pack2(scale, scale);
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t h;
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %1;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
            : "=r"(h) : "r"(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        if (kCtas == 2) {
            const float2 x = unpack2(mul2(pack2(f.x, f.y), s2));
            const __nv_bfloat162 r = __floats2bfloat162_rn(x.x, x.y);
            o[i] = *reinterpret_cast<const uint32_t *>(&r);
        } else {
            const __nv_bfloat162 r = __hmul2(__floats2bfloat162_rn(f.x, f.y), __float2bfloat162_rn(scale));
            o[i] = *reinterpret_cast<const uint32_t *>(&r);
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                     ::"r"(row_addr + (((unit + h) ^ sw) << 4)), "r"(o[4 * h]), "r"(o[4 * h + 1]), "r"(o[4 * h + 2]),
                       "r"(o[4 * h + 3])
                     : "memory");
}

template <bool kFp8, int kCtas>
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__((TcCfg<kFp8, kCtas>::kThreads), 1)
chunk_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_q4,
                const ChunkArgs a, int2 *__restrict__ pieces)
{
    using C = TcCfg<kFp8, kCtas>;
    constexpr int kKeys = C::kKeys;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem, *ring = smem + C::kOffRing;
    TcShared *sh = reinterpret_cast<TcShared *>(smem + C::kOffShared);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    const int64_t worker = blockIdx.x / kCtas, workers = gridDim.x / kCtas;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&sh->kv_full[i], C::kFills);
            mbar_init(&sh->kv_peer[i], 1);
            mbar_init(&sh->kv_empty[i], 1);
        }
        mbar_init(&sh->q_full, 1);
        mbar_init(&sh->q_peer, 1);
        mbar_init(&sh->q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->s_full[i], 1);
            mbar_init(&sh->p_full[i], 4 * kCtas);
        }
        mbar_init(&sh->pv_done, 1);
        mbar_init(&sh->drained, 1);
        mbar_init(&sh->o_full, 1);
        mbar_init(&sh->o_empty, 4 * kCtas);
        for (int i = 0; i < kTcTables; ++i) {
            mbar_init(&sh->tab_full[i], 2);
            mbar_init(&sh->tab_empty[i], 8);
        }
        sh->abort_flag = 0;
        fence_barrier_init();
    }
    pdl_enter();  // before the allocation: no CTA waits while it holds tensor memory
    if (warp == 1) {
        if (kCtas == 1) {
            tmem_alloc(&sh->tmem_base, kTcCols);
            tmem_relinquish();
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                         ::"r"(smem_u32(&sh->tmem_base)), "r"(kTcCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
    }
    sh->lengths.fill(a);
    chunk_share<C::kTok, kKeys, C::kThreads, C::kRestart>(a, worker, workers, &sh->share, sh->scan,
                                                          blockIdx.x == 0 ? pieces : nullptr, &sh->lengths);
    tc_fence_before();
    __syncthreads();
    if (kCtas == 2) cluster_sync();  // both CTAs' barriers are initialised
    tc_fence_after();
    const uint32_t tmem = sh->tmem_base;
    volatile int *abort_flag = &sh->abort_flag;
    TcWalk<C::kTok, kKeys, !kFp8> it(sh, sh->walk[warp]);
    bool ok = true;
    if (warp == 0) {
        // ---------------- Q ----------------
        uint32_t n = 0;
        while (ok && it.next<true>(a)) {
            ok = mbar_wait(&sh->q_empty, (n & 1) ^ 1, abort_flag);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            // Ten tokens, or of 21 CTA 0 the tokens 0 .. 9 and heads 0 .. 7 of token 10, CTA 1 its other heads and
            // the tokens 11 .. 20 (what lies behind the group's tokens is not written, and zeros come from
            // behind the tensor).  In few copies: one of 4 rows takes the 75 cycles of a longer one.
            if (lane == 0) {
                const int g = it.hd * kGrp;
                mbar_arrive_expect_tx(&sh->q_full, (kCtas == 1 ? 120 : (rank == 0 ? 128 : 124)) * kD * 2);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint8_t *dst = sQ + c * kTcQChunk;
                    if (rank == 0) {
                        tma_load_3d(dst, &map_q, &sh->q_full, c * 64, g, it.row0);
                        if (kCtas == 2) {
                            tma_load_3d(dst + 120 * 128, &map_q4, &sh->q_full, c * 64, g, it.row0 + 10);
                            tma_load_3d(dst + 124 * 128, &map_q4, &sh->q_full, c * 64, g + 4, it.row0 + 10);
                        }
                    } else {
                        tma_load_3d(dst, &map_q4, &sh->q_full, c * 64, g + 8, it.row0 + 10);
                        tma_load_3d(dst + 4 * 128, &map_q, &sh->q_full, c * 64, g, it.row0 + 11);
                    }
                }
            }
            __syncwarp();
            ++n;
        }
        // where a role has given up, the last copies may be on their way still: they land before the CTA exits
        if (lane == 0 && n > 0) mbar_wait(&sh->q_full, (n - 1) & 1, nullptr);
    } else if (warp == 1) {
        if (elect_one()) {
            uint32_t stage = 0, ph = 0, n = 0;
            auto advance = [&]() {
                if (++stage == C::kStages) {
                    stage = 0;
                    ph ^= 1u;
                }
            };
            if (rank == 0) {
                // ---------------- products ----------------
                constexpr uint32_t idesc_s = idesc_bf16_f32(128 * kCtas, kKeys, 0, 0);
                constexpr uint32_t idesc_o = idesc_bf16_f32(128 * kCtas, kD, 0, 1);
                const uint32_t q_addr = smem_u32(sQ), ring_u = smem_u32(ring);
                uint32_t T = 0;  // tiles so far
                auto slot_full = [&]() -> bool {
                    if (!mbar_wait(&sh->kv_full[stage], ph, abort_flag)) return false;
                    fence_proxy_async_smem();
                    return kCtas == 1 || wait_pair(&sh->kv_peer[stage], ph, abort_flag);
                };
                auto do_s = [&](uint32_t t) -> bool {
                    if (!slot_full()) return false;
                    tc_fence_after();
                    const uint32_t k_addr = ring_u + stage * kTcSlot, d = tmem + (t & 1) * kKeys;
#pragma unroll
                    for (int ks = 0; ks < kD / 16; ++ks)
                        mma_ss<kCtas>(d, sdesc_sw128(q_addr + (ks >> 2) * kTcQChunk + (ks & 3) * 32, 16, 1024),
                                sdesc_sw128(k_addr + (ks >> 2) * kTcKChunk + (ks & 3) * 32, 16, 1024), idesc_s,
                                ks > 0 ? 1u : 0u);
                    commit_all<kCtas>(&sh->kv_empty[stage]);
                    commit_all<kCtas>(&sh->s_full[t & 1]);
                    advance();
                    return true;
                };
                while (ok && it.next<false>(a)) {
                    const int nt = it.i1 - it.i0;
                    ok = mbar_wait(&sh->q_full, n & 1, abort_flag) && (kCtas == 1 || wait_pair(&sh->q_peer, n & 1, abort_flag));
                    ok = ok && do_s(T);
                    if (ok && nt == 1) commit_all<kCtas>(&sh->q_empty);
                    for (int i = 0; ok && i < nt; ++i, ++T) {
                        if (i + 1 < nt) {
                            if (!(ok = do_s(T + 1))) break;
                            if (i + 2 == nt) commit_all<kCtas>(&sh->q_empty);
                        }
                        if (i == 0 && !(ok = wait_pair(&sh->o_empty, (n & 1) ^ 1, abort_flag))) break;
                        if (!(ok = wait_pair(&sh->p_full[T & 1], (T >> 1) & 1, abort_flag))) break;
                        if (!(ok = slot_full())) break;
                        tc_fence_after();
                        const uint32_t v_addr = ring_u + stage * kTcSlot, p = tmem + (T & 1) * kKeys;
#pragma unroll
                        for (int ks = 0; ks < kKeys / 16; ++ks)
                            mma_ts<kCtas>(tmem + kTcO, p + ks * 8, sdesc_sw128(v_addr + ks * 2048, C::kVChunk, 1024), idesc_o,
                                    (i == 0 && ks == 0) ? 0u : 1u);
                        commit_all<kCtas>(&sh->kv_empty[stage]);
                        commit_all<kCtas>(&sh->pv_done);
                        if (i + 1 == nt) commit_all<kCtas>(&sh->o_full);
                        advance();
                    }
                    ++n;
                }
                // and likewise the products that have been issued: no tensor memory is freed under them (CTA 1
                // waits for this CTA at the end)
                commit_all<kCtas>(&sh->drained);
                mbar_wait(&sh->drained, 0, nullptr);
            } else {
                // ---------------- CTA 1: its Q and slots are full ----------------
                while (ok && it.next<false>(a)) {
                    for (int e = 0; ok && e < 2 * (it.i1 - it.i0); ++e) {
                        ok = mbar_wait(&sh->kv_full[stage], ph, abort_flag);
                        fence_proxy_async_smem();
                        if (ok) arrive_leader(&sh->kv_peer[stage]);
                        advance();
                        if (e == 0 && ok) {
                            ok = mbar_wait(&sh->q_full, n & 1, abort_flag);
                            if (ok) arrive_leader(&sh->q_peer);
                        }
                    }
                    ++n;
                }
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        if (!kFp8) {
            // ---------------- bf16 K and V ----------------
            // Warp w copies K of the keys 32 w .. of the CTA's 64, and V of these and, in a pair, of the same keys
            // of the other CTA's 64; a lane looks up one key of each (row of the KV head, -1: none).  A slot's
            // barrier counts the threads whose copies have arrived.
            const int w = warp - 2, u = lane & 7, k4 = lane >> 3;
            const uint32_t ring_u = smem_u32(ring);
            const uint8_t *kp = static_cast<const uint8_t *>(a.pool.k) + u * 16;
            const uint8_t *vp = static_cast<const uint8_t *>(a.pool.v) + u * 16 + rank * 256;
            uint32_t stage = 0, ph = 1;
            auto slot_ready = [&]() -> bool {
                const bool good = mbar_wait(&sh->kv_empty[stage], ph, abort_flag);
                return __all_sync(0xffffffffu, good);
            };
#ifdef QSA_DEBUG_CHECKS
            // injected fault: the second slot of CTA 1, or of the only CTA, is never full
            bool withhold = g_debug_fault_site == 2 && rank == kCtas - 1;
#endif
            auto slot_issued = [&]() {
#ifdef QSA_DEBUG_CHECKS
                if (withhold && stage == 1) withhold = false;
                else
#endif
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];"
                             ::"r"(smem_u32(&sh->kv_full[stage])) : "memory");
                if (++stage == C::kStages) {
                    stage = 0;
                    ph ^= 1u;
                }
            };
            while (ok && it.next<true>(a)) {
                int32_t page[kCtas];
                uint32_t off[kCtas] = {};
                auto fetch = [&](int i) {
#pragma unroll
                    for (int e = 0; e < kCtas; ++e) page[e] = it.page_of(a, i, ((int)rank ^ e) * 64 + w * 32 + lane, &off[e]);
                };
                auto resolve = [&](int32_t (&r)[kCtas]) {
#pragma unroll
                    for (int e = 0; e < kCtas; ++e) r[e] = it.row_of(a, page[e], off[e]);
                };
                auto load_k = [&](const int32_t (&r)[kCtas]) -> bool {
                    if (!slot_ready()) return false;
                    const uint32_t dst = ring_u + stage * kTcSlot + (w * 32 + k4) * 128;
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const int32_t row = __shfl_sync(0xffffffffu, r[0], x * 4 + k4);
                        const uint8_t *src = kp + (int64_t)(row < 0 ? 0 : row) * 512;
                        const uint32_t d = dst + x * 512 + (((uint32_t)u ^ ((x * 4 + k4) & 7)) << 4);
#pragma unroll
                        for (int c = 0; c < 4; ++c) copy16(d + c * kTcKChunk, src + c * 128, row >= 0);
                    }
                    slot_issued();
                    return true;
                };
                auto load_v = [&](const int32_t (&r)[kCtas]) -> bool {
                    if (!slot_ready()) return false;
#pragma unroll
                    for (int x = 0; x < 8 * kCtas; ++x) {
                        const int key = (x & 7) * 4 + k4;
                        const uint32_t dst = ring_u + stage * kTcSlot + (((int)rank ^ (x >> 3)) * 64 + w * 32 + key) * 128;
                        const int32_t row = __shfl_sync(0xffffffffu, r[x >> 3], key);
                        const uint8_t *src = vp + (int64_t)(row < 0 ? 0 : row) * 512;
                        const uint32_t d = dst + (((uint32_t)u ^ (key & 7)) << 4);
#pragma unroll
                        for (int c = 0; c < C::kVChunks; ++c) copy16(d + c * C::kVChunk, src + c * 128, row >= 0);
                    }
                    slot_issued();
                    return true;
                };
                int32_t r0[kCtas], r1[kCtas];
                fetch(it.i0);
                resolve(r0);
                fetch(it.i0 + 1);
                ok = load_k(r0);
                for (int i = it.i0; ok && i < it.i1; ++i) {
                    resolve(r1);
                    fetch(i + 2);
                    if (i + 1 < it.i1) ok = load_k(r1);
                    ok = ok && load_v(r0);
#pragma unroll
                    for (int e = 0; e < kCtas; ++e) r0[e] = r1[e];
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");  // none is on its way when the CTA exits
        } else {
            // ---------------- rows and scales of e4m3 pools ----------------
            // A key or two per lane; a tile's pages are looked up one tile ahead of its scales, and these
            // one ahead of the table's writing.
            TcTable<kCtas> *tab = reinterpret_cast<TcTable<kCtas> *>(smem + C::kOffTable);
            const int key = (warp - 2) * 32 * kCtas + lane;
            uint32_t n = 0;  // tables written
            while (ok && it.next<true>(a)) {
                int32_t page[kCtas], row[kCtas];
                uint32_t off[kCtas] = {}, kb[kCtas], vb[kCtas];
                auto fetch = [&](int i) {
#pragma unroll
                    for (int e = 0; e < kCtas; ++e) page[e] = it.page_of(a, i, key + 32 * e, &off[e]);
                };
                auto resolve = [&]() {
#pragma unroll
                    for (int e = 0; e < kCtas; ++e) {
                        row[e] = it.row_of(a, page[e], off[e]);
                        kb[e] = row[e] >= 0 ? __ldg(a.pool.k_scales + row[e]) : 127u;
                        vb[e] = row[e] >= 0 ? __ldg(a.pool.v_scales + row[e]) : 127u;
                    }
                };
                fetch(it.i0);
                resolve();
                fetch(it.i0 + 1);
                for (int i = it.i0; i < it.i1; ++i, ++n) {
                    const uint32_t x = n % kTcTables;
                    int32_t r[kCtas];
                    uint32_t k[kCtas], v[kCtas];
#pragma unroll
                    for (int e = 0; e < kCtas; ++e) {
                        r[e] = row[e];
                        k[e] = kb[e];
                        v[e] = vb[e];
                    }
                    resolve();
                    fetch(i + 2);
                    ok = mbar_wait(&sh->tab_empty[x], ((n / kTcTables) & 1) ^ 1, abort_flag);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
#pragma unroll
                    for (int e = 0; e < kCtas; ++e) {
                        tab->row[x][key + 32 * e] = r[e];
                        tab->ks[x][key + 32 * e] = (uint8_t)k[e];
                        tab->vs[x][key + 32 * e] = (uint8_t)v[e];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->tab_full[x]);
                }
            }
        }
    } else if (warp < 8) {
        // ---------------- softmax and epilogue ----------------
        constexpr int kPart = 64;  // a tile's keys, or half of them
        const int quad = warp & 3, rl = quad * 32 + lane, r = (int)rank * 128 + rl;
        const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
        const float c2 = a.scale * 1.4426950408889634f;
        uint32_t T = 0, n = 0;
        auto await = [&](uint64_t *bar, uint32_t parity) -> bool {
            ok = mbar_wait(bar, parity, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            return ok;
        };
        while (ok && it.next<true>(a)) {
            const int t = it.t0 + r / kGrp;  // this row's position (rows past the tokens: not written)
            float m = -INFINITY, l = 0.f;          // running maximum of c2 s, sum of exp2(c2 s - m)
            for (int i = it.i0; i < it.i1; ++i, ++T) {
                const uint32_t buf = T & 1, s_addr = lane_addr + buf * kKeys;
                if (!await(&sh->s_full[buf], (T >> 1) & 1)) break;
                const int j0 = it.tile(i);
                // unless every row sees every key of the tile: columns hi and below, from lo on or below sk
                const bool edge = !(j0 + kKeys - 1 <= it.t0 &&
                                    (a.window <= 0 || it.t_last - j0 < a.window || j0 + kKeys <= a.sinks));
                int hi = kKeys, lo = 0, sk = 0;
                if (edge) {
                    hi = t - j0;
                    lo = a.window > 0 && a.window <= hi ? hi - (int)a.window + 1 : 0;
                    sk = it.sinks - j0;
                }
                auto load = [&](int h, float (&s)[kPart]) {
#pragma unroll
                    for (int c = 0; c < kPart / 32; ++c) tmem_ld32(s_addr + h * kPart + c * 32, s + c * 32);
                };
                auto mask = [&](int h, float (&s)[kPart]) {
                    if (edge) {
#pragma unroll
                        for (int c = 0; c < kPart; ++c)
                            if (h * kPart + c > hi || (h * kPart + c < lo && h * kPart + c >= sk)) s[c] = -INFINITY;
                    }
                };
                auto largest = [&](float x, const float (&s)[kPart]) -> float {
                    float y = s[0], z = s[1], w = s[2];
                    x = fmaxf(x, s[3]);
#pragma unroll
                    for (int c = 4; c + 8 <= kPart; c += 8) {
                        x = max3(x, s[c], s[c + 1]);
                        y = max3(y, s[c + 2], s[c + 3]);
                        z = max3(z, s[c + 4], s[c + 5]);
                        w = max3(w, s[c + 6], s[c + 7]);
                    }
                    x = max3(x, s[kPart - 4], s[kPart - 3]);
                    y = max3(y, s[kPart - 2], s[kPart - 1]);
                    return fmaxf(max3(x, y, z), w);
                };
                // The maximum first.  bf16 pools keep all scores in registers from here on; with 16 warps
                // there is room for the first half only, and the second is read again below.
                float s0[kPart], s1[kPart];
                float mx = -INFINITY;
                if (kCtas == 2) {
                    load(1, s1);
                    if (!kFp8) load(0, s0);
                    tmem_wait_ld();
                    mask(1, s1);
                    mx = largest(mx, s1);
                }
                if (kFp8 || kCtas == 1) {
                    load(0, s0);
                    tmem_wait_ld();
                }
                mask(0, s0);
                mx = largest(mx, s0);
                mx *= c2;
                // O and l are zero until a key is visible, rescaled after that
                const bool grow = m != -INFINITY && mx > m + kTcRescale;
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? ex2(m - mx) : 1.f;
                    if (grow) m = mx;
                    l *= f;
                    // O of the tiles before: T - 1 products have completed at least (S(T) came behind them)
                    if (!await(&sh->pv_done, (T - 1) & 1)) break;
#pragma unroll 1
                    for (int c = 0; c < kD / 32; ++c) {
                        float o[32];
                        tmem_ld32(lane_addr + kTcO + c * 32, o);
                        tmem_wait_ld();
                        tmem_st16(lane_addr + kTcO + c * 32, o, f);
                        tmem_st16(lane_addr + kTcO + c * 32 + 16, o + 16, f);
                    }
                }
                if (m == -INFINITY) m = mx;
                const float base = m == -INFINITY ? 0.f : m;
                const uint64_t c22 = pack2(c2, c2), b22 = pack2(-base, -base);
                uint64_t l01 = pack2(l, 0.f), l23 = pack2(0.f, 0.f);
                // half h's keys as columns 32 h ..: the scores there have been read by now
                auto probabilities = [&](int h, const float (&s)[kPart]) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const int c = 32 * x + 2 * e;
                            const float2 y = unpack2(fma2(pack2(s[c], s[c + 1]), c22, b22));
                            const float2 z = unpack2(fma2(pack2(s[c + 2], s[c + 3]), c22, b22));
                            const float p0 = ex2(y.x), p1 = ex2(y.y), p2 = ex2(z.x), p3 = ex2(z.y);
                            l01 = add2(l01, pack2(p0, p1));
                            l23 = add2(l23, pack2(p2, p3));
                            const __nv_bfloat162 a0 = __floats2bfloat162_rn(p0, p1), a1 = __floats2bfloat162_rn(p2, p3);
                            p[e] = *reinterpret_cast<const uint32_t *>(&a0);
                            p[e + 1] = *reinterpret_cast<const uint32_t *>(&a1);
                        }
                        tmem_st16u(s_addr + h * 32 + x * 16, p);
                    }
                };
                probabilities(0, s0);
                if (kCtas == 2) {
                    if (kFp8) {
                        load(1, s0);
                        tmem_wait_ld();
                        mask(1, s0);
                    }
                    probabilities(1, kFp8 ? s0 : s1);
                }
                const float2 la = unpack2(add2(l01, l23));
                l = la.x + la.y;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_leader_relaxed(&sh->p_full[buf]);
            }
            // O of the whole item
            if (!ok || !await(&sh->o_full, n & 1)) break;
            ++n;
            const bool mine = r / kGrp < it.nq && r < C::kRows, none = l == 0.f;
            const float inv = none ? 0.f : 1.f / l;
            const bool complete = it.i0 == 0 && it.i1 == it.nt;
            const int64_t piece = 2 * worker + (it.i0 == 0 ? 1 : 0);
            const int64_t row = (int64_t)(it.row0 + r / kGrp) * kHQ + it.hd * kGrp + r % kGrp;
            // four lanes exchange 16-byte pieces of their four rows, so that a store writes 64 bytes of each
            const int r4 = r & ~3, q = lane & 3;
            const int rows = it.nq * kGrp - r4;  // of the four, those that are written
#pragma unroll 1
            for (int c = 0; c < kD / 32; ++c) {
                float o[32];
                tmem_ld32(lane_addr + kTcO + c * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = none ? 0.f : o[e] * inv;
                if (complete) {
                    uint4 v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        __nv_bfloat162 h[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) h[x] = __floats2bfloat162_rn(o[e * 8 + 2 * x], o[e * 8 + 2 * x + 1]);
                        v[e] = *reinterpret_cast<const uint4 *>(h);
                    }
                    transpose4(v, lane);
                    // (the four rows are heads of one token: 12 is a multiple of 4)
                    __nv_bfloat16 *dst = a.o + (row - q) * kD + c * 32 + q * 8;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < rows) *reinterpret_cast<uint4 *>(dst + j * kD) = v[j];
                } else {
                    float *dst = a.ws + (piece * C::kRows + r4) * kD + c * 32 + q * 4;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint4 v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = make_uint4(__float_as_uint(o[h * 16 + 4 * e]), __float_as_uint(o[h * 16 + 4 * e + 1]),
                                              __float_as_uint(o[h * 16 + 4 * e + 2]), __float_as_uint(o[h * 16 + 4 * e + 3]));
                        transpose4(v, lane);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < rows) *reinterpret_cast<uint4 *>(dst + j * kD + h * 16) = v[j];
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader_relaxed(&sh->o_empty);
            if (mine) {
                const float lse2 = none ? -INFINITY : m + log2f(l);
                if (!complete) a.ws[2 * workers * C::kRows * kD + piece * C::kRows + r] = lse2;
                else if (a.lse != nullptr) a.lse[row] = lse2 * 0.6931471805599453f;
            }
        }
    } else if (kFp8) {
        // ---------------- e4m3 codes to bf16 ----------------
        const TcTable<kCtas> *tab = reinterpret_cast<const TcTable<kCtas> *>(smem + C::kOffTable);
        const int cw = warp - 8, k8 = lane >> 2, piece = lane & 3;
        const uint32_t ring_u = smem_u32(ring);
        const uint8_t *kp = static_cast<const uint8_t *>(a.pool.k) + piece * 16;
        const uint8_t *vp = static_cast<const uint8_t *>(a.pool.v) + rank * 128 + piece * 16;
        uint32_t stage = 0, ph = 1, n = 0;
        // A warp converts 8 keys of K (all dims) and 8 or, in a pair, 16 of V (this CTA's dims) per tile; the next
        // half tile of the other kind is loaded before one is converted.
        uint4 kreg[4], vreg[4];
        uint32_t kb, vb[kCtas];
        auto load_k = [&](uint32_t x) {
            const int key = (int)rank * 64 + cw * 8 + k8;
            const int32_t row = tab->row[x][key];
            kb = tab->ks[x][key];
            const uint8_t *src = kp + (int64_t)row * kD;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                kreg[c] = row >= 0 ? __ldg(reinterpret_cast<const uint4 *>(src + c * 64)) : make_uint4(0u, 0u, 0u, 0u);
        };
        auto load_v = [&](uint32_t x) {
#pragma unroll
            for (int q = 0; q < kCtas; ++q) {
                const int key = (cw * kCtas + q) * 8 + k8;
                const int32_t row = tab->row[x][key];
                vb[q] = tab->vs[x][key];
                const uint8_t *src = vp + (int64_t)row * kD;
#pragma unroll
                for (int c = 0; c < C::kVChunks; ++c)
                    vreg[q * C::kVChunks + c] = row >= 0 ? __ldg(reinterpret_cast<const uint4 *>(src + c * 64)) : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        auto table_ready = [&](uint32_t t) -> bool {
            ok = mbar_wait(&sh->tab_full[t % kTcTables], (t / kTcTables) & 1, abort_flag);
            return ok = __all_sync(0xffffffffu, ok);
        };
        auto slot_ready = [&]() -> bool {
            ok = mbar_wait(&sh->kv_empty[stage], ph, abort_flag);
            return ok = __all_sync(0xffffffffu, ok);
        };
#ifdef QSA_DEBUG_CHECKS
        bool withhold = g_debug_fault_site == 2 && rank == kCtas - 1;  // as above
#endif
        auto slot_done = [&]() {
            __syncwarp();
#ifdef QSA_DEBUG_CHECKS
            if (withhold && stage == 1) withhold = false;
            else
#endif
            if (lane == 0) mbar_arrive(&sh->kv_full[stage]);
            if (++stage == C::kStages) {
                stage = 0;
                ph ^= 1u;
            }
        };
        while (ok && it.next<true>(a)) {
            const uint32_t nt = (uint32_t)(it.i1 - it.i0);
            if (!table_ready(n)) break;
            load_k(n % kTcTables);
            for (uint32_t i = 0; i <= nt; ++i) {
                if (i < nt) {  // K(i)
                    if (!slot_ready()) break;
                    const float sc = scale_of_byte(kb);
                    const uint32_t dst = ring_u + stage * kTcSlot + (cw * 8 + k8) * 128;
#pragma unroll
                    for (int c = 0; c < 4; ++c) codes_to_slot<kCtas>(kreg[c], sc, dst + c * kTcKChunk, 2 * piece, k8);
                    slot_done();
                }
                if (i + 1 < nt) {
                    if (!table_ready(n + i + 1)) break;
                    load_k((n + i + 1) % kTcTables);
                }
                if (i > 0) {  // V(i - 1)
                    if (!slot_ready()) break;
#pragma unroll
                    for (int q = 0; q < kCtas; ++q) {
                        const float sc = scale_of_byte(vb[q]);
                        const uint32_t dst = ring_u + stage * kTcSlot + ((cw * kCtas + q) * 8 + k8) * 128;
#pragma unroll
                        for (int c = 0; c < C::kVChunks; ++c) codes_to_slot<kCtas>(vreg[q * C::kVChunks + c], sc, dst + c * C::kVChunk, 2 * piece, k8);
                    }
                    slot_done();
                }
                if (i < nt) {
                    load_v((n + i) % kTcTables);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->tab_empty[(n + i) % kTcTables]);
                }
            }
            n += nt;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (kCtas == 2) cluster_sync();  // no arrival of the peer is under way
    if (warp == 1) {
        tc_fence_after();
        if (kCtas == 1)
            tmem_dealloc(tmem, kTcCols);
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTcCols) : "memory");
    }
}

// pairs of CTAs that run at the same time on the current device
template <bool kFp8>
cudaError_t tc_workers(int64_t *out)
{
    static std::mutex mu;
    static int known[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 64 && known[dev] > 0) {
        *out = known[dev];
        return cudaSuccess;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * kTcMaxPairs);
    cfg.blockDim = dim3(TcCfg<kFp8, 2>::kThreads);
    cfg.dynamicSmemBytes = TcCfg<kFp8, 2>::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, chunk_tc_kernel<kFp8, 2>, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    if (n > kTcMaxPairs) n = (int)kTcMaxPairs;
    if (dev < 64) known[dev] = n;
    *out = n;
    return cudaSuccess;
}

size_t tc_pieces_offset()
{
    static_assert(kTcMaxPairs * 252 >= kTcMaxSingles * 120, "the pairs' pieces are the larger ones");
    return (size_t)(2 * kTcMaxPairs) * 252 * (kD + 1) * sizeof(float);
}

template <bool kFp8, int kCtas>
cudaError_t launch_tc(const ChunkArgs &a, cudaStream_t stream)
{
    using C = TcCfg<kFp8, kCtas>;
    CUtensorMap mq, mq4;  // ten tokens, and four heads of one, of 64 dims
    if (!make_tmap_3d(&mq, a.q, kD, kHQ, (uint64_t)a.total_q, kD * 2, (uint64_t)kHQ * kD * 2, 64, kGrp, 10) ||
        !make_tmap_3d(&mq4, a.q, kD, kHQ, (uint64_t)a.total_q, kD * 2, (uint64_t)kHQ * kD * 2, 64, 4, 1))
        return cudaErrorInvalidValue;
    cudaError_t e = set_smem_attr_once(reinterpret_cast<const void *>(chunk_tc_kernel<kFp8, kCtas>), C::kSmem);
    if (e != cudaSuccess) return e;
    int64_t workers = num_sms();
    if (workers > kTcMaxSingles) workers = kTcMaxSingles;
    if (kCtas == 2) {
        e = tc_workers<kFp8>(&workers);
        if (e != cudaSuccess) return e;
    }
    int2 *pieces = reinterpret_cast<int2 *>(reinterpret_cast<uint8_t *>(a.ws) + tc_pieces_offset());
    e = launch_pdl(chunk_tc_kernel<kFp8, kCtas>, dim3((unsigned)(kCtas * workers)), dim3(C::kThreads), C::kSmem, stream, mq,
                   mq4, a, pieces);
    if (e != cudaSuccess) return e;
    return launch_chunk_merge<C::kTok, C::kKeys, C::kRestart>(a, pieces, workers, stream);
}

}  // namespace

size_t chunk_tc_workspace_bytes(int batch, int64_t total_q)
{
    return tc_pieces_offset() + (size_t)chunk_slots<10>(total_q, batch) * 2 * sizeof(int2);
}

// the single CTA's kernel where all groups are small (see above)
cudaError_t launch_chunk_tc(const ChunkArgs &a, cudaStream_t stream)
{
    if (a.max_len_q <= 10) return a.pool.fp8 ? launch_tc<true, 1>(a, stream) : launch_tc<false, 1>(a, stream);
    return a.pool.fp8 ? launch_tc<true, 2>(a, stream) : launch_tc<false, 2>(a, stream);
}

}  // namespace qsa
