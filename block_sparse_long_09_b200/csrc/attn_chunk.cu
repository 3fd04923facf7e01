// attn_chunk.cu -- attention of the new tokens of every sequence over its paged cache,
// rows kernel: up to kTok new tokens (12 kTok query rows of a KV head) per item.
//
//   o[t, h] = sum_j p_j v[j, g] / sum_j p_j,  p_j = exp(scale <q[t, h], k[j, g]> - m)
// over the cached positions j <= t with t - j < window or j < sinks (no window: all).
//
// One decoded token brings 12 rows to 512 B (e4m3) or 1 KB (bf16) of K and V per key, so this
// kernel is bound by HBM; it is built to keep 64 KB of loads per CTA in flight, two CTAs per
// SM, with nothing between memory and the matrix instructions but registers:
//   * S = Q K^T by mma.m16n8k16: a warp takes 16 (e4m3) or 8 (bf16) keys of the tile, its
//     lanes load 16 B pieces of the keys' rows straight into B fragments.  The order of the
//     256 dims inside the sums is free, so it is chosen to make a lane's dims contiguous,
//     and Q is laid out once per item in the same order (A fragments in shared memory).
//   * e4m3 codes become bf16 by moving their 7 low bits to the top of a bf16 and
//     multiplying by 2^120; exact.  The keys' scales multiply S, the values' scales multiply P:
//     powers of two, exact as well.
//   * the softmax statistics are shared through 8 row maxima in shared memory; P goes to
//     shared memory as bf16 (its rounding: 2^-9 relative per term, as in every attention
//     kernel of this library).
//   * O += P V: a warp owns 32 of the 256 dims for all the tile's keys.  Its lanes load 4
//     dims of 4 consecutive keys; byte permutes pair the keys for the B fragments, so V
//     needs no transpose through shared memory.
// The next tile's K loads are issued as soon as S is computed, its pool rows two tiles ahead.
// Tiles that no row sees are never read, and keys that no row of the item sees (behind the
// sequence's end, before the window) are replaced by zeros, whatever their memory holds.
#include "chunk_common.cuh"

namespace qsa {

namespace {

constexpr int kRowWarps = 8, kRowThreads = kRowWarps * 32;

template <bool kFp8>
struct RowCfg {
    static constexpr int kKeys = kFp8 ? 128 : 64;         // keys per tile: 64 KB of K and V
    static constexpr int kNT = kKeys / (8 * kRowWarps);   // 8-key column tiles of a warp's S
    static constexpr int kPieces = kFp8 ? 4 : 8;          // 16 B pieces of a key's row per lane
    static constexpr int kKS = kKeys / 16;                // k steps of P V
    static constexpr int kPitch = kKeys + 8;              // P row pitch: ldmatrix without bank conflicts
};

__device__ __forceinline__ uint4 ld_stream16(const void *p)
{
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldmatrix4(uint32_t addr)
{
    uint4 r;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
    return r;
}

// two codes in the high bytes of a register's halves -> bf16 pair
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t x)
{
    const uint32_t y = (x & 0x80008000u) | ((x >> 4) & 0x07F007F0u);
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&y),
                                     __halves2bfloat162(__ushort_as_bfloat16(0x7B80), __ushort_as_bfloat16(0x7B80)));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// kMT 16-row tiles of (token, head) rows: 1 token in 16, or 4 tokens in 48
template <int kMT>
constexpr int row_tokens() { return kMT * 16 / kGrp; }

template <int kMT, bool kFp8>
struct RowShared {
    uint4 q[kMT][16][32];                                        // A fragments of Q
    __nv_bfloat16 p[kMT * 16][RowCfg<kFp8>::kPitch];
    float wmax[kRowWarps][kMT * 16], wsum[kRowWarps][kMT * 16];
    alignas(16) int32_t row[3][RowCfg<kFp8>::kKeys];             // pool rows of the tiles' keys, -1: none
    float ks[2][RowCfg<kFp8>::kKeys], vs[2][RowCfg<kFp8>::kKeys];
    int64_t scan[kRowWarps];
    ChunkShare share;
};

template <int kMT, bool kFp8>
__global__ void __launch_bounds__(kRowThreads, 2)
chunk_rows_kernel(const ChunkArgs a, int64_t *__restrict__ prefix)
{
    using C = RowCfg<kFp8>;
    constexpr int kKeys = C::kKeys, kTok = row_tokens<kMT>(), kRows = kTok * kGrp;
    constexpr int kBytes = kFp8 ? kD : 2 * kD;  // of a key's row of one KV head
    __shared__ RowShared<kMT, kFp8> sh;
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = lane >> 2, c = lane & 3;      // fragment coordinates
    chunk_share<kTok, kKeys, kRowThreads>(a, blockIdx.x, gridDim.x, &sh.share, sh.scan,
                                          blockIdx.x == 0 ? prefix : nullptr);
    int64_t at = sh.share.ts;
    const int64_t te = sh.share.te;
    int64_t slot = sh.share.slot, slot_first = sh.share.first;
    const float c2 = a.scale * 1.4426950408889634f;
    const uint8_t *kp = static_cast<const uint8_t *>(a.pool.k), *vp = static_cast<const uint8_t *>(a.pool.v);

    while (at < te) {
        ChunkGroup g = chunk_group<kTok, kKeys>(a, slot);
        while (at >= slot_first + 2 * (int64_t)g.nt) {  // empty slots between two groups
            slot_first += 2 * (int64_t)g.nt;
            g = chunk_group<kTok, kKeys>(a, ++slot);
        }
        const int hd = at >= slot_first + g.nt ? 1 : 0;  // KV head
        const int64_t item_first = slot_first + (int64_t)hd * g.nt;
        const int i0 = (int)(at - item_first);
        const int i1 = te - item_first < g.nt ? (int)(te - item_first) : g.nt;
        const int64_t t_first = g.t0 > 0 ? g.t0 : 0, t_last = g.t0 + g.nq - 1;

        // the pool rows of tile i's keys: 0 .. kKeys - 1 threads, one key each
        auto key_row = [&](int i) -> int32_t {
            if (i >= i1) return -1;
            const int64_t j = tile_start(g, i, kKeys) + tid;
            const bool any = j <= t_last && (a.window <= 0 || t_first - j < a.window || j < a.sinks);
            return any ? (int32_t)chunk_pool_row(a.pool, g.s, j) : -1;
        };
        __syncthreads();  // the previous item's last reads of shared memory
        if (tid < kKeys) {
            sh.row[0][tid] = key_row(i0);
            sh.row[1][tid] = key_row(i0 + 1);
            if (kFp8) {
                const int32_t r = sh.row[0][tid];
                sh.ks[0][tid] = r >= 0 ? scale_of_byte(__ldg(a.pool.k_scales + (int64_t)r * 2 + hd)) : 0.f;
                sh.vs[0][tid] = r >= 0 ? scale_of_byte(__ldg(a.pool.v_scales + (int64_t)r * 2 + hd)) : 0.f;
            }
        }
        for (int x = tid; x < kMT * 16 * 32; x += kRowThreads) {
            const int mt = x / 512, st = (x / 32) % 16, ln = x & 31;
            const int r0 = mt * 16 + (ln >> 2);
            const int d = kFp8 ? (st >> 2) * 64 + (ln & 3) * 16 + (st & 3) * 4 : (st >> 1) * 32 + (ln & 3) * 8 + (st & 1) * 4;
            uint2 lo = make_uint2(0u, 0u), hi = lo;
            const __nv_bfloat16 *src = a.q + (g.row0 * kHQ + hd * kGrp) * kD + d;
            if (r0 / kGrp < g.nq)
                lo = __ldg(reinterpret_cast<const uint2 *>(src + ((int64_t)(r0 / kGrp) * kHQ + r0 % kGrp) * kD));
            if ((r0 + 8) / kGrp < g.nq)
                hi = __ldg(reinterpret_cast<const uint2 *>(src + ((int64_t)((r0 + 8) / kGrp) * kHQ + (r0 + 8) % kGrp) * kD));
            sh.q[mt][st][ln] = make_uint4(lo.x, hi.x, lo.y, hi.y);
        }
        __syncthreads();

        uint4 kr[C::kNT][C::kPieces];
        auto load_k = [&](int buf) {
#pragma unroll
            for (int nt = 0; nt < C::kNT; ++nt) {
                const int32_t r = sh.row[buf][warp * (kKeys / kRowWarps) + nt * 8 + n];
                const uint8_t *src = kp + ((int64_t)r * kHKV + hd) * kBytes + c * 16;
#pragma unroll
                for (int i = 0; i < C::kPieces; ++i)
                    kr[nt][i] = r >= 0 ? ld_stream16(src + i * 64) : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        load_k(0);

        float o[kMT][4][4];
        float m[kMT][2], l[kMT][2];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][j][e] = 0.f;
            m[mt][0] = m[mt][1] = -INFINITY;
            l[mt][0] = l[mt][1] = 0.f;
        }
        // positions of this thread's rows; a row without a token sees no key
        int64_t t_row[kMT][2];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = mt * 16 + n + 8 * e;
                t_row[mt][e] = r / kGrp < g.nq ? g.t0 + r / kGrp : (int64_t)-1;
            }

        int cur = 0, nxt = 1, aft = 2;  // ring of the pool rows: this tile's, the next one's, the one after
        for (int i = i0; i < i1; ++i) {
            const int par = (i - i0) & 1;
            // V of this tile
            uint32_t vr[C::kKS][4][kFp8 ? 1 : 2];
#pragma unroll
            for (int ks = 0; ks < C::kKS; ++ks) {
                const int4 r4 = *reinterpret_cast<const int4 *>(&sh.row[cur][ks * 16 + c * 4]);
                const int32_t r[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint8_t *src = vp + ((int64_t)r[e] * kHKV + hd) * kBytes + (warp * 32 + n * 4) * (kFp8 ? 1 : 2);
                    if (kFp8) {
                        vr[ks][e][0] = r[e] >= 0 ? __ldg(reinterpret_cast<const uint32_t *>(src)) : 0u;
                    } else {
                        const uint2 x = r[e] >= 0 ? __ldg(reinterpret_cast<const uint2 *>(src)) : make_uint2(0u, 0u);
                        vr[ks][e][0] = x.x;
                        vr[ks][e][kFp8 ? 0 : 1] = x.y;
                    }
                }
            }
            // S of this warp's keys
            float s[C::kNT][kMT][4];
#pragma unroll
            for (int nt = 0; nt < C::kNT; ++nt)
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[nt][mt][e] = 0.f;
#pragma unroll
            for (int st = 0; st < 16; ++st) {
                uint4 qa[kMT];
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) qa[mt] = sh.q[mt][st][lane];
#pragma unroll
                for (int nt = 0; nt < C::kNT; ++nt) {
                    uint32_t b0, b1;
                    if (kFp8) {
                        const uint4 &x = kr[nt][st >> 2];
                        const uint32_t w = (st & 3) == 0 ? x.x : ((st & 3) == 1 ? x.y : ((st & 3) == 2 ? x.z : x.w));
                        b0 = codes_to_bf16(__byte_perm(w, 0u, 0x1100));
                        b1 = codes_to_bf16(__byte_perm(w, 0u, 0x3322));
                    } else {
                        const uint4 &x = kr[nt][(st >> 1) % C::kPieces];
                        b0 = (st & 1) ? x.z : x.x;
                        b1 = (st & 1) ? x.w : x.y;
                    }
#pragma unroll
                    for (int mt = 0; mt < kMT; ++mt) mma_16816(s[nt][mt], qa[mt], b0, b1);
                }
            }
            // the next tile's K, its scales, and the pool rows of the tile after it
            int32_t row2 = -1;
            uint32_t kb = 0u, vb = 0u;
            if (i + 1 < i1) {
                load_k(nxt);
                if (tid < kKeys) {
                    row2 = key_row(i + 2);
                    if (kFp8) {
                        const int64_t r = sh.row[nxt][tid];
                        kb = r >= 0 ? __ldg(a.pool.k_scales + r * 2 + hd) : 0u;
                        vb = r >= 0 ? __ldg(a.pool.v_scales + r * 2 + hd) : 0u;
                    }
                }
            }
            // scale, mask, row maxima
            const int64_t j0 = tile_start(g, i, kKeys);
            // every row sees every key of the tile: no test per entry
            const bool whole = g.t0 >= 0 && j0 + kKeys - 1 <= g.t0 && g.nq == kTok &&
                               (a.window <= 0 || t_last - j0 < a.window || j0 + kKeys <= a.sinks);
            float mx[kMT][2];
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) mx[mt][0] = mx[mt][1] = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < C::kNT; ++nt) {
                const int key = warp * (kKeys / kRowWarps) + nt * 8 + 2 * c;
                const float f0 = kFp8 ? c2 * sh.ks[par][key] : c2, f1 = kFp8 ? c2 * sh.ks[par][key + 1] : c2;
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = s[nt][mt][e] * ((e & 1) ? f1 : f0);
                        if (!whole && !chunk_sees(t_row[mt][e >> 1], j0 + key + (e & 1), a.window, a.sinks)) x = -INFINITY;
                        s[nt][mt][e] = x;
                        mx[mt][e >> 1] = fmaxf(mx[mt][e >> 1], x);
                    }
            }
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = mx[mt][e];
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    if (c == 0) sh.wmax[warp][mt * 16 + n + 8 * e] = x;
                }
            __syncthreads();
            float f[kMT][2];
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = m[mt][e];
#pragma unroll
                    for (int w = 0; w < kRowWarps; ++w) x = fmaxf(x, sh.wmax[w][mt * 16 + n + 8 * e]);
                    const float base = x == -INFINITY ? 0.f : x;  // no visible key yet
                    f[mt][e] = exp2f(m[mt][e] - base);
                    m[mt][e] = x;
                    mx[mt][e] = base;
                    l[mt][e] *= f[mt][e];
                }
            // P, its row sums (of the unrounded values), and the values' scales folded in
#pragma unroll
            for (int nt = 0; nt < C::kNT; ++nt) {
                const int key = warp * (kKeys / kRowWarps) + nt * 8 + 2 * c;
                const float v0 = kFp8 ? sh.vs[par][key] : 1.f, v1 = kFp8 ? sh.vs[par][key + 1] : 1.f;
                // key 4 x + y of a 16-key step is column 2 x + (y & 1) + 8 (y >> 1): a lane's four
                // keys of a step are then consecutive in the cache
                const int k16 = key & 15, col = (key & ~15) + 2 * (k16 >> 2) + ((k16 & 2) << 2);
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float p0 = exp2f(s[nt][mt][2 * e] - mx[mt][e]), p1 = exp2f(s[nt][mt][2 * e + 1] - mx[mt][e]);
                        l[mt][e] += p0 + p1;
                        // a masked key's scale may be a NaN (a row with a non-finite value): P stays 0
                        const float w0 = kFp8 ? (p0 == 0.f ? 0.f : p0 * v0) : p0, w1 = kFp8 ? (p1 == 0.f ? 0.f : p1 * v1) : p1;
                        *reinterpret_cast<__nv_bfloat162 *>(&sh.p[mt * 16 + n + 8 * e][col]) = __floats2bfloat162_rn(w0, w1);
                    }
            }
            if (tid < kKeys && i + 1 < i1) {
                sh.row[aft][tid] = row2;
                if (kFp8) {
                    sh.ks[par ^ 1][tid] = scale_of_byte(kb);
                    sh.vs[par ^ 1][tid] = scale_of_byte(vb);
                }
            }
            __syncthreads();
            // O = O f + P V
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[mt][j][e] *= f[mt][e >> 1];
#pragma unroll
            for (int ks = 0; ks < C::kKS; ++ks) {
                uint4 pa[kMT];
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
                    pa[mt] = ldmatrix4(smem_u32(&sh.p[mt * 16 + (lane & 15)][ks * 16 + (lane >> 4) * 8]));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t b0, b1;
                    if (kFp8) {
                        const uint32_t sel = j * 0x11u | (4 + j) * 0x1100u;
                        b0 = codes_to_bf16(__byte_perm(vr[ks][0][0], vr[ks][1][0], sel));
                        b1 = codes_to_bf16(__byte_perm(vr[ks][2][0], vr[ks][3][0], sel));
                    } else {
                        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
                        const int hh = kFp8 ? 0 : j >> 1;
                        b0 = __byte_perm(vr[ks][0][hh], vr[ks][1][hh], sel);
                        b1 = __byte_perm(vr[ks][2][hh], vr[ks][3][hh], sel);
                    }
#pragma unroll
                    for (int mt = 0; mt < kMT; ++mt) mma_16816(o[mt][j], pa[mt], b0, b1);
                }
            }
            const int t = cur;
            cur = nxt;
            nxt = aft;
            aft = t;
        }

        // row sums over the warps' keys
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[mt][e];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (c == 0) sh.wsum[warp][mt * 16 + n + 8 * e] = x;
            }
        __syncthreads();
        const bool complete = i0 == 0 && i1 == g.nt;
        const int64_t piece = 2 * (int64_t)blockIdx.x + (i0 == 0 ? 1 : 0);
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = mt * 16 + n + 8 * e;
                if (r / kGrp >= g.nq) continue;
                float L = 0.f;
#pragma unroll
                for (int w = 0; w < kRowWarps; ++w) L += sh.wsum[w][r];
                const bool none = L == 0.f;  // (a NaN is not)
                const float inv = none ? 0.f : 1.f / L;
                const float lse2 = none ? -INFINITY : m[mt][e] + log2f(L);
                float x[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] = none ? 0.f : o[mt][j][2 * e] * inv;
                    x[4 + j] = none ? 0.f : o[mt][j][2 * e + 1] * inv;
                }
                const int d = warp * 32 + c * 8;
                if (complete) {
                    const int64_t row = (g.row0 + r / kGrp) * kHQ + hd * kGrp + r % kGrp;
                    __nv_bfloat162 h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                    *reinterpret_cast<uint4 *>(a.o + row * kD + d) = *reinterpret_cast<const uint4 *>(h);
                    if (a.lse != nullptr && warp == 0 && c == 0) a.lse[row] = lse2 * 0.6931471805599453f;
                } else {
                    float *dst = a.ws + (piece * kRows + r) * kD + d;
                    *reinterpret_cast<float4 *>(dst) = make_float4(x[0], x[1], x[2], x[3]);
                    *reinterpret_cast<float4 *>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
                    if (warp == 0 && c == 0) a.ws[2 * (int64_t)gridDim.x * kRows * kD + piece * kRows + r] = lse2;
                }
            }
        at = item_first + i1;
    }
}

constexpr int64_t kMaxWorkers = 512;  // CTAs of the rows kernel, at most (the workspace's bound)

size_t rows_prefix_offset(int rows) { return (size_t)(2 * kMaxWorkers) * rows * (kD + 1) * sizeof(float); }

template <int kMT, bool kFp8>
cudaError_t launch_rows(const ChunkArgs &a, cudaStream_t stream)
{
    constexpr int kTok = row_tokens<kMT>(), kRows = kTok * kGrp, kKeys = RowCfg<kFp8>::kKeys;
    int64_t *prefix = reinterpret_cast<int64_t *>(reinterpret_cast<uint8_t *>(a.ws) + rows_prefix_offset(kRows));
    int64_t workers = (int64_t)num_sms() * 2;
    if (workers > kMaxWorkers) workers = kMaxWorkers;
    cudaError_t e = launch_pdl(chunk_rows_kernel<kMT, kFp8>, dim3((unsigned)workers), dim3(kRowThreads), 0, stream, a, prefix);
    if (e != cudaSuccess) return e;
    return launch_chunk_merge<kTok, kKeys>(a, prefix, workers, stream);
}

}  // namespace

size_t chunk_workspace_bytes(int batch, int64_t total_q)
{
    const size_t rows = row_tokens<3>() * kGrp;
    const size_t own = rows_prefix_offset(rows) + (size_t)(chunk_slots<1>(total_q, batch) + 1) * sizeof(int64_t);
    const size_t tc = chunk_tc_workspace_bytes(batch, total_q);
    return own > tc ? own : tc;
}

cudaError_t launch_chunk_attn(const ChunkArgs &a, cudaStream_t stream)
{
    if (a.total_q <= 0) return cudaSuccess;
    if (a.max_len_q <= 1) return a.pool.fp8 ? launch_rows<1, true>(a, stream) : launch_rows<1, false>(a, stream);
    return launch_chunk_tc(a, stream);
}

}  // namespace qsa
