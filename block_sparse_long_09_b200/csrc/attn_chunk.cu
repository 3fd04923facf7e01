// attn_chunk.cu -- attention of the new tokens of every sequence over its paged cache:
// the kernel for single new tokens (decoding), and the choice between the two kernels.
//
//   o[h] = sum_j p_j v[j, g] / sum_j p_j,  p_j = exp2(c2 <q[h], k[j, g]> - m)     c2 = scale log2(e)
// over the cached positions j <= t with t - j < window or j < sinks (no window: all).
//
// One decoded token brings 12 rows to 512 B (e4m3) or 1 KB (bf16) of K and V per key: bound by
// HBM, 22 or 43 cycles of an SM per key.  So nothing may interrupt the loads: a CTA per SM, whose
// eight warps work alone.  Of every tile of 128 keys a warp takes 16, copies their K and V into a ring
// of its own (16-byte asynchronous copies, 130 KB on their way per SM, zeros for keys that the
// row does not see), and keeps its own running maximum, sum and all 256 dims of O in registers.
// There is no barrier until the item ends, where the eight states are added up.  Measured at batch 64
// of 32768 cached tokens, e4m3: 403 us, 5.3 TB/s, 83 % of the copy rate; what bounds it is the latency
// of the two warps per scheduler that the registers of O leave room for (38 % of the issue slots).
// (A CTA-wide softmax with K and V in registers reached 39 % of the copy rate: it waited at two
// barriers per tile.  Sixteen warps in pairs, each with half of O's dims: 438 us, for the lookups and
// the softmax that both do.)
//   * S = Q K^T and O += P V by mma.m16n8k16, the twelve heads in 16 rows.  S's accumulators are
//     P's operand as they are; the order of the 256 dims inside S, of the dims of O and of a
//     warp's 16 keys is free, and chosen so that a lane's loads are 16 contiguous bytes
//     without bank conflicts (rows of the ring are padded by 16 or 32 bytes for that).
//   * e4m3 codes become fp16, two per conversion instruction, exactly; so Q and P are fp16 too.
//     (Made bf16 by shifts and masks the codes cost 700 integer operations per 16 keys, the bound:
//     568 us at batch 64; as e4m3 operands of m16n8k32 against Q in three e4m3 parts 714 us.)
//     Q is scaled by a power of two per row, its largest value into [2^14, 2^15): exact for
//     values down to 2^-31 of the row's largest, off by 2^-39 of it below.
//     The keys' scales multiply S.  The values' scales multiply P, p 2^e, which is held relative
//     to the row's largest so far (a power of two): 2^-12 relative, or below 2^-18 of the largest an
//     absolute 2^-29 of it.  The running maximum moves by whole powers of two, and this reference
//     with it, since what an early key left in O shrinks as the maximum grows: a late key far above the rest
//     counts by its own size, however small its value's scale is beside theirs.
//   * bf16 pools: P rounds to bf16, 2^-8 relative at most, as in every attention kernel here.
//   * O is rescaled only when a row's maximum grows by more than 2^8.
#include <cuda_fp16.h>

#include "chunk_common.cuh"

namespace qsa {

namespace {

constexpr int kDecWarps = 8, kDecThreads = kDecWarps * 32, kDecKeys = 16 * kDecWarps;
constexpr int kUpRange = 110;   // e4m3: exponents of O's reference, -kUpRange .. kUpRange
constexpr int kDecRestart = 2;  // tiles that another item on a worker costs (5 us, a tile 2.5)

template <bool kFp8>
struct DecCfg {
    static constexpr int kRow = kFp8 ? kD : 2 * kD;                  // bytes of a key's row of one KV head
    static constexpr int kPitchK = kRow + 16, kPitchV = kRow + (kFp8 ? 32 : 16);
    static constexpr int kSlot = 16 * kPitchV;                       // K or V of 16 keys
    static constexpr int kAhead = kFp8 ? 2 : 1;                      // tiles on their way beside the current one
    static constexpr int kRing = 2 * kAhead + 1;
    static constexpr int kOffRing = 16 * 32 * 16;                    // behind Q's fragments
    static constexpr int kMergePitch = kD + 16;                      // floats per row of a warp's state
    static constexpr int kOffStats = kOffRing + kDecWarps * kRing * kSlot;
    static constexpr int kOffScale = kOffStats + 2 * kDecWarps * 16 * (int)sizeof(float);
    static constexpr int kSmem = kOffScale + 16 * (int)sizeof(float);
    static_assert(kDecWarps * kGrp * kMergePitch * 4 <= kDecWarps * kRing * kSlot, "the merge reuses the ring");
    static_assert(kSmem + 2048 <= 232448, "shared memory of one CTA");
};

template <bool kHalf>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1)
{
    if (kHalf)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
            " {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
    else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldmatrix4t(uint32_t addr)
{
    uint4 r;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr) : "memory");
    return r;
}

__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr) : "memory");
    return r;
}

// four e4m3 codes -> the fp16 pairs of codes (0, 1) and (2, 3)
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t &p01, uint32_t &p23)
{
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(p01), "=r"(p23) : "r"(w));
}

__device__ __forceinline__ uint32_t half2(float x, float y)
{
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ float dec_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool kFp8>
__global__ void __launch_bounds__(kDecThreads, 1)
chunk_decode_kernel(const ChunkArgs a, int2 *__restrict__ pieces)
{
    using C = DecCfg<kFp8>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ ChunkShare share;
    __shared__ int64_t scan[2 * kDecWarps];
    __shared__ ChunkLengths lengths;
    pdl_enter();
    lengths.fill(a);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = lane >> 2, c = lane & 3;  // fragment coordinates
    uint4 *sq = reinterpret_cast<uint4 *>(smem);
    float *stats = reinterpret_cast<float *>(smem + C::kOffStats);  // [maximum, sum][warp][16 rows]
    float *states = reinterpret_cast<float *>(smem + C::kOffRing);  // [warp][12 rows][kMergePitch], at an item's end
    const uint32_t ring = smem_u32(smem + C::kOffRing) + warp * C::kRing * C::kSlot;
    chunk_share<1, kDecKeys, kDecThreads, kDecRestart>(a, blockIdx.x, gridDim.x, &share, scan,
                                                       blockIdx.x == 0 ? pieces : nullptr, &lengths);
    int64_t at = share.ts, first = share.first;
    int slot = share.slot;
    const int64_t te = share.te;
    const float c2 = a.scale * 1.4426950408889634f;

    while (at < te) {
        ChunkGroup g = slot == share.slot ? share.g : chunk_group<1, kDecKeys>(ChunkDims(a, &lengths), slot);
        while (at >= first + 2 * (int64_t)g.nt) {  // empty slots between two tokens
            first += 2 * (int64_t)g.nt;
            g = chunk_group<1, kDecKeys>(ChunkDims(a, &lengths), ++slot);
        }
        const int hd = at >= first + g.nt ? 1 : 0;  // KV head
        const int64_t item = first + (int64_t)hd * g.nt;
        const int i0 = (int)(at - item), i1 = te - item < g.nt ? (int)(te - item) : g.nt;
        const int t = g.t0, ns = g.ns, w_tile = g.w_tile;
        const int near = a.window > 0 && a.window <= t ? t - (int)a.window + 1 : 0, sinks = (int)a.sinks;
        const int64_t row_q = (int64_t)g.row0 * kHQ + hd * kGrp;
        const int32_t *table = a.pool.table + (int64_t)g.s * a.pool.max_pages;
        auto sees = [&](int j) -> bool { return j <= t && (j >= near || j < sinks); };
        auto tile = [&](int i) -> int { return (i < ns ? i : w_tile + (i - ns)) * kDecKeys + warp * 16; };

        // A lane looks up key lane mod 16 of the warp's 16.  The page is fetched a tile ahead of its use.
        constexpr int32_t kUnseen = -2;
        int32_t page = kUnseen, row = -1;
        uint32_t off = 0u, sc[C::kAhead + 1];
        auto fetch = [&](int i) {
            page = kUnseen;
            if (i >= i1) return;
            const int j = tile(i) + (lane & 15);
            if (!sees(j)) return;
            const uint32_t p = a.pool.page_of((uint32_t)j, &off);
            page = p < (uint32_t)a.pool.max_pages ? __ldg(table + p) : -1;
        };
        auto resolve = [&]() -> uint32_t {  // -> this lane's scale: of K (lanes 0 .. 15) or V
            row = -1;
            if (page != kUnseen) {
                if ((uint32_t)page < (uint32_t)a.pool.num_pages)
                    row = (page * a.pool.page_size + (int32_t)off) * kHKV + hd;
                else
                    set_device_status(QSA_ERR_DEVICE_CHECK);
            }
            if (!kFp8) return 0u;
            return row >= 0 ? (uint32_t)__ldg((lane < 16 ? a.pool.k_scales : a.pool.v_scales) + row) : 127u;
        };
        uint32_t put = 0, get = 0;  // ring slots
        auto copy = [&](const void *base, int pitch) {
            const uint32_t dst = ring + put * C::kSlot;
            put = put + 1 == C::kRing ? 0 : put + 1;
#pragma unroll
            for (int x = 0; x < (kFp8 ? 8 : 16); ++x) {
                const int key = kFp8 ? 2 * x + (lane >> 4) : x, col = (kFp8 ? lane & 15 : lane) * 16;
                const int32_t r = __shfl_sync(0xffffffffu, row, key);
                const uint8_t *src = static_cast<const uint8_t *>(base) + (int64_t)(r < 0 ? 0 : r) * C::kRow + col;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                             ::"r"(dst + key * pitch + col), "l"(src), "r"(r >= 0 ? 16 : 0) : "memory");
            }
        };
        auto commit = [&]() { asm volatile("cp.async.commit_group;" ::: "memory"); };
        auto arrived = [&]() {  // the oldest half tile on its way
            asm volatile("cp.async.wait_group %0;" ::"n"(C::kRing - 1) : "memory");
            __syncwarp();
        };

        // the first tiles are on their way while Q is laid out
        fetch(i0);
#pragma unroll
        for (int x = 0; x < C::kAhead; ++x) {
            sc[x] = resolve();
            fetch(i0 + x + 1);
            copy(a.pool.k, C::kPitchK);
            commit();
            copy(a.pool.v, C::kPitchV);
            commit();
        }
        // Q's fragments in the order of K's dims; e4m3: as fp16, scaled per row
        if (kFp8) {
            float *qs = reinterpret_cast<float *>(smem + C::kOffScale);
            for (int r = warp; r < 16; r += kDecWarps) {
                float top = 0.f;
                if (r < kGrp) {
                    const uint4 w = __ldg(reinterpret_cast<const uint4 *>(a.q + (row_q + r) * kD + lane * 8));
                    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(v[e] << 16)), fabsf(__uint_as_float(v[e] & 0xFFFF0000u))));
                }
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                // the largest times 2^(14 - E) lies in [2^14, 2^15); an infinity stays one
                const int E = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127);
                if (lane == 0) qs[r] = pow2(E - 14);
            }
            __syncthreads();
        }
        for (int x = tid; x < 16 * 32; x += kDecThreads) {
            const int st = x >> 5, ln = x & 31, r0 = ln >> 2;
            const int d = kFp8 ? (st >> 2) * 64 + (ln & 3) * 16 + (st & 3) * 4 : (st >> 1) * 32 + (ln & 3) * 8 + (st & 1) * 4;
            const __nv_bfloat16 *src = a.q + (row_q + r0) * kD + d;
            uint2 lo = __ldg(reinterpret_cast<const uint2 *>(src));
            uint2 hi = r0 + 8 < kGrp ? __ldg(reinterpret_cast<const uint2 *>(src + 8 * kD)) : make_uint2(0u, 0u);
            if (kFp8) {
                const float *qs = reinterpret_cast<const float *>(smem + C::kOffScale);
                auto halves = [](uint32_t v, float up) -> uint32_t {
                    return half2(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xFFFF0000u) * up);
                };
                const float u0 = 1.f / qs[r0], u1 = 1.f / qs[r0 + 8];  // (powers of two)
                lo = make_uint2(halves(lo.x, u0), halves(lo.y, u0));
                hi = make_uint2(halves(hi.x, u1), halves(hi.y, u1));
            }
            sq[x] = make_uint4(lo.x, hi.x, lo.y, hi.y);
        }
        __syncthreads();

        float q_down[2] = {1.f, 1.f};
        if (kFp8) {
            q_down[0] = reinterpret_cast<const float *>(smem + C::kOffScale)[n];
            q_down[1] = reinterpret_cast<const float *>(smem + C::kOffScale)[n + 8];
        }

        float o[32][4];
#pragma unroll
        for (int j = 0; j < 32; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // of rows n and n + 8
        float up[2] = {INFINITY, INFINITY};                      // e4m3: O is held times this (infinity: still 0)

        for (int i = i0; i < i1; ++i) {
            // K of this tile; a warp's key (x >> 1) + 4 (x & 1) + 8 y is column x of S's part y
            sc[C::kAhead] = resolve();
            fetch(i + C::kAhead + 1);
            __syncwarp();  // all lanes have read the slot that is filled next
            copy(a.pool.k, C::kPitchK);
            commit();
            arrived();
            const uint32_t k_slot = ring + get * C::kSlot + c * 16 + ((n >> 1) + 4 * (n & 1)) * C::kPitchK;
            get = get + 1 == C::kRing ? 0 : get + 1;
            float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}, s2[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int x = 0; x < (kFp8 ? 4 : 8); ++x) {
                uint4 w[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) w[y] = lds16(k_slot + y * 8 * C::kPitchK + x * 64);
#pragma unroll
                for (int z = 0; z < (kFp8 ? 4 : 2); ++z) {
                    const uint4 qa = sq[(x * (kFp8 ? 4 : 2) + z) * 32 + lane];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        uint32_t b0, b1;
                        if (kFp8) {
                            codes_to_half(z == 0 ? w[y].x : (z == 1 ? w[y].y : (z == 2 ? w[y].z : w[y].w)), b0, b1);
                        } else {
                            b0 = z == 0 ? w[y].x : w[y].z;
                            b1 = z == 0 ? w[y].y : w[y].w;
                        }
                        // even and odd steps apart: shorter chains of dependent products
                        mma_16816<kFp8>((z & 1) ? s2[y] : s[y], qa, b0, b1);
                    }
                }
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[y][e] = (s[y][e] + s2[y][e]) * (kFp8 ? q_down[e >> 1] : 1.f);
            // scale, mask, row maxima: this lane's keys are c, c + 4 (part 0), c + 8, c + 12 (part 1)
            const int j0 = tile(i);
            const bool whole = j0 + 15 <= t && (j0 >= near || j0 + 16 <= sinks);
            float vs[2][2], mx[2];
            const float own = kFp8 ? scale_of_byte(sc[0]) : 1.f;  // of key lane mod 16: K's, from lane 16 on V's
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float f = c2;
                    if (kFp8) {
                        f *= __shfl_sync(0xffffffffu, own, c + 4 * x + 8 * y);
                        vs[y][x] = __shfl_sync(0xffffffffu, own, c + 4 * x + 8 * y + 16);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) s[y][2 * h + x] *= f;
                }
            if (!whole) {
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        if (!sees(j0 + c + 4 * x + 8 * y)) s[y][x] = s[y][2 + x] = -INFINITY;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
                mx[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
            bool grow = false;
            float base[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                if (kFp8) mx[h] = ceilf(mx[h]);
                grow |= m[h] != -INFINITY && mx[h] > m[h] + 8.f;
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float to = fmaxf(m[h], mx[h]);
                    float f;
                    if (kFp8) {
                        // the maximum is a whole number here: O's reference moves with it, and O stays as it is
                        // held (but where the reference would leave its range)
                        const int grown = m[h] == -INFINITY ? 0 : (int)fminf(to - m[h], 400.f);
                        const int e = (int)(__float_as_uint(up[h]) >> 23) - 127;
                        const int moved = up[h] == INFINITY ? 0 : min(grown, kUpRange - e);
                        l[h] *= grown > 126 ? 0.f : pow2(-grown);
                        if (moved > 0) up[h] = pow2(e + moved);
                        f = grown - moved > 126 ? 0.f : pow2(moved - grown);
                    } else {
                        f = m[h] == -INFINITY ? 1.f : dec_ex2(m[h] - to);
                        l[h] *= f;
                    }
                    m[h] = to;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        o[j][2 * h] *= f;
                        o[j][2 * h + 1] *= f;
                    }
                }
            }
            float p[2][2][2], px[2] = {0.f, 0.f};  // [row half][part][key], a row's largest
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (m[h] == -INFINITY) m[h] = mx[h];
                base[h] = m[h] == -INFINITY ? 0.f : m[h];  // no visible key yet
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float e = dec_ex2(s[y][2 * h + x] - base[h]);
                        l[h] += e;
                        // (a key that the row does not see has the scale 1; a NaN scale of one that it
                        // sees makes a NaN of the row however small its probability)
                        p[h][y][x] = kFp8 ? e * vs[y][x] : e;
                        px[h] = fmaxf(px[h], p[h][y][x]);
                    }
            }
            if (kFp8) {
                // p 2^e relative to 2^-up of its row: at most 2^15, at 2^4 when the reference is set
                if (__any_sync(0xffffffffu, px[0] * up[0] > 32768.f || px[1] * up[1] > 32768.f)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        px[h] = fmaxf(px[h], __shfl_xor_sync(0xffffffffu, px[h], 1));
                        px[h] = fmaxf(px[h], __shfl_xor_sync(0xffffffffu, px[h], 2));
                        if (px[h] * up[h] > 32768.f) {
                            const float to = pow2(min(max(131 - (int)(__float_as_uint(px[h]) >> 23), -kUpRange), kUpRange));
                            const float f = up[h] == INFINITY ? 0.f : to / up[h];  // (powers of two)
                            up[h] = to;
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                o[j][2 * h] *= f;
                                o[j][2 * h + 1] *= f;
                            }
                        }
                    }
                }
            }
            uint32_t pa[2][2];  // [part][row half]
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    if (kFp8) {
                        const float u = up[h] == INFINITY ? 0.f : up[h];
                        pa[y][h] = half2(p[h][y][0] * u, p[h][y][1] * u);
                    } else {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(p[h][y][0], p[h][y][1]);
                        pa[y][h] = *reinterpret_cast<const uint32_t *>(&b);
                    }
                }
            const uint4 pf = make_uint4(pa[0][0], pa[0][1], pa[1][0], pa[1][1]);
            // V
            __syncwarp();
            copy(a.pool.v, C::kPitchV);
            commit();
            arrived();
            const uint32_t v_slot = ring + get * C::kSlot;
            get = get + 1 == C::kRing ? 0 : get + 1;
            if (kFp8) {
                // dims 128 x + 16 n .. + 15 of the keys c, c + 4, c + 8, c + 12: 16 column tiles
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint4 w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = lds16(v_slot + (c + 4 * e) * C::kPitchV + x * 128 + n * 16);
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        uint32_t k[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) k[e] = z == 0 ? w[e].x : (z == 1 ? w[e].y : (z == 2 ? w[e].z : w[e].w));
                        uint32_t b0[4], b1[4];
                        codes_to_half(__byte_perm(k[0], k[1], 0x5140), b0[0], b0[1]);
                        codes_to_half(__byte_perm(k[0], k[1], 0x7362), b0[2], b0[3]);
                        codes_to_half(__byte_perm(k[2], k[3], 0x5140), b1[0], b1[1]);
                        codes_to_half(__byte_perm(k[2], k[3], 0x7362), b1[2], b1[3]);
#pragma unroll
                        for (int b = 0; b < 4; ++b) mma_16816<kFp8>(o[x * 16 + z * 4 + b], pf, b0[b], b1[b]);
                    }
                }
            } else {
                // matrices of 8 keys by 8 dims, transposed: rows are the keys of S's columns
                const int kr = lane & 7, part = (lane >> 3) & 1;
                const uint32_t src = v_slot + ((kr >> 1) + 4 * (kr & 1) + 8 * part) * C::kPitchV + (lane >> 4) * 16;
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const uint4 b = ldmatrix4t(src + x * 32);
                    mma_16816<kFp8>(o[2 * x], pf, b.x, b.y);
                    mma_16816<kFp8>(o[2 * x + 1], pf, b.z, b.w);
                }
            }
#pragma unroll
            for (int x = 0; x < C::kAhead; ++x) sc[x] = sc[x + 1];
        }
        asm volatile("cp.async.wait_all;" ::: "memory");

        // the eight warps' states, through shared memory in the place of their rings
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (kFp8) {
                const float down = up[h] == INFINITY ? 1.f : 1.f / up[h];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    o[j][2 * h] *= down;
                    o[j][2 * h + 1] *= down;
                }
            }
            if (c == 0) {
                stats[warp * 16 + n + 8 * h] = m[h];
                stats[(kDecWarps + warp) * 16 + n + 8 * h] = l[h];
            }
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = n + 8 * h;
            if (r >= kGrp) continue;
            float *dst = states + (warp * kGrp + r) * C::kMergePitch;
            if (kFp8) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const int j = x * 16 + z * 4;
                            *reinterpret_cast<float4 *>(dst + x * 128 + (2 * c + e) * 16 + ((z + c) & 3) * 4) =  // (no bank conflicts)
                                make_float4(o[j][2 * h + e], o[j + 1][2 * h + e], o[j + 2][2 * h + e], o[j + 3][2 * h + e]);
                        }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    *reinterpret_cast<float2 *>(dst + 8 * j + 2 * c) = make_float2(o[j][2 * h], o[j][2 * h + 1]);
            }
        }
        __syncthreads();
        const bool complete = i0 == 0 && i1 == g.nt;
        const int64_t piece = 2 * (int64_t)blockIdx.x + (i0 == 0 ? 1 : 0);
        // a thread adds up 12 dims: four of rows tid / 64, + 4 and + 8
        for (int r = tid >> 6; r < kGrp; r += 4) {
            const int d = (tid & 63) * 4, at_d = kFp8 ? (d & ~15) + (((d >> 2) + (d >> 5)) & 3) * 4 : d;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kDecWarps; ++w) top = fmaxf(top, stats[w * 16 + r]);
            const float b = top == -INFINITY ? 0.f : top;
            float L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kDecWarps; ++w) {
                const float f = exp2f(stats[w * 16 + r] - b);
                const float4 x = *reinterpret_cast<const float4 *>(states + (w * kGrp + r) * C::kMergePitch + at_d);
                L = fmaf(f, stats[(kDecWarps + w) * 16 + r], L);
                acc.x = fmaf(f, x.x, acc.x);
                acc.y = fmaf(f, x.y, acc.y);
                acc.z = fmaf(f, x.z, acc.z);
                acc.w = fmaf(f, x.w, acc.w);
            }
            const bool none = L == 0.f;  // (a NaN is not)
            const float inv = none ? 0.f : 1.f / L;
            const float lse2 = none ? -INFINITY : top + log2f(L);
            acc = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            if (complete) {
                const __nv_bfloat162 h0 = __floats2bfloat162_rn(acc.x, acc.y), h1 = __floats2bfloat162_rn(acc.z, acc.w);
                *reinterpret_cast<uint2 *>(a.o + (row_q + r) * kD + d) =
                    make_uint2(*reinterpret_cast<const uint32_t *>(&h0), *reinterpret_cast<const uint32_t *>(&h1));
                if (a.lse != nullptr && d == 0) a.lse[row_q + r] = lse2 * 0.6931471805599453f;
            } else {
                *reinterpret_cast<float4 *>(a.ws + (piece * kGrp + r) * kD + d) = acc;
                if (d == 0) a.ws[2 * (int64_t)gridDim.x * kGrp * kD + piece * kGrp + r] = lse2;
            }
        }
        __syncthreads();  // the next item's copies overwrite the states
        at = item + i1;
    }
}

constexpr int64_t kMaxWorkers = 160;  // CTAs of the kernel, at most (the workspace's bound)

size_t dec_pieces_offset() { return (size_t)(2 * kMaxWorkers) * kGrp * (kD + 1) * sizeof(float); }

template <bool kFp8>
cudaError_t launch_decode(const ChunkArgs &a, cudaStream_t stream)
{
    int2 *pieces = reinterpret_cast<int2 *>(reinterpret_cast<uint8_t *>(a.ws) + dec_pieces_offset());
    int64_t workers = num_sms();
    if (workers > kMaxWorkers) workers = kMaxWorkers;
    cudaError_t e = set_smem_attr_once(reinterpret_cast<const void *>(chunk_decode_kernel<kFp8>), DecCfg<kFp8>::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(chunk_decode_kernel<kFp8>, dim3((unsigned)workers), dim3(kDecThreads), DecCfg<kFp8>::kSmem, stream, a,
                   pieces);
    if (e != cudaSuccess) return e;
    return launch_chunk_merge<1, kDecKeys, kDecRestart>(a, pieces, workers, stream);
}

}  // namespace

size_t chunk_workspace_bytes(int batch, int64_t total_q)
{
    const size_t own = dec_pieces_offset() + (size_t)chunk_slots<1>(total_q, batch) * 2 * sizeof(int2);
    const size_t tc = chunk_tc_workspace_bytes(batch, total_q);
    return own > tc ? own : tc;
}

// Single tokens (max_len_q <= 1): e4m3 pages here, 403 us against 790 us of the tensor-core kernel at batch
// 64 of 32768 cached tokens, whose warps that make bf16 of the codes are its bound; bf16 pages there, but for a few
// tokens, where its longer start counts.  Here and there, caches not in L2: one token over 1000, 8192 or 32768 cached
// 16.4 and 20.5, 22.5 and 26.6, 30.7 and 36.9 us; seven 22.5 and 24.6, 43.0 and 43.0, 110.6 and 102.4 us; ten 26.6 and
// 28.7, 57.3 and 57.3, 147.5 and 135.2 us; 32 36.9 and 34.8, 127.0 and 116.7, 387 and 346 us.
cudaError_t launch_chunk_attn(const ChunkArgs &a, cudaStream_t stream)
{
    if (a.total_q <= 0) return cudaSuccess;
    if (a.max_len_q <= 1 && a.pool.fp8) return launch_decode<true>(a, stream);
    if (a.max_len_q <= 1 && a.total_q < 8) return launch_decode<false>(a, stream);
    return launch_chunk_tc(a, stream);
}

}  // namespace qsa
