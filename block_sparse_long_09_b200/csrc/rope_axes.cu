// rope_axes.cu -- rotary positions with three axes (time, height, width) for the
// attention's q and k, and the gradient of that rotation.
//
// Pair i < h = s0 + s1 + s2 of a head is the dims (i, i + h); it rotates by
//   theta = pos[axis(i)] * base^(-i / h)
//   (a, b) -> (a cos - b sin, a sin + b cos),        dims from 2 h on stay as they are.
// axis(i): s0 pairs of axis 0, then s1 of axis 1, then s2 of axis 2; interleaved, the s1
// pairs 1, 4, 7, ... are axis 1, the s2 pairs 2, 5, 8, ... axis 2 and the rest axis 0.
// The rotation is orthogonal, so the gradient of its input is the rotation by -theta of
// its output's gradient (kInverse).
//
// Angles in fp64 (a position of 2^20 leaves an fp32 angle off by 0.06 rad), as multiples of pi, so
// that no position needs a long argument reduction; cosines and sines rounded to fp32 once, the
// products in fp32, one rounding to bf16.
//
// Bound by HBM: 26 heads x 512 B read and written per token.  A warp per token: its lanes
// compute the token's cosines and sines, exchange them through shared memory, and keep the ones of
// their 8 dims for all heads; the rows come four at a time.  (A table per 8 tokens shared by a
// CTA, its barriers in the way of the loads: 3.8 TB/s at 16384 tokens.)  Few tokens: up to four
// warps share a token's heads, so that the SMs have loads enough on their way.
#include "kernels.cuh"

namespace qsa {

namespace {

constexpr int kRopeWarps = 4, kMaxPairs = 128, kRopeRows = 4;
constexpr int kHQ = 24, kHKV = 2, kD = 256;

template <bool kAligned>
__global__ void __launch_bounds__(kRopeWarps * 32)
rope_axes_kernel(const __nv_bfloat16 *q, const __nv_bfloat16 *k, const int32_t *__restrict__ pos,
                 int64_t total, int s0, int s1, int s2, double log2_base, int interleaved, int inverse, int parts,
                 __nv_bfloat16 *q_out, __nv_bfloat16 *k_out)
{
    __shared__ float2 table[kRopeWarps][kMaxPairs];  // (cos, sin) of a warp's token
    __shared__ __nv_bfloat16 copy[kAligned ? 1 : kRopeWarps][kAligned ? 1 : kRopeRows][kAligned ? 8 : kD];
    pdl_enter();
    const int h = s0 + s1 + s2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kRopeWarps + warp, token = unit / parts;
    if (token >= total) return;  // uniform for the warp
    const int hq = q != nullptr ? kHQ : 0, heads = hq + (k != nullptr ? kHKV : 0);
    const int per = (heads + parts - 1) / parts, first = (int)(unit - token * parts) * per;
    const int last = first + per < heads ? first + per : heads;
    // row x of the token, this lane's 8 dims
    auto offset = [&](int x) -> int64_t {
        return (x < hq ? token * kHQ + x : token * kHKV + (x - hq)) * (int64_t)kD + lane * 8;
    };
    // the first rows are on their way while the angles are computed; in place only dims that rotate move
    const bool rot_q = q != q_out || lane * 8 < 2 * h, rot_k = k != k_out || lane * 8 < 2 * h;
    uint4 raw[kRopeRows];
    auto load = [&](int x0) {
#pragma unroll
        for (int u = 0; u < kRopeRows; ++u) {
            const int x = x0 + u;
            raw[u] = make_uint4(0u, 0u, 0u, 0u);
            if (x < last && (x < hq ? rot_q : rot_k)) raw[u] = *reinterpret_cast<const uint4 *>((x < hq ? q : k) + offset(x));
        }
    };
    load(first);
    for (int i = lane; i < h; i += 32) {
        const int axis = interleaved ? (i % 3 == 1 && i / 3 < s1 ? 1 : (i % 3 == 2 && i / 3 < s2 ? 2 : 0))
                                     : (i >= s0 ? (i >= s0 + s1 ? 2 : 1) : 0);
        const double freq = exp2(-log2_base * (double)i / (double)h) * 0.31830988618379067154;  // 1 / pi
        double sn, cs;
        sincospi((double)__ldg(pos + axis * total + token) * freq, &sn, &cs);
        table[warp][i] = make_float2((float)cs, inverse ? -(float)sn : (float)sn);
    }
    __syncwarp();
    // of dim lane * 8 + e: cos, and sin with the sign that the partner dim has in it
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int d = lane * 8 + e;
        const float2 f = d < 2 * h ? table[warp][d < h ? d : d - h] : make_float2(1.f, 0.f);
        cs[e] = f.x;
        sn[e] = d < h ? -f.y : f.y;
    }
    const int hl = h / 8;  // aligned: lanes of the low half
    const int partner = lane < hl ? lane + hl : (lane < 2 * hl ? lane - hl : lane);

    for (int x0 = first; x0 < last; x0 += kRopeRows) {
        uint32_t w[kRopeRows][4];
#pragma unroll
        for (int u = 0; u < kRopeRows; ++u) {
            w[u][0] = raw[u].x;
            w[u][1] = raw[u].y;
            w[u][2] = raw[u].z;
            w[u][3] = raw[u].w;
            if (!kAligned) *reinterpret_cast<uint4 *>(&copy[warp][u][lane * 8]) = raw[u];
        }
        if (x0 + kRopeRows < last) load(x0 + kRopeRows);
        if (!kAligned) __syncwarp();
#pragma unroll
        for (int u = 0; u < kRopeRows; ++u) {
            const int x = x0 + u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float y0, y1;  // the partner dims
                if (kAligned) {
                    const uint32_t o = __shfl_sync(0xffffffffu, w[u][j], partner);
                    y0 = __uint_as_float(o << 16);
                    y1 = __uint_as_float(o & 0xFFFF0000u);
                } else {
                    const int d = lane * 8 + 2 * j;
                    const __nv_bfloat16 *r = copy[warp][u];
                    y0 = d < 2 * h ? __bfloat162float(r[d < h ? d + h : d - h]) : 0.f;
                    y1 = d + 1 < 2 * h ? __bfloat162float(r[d + 1 < h ? d + 1 + h : d + 1 - h]) : 0.f;
                }
                const float x0f = __uint_as_float(w[u][j] << 16), x1f = __uint_as_float(w[u][j] & 0xFFFF0000u);
                const __nv_bfloat162 b = __floats2bfloat162_rn(x0f * cs[2 * j] + y0 * sn[2 * j],
                                                               x1f * cs[2 * j + 1] + y1 * sn[2 * j + 1]);
                const uint32_t nw = *reinterpret_cast<const uint32_t *>(&b);
                // dims that do not rotate keep their bits (a NaN's payload too)
                const int d = lane * 8 + 2 * j;
                if (d + 1 < 2 * h) w[u][j] = nw;
                else if (d < 2 * h) w[u][j] = (w[u][j] & 0xFFFF0000u) | (nw & 0xFFFFu);
            }
            if (x < last && (x < hq ? rot_q : rot_k))
                *reinterpret_cast<uint4 *>((x < hq ? q_out : k_out) + offset(x)) = make_uint4(w[u][0], w[u][1], w[u][2], w[u][3]);
        }
        if (!kAligned) __syncwarp();  // the copies have been read
    }
}

}  // namespace

cudaError_t launch_rope_axes(const __nv_bfloat16 *q, const __nv_bfloat16 *k, const int32_t *pos, int64_t total, int s0,
                             int s1, int s2, float base, bool interleaved, bool inverse, __nv_bfloat16 *q_out,
                             __nv_bfloat16 *k_out, cudaStream_t stream)
{
    if (total <= 0 || (q == nullptr && k == nullptr)) return cudaSuccess;
    // warps per token: enough for 16 per SM (a second one costs its angles again)
    const int64_t want = (int64_t)num_sms() * 16;
    const int parts = q == nullptr || total >= want ? 1 : (2 * total >= want ? 2 : 4);
    const int64_t grid = (total * parts + kRopeWarps - 1) / kRopeWarps;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    const bool aligned = (s0 + s1 + s2) % 8 == 0;
    return launch_pdl(aligned ? rope_axes_kernel<true> : rope_axes_kernel<false>, dim3((unsigned)grid),
                      dim3(kRopeWarps * 32), 0, stream, q, k, pos, total, s0, s1, s2, log2((double)base),
                      interleaved ? 1 : 0, inverse ? 1 : 0, parts, q_out, k_out);
}

}  // namespace qsa
