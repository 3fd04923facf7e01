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
// Angles, their cosines and sines in fp64 (a position of 2^20 leaves an fp32 angle off by
// 0.06 rad), rounded to fp32 once; the products in fp32, one rounding to bf16.
//
// Bound by HBM: 26 heads x 512 B read and written per token.  A CTA takes 8 tokens at a
// time: 256 threads fill a table of their cosines and sines, shared by the 26 heads (one fp64
// sincos per 26 x 2 values), then a warp rotates a (token, head) row, 16 B per lane, the
// partner dims from the lane h / 8 away (any other h: from a copy of the row in shared memory).
#include "kernels.cuh"

namespace qsa {

namespace {

constexpr int kRopeWarps = 8, kRopeTok = 8, kMaxPairs = 128;
constexpr int kHQ = 24, kHKV = 2, kD = 256;

template <bool kAligned>
__global__ void __launch_bounds__(kRopeWarps * 32)
rope_axes_kernel(const __nv_bfloat16 *q, const __nv_bfloat16 *k, const int32_t *__restrict__ pos,
                 int64_t total, int s0, int s1, int s2, double log2_base, int interleaved, int inverse,
                 __nv_bfloat16 *q_out, __nv_bfloat16 *k_out)
{
    __shared__ double freq[kMaxPairs];
    __shared__ int8_t axis[kMaxPairs];
    __shared__ float2 cs[kRopeTok][kMaxPairs];  // (cos, sin)
    __shared__ __nv_bfloat16 copy[kAligned ? 1 : kRopeWarps][kAligned ? 1 : kD];
    pdl_enter();
    const int h = s0 + s1 + s2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < h; i += kRopeWarps * 32) {
        freq[i] = exp2(-log2_base * (double)i / (double)h);
        axis[i] = interleaved ? (i % 3 == 1 && i / 3 < s1 ? 1 : (i % 3 == 2 && i / 3 < s2 ? 2 : 0))
                              : (i >= s0 ? (i >= s0 + s1 ? 2 : 1) : 0);
    }
    const int hq = q != nullptr ? kHQ : 0, heads = hq + (k != nullptr ? kHKV : 0);
    // the lanes whose dims are read and written: all, or in place only those that rotate
    for (int64_t t0 = (int64_t)blockIdx.x * kRopeTok; t0 < total; t0 += (int64_t)gridDim.x * kRopeTok) {
        const int nt = (int)(total - t0 < kRopeTok ? total - t0 : kRopeTok);
        __syncthreads();  // freq is there; the previous tokens' table has been read
        for (int x = threadIdx.x; x < nt * h; x += kRopeWarps * 32) {
            const int t = x / h, i = x % h;
            double sn, c;
            sincos((double)__ldg(pos + axis[i] * total + t0 + t) * freq[i], &sn, &c);
            cs[t][i] = make_float2((float)c, inverse ? -(float)sn : (float)sn);
        }
        __syncthreads();
        for (int x = warp; x < nt * heads; x += kRopeWarps) {
            const int t = x / heads, hd = x % heads;
            const bool is_q = hd < hq;
            const int64_t off = (is_q ? ((t0 + t) * kHQ + hd) : ((t0 + t) * kHKV + (hd - hq))) * (int64_t)kD + lane * 8;
            const __nv_bfloat16 *src = (is_q ? q : k) + off;
            __nv_bfloat16 *dst = (is_q ? q_out : k_out) + off;
            const bool mine = src != dst || lane * 8 < 2 * h;
            uint4 raw = make_uint4(0u, 0u, 0u, 0u);
            if (mine) raw = *reinterpret_cast<const uint4 *>(src);
            uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
            if (kAligned) {
                const int hl = h / 8;  // lanes of the low half
                const bool lo = lane < hl, rot = lane < 2 * hl;
                const int partner = lo ? lane + hl : (rot ? lane - hl : lane);
                const int p0 = (lo ? lane : lane - hl) * 8;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t o = __shfl_sync(0xffffffffu, w[j], partner);
                    if (rot) {
                        const float4 f = *reinterpret_cast<const float4 *>(&cs[t][p0 + 2 * j]);
                        const float x0 = __uint_as_float(w[j] << 16), x1 = __uint_as_float(w[j] & 0xFFFF0000u);
                        const float y0 = __uint_as_float(o << 16), y1 = __uint_as_float(o & 0xFFFF0000u);
                        const float r0 = lo ? x0 * f.x - y0 * f.y : y0 * f.y + x0 * f.x;
                        const float r1 = lo ? x1 * f.z - y1 * f.w : y1 * f.w + x1 * f.z;
                        const __nv_bfloat162 b = __floats2bfloat162_rn(r0, r1);
                        w[j] = *reinterpret_cast<const uint32_t *>(&b);
                    }
                }
            } else {
                __nv_bfloat16 *row = copy[warp];
                __syncwarp();
                *reinterpret_cast<uint4 *>(row + lane * 8) = raw;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float r[2] = {__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u)};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int d = lane * 8 + 2 * j + e;
                        if (d < h) {
                            const float2 f = cs[t][d];
                            r[e] = r[e] * f.x - __bfloat162float(row[d + h]) * f.y;
                        } else if (d < 2 * h) {
                            const float2 f = cs[t][d - h];
                            r[e] = __bfloat162float(row[d - h]) * f.y + r[e] * f.x;
                        }
                    }
                    const __nv_bfloat162 b = __floats2bfloat162_rn(r[0], r[1]);
                    const uint32_t nw = *reinterpret_cast<const uint32_t *>(&b);
                    // dims that do not rotate keep their bits (a NaN's payload too)
                    const int d0 = lane * 8 + 2 * j;
                    if (d0 + 1 < 2 * h) w[j] = nw;
                    else if (d0 < 2 * h) w[j] = (w[j] & 0xFFFF0000u) | (nw & 0xFFFFu);
                }
            }
            if (mine) *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

}  // namespace

cudaError_t launch_rope_axes(const __nv_bfloat16 *q, const __nv_bfloat16 *k, const int32_t *pos, int64_t total, int s0,
                             int s1, int s2, float base, bool interleaved, bool inverse, __nv_bfloat16 *q_out,
                             __nv_bfloat16 *k_out, cudaStream_t stream)
{
    if (total <= 0 || (q == nullptr && k == nullptr)) return cudaSuccess;
    const int64_t groups = (total + kRopeTok - 1) / kRopeTok, most = (int64_t)num_sms() * 8;
    const bool aligned = (s0 + s1 + s2) % 8 == 0;
    return launch_pdl(aligned ? rope_axes_kernel<true> : rope_axes_kernel<false>,
                      dim3((unsigned)(groups < most ? groups : most)), dim3(kRopeWarps * 32), 0, stream, q, k, pos,
                      total, s0, s1, s2, log2((double)base), interleaved ? 1 : 0, inverse ? 1 : 0, q_out, k_out);
}

}  // namespace qsa
