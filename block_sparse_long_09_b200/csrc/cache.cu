// cache.cu -- writing new tokens into a paged K/V pool and reading a range of tokens back.
//
// Formats of a pool's rows (256 values of one token and KV head):
//   bf16   the values as they are
//   e4m3   x ~ code * 2^e with one exponent per row, the smallest e >= -127 with
//          max|x| <= 448 * 2^e, stored as the byte e + 127; code = x * 2^-e rounded to
//          nearest even.  A power of two makes both directions exact but for that one
//          rounding: x * 2^-e is exact in fp32, code * 2^e is exact in bf16.  A row that is
//          written, read back and written again has the same values; its codes and byte are
//          the same too, or the byte is one less and the codes stand for twice as much (a maximum just
//          above 448 * 2^e that was rounded down to it: 450 is held as 224 * 2, and 448 then as
//          448 * 1).  A scale max|x| / 448 would use the codes' last factor of two at most,
//          for a division per value and a second rounding.
//          A row that holds an infinity or a NaN is stored as the byte 255 with zero codes
//          and reads back as NaN.  The codes that are written are finite; a pool filled otherwise may
//          hold the type's NaN codes, which read back as NaN.
//
// Bound by HBM in both directions (2 KB of bf16 and 1028 B of e4m3 per token).  Writing: a warp
// per (token, K or V): both heads' 512 values are 16 per lane, 32 bytes of bf16 memory and one
// 16-byte access to codes; the row maximum is four shuffles over 16 lanes.  The loads of a
// token's values do not wait for its page lookup.  Reading: a warp takes K or V of four tokens, whose
// lookups its lanes make side by side (a token per warp: 4.0 TB/s of 131072 e4m3 tokens).
#include <cuda_fp8.h>

#include "kernels.cuh"

namespace qsa {

namespace {

constexpr int kCacheWarps = 8;
constexpr int kReadTok = 4;    // tokens that a warp reads at a time
constexpr int kRowVals = 512;  // values of one token: 2 KV heads x 256

// pool row of position tok of sequence s, or -1 when the table has no valid page for it
__device__ __forceinline__ int64_t pool_row(const CachePool &c, int64_t s, int64_t tok)
{
    if (tok < 0) return -1;
    uint32_t off;
    const uint32_t j = c.page_of((uint32_t)tok, &off);  // (a length is an int32)
    const int32_t page = j < (uint32_t)c.max_pages ? __ldg(c.table + s * c.max_pages + j) : -1;
    if (page < 0 || page >= c.num_pages) return -1;
    return (int64_t)page * c.page_size + off;
}

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

template <bool kFp8>
__global__ void __launch_bounds__(kCacheWarps * 32)
cache_write_kernel(const __nv_bfloat16 *__restrict__ k, const __nv_bfloat16 *__restrict__ v, const CachePool c,
                   const int32_t *__restrict__ cu_q, const int32_t *__restrict__ cu_k, int batch, int64_t total_q)
{
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kCacheWarps + (threadIdx.x >> 5);
    if (item >= 2 * total_q) return;  // uniform for the warp
    const int64_t i = item >> 1;
    const bool is_v = item & 1;
    const uint4 *src = reinterpret_cast<const uint4 *>((is_v ? v : k) + i * kRowVals) + (kFp8 ? 2 * lane : lane);
    const uint4 a = __ldcs(src), b = __ldcs(src + (kFp8 ? 1 : 32));
    if (i < __ldg(cu_q) || i >= __ldg(cu_q + batch)) return;  // not a sequence's row
    const int s = find_seq(cu_q, batch, i);
    const int64_t q0 = __ldg(cu_q + s), Lq = (int64_t)__ldg(cu_q + s + 1) - q0;
    const int64_t Lk = (int64_t)__ldg(cu_k + s + 1) - __ldg(cu_k + s);
    const int64_t row = pool_row(c, s, Lk - Lq + (i - q0));
    if (row < 0) {
        if (lane == 0) set_device_status(QSA_ERR_DEVICE_CHECK);
        return;
    }
    if (!kFp8) {
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(is_v ? c.v : c.k) + row * kRowVals) + lane;
        dst[0] = a;
        dst[32] = b;
        return;
    }
    // max|x| as bf16 bits: magnitudes order like their bits, NaNs above infinity
    uint32_t m = max2(max2(max2(a.x & 0x7FFF7FFFu, a.y & 0x7FFF7FFFu), max2(a.z & 0x7FFF7FFFu, a.w & 0x7FFF7FFFu)),
                      max2(max2(b.x & 0x7FFF7FFFu, b.y & 0x7FFF7FFFu), max2(b.z & 0x7FFF7FFFu, b.w & 0x7FFF7FFFu)));
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = max2(m, __shfl_xor_sync(0xffffffffu, m, off));
    const uint32_t top = (m & 0xFFFFu) > (m >> 16) ? (m & 0xFFFFu) : (m >> 16);
    const bool finite = top < 0x7F80u;
    // top = (1 + f / 128) 2^(E - 127); 448 = 1.75 * 2^8, so e = E - 135, one more when f > 96
    const int byte0 = (int)(top >> 7) - 8 + ((top & 0x7Fu) > 96u ? 1 : 0);
    const int byte = finite ? (byte0 > 0 ? byte0 : 0) : 255;
    const float inv = finite ? __uint_as_float((uint32_t)(254 - byte) << 23) : 0.f;  // 2^-e
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t r = 0u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t x = w[2 * j + h];
            const float2 f = make_float2(__uint_as_float(x << 16) * inv, __uint_as_float(x & 0xFFFF0000u) * inv);
            r |= (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3) << (16 * h);
        }
        out[j] = finite ? r : 0u;  // an infinity times zero is a NaN
    }
    *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(is_v ? c.v : c.k) + row * kRowVals + lane * 16) =
        make_uint4(out[0], out[1], out[2], out[3]);
    if ((lane & 15) == 0) (is_v ? c.v_scales : c.k_scales)[row * 2 + (lane >> 4)] = (uint8_t)byte;
}

// two e4m3 codes' values (the type's NaN codes, 0x7F and 0xFF, among them)
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two)
{
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3)));
}

template <bool kFp8>
__global__ void __launch_bounds__(kCacheWarps * 32)
cache_read_kernel(const CachePool c, const int32_t *__restrict__ cu_k, const int32_t *__restrict__ tok_begin,
                  const int32_t *__restrict__ cu_out, int batch, int64_t total_out, __nv_bfloat16 *__restrict__ k_out,
                  __nv_bfloat16 *__restrict__ v_out)
{
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kCacheWarps + (threadIdx.x >> 5);
    const int64_t i0 = (item >> 1) * kReadTok;
    if (i0 >= total_out) return;  // uniform for the warp
    const bool is_v = item & 1;
    // lane u looks up token u: its pool row, -1 a token that the cache does not hold, -2 no sequence's row
    int64_t mine = -2;
    if (lane < kReadTok && i0 + lane < total_out && i0 + lane >= __ldg(cu_out) && i0 + lane < __ldg(cu_out + batch)) {
        const int64_t i = i0 + lane;
        const int s = find_seq(cu_out, batch, i);
        const int64_t Lk = (int64_t)__ldg(cu_k + s + 1) - __ldg(cu_k + s);
        const int64_t tok = (tok_begin != nullptr ? (int64_t)__ldg(tok_begin + s) : 0) + (i - __ldg(cu_out + s));
        mine = tok < Lk ? pool_row(c, s, tok) : -1;
        if (mine < 0) set_device_status(QSA_ERR_DEVICE_CHECK);
    }
    const void *pages = is_v ? c.v : c.k;
    int64_t row[kReadTok];
    uint4 a[kReadTok], b[kReadTok];
    uint32_t byte[kReadTok];
#pragma unroll
    for (int u = 0; u < kReadTok; ++u) {
        row[u] = __shfl_sync(0xffffffffu, mine, u);
        a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
        byte[u] = 127u;
        if (row[u] < 0) continue;
        if (kFp8) {
            a[u] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(pages) + row[u] * kRowVals + lane * 16));
            byte[u] = __ldg((is_v ? c.v_scales : c.k_scales) + row[u] * 2 + (lane >> 4));
        } else {
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(pages) + row[u] * kRowVals) + lane;
            a[u] = __ldcs(src);
            b[u] = __ldcs(src + 32);
        }
    }
#pragma unroll
    for (int u = 0; u < kReadTok; ++u) {
        if (row[u] == -2) continue;
        __nv_bfloat16 *dst = (is_v ? v_out : k_out) + (i0 + u) * kRowVals;
        if (!kFp8) {
            __stcs(reinterpret_cast<uint4 *>(dst) + lane, a[u]);
            __stcs(reinterpret_cast<uint4 *>(dst) + lane + 32, b[u]);
            continue;
        }
        const float scale = scale_of_byte(byte[u]);
        const uint32_t w[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
        uint32_t out[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 x = e4m3x2_to_float2((w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
            const __nv_bfloat162 p = __floats2bfloat162_rn(x.x * scale, x.y * scale);
            out[j] = *reinterpret_cast<const uint32_t *>(&p);
        }
        // a lane's 16 values are two pieces of 16 bytes; two lanes exchange one, so that a store covers
        // whole 32-byte sectors
        const bool odd = lane & 1;
        uint4 lo = make_uint4(out[0], out[1], out[2], out[3]), hi = make_uint4(out[4], out[5], out[6], out[7]);
        const uint4 give = odd ? lo : hi;
        uint4 got;
        got.x = __shfl_xor_sync(0xffffffffu, give.x, 1);
        got.y = __shfl_xor_sync(0xffffffffu, give.y, 1);
        got.z = __shfl_xor_sync(0xffffffffu, give.z, 1);
        got.w = __shfl_xor_sync(0xffffffffu, give.w, 1);
        // of pieces 2 l, 2 l + 1 of lane l the even lane now has 2 l and 2 l + 2, the odd one 2 l - 1 and 2 l + 1
        if (odd) lo = got; else hi = got;
        uint4 *d = reinterpret_cast<uint4 *>(dst);
        __stcs(d + (odd ? 2 * lane - 1 : 2 * lane), lo);
        __stcs(d + (odd ? 2 * lane + 1 : 2 * lane + 2), hi);
    }
}

}  // namespace

cudaError_t launch_cache_write(const CachePool &c, const __nv_bfloat16 *k, const __nv_bfloat16 *v, const int32_t *cu_q,
                               const int32_t *cu_k, int batch, int64_t total_q, cudaStream_t stream)
{
    const int64_t grid = (2 * total_q + kCacheWarps - 1) / kCacheWarps;
    if (grid <= 0) return cudaSuccess;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return launch_pdl(c.fp8 ? cache_write_kernel<true> : cache_write_kernel<false>, dim3((unsigned)grid),
                      dim3(kCacheWarps * 32), 0, stream, k, v, c, cu_q, cu_k, batch, total_q);
}

cudaError_t launch_cache_read(const CachePool &c, const int32_t *cu_k, const int32_t *tok_begin, const int32_t *cu_out,
                              int batch, int64_t total_out, __nv_bfloat16 *k_out, __nv_bfloat16 *v_out,
                              cudaStream_t stream)
{
    const int64_t grid = (2 * ((total_out + kReadTok - 1) / kReadTok) + kCacheWarps - 1) / kCacheWarps;
    if (grid <= 0) return cudaSuccess;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return launch_pdl(c.fp8 ? cache_read_kernel<true> : cache_read_kernel<false>, dim3((unsigned)grid),
                      dim3(kCacheWarps * 32), 0, stream, c, cu_k, tok_begin, cu_out, batch, total_out, k_out, v_out);
}

}  // namespace qsa
