// Quantised cache of recurrent states: fp32 states to 8-bit codes with a scale for each key channel,
// and back.
//
// A state's rows (key channels) decay and are written at their own rates, so their sizes differ; a
// scale for each (slot, head, key channel) costs 4 bytes in d_v.  With A = max |x| of the row and
// TOP = 127 (int8) or 448 (e4m3):
//   scale = A / TOP,   code = the code nearest to x TOP / A (ties to even),   value = code * scale.
// The code is that of the exact quotient: x (TOP / A) in fp32 is off by a few units in the last
// place, so only a quotient that close to a border between two codes can go to the wrong one, and
// there the border times A is compared with x TOP in fp64, where both products are exact.
//
// Bound by HBM: 5 bytes for each value in each direction.  A warp takes whole rows (16 bytes of state
// and 4 bytes of codes for each lane), 4 of them in flight for each lane; the sum over a row's maximum
// is a butterfly over the row's lanes.  128 slots of 32 heads, 128 x 128 (335 MB each way): to int8 66 us (5.1 TB/s; a
// branch for each value instead of one for four: 71), to e4m3 78 us, back 46 (58 from HBM alone).
#include <cuda_fp8.h>

#include "common.cuh"
#include "linattn.cuh"

namespace kda {
namespace {

constexpr int FMT_INT8 = 0;
constexpr unsigned DEV_BAD_INDEX = 4u;
constexpr int SC_NT = 256;
constexpr int SC_UNROLL = 4;

// |x| TOP / A against the border m > 0 between two codes: -1, 0, 1 as it lies below, on, above
__device__ __noinline__ int border_side(float ax, float amax, float top, float m)
{
    const double l = (double)ax * (double)top, r = (double)m * (double)amax;
    return l < r ? -1 : (l > r ? 1 : 0);
}
// Adding 1.5 * 2^23 rounds to a whole number (ties to even) and leaves it in the low bits, in two's complement:
// the conversion instructions run at a quarter of this rate and bound the kernel (91 against 51 us of traffic).
constexpr float MAGIC = 12582912.f;
// x TOP / A (inv = TOP / A) as an int8 code in the low byte of the result, and how far it is from it
__device__ __forceinline__ uint32_t int8_code(float x, float inv, float &d)
{
    const float whole = fmaf(x, inv, MAGIC);
    d = fabsf(fmaf(x, inv, MAGIC - whole));
    return __float_as_uint(whole);
}
constexpr float INT8_NEAR = 0.5f - 6e-5f;   // inv is off by 2 units of 2^-23: 127 of those are 3e-5
__device__ __noinline__ uint32_t int8_code_near(float x, float amax, float inv)
{
    const float whole = fmaf(x, inv, MAGIC), r = whole - MAGIC, d = fmaf(x, inv, -r);
    if (fabsf(d) <= INT8_NEAR) return __float_as_uint(whole);
    const float m = fabsf(r + copysignf(0.5f, d));
    const int side = border_side(fabsf(x), amax, 127.f, m);
    const int below = (int)(m - 0.5f), mag = side < 0 ? below : side > 0 ? below + 1 : below + (below & 1);
    return (uint32_t)(x < 0.f ? -mag : mag);
}
// e4m3: |x| TOP / A, and whether it may be on the wrong side of a border between two codes
__device__ __forceinline__ float e4m3_mag(float ax, float inv, bool &near)
{
    const float t = ax * inv, u = t * 512.f, r = (u + MAGIC) - MAGIC;
    const uint32_t b = __float_as_uint(t);
    // 3 stored bits, the border has the 20 below them at half; below 2^-6: steps of 2^-9.  t is off by 3 units at most
    near |= t >= 0.015625f ? ((b + 0x80008u) & 0xFFFFFu) <= 16u : fabsf(u - r) > 0.5f - 1.6e-5f;
    return t;
}
// a value that rounds (to nearest even) to the exact quotient's code
__device__ __noinline__ float e4m3_mag_near(float ax, float amax, float inv)
{
    bool near = false;
    const float t = e4m3_mag(ax, inv, near);
    if (!near) return t;
    const uint32_t b = __float_as_uint(t);
    const float u = t * 512.f, r = (u + MAGIC) - MAGIC;
    const float m = t >= 0.015625f ? __uint_as_float((b & ~0xFFFFFu) | 0x80000u)
                                   : (r + copysignf(0.5f, u - r)) * (1.f / 512.f);
    const int side = border_side(ax, amax, 448.f, m);
    return side == 0 ? m : __uint_as_float(__float_as_uint(m) + side);
}

// LPR lanes of a row (4 values each)
template <int DV, int FMT>
__global__ void __launch_bounds__(SC_NT) state_quantize_kernel(const StateCache a)
{
    constexpr int LPR = DV / 4, RPW = 32 / LPR;   // rows of a warp's pass
    constexpr float TOP = FMT == FMT_INT8 ? 127.f : 448.f;
    const int i = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = a.rows ? a.rows[i] : i, slot = a.slots ? a.slots[i] : i;
    if (row < 0 || slot < 0) return;
    if (row >= a.M || slot >= a.S) {
        if (tid == 0) atomicOr(a.status, DEV_BAD_INDEX);
        return;
    }
    if (a.slots) {   // of several entries with one slot the last is written
        bool later = false;
        for (int j = i + 1 + tid; j < a.n; j += SC_NT) {
            const int r = a.rows ? a.rows[j] : j;
            later |= a.slots[j] == slot && r >= 0 && r < a.M;
        }
        if (__syncthreads_or(later)) return;
    }
    const float4 *src = reinterpret_cast<const float4 *>(a.states + ((size_t)row * a.H + h) * a.dk * DV);
    uint32_t *dst = reinterpret_cast<uint32_t *>(a.codes + ((size_t)slot * a.H + h) * a.dk * DV);
    float *scales = a.scales + ((size_t)slot * a.H + h) * a.dk;
    const int c = lane % LPR, sub = lane / LPR;
    constexpr int PASS = SC_NT / 32 * RPW;        // rows of the CTA's pass
    for (int base = 0; base < a.dk; base += PASS * SC_UNROLL) {
        float4 x[SC_UNROLL];
        uint32_t amax[SC_UNROLL];
#pragma unroll
        for (int u = 0; u < SC_UNROLL; ++u) {
            const int k = base + u * PASS + warp * RPW + sub;
            x[u] = k < a.dk ? __ldcs(src + (size_t)k * LPR + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < SC_UNROLL; ++u) {
            const int k = base + u * PASS + warp * RPW + sub;
            float v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            // as integers, magnitudes order like the values, infinity and NaN above them
            uint32_t most = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) most = max(most, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
            for (int off = LPR / 2; off; off >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
            amax[u] = most;
            uint32_t word = 0;
            if (most < 0x7f800000u && most > 0u) {
                float am = __uint_as_float(most);
                if (am < 1e-30f || am > 1e30f) {   // keep the quotient's parts in range: exact scaling of row and maximum
                    const float by = am < 1.f ? 18446744073709551616.f : 5.421010862427522e-20f;
                    am *= by;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] *= by;
                }
                const float inv = __fdividef(TOP, am);
                // the four values' borders are looked at together: one branch, seldom taken
                if (FMT == FMT_INT8) {
                    uint32_t code[4];
                    float d[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) code[e] = int8_code(v[e], inv, d[e]);
                    if (fmaxf(fmaxf(d[0], d[1]), fmaxf(d[2], d[3])) > INT8_NEAR) {
#pragma unroll 1
                        for (int e = 0; e < 4; ++e)
                            word = word >> 8 | int8_code_near(e == 0 ? v[0] : e == 1 ? v[1] : e == 2 ? v[2] : v[3], am, inv) << 24;
                    } else {
                        word = __byte_perm(__byte_perm(code[0], code[1], 0x0040), __byte_perm(code[2], code[3], 0x0040), 0x5410);
                    }
                } else {
                    float t[4];
                    bool near = false;
#pragma unroll
                    for (int e = 0; e < 4; ++e) t[e] = e4m3_mag(fabsf(v[e]), inv, near);
                    if (near) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) t[e] = e4m3_mag_near(fabsf(v[e]), am, inv);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) t[e] = copysignf(t[e], v[e]);
                    word = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(t[0], t[1]), __NV_SATFINITE, __NV_E4M3) |
                           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(t[2], t[3]), __NV_SATFINITE, __NV_E4M3) << 16;
                }
            }
            if (k < a.dk) dst[(size_t)k * LPR + c] = word;
        }
        // a row's scale is one lane's: the u-th of its lanes has the u-th row's
        uint32_t mine = amax[0];
#pragma unroll
        for (int u = 1; u < SC_UNROLL; ++u) mine = c == u ? amax[u] : mine;
        const int k = base + c * PASS + warp * RPW + sub;
        if (c < SC_UNROLL && k < a.dk) {
            // a 127th of the largest finite value rounds up, and 127 times that is infinite: the scale below it there
            const float s = fminf(__fdiv_rn(__uint_as_float(mine), TOP), FMT == FMT_INT8 ? 0x1.020406p121f : 1e38f);
            scales[k] = mine < 0x7f800000u ? s : __int_as_float(0x7fc00000);
        }
    }
}

template <int FMT> __device__ __forceinline__ float4 widen_codes(uint32_t w, float s)
{
    if (FMT == FMT_INT8)
        return make_float4((float)(int8_t)(w & 0xff) * s, (float)(int8_t)(w >> 8 & 0xff) * s,
                           (float)(int8_t)(w >> 16 & 0xff) * s, (float)(int8_t)(w >> 24) * s);
    const __half2 lo(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffff), __NV_E4M3));
    const __half2 hi(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3));
    const float2 l = __half22float2(lo), u = __half22float2(hi);
    return make_float4(l.x * s, l.y * s, u.x * s, u.y * s);
}

template <int DV, int FMT>
__global__ void __launch_bounds__(SC_NT) state_dequantize_kernel(const StateCache a)
{
    constexpr int LPR = DV / 4;
    const int i = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const int tid = threadIdx.x;
    const int slot = a.slots ? a.slots[i] : i;
    float4 *dst = reinterpret_cast<float4 *>(a.out + ((size_t)i * a.H + h) * a.dk * DV);
    const int words = a.dk * LPR;
    if (slot < 0 || slot >= a.S) {   // an empty state, or a bad index: NaN
        const float f = slot < 0 ? 0.f : __int_as_float(0x7fc00000);
        if (slot >= a.S && tid == 0) atomicOr(a.status, DEV_BAD_INDEX);
        for (int e = tid; e < words; e += SC_NT) __stcs(dst + e, make_float4(f, f, f, f));
        return;
    }
    const uint32_t *src = reinterpret_cast<const uint32_t *>(a.codes + ((size_t)slot * a.H + h) * a.dk * DV);
    const float *scales = a.scales + ((size_t)slot * a.H + h) * a.dk;
    for (int base = 0; base < words; base += SC_NT * 2 * SC_UNROLL) {
        uint32_t w[2 * SC_UNROLL];
        float s[2 * SC_UNROLL];
#pragma unroll
        for (int u = 0; u < 2 * SC_UNROLL; ++u) {
            const int e = base + u * SC_NT + tid;
            w[u] = e < words ? __ldcs(src + e) : 0u;
            s[u] = e < words ? __ldg(scales + e / LPR) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 2 * SC_UNROLL; ++u) {
            const int e = base + u * SC_NT + tid;
            if (e < words) __stcs(dst + e, widen_codes<FMT>(w[u], s[u]));
        }
    }
}

template <int DV> cudaError_t launch_dv(const StateCache &a, bool write, cudaStream_t st)
{
    const unsigned grid = (unsigned)((long long)a.n * a.H);
    if (write) {
        if (a.format == FMT_INT8) state_quantize_kernel<DV, 0><<<grid, SC_NT, 0, st>>>(a);
        else state_quantize_kernel<DV, 1><<<grid, SC_NT, 0, st>>>(a);
    } else {
        if (a.format == FMT_INT8) state_dequantize_kernel<DV, 0><<<grid, SC_NT, 0, st>>>(a);
        else state_dequantize_kernel<DV, 1><<<grid, SC_NT, 0, st>>>(a);
    }
    return cudaGetLastError();
}
cudaError_t launch(const StateCache &a, bool write, cudaStream_t st)
{
    switch (a.dv) {
    case 16: return launch_dv<16>(a, write, st);
    case 32: return launch_dv<32>(a, write, st);
    case 64: return launch_dv<64>(a, write, st);
    case 128: return launch_dv<128>(a, write, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_state_quantize(const StateCache &a, cudaStream_t st) { return launch(a, true, st); }
cudaError_t launch_state_dequantize(const StateCache &a, cudaStream_t st) { return launch(a, false, st); }

}  // namespace kda
