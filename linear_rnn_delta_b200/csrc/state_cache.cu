// Quantised cache of recurrent states: fp32 states to 8-bit codes with a scale for each key channel,
// and back.
//
// A state's rows (key channels) decay and are written at their own rates, so their sizes differ; a
// scale for each (slot, head, key channel) costs 4 bytes in d_v.  With A = max |x| of the row and
// TOP = 127 (int8) or 448 (e4m3):
//   scale = A / TOP,   code = the code nearest to x TOP / A (ties to even),   value = code * scale.
// The code is that of the exact quotient: x (TOP / A) in fp32 is off by at most 1.5 units in the last
// place, so only a quotient that close to a border between two codes can go to the wrong one, and
// there the border times A is compared with x TOP in fp64, where both products are exact.
//
// Bound by HBM: 5 bytes for each value in each direction.  A warp takes whole rows (16 bytes of state
// and 4 bytes of codes for each lane), 4 of them in flight for each lane; the sum over a row's maximum
// is a butterfly over the row's lanes.
#include <cuda_fp8.h>

#include "common.cuh"
#include "linattn.cuh"

namespace kda {
namespace {

constexpr int FMT_INT8 = 0;
constexpr unsigned DEV_BAD_INDEX = 4u;
constexpr int SC_NT = 256;
constexpr int SC_UNROLL = 4;

// x TOP / A next to the border `m` (m > 0, |x| of it): -1, 0, 1 as the exact quotient lies below, on, above
__device__ __noinline__ int border_side(float ax, float amax, float top, float m)
{
    const double l = (double)ax * (double)top, r = (double)m * (double)amax;
    return l < r ? -1 : (l > r ? 1 : 0);
}
// |x| TOP / A as t (inv = TOP / A): int8 magnitude
__device__ __forceinline__ float int8_mag(float ax, float amax, float inv)
{
    const float t = ax * inv;
    float r = rintf(t);
    const float f = floorf(t);
    if (fabsf(t - f - 0.5f) < 6e-5f) {   // 127 * 1.5 units of 2^-23 is 2.3e-5
        const int side = border_side(ax, amax, 127.f, f + 0.5f);
        r = side < 0 ? f : (side > 0 ? f + 1.f : 2.f * rintf(0.5f * (f + 0.5f)));   // tie: the even neighbour
    }
    return r;
}
// e4m3: a value that rounds (to nearest even) to the exact quotient's code
__device__ __forceinline__ float e4m3_mag(float ax, float amax, float inv)
{
    float t = ax * inv;
    float m;
    bool near;
    if (t >= 0.015625f) {   // normal codes: 3 stored bits, the border has the 20 below them at half
        const uint32_t b = __float_as_uint(t);
        const int d = (int)(b & 0xFFFFFu) - 0x80000;
        near = d >= -4 && d <= 4;
        m = __uint_as_float((b & ~0xFFFFFu) | 0x80000u);
    } else {                // steps of 2^-9
        const float u = t * 512.f, f = floorf(u) + 0.5f;
        near = fabsf(u - f) < 8e-6f;
        m = f * (1.f / 512.f);
    }
    if (near) {
        const int side = border_side(ax, amax, 448.f, m);
        t = side == 0 ? m : __uint_as_float(__float_as_uint(m) + side);
    }
    return t;
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
#pragma unroll
        for (int u = 0; u < SC_UNROLL; ++u) {
            const int k = base + u * PASS + warp * RPW + sub;
            x[u] = k < a.dk ? __ldcs(src + (size_t)k * LPR + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < SC_UNROLL; ++u) {
            const int k = base + u * PASS + warp * RPW + sub;
            float v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            float amax = 0.f;
            bool bad = false;   // NaN or infinity: fmaxf would drop a NaN
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                amax = fmaxf(amax, fabsf(v[e]));
                bad |= !(fabsf(v[e]) <= 3.402823466e38f);
            }
            if (bad) amax = __int_as_float(0x7f800000);
#pragma unroll
            for (int off = LPR / 2; off; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            float scale = __fdiv_rn(amax, TOP);
            const bool finite = amax <= 3.402823466e38f;
            if (!finite) scale = __int_as_float(0x7fc00000);
            uint32_t word = 0;
            if (finite && amax > 0.f) {
                float am = amax;
                if (amax < 1e-30f) {   // keep TOP / A in range: exact scaling of row and maximum
                    am *= 18446744073709551616.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] *= 18446744073709551616.f;
                }
                const float inv = __fdiv_rn(TOP, am);
                if (FMT == FMT_INT8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int m = (int)int8_mag(fabsf(v[e]), am, inv);
                        word |= (uint32_t)(uint8_t)(int8_t)(v[e] < 0.f ? -m : m) << (8 * e);
                    }
                } else {
                    float t[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) t[e] = copysignf(e4m3_mag(fabsf(v[e]), am, inv), v[e]);
                    word = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(t[0], t[1]), __NV_SATFINITE, __NV_E4M3) |
                           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(t[2], t[3]), __NV_SATFINITE, __NV_E4M3) << 16;
                }
            }
            if (k < a.dk) {
                dst[(size_t)k * LPR + c] = word;
                if (c == 0) scales[k] = scale;
            }
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
