// Shared parts of linear attention's tensor-core kernels: waits, fixed-point decays, tensor maps.
#pragma once

#include <cuda.h>
#include <mutex>
#include <cstring>

#include "common.cuh"
#include "linattn.cuh"
#include "sm100.cuh"

namespace kda {
namespace lin {

using namespace sm100;

constexpr int C = 64;                                 // tokens of a chunk
constexpr uint32_t TILE = 16384;                      // [64 tokens][128 channels] bf16: two panels of 64 channels
constexpr uint32_t STAGE = 3 * TILE;                  // X, Y, Z

constexpr long long WAIT_LIMIT = 1ll << 32;           // cycles, about 2 s (hand-overs and the last waits of a CTA)
// Polls that sleep for 4 us: about 2 s.  (Given more time, a poll was measured to sleep 4 us all the same, and a limit
// of 2000 polls of 1 ms to be over after 8 ms: less than a CTA may wait for the segments before its own.  Reading a
// timer between polls made the walks 1 to 2 % longer.)
constexpr uint32_t WAIT_NS = 4000, WAIT_POLLS = 500000;
constexpr long long STALL_LIMIT = 1ll << 21;          // testing aid: about 1 ms
constexpr unsigned DEV_WAIT_TIMEOUT = 1u;

// What a CTA walks, in chunks of U tokens: chunks c0 .. c0 + nch - 1 of sequence n (nall in all; none: the slot is nobody's).
struct Work {
    int n, slot, row0, len, c0, nch, nall;
};
template <int U = C> __device__ __forceinline__ Work lin_work(const LinRun &a, int unit)
{
    Work w;
    w.slot = unit;
    if (a.seg_chunks) {   // the last sequence whose first slot is not behind this one (first slots increase)
        int lo = 0, hi = a.num_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (mid + lin_row0(a, mid) / a.seg_tokens <= unit) lo = mid;
            else hi = mid - 1;
        }
        w.n = lo;
    } else {
        w.n = unit;
    }
    w.row0 = lin_row0(a, w.n);
    w.len = lin_len(a, w.n);
    w.nall = (w.len + U - 1) / U;
    w.c0 = a.seg_chunks ? (unit - w.n - w.row0 / a.seg_tokens) * a.seg_chunks : 0;
    w.nch = a.seg_chunks ? min(a.seg_chunks, w.nall - w.c0) : w.nall;
    return w;
}

// Segments in turn: the ticket's one, by the whole block.  Segments are given out by what their sequence has yet to
// walk (its last segments count 1), the longest first, which fills the SMs until the longest sequences end; a
// sequence's earlier ones come before its later ones, so that the one that hands over a state is running or done
// already.  `scratch` holds 2 * 32 words.  A slot of -1: no segment is left.
constexpr int TURN_SEQS = 896;   // packed sequences at most: one to a thread
// A sequence's tokens at most: its last segment may wait for the walk of all others, 2.2 us a chunk of 128 x 128, 5.5
// with a reset and a NaN in each (0.29 to 0.72 s in all, where a wait gives up after 2).
constexpr int TURN_ROWS = 1 << 23;
__device__ __forceinline__ Work lin_turn(const LinRun &a, int h, int *scratch)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int tokens = a.seg_tokens, all = (int)((a.rows + tokens - 1) / tokens);
    if (tid == 0) scratch[0] = atomicAdd(a.tickets + h, 1);
    __syncthreads();
    const int ticket = scratch[0];
    int n = -1, part = 0;   // part: in time
    if (!a.cu_seqlens) {
        const int parts = max(1, (a.T + tokens - 1) / tokens);
        part = ticket / a.num_seqs;
        if (part < parts) n = ticket % a.num_seqs;
        __syncthreads();
    } else {
        const int mine = tid < a.num_seqs ? min(max(1, (lin_len(a, tid) + tokens - 1) / tokens), all + 1) : 0;
        // segments with `level` or more to walk, themselves included
        auto sum = [&](int v, int buf) {
            v = __reduce_add_sync(0xffffffffu, v);
            if (lane == 0) scratch[32 * buf + warp] = v;
            __syncthreads();
            return __reduce_add_sync(0xffffffffu, lane < warps ? scratch[32 * buf + lane] : 0);
        };
        __syncthreads();
        int lo = 0, hi = all + 2, above = 0, buf = 1;   // more than `ticket` at lo, `above` (no more) at hi
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1, cnt = sum(max(0, mine - mid + 1), buf);
            buf ^= 1;
            if (cnt > ticket) lo = mid;
            else {
                hi = mid;
                above = cnt;
            }
        }
        // the (ticket - above)-th sequence of lo segments or more
        const unsigned has = __ballot_sync(0xffffffffu, mine >= lo && lo > 0);
        if (lane == 0) scratch[32 * buf + warp] = __popc(has);
        __syncthreads();
        int before = __popc(has & ((1u << lane) - 1));
        for (int w = 0; w < warp; ++w) before += scratch[32 * buf + w];
        buf ^= 1;
        if (tid == 0) scratch[32 * buf] = -1;
        __syncthreads();
        if ((has >> lane & 1) && before == ticket - above) {
            scratch[32 * buf] = tid;
            scratch[32 * buf + 1] = mine - lo;
        }
        __syncthreads();
        n = scratch[32 * buf];
        part = scratch[32 * buf + 1];
        __syncthreads();
    }
    Work w{};
    w.slot = -1;
    if (n < 0) return w;
    w.n = n;
    w.row0 = lin_row0(a, n);
    w.len = lin_len(a, n);
    w.nall = max(0, (w.len + C - 1) / C);
    const int j = a.reverse ? max(1, (w.nall + a.seg_chunks - 1) / a.seg_chunks) - 1 - part : part;
    w.slot = n + w.row0 / tokens + j;
    w.c0 = j * a.seg_chunks;
    w.nch = min(a.seg_chunks, w.nall - w.c0);
    return w;
}

// 4 consecutive elements as fp32
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p)
{
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

// Descriptors (low words): K step kk of a K-major tile in panels of 64 elements, and of an MN-major
// [token][channel] tile in panels of 64 channels; `base` the tile's own.
__device__ __forceinline__ uint32_t k_tile(uint32_t saddr) { return desc_sw128_lo(saddr, 16); }
__device__ __forceinline__ uint32_t dK(uint32_t base, int kk) { return base + (uint32_t)((kk >> 2) * 512 + (kk & 3) * 2); }
__device__ __forceinline__ uint32_t mn_tile(uint32_t saddr) { return desc_sw128_lo(saddr, 8192); }
__device__ __forceinline__ uint32_t dMN(uint32_t base, int kk) { return base + (uint32_t)(kk * 128); }

// Waits for a phase; false if the wait ran out here (recorded for the others) or elsewhere.  A warp has one
// answer.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    uint32_t polls = 0;
    while (!__all_sync(0xffffffffu, mbar_try_wait_ns(bar, parity, WAIT_NS) != 0)) {
        if (__any_sync(0xffffffffu, *abort != 0) || ++polls > WAIT_POLLS) {
            *abort = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ void warp_arrive(uint64_t *bar)   // one arrival for the warp, behind all its lanes
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ float2 unpack(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// next bf16 part of a pair: rounds x, leaves the rest in x
__device__ __forceinline__ uint32_t take_part(float2 &x)
{
    const uint32_t w = pack_bf16(x.x, x.y);
    x = __ffma2_rn(unpack(w), make_float2(-1.f, -1.f), x);
    return w;
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Log2-decays are summed as 64-bit fixed point with 32 bits behind the point: sums and differences are exact,
// a term is off by less than 3 2^-33.
__device__ __forceinline__ long long fix_log2(float g)
{
    // g log2(e) as two floats: the rounding of the product, and of log2(e), would show in long sums
    const float hi = g * 1.44269502f, lo = fmaf(g, 1.44269502f, -hi) + g * 1.92596303e-8f;
    const float n = rintf(hi);
    // hi - n and lo each on its own: their sum would be rounded to 24 bits (2^-26 off, the same for every token of a
    // steady decay)
    return ((long long)(int)n << 32) + __float2int_rn((hi - n) * 4294967296.f) + __float2int_rn(lo * 4294967296.f);
}
// Sums over a whole segment stop at 2^-256, whose decay is 0: resets count 2^-14427 each, and 150000 of them would
// leave the 31 bits before the point.
constexpr long long FIX_LEAST = -(256ll << 32);
// integer part and rest in [-1/2, 1/2)
__device__ __forceinline__ int fix_int(long long x) { return (int)((x + 0x80000000ll) >> 32); }
__device__ __forceinline__ float fix_rest(long long x) { return (float)(int)(unsigned)x * 2.3283064365386963e-10f; }
// 2^x, its error that of the rest's exponential whatever the size of x; below 2^-126 it is 0
__device__ __forceinline__ float fix_exp2(long long x)
{
    const int n = fix_int(x);
    const float by = n < -126 ? 0.f : __int_as_float(n > 127 ? 0x7f800000 : (n + 127) << 23);
    return ex2(fix_rest(x)) * by;
}
// The same within 0.6 units in the last place, for the factors that a state is multiplied with again and again: with a
// steady decay the same error compounds (ex2 is off by up to 2 units).  e^x - 1 = x (1 + x/2 (1 + x/3 (...))) with
// x = ln 2 times the rest, |x| < 0.347, to x^8: what follows is below 2^-28.
__device__ __forceinline__ float fix_exp2_steady(long long x)
{
    const int n = fix_int(x);
    const float by = n < -126 ? 0.f : __int_as_float(n > 127 ? 0x7f800000 : (n + 127) << 23);
    const float f = fix_rest(x), hi = f * 0.693147182f, lo = fmaf(f, 0.693147182f, -hi) - f * 1.90465421e-9f;
    float y = 1.f / 40320.f;
    y = fmaf(y, hi, 1.f / 5040.f);
    y = fmaf(y, hi, 1.f / 720.f);
    y = fmaf(y, hi, 1.f / 120.f);
    y = fmaf(y, hi, 1.f / 24.f);
    y = fmaf(y, hi, 1.f / 6.f);
    y = fmaf(y, hi, 0.5f);
    // 1 + (hi + (lo + hi^2 y)), lo's own powers below 2^-25 of the last place
    const float rest = fmaf(hi * hi, y, fmaf(lo, hi, lo)), sum = 1.f + hi;
    return (sum + ((hi - (sum - 1.f)) + rest)) * by;
}
__device__ __forceinline__ float diff(float2 a, float2 b) { return (a.x - b.x) + (a.y - b.y); }

// max of the magnitudes of two bf16 pairs, NaN if either is one
__device__ __forceinline__ uint32_t max_abs2(uint32_t x, uint32_t y)
{
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}

// ---- host side --------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// [rows][heads][d] bf16; box of 64 channels of one head, 64 rows, 128-byte swizzle (one operand panel)
inline bool make_map(CUtensorMap *m, const void *base, long long rows, int heads, int d)
{
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2};
    cuuint32_t box[3] = {64, 1, 64}, es[3] = {1, 1, 1};
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Makes the current device's context the thread's own, which encoding a tensor map needs: a thread that has
// made no runtime call yet (autograd's) has none.
inline cudaError_t bind_context()
{
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e != cudaSuccess ? e : cudaSetDevice(dev);
}

// Per-device one-time set-up of a kernel: its dynamic shared memory.
template <typename K> cudaError_t opt_in(K kernel, uint32_t bytes, bool (&done)[64])
{
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
        done[dev] = true;
    }
    return cudaSuccess;
}

}  // namespace lin
}  // namespace kda
