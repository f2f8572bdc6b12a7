// Chunked linear attention with one decay per head on the tensor cores (bf16 inputs, d_x and d_z of
// 64 or 128, fp32 accumulation and state).
//
// One pass (LinRun): out_r = R_r^T x_r with R_r = a_r R_{r-1} + y_r z_r^T.  Over a chunk of C = 64
// tokens, c_r the running sum of log-decays within it and R_0 the state before it,
//   out_r = w_r R_0^T x_r + sum_s L_rs (x_r . y_s) z_s,      w_r = e^{c_r},  L_rs = e^{c_r - c_s} (s <= r)
//   R_C   = e^{c_C} R_0 + sum_s u_s y_s z_s^T,               u_s = e^{c_C - c_s}.
// Backward in time the chunks run from the last to the first, R_0 is the state that enters the chunk's
// last token, L_rs = e^{c_s - c_r} (s >= r), w_r = e^{c_C - c_r} and u_s = e^{c_s} (which includes the
// decay of the chunk's first token, so the state handed on enters the token before it).
//
// Tensor-core products per chunk, D in tensor memory, lanes = value channel j except for the first:
//   QK    [r][s]  = X Y^T
//   KV    [j][i]  = Z^T Ybar          Ybar = u_s y_s in three bf16 parts
//   inter [j][r]  = R_0^T X^T         R_0^T in two or three bf16 parts, A operand in tensor memory
//   intra [j][r]  = Z^T P^T           P = L o QK in two bf16 parts
// x, y, z enter exactly.  What is fp32 and has to be an operand is split into bf16 parts, each the
// rounding of what the parts before it leave: two parts are off by at most 2^-18 of the value, which is
// far below the bf16 step of the outputs; the state and what is returned in fp32 take three (2^-27).
// Decays are differences of running sums kept as two floats each (summed in fp64), so that a strong
// decay or a reset in a chunk costs the pairs on one side of it nothing.  Log-decays below -10^4 count
// as -10^4, whose e^g is 0, so that -infinity needs no case of its own.
//
// A CTA of 16 warps walks one (sequence, head), one role for each warpgroup and a bounded wait on every
// mbarrier:
//   warps 0-1   P: QK lanes 0-63 -> decay, mask, split -> shared memory (row r is a thread's)
//   warp 2      loads (TMA, three stages of X, Y, Z) and the chunk's decays
//   warp 3      issues every MMA, in the order KV_i, QK_{i+1}, inter_i, intra_i: the state's way from KV_i
//               to inter_{i+1} has the other products in between
//   warps 4-7   Ybar (and Z's rows behind the sequence's end, which belong to the next one: zeroed)
//   warps 8-11  the state, fp32 in registers (a thread has row j of R^T): R = e^{c_C} R + KV, split
//   warps 12-15 outputs: w_r inter + intra, rounded and stored (a warp's 32 channels are 64 bytes)
// Infinities and NaN: masked entries of P are selected, not multiplied, but 0 * NaN in `intra` would
// carry a token's z to tokens it must not reach.  Warps 4-7 look for them; in a chunk that has any they
// are taken out of Z and the outputs of that channel from that token on, and the channel's state, become
// NaN instead.
#include <cuda.h>
#include <mutex>
#include <cstring>

#include "common.cuh"
#include "linattn.cuh"
#include "sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int C = 64;
constexpr int NT = 768;
constexpr int NS = 3;                                 // load stages
constexpr uint32_t TILE = 16384;                      // [64 tokens][128 channels] bf16: two panels of 64 channels
constexpr uint32_t STAGE = 3 * TILE;                  // X, Y, Z
constexpr uint32_t SM_KB = NS * STAGE;                // Ybar, three parts
constexpr uint32_t SM_P = SM_KB + 3 * TILE;           // P: two tiles of [64][64] bf16 (two chunks', or two parts)
constexpr uint32_t SM_GATE = SM_P + 2 * 8192;
struct GateStage {
    float2 c[C];        // running sums of log2-decays, two floats
    float a[C], b[C];   // 2^{c_r - m}, 2^{m - c_s} with m half the chunk's sum: their product is L_rs (`narrow`)
    float w_in[C];      // w_r
    float w_out[C];     // u_s
    float total;        // e^{c_C}
    int nv;             // tokens of the chunk
    int bad;            // Z holds an infinity or a NaN
    int narrow;         // a and b are within 2^100 of 1
    short from[128];    // ... of channel j, first (backward: last) token
};
constexpr uint32_t SM_BAR = SM_GATE + NS * sizeof(GateStage);
enum { B_FULL = 0, B_GATE = NS, B_EMPTY = 2 * NS, B_QKF = 3 * NS, B_QKE = B_QKF + 2, B_PF = B_QKE + 2, B_OF = B_PF + 2,
       B_KBF = B_OF + 2, B_KVF, B_KVE, B_SF, B_SE, B_OE, B_DRAIN, NBAR };
constexpr uint32_t SM_MISC = SM_BAR + NBAR * 8;       // tensor-memory address, abort flag
constexpr uint32_t SM_ALLOC = SM_MISC + 16 + 1024;
static_assert(SM_ALLOC <= 232448, "shared memory budget");

// registers of the six warpgroups: what they give up or take adds up to the launch's 80 each
constexpr int RG_P = 72, RG_YBAR = 64, RG_OUT = 72, RG_STATE = 104;
static_assert(RG_P + 2 * RG_YBAR + RG_OUT + 2 * RG_STATE <= 6 * 80, "more registers than the block has");

// tensor-memory columns: KV, the state's parts, inter, intra, QK.  With two parts QK has room for two chunks
constexpr uint32_t TM_KV = 0, TM_S = 128, TM_COLS = 512;
__host__ __device__ constexpr uint32_t tm_inter(int nsp) { return TM_S + 64 * nsp; }
__host__ __device__ constexpr uint32_t tm_intra(int nsp) { return tm_inter(nsp) + 64; }
__host__ __device__ constexpr uint32_t tm_qk(int nsp) { return tm_intra(nsp) + 64; }

constexpr long long WAIT_LIMIT = 1ll << 32;           // cycles, about 2 s
constexpr unsigned DEV_WAIT_TIMEOUT = 1u;
constexpr double LOG2E = 1.4426950408889634;

struct LinChunkParams {
    LinRun a;
    CUtensorMap tx, ty, tz;
    unsigned *status;
};

// K-major descriptor, K step kk of 16 elements, panels of 64 elements `pstride` bytes apart
__device__ __forceinline__ uint64_t dK(uint32_t base, int kk)
{
    return make_desc_sw128(base, 16) + (uint64_t)(((uint32_t)(kk >> 2) * 8192u + (uint32_t)(kk & 3) * 32u) >> 4);
}
// MN-major descriptor of a [token][channel] tile (two panels of 64 channels), K step kk of 16 tokens
__device__ __forceinline__ uint64_t dMN(uint32_t base, int kk)
{
    return make_desc_sw128(base, 8192) + (uint64_t)((uint32_t)kk * (2048u >> 4));
}

// Waits for a phase; false if the wait ran out here (recorded for the others) or elsewhere.
__device__ __forceinline__ bool wait_one(uint64_t *bar, uint32_t parity, volatile int *abort)   // one thread
{
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort) return false;
        if (clock64() - t0 > WAIT_LIMIT) {
            *abort = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    const long long t0 = clock64();
    for (;;) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity) != 0)) return true;
        if (__any_sync(0xffffffffu, *abort != 0 || clock64() - t0 > WAIT_LIMIT)) {
            *abort = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort)   // a warp, one answer
{
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity) != 0) || wait_slow(bar, parity, abort);
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
// 2^x, the error that of exp2f on [-1/2, 1/2] whatever the size of x
__device__ __forceinline__ float exp2_wide(double x)
{
    if (!(x > -126.0 && x < 127.0)) return exp2f((float)x);   // (nearly) nothing, overflow or NaN
    const double n = rint(x);
    return exp2f((float)(x - n)) * __int_as_float(((int)n + 127) << 23);
}
__device__ __forceinline__ float diff(float2 a, float2 b) { return (a.x - b.x) + (a.y - b.y); }

// max of the magnitudes of two bf16 pairs, NaN if either is one
__device__ __forceinline__ uint32_t max_abs2(uint32_t x, uint32_t y)
{
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}

// NSP: bf16 parts of the state in `inter`.  NPP: parts of P; with one, P and its accumulator have two
// buffers each and the next chunk's P is formed while this one's is multiplied.
template <int DX, int DZ, int NSP, int NPP, typename TOut>
__global__ void __launch_bounds__(NT, 1) lin_chunk_kernel(const __grid_constant__ LinChunkParams P)
{
    constexpr int JW = DZ / 32;                // warps with value channels of their own
    constexpr int NB = NPP == 1 ? 2 : 1;       // buffers of P and QK
    constexpr bool BF16_OUT = sizeof(TOut) == 2;
    constexpr uint32_t TM_INTER = tm_inter(NSP), TM_INTRA = tm_intra(NSP), TM_QK = tm_qk(NSP);
    static_assert(TM_QK + 64 * NB <= TM_COLS, "tensor memory");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + SM_BAR);
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(sm + SM_MISC);
    volatile int *s_abort = reinterpret_cast<volatile int *>(sm + SM_MISC + 8);
    GateStage *gates = reinterpret_cast<GateStage *>(sm + SM_GATE);
    const LinRun &a = P.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
    const int n = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const int row0 = lin_row0(a, n), len = lin_len(a, n);
    const int nch = (len + C - 1) / C;
    const bool rev = a.reverse != 0;
    const size_t soff = ((size_t)n * a.H + h) * DX * DZ;

    if (warp == 3) tmem_alloc(s_tmem, TM_COLS);
    if (tid == 0) {
        *s_abort = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar + B_FULL + s, 1);
            mbar_init(bar + B_GATE + s, 1);
            mbar_init(bar + B_EMPTY + s, 1 + 2 * JW + (BF16_OUT ? 4 : JW));
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar + B_QKF + s, 1);
            mbar_init(bar + B_QKE + s, 2);
            mbar_init(bar + B_PF + s, 2);
            mbar_init(bar + B_OF + s, 1);
        }
        mbar_init(bar + B_KBF, 8);
        mbar_init(bar + B_KVF, 1);
        mbar_init(bar + B_KVE, 2 * JW);
        mbar_init(bar + B_SF, 2 * JW);
        mbar_init(bar + B_SE, 1);
        mbar_init(bar + B_OE, JW);
        mbar_init(bar + B_DRAIN, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *s_tmem;
    const uint32_t tlane = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    // chunk of iteration i
    auto chunk = [&](int i) { return rev ? nch - 1 - i : i; };
    // phase parity of the i-th use of a barrier that alternates between NB
    auto par = [](int i) { return (uint32_t)(i / NB) & 1u; };

    if (wg == 0) {
        regs_dec<RG_P>();
        if (warp < 2) {
            // ---- P: row r of QK
            const int r = tid;
            for (int i = 0; i < nch; ++i) {
                const int s = i % NS, pb = i % NB;
                const GateStage &G = gates[s];
                // P's buffer is free once intra_{i-NB} has read it
                if (!wait(bar + B_GATE + s, (i / NS) & 1, s_abort) || !wait(bar + B_QKF + pb, par(i), s_abort) ||
                    (i >= NB && !wait(bar + B_OF + pb, par(i - NB), s_abort)))
                    break;
                tc_fence_after();
                const int first = rev ? r : 0, last = rev ? G.nv - 1 : r;   // the row's tokens
                // columns that no row of the warp masks
                const int clear_from = rev ? warp * 32 + 31 : 0, clear_to = rev ? G.nv - 1 : warp * 32;
                const float2 cr = G.c[r];
                const bool narrow = G.narrow != 0;
                const float af = rev ? G.b[r] : G.a[r];
                const float2 ar = make_float2(af, af);
                const float *bcol = rev ? G.a : G.b;
                uint8_t *prow = sm + SM_P + pb * 8192 + r * 128;
#pragma unroll 1
                for (int blk = 0; blk < 4; ++blk) {
                    uint32_t hi[8], lo[NPP == 2 ? 8 : 1];
                    if (rev ? blk * 16 + 15 < warp * 32 : blk * 16 > warp * 32 + 31) {   // masked for all of the warp's rows
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            hi[e] = 0u;
                            if (NPP == 2) lo[e] = 0u;
                        }
                    } else {
                        float2 v[8];
                        tmem_ld16(tlane + TM_QK + pb * 64 + blk * 16, &v[0].x);
                        tmem_wait_ld();
                        if (narrow) {
#pragma unroll
                            for (int e = 0; e < 8; e += 2) {
                                const float4 bs = *reinterpret_cast<const float4 *>(bcol + blk * 16 + 2 * e);
                                v[e] = __fmul2_rn(__fmul2_rn(v[e], ar), make_float2(bs.x, bs.y));
                                v[e + 1] = __fmul2_rn(__fmul2_rn(v[e + 1], ar), make_float2(bs.z, bs.w));
                            }
                        } else {   // a strong decay or a reset in the chunk: each pair's own exponential
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float4 cs = *reinterpret_cast<const float4 *>(&G.c[blk * 16 + 2 * e]);
                                const float d0 = diff(cr, make_float2(cs.x, cs.y)), d1 = diff(cr, make_float2(cs.z, cs.w));
                                v[e].x *= ex2(rev ? -d0 : d0);
                                v[e].y *= ex2(rev ? -d1 : d1);
                            }
                        }
                        if (blk * 16 + 15 > clear_to || blk * 16 < clear_from) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int s0 = blk * 16 + 2 * e;
                                if (s0 < first || s0 > last) v[e].x = 0.f;
                                if (s0 + 1 < first || s0 + 1 > last) v[e].y = 0.f;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            if (NPP == 2) {
                                hi[e] = take_part(v[e]);
                                lo[e] = pack_bf16(v[e].x, v[e].y);
                            } else {
                                hi[e] = pack_bf16(v[e].x, v[e].y);
                            }
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint4 *at = reinterpret_cast<uint4 *>(prow + (((blk * 2 + q) ^ (r & 7)) << 4));
                        at[0] = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
                        if (NPP == 2) at[512] = make_uint4(lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
                    }
                }
                tc_fence_before();
                warp_arrive(bar + B_QKE + pb);
                fence_async_smem();
                warp_arrive(bar + B_PF + pb);
            }
        } else if (warp == 2) {
            // ---- loads and decays (a chunk's log-decays are on their way while the one before is summed)
            float next[2] = {0.f, 0.f};
            auto gate_load = [&](int i) {
                const int t0 = chunk(i) * C;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = t0 + 2 * lane + e;
                    next[e] = t < len ? a.g[((size_t)row0 + t) * a.g_ld + h] : 0.f;
                }
            };
            if (nch > 0) gate_load(0);
            int i = 0;
            for (; i < nch; ++i) {
                const int s = i % NS, t0 = chunk(i) * C;
                if (i >= NS && !wait(bar + B_EMPTY + s, (i / NS - 1) & 1, s_abort)) break;
                if (lane == 0) {
                    uint8_t *st = sm + s * STAGE;
                    mbar_expect_tx(bar + B_FULL + s, (2 * DX + DZ) * C * 2);
#pragma unroll
                    for (int p = 0; p < DX / 64; ++p) {
                        tma_load_3d(st + p * 8192, &P.tx, bar + B_FULL + s, p * 64, h / a.gx, row0 + t0);
                        tma_load_3d(st + TILE + p * 8192, &P.ty, bar + B_FULL + s, p * 64, h / a.gy, row0 + t0);
                    }
#pragma unroll
                    for (int p = 0; p < DZ / 64; ++p)
                        tma_load_3d(st + 2 * TILE + p * 8192, &P.tz, bar + B_FULL + s, p * 64, h / a.gz, row0 + t0);
                }
                GateStage &G = gates[s];
                const int nv = min(C, len - t0);
                double g2[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) g2[e] = (double)(next[e] < -1e4f ? -1e4f : next[e]) * LOG2E;   // NaN stays
                if (i + 1 < nch) gate_load(i + 1);
                double run = g2[0] + g2[1];
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const double o = __shfl_up_sync(0xffffffffu, run, off);
                    if (lane >= off) run += o;
                }
                const double end = __shfl_sync(0xffffffffu, run, 31), mid = 0.5 * end;
                bool narrow = true;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = 2 * lane + e;
                    const double c = e ? run : run - g2[1];
                    const float hi = (float)c;
                    G.c[t] = make_float2(hi, (float)(c - (double)hi));
                    G.a[t] = exp2_wide(c - mid);
                    G.b[t] = exp2_wide(mid - c);
                    narrow = narrow && c - mid < 100.0 && mid - c < 100.0;
                    const float since = exp2_wide(c), left = exp2_wide(end - c);
                    G.w_in[t] = rev ? left : since;
                    G.w_out[t] = rev ? since : left;
                }
                narrow = __all_sync(0xffffffffu, narrow);
                if (lane == 0) {
                    G.total = exp2_wide(end);
                    G.nv = nv;
                    G.narrow = narrow;
                }
                warp_arrive(bar + B_GATE + s);
            }
            // no load is in flight when the CTA ends, wound down early or not
            if (lane == 0)
                for (int j = max(0, i - NS); j < i; ++j) mbar_wait_cycles(bar + B_FULL + j % NS, (j / NS) & 1, WAIT_LIMIT);
        } else if (lane == 0) {
            // ---- MMA issue
            constexpr uint32_t ID_QK = idesc_bf16(128, C, false, false), ID_KV = idesc_bf16(128, DX, true, true);
            constexpr uint32_t ID_INTER = idesc_bf16(128, C, false, false), ID_INTRA = idesc_bf16(128, C, true, false);
            bool ok = true;
            auto qk = [&](int i) {   // rows 64-127 of A are what lies behind X: lanes nobody reads
                const uint32_t st = sb + (i % NS) * STAGE, d = tbase + TM_QK + (i % NB) * 64;
                ok = ok && wait_one(bar + B_FULL + i % NS, (i / NS) & 1, s_abort);
                if (i >= NB) ok = ok && wait_one(bar + B_QKE + i % NB, par(i - NB), s_abort);
                if (!ok) return;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < DX / 16; ++kk) mma_bf16(d, dK(st, kk), dK(st + TILE, kk), ID_QK, kk > 0);
                mma_commit(bar + B_QKF + i % NB);
            };
            for (int i = -1; i < nch && ok; ++i) {
                const uint32_t st = sb + ((i + NS) % NS) * STAGE;
                if (i >= 0) {
                    ok = wait_one(bar + B_KBF, i & 1, s_abort) &&
                         (i == 0 || wait_one(bar + B_KVE, (i - 1) & 1, s_abort));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int p = 0; p < 3; ++p)
#pragma unroll
                        for (int kk = 0; kk < C / 16; ++kk)
                            mma_bf16(tbase + TM_KV, dMN(st + 2 * TILE, kk), dMN(sb + SM_KB + p * TILE, kk), ID_KV, p + kk > 0);
                    mma_commit(bar + B_KVF);
                }
                if (i + 1 < nch) qk(i + 1);
                if (i < 0) continue;
                ok = ok && wait_one(bar + B_SF, i & 1, s_abort) &&
                     (i == 0 || wait_one(bar + B_OE, (i - 1) & 1, s_abort));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int p = 0; p < NSP; ++p)
#pragma unroll
                    for (int kk = 0; kk < DX / 16; ++kk)
                        mma_bf16_ts(tbase + TM_INTER, tbase + TM_S + p * 64 + kk * 8, dK(st, kk), ID_INTER, p + kk > 0);
                mma_commit(bar + B_SE);
                ok = wait_one(bar + B_PF + i % NB, par(i), s_abort);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int p = 0; p < NPP; ++p)
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk)
                        mma_bf16(tbase + TM_INTRA, dMN(st + 2 * TILE, kk), dK(sb + SM_P + (i % NB + p) * 8192, kk), ID_INTRA,
                                 p + kk > 0);
                mma_commit(bar + B_OF + i % NB);
                mma_commit(bar + B_EMPTY + i % NS);
            }
            // products still running are waited for below (every product of a full run is, by its readers)
            if (!ok) {
                mma_commit(bar + B_DRAIN);
                mbar_wait_cycles(bar + B_DRAIN, 0, WAIT_LIMIT);
            }
        }
    } else if (wg <= 2) {
        regs_dec<RG_YBAR>();
        // ---- Ybar
        constexpr int YT = 256;
        const int t = tid - 128;
        bool ok = true;
        for (int i = 0; i < nch; ++i) {
            const int s = i % NS;
            GateStage &G = gates[s];
            uint8_t *st = sm + s * STAGE;
            ok = ok && wait(bar + B_GATE + s, (i / NS) & 1, s_abort) && wait(bar + B_FULL + s, (i / NS) & 1, s_abort);
            if (!group_sync_and(1, YT, ok)) break;   // the group's barriers need all of it
            const int nv = G.nv;
            // rows behind the sequence's end belong to another one (or hold nothing): zero
            if (nv < C) {
                for (int e = t; e < (DZ / 64) * (C - nv) * 8; e += YT) {
                    const int p = e / ((C - nv) * 8), q = e % ((C - nv) * 8);
                    *reinterpret_cast<uint4 *>(st + 2 * TILE + p * 8192 + nv * 128 + q * 16) = make_uint4(0, 0, 0, 0);
                }
                group_sync(1, YT);
            }
            uint32_t most = 0;
#pragma unroll
            for (int q = 0; q < DZ / 32; ++q) {
                const uint4 w = *reinterpret_cast<const uint4 *>(st + 2 * TILE + (t + YT * q) * 16);
                most = max_abs2(max_abs2(most, max_abs2(w.x, w.y)), max_abs2(w.z, w.w));
            }
            const bool clean = group_sync_and(1, YT, (most & 0x7fffu) < 0x7f80u && (most & 0x7fff0000u) < 0x7f800000u);
            if (t == 0) G.bad = !clean;
            if (!clean && t < 128) {
                int from = rev ? -1 : C;
                if (t < DZ) {
                    for (int u = 0; u < C; ++u) {
                        const int r = rev ? u : C - 1 - u;   // the last write is the first token in time
                        uint8_t *at = st + 2 * TILE + (t >> 6) * 8192 + r * 128 + (((t & 63) * 2) ^ ((r & 7) << 4));
                        unsigned short &w = *reinterpret_cast<unsigned short *>(at);
                        if ((w & 0x7f80u) == 0x7f80u) {
                            w = 0;
                            from = r;
                        }
                    }
                }
                G.from[t] = (short)from;
            }
            ok = i == 0 || wait(bar + B_KVF, (i - 1) & 1, s_abort);   // KV_{i-1} has read Ybar
            if (!ok) continue;
#pragma unroll 2
            for (int q = 0; q < DX / 32; ++q) {
                const int off = (t + YT * q) * 16, r = (off & 8191) >> 7;
                uint4 w = *reinterpret_cast<const uint4 *>(st + TILE + off);
                if (r >= nv) w = make_uint4(0, 0, 0, 0);
                const float u = G.w_out[r];
                const float2 u2 = make_float2(u, u);
                uint32_t part[3][4];
                const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 x = __fmul2_rn(unpack(in[e]), u2);
                    part[0][e] = take_part(x);
                    part[1][e] = take_part(x);
                    part[2][e] = pack_bf16(x.x, x.y);
                }
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    *reinterpret_cast<uint4 *>(sm + SM_KB + p * TILE + off) =
                        make_uint4(part[p][0], part[p][1], part[p][2], part[p][3]);
            }
            fence_async_smem();
            warp_arrive(bar + B_KBF);
        }
    } else if (wg == 3) {
        regs_dec<RG_OUT>();
        // ---- outputs
        const size_t ld = (size_t)a.H * DZ;
        if constexpr (BF16_OUT) {
            // Fragments of O^T (channel, token pair) go transposed into [token][channel] rows over this
            // stage's X and Y, which nobody reads any more; rows of DZ channels then leave by bulk copies.
            constexpr uint32_t RS = DZ * 2 + 16;   // the 16 bytes spread 8 rows over all banks
            const int q = warp & 3;
            bool ok = true;
            for (int i = 0; i < nch; ++i) {
                const int s = i % NS, t0 = chunk(i) * C;
                ok = wait(bar + B_OF + i % NB, par(i), s_abort);
                if (!group_sync_and(2, 128, ok)) break;
                tc_fence_after();
                const GateStage &G = gates[s];
                const int nv = G.nv;
                const uint32_t stage = sb + s * STAGE;
                if (q < JW) {
                    const bool bad = G.bad != 0;
#pragma unroll 1
                    for (int x = 0; x < 4; ++x) {
                        const int half = x >> 1, g = x & 1;   // 32 tokens, 16 channels
                        float u[16], v[16];
                        const uint32_t at = tlane + ((uint32_t)(g * 16) << 16) + half * 32;
                        tmem_ld_frag4(at + TM_INTER, u);
                        tmem_ld_frag4(at + TM_INTRA, v);
                        tmem_wait_ld();
                        if (x == 3) {   // the accumulators are read
                            tc_fence_before();
                            warp_arrive(bar + B_OE);
                        }
                        uint32_t pk[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 w = *reinterpret_cast<const float2 *>(&G.w_in[half * 32 + k * 8 + 2 * (lane & 3)]);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float2 o = __ffma2_rn(make_float2(u[4 * k + 2 * e], u[4 * k + 2 * e + 1]), w,
                                                      make_float2(v[4 * k + 2 * e], v[4 * k + 2 * e + 1]));
                                if (bad) {
                                    const int r = half * 32 + k * 8 + 2 * (lane & 3);
                                    const int from = G.from[q * 32 + g * 16 + 8 * e + (lane >> 2)];
                                    if (rev ? r <= from : r >= from) o.x = __int_as_float(0x7fc00000);
                                    if (rev ? r + 1 <= from : r + 1 >= from) o.y = __int_as_float(0x7fc00000);
                                }
                                pk[2 * k + e] = pack_bf16(o.x, o.y);
                            }
                        }
                        // matrices: channels +0 / +8 of token group k, then of k + 1
                        const uint32_t to = stage + (half * 32 + (lane >> 4) * 8 + (lane & 7)) * RS +
                                            (q * 32 + g * 16 + ((lane >> 3) & 1) * 8) * 2;
                        stmatrix_x4_trans(to, pk[0], pk[1], pk[2], pk[3]);
                        stmatrix_x4_trans(to + 16 * RS, pk[4], pk[5], pk[6], pk[7]);
                    }
                }
                fence_async_smem();
                group_sync(2, 128);
                const int r = q * 16 + lane;
                if (lane < 16 && r < nv)
                    bulk_store((TOut *)a.out + ((size_t)row0 + t0 + r) * ld + (size_t)h * DZ, sm + s * STAGE + r * RS, DZ * 2);
                bulk_commit();
                bulk_wait_read();
                warp_arrive(bar + B_EMPTY + s);
            }
            bulk_wait_all();
        } else if ((warp & 3) < JW) {
            const int j = (warp & 3) * 32 + lane;
            for (int i = 0; i < nch; ++i) {
                const int s = i % NS, t0 = chunk(i) * C;
                if (!wait(bar + B_OF + i % NB, par(i), s_abort)) break;
                tc_fence_after();
                const GateStage &G = gates[s];
                const int nv = G.nv;
                const bool bad = G.bad != 0;
                const int from = bad ? G.from[j] : 0;
                TOut *o = (TOut *)a.out + ((size_t)row0 + t0) * ld + (size_t)h * DZ + j;
#pragma unroll 1
                for (int blk = 0; blk < 4; ++blk, o += 16 * ld) {
                    float u[16], v[16];
                    tmem_ld16(tlane + TM_INTER + blk * 16, u);
                    tmem_ld16(tlane + TM_INTRA + blk * 16, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 w = *reinterpret_cast<const float4 *>(&G.w_in[blk * 16 + e]);
                        v[e] = fmaf(w.x, u[e], v[e]);
                        v[e + 1] = fmaf(w.y, u[e + 1], v[e + 1]);
                        v[e + 2] = fmaf(w.z, u[e + 2], v[e + 2]);
                        v[e + 3] = fmaf(w.w, u[e + 3], v[e + 3]);
                    }
                    if (blk == 3) {   // the accumulators and this stage are read
                        tc_fence_before();
                        warp_arrive(bar + B_OE);
                        warp_arrive(bar + B_EMPTY + s);
                    }
                    TOut *at = o;
#pragma unroll
                    for (int e = 0; e < 16; ++e, at += ld) {
                        const int r = blk * 16 + e;
                        if (bad && (rev ? r <= from : r >= from)) v[e] = __int_as_float(0x7fc00000);
                        if (r < nv) st_out(at, v[e]);
                    }
                }
            }
        }
    } else {
        regs_inc<RG_STATE>();
        // ---- state: row j of R^T, half of its columns
        constexpr int CX = DX / 2;
        if ((warp & 3) < JW) {
            const int j = (warp & 3) * 32 + lane, i0 = (wg - 4) * CX;
            float2 S[CX / 2];
            if (a.s_in && a.in_t) {
#pragma unroll
                for (int e = 0; e < CX / 2; ++e)
                    S[e] = *reinterpret_cast<const float2 *>(a.s_in + soff + (size_t)j * DX + i0 + 2 * e);
            } else if (a.s_in) {
                const float *at = a.s_in + soff + (size_t)i0 * DZ + j;
#pragma unroll
                for (int e = 0; e < CX / 2; ++e) S[e] = make_float2(at[2 * e * DZ], at[(2 * e + 1) * DZ]);
            } else {
#pragma unroll
                for (int e = 0; e < CX / 2; ++e) S[e] = make_float2(0.f, 0.f);
            }
            bool ok = true;
            // iteration i: the state before it is published (and written where it is a boundary's or the last)
            for (int i = 0;; ++i) {
                float *to[2] = {nullptr, nullptr};
                // the token whose boundary this state is: backward the chunk to come ends there, forward the last one did
                const int edge = rev ? (i < nch ? min(len, (chunk(i) + 1) * C) - 1 : -1) : min(len, i * C) - 1;
                if (a.snap && edge >= 0 && (edge == len - 1 || (edge + 1) % a.snap_tokens == 0))
                    to[0] = a.snap + ((size_t)(n + row0 / a.snap_tokens + edge / a.snap_tokens) * a.H + h) * DX * DZ;
                if (i == nch && a.s_out) to[1] = a.s_out + soff;
#pragma unroll 1
                for (int w = 0; w < 2; ++w) {
                    float *dst = w ? to[1] : to[0];
                    if (!dst) continue;
                    dst += (size_t)i0 * DZ + j;
#pragma unroll
                    for (int e = 0; e < CX / 2; ++e) {
                        dst[2 * e * DZ] = S[e].x;
                        dst[(2 * e + 1) * DZ] = S[e].y;
                    }
                }
                if (i == nch) break;
                if (i > 0) {
                    ok = wait(bar + B_SE, (i - 1) & 1, s_abort);   // inter_{i-1} has read the parts
                    if (!ok) break;
                    tc_fence_after();
                }
                // the bf16 parts of the state, for `inter`
#pragma unroll
                for (int b = 0; b < CX / 16; ++b) {
                    uint32_t part[NSP][8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float2 x = S[b * 8 + e];
#pragma unroll
                        for (int p = 0; p < NSP - 1; ++p) part[p][e] = take_part(x);
                        part[NSP - 1][e] = pack_bf16(x.x, x.y);
                    }
#pragma unroll
                    for (int p = 0; p < NSP; ++p) tmem_st8(tlane + TM_S + p * 64 + i0 / 2 + b * 8, part[p]);
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar + B_SF);
                const int s = i % NS;
                ok = wait(bar + B_KVF, i & 1, s_abort);
                if (!ok) break;
                tc_fence_after();
                const GateStage &G = gates[s];
                const float2 tot = make_float2(G.total, G.total);
#pragma unroll
                for (int b = 0; b < CX / 16; ++b) {
                    float v[16];
                    tmem_ld16(tlane + TM_KV + i0 + b * 16, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        S[b * 8 + e] = __ffma2_rn(S[b * 8 + e], tot, make_float2(v[2 * e], v[2 * e + 1]));
                }
                tc_fence_before();
                warp_arrive(bar + B_KVE);
                if (G.bad && G.from[j] >= 0 && G.from[j] < C) {
#pragma unroll
                    for (int e = 0; e < CX / 2; ++e) S[e] = make_float2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
                }
                warp_arrive(bar + B_EMPTY + s);
            }
            if (!ok && a.s_out)
                for (int e = 0; e < CX; ++e) a.s_out[soff + (size_t)(i0 + e) * DZ + j] = __int_as_float(0x7fc00000);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 3) tmem_dealloc(tbase, TM_COLS);
    if (tid == 0 && *s_abort) atomicOr(P.status, DEV_WAIT_TIMEOUT);
}

// ---- host side --------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
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
bool make_map(CUtensorMap *m, const void *base, long long rows, int heads, int d)
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

// Per-device one-time set-up of a kernel: its dynamic shared memory.
template <typename K> cudaError_t opt_in(K kernel, uint32_t bytes, bool (&done)[64])
{
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    // makes the device's context the thread's current one, which encoding a tensor map needs: a thread
    // that has made no runtime call yet (autograd's) has none
    if ((e = cudaSetDevice(dev)) != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
        done[dev] = true;
    }
    return cudaSuccess;
}

template <int DX, int DZ, int NSP, int NPP, typename TOut> cudaError_t launch_dims(const LinRun &r, cudaStream_t st)
{
    static bool done[64] = {};
    cudaError_t e = opt_in(lin_chunk_kernel<DX, DZ, NSP, NPP, TOut>, SM_ALLOC, done);
    if (e != cudaSuccess) return e;
    LinChunkParams p;
    memset(&p, 0, sizeof(p));
    p.a = r;
    if ((e = device_status_word(&p.status)) != cudaSuccess) return e;
    const long long rows = r.rows;
    if (rows > 0 && (!make_map(&p.tx, r.x, rows, r.H / r.gx, DX) || !make_map(&p.ty, r.y, rows, r.H / r.gy, DX) ||
                     !make_map(&p.tz, r.z, rows, r.H / r.gz, DZ)))
        return cudaErrorInvalidValue;
    lin_chunk_kernel<DX, DZ, NSP, NPP, TOut><<<(unsigned)(r.num_seqs * r.H), NT, SM_ALLOC, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

bool lin_chunk_takes(int dx, int dz) { return (dx == 64 || dx == 128) && (dz == 64 || dz == 128); }

cudaError_t launch_lin_chunk(const LinRun &r, int dx, int dz, cudaStream_t st)
{
    const bool fine = r.out_f32 != 0;
    if (dx == 128 && dz == 128) return fine ? launch_dims<128, 128, 3, 2, float>(r, st) : launch_dims<128, 128, 2, 1, __nv_bfloat16>(r, st);
    if (dx == 128 && dz == 64) return fine ? launch_dims<128, 64, 3, 2, float>(r, st) : launch_dims<128, 64, 2, 1, __nv_bfloat16>(r, st);
    if (dx == 64 && dz == 128) return fine ? launch_dims<64, 128, 3, 2, float>(r, st) : launch_dims<64, 128, 2, 1, __nv_bfloat16>(r, st);
    if (dx == 64 && dz == 64) return fine ? launch_dims<64, 64, 3, 2, float>(r, st) : launch_dims<64, 64, 2, 1, __nv_bfloat16>(r, st);
    return cudaErrorInvalidValue;
}

}  // namespace kda
