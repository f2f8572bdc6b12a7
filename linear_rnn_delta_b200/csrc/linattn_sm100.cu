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
constexpr int NT = 512;
constexpr int NS = 3;                                 // load stages
constexpr uint32_t TILE = 16384;                      // [64 tokens][128 channels] bf16: two panels of 64 channels
constexpr uint32_t STAGE = 3 * TILE;                  // X, Y, Z
constexpr uint32_t SM_KB = NS * STAGE;                // Ybar, three parts
constexpr uint32_t SM_P = SM_KB + 3 * TILE;           // P, two parts of [64][64] bf16
constexpr uint32_t SM_GATE = SM_P + 2 * 8192;
struct GateStage {
    float2 c[C];        // running sums of log2-decays, two floats
    float w_in[C];      // w_r
    float w_out[C];     // u_s, 0 behind the sequence's end
    float total;        // e^{c_C}
    int nv;             // tokens of the chunk
    int bad;            // Z holds an infinity or a NaN
    int pad;
    short from[128];    // ... of channel j, first (backward: last) token
};
constexpr uint32_t SM_BAR = SM_GATE + NS * sizeof(GateStage);
enum { B_FULL = 0, B_GATE = NS, B_EMPTY = 2 * NS, B_QKF = 3 * NS, B_QKE, B_PF, B_KBF, B_KVF, B_KVE, B_SF, B_SE, B_OF,
       B_OE, B_DRAIN, NBAR };
constexpr uint32_t SM_MISC = SM_BAR + NBAR * 8;       // tensor-memory address, abort flag
constexpr uint32_t SM_ALLOC = SM_MISC + 16 + 1024;
static_assert(SM_ALLOC <= 232448, "shared memory budget");

// tensor-memory columns
constexpr uint32_t TM_KV = 0, TM_S = 128, TM_INTER = 320, TM_INTRA = 384, TM_QK = 448, TM_COLS = 512;

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
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort)   // a warp, one answer
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity) != 0)) return true;
    const long long t0 = clock64();
    for (;;) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity) != 0)) return true;
        if (__any_sync(0xffffffffu, *abort != 0 || clock64() - t0 > WAIT_LIMIT)) {
            *abort = 1;
            return false;
        }
    }
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
__device__ __forceinline__ float diff(float2 a, float2 b) { return (a.x - b.x) + (a.y - b.y); }

template <int DX, int DZ, int NSP>
__global__ void __launch_bounds__(NT, 1) lin_chunk_kernel(const __grid_constant__ LinChunkParams P)
{
    constexpr int JW = DZ / 32;   // warps with value channels of their own
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
            mbar_init(bar + B_EMPTY + s, 1 + 2 * JW);
        }
        mbar_init(bar + B_QKF, 1);
        mbar_init(bar + B_QKE, 2);
        mbar_init(bar + B_PF, 2);
        mbar_init(bar + B_KBF, 4);
        mbar_init(bar + B_KVF, 1);
        mbar_init(bar + B_KVE, JW);
        mbar_init(bar + B_SF, JW);
        mbar_init(bar + B_SE, 1);
        mbar_init(bar + B_OF, 1);
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

    if (wg == 0) {
        regs_dec<112>();
        if (warp < 2) {
            // ---- P: row r of QK
            const int r = tid;
            for (int i = 0; i < nch; ++i) {
                const int s = i % NS;
                const GateStage &G = gates[s];
                if (!wait(bar + B_GATE + s, (i / NS) & 1, s_abort) || !wait(bar + B_QKF, i & 1, s_abort)) break;
                tc_fence_after();
                const int nv = G.nv;
                const float2 cr = G.c[r];
                uint32_t hi[2][16], lo[2][16];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    // the half that lies wholly on the masked side of this warp's rows
                    if (rev ? (warp == 1 && half == 0) : (warp == 0 && half == 1)) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) hi[half][e] = lo[half][e] = 0u;
                        continue;
                    }
                    float v[32];
                    tmem_ld32(tlane + TM_QK + half * 32, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const int s0 = half * 32 + e;
                        const float4 cs = *reinterpret_cast<const float4 *>(&G.c[s0]);
                        const float d0 = diff(cr, make_float2(cs.x, cs.y)), d1 = diff(cr, make_float2(cs.z, cs.w));
                        float2 p = make_float2(v[e] * ex2(rev ? -d0 : d0), v[e + 1] * ex2(rev ? -d1 : d1));
                        if (!(rev ? (s0 >= r && s0 < nv) : (s0 <= r))) p.x = 0.f;
                        if (!(rev ? (s0 + 1 >= r && s0 + 1 < nv) : (s0 + 1 <= r))) p.y = 0.f;
                        hi[half][e / 2] = take_part(p);
                        lo[half][e / 2] = pack_bf16(p.x, p.y);
                    }
                }
                tc_fence_before();
                warp_arrive(bar + B_QKE);
                if (i > 0 && !wait(bar + B_OF, (i - 1) & 1, s_abort)) break;   // intra_{i-1} has read P
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const uint32_t off = SM_P + r * 128 + ((q ^ (r & 7)) << 4);
                    const uint32_t *x = &hi[q >> 2][(q & 3) * 4], *y = &lo[q >> 2][(q & 3) * 4];
                    *reinterpret_cast<uint4 *>(sm + off) = make_uint4(x[0], x[1], x[2], x[3]);
                    *reinterpret_cast<uint4 *>(sm + off + 8192) = make_uint4(y[0], y[1], y[2], y[3]);
                }
                fence_async_smem();
                warp_arrive(bar + B_PF);
            }
        } else if (warp == 2) {
            // ---- loads and decays
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
                for (int e = 0; e < 2; ++e) {
                    const int t = 2 * lane + e;
                    const float g = t < nv ? a.g[((size_t)row0 + t0 + t) * a.g_ld + h] : 0.f;
                    g2[e] = (double)(g < -1e4f ? -1e4f : g) * LOG2E;   // NaN stays
                }
                double run = g2[0] + g2[1];
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const double o = __shfl_up_sync(0xffffffffu, run, off);
                    if (lane >= off) run += o;
                }
                const double end = __shfl_sync(0xffffffffu, run, 31);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = 2 * lane + e;
                    const double c = e ? run : run - g2[1];
                    const float hi = (float)c;
                    G.c[t] = make_float2(hi, (float)(c - (double)hi));
                    const float since = exp2f((float)c), left = exp2f((float)(end - c));
                    G.w_in[t] = rev ? left : since;
                    G.w_out[t] = rev ? since : left;
                }
                if (lane == 0) {
                    G.total = exp2f((float)end);
                    G.nv = nv;
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
                const uint32_t st = sb + (i % NS) * STAGE;
                ok = ok && wait_one(bar + B_FULL + i % NS, (i / NS) & 1, s_abort);
                if (i > 0) ok = ok && wait_one(bar + B_QKE, (i - 1) & 1, s_abort);
                if (!ok) return;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < DX / 16; ++kk)
                    mma_bf16(tbase + TM_QK, dK(st, kk), dK(st + TILE, kk), ID_QK, kk > 0);
                mma_commit(bar + B_QKF);
            };
            if (nch > 0) qk(0);
            for (int i = 0; i < nch && ok; ++i) {
                const uint32_t st = sb + (i % NS) * STAGE;
                ok = wait_one(bar + B_KBF, i & 1, s_abort) && (i == 0 || wait_one(bar + B_KVE, (i - 1) & 1, s_abort));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int p = 0; p < 3; ++p)
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk)
                        mma_bf16(tbase + TM_KV, dMN(st + 2 * TILE, kk), dMN(sb + SM_KB + p * TILE, kk), ID_KV, p + kk > 0);
                mma_commit(bar + B_KVF);
                if (i + 1 < nch) qk(i + 1);
                ok = ok && wait_one(bar + B_SF, i & 1, s_abort) && (i == 0 || wait_one(bar + B_OE, (i - 1) & 1, s_abort));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int p = 0; p < NSP; ++p)
#pragma unroll
                    for (int kk = 0; kk < DX / 16; ++kk)
                        mma_bf16_ts(tbase + TM_INTER, tbase + TM_S + p * 64 + kk * 8, dK(st, kk), ID_INTER, p + kk > 0);
                mma_commit(bar + B_SE);
                ok = wait_one(bar + B_PF, i & 1, s_abort);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk)
                        mma_bf16(tbase + TM_INTRA, dMN(st + 2 * TILE, kk), dK(sb + SM_P + p * 8192, kk), ID_INTRA,
                                 p + kk > 0);
                mma_commit(bar + B_OF);
                mma_commit(bar + B_EMPTY + i % NS);
            }
            // products still running are waited for below (every product of a full run is, by its readers)
            if (!ok) {
                mma_commit(bar + B_DRAIN);
                mbar_wait_cycles(bar + B_DRAIN, 0, WAIT_LIMIT);
            }
        }
    } else if (wg == 1) {
        regs_dec<96>();
        // ---- Ybar
        const int t = tid - 128;
        bool ok = true;
        for (int i = 0; i < nch; ++i) {
            const int s = i % NS;
            GateStage &G = gates[s];
            uint8_t *st = sm + s * STAGE;
            ok = ok && wait(bar + B_GATE + s, (i / NS) & 1, s_abort) && wait(bar + B_FULL + s, (i / NS) & 1, s_abort);
            if (!group_sync_and(1, 128, ok)) break;   // the group's barriers need all of it
            const int nv = G.nv;
            // rows behind the sequence's end belong to another one (or hold nothing): zero
            if (nv < C) {
                for (int e = t; e < (DZ / 64) * (C - nv) * 8; e += 128) {
                    const int p = e / ((C - nv) * 8), q = e % ((C - nv) * 8);
                    *reinterpret_cast<uint4 *>(st + 2 * TILE + p * 8192 + nv * 128 + q * 16) = make_uint4(0, 0, 0, 0);
                }
                group_sync(1, 128);
            }
            uint32_t bad = 0;
#pragma unroll
            for (int q = 0; q < DZ / 16; ++q) {
                const uint4 w = *reinterpret_cast<const uint4 *>(st + 2 * TILE + (t + 128 * q) * 16);
                // an exponent of all ones carries into the sign bit
                bad |= ((w.x & 0x7f807f80u) + 0x00800080u) | ((w.y & 0x7f807f80u) + 0x00800080u) |
                       ((w.z & 0x7f807f80u) + 0x00800080u) | ((w.w & 0x7f807f80u) + 0x00800080u);
            }
            const bool clean = group_sync_and(1, 128, (bad & 0x80008000u) == 0);
            if (t == 0) G.bad = !clean;
            if (!clean) {
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
#pragma unroll
            for (int q = 0; q < DX / 16; ++q) {
                const int off = (t + 128 * q) * 16, r = (off & 8191) >> 7;
                const uint4 w = *reinterpret_cast<const uint4 *>(st + TILE + off);
                const float u = G.w_out[r];
                const float2 u2 = make_float2(u, u);
                uint32_t part[3][4];
                const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 x = __fmul2_rn(unpack(in[e]), u2);
                    if (r >= nv) x = make_float2(0.f, 0.f);
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
    } else if (wg == 2) {
        regs_inc<208>();
        // ---- state: row j of R^T
        if ((warp & 3) < JW) {
            const int j = (warp & 3) * 32 + lane;
            float2 S[DX / 2];
#pragma unroll
            for (int i = 0; i < DX; i += 2) {
                float2 v = make_float2(0.f, 0.f);
                if (a.s_in && a.in_t) v = *reinterpret_cast<const float2 *>(a.s_in + soff + (size_t)j * DX + i);
                else if (a.s_in) v = make_float2(a.s_in[soff + (size_t)i * DZ + j], a.s_in[soff + (size_t)(i + 1) * DZ + j]);
                S[i / 2] = v;
            }
            auto publish = [&]() {   // the bf16 parts of the state, for `inter`
#pragma unroll
                for (int b = 0; b < DX / 32; ++b) {
                    uint32_t part[3][16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 x = S[b * 16 + e];
#pragma unroll
                        for (int p = 0; p < NSP - 1; ++p) part[p][e] = take_part(x);
                        part[NSP - 1][e] = pack_bf16(x.x, x.y);
                    }
#pragma unroll
                    for (int p = 0; p < NSP; ++p)
                        tmem_st16(tlane + TM_S + p * 64 + b * 16, reinterpret_cast<const float *>(part[p]));
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(bar + B_SF);
            };
            auto write = [&](float *dst) {
#pragma unroll
                for (int i = 0; i < DX; i += 2) {
                    dst[(size_t)i * DZ + j] = S[i / 2].x;
                    dst[(size_t)(i + 1) * DZ + j] = S[i / 2].y;
                }
            };
            auto snap = [&](int t) {   // boundary state of the segment that token t belongs to
                write(a.snap + ((size_t)(n + row0 / a.snap_tokens + t / a.snap_tokens) * a.H + h) * DX * DZ);
            };
            bool ok = true;
            if (nch > 0) publish();
            for (int i = 0; i < nch; ++i) {
                const int s = i % NS, last = min(len, (chunk(i) + 1) * C) - 1;   // the chunk's last token
                const bool edge = a.snap && (last == len - 1 || (last + 1) % a.snap_tokens == 0);
                if (rev && edge) snap(last);
                ok = wait(bar + B_KVF, i & 1, s_abort);
                if (!ok) break;
                tc_fence_after();
                const GateStage &G = gates[s];
                const float2 tot = make_float2(G.total, G.total);
#pragma unroll
                for (int b = 0; b < DX / 32; ++b) {
                    float v[32];
                    tmem_ld32(tlane + TM_KV + b * 32, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        S[b * 16 + e] = __ffma2_rn(S[b * 16 + e], tot, make_float2(v[2 * e], v[2 * e + 1]));
                }
                tc_fence_before();
                warp_arrive(bar + B_KVE);
                if (G.bad && G.from[j] >= 0 && G.from[j] < C) {
#pragma unroll
                    for (int e = 0; e < DX / 2; ++e) S[e] = make_float2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
                }
                warp_arrive(bar + B_EMPTY + s);
                if (!rev && edge) snap(last);
                if (i + 1 < nch) {
                    ok = wait(bar + B_SE, i & 1, s_abort);   // inter_i has read the parts
                    if (!ok) break;
                    tc_fence_after();
                    publish();
                }
            }
            if (a.s_out) {
                if (!ok) {
#pragma unroll
                    for (int e = 0; e < DX / 2; ++e) S[e] = make_float2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
                }
                write(a.s_out + soff);
            }
        }
    } else {
        regs_dec<96>();
        // ---- outputs of channel j
        if ((warp & 3) < JW) {
            const int j = (warp & 3) * 32 + lane;
            const size_t ld = (size_t)a.H * DZ;
            for (int i = 0; i < nch; ++i) {
                const int s = i % NS, t0 = chunk(i) * C;
                if (!wait(bar + B_OF, i & 1, s_abort)) break;
                tc_fence_after();
                const GateStage &G = gates[s];
                const int nv = G.nv;
                const bool bad = G.bad != 0;
                const int from = bad ? G.from[j] : 0;
                const size_t at = ((size_t)row0 + t0) * ld + (size_t)h * DZ + j;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float u[32], v[32];
                    tmem_ld32(tlane + TM_INTER + half * 32, u);
                    tmem_ld32(tlane + TM_INTRA + half * 32, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 w = *reinterpret_cast<const float4 *>(&G.w_in[half * 32 + e]);
                        v[e] = fmaf(w.x, u[e], v[e]);
                        v[e + 1] = fmaf(w.y, u[e + 1], v[e + 1]);
                        v[e + 2] = fmaf(w.z, u[e + 2], v[e + 2]);
                        v[e + 3] = fmaf(w.w, u[e + 3], v[e + 3]);
                    }
                    if (half == 1) {   // the accumulators and this stage are read
                        tc_fence_before();
                        warp_arrive(bar + B_OE);
                        warp_arrive(bar + B_EMPTY + s);
                    }
                    if (bad) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int r = half * 32 + e;
                            if (rev ? r <= from : r >= from) v[e] = __int_as_float(0x7fc00000);
                        }
                    }
                    if (a.out_f32) {
                        float *o = (float *)a.out + at + (size_t)(half * 32) * ld;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (half * 32 + e < nv) o[e * ld] = v[e];
                    } else {
                        __nv_bfloat16 *o = (__nv_bfloat16 *)a.out + at + (size_t)(half * 32) * ld;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (half * 32 + e < nv) o[e * ld] = __float2bfloat16_rn(v[e]);
                    }
                }
            }
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

template <int DX, int DZ, int NSP> cudaError_t launch_dims(const LinRun &r, cudaStream_t st)
{
    static bool done[64] = {};
    cudaError_t e = opt_in(lin_chunk_kernel<DX, DZ, NSP>, SM_ALLOC, done);
    if (e != cudaSuccess) return e;
    LinChunkParams p;
    memset(&p, 0, sizeof(p));
    p.a = r;
    if ((e = device_status_word(&p.status)) != cudaSuccess) return e;
    const long long rows = r.rows;
    if (rows > 0 && (!make_map(&p.tx, r.x, rows, r.H / r.gx, DX) || !make_map(&p.ty, r.y, rows, r.H / r.gy, DX) ||
                     !make_map(&p.tz, r.z, rows, r.H / r.gz, DZ)))
        return cudaErrorInvalidValue;
    lin_chunk_kernel<DX, DZ, NSP><<<(unsigned)(r.num_seqs * r.H), NT, SM_ALLOC, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

bool lin_chunk_takes(int dx, int dz) { return (dx == 64 || dx == 128) && (dz == 64 || dz == 128); }

cudaError_t launch_lin_chunk(const LinRun &r, int dx, int dz, cudaStream_t st)
{
    const bool fine = r.out_f32 != 0;
    if (dx == 128 && dz == 128) return fine ? launch_dims<128, 128, 3>(r, st) : launch_dims<128, 128, 2>(r, st);
    if (dx == 128 && dz == 64) return fine ? launch_dims<128, 64, 3>(r, st) : launch_dims<128, 64, 2>(r, st);
    if (dx == 64 && dz == 128) return fine ? launch_dims<64, 128, 3>(r, st) : launch_dims<64, 128, 2>(r, st);
    if (dx == 64 && dz == 64) return fine ? launch_dims<64, 64, 3>(r, st) : launch_dims<64, 64, 2>(r, st);
    return cudaErrorInvalidValue;
}

}  // namespace kda
