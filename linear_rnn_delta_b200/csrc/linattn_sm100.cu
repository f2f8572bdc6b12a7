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
// Tensor-core products per chunk; D in tensor memory, lanes = value channel j except for QK:
//   QK [r][s] = X Y^T
//   KV [j][i] = (Z^T u) Y           Z^T u, its columns scaled by u_s, in three bf16 parts
//   O  [j][r] = R_0^T X^T + Z^T P^T   R_0^T in two bf16 parts,  P_rs = (L_rs / w_r) (x_r . y_s) rounded once
// and out_r = w_r O_r: with the weights divided by w_r the two products share one accumulator.  L_rs / w_r
// is e^{-c_s}, which stays in range while the chunk's decays multiply to no less than 2^-96 (`narrow`).  A chunk
// that decays further (a reset, say) has P_rs = L_rs (x_r . y_s), out_r = O_r, and w_r goes to X, rounded.
// Both kinds keep O and P 2^32 times smaller (exactly: a shift of exponents, taken back with w_r): e^{-c_s} (x_r . y_s) z_s
// may be 2^96 times the output's own term, and unshifted it overflowed where that term was no more than 2^32.  Sums up
// to 2^64 have room now, and what is lost at the other end lies below 2^-94.
// All A operands but QK's are in tensor memory: the tensor core reads 128 bytes of shared memory a cycle,
// and with A from there, too, operands alone would keep it busy for 1600 cycles a chunk and everybody
// else's shared-memory accesses waiting.  Z^T gets there from Z by transposing matrix loads.
//
// Precision.  x, y, z enter exactly.  A value in n bf16 parts (each the rounding of what the ones before
// leave) is off by at most 2^-8n of itself: three for what is summed into the fp32 state, two for the state
// in the outputs, one for P, an error of the outputs' own rounding's size.  Log-decays are summed in fixed
// point, so that a strong decay costs the pairs on one side of it nothing; those below -10^4 count as
// -10^4, whose e^g is 0, so that -infinity needs no case of its own.
//
// A CTA of 28 warps walks one (sequence, head), or a segment of one, with a bounded wait on every mbarrier:
//   warps 0-1   P: QK lanes 0-63 (a thread has row r) -> decay, mask -> shared memory, two buffers
//   warp 2      the chunk's decays
//   warps 4-11  Z^T and its scaled parts to tensor memory
//   warps 12-15 outputs: w_r O -> bf16 -> [token][channel] tile -> TMA store
//   warps 16-23 the state, fp32 in registers (a thread has half a row of R^T): R = e^{c_C} R + KV, split
//   warp 24     loads (TMA, four stages of X, Y, Z)
//   warps 25-27 issue KV_i, O_i and QK_i (one warp for all products spent longer on waits and issue than they
//               take, and QK waited behind KV)
// Instruction fetch bounds such a kernel as soon as the roles' loops outgrow the SM's instruction cache:
// loop bodies are kept short (rolled where registers allow), and waits sleep instead of polling.
// Infinities and NaN: masked entries of P are selected, not multiplied, but 0 * NaN in Z^T P^T would
// carry a token's z to tokens it must not reach.  Warps 4-11 look for them; in a chunk that has any they
// are taken out of Z, and the outputs of that channel from that token on, and the channel's state, become
// NaN instead.
#include <algorithm>
#include <cmath>

#include "linattn_sm100.cuh"

namespace kda {
namespace {

using namespace lin;

constexpr int NT = 896;
constexpr int NS = 4;                                 // load stages
constexpr uint32_t SM_P = NS * STAGE;                 // P, two chunks' [64][64] bf16
constexpr uint32_t SM_GATE = SM_P + 2 * 8192;
struct GateStage {
    float2 c[C];        // running sums of log2-decays, two floats
    float b[C];         // 2^-SHIFT L_rs / w_r
    float w[C];         // 2^SHIFT w_r
    float u[C];         // u_s
    float total;        // e^{c_C}
    int nv;             // tokens of the chunk
    int bad;            // Z holds an infinity or a NaN
    int narrow;
    short from[128];    // ... of channel j, first (backward: last) token
};
constexpr uint32_t SM_BAR = SM_GATE + NS * sizeof(GateStage);
enum { B_FULL = 0, B_EMPTY = NS, B_QKF = 2 * NS, B_QKE = B_QKF + NS, B_PZ, B_OF = B_PZ + 2, B_KB = B_OF + 2,
       B_KVF, B_S, B_SE, B_DRAIN, NBAR = B_DRAIN + 3 };
// full: a stage's tiles and decays; empty: it may be loaded again; QKF, KVF, SE, OF: QK, KV, the state's product,
// O are complete; QKE: QK is read; and what an MMA needs, all of it on one barrier (a wait costs the issuing
// warp some 200 cycles even when it is over): PZ: P and Z^T for Z^T P^T; KB: Z^T's parts, and KV read, for KV;
// S: the state's parts, and O read, for the state's product.
// A wait for a phase by its parity needs that the phase after it cannot end first.  Whoever waits is among those who
// let that one begin, but for QKF: warps 4-11 wait for it in some chunks only, and QK_{i+2} needs nothing later from
// them than PZ_{i-1}.  It has a barrier for each load stage (QK_{i+4} needs PZ_{i+1}).
constexpr uint32_t SM_MISC = SM_BAR + NBAR * 8;       // tensor-memory address, abort flag
constexpr uint32_t SM_ALLOC = SM_MISC + 16 + 1024;
static_assert(SM_ALLOC <= 232448, "shared memory budget");

constexpr long long NARROW = 96ll << 32;
constexpr int SHIFT = 32;                  // O and P are 2^-SHIFT times what they stand for
constexpr float DOWN = 1.f / 4294967296.f, UP = 4294967296.f;

// registers of the seven warpgroups: what they give up or take adds up to the launch's 72 each
constexpr int RG_P = 72 /* the launch's own */, RG_Z = 64, RG_OUT = 56, RG_STATE = 104, RG_MMA = 40;
static_assert(RG_P + 2 * RG_Z + RG_OUT + 2 * RG_STATE + RG_MMA <= 7 * 72, "more registers than the block has");

// tensor-memory columns: KV, O, QK, the state's two parts, the scaled Z^T's three, Z^T
constexpr uint32_t TM_KV = 0, TM_O = 128, TM_QK = 192, TM_S = 256, TM_ZP = 384, TM_Z = 480, TM_COLS = 512;

// A state between the CTAs of two segments: each warp that wrote its part counts it, and all are waited for.
__device__ __forceinline__ void hand_over(int *count)
{
    asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(count) : "memory");
}
__device__ __forceinline__ bool wait_handed(const int *count, int all, long long limit, volatile int *abort)
{
    bool ok = true;
    if ((threadIdx.x & 31) == 0) {
        const long long t0 = clock64();
        for (;;) {
            int v;
            asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
            if (v >= all) break;
            if (*abort || clock64() - t0 > limit) {
                *abort = 1;
                ok = false;
                break;
            }
            __nanosleep(200);
        }
    }
    ok = __all_sync(0xffffffffu, ok);
    __syncwarp();   // passes lane 0's acquire on to the lanes that read the state (a vote does not)
    return ok;
}

// Up to three passes of one shape; CTAs of a unit's passes and heads are neighbours
struct LinChunkParams {
    int passes;
    LinRun a[3];
    CUtensorMap x[3], y[3], z[3], o[3];
    unsigned *status;
};

// STATE: only the state that a segment adds from nothing, and its decay.  OUT32: fp32 outputs.
template <int DX, int DZ, bool STATE, bool OUT32>
__global__ void __launch_bounds__(NT, 1) lin_chunk_kernel(const __grid_constant__ LinChunkParams P)
{
    constexpr int JW = DZ / 32;                // warps with value channels of their own
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + SM_BAR);
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(sm + SM_MISC);
    volatile int *s_abort = reinterpret_cast<volatile int *>(sm + SM_MISC + 8);
    GateStage *gates = reinterpret_cast<GateStage *>(sm + SM_GATE);
    const int h = blockIdx.x % P.a[0].H, pass = blockIdx.x / P.a[0].H % P.passes;
    const LinRun &a = P.a[pass];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
    const bool rev = a.reverse != 0;
    const bool turns = !STATE && a.tickets;
    const Work work = turns ? lin_turn(a, h, reinterpret_cast<int *>(sm + SM_GATE)) : lin_work(a, blockIdx.x / a.H / P.passes);
    const int n = work.n, row0 = work.row0, len = work.len, nch = work.nch;
    if (turns ? work.slot < 0 : a.seg_chunks && nch <= 0) return;
    // the sequence's first and last segment in time
    const bool opening = rev ? work.c0 + nch >= work.nall : work.c0 == 0;
    const bool closing = rev ? work.c0 == 0 : work.c0 + nch >= work.nall;
    if (STATE && closing) return;   // nobody asks for the state behind it
    const size_t soff = ((size_t)n * a.H + h) * DX * DZ, woff = ((size_t)work.slot * a.H + h) * DX * DZ;

    if (warp == 3) tmem_alloc(s_tmem, TM_COLS);
    if (tid == 0) {
        *s_abort = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar + B_FULL + s, 2);   // the loads' bytes, the decays
            mbar_init(bar + B_EMPTY + s, STATE ? 1 + 2 * JW : 2 + 2 * JW + 4);   // products, state, outputs
        }
        for (int s = 0; s < NS; ++s) mbar_init(bar + B_QKF + s, 1);
        mbar_init(bar + B_QKE, 2);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar + B_PZ + s, 2 + 8);
            mbar_init(bar + B_OF + s, 1);
        }
        for (int s = 0; s < 3; ++s) mbar_init(bar + B_DRAIN + s, 1);
        mbar_init(bar + B_KB, 8 + 2 * JW);
        mbar_init(bar + B_KVF, 1);
        mbar_init(bar + B_S, 2 * JW + JW);
        mbar_init(bar + B_SE, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *s_tmem;
    const uint32_t tlane = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    // chunk of iteration i
    auto chunk = [&](int i) { return work.c0 + (rev ? nch - 1 - i : i); };

    if (wg == 0) {
        if (warp < 2) {
          if constexpr (!STATE) {
            // ---- P: row r of QK
            const int r = tid;
            for (int i = 0; i < nch; ++i) {
                const int s = i % NS, pb = i & 1;
                const GateStage &G = gates[s];
                // P's buffer is free once O_{i-2} has read it
                if (!wait(bar + B_FULL + s, (i / NS) & 1, s_abort) || !wait(bar + B_QKF + s, (i / NS) & 1, s_abort) ||
                    (i >= 2 && !wait(bar + B_OF + pb, ((i >> 1) - 1) & 1, s_abort)))
                    break;
                tc_fence_after();
                const bool narrow = G.narrow != 0;
                uint8_t *prow = sm + SM_P + pb * 8192 + r * 128;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    // the row's tokens among these 32, as bits: s <= r, or backward r <= s < nv
                    const int lo = rev ? r - half * 32 : 0, hi = (rev ? G.nv - 1 : r) - half * 32;
                    uint32_t keep = hi < 0 || lo > 31 ? 0u : 0xffffffffu >> (31 - min(hi, 31));
                    if (lo > 0 && lo <= 31) keep &= 0xffffffffu << lo;
                    if (rev ? half < warp : half > warp) {   // nobody's
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *reinterpret_cast<uint4 *>(prow + (((half * 4 + q) ^ (r & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                    } else if (narrow) {
                        float2 v[16];
                        uint32_t pk[16];
                        tmem_ld32(tlane + TM_QK + half * 32, &v[0].x);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float4 bs = *reinterpret_cast<const float4 *>(&G.b[half * 32 + 2 * e]);
                            v[e] = __fmul2_rn(v[e], make_float2(bs.x, bs.y));
                            v[e + 1] = __fmul2_rn(v[e + 1], make_float2(bs.z, bs.w));
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (!(keep & (1u << (2 * e)))) v[e].x = 0.f;
                            if (!(keep & (2u << (2 * e)))) v[e].y = 0.f;
                            pk[e] = pack_bf16(v[e].x, v[e].y);
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *reinterpret_cast<uint4 *>(prow + (((half * 4 + q) ^ (r & 7)) << 4)) =
                                make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
                    } else {   // a strong decay or a reset in the chunk: each pair's own exponential
                        const float2 cr = make_float2(G.c[r].x + (rev ? SHIFT : -SHIFT), G.c[r].y);
#pragma unroll 1
                        for (int q = 0; q < 4; ++q, keep >>= 8) {
                            float v[8];
                            tmem_ld8(tlane + TM_QK + half * 32 + q * 8, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float d = diff(cr, G.c[half * 32 + q * 8 + e]);
                                v[e] = keep & (1u << e) ? v[e] * ex2(rev ? -d : d) : 0.f;
                            }
                            *reinterpret_cast<uint4 *>(prow + (((half * 4 + q) ^ (r & 7)) << 4)) =
                                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                           pack_bf16(v[6], v[7]));
                        }
                    }
                }
                tc_fence_before();
                warp_arrive(bar + B_QKE);
                fence_async_smem();
                warp_arrive(bar + B_PZ + pb);
            }
          }
        } else if (warp == 2) {
            // ---- decays (a chunk's are on their way while the one before is summed)
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
            long long sum = 0;   // of the segment's log-decays
            bool any_nan = false;
            for (int i = 0; i < nch; ++i) {
                const int s = i % NS, t0 = chunk(i) * C;
                if (i >= NS && !wait(bar + B_EMPTY + s, (i / NS - 1) & 1, s_abort)) break;
                GateStage &G = gates[s];
                // e^g is 0 far before -10^4 (and infinite before 10^4, which breaks the contract)
                const float ga = fminf(fmaxf(next[0], -1e4f), 1e4f), gb = fminf(fmaxf(next[1], -1e4f), 1e4f);
                const unsigned nan_a = __ballot_sync(0xffffffffu, next[0] != next[0]);
                const unsigned nan_b = __ballot_sync(0xffffffffu, next[1] != next[1]);
                if (i + 1 < nch) gate_load(i + 1);
                const long long fb = fix_log2(gb);
                long long run = fix_log2(ga) + fb;
#pragma unroll 1
                for (int off = 1; off < 32; off <<= 1) {
                    const long long o = __shfl_up_sync(0xffffffffu, run, off);
                    if (lane >= off) run += o;
                }
                const long long end = __shfl_sync(0xffffffffu, run, 31);
                const float nan = __int_as_float(0x7fc00000);
                bool narrow = (nan_a | nan_b) == 0;
#pragma unroll 1
                for (int e = 0; e < 2; ++e) {
                    const int t = 2 * lane + e;
                    const long long c = e ? run : run - fb, left = end - c;
                    float2 cc = make_float2((float)fix_int(c), fix_rest(c));
                    float w = fix_exp2((rev ? left : c) + ((long long)SHIFT << 32)), u = fix_exp2(rev ? c : left);
                    narrow = narrow && c < NARROW && -c < NARROW && left < NARROW && -left < NARROW;
                    G.b[t] = fix_exp2((rev ? -left : -c) - ((long long)SHIFT << 32));
                    if (nan_a | nan_b) {   // a NaN decay is part of every sum from its token on
                        const unsigned upto = 0xffffffffu >> (31 - lane);
                        const bool seen = (nan_a & upto) || (nan_b & (e ? upto : upto >> 1));
                        if (seen) cc.x = nan;
                        if (seen || rev) w = nan;
                        if (seen || !rev) u = nan;
                    }
                    G.c[t] = cc;
                    G.w[t] = w;
                    G.u[t] = u;
                }
                if (STATE) sum = max(sum + end, FIX_LEAST), any_nan = any_nan || (nan_a | nan_b);
                narrow = __all_sync(0xffffffffu, narrow);
                if (lane == 0) {
                    G.total = (nan_a | nan_b) ? nan : fix_exp2(end);
                    G.nv = min(C, len - t0);
                    G.narrow = narrow;
                }
                warp_arrive(bar + B_FULL + s);
            }
            if (STATE && lane == 0)
                a.seg_total[(size_t)work.slot * a.H + h] = any_nan ? __int_as_float(0x7fc00000) : fix_exp2(sum);
        }
    } else if (wg <= 2) {
        regs_dec<RG_Z>();
        // ---- Z^T and its scaled parts: a warp has 32 channels and (by warpgroup) half of the tokens
        constexpr int ZT = 256;
        const int t = tid - 128, q = warp & 3, part0 = (wg - 1) * 16;   // columns of 2 tokens
        // this lane's row of the first 8x8 piece (a piece of 16 more tokens is 2048 bytes on, of 16 more
        // channels two 16-byte columns on, under the swizzle)
        const int ch = (q & 1) * 4 + ((lane >> 3) & 1), zr = (lane >> 4) * 8 + (lane & 7);
        const uint32_t zaddr = sb + 2 * TILE + (q >> 1) * 8192 + (wg - 1) * 4096 + zr * 128 + ((ch ^ (zr & 7)) << 4);
        const uint32_t zstep = (((ch + 2) ^ (zr & 7)) << 4) - ((ch ^ (zr & 7)) << 4);
        bool ok = true;
        for (int i = 0; i < nch; ++i) {
            const int s = i % NS;
            GateStage &G = gates[s];
            uint8_t *st = sm + s * STAGE;
            ok = ok && wait(bar + B_FULL + s, (i / NS) & 1, s_abort);
            const int nv = min(C, len - chunk(i) * C);   // (not from G: barriers below depend on it, come what may)
            // rows of Y and Z behind the sequence's end belong to another one (or hold nothing): zero
            if (nv < C) {
                const int p = (t & 31) >> 3;   // panel: Y's, then Z's
                if (p < 2 ? p < DX / 64 : p - 2 < DZ / 64) {
#pragma unroll 1
                    for (int r = nv + (t >> 5); r < C; r += ZT / 32)
                        *reinterpret_cast<uint4 *>(st + TILE + p * 8192 + r * 128 + (t & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                group_sync(1, ZT);
            }
            uint32_t z[2][8];   // 16 channels, 32 tokens each
            bool clean = true;
#pragma unroll 1
            for (int pass = 0;; ++pass) {
                uint32_t most = 0;
                if (q < JW) {
#pragma unroll
                    for (int g = 0; g < 2; ++g)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            ldmatrix_x4_trans(zaddr + s * STAGE + k * 2048 + (g ? zstep : 0), z[g] + 4 * k);
#pragma unroll
                    for (int e = 0; e < 8; ++e) most = max_abs2(most, max_abs2(z[0][e], z[1][e]));
                }
                if (pass) break;
                clean = group_sync_and(1, ZT, ok && (most & 0x7fffu) < 0x7f80u && (most & 0x7fff0000u) < 0x7f800000u);
                if (t == 0) G.bad = !clean;
                if (clean) break;
                ok = group_sync_and(1, ZT, ok);   // the group's barriers need all of it: it gives up together
                if (!ok) break;
                if (t < 128) {
                    int from = rev ? -1 : C;
                    if (t < DZ) {
#pragma unroll 1
                        for (int x = 0; x < C; ++x) {
                            const int r = rev ? x : C - 1 - x;   // the last write is the first token in time
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
                group_sync(1, ZT);   // once more, without them
            }
            if (!ok) break;
            if (!STATE && !G.narrow) {   // w_r goes to X, which QK_i has read
                ok = ok && wait(bar + B_QKF + s, (i / NS) & 1, s_abort);
#pragma unroll 1
                for (int e = t; e < C * DX / 8; e += ZT) {
                    uint32_t *x = reinterpret_cast<uint32_t *>(st + e * 16);
                    const float w = G.w[(e & 511) >> 3] * DOWN;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float2 v = __fmul2_rn(unpack(x[y]), make_float2(w, w));
                        x[y] = pack_bf16(v.x, v.y);
                    }
                }
                fence_async_smem();
            }
            uint32_t part[3][8];
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {
                if (q < JW) {
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {   // 8 tokens: u[k] channel lane/4, u[k+1] channel lane/4 + 8
                        const float2 u = *reinterpret_cast<const float2 *>(&G.u[part0 * 2 + 4 * k + 2 * (lane & 3)]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float2 x = __fmul2_rn(unpack(g ? z[1][k + e] : z[0][k + e]), u);
                            part[0][k + e] = take_part(x);
                            part[1][k + e] = take_part(x);
                            part[2][k + e] = pack_bf16(x.x, x.y);
                        }
                    }
                }
                if (g == 0) {   // KV_{i-1} has read the parts
                    if (i > 0) ok = ok && wait(bar + B_KVF, (i - 1) & 1, s_abort);
                    if (!ok) break;
                    tc_fence_after();
                }
                if (q < JW) {
#pragma unroll
                    for (int p = 0; p < 3; ++p)
                        tmem_st_frag4(tlane + ((uint32_t)(g * 16) << 16) + TM_ZP + p * 32 + part0, part[p]);
                }
            }
            if (!ok) continue;
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(bar + B_KB);
            if (STATE) continue;
            // Z^T itself: O_{i-1} has read the last one
            if (i > 0) ok = ok && wait(bar + B_OF + ((i - 1) & 1), ((i - 1) >> 1) & 1, s_abort);
            if (!ok) continue;
            if (q < JW) {
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < 2; ++g) tmem_st_frag4(tlane + ((uint32_t)(g * 16) << 16) + TM_Z + part0, z[g]);
                tmem_wait_st();
                tc_fence_before();
            }
            warp_arrive(bar + B_PZ + (i & 1));
        }
    } else if (wg == 3) {
        regs_dec<RG_OUT>();
      if constexpr (!STATE) {
        // ---- outputs: fragments of O^T (channel, token pair) go transposed into [token][channel] panels over
        // this stage's X, which nobody reads any more, and leave from there by TMA (the last, ragged chunk of
        // a sequence row by row: what lies behind it is another sequence's)
        const size_t ld = (size_t)a.H * DZ;
        const int q = warp & 3;
        bool ok = true;
        if (q < JW) warp_arrive(bar + B_S);   // O has nothing to be read yet
        for (int i = 0; i < nch; ++i) {
            const int s = i % NS, t0 = chunk(i) * C;
            ok = wait(bar + B_OF + (i & 1), (i >> 1) & 1, s_abort);
            if (!group_sync_and(2, 128, ok)) break;
            tc_fence_after();
            const GateStage &G = gates[s];
            const int nv = G.nv;
            const bool bad = G.bad != 0, narrow = G.narrow != 0;
            if (q < JW) {
                const int r0 = (lane >> 4) * 8 + (lane & 7), c0 = (q & 1) * 4 + ((lane >> 3) & 1);
                const uint32_t rows = sb + s * STAGE + (q >> 1) * 8192 + r0 * 128;
#pragma unroll 1
                for (int x = 0; x < 4; ++x) {
                    const int half = x >> 1, g = x & 1;   // 32 tokens, 16 channels
                    float2 v[8];
                    tmem_ld_frag4(tlane + ((uint32_t)(g * 16) << 16) + TM_O + half * 32, &v[0].x);
                    tmem_wait_ld();
                    if (x == 3) {   // the accumulator is read
                        tc_fence_before();
                        warp_arrive(bar + B_S);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float2 w = make_float2(UP, UP);
                        if (narrow) w = *reinterpret_cast<const float2 *>(&G.w[half * 32 + k * 8 + 2 * (lane & 3)]);
                        v[2 * k] = __fmul2_rn(v[2 * k], w);
                        v[2 * k + 1] = __fmul2_rn(v[2 * k + 1], w);
                    }
                    if (bad) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int r = half * 32 + (k >> 1) * 8 + 2 * (lane & 3);
                            const int from = G.from[q * 32 + g * 16 + 8 * (k & 1) + (lane >> 2)];
                            if (rev ? r <= from : r >= from) v[k].x = __int_as_float(0x7fc00000);
                            if (rev ? r + 1 <= from : r + 1 >= from) v[k].y = __int_as_float(0x7fc00000);
                        }
                    }
                    if constexpr (OUT32) {   // a register's 32 values are 8 channels of 4 tokens: whole sectors
                        float *o = (float *)a.out + ((size_t)row0 + t0) * ld + (size_t)h * DZ + q * 32 + g * 16 + (lane >> 2);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int r = half * 32 + (k >> 1) * 8 + 2 * (lane & 3);
                            if (r < nv) o[r * ld + 8 * (k & 1)] = v[k].x;
                            if (r + 1 < nv) o[(r + 1) * ld + 8 * (k & 1)] = v[k].y;
                        }
                    } else {
                        uint32_t pk[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) pk[k] = pack_bf16(v[k].x, v[k].y);
                        // matrices: channels +0 / +8 of token group k, then of k + 1
                        const uint32_t to = rows + half * 4096 + (((c0 + g * 2) ^ (r0 & 7)) << 4);
                        stmatrix_x4_trans(to, pk[0], pk[1], pk[2], pk[3]);
                        stmatrix_x4_trans(to + 2048, pk[4], pk[5], pk[6], pk[7]);
                    }
                }
            }
            if constexpr (!OUT32) {
                fence_async_smem();
                group_sync(2, 128);
                if (nv == C) {
                    if (tid == 3 * 128) {
#pragma unroll
                        for (int p = 0; p < DZ / 64; ++p)
                            tma_store_3d(&P.o[pass], sm + s * STAGE + p * 8192, p * 64, h, row0 + t0);
                        bulk_commit();
                        bulk_wait_read();
                    }
                } else {
                    __nv_bfloat16 *o = (__nv_bfloat16 *)a.out + ((size_t)row0 + t0) * ld + (size_t)h * DZ;
#pragma unroll 1
                    for (int e = tid - 3 * 128; e < nv * (DZ / 8); e += 128) {
                        const int r = e / (DZ / 8), ch = e % (DZ / 8);
                        *reinterpret_cast<uint4 *>(o + r * ld + ch * 8) = *reinterpret_cast<const uint4 *>(
                            sm + s * STAGE + (ch >> 3) * 8192 + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
                    }
                }
            }
            warp_arrive(bar + B_EMPTY + s);
        }
        bulk_wait_all();
      }
    } else if (wg <= 5) {
        regs_inc<RG_STATE>();
        // ---- state: row j of R^T, half of its columns
        constexpr int CX = DX / 2;
        if ((warp & 3) < JW) {
            const int j = (warp & 3) * 32 + lane, i0 = (wg - 4) * CX;
            const bool given = !STATE && a.seg_chunks && !(turns && opening);   // by other segments' walks
            const float *s_in = STATE ? nullptr : given ? a.seg_state + woff : a.s_in ? a.s_in + soff : nullptr;
            const bool gives = turns && !closing;   // in turn: to the slot behind this one in time
            const size_t to_slot = (size_t)(work.slot + (rev ? -1 : 1)) * a.H + h;
            float *s_out = STATE ? a.seg_state + woff : gives ? a.seg_state + to_slot * (DX * DZ)
                           : a.s_out && closing ? a.s_out + soff : nullptr;
            bool ok = true;
            const bool stall = a.stall && n == 0 && h == 0;
            if (turns && given)
                ok = wait_handed(a.handed + (size_t)work.slot * a.H + h, 2 * JW,
                                 stall && work.c0 == a.seg_chunks ? STALL_LIMIT : WAIT_LIMIT, s_abort);
            // between memory and the registers by way of the tensor memory that KV has later: short loops
            const uint32_t scratch = tlane + TM_KV + i0;
            {
                const bool t = s_in && a.in_t && !given;
                const float *at = s_in + (t ? (size_t)j * DX + i0 : (size_t)i0 * DZ + j);
                const int step = t ? 1 : DZ;
#pragma unroll 1
                for (int b = 0; b < CX / 16; ++b, at += 16 * step) {
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = s_in ? __ldcg(at + e * step) : 0.f;
                    tmem_st16(scratch + b * 16, v);
                }
                tmem_wait_st();
            }
            float2 S[CX / 2];
#pragma unroll
            for (int b = 0; b < CX / 16; ++b) tmem_ld16(scratch + b * 16, &S[b * 8].x);
            tmem_wait_ld();
            // iteration i: the state before it is published (and written where it is a boundary's or the last)
            for (int i = 0; ok; ++i) {
                if ((!STATE && a.snap) || i == nch) {
                    float *to[2] = {nullptr, nullptr};
                    // the token whose boundary this state is: backward the chunk to come ends there, forward the
                    // last one did
                    const int edge = rev ? (i < nch ? min(len, (chunk(i) + 1) * C) - 1 : -1)
                                         : (i > 0 ? min(len, (work.c0 + i) * C) - 1 : -1);
                    if (!STATE && a.snap && edge >= 0 && (edge == len - 1 || (edge + 1) % a.snap_tokens == 0))
                        to[0] = a.snap + ((size_t)(n + row0 / a.snap_tokens + edge / a.snap_tokens) * a.H + h) * DX * DZ;
                    if (i == nch) to[1] = s_out;
                    if (to[0] || to[1]) {
#pragma unroll
                        for (int b = 0; b < CX / 16; ++b) tmem_st16(scratch + b * 16, &S[b * 8].x);
                        tmem_wait_st();
#pragma unroll 1
                        for (int b = 0; b < CX / 8; ++b) {   // half of them for the second destination
                            float v[16];
                            float *dst = b < CX / 16 ? to[0] : to[1];
                            if (!dst) continue;
                            const int b16 = (b & (CX / 16 - 1)) * 16;
                            tmem_ld16(scratch + b16, v);
                            tmem_wait_ld();
                            dst += (size_t)(i0 + b16) * DZ + j;
#pragma unroll
                            for (int e = 0; e < 16; ++e) dst[e * DZ] = v[e];
                        }
                    }
                    if (i == nch) break;
                }
                tc_fence_before();
                warp_arrive(bar + B_KB);   // KV is read (the first time there is nothing to be read)
                if constexpr (!STATE) {
                    if (i > 0) {
                        ok = wait(bar + B_SE, (i - 1) & 1, s_abort);   // O_{i-1} has read the parts
                        if (!ok) break;
                        tc_fence_after();
                    }
#pragma unroll
                    for (int b = 0; b < CX / 16; ++b) {
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float2 x = __fmul2_rn(S[b * 8 + e], make_float2(DOWN, DOWN));
                            hi[e] = take_part(x);
                            lo[e] = pack_bf16(x.x, x.y);
                        }
                        tmem_st8(tlane + TM_S + i0 / 2 + b * 8, hi);
                        tmem_st8(tlane + TM_S + 64 + i0 / 2 + b * 8, lo);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    warp_arrive(bar + B_S);
                }
                const int s = i % NS;
                ok = wait(bar + B_KVF, i & 1, s_abort);
                if (!ok) break;
                tc_fence_after();
                const GateStage &G = gates[s];
                const float2 tot = make_float2(G.total, G.total);
#pragma unroll
                for (int b = 0; b < CX / 16; ++b) {
                    float v[16];
                    tmem_ld16(scratch + b * 16, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        S[b * 8 + e] = __ffma2_rn(S[b * 8 + e], tot, make_float2(v[2 * e], v[2 * e + 1]));
                }
                if (G.bad && G.from[j] >= 0 && G.from[j] < C) {
#pragma unroll
                    for (int e = 0; e < CX / 2; ++e) S[e] = make_float2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
                }
                warp_arrive(bar + B_EMPTY + s);
            }
            if (!ok && s_out)
#pragma unroll 1
                for (int e = 0; e < CX; ++e) s_out[(size_t)(i0 + e) * DZ + j] = __int_as_float(0x7fc00000);
            if (gives && !(stall && opening)) {
                __syncwarp();
                if (lane == 0) hand_over(a.handed + to_slot);
            }
        }
    } else {
        regs_dec<RG_MMA>();
        const uint32_t lead = elect_one();
        bool ok = true;
        if (warp == 24) {
            // ---- loads
            const int hx = h / a.gx, hy = h / a.gy, hz = h / a.gz;
            int i = 0;
            for (; i < nch; ++i) {
                const int s = i % NS, t0 = chunk(i) * C;
                if (i >= NS && !wait(bar + B_EMPTY + s, (i / NS - 1) & 1, s_abort)) break;
                if (lane == 0) {
                    uint8_t *st = sm + s * STAGE;
                    mbar_expect_tx(bar + B_FULL + s, ((STATE ? 1 : 2) * DX + DZ) * C * 2);
#pragma unroll
                    for (int p = 0; p < DX / 64; ++p) {
                        if (!STATE) tma_load_3d(st + p * 8192, &P.x[pass], bar + B_FULL + s, p * 64, hx, row0 + t0);
                        tma_load_3d(st + TILE + p * 8192, &P.y[pass], bar + B_FULL + s, p * 64, hy, row0 + t0);
                    }
#pragma unroll
                    for (int p = 0; p < DZ / 64; ++p)
                        tma_load_3d(st + 2 * TILE + p * 8192, &P.z[pass], bar + B_FULL + s, p * 64, hz, row0 + t0);
                }
            }
            // no load is in flight when the CTA ends, wound down early or not
            if (lane == 0)
                for (int j = max(0, i - NS); j < i; ++j) mbar_wait_cycles(bar + B_FULL + j % NS, (j / NS) & 1, WAIT_LIMIT);
        } else if (warp == 25) {
            // ---- KV_i
            constexpr uint32_t ID_KV = idesc_bf16(128, DX, false, true);
            for (int i = 0; i < nch; ++i) {
                ok = wait(bar + B_KB, i & 1, s_abort);
                if (!ok) break;
                tc_fence_after();
                const uint32_t y = mn_tile(sb + i % NS * STAGE + TILE);
#pragma unroll 2
                for (int k = 0; k < 3 * C / 16; ++k)   // the parts' columns follow one another
                    mma_bf16_ts_warp(tbase + TM_KV, tbase + TM_ZP + k * 8, dMN(y, k & (C / 16 - 1)), ID_KV, k > 0, lead);
                mma_commit_warp(bar + B_KVF, lead);
                mma_commit_warp(bar + B_EMPTY + i % NS, lead);
            }
        } else if (!STATE && warp == 27) {
            // ---- QK_i; rows 64-127 of A are what lies behind X: lanes nobody reads
            constexpr uint32_t ID_QK = idesc_bf16(128, C, false, false);
            for (int i = 0; i < nch; ++i) {
                const int s = i % NS;
                ok = wait(bar + B_FULL + s, (i / NS) & 1, s_abort) && (i == 0 || wait(bar + B_QKE, (i - 1) & 1, s_abort));
                if (!ok) break;
                tc_fence_after();
                const uint32_t x = k_tile(sb + s * STAGE), y = k_tile(sb + s * STAGE + TILE);
#pragma unroll 2
                for (int k = 0; k < DX / 16; ++k)
                    mma_bf16_warp(tbase + TM_QK, dK(x, k), dK(y, k), ID_QK, k > 0, lead);
                mma_commit_warp(bar + B_QKF + s, lead);
            }
        } else if (!STATE && warp == 26) {
            // ---- O_i: the state's product and the chunk's
            constexpr uint32_t ID_O = idesc_bf16(128, C, false, false);
            const uint32_t pt = k_tile(sb + SM_P);
            for (int i = 0; i < nch; ++i) {
                ok = wait(bar + B_PZ + (i & 1), (i >> 1) & 1, s_abort) && wait(bar + B_S, i & 1, s_abort);
                if (!ok) break;
                tc_fence_after();
                const uint32_t x = k_tile(sb + i % NS * STAGE);
#pragma unroll 4
                for (int k = 0; k < 2 * DX / 16; ++k) {   // both parts
                    const int kk = k & (DX / 16 - 1);
                    mma_bf16_ts_warp(tbase + TM_O, tbase + TM_S + (k / (DX / 16)) * 64 + kk * 8, dK(x, kk), ID_O, k > 0, lead);
                }
                mma_commit_warp(bar + B_SE, lead);
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk)
                    mma_bf16_ts_warp(tbase + TM_O, tbase + TM_Z + kk * 8, dK(pt + (i & 1) * 512, kk), ID_O, 1, lead);
                mma_commit_warp(bar + B_OF + (i & 1), lead);
                mma_commit_warp(bar + B_EMPTY + i % NS, lead);
            }
        }
        // no product runs on: this warp may have issued all of its own and a reader have given up since
        if (nch > 0 && (warp == 25 || (!STATE && warp > 25))) {
            mma_commit_warp(bar + B_DRAIN + warp - 25, lead);
            if (lane == 0) mbar_wait_cycles(bar + B_DRAIN + warp - 25, 0, WAIT_LIMIT);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 3) tmem_dealloc(tbase, TM_COLS);
    if (tid == 0 && *s_abort) atomicOr(P.status, DEV_WAIT_TIMEOUT);
}

constexpr int SEG_AHEAD = 8;

// The states that enter the segments, in place of what each adds: one pass over a sequence's segments in time.
// A thread has 4 values of one (sequence, head)'s state.
__global__ void __launch_bounds__(256) lin_segment_kernel(const __grid_constant__ LinRuns P, int dx, int dz)
{
    const LinRun &a = P.a[blockIdx.z];
    const int nh = blockIdx.x, n = nh / a.H, h = nh % a.H, size = dx * dz;
    const int e = (blockIdx.y * 256 + threadIdx.x) * 4;
    if (e >= size) return;
    const int row0 = lin_row0(a, n), len = lin_len(a, n), tokens = a.seg_tokens;
    const int first = n + row0 / tokens, nseg = (len + tokens - 1) / tokens;
    float4 cur = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.s_in) {
        const float *s = a.s_in + (size_t)nh * size;
        if (a.in_t) {   // stored [dz][dx]; 4 values of a row i are 4 rows there
            const int i = e / dz, j = e % dz;
            cur = make_float4(s[j * dx + i], s[(j + 1) * dx + i], s[(j + 2) * dx + i], s[(j + 3) * dx + i]);
        } else {
            cur = *reinterpret_cast<const float4 *>(s + e);
        }
    }
    // SEG_AHEAD segments' loads in flight: one by one their latencies add up (3 us a segment)
    for (int t0 = 0; t0 < nseg; t0 += SEG_AHEAD) {
        float4 *at[SEG_AHEAD], add[SEG_AHEAD];
        float d[SEG_AHEAD];
#pragma unroll
        for (int b = 0; b < SEG_AHEAD; ++b) {
            const int t = t0 + b;
            if (t >= nseg) break;
            const size_t slot = (size_t)(first + (a.reverse ? nseg - 1 - t : t)) * a.H + h;
            at[b] = reinterpret_cast<float4 *>(a.seg_state + slot * size + e);
            if (t + 1 < nseg) {   // (nothing was written for the last one)
                add[b] = *at[b];
                d[b] = a.seg_total[slot];
            }
        }
#pragma unroll
        for (int b = 0; b < SEG_AHEAD; ++b) {
            if (t0 + b >= nseg) break;
            *at[b] = cur;
            if (t0 + b + 1 < nseg)
                cur = make_float4(fmaf(d[b], cur.x, add[b].x), fmaf(d[b], cur.y, add[b].y),
                                  fmaf(d[b], cur.z, add[b].z), fmaf(d[b], cur.w, add[b].w));
        }
    }
    if (nseg == 0 && a.s_out) *reinterpret_cast<float4 *>(a.s_out + (size_t)nh * size + e) = cur;
}

template <int DX, int DZ> cudaError_t make_params(LinChunkParams &p, const LinRun *r, int passes)
{
    memset(&p, 0, sizeof(p));
    p.passes = passes;
    cudaError_t e = bind_context();
    if (e != cudaSuccess || (e = device_status_word(&p.status)) != cudaSuccess) return e;
    for (int i = 0; i < passes; ++i) {
        p.a[i] = r[i];
        if (r[i].rows > 0 && (!make_map(&p.x[i], r[i].x, r[i].rows, r[i].H / r[i].gx, DX) ||
                              !make_map(&p.y[i], r[i].y, r[i].rows, r[i].H / r[i].gy, DX) ||
                              !make_map(&p.z[i], r[i].z, r[i].rows, r[i].H / r[i].gz, DZ) ||
                              (!r[i].out_f32 && !make_map(&p.o[i], r[i].out, r[i].rows, r[i].H, DZ))))
            return cudaErrorInvalidValue;
    }
    return cudaSuccess;
}

template <int DX, int DZ, bool STATE, bool OUT32>
cudaError_t launch_kernel(const LinChunkParams &p, cudaStream_t st)
{
    static bool done[64] = {};
    const cudaError_t e = opt_in(lin_chunk_kernel<DX, DZ, STATE, OUT32>, SM_ALLOC, done);
    if (e != cudaSuccess) return e;
    const LinRun &r = p.a[0];
    // in turn, sequences of one length have as many segments each; packed ones have no more than there are slots
    const int each = r.tickets && !r.cu_seqlens ? std::max(1, (r.T + r.seg_tokens - 1) / r.seg_tokens) : 0;
    const unsigned units = (unsigned)(each ? r.num_seqs * each : r.seg_chunks ? r.slots : r.num_seqs);
    lin_chunk_kernel<DX, DZ, STATE, OUT32><<<units * r.H * p.passes, NT, SM_ALLOC, st>>>(p);
    return cudaGetLastError();
}

template <int DX, int DZ> cudaError_t launch_dims(const LinRuns &r, int passes, cudaStream_t st)
{
    LinChunkParams p;
    cudaError_t e = make_params<DX, DZ>(p, r.a, passes);
    if (e != cudaSuccess) return e;
    if (r.a[0].seg_chunks && !r.a[0].tickets) {
        if ((e = launch_kernel<DX, DZ, true, false>(p, st)) != cudaSuccess) return e;
        if ((e = launch_lin_segments(r, passes, DX, DZ, st)) != cudaSuccess) return e;
    }
    // passes of one launch have outputs of one type
    return r.a[0].out_f32 ? launch_kernel<DX, DZ, false, true>(p, st) : launch_kernel<DX, DZ, false, false>(p, st);
}

}  // namespace

cudaError_t launch_lin_segments(const LinRuns &r, int passes, int dx, int dz, cudaStream_t st)
{
    lin_segment_kernel<<<dim3(r.a[0].num_seqs * r.a[0].H, (dx * dz + 1023) / 1024, passes), 256, 0, st>>>(r, dx, dz);
    return cudaGetLastError();
}

bool lin_chunk_takes(int dx, int dz) { return (dx == 64 || dx == 128) && (dz == 64 || dz == 128); }

LinCut lin_cut(int num_seqs, int T, int H, int passes, long long rows, bool packed)
{
    // Time in chunks of the kernel's walk (1.85 us each at 128 x 128).  Whole: the waves of (sequence, head) pairs over
    // the SMs, each of a sequence and a start (6 chunks).  Cut, side by side: every chunk is walked twice, the first
    // time for its state alone, and each of a segment's two walks has a start (1.7 chunks a chunk and 16 a segment; 5
    // for the two further launches).  Cut, in turn: each is walked once, but a sequence's one after the other.
    // Packed lengths, unknown here, are taken as exponential, cu_seqlens' rows divided by the sequences their mean:
    // the longest of n has about mean (ln n + 0.58) chunks, and a sequence gives 1 / (1 - exp(-seg / mean)) segments.
    // CTAs of unequal work fill the SMs but for half of the last one's.
    // Measured, whole and as taken, 16 heads of 128 x 128: 1x32768 953 and 241 us, 1x8192 248 and 84, 4x8192 whole 250
    // (side by side 261), 12x4096 283 and 222 (in turn), 10x8192 543 and 386 (in turn), backward of 4x4096 670 and 595
    // (in turn); packed, 30 sequences of 65536 tokens, 4 heads, 246 and 186 (side by side); 7 of 16384 whole 129
    // (in turn 140); 16 of 32768, 32 heads, 427 and 359 (in turn).
    // A B200's SMs: a constant, so that the workspace's size follows from the call's sizes alone.  The costs were measured
    // at 128 x 128 and serve the smaller head sizes, too, whose chunks take 15 % less.
    const int S = 148;
    const double units = (double)num_seqs * H * passes;
    const double mean = packed ? std::max(1.0, (double)rows / C / num_seqs) : (double)((T + C - 1) / C);
    const double all = mean * units;
    const double longest = mean * (packed ? std::max(1.0, std::log((double)num_seqs) + 0.58) : 1.0);
    const double whole = packed ? std::max(longest + 6, (all + 6 * units) / S + 0.5 * longest)
                                : std::ceil(units / S) * (mean + 6);
    double least = 0.9 * whole;
    LinCut best{0, false};
    for (int seg = 4; seg < longest; seg += 1 + seg / 16) {
        const double count = units * (packed ? 1 / (1 - std::exp(-seg / mean)) : std::ceil(mean / seg));
        for (int turns = 0; turns < 2; ++turns) {
            if (turns && ((packed && num_seqs > TURN_SEQS) || (packed ? rows : T) > TURN_ROWS)) break;
            const double rate = turns ? 1 : 1.7, start = turns ? 6 : 16, walk = rate * seg + start;
            double cut = std::max(walk, (rate * all + start * count) / S + 0.5 * walk);
            if (!packed) cut = turns ? std::max(cut, std::ceil(count / S) * walk) : std::ceil(count / S) * walk;
            cut = turns ? std::max(cut, longest + start * std::ceil(longest / seg)) + 1 : cut + 5;
            if (cut < least) {
                least = cut;
                best = LinCut{seg, turns != 0};
            }
        }
    }
    return best;
}

cudaError_t launch_lin_chunk(const LinRuns &r, int passes, int dx, int dz, cudaStream_t st)
{
    if (dx == 128 && dz == 128) return launch_dims<128, 128>(r, passes, st);
    if (dx == 128 && dz == 64) return launch_dims<128, 64>(r, passes, st);
    if (dx == 64 && dz == 128) return launch_dims<64, 128>(r, passes, st);
    if (dx == 64 && dz == 64) return launch_dims<64, 64>(r, passes, st);
    return cudaErrorInvalidValue;
}

}  // namespace kda
