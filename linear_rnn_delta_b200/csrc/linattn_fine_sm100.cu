// Chunked linear attention with one decay per head on the tensor cores, fp32 outputs: the passes whose
// outputs the gate gradient is a difference of (dq and dk).  The chunk's formulas, roles and waits are those
// of linattn_sm100.cu; what differs is the precision: the state enters `inter` in three bf16 parts and P in
// two, and the outputs leave as fp32.  Three parts of the state fill the tensor memory, so Z is read from shared memory and
// Ybar = u_s y_s is what carries u_s, in three parts:
//   QK    [r][s]  = X Y^T
//   KV    [j][i]  = Z^T Ybar
//   inter [j][r]  = R_0^T X^T
//   intra [j][r]  = Z^T P^T           P = L o QK,   out_r = w_r inter + intra
#include "linattn_sm100.cuh"

namespace kda {
namespace {

using namespace lin;

constexpr int NT = 768;
constexpr int NS = 3;                                 // load stages
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
enum { B_FULL = 0, B_GATE = NS, B_EMPTY = 2 * NS, B_QKF = 3 * NS, B_QKE, B_PF, B_OF = B_PF + 2,
       B_KBF = B_OF + 2, B_KVF, B_KVE, B_SF, B_SE, B_OE, B_DRAIN, NBAR };
constexpr uint32_t SM_MISC = SM_BAR + NBAR * 8;       // tensor-memory address, abort flag
constexpr uint32_t SM_ALLOC = SM_MISC + 16 + 1024;
static_assert(SM_ALLOC <= 232448, "shared memory budget");

// registers of the six warpgroups: what they give up or take adds up to the launch's 80 each
constexpr int RG_P = 72, RG_YBAR = 64, RG_OUT = 72, RG_STATE = 104;
static_assert(RG_P + 2 * RG_YBAR + RG_OUT + 2 * RG_STATE <= 6 * 80, "more registers than the block has");

// tensor-memory columns: KV, inter, intra, QK, the state's parts, Z^T (two chunks' with two parts)
constexpr uint32_t TM_KV = 0, TM_INTER = 128, TM_INTRA = 192, TM_QK = 256, TM_S = 320, TM_COLS = 512;

struct LinChunkParams {
    LinRun a;
    CUtensorMap tx, ty, tz, to;
    unsigned *status;
};

template <int DX, int DZ, int NSP, int NPP, typename TOut>
__global__ void __launch_bounds__(NT, 1) lin_chunk_fine_kernel(const __grid_constant__ LinChunkParams P)
{
    constexpr int JW = DZ / 32;                // warps with value channels of their own
    constexpr int NB = NPP == 1 ? 2 : 1;       // buffers of P
    constexpr bool ZT = NSP <= 2;              // Z^T in tensor memory, two buffers; no room beside three parts
    constexpr bool BF16_OUT = sizeof(TOut) == 2;
    constexpr uint32_t TM_ZT = TM_S + 64 * NSP;
    static_assert(TM_ZT + (ZT ? 64 : 0) <= TM_COLS, "tensor memory");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + SM_BAR);
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(sm + SM_MISC);
    volatile int *s_abort = reinterpret_cast<volatile int *>(sm + SM_MISC + 8);
    GateStage *gates = reinterpret_cast<GateStage *>(sm + SM_GATE);
    const LinRun &a = P.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
    const int h = blockIdx.x % a.H;
    const bool rev = a.reverse != 0;
    const Work work = lin_work(a, blockIdx.x / a.H);
    const int n = work.n, row0 = work.row0, len = work.len, nch = work.nch;
    if (a.seg_chunks && nch <= 0) return;
    const bool closing = rev ? work.c0 == 0 : work.c0 + nch == work.nall;   // the sequence's last segment in time
    const size_t soff = ((size_t)n * a.H + h) * DX * DZ, woff = ((size_t)work.slot * a.H + h) * DX * DZ;

    if (warp == 3) tmem_alloc(s_tmem, TM_COLS);
    if (tid == 0) {
        *s_abort = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar + B_FULL + s, 1);
            mbar_init(bar + B_GATE + s, 1);
            mbar_init(bar + B_EMPTY + s, 1 + 2 * JW + (BF16_OUT ? 4 : JW));
        }
        mbar_init(bar + B_QKF, 1);
        mbar_init(bar + B_QKE, 2);
        for (int s = 0; s < 2; ++s) {
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
    auto chunk = [&](int i) { return work.c0 + (rev ? nch - 1 - i : i); };
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
                if (!wait(bar + B_GATE + s, (i / NS) & 1, s_abort) || !wait(bar + B_QKF, i & 1, s_abort) ||
                    (i >= NB && !wait(bar + B_OF + pb, par(i - NB), s_abort)))
                    break;
                tc_fence_after();
                const int first = rev ? r : 0, last = rev ? G.nv - 1 : r;   // the row's tokens
                const float2 cr = G.c[r];
                const bool narrow = G.narrow != 0;
                const float af = rev ? G.b[r] : G.a[r];
                const float2 ar = make_float2(af, af);
                const float *bcol = rev ? G.a : G.b;
                uint8_t *prow = sm + SM_P + pb * 8192 + r * 128;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint32_t hi[16], lo[NPP == 2 ? 16 : 1];
                    if (rev ? half < warp : half > warp) {   // masked for all of the warp's rows
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            hi[e] = 0u;
                            if (NPP == 2) lo[e] = 0u;
                        }
                    } else {
                        float2 v[16];
                        tmem_ld32(tlane + TM_QK + half * 32, &v[0].x);
                        tmem_wait_ld();
                        if (narrow) {
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const float4 bs = *reinterpret_cast<const float4 *>(bcol + half * 32 + 2 * e);
                                v[e] = __fmul2_rn(__fmul2_rn(v[e], ar), make_float2(bs.x, bs.y));
                                v[e + 1] = __fmul2_rn(__fmul2_rn(v[e + 1], ar), make_float2(bs.z, bs.w));
                            }
                        } else {   // a strong decay or a reset in the chunk: each pair's own exponential
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float4 cs = *reinterpret_cast<const float4 *>(&G.c[half * 32 + 2 * e]);
                                const float d0 = diff(cr, make_float2(cs.x, cs.y)), d1 = diff(cr, make_float2(cs.z, cs.w));
                                v[e].x *= ex2(rev ? -d0 : d0);
                                v[e].y *= ex2(rev ? -d1 : d1);
                            }
                        }
                        if (half == warp || (rev && G.nv < C)) {   // columns that some row of the warp masks
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const int s0 = half * 32 + 2 * e;
                                if (s0 < first || s0 > last) v[e].x = 0.f;
                                if (s0 + 1 < first || s0 + 1 > last) v[e].y = 0.f;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (NPP == 2) {
                                hi[e] = take_part(v[e]);
                                lo[e] = pack_bf16(v[e].x, v[e].y);
                            } else {
                                hi[e] = pack_bf16(v[e].x, v[e].y);
                            }
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint4 *at = reinterpret_cast<uint4 *>(prow + (((half * 4 + q) ^ (r & 7)) << 4));
                        at[0] = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
                        if (NPP == 2) at[512] = make_uint4(lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
                    }
                }
                tc_fence_before();
                warp_arrive(bar + B_QKE);
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
                // e^g is 0 far before -10^4 (and infinite before 10^4, which breaks the contract)
                const float ga = fminf(fmaxf(next[0], -1e4f), 1e4f), gb = fminf(fmaxf(next[1], -1e4f), 1e4f);
                const unsigned nan_a = __ballot_sync(0xffffffffu, next[0] != next[0]);
                const unsigned nan_b = __ballot_sync(0xffffffffu, next[1] != next[1]);
                if (i + 1 < nch) gate_load(i + 1);
                const long long fb = fix_log2(gb);
                long long run = fix_log2(ga) + fb;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const long long o = __shfl_up_sync(0xffffffffu, run, off);
                    if (lane >= off) run += o;
                }
                const long long end = __shfl_sync(0xffffffffu, run, 31), mid = end >> 1;
                const float nan = __int_as_float(0x7fc00000);
                bool narrow = (nan_a | nan_b) == 0;
#pragma unroll 1
                for (int e = 0; e < 2; ++e) {
                    const int t = 2 * lane + e;
                    const long long c = e ? run : run - fb;
                    float2 cc = make_float2((float)fix_int(c), fix_rest(c));
                    float since = fix_exp2(c), left = fix_exp2(end - c);
                    G.a[t] = fix_exp2(c - mid);
                    G.b[t] = fix_exp2(mid - c);
                    narrow = narrow && c - mid < (100ll << 32) && mid - c < (100ll << 32);
                    if (nan_a | nan_b) {   // a NaN decay is part of every sum from its token on
                        const unsigned upto = 0xffffffffu >> (31 - lane);
                        if ((nan_a & upto) || (nan_b & (e ? upto : upto >> 1))) cc.x = since = nan;
                        left = nan;
                    }
                    G.c[t] = cc;
                    G.w_in[t] = rev ? left : since;
                    G.w_out[t] = rev ? since : left;
                }
                narrow = __all_sync(0xffffffffu, narrow);
                if (lane == 0) {
                    G.total = (nan_a | nan_b) ? nan : fix_exp2(end);
                    G.nv = nv;
                    G.narrow = narrow;
                }
                warp_arrive(bar + B_GATE + s);
            }
            // no load is in flight when the CTA ends, wound down early or not
            if (lane == 0)
                for (int j = max(0, i - NS); j < i; ++j) mbar_wait_cycles(bar + B_FULL + j % NS, (j / NS) & 1, WAIT_LIMIT);
        } else {
            // ---- MMA issue
            const uint32_t lead = lane == 0;
            constexpr uint32_t ID_QK = idesc_bf16(128, C, false, false), ID_KV = idesc_bf16(128, DX, !ZT, true);
            constexpr uint32_t ID_INTER = idesc_bf16(128, C, false, false), ID_INTRA = idesc_bf16(128, C, !ZT, false);
            bool ok = true;
            const uint32_t kb = mn_tile(sb + SM_KB), pt = k_tile(sb + SM_P);
            uint32_t xt = k_tile(sb);                    // X of the chunk at hand, its Y and Z one and two tiles on
            int s = 0;
            for (int i = -1; i < nch && ok; ++i) {
                const uint32_t zt = tbase + TM_ZT + (i & 1) * 32;
                if (i >= 0) {
                    ok = wait(bar + B_KBF, i & 1, s_abort) && (i == 0 || wait(bar + B_KVE, (i - 1) & 1, s_abort));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t za = mn_tile(sb + s * STAGE + 2 * TILE);
#pragma unroll 1
                    for (int p = 0; p < 3; ++p)
#pragma unroll
                        for (int kk = 0; kk < C / 16; ++kk) {
                            const uint32_t b = dMN(kb, kk) + p * (TILE >> 4);
                            if (ZT) mma_bf16_ts_warp(tbase + TM_KV, zt + kk * 8, b, ID_KV, p + kk > 0, lead);
                            else mma_bf16_warp(tbase + TM_KV, dMN(za, kk), b, ID_KV, p + kk > 0, lead);
                        }
                    mma_commit_warp(bar + B_KVF, lead);
                }
                if (i + 1 < nch) {   // QK of the next one; rows 64-127 of A are what lies behind X: lanes nobody reads
                    const int sn = (i + 1) % NS;
                    const uint32_t xn = k_tile(sb + sn * STAGE);
                    ok = wait(bar + B_FULL + sn, ((i + 1) / NS) & 1, s_abort) &&
                         (i < 0 || wait(bar + B_QKE, i & 1, s_abort));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int p = 0; p < DX / 64; ++p)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_bf16_warp(tbase + TM_QK, dK(xn, kk) + p * 512, dK(xn + (TILE >> 4), kk) + p * 512, ID_QK,
                                          p + kk > 0, lead);
                    mma_commit_warp(bar + B_QKF, lead);
                }
                if (i < 0) continue;
                ok = wait(bar + B_SF, i & 1, s_abort) && (i == 0 || wait(bar + B_OE, (i - 1) & 1, s_abort));
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int p = 0; p < NSP * (DX / 64); ++p) {   // a part's panel of 64 key channels
                    const int part = p / (DX / 64), panel = p % (DX / 64);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16_ts_warp(tbase + TM_INTER, tbase + TM_S + part * 64 + panel * 32 + kk * 8,
                                         dK(xt, kk) + panel * 512, ID_INTER, p + kk > 0, lead);
                }
                mma_commit_warp(bar + B_SE, lead);
                ok = wait(bar + B_PF + i % NB, par(i), s_abort);
                if (!ok) break;
                tc_fence_after();
                const uint32_t za = mn_tile(sb + s * STAGE + 2 * TILE);
#pragma unroll
                for (int p = 0; p < NPP; ++p)
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk) {
                        const uint32_t b = dK(pt + (i % NB + p) * 512, kk);
                        if (ZT) mma_bf16_ts_warp(tbase + TM_INTRA, zt + kk * 8, b, ID_INTRA, p + kk > 0, lead);
                        else mma_bf16_warp(tbase + TM_INTRA, dMN(za, kk), b, ID_INTRA, p + kk > 0, lead);
                    }
                mma_commit_warp(bar + B_OF + i % NB, lead);
                mma_commit_warp(bar + B_EMPTY + s, lead);
                s = s == NS - 1 ? 0 : s + 1;
                xt = k_tile(sb + s * STAGE);
            }
            // products still running are waited for below (every product of a full run is, by its readers)
            if (!ok) {
                mma_commit_warp(bar + B_DRAIN, lead);
                mbar_wait_cycles(bar + B_DRAIN, 0, WAIT_LIMIT);
            }
        }
    } else if (wg <= 2) {
        regs_dec<RG_YBAR>();
        // ---- Ybar
        constexpr int YT = 256;
        const int t = tid - 128, zq = warp & 3;
        // this lane's row of the first 8x8 piece of channels 32 zq (a piece of 16 more tokens is 2048 bytes on,
        // of 16 more channels two 16-byte columns on, under the swizzle)
        const int zch = (zq & 1) * 4 + ((lane >> 3) & 1), zr = (lane >> 4) * 8 + (lane & 7);
        const uint32_t zaddr0 = sb + 2 * TILE + (zq >> 1) * 8192 + zr * 128 + ((zch ^ (zr & 7)) << 4);
        const uint32_t zstep = ((((zch + 2) ^ (zr & 7)) << 4)) - ((zch ^ (zr & 7)) << 4);
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
            // Z^T, the A operand of KV and intra: 8x8 pieces, transposed on their way to registers
            uint32_t zt[2][16];
            bool clean = true;
#pragma unroll 1
            for (int pass = 0;; ++pass) {
                uint32_t most = 0;
                if (wg == 1 && zq < JW) {
#pragma unroll
                    for (int g = 0; g < 2; ++g)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            ldmatrix_x4_trans(zaddr0 + s * STAGE + k * 2048 + (g ? zstep : 0), zt[g] + 4 * k);
                        }
#pragma unroll
                    for (int e = 0; e < 16; ++e) most = max_abs2(most, max_abs2(zt[0][e], zt[1][e]));
                }
                if (pass) break;
                clean = group_sync_and(1, YT, (most & 0x7fffu) < 0x7f80u && (most & 0x7fff0000u) < 0x7f800000u);
                if (t == 0) G.bad = !clean;
                if (clean) break;
                if (t < 128) {
                    int from = rev ? -1 : C;
                    if (t < DZ) {
#pragma unroll 1
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
                group_sync(1, YT);   // once more, without them
            }
            // KV_{i-1} has read Ybar, and what was issued before it (intra_{i-2}) this buffer of Z^T
            ok = i == 0 || wait(bar + B_KVF, (i - 1) & 1, s_abort);
            if (!ok) continue;
            if (ZT && wg == 1 && zq < JW) {
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    tmem_st_frag8(tlane + ((uint32_t)(g * 16) << 16) + TM_ZT + (i & 1) * 32, zt[g]);
                tmem_wait_st();
                tc_fence_before();
            }
#pragma unroll 1
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
            // Fragments of O^T (channel, token pair) go transposed into [token][channel] panels over this
            // stage's X, which nobody reads any more, and leave from there by TMA (the last, ragged chunk of
            // a sequence row by row: what lies behind it is another sequence's).
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
                        const int r = half * 32 + (lane >> 4) * 8 + (lane & 7), ch = (q & 1) * 4 + g * 2 + ((lane >> 3) & 1);
                        const uint32_t to = stage + (q >> 1) * 8192 + r * 128 + ((ch ^ (r & 7)) << 4);
                        stmatrix_x4_trans(to, pk[0], pk[1], pk[2], pk[3]);
                        stmatrix_x4_trans(to + 16 * 128, pk[4], pk[5], pk[6], pk[7]);
                    }
                }
                fence_async_smem();
                group_sync(2, 128);
                if (nv == C) {
                    if (tid == 3 * 128) {
#pragma unroll
                        for (int p = 0; p < DZ / 64; ++p)
                            tma_store_3d(&P.to, sm + s * STAGE + p * 8192, p * 64, h, row0 + t0);
                        bulk_commit();
                        bulk_wait_read();
                    }
                } else {
                    for (int e = tid - 3 * 128; e < nv * (DZ / 8); e += 128) {
                        const int r = e / (DZ / 8), ch = e % (DZ / 8);
                        *reinterpret_cast<uint4 *>((TOut *)a.out + ((size_t)row0 + t0 + r) * ld + (size_t)h * DZ + ch * 8) =
                            *reinterpret_cast<const uint4 *>(sm + s * STAGE + (ch >> 3) * 8192 + r * 128 +
                                                             (((ch & 7) ^ (r & 7)) << 4));
                    }
                }
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
            const float *s_in = a.seg_chunks ? a.seg_state + woff : a.s_in ? a.s_in + soff : nullptr;
            float *s_out = a.s_out && closing ? a.s_out + soff : nullptr;
            if (s_in && a.in_t && !a.seg_chunks) {
#pragma unroll
                for (int e = 0; e < CX / 2; ++e)
                    S[e] = *reinterpret_cast<const float2 *>(s_in + (size_t)j * DX + i0 + 2 * e);
            } else if (s_in) {
                const float *at = s_in + (size_t)i0 * DZ + j;
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
                const int edge = rev ? (i < nch ? min(len, (chunk(i) + 1) * C) - 1 : -1)
                                     : (i > 0 ? min(len, (work.c0 + i) * C) - 1 : -1);
                if (a.snap && edge >= 0 && (edge == len - 1 || (edge + 1) % a.snap_tokens == 0))
                    to[0] = a.snap + ((size_t)(n + row0 / a.snap_tokens + edge / a.snap_tokens) * a.H + h) * DX * DZ;
                if (i == nch) to[1] = s_out;
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
            if (!ok && s_out)
                for (int e = 0; e < CX; ++e) s_out[(size_t)(i0 + e) * DZ + j] = __int_as_float(0x7fc00000);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 3) tmem_dealloc(tbase, TM_COLS);
    if (tid == 0 && *s_abort) atomicOr(P.status, DEV_WAIT_TIMEOUT);
}

template <int DX, int DZ, int NSP, int NPP, typename TOut> cudaError_t launch_dims(const LinRun &r, cudaStream_t st)
{
    static bool done[64] = {};
    cudaError_t e = opt_in(lin_chunk_fine_kernel<DX, DZ, NSP, NPP, TOut>, SM_ALLOC, done);
    if (e != cudaSuccess) return e;
    LinChunkParams p;
    memset(&p, 0, sizeof(p));
    p.a = r;
    if ((e = device_status_word(&p.status)) != cudaSuccess) return e;
    const long long rows = r.rows;
    if (rows > 0 && (!make_map(&p.tx, r.x, rows, r.H / r.gx, DX) || !make_map(&p.ty, r.y, rows, r.H / r.gy, DX) ||
                     !make_map(&p.tz, r.z, rows, r.H / r.gz, DZ) ||
                     (sizeof(TOut) == 2 && !make_map(&p.to, r.out, rows, r.H, DZ))))
        return cudaErrorInvalidValue;
    lin_chunk_fine_kernel<DX, DZ, NSP, NPP, TOut><<<(unsigned)((r.seg_chunks ? r.slots : r.num_seqs) * r.H), NT, SM_ALLOC, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_chunk_fine(const LinRun &r, int dx, int dz, cudaStream_t st)
{
    if (dx == 128 && dz == 128) return launch_dims<128, 128, 3, 2, float>(r, st);
    if (dx == 128 && dz == 64) return launch_dims<128, 64, 3, 2, float>(r, st);
    if (dx == 64 && dz == 128) return launch_dims<64, 128, 3, 2, float>(r, st);
    if (dx == 64 && dz == 64) return launch_dims<64, 64, 3, 2, float>(r, st);
    return cudaErrorInvalidValue;
}

}  // namespace kda
