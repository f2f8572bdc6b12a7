// Gate gradient of linear attention's chunk form on the tensor cores: the sums of lin_gate_chunk_kernel
// (linattn_grad.cu), for one chunk of 64 tokens and head,
//   dg_t = sum_{s < t <= r} L_rs (q_r . k_s) (do_r . v_s) + sum_{r >= t} w_r do_r^T S_0 q_r
//        + sum_{s < t} u_s v_s^T G_C k_s + e^{c_C} <S_0, G_C>,
// S_0 and G_C as the dq and dk passes left them at the chunk's ends ([d_v][d_k], fp32).
// Four products, D in tensor memory:  Q K^T and dO V^T (bf16 operands as loaded), and S_0 dO^T, G_C V^T
// with lanes = key channels (in which the states are contiguous) and the state in three bf16 parts (2^-24), A from
// tensor memory.  The rest is fp32: the inner products with q and k are lane sums, 16 tokens exchanged at once.
// A chunk and head have 2 states (8 d_k d_v bytes) and 4 tiles to read.  What takes the time are the steps that wait for
// one another (tiles, products, states, products): two CTAs an SM cover each other's, and 16 warps a CTA (8: 247 us)
// shorten them.  4 x 4096 tokens, 16 heads, 128 x 128: 233 us, 2.9 TB/s.
#include "linattn_sm100.cuh"

namespace kda {
namespace {

using namespace lin;

constexpr int NT = 512, ROWS = NT / 128;                 // warps of each quarter of the lanes
constexpr int TW = C / ROWS;                             // tokens of a warp
constexpr uint32_t SM_W = 4 * TILE;                      // q, k, dO, v tiles, then W [64][66]
constexpr int WP = 66;                                   // W's row pitch
constexpr uint32_t SM_END = SM_W + 64 * WP * 4;
constexpr uint32_t SM_ALLOC = SM_END + 1024;
constexpr uint32_t TM_D = 0, TM_S = 64, TM_COLS = 256;   // accumulator (the first product's second at TM_S), state parts

struct GateParams {
    LinGateGrad a;
    CUtensorMap q, k, v, d_o;
    unsigned *status;
};

template <int DK, int DV>
__global__ void __launch_bounds__(NT, 2) lin_gate_kernel(const __grid_constant__ GateParams P)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    float *s_w = reinterpret_cast<float *>(sm + SM_W);
    __shared__ __align__(8) uint64_t s_bar[2];   // tiles; products
    __shared__ uint32_t s_tmem;
    __shared__ float2 s_c[C];
    __shared__ float s_win[C], s_uout[C], s_red[2][4][C], s_dq[C], s_dk[C], s_x[NT / 32], s_tot, s_pre[NT / 32][C];
    const LinGateGrad &a = P.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quarter = warp & 3, part_of = warp >> 2;
    const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H;
    // sequence of the slot: the last one whose first slot is not behind it (first slots increase)
    int n = 0;
    {
        int lo = 0, hi = a.num_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (mid + (a.cu_seqlens ? a.cu_seqlens[mid] : mid * a.T) / C <= slot) lo = mid;
            else hi = mid - 1;
        }
        n = lo;
    }
    const int row0 = a.cu_seqlens ? a.cu_seqlens[n] : n * a.T;
    const int len = a.cu_seqlens ? a.cu_seqlens[n + 1] - row0 : a.T;
    const int t0 = (slot - n - row0 / C) * C;
    if (t0 < 0 || t0 >= len) {   // no chunk has this slot
        if (a.partial && tid == 0) a.partial[(size_t)slot * a.H + h] = 0.f;
        return;
    }
    const int nt = min(C, len - t0), hk = h / (a.H / a.Hk);
    const size_t row = (size_t)row0 + t0;

    // the states, on their way to L2 while the tiles are worked on
    const bool first = t0 == 0, last = t0 + nt >= len;
    const size_t size = (size_t)DK * DV;
    const float *st0 = first ? (a.s_init ? a.s_init + ((size_t)n * a.H + h) * size : nullptr)
                  : a.snap_s + ((size_t)(slot - 1) * a.H + h) * size;
    const float *st1 = last ? (a.g_end ? a.g_end + ((size_t)n * a.H + h) * size : nullptr)
                 : a.snap_g + ((size_t)slot * a.H + h) * size;
    for (int e = tid; e < DK * DV / 32; e += NT) {
        if (st0) asm volatile("prefetch.global.L2 [%0];" :: "l"(st0 + e * 32));
        if (st1) asm volatile("prefetch.global.L2 [%0];" :: "l"(st1 + e * 32));
    }

    const bool stall = a.stall && blockIdx.x == 0;
    if (warp == 0) tmem_alloc(&s_tmem, TM_COLS);
    if (tid == 0) {
        mbar_init(s_bar, 1);
        mbar_init(s_bar + 1, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (!stall) {
            mbar_expect_tx(s_bar, (DK + DV) * 2 * C * 2);
#pragma unroll
            for (int p = 0; p < DK / 64; ++p) {
                tma_load_3d(sm + p * 8192, &P.q, s_bar, p * 64, hk, (int)row);
                tma_load_3d(sm + TILE + p * 8192, &P.k, s_bar, p * 64, hk, (int)row);
            }
#pragma unroll
            for (int p = 0; p < DV / 64; ++p) {
                tma_load_3d(sm + 2 * TILE + p * 8192, &P.d_o, s_bar, p * 64, h, (int)row);
                tma_load_3d(sm + 3 * TILE + p * 8192, &P.v, s_bar, p * 64, h, (int)row);
            }
        }
    }
    if (warp == 1) {   // sums of log2-decays
        const float g0 = 2 * lane < nt ? a.g[(row + 2 * lane) * a.g_ld + h] : 0.f;
        const float g1 = 2 * lane + 1 < nt ? a.g[(row + 2 * lane + 1) * a.g_ld + h] : 0.f;
        const bool nan = __any_sync(0xffffffffu, g0 != g0 || g1 != g1);
        const long long f1 = fix_log2(fminf(fmaxf(g1, -1e4f), 1e4f));
        long long run = fix_log2(fminf(fmaxf(g0, -1e4f), 1e4f)) + f1;
        for (int off = 1; off < 32; off <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, run, off);
            if (lane >= off) run += o;
        }
        const long long end = __shfl_sync(0xffffffffu, run, 31);
        for (int e = 0; e < 2; ++e) {
            const long long c = e ? run : run - f1;
            const int t = 2 * lane + e;
            s_c[t] = make_float2(nan ? NAN : (float)fix_int(c), fix_rest(c));
            s_win[t] = nan ? NAN : fix_exp2(c);
            s_uout[t] = nan ? NAN : fix_exp2(end - c);
        }
        if (lane == 0) s_tot = nan ? NAN : fix_exp2(end);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = s_tmem, tlane = tbase + ((uint32_t)(quarter * 32) << 16);
    bool ok = mbar_wait_cycles(s_bar, 0, stall ? STALL_LIMIT : WAIT_LIMIT);
    ok = __syncthreads_and(ok) != 0;
    uint32_t products = 0;   // of which all but the last are complete
    // products are issued by warp 0, everybody waits for them
    auto finish = [&]() {
        if (warp == 0) mma_commit_warp(s_bar + 1, lane == 0);
        ok = __syncthreads_and(mbar_wait_cycles(s_bar + 1, products & 1, WAIT_LIMIT)) != 0 && ok;
        ++products;
        tc_fence_after();
    };

    if (ok) {
        // Q K^T and dO V^T; rows 64-127 of A are what lies behind: lanes nobody reads
        constexpr uint32_t ID = idesc_bf16(128, C, false, false);
        if (warp == 0) {
            const uint32_t lead = lane == 0, q = k_tile(sb), k = k_tile(sb + TILE), d = k_tile(sb + 2 * TILE), v = k_tile(sb + 3 * TILE);
#pragma unroll
            for (int e = 0; e < DK / 16; ++e) mma_bf16_warp(tbase + TM_D, dK(q, e), dK(k, e), ID, e > 0, lead);
#pragma unroll
            for (int e = 0; e < DV / 16; ++e) mma_bf16_warp(tbase + TM_S, dK(d, e), dK(v, e), ID, e > 0, lead);
        }
        finish();
        if (ok && quarter < 2) {   // row r of W, 16 columns
            const int r = quarter * 32 + lane, s0 = part_of * TW;
            float x[TW], y[TW];
            tmem_ld16(tlane + TM_D + s0, x);
            tmem_ld16(tlane + TM_S + s0, y);
            tmem_wait_ld();
            const float2 cr = s_c[r];
#pragma unroll
            for (int e = 0; e < TW; ++e)
                s_w[r * WP + s0 + e] = s0 + e < r ? x[e] * y[e] * ex2(diff(cr, s_c[s0 + e])) : 0.f;
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }

    // the two state products: S_0 with dO, weighed by q; G_C with v, weighed by k
    const int i = quarter * 32 + lane, j0 = part_of * (DV / ROWS);
    float accx = 0.f;
#pragma unroll 1
    for (int m = 0; m < 2; ++m) {
        if (!ok || !(m ? st1 : st0)) continue;   // (uniform)
        if (i < DK) {
            // the caller's states are [dk][dv], the passes' [dv][dk]
            const bool nat = m ? last : first;
            const float *at = (m ? st1 : st0) + (nat ? (size_t)i * DV + j0 : (size_t)j0 * DK + i);
            const float *other = m == 0 && st1 ? st1 + (last ? (size_t)i * DV + j0 : (size_t)j0 * DK + i) : nullptr;
            const int step = nat ? 1 : DK, ostep = last ? 1 : DK;
#pragma unroll 1
            for (int b = 0; b < DV / ROWS / 16; ++b) {   // 16 value channels
                float x[16], z[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = at[(b * 16 + e) * step];
                if (other) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) z[e] = other[(b * 16 + e) * ostep];
#pragma unroll
                    for (int e = 0; e < 16; ++e) accx = fmaf(x[e], z[e], accx);
                }
                uint32_t part[3][8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float2 w = make_float2(x[2 * e], x[2 * e + 1]);
                    part[0][e] = take_part(w);
                    part[1][e] = take_part(w);
                    part[2][e] = pack_bf16(w.x, w.y);
                }
#pragma unroll
                for (int p = 0; p < 3; ++p) tmem_st8(tlane + TM_S + p * 64 + j0 / 2 + b * 8, part[p]);
            }
            tmem_wait_st();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == 0) {
            constexpr uint32_t ID = idesc_bf16(128, C, false, false);
            const uint32_t b = k_tile(sb + (2 + m) * TILE);
#pragma unroll 4
            for (int e = 0; e < 3 * DV / 16; ++e) {
                const int kk = e % (DV / 16);
                mma_bf16_ts_warp(tbase + TM_D, tbase + TM_S + (e / (DV / 16)) * 64 + kk * 8, dK(b, kk), ID, e > 0, lane == 0);
            }
        }
        finish();
        if (ok) {
            // this warp's 32 channels and 16 tokens: lane sums, halved and exchanged; lanes 2 l, 2 l + 1 keep token l
            float y[TW];
            tmem_ld16(tlane + TM_D + part_of * TW, y);
            tmem_wait_ld();
            const uint8_t *tile = sm + m * TILE + (i >> 6) * 8192;
#pragma unroll
            for (int e = 0; e < TW; ++e) {
                const int r = part_of * TW + e;
                const unsigned short w = *reinterpret_cast<const unsigned short *>(tile + r * 128 + (((i & 63) * 2) ^ ((r & 7) << 4)));
                y[e] = i < DK ? y[e] * __uint_as_float((uint32_t)w << 16) : 0.f;
            }
#pragma unroll
            for (int off = 16, cnt = 8; cnt; off >>= 1, cnt >>= 1) {
                const bool up = (lane & off) != 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (e < cnt) {
                        const float send = up ? y[e] : y[e + cnt], keep = up ? y[e + cnt] : y[e];
                        y[e] = keep + __shfl_xor_sync(0xffffffffu, send, off);
                    }
                }
            }
            y[0] += __shfl_xor_sync(0xffffffffu, y[0], 1);
            if (!(lane & 1)) s_red[m][quarter][part_of * TW + (lane >> 1)] = y[0];
        }
        tc_fence_before();
        __syncthreads();   // D and the parts are read
        tc_fence_after();
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) accx += __shfl_xor_sync(0xffffffffu, accx, off);
    if (lane == 0) s_x[warp] = accx;
    __syncthreads();
    if (tid < 2 * C) {
        const int m = tid >> 6, r = tid & 63;
        const float sum = (m ? st1 : st0) ? (s_red[m][0][r] + s_red[m][1][r]) + (s_red[m][2][r] + s_red[m][3][r]) : 0.f;
        if (m == 0) s_dq[r] = r < nt && st0 ? s_win[r] * sum : 0.f;
        else s_dk[r] = r < nt && st1 ? s_uout[r] * sum : 0.f;
    }
    {   // p_r(t) = sum_{s < t} W_rs, summed over the warp's rows r >= t; a lane has t = 2 lane, 2 lane + 1
        float y0 = 0.f, y1 = 0.f;
#pragma unroll
        for (int e = 0; e < C * 32 / NT; ++e) {
            const int r = warp * (C * 32 / NT) + e;
            const float2 w = *reinterpret_cast<const float2 *>(s_w + r * WP + 2 * lane);
            float run = w.x + w.y;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float o = __shfl_up_sync(0xffffffffu, run, off);
                if (lane >= off) run += o;
            }
            float before = __shfl_up_sync(0xffffffffu, run, 1);
            if (lane == 0) before = 0.f;
            if (r >= 2 * lane && r < nt) y0 += before;
            if (r >= 2 * lane + 1 && r < nt) y1 += before + w.x;
        }
        s_pre[warp][2 * lane] = y0;
        s_pre[warp][2 * lane + 1] = y1;
    }
    __syncthreads();
    if (warp == 0) {   // t = 2 lane, 2 lane + 1
        const int t = 2 * lane;
        float x[2] = {0.f, 0.f};
        for (int w = 0; w < NT / 32; ++w) {
            x[0] += s_pre[w][t];
            x[1] += s_pre[w][t + 1];
        }
        const float q0 = s_dq[t], q1 = s_dq[t + 1], k0 = s_dk[t], k1 = s_dk[t + 1];
        float after = q0 + q1, before = k0 + k1;   // sums of dq from t on, of dk up to t + 1
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const float o = __shfl_down_sync(0xffffffffu, after, off), u = __shfl_up_sync(0xffffffffu, before, off);
            if (lane + off < 32) after += o;
            if (lane >= off) before += u;
        }
        float sq = __shfl_down_sync(0xffffffffu, after, 1), sk = __shfl_up_sync(0xffffffffu, before, 1);
        if (lane == 31) sq = 0.f;
        if (lane == 0) sk = 0.f;
        float cross = 0.f;
        if (st0 && st1) {
            for (int w = 0; w < NT / 32; ++w) cross += s_x[w];
            cross *= s_tot;
        }
        x[0] = (x[0] + (q0 + q1 + sq)) + (sk + cross);
        x[1] = (x[1] + (q1 + sq)) + (sk + k0 + cross);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (t + e >= nt) continue;
            float d = ok ? x[e] : NAN;
            // e^g has slope 0 at -infinity (the states' products may have an infinity's NaN there)
            if (a.g[(row + t + e) * a.g_ld + h] == -INFINITY) d = 0.f;
            if (a.dg) a.dg[(row + t + e) * a.H + h] = d;
            sum += d;
        }
        if (a.partial) {
#pragma unroll
            for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (lane == 0) a.partial[(size_t)slot * a.H + h] = sum;
        }
    }
    if (!ok && tid == 0) {   // what was started ends before the CTA does
        atomicOr(P.status, DEV_WAIT_TIMEOUT);
        if (!stall) mbar_wait_cycles(s_bar, 0, WAIT_LIMIT);
        if (products) mbar_wait_cycles(s_bar + 1, (products - 1) & 1, WAIT_LIMIT);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tbase, TM_COLS);
}

template <int DK, int DV> cudaError_t launch_dims(const LinGateGrad &a, cudaStream_t st)
{
    static bool done[64] = {};
    cudaError_t e = opt_in(lin_gate_kernel<DK, DV>, SM_ALLOC, done);
    GateParams p;
    memset(&p, 0, sizeof(p));
    p.a = a;
    if (e != cudaSuccess || (e = bind_context()) != cudaSuccess || (e = device_status_word(&p.status)) != cudaSuccess) return e;
    if (!make_map(&p.q, a.q, a.rows, a.Hk, DK) || !make_map(&p.k, a.k, a.rows, a.Hk, DK) ||
        !make_map(&p.v, a.v, a.rows, a.H, DV) || !make_map(&p.d_o, a.d_o, a.rows, a.H, DV))
        return cudaErrorInvalidValue;
    lin_gate_kernel<DK, DV><<<(unsigned)((long long)a.slots * a.H), NT, SM_ALLOC, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_gate_chunk(const LinGateGrad &a, cudaStream_t st)
{
    if (a.dk == 128 && a.dv == 128) return launch_dims<128, 128>(a, st);
    if (a.dk == 128 && a.dv == 64) return launch_dims<128, 64>(a, st);
    if (a.dk == 64 && a.dv == 128) return launch_dims<64, 128>(a, st);
    if (a.dk == 64 && a.dv == 64) return launch_dims<64, 64>(a, st);
    return cudaErrorInvalidValue;
}

}  // namespace kda
