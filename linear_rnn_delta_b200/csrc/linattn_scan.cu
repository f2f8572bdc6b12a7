// Token-by-token fp32 scan of linear attention with one decay per head.
//
// Serves fp32 inputs and the head sizes that the tensor-core chunked kernel does not take.  Columns of the
// state evolve independently, so a CTA owns a block of value columns of one (sequence, head), or of a
// segment of it.  KS = d_x / 8 adjacent lanes form a group that owns 4 columns: lane p of it keeps rows
// 8p .. 8p+7 of them in registers.  Tokens go in blocks of 8 by their place in the sequence.  Within a
// block the state is kept without its decay, S = 2^{L_u} Z with L_u the sum of log2-decays up to step u:
//   Z += y_u (2^{-L_u} z_u)^T,   out_u = 2^{L_u} Z^T x_u,
// two packed multiply-adds for two elements where S = a S + y z^T costs three operations and rounds
// twice as often; S is formed at the block's end.  A block that decays by more than 2^-60 (a reset, say)
// takes the plain way.  The sum over a group's lanes is taken for 4 tokens at once: 16 partial sums
// (4 tokens x 4 columns) are halved and exchanged log2(KS) times, so that a group spends 16 - 16/KS shuffles
// where a butterfly for each value would take 16 log2(KS).
//
// Blocks are double buffered in shared memory as fp32: block b+1 is loaded into registers while block b is
// computed.  Backward in time a step's decay is that of the token behind it (none at a segment's last
// token, whose entering state has it already; the state that leaves a segment has its first token's).  Steps
// without a token have x = y = z = 0 and no decay: they leave the state as it is.
// Bound by issue: 8 packed multiply-adds, 5 16-byte shared loads and 4 shuffles a token for 32 elements a lane.  One
// warp an SM sub-partition takes 200 ns a token, so few (sequence, head) pairs are cut into segments, like the
// chunk form's: their states first (two thirds of the work), then all segments side by side.  2 x 300 tokens, 2 heads,
// 32 x 64: 4 and 6 us in segments of 16 tokens (of 64: 9 and 15); 2 x 1001, 8 heads, 64 x 128: 19 and 41 us.
#include <algorithm>
#include <cmath>

#include "linattn_sm100.cuh"

namespace kda {
namespace {

using lin::fix_exp2;
using lin::fix_exp2_steady;
using lin::fix_log2;
using lin::load4;

constexpr int TB = 8;    // tokens of a block
constexpr int TU = 4;    // tokens whose sums are exchanged together
constexpr long long NARROW = 60ll << 32;

template <int DX, int DZ> struct LinScanShape {
    static constexpr int KS = DX / 8;                             // lanes of a group
    static constexpr int MAXG = 128 / KS;                         // groups of a CTA of 128 threads
    static constexpr int CB = DZ / 4 <= MAXG ? DZ : MAXG * 4;     // columns of a CTA
    static constexpr int LIVE = CB / 4 * KS;                      // lanes with work
    static constexpr int NTH = LIVE < 32 ? 32 : LIVE;
    static constexpr int CTAS = DZ / CB;
    static_assert(NTH % 32 == 0 && (LIVE % 32 == 0 || LIVE < 32), "whole warps");
};

// STATE: only the state that a segment adds from nothing, and its decay.
template <int DX, int DZ, typename TIn, bool STATE>
__global__ void __launch_bounds__(LinScanShape<DX, DZ>::NTH) lin_scan_kernel(const __grid_constant__ LinRuns P)
{
    const LinRun &a = P.a[blockIdx.y];
    using SH = LinScanShape<DX, DZ>;
    constexpr int KS = SH::KS, CB = SH::CB, LIVE = SH::LIVE, NTH = SH::NTH, CTAS = SH::CTAS;
    __shared__ __align__(16) float s_x[2][STATE ? 1 : TB][DX], s_y[2][TB][DX], s_z[2][TB][CB];
    __shared__ float s_dec[2][TB], s_in[2][TB], s_out[2][TB], s_end[2];   // a_u; 2^{-L_u}, 2^{L_u} (1 in a wide block)
    __shared__ int s_wide[2];

    const int pair = blockIdx.x / CTAS, cblk = blockIdx.x % CTAS;
    const int h = pair % a.H;
    const lin::Work work = lin::lin_work<SCAN_CHUNK>(a, pair / a.H);
    if (a.seg_chunks && work.nch <= 0) return;
    const bool rev = a.reverse != 0;
    const bool closing = rev ? work.c0 == 0 : work.c0 + work.nch == work.nall;   // the sequence's last segment in time
    if (STATE && closing) return;   // nobody asks for the state behind it
    const int tid = threadIdx.x;
    const bool live = tid < LIVE;
    const int p = tid % KS, grp = live ? tid / KS : 0;
    const int j = cblk * CB + grp * 4;                 // first of the group's columns
    const int n = work.n, row0 = work.row0, len = work.len;
    const int beg = work.c0 * SCAN_CHUNK, end = min(len, beg + work.nch * SCAN_CHUNK);   // the segment's tokens
    const int hx = a.H / a.gx, hy = a.H / a.gy, hz = a.H / a.gz;
    const TIn *x = (const TIn *)a.x + (size_t)(h / a.gx) * DX, *y = (const TIn *)a.y + (size_t)(h / a.gy) * DX;
    const TIn *z = (const TIn *)a.z + (size_t)(h / a.gz) * DZ + cblk * CB;
    const size_t soff = ((size_t)n * a.H + h) * DX * DZ, woff = ((size_t)work.slot * a.H + h) * DX * DZ;

    const float *sin = STATE ? nullptr : a.seg_chunks ? a.seg_state + woff : a.s_in ? a.s_in + soff : nullptr;
    const bool in_t = a.in_t && !a.seg_chunks;
    float2 S[8][2];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const int i = 8 * p + r;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (sin && live) {
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = in_t ? sin[(size_t)(j + c) * DX + i] : sin[(size_t)i * DZ + j + c];
        }
        S[r][0] = make_float2(v[0], v[1]);
        S[r][1] = make_float2(v[2], v[3]);
    }

    constexpr int UX = TB * DX / 4, UZ = TB * CB / 4;   // groups of 4 elements of a block
    constexpr int EX = (UX + NTH - 1) / NTH, EZ = (UZ + NTH - 1) / NTH;
    float4 px[STATE ? 1 : EX], py[EX], pz[EZ];
    float pg = 0.f;
    long long sum = 0;   // STATE: this lane's share of the segment's log-decays
    bool any_nan = false;
    const int nblk = (end - beg + TB - 1) / TB;          // beg is a multiple of TB
    // token of step u of the b-th block in time
    auto token = [&](int b, int u) { return rev ? beg + (nblk - 1 - b) * TB + TB - 1 - u : beg + b * TB + u; };
    auto fetch = [&](int b) {
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int e = 0; e < EX; ++e) {
            const int w = tid + e * NTH, u = w / (DX / 4), i = w % (DX / 4) * 4, t = token(b, u);
            py[e] = zero;
            if (!STATE) px[e] = zero;
            if (u < TB && t < end) {
                const size_t row = (size_t)row0 + t;
                if (!STATE) px[e] = load4(x + row * hx * DX + i);
                py[e] = load4(y + row * hy * DX + i);
            }
        }
#pragma unroll
        for (int e = 0; e < EZ; ++e) {
            const int w = tid + e * NTH, u = w / (CB / 4), i = w % (CB / 4) * 4, t = token(b, u);
            pz[e] = zero;
            if (u < TB && t < end) pz[e] = load4(z + ((size_t)row0 + t) * hz * DZ + i);
        }
        if (tid < TB) {   // whose decay the step has
            const int t = token(b, tid) + (rev ? 1 : 0);
            pg = t < end ? a.g[((size_t)row0 + t) * a.g_ld + h] : 0.f;
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int e = 0; e < EX; ++e) {
            const int w = tid + e * NTH, u = w / (DX / 4), i = w % (DX / 4) * 4;
            if (u < TB) {
                if (!STATE) *reinterpret_cast<float4 *>(&s_x[buf][STATE ? 0 : u][i]) = px[e];
                *reinterpret_cast<float4 *>(&s_y[buf][u][i]) = py[e];
            }
        }
#pragma unroll
        for (int e = 0; e < EZ; ++e) {
            const int w = tid + e * NTH, u = w / (CB / 4), i = w % (CB / 4) * 4;
            if (u < TB) *reinterpret_cast<float4 *>(&s_z[buf][u][i]) = pz[e];
        }
        if (tid < 32) {   // lanes 0-7 have the block's decays
            const long long f = fix_log2(fminf(fmaxf(pg, -1e4f), 1e4f));
            const bool nan = pg != pg;
            long long L = tid < TB ? f : 0;
#pragma unroll
            for (int off = 1; off < TB; off <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, L, off);
                if (tid >= off) L += o;
            }
            const bool fits = L < NARROW && -L < NARROW && !nan;
            const bool wide = __any_sync(0xffffffffu, tid < TB && !fits);
            if (tid < TB) {
                s_dec[buf][tid] = wide ? (nan ? pg : fix_exp2_steady(f)) : 1.f;
                s_in[buf][tid] = wide ? 1.f : fix_exp2(-L);
                s_out[buf][tid] = wide ? 1.f : fix_exp2(L);
                if (tid == TB - 1) {
                    s_end[buf] = wide ? 1.f : fix_exp2_steady(L);
                    s_wide[buf] = wide;
                }
                if (STATE) {
                    sum = max(sum + f, lin::FIX_LEAST);
                    any_nan = any_nan || nan;
                }
            }
        }
    };
    auto write_state = [&](float *dst, float by) {   // [DX][DZ]
        if (!live) return;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int i = 8 * p + r;
            *reinterpret_cast<float4 *>(dst + (size_t)i * DZ + j) =
                make_float4(S[r][0].x * by, S[r][0].y * by, S[r][1].x * by, S[r][1].y * by);
        }
    };
    // the state at a boundary: behind token t forward, entering it backward
    auto snap = [&](int t) {
        if (STATE || !a.snap || t < 0 || (t != len - 1 && (t + 1) % a.snap_tokens)) return;
        write_state(a.snap + ((size_t)(n + row0 / a.snap_tokens + t / a.snap_tokens) * a.H + h) * DX * DZ, 1.f);
    };

    if (nblk > 0) fetch(0);
    if (rev && nblk > 0) snap(end - 1);
    for (int b = 0, buf = 0; b < nblk; ++b, buf ^= 1) {
        stage(buf);
        __syncthreads();   // this block is staged, and nobody reads the buffer of the one before the last
        if (b + 1 < nblk) fetch(b + 1);
        const bool wide = s_wide[buf] != 0;
#pragma unroll 1
        for (int u0 = 0; u0 < TB; u0 += TU) {
            float acc[4 * TU];
#pragma unroll
            for (int u = 0; u < TU; ++u) {
                const int w = u0 + u;
                if (wide) {
                    const float2 d = make_float2(s_dec[buf][w], s_dec[buf][w]);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        S[r][0] = __fmul2_rn(S[r][0], d);
                        S[r][1] = __fmul2_rn(S[r][1], d);
                    }
                }
                const float f = s_in[buf][w];
                const float4 z4 = *reinterpret_cast<const float4 *>(&s_z[buf][w][grp * 4]);
                const float2 z01 = make_float2(z4.x * f, z4.y * f), z23 = make_float2(z4.z * f, z4.w * f);
                float yv[8];
                *reinterpret_cast<float4 *>(yv) = *reinterpret_cast<const float4 *>(&s_y[buf][w][8 * p]);
                *reinterpret_cast<float4 *>(yv + 4) = *reinterpret_cast<const float4 *>(&s_y[buf][w][8 * p + 4]);
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const float2 y2 = make_float2(yv[r], yv[r]);
                    S[r][0] = __ffma2_rn(y2, z01, S[r][0]);
                    S[r][1] = __ffma2_rn(y2, z23, S[r][1]);
                }
                if (!STATE) {
                    float xv[8];
                    *reinterpret_cast<float4 *>(xv) = *reinterpret_cast<const float4 *>(&s_x[buf][STATE ? 0 : w][8 * p]);
                    *reinterpret_cast<float4 *>(xv + 4) = *reinterpret_cast<const float4 *>(&s_x[buf][STATE ? 0 : w][8 * p + 4]);
                    float2 o01 = make_float2(0.f, 0.f), o23 = o01;
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float2 x2 = make_float2(xv[r], xv[r]);
                        o01 = __ffma2_rn(x2, S[r][0], o01);
                        o23 = __ffma2_rn(x2, S[r][1], o23);
                    }
                    acc[4 * u] = o01.x; acc[4 * u + 1] = o01.y; acc[4 * u + 2] = o23.x; acc[4 * u + 3] = o23.y;
                }
            }
            if (!STATE) {
                // halve and exchange: lane p ends with the sums of values p*NV .. p*NV+NV-1 (token-major)
                constexpr int NV = 4 * TU / KS;
                int nv = 4 * TU;
#pragma unroll
                for (int off = KS / 2; off >= 1; off >>= 1) {
                    nv >>= 1;
                    const bool up = (p & off) != 0;
#pragma unroll
                    for (int i = 0; i < 4 * TU / 2; ++i) {
                        if (i < nv) {
                            const float send = up ? acc[i] : acc[i + nv], keep = up ? acc[i + nv] : acc[i];
                            acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
                        }
                    }
                }
                if (live) {
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int u = u0 + (p * NV + i) / 4, c = (p * NV + i) % 4, t = token(b, u);
                        if (t < end) {
                            const size_t at = (((size_t)row0 + t) * a.H + h) * DZ + j + c;
                            const float o = acc[i] * s_out[buf][u];
                            if (a.out_f32) ((float *)a.out)[at] = o;
                            else st_out((TIn *)a.out + at, o);
                        }
                    }
                }
            }
        }
        if (!wide) {
            const float2 d = make_float2(s_end[buf], s_end[buf]);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                S[r][0] = __fmul2_rn(S[r][0], d);
                S[r][1] = __fmul2_rn(S[r][1], d);
            }
        }
        if (!rev) {
            snap(min(token(b, TB - 1), end - 1));
        } else if (!STATE && a.snap && b + 1 < nblk) {
            // entering the token before this block, with this block's first token's decay
            const int t = token(b, TB - 1);   // the block's first token
            if (t % a.snap_tokens == 0) {
                const float g = a.g[((size_t)row0 + t) * a.g_ld + h];
                const float by = g != g ? g : fix_exp2(fix_log2(fminf(fmaxf(g, -1e4f), 1e4f)));
                write_state(a.snap + ((size_t)(n + row0 / a.snap_tokens + (t - 1) / a.snap_tokens) * a.H + h) * DX * DZ, by);
            }
        }
    }
    // backward in time, the state that leaves the segment has its first token's decay, too
    float by = 1.f;
    if (rev && nblk > 0) {
        const float g = a.g[((size_t)row0 + beg) * a.g_ld + h];
        by = g != g ? g : fix_exp2(fix_log2(fminf(fmaxf(g, -1e4f), 1e4f)));
    }
    if (STATE) {
        write_state(a.seg_state + woff, by);
        if (cblk == 0 && tid < 32) {
            if (rev && tid == 0) {   // the steps had the decays of the tokens behind theirs: this one is still to come
                const float g = a.g[((size_t)row0 + beg) * a.g_ld + h];
                sum += fix_log2(fminf(fmaxf(g, -1e4f), 1e4f));
                any_nan = any_nan || g != g;
            }
#pragma unroll
            for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            any_nan = __any_sync(0xffffffffu, any_nan);
            if (tid == 0) a.seg_total[(size_t)work.slot * a.H + h] = any_nan ? NAN : fix_exp2(sum);
        }
    } else if (a.s_out && closing) {
        write_state(a.s_out + soff, by);
    }
}

template <int DX, int DZ, typename TIn> cudaError_t launch_type(const LinRuns &p, int passes, cudaStream_t st)
{
    using SH = LinScanShape<DX, DZ>;
    const LinRun &r = p.a[0];
    const long long ctas = (long long)(r.seg_chunks ? r.slots : r.num_seqs) * r.H * SH::CTAS;
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)ctas, passes);
    if (r.seg_chunks) {
        lin_scan_kernel<DX, DZ, TIn, true><<<grid, SH::NTH, 0, st>>>(p);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess || (e = launch_lin_segments(p, passes, DX, DZ, st)) != cudaSuccess) return e;
    }
    lin_scan_kernel<DX, DZ, TIn, false><<<grid, SH::NTH, 0, st>>>(p);
    return cudaGetLastError();
}
template <int DX, int DZ>
cudaError_t launch_dims(const LinRuns &p, int passes, bool bf16, cudaStream_t st)
{
    return bf16 ? launch_type<DX, DZ, __nv_bfloat16>(p, passes, st) : launch_type<DX, DZ, float>(p, passes, st);
}
template <int DX>
cudaError_t launch_dz(const LinRuns &p, int passes, int dz, bool bf16, cudaStream_t st)
{
    switch (dz) {
    case 16: return launch_dims<DX, 16>(p, passes, bf16, st);
    case 32: return launch_dims<DX, 32>(p, passes, bf16, st);
    case 64: return launch_dims<DX, 64>(p, passes, bf16, st);
    case 128: return launch_dims<DX, 128>(p, passes, bf16, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

int lin_scan_segment_chunks(int num_seqs, int H, int passes, int dx, int dz, long long rows)
{
    // An SM holds 8 CTAs of 128 threads and needs about 4 to hide their latencies.  Cut, a token costs 5/3, and a
    // segment's two walks a start of 2 us each (10 tokens): not shorter than 16 tokens.
    const double ctas = (double)num_seqs * H * passes * std::max(1, dx * dz / 4096);
    const double chunks = (double)(rows + SCAN_CHUNK - 1) / SCAN_CHUNK / num_seqs;
    const double wanted = std::min(chunks, 4 * 148 / ctas);
    return wanted < 3 ? 0 : (int)std::max(1.0, std::ceil(chunks / wanted));
}

cudaError_t launch_lin_scan(const LinRuns &r, int passes, int dx, int dz, bool bf16, cudaStream_t st)
{
    switch (dx) {
    case 16: return launch_dz<16>(r, passes, dz, bf16, st);
    case 32: return launch_dz<32>(r, passes, dz, bf16, st);
    case 64: return launch_dz<64>(r, passes, dz, bf16, st);
    case 128: return launch_dz<128>(r, passes, dz, bf16, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace kda
