// Token-by-token fp32 scan of linear attention with one decay per head.
//
// Serves fp32 inputs and the head sizes that the tensor-core chunked kernel does not take; it is also
// the exact-order path.  Columns of the state evolve independently, so a CTA owns a block of value
// columns of one (sequence, head) and the whole token axis.  KS = d_x / 8 adjacent lanes form a group
// that owns 4 columns: lane p of it keeps rows 8p .. 8p+7 of them in registers.  A token costs
//   S = a S + k v^T        (packed fp32 multiply and multiply-add)
//   partial o_j = sum over the lane's 8 rows of q_i S_ij
// and the sum over a group's lanes is taken for 4 tokens at once: 16 partial sums (4 tokens x 4
// columns) are halved and exchanged log2(KS) times, so that a group spends 16 - 16/KS shuffles where
// a butterfly for each value would take 16 log2(KS).
//
// Tokens are staged TB at a time in shared memory as fp32, double buffered: block b+1 is loaded into
// registers while block b is computed.  Positions p = 0 .. len-1 run forward (t = p) or backward in
// time (t = len-1-p); backward, the decay of position p is that of token t+1 (1 at p = 0), so that
// the state entering a token is a_{t+1} G_{t+1}.  Steps behind the last one are staged as k = q = 0
// and decay 1: they leave the state as it is.
#include "common.cuh"
#include "linattn.cuh"

namespace kda {
namespace {

constexpr int TB = 8;    // tokens of a staged block
constexpr int TU = 4;    // tokens whose sums are exchanged together

template <int DX, int DZ> struct LinScanShape {
    static constexpr int KS = DX / 8;                             // lanes of a group
    static constexpr int MAXG = 128 / KS;                         // groups of a CTA of 128 threads
    static constexpr int CB = DZ / 4 <= MAXG ? DZ : MAXG * 4;     // columns of a CTA
    static constexpr int LIVE = CB / 4 * KS;                      // lanes with work
    static constexpr int NTH = LIVE < 32 ? 32 : LIVE;
    static constexpr int CTAS = DZ / CB;
    static_assert(NTH % 32 == 0 && (LIVE % 32 == 0 || LIVE < 32), "whole warps");
};

// 4 consecutive elements as fp32
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p)
{
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

template <int DX, int DZ, typename TIn>
__global__ void __launch_bounds__(LinScanShape<DX, DZ>::NTH) lin_scan_kernel(const LinRun a)
{
    using SH = LinScanShape<DX, DZ>;
    constexpr int KS = SH::KS, CB = SH::CB, LIVE = SH::LIVE, NTH = SH::NTH, CTAS = SH::CTAS;
    __shared__ __align__(16) float s_x[2][TB][DX], s_y[2][TB][DX], s_z[2][TB][CB];
    __shared__ float s_a[2][TB];

    const int pair = blockIdx.x / CTAS, cblk = blockIdx.x % CTAS;
    const int n = pair / a.H, h = pair % a.H;
    const int tid = threadIdx.x;
    const bool live = tid < LIVE;
    const int p = tid % KS, grp = live ? tid / KS : 0;
    const int j = cblk * CB + grp * 4;                 // first of the group's columns
    const int row0 = lin_row0(a, n), len = lin_len(a, n);
    const int hx = a.H / a.gx, hy = a.H / a.gy, hz = a.H / a.gz;
    const TIn *x = (const TIn *)a.x + (size_t)(h / a.gx) * DX, *y = (const TIn *)a.y + (size_t)(h / a.gy) * DX;
    const TIn *z = (const TIn *)a.z + (size_t)(h / a.gz) * DZ + cblk * CB;
    const size_t soff = (size_t)pair * DX * DZ;

    float2 S[8][2];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const int i = 8 * p + r;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (a.s_in && live) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                v[c] = a.in_t ? a.s_in[soff + (size_t)(j + c) * DX + i] : a.s_in[soff + (size_t)i * DZ + j + c];
        }
        S[r][0] = make_float2(v[0], v[1]);
        S[r][1] = make_float2(v[2], v[3]);
    }

    constexpr int UX = TB * DX / 4, UZ = TB * CB / 4;   // groups of 4 elements of a block
    constexpr int EX = (UX + NTH - 1) / NTH, EZ = (UZ + NTH - 1) / NTH;
    float4 px[EX], py[EX], pz[EZ];
    float pa = 0.f;
    auto token = [&](int pos) { return a.reverse ? len - 1 - pos : pos; };
    auto fetch = [&](int base) {
        const int nt = min(TB, len - base);
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < EX; ++u) {
            const int e = tid + u * NTH, tt = e / (DX / 4), i = e % (DX / 4) * 4;
            px[u] = py[u] = zero;
            if (tt < nt) {
                const size_t row = (size_t)row0 + token(base + tt);
                px[u] = load4(x + row * hx * DX + i);
                py[u] = load4(y + row * hy * DX + i);
            }
        }
#pragma unroll
        for (int u = 0; u < EZ; ++u) {
            const int e = tid + u * NTH, tt = e / (CB / 4), i = e % (CB / 4) * 4;
            pz[u] = zero;
            if (tt < nt) pz[u] = load4(z + ((size_t)row0 + token(base + tt)) * hz * DZ + i);
        }
        if (tid < TB) {
            pa = 1.f;
            const int t = token(base + tid) + (a.reverse ? 1 : 0);   // whose decay the step has
            if (tid < nt && t < len) pa = expf(a.g[(size_t)((size_t)row0 + t) * a.g_ld + h]);
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int u = 0; u < EX; ++u) {
            const int e = tid + u * NTH, tt = e / (DX / 4), i = e % (DX / 4) * 4;
            if (tt < TB) {
                *reinterpret_cast<float4 *>(&s_x[buf][tt][i]) = px[u];
                *reinterpret_cast<float4 *>(&s_y[buf][tt][i]) = py[u];
            }
        }
#pragma unroll
        for (int u = 0; u < EZ; ++u) {
            const int e = tid + u * NTH, tt = e / (CB / 4), i = e % (CB / 4) * 4;
            if (tt < TB) *reinterpret_cast<float4 *>(&s_z[buf][tt][i]) = pz[u];
        }
        if (tid < TB) s_a[buf][tid] = pa;
    };
    auto write_state = [&](float *dst, bool t, float by) {   // [DX][DZ], or transposed
        if (!live) return;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int i = 8 * p + r;
            const float v[4] = {S[r][0].x * by, S[r][0].y * by, S[r][1].x * by, S[r][1].y * by};
            if (t) {
#pragma unroll
                for (int c = 0; c < 4; ++c) dst[(size_t)(j + c) * DX + i] = v[c];
            } else {
                *reinterpret_cast<float4 *>(dst + (size_t)i * DZ + j) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
    };
    auto snap_at = [&](int t) {   // boundary state of the segment that token t belongs to
        float *dst = a.snap + ((size_t)(n + row0 / a.snap_tokens + t / a.snap_tokens) * a.H + h) * DX * DZ;
        write_state(dst, false, 1.f);
    };

    fetch(0);
    for (int base = 0, buf = 0; base < len; base += TB, buf ^= 1) {
        stage(buf);
        __syncthreads();   // this block is staged, and nobody reads the buffer of the one before the last
        if (base + TB < len) fetch(base + TB);
#pragma unroll
        for (int t0 = 0; t0 < TB; t0 += TU) {
            if (base + t0 >= len) break;
            float acc[4 * TU];
#pragma unroll
            for (int u = 0; u < TU; ++u) {
                const int tt = t0 + u, pos = base + tt;
                const float2 a2 = make_float2(s_a[buf][tt], s_a[buf][tt]);
                const float4 z4 = *reinterpret_cast<const float4 *>(&s_z[buf][tt][grp * 4]);
                const float2 z01 = make_float2(z4.x, z4.y), z23 = make_float2(z4.z, z4.w);
                float yv[8], xv[8];
                *reinterpret_cast<float4 *>(yv) = *reinterpret_cast<const float4 *>(&s_y[buf][tt][8 * p]);
                *reinterpret_cast<float4 *>(yv + 4) = *reinterpret_cast<const float4 *>(&s_y[buf][tt][8 * p + 4]);
                *reinterpret_cast<float4 *>(xv) = *reinterpret_cast<const float4 *>(&s_x[buf][tt][8 * p]);
                *reinterpret_cast<float4 *>(xv + 4) = *reinterpret_cast<const float4 *>(&s_x[buf][tt][8 * p + 4]);
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    S[r][0] = __fmul2_rn(S[r][0], a2);
                    S[r][1] = __fmul2_rn(S[r][1], a2);
                }
                if (a.reverse && a.snap && pos < len) {
                    const int t = len - 1 - pos;
                    if (t == len - 1 || (t + 1) % a.snap_tokens == 0) snap_at(t);
                }
                float2 o01 = make_float2(0.f, 0.f), o23 = o01;
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const float2 y2 = make_float2(yv[r], yv[r]), x2 = make_float2(xv[r], xv[r]);
                    S[r][0] = __ffma2_rn(y2, z01, S[r][0]);
                    S[r][1] = __ffma2_rn(y2, z23, S[r][1]);
                    o01 = __ffma2_rn(x2, S[r][0], o01);
                    o23 = __ffma2_rn(x2, S[r][1], o23);
                }
                acc[4 * u] = o01.x; acc[4 * u + 1] = o01.y; acc[4 * u + 2] = o23.x; acc[4 * u + 3] = o23.y;
                if (!a.reverse && a.snap && pos < len && (pos == len - 1 || (pos + 1) % a.snap_tokens == 0))
                    snap_at(pos);
            }
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
                    const int u = (p * NV + i) / 4, c = (p * NV + i) % 4, pos = base + t0 + u;
                    if (pos < len) {
                        const size_t at = (((size_t)row0 + token(pos)) * a.H + h) * DZ + j + c;
                        if (a.out_f32) ((float *)a.out)[at] = acc[i];
                        else st_out((TIn *)a.out + at, acc[i]);
                    }
                }
            }
        }
    }
    if (a.s_out) {
        // backward in time, the state at the sequence's start has the first token's decay too
        const float by = (a.reverse && len > 0) ? expf(a.g[(size_t)row0 * a.g_ld + h]) : 1.f;
        write_state(a.s_out + soff, a.out_t != 0, by);
    }
}

template <int DX, int DZ>
cudaError_t launch_dims(const LinRun &r, bool bf16, cudaStream_t st)
{
    using SH = LinScanShape<DX, DZ>;
    const long long ctas = (long long)r.num_seqs * r.H * SH::CTAS;
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    if (bf16) lin_scan_kernel<DX, DZ, __nv_bfloat16><<<(unsigned)ctas, SH::NTH, 0, st>>>(r);
    else lin_scan_kernel<DX, DZ, float><<<(unsigned)ctas, SH::NTH, 0, st>>>(r);
    return cudaGetLastError();
}
template <int DX>
cudaError_t launch_dz(const LinRun &r, int dz, bool bf16, cudaStream_t st)
{
    switch (dz) {
    case 16: return launch_dims<DX, 16>(r, bf16, st);
    case 32: return launch_dims<DX, 32>(r, bf16, st);
    case 64: return launch_dims<DX, 64>(r, bf16, st);
    case 128: return launch_dims<DX, 128>(r, bf16, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_lin_scan(const LinRun &r, int dx, int dz, bool bf16, cudaStream_t st)
{
    switch (dx) {
    case 16: return launch_dz<16>(r, dz, bf16, st);
    case 32: return launch_dz<32>(r, dz, bf16, st);
    case 64: return launch_dz<64>(r, dz, bf16, st);
    case 128: return launch_dz<128>(r, dz, bf16, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace kda
