// Closing kernels of linear attention's backward pass: gradients of shared heads, and the gradient of the
// log-decays.
//
// With c_t the running sum of g, g enters the output through e^{c_r - c_s} (q_r . k_s), s <= r, so dL/dg_t is
// the sum over all pairs s < t <= r of their share of L.  The short form of that sum,
//   sum_{r >= t} (q_r . dq_r - k_r . dk_r) + <S_T, dL/dS_T>,
// takes small differences of large sums: with a decay of e^{-1} a token it left 2e-5 of dg (and 4e-4 of a decay's
// own, which is a sum over tokens) where fp32 should leave 1e-7.  So the pairs are summed as they are: those
// within a chunk one by one, the others through the states at the chunk's two ends.

#include "linattn_sm100.cuh"

namespace kda {
namespace {

using lin::load4;

// Sums the value heads' gradients of a shared key head, in head order; 4 channels a thread, 8 heads' loads in flight.
// Bound by HBM: 8191 tokens of 16 heads over 2, 128 channels, 134 MB in 25 us (5.3 TB/s; one head after the other: 29 us).
template <typename TOut>
__global__ void __launch_bounds__(256) lin_share_kernel(const float *dqf, const float *dkf, TOut *dq, TOut *dk,
                                                        long long rows, int Hk, int H, int d)
{
    const int group = H / Hk, quads = d / 4;
    const long long items = rows * Hk * quads;
    for (long long it = blockIdx.x * 256ll + threadIdx.x; it < items; it += gridDim.x * 256ll) {
        const long long rk = it / quads;             // (row, key head)
        const int c = (int)(it % quads) * 4;
        const size_t from = ((size_t)(rk / Hk) * H + (size_t)(rk % Hk) * group) * d + c;
        float4 q = make_float4(0.f, 0.f, 0.f, 0.f), k = q;
#pragma unroll 8
        for (int m = 0; m < group; ++m) {
            const float4 u = __ldcs(reinterpret_cast<const float4 *>(dqf + from + (size_t)m * d));
            const float4 w = __ldcs(reinterpret_cast<const float4 *>(dkf + from + (size_t)m * d));
            q.x += u.x; q.y += u.y; q.z += u.z; q.w += u.w;
            k.x += w.x; k.y += w.y; k.z += w.z; k.w += w.w;
        }
        const size_t to = (size_t)rk * d + c;
        st_out(dq + to, q.x); st_out(dq + to + 1, q.y); st_out(dq + to + 2, q.z); st_out(dq + to + 3, q.w);
        st_out(dk + to, k.x); st_out(dk + to + 1, k.y); st_out(dk + to + 2, k.z); st_out(dk + to + 3, k.w);
    }
}

// dg of one chunk (64 tokens) and head, every pair of tokens on its own:
//   dg_t = sum_{s < t <= r} W_rs                          both in the chunk, W_rs = L_rs (q_r . k_s) (do_r . v_s)
//        + sum_{r >= t} w_r q_r^T S_0 do_r                s before the chunk
//        + sum_{s < t} u_s k_s^T G_C v_s                  r behind it
//        + e^{c_C} <S_0, G_C>                             s before, r behind
// S_0 the state before the chunk, G_C what enters its last token from behind.  The state products are
// taken 16 rows of S^T and G^T (value channels) at a time.  Bound by fp32 arithmetic: 2 d_k d_v + 64 (d_k + d_v)
// multiply-adds a token, beside 6 d_k d_v / 2 packed ones of the three passes.
constexpr int GT = 256;
constexpr int GC = 64;
constexpr int GROWS = 16;

template <int DK, int DV, typename TIn>
__global__ void __launch_bounds__(GT) lin_gate_chunk_kernel(const LinGateGrad a)
{
    constexpr int PK = DK + 4, PV = DV + 4;   // padded rows: 16-byte steps over all banks
    extern __shared__ __align__(16) float sm[];
    float *s_q = sm, *s_k = s_q + GC * PK, *s_do = s_k + GC * PK, *s_v = s_do + GC * PV;
    float *s_s = s_v + GC * PV, *s_g = s_s + GROWS * PK;            // rows of S^T and G^T
    float *s_w = s_g + GROWS * PK;                                  // [64][65]
    __shared__ float2 s_c[GC];
    __shared__ float s_win[GC], s_uout[GC], s_dq[GC], s_dk[GC], s_x[GT / 32], s_tot, s_pre[GT / 32][GC];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H;
    // sequence of the slot: the last one whose first slot is not behind it (first slots increase)
    int n = 0;
    {
        int lo = 0, hi = a.num_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (mid + (a.cu_seqlens ? a.cu_seqlens[mid] : mid * a.T) / GC <= slot) lo = mid;
            else hi = mid - 1;
        }
        n = lo;
    }
    const int row0 = a.cu_seqlens ? a.cu_seqlens[n] : n * a.T;
    const int len = a.cu_seqlens ? a.cu_seqlens[n + 1] - row0 : a.T;
    const int t0 = (slot - n - row0 / GC) * GC;
    if (t0 < 0 || t0 >= len) {   // no chunk has this slot
        if (a.partial && tid == 0) a.partial[(size_t)slot * a.H + h] = 0.f;
        return;
    }
    const int nt = min(GC, len - t0), hk = h / (a.H / a.Hk);
    const size_t row = (size_t)row0 + t0;

    // tiles, zero behind the sequence's end
    const TIn *q = (const TIn *)a.q + (row * a.Hk + hk) * DK, *k = (const TIn *)a.k + (row * a.Hk + hk) * DK;
    const TIn *v = (const TIn *)a.v + (row * a.H + h) * DV, *d = (const TIn *)a.d_o + (row * a.H + h) * DV;
#pragma unroll
    for (int e = tid; e < GC * DK / 4; e += GT) {
        const int r = e / (DK / 4), i = e % (DK / 4) * 4;
        const bool in = r < nt;
        *reinterpret_cast<float4 *>(s_q + r * PK + i) = in ? load4(q + (size_t)r * a.Hk * DK + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(s_k + r * PK + i) = in ? load4(k + (size_t)r * a.Hk * DK + i) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int e = tid; e < GC * DV / 4; e += GT) {
        const int r = e / (DV / 4), j = e % (DV / 4) * 4;
        const bool in = r < nt;
        *reinterpret_cast<float4 *>(s_do + r * PV + j) = in ? load4(d + (size_t)r * a.H * DV + j) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(s_v + r * PV + j) = in ? load4(v + (size_t)r * a.H * DV + j) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (warp == 0) {   // sums of log2-decays
        const float g0 = 2 * lane < nt ? a.g[(row + 2 * lane) * a.g_ld + h] : 0.f;
        const float g1 = 2 * lane + 1 < nt ? a.g[(row + 2 * lane + 1) * a.g_ld + h] : 0.f;
        const bool nan = __any_sync(0xffffffffu, g0 != g0 || g1 != g1);
        const long long f1 = lin::fix_log2(fminf(fmaxf(g1, -1e4f), 1e4f));
        long long run = lin::fix_log2(fminf(fmaxf(g0, -1e4f), 1e4f)) + f1;
        for (int off = 1; off < 32; off <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, run, off);
            if (lane >= off) run += o;
        }
        const long long end = __shfl_sync(0xffffffffu, run, 31);
        for (int e = 0; e < 2; ++e) {
            const long long c = e ? run : run - f1;
            const int t = 2 * lane + e;
            s_c[t] = make_float2(nan ? NAN : (float)lin::fix_int(c), lin::fix_rest(c));
            s_win[t] = nan ? NAN : lin::fix_exp2(c);
            s_uout[t] = nan ? NAN : lin::fix_exp2(end - c);
        }
        if (lane == 0) s_tot = nan ? NAN : lin::fix_exp2(end);
    }
    __syncthreads();

    // W, 4 x 4 of it a thread (rows ty + 16 x, columns tx + 16 y)
    {
        const int tx = tid & 15, ty = tid >> 4;
        float qk[4][4] = {}, dv[4][4] = {};
        for (int i = 0; i < DK; i += 4) {
            float4 x[4], y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = *reinterpret_cast<const float4 *>(s_q + (ty + 16 * e) * PK + i);
                y[e] = *reinterpret_cast<const float4 *>(s_k + (tx + 16 * e) * PK + i);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    qk[e][f] = fmaf(x[e].x, y[f].x, fmaf(x[e].y, y[f].y, fmaf(x[e].z, y[f].z, fmaf(x[e].w, y[f].w, qk[e][f]))));
        }
        for (int j = 0; j < DV; j += 4) {
            float4 x[4], y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = *reinterpret_cast<const float4 *>(s_do + (ty + 16 * e) * PV + j);
                y[e] = *reinterpret_cast<const float4 *>(s_v + (tx + 16 * e) * PV + j);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    dv[e][f] = fmaf(x[e].x, y[f].x, fmaf(x[e].y, y[f].y, fmaf(x[e].z, y[f].z, fmaf(x[e].w, y[f].w, dv[e][f]))));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int r = ty + 16 * e, s = tx + 16 * f;
                const float2 cr = s_c[r], cs = s_c[s];
                s_w[r * 65 + s] = s < r ? qk[e][f] * dv[e][f] * exp2f((cr.x - cs.x) + (cr.y - cs.y)) : 0.f;
            }
    }

    // state products.  Thread: token r = tid / 4, rows (tid % 4) + 4 x of the 16; state layout [dv][dk]
    const bool first = t0 == 0, last = t0 + nt >= len;
    const size_t size = (size_t)DK * DV;
    const float *S0 = first ? (a.s_init ? a.s_init + ((size_t)n * a.H + h) * size : nullptr)
                            : a.snap_s + ((size_t)(slot - 1) * a.H + h) * size;
    const float *GC_ = last ? (a.g_end ? a.g_end + ((size_t)n * a.H + h) * size : nullptr)
                            : a.snap_g + ((size_t)slot * a.H + h) * size;
    const int r = tid >> 2, sub = tid & 3;
    float accq = 0.f, acck = 0.f, accx = 0.f;
    for (int j0 = 0; j0 < DV && (S0 || GC_); j0 += GROWS) {
        __syncthreads();
        for (int e = tid; e < GROWS * DK; e += GT) {
            const int j = e / DK, i = e % DK;   // the caller's states are [dk][dv], the passes' boundary states [dv][dk]
            const float x = !S0 ? 0.f : first ? S0[(size_t)i * DV + j0 + j] : S0[(size_t)(j0 + j) * DK + i];
            const float y = !GC_ ? 0.f : last ? GC_[(size_t)i * DV + j0 + j] : GC_[(size_t)(j0 + j) * DK + i];
            s_s[j * PK + i] = x;
            s_g[j * PK + i] = y;
            accx = fmaf(x, y, accx);
        }
        __syncthreads();
        float yq[GROWS / 4] = {}, yk[GROWS / 4] = {};
        for (int i = 0; i < DK; i += 4) {
            const float4 xq = *reinterpret_cast<const float4 *>(s_q + r * PK + i);
            const float4 xk = *reinterpret_cast<const float4 *>(s_k + r * PK + i);
#pragma unroll
            for (int e = 0; e < GROWS / 4; ++e) {
                const float4 u = *reinterpret_cast<const float4 *>(s_s + (sub + 4 * e) * PK + i);
                const float4 w = *reinterpret_cast<const float4 *>(s_g + (sub + 4 * e) * PK + i);
                yq[e] = fmaf(u.x, xq.x, fmaf(u.y, xq.y, fmaf(u.z, xq.z, fmaf(u.w, xq.w, yq[e]))));
                yk[e] = fmaf(w.x, xk.x, fmaf(w.y, xk.y, fmaf(w.z, xk.z, fmaf(w.w, xk.w, yk[e]))));
            }
        }
#pragma unroll
        for (int e = 0; e < GROWS / 4; ++e) {
            accq = fmaf(yq[e], s_do[r * PV + j0 + sub + 4 * e], accq);
            acck = fmaf(yk[e], s_v[r * PV + j0 + sub + 4 * e], acck);
        }
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
        accq += __shfl_xor_sync(0xffffffffu, accq, off);
        acck += __shfl_xor_sync(0xffffffffu, acck, off);
    }
    if (sub == 0) {
        s_dq[r] = r < nt && S0 ? s_win[r] * accq : 0.f;
        s_dk[r] = r < nt && GC_ ? s_uout[r] * acck : 0.f;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) accx += __shfl_xor_sync(0xffffffffu, accx, off);
    if (lane == 0) s_x[warp] = accx;
    __syncthreads();

    {   // p_r(t) = sum_{s < t} W_rs, summed over the warp's 8 rows r >= t; a lane has t = 2 lane, 2 lane + 1
        float y0 = 0.f, y1 = 0.f;
#pragma unroll
        for (int e = 0; e < GC * 32 / GT; ++e) {
            const int r2 = warp * (GC * 32 / GT) + e;
            const float w0 = s_w[r2 * 65 + 2 * lane], w1 = s_w[r2 * 65 + 2 * lane + 1];
            float run = w0 + w1;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float o = __shfl_up_sync(0xffffffffu, run, off);
                if (lane >= off) run += o;
            }
            float before = __shfl_up_sync(0xffffffffu, run, 1);
            if (lane == 0) before = 0.f;
            if (r2 >= 2 * lane && r2 < nt) y0 += before;
            if (r2 >= 2 * lane + 1 && r2 < nt) y1 += before + w0;
        }
        s_pre[warp][2 * lane] = y0;
        s_pre[warp][2 * lane + 1] = y1;
    }
    __syncthreads();
    if (warp == 0) {   // t = 2 lane, 2 lane + 1
        const int t = 2 * lane;
        float x[2] = {0.f, 0.f};
#pragma unroll
        for (int w = 0; w < GT / 32; ++w) {
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
        if (S0 && GC_) {
            for (int w = 0; w < GT / 32; ++w) cross += s_x[w];
            cross *= s_tot;
        }
        x[0] = (x[0] + (q0 + q1 + sq)) + (sk + cross);
        x[1] = (x[1] + (q1 + sq)) + (sk + k0 + cross);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (t + e >= nt) continue;
            // e^g has slope 0 at -infinity (the states' products may have an infinity's NaN there)
            if (a.g[(row + t + e) * a.g_ld + h] == -INFINITY) x[e] = 0.f;
            if (a.dg) a.dg[(row + t + e) * a.H + h] = x[e];
            sum += x[e];
        }
        if (a.partial) {
#pragma unroll
            for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (lane == 0) a.partial[(size_t)slot * a.H + h] = sum;
        }
    }
}

// dg of a head's own decay: the sum over its chunks (slots of 64 tokens), in slot order and 64 bits
__global__ void __launch_bounds__(128) lin_gate_head_kernel(const float *partial, int slots, int H, float *dg)
{
    __shared__ double s_red[128];
    const int h = blockIdx.x, tid = threadIdx.x;
    double acc = 0.0;
    for (int s = tid; s < slots; s += 128) acc += (double)partial[(size_t)s * H + h];
    s_red[tid] = acc;
    __syncthreads();
    for (int off = 64; off; off >>= 1) {
        if (tid < off) s_red[tid] += s_red[tid + off];
        __syncthreads();
    }
    if (tid == 0) dg[h] = (float)s_red[0];
}

}  // namespace

cudaError_t launch_lin_share(const float *dqf, const float *dkf, void *dq, void *dk, long long rows, int Hk, int H,
                             int d_k, bool bf16, cudaStream_t st)
{
    const long long items = rows * Hk * (d_k / 4);
    if (items == 0) return cudaSuccess;
    const unsigned grid = (unsigned)min((items + 255) / 256, 148ll * 16);
    if (bf16) lin_share_kernel<<<grid, 256, 0, st>>>(dqf, dkf, (__nv_bfloat16 *)dq, (__nv_bfloat16 *)dk, rows, Hk, H, d_k);
    else lin_share_kernel<<<grid, 256, 0, st>>>(dqf, dkf, (float *)dq, (float *)dk, rows, Hk, H, d_k);
    return cudaGetLastError();
}

namespace {

template <int DK, int DV, typename TIn> cudaError_t launch_gate(const LinGateGrad &a, cudaStream_t st)
{
    constexpr uint32_t bytes = (2 * GC * (DK + 4) + 2 * GC * (DV + 4) + 2 * GROWS * (DK + 4) + GC * 65) * 4;
    static bool done[64] = {};
    const cudaError_t e = lin::opt_in(lin_gate_chunk_kernel<DK, DV, TIn>, bytes, done);
    if (e != cudaSuccess) return e;
    lin_gate_chunk_kernel<DK, DV, TIn><<<(unsigned)((long long)a.slots * a.H), GT, bytes, st>>>(a);
    return cudaGetLastError();
}
template <int DK, typename TIn> cudaError_t launch_gate_dv(const LinGateGrad &a, cudaStream_t st)
{
    switch (a.dv) {
    case 16: return launch_gate<DK, 16, TIn>(a, st);
    case 32: return launch_gate<DK, 32, TIn>(a, st);
    case 64: return launch_gate<DK, 64, TIn>(a, st);
    case 128: return launch_gate<DK, 128, TIn>(a, st);
    }
    return cudaErrorInvalidValue;
}
template <typename TIn> cudaError_t launch_gate_dims(const LinGateGrad &a, cudaStream_t st)
{
    switch (a.dk) {
    case 16: return launch_gate_dv<16, TIn>(a, st);
    case 32: return launch_gate_dv<32, TIn>(a, st);
    case 64: return launch_gate_dv<64, TIn>(a, st);
    case 128: return launch_gate_dv<128, TIn>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_lin_gate_grad(const LinGateGrad &a, bool bf16, bool chunk, cudaStream_t st)
{
    if ((long long)a.slots * a.H > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaSuccess;
    if (a.rows > 0) e = chunk ? launch_lin_gate_chunk(a, st) : bf16 ? launch_gate_dims<__nv_bfloat16>(a, st) : launch_gate_dims<float>(a, st);
    if (e == cudaSuccess && a.dg_head) {
        lin_gate_head_kernel<<<a.H, 128, 0, st>>>(a.partial, a.rows > 0 ? a.slots : 0, a.H, a.dg_head);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace kda
