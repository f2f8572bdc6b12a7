// Closing kernels of linear attention's backward pass: gradients of shared heads, the dots q.dq and
// k.dk of every token, and the gradient of the log-decays.
//
// With c_t the running sum of g, g enters the output through e^{c_r - c_s} (q_r . k_s), s <= r, so
//   dL/dg_t = sum over pairs s < t <= r of their share of L
//           = sum_{r >= t} (q_r . dq_r - k_r . dk_r) + <S_T, dL/dS_T>.
// Far from the end that sum is a small difference of large ones: its terms reach back to the end of
// the sequence while dg_t only knows pairs that the decay leaves alive.  Both recurrences leave their
// state at boundaries every LIN_SEG tokens, and there the rest of the sum is an inner product:
//   dg_t = sum_{t <= r <= e} (q_r . dq_r - k_r . dk_r) + <S_e, a_{e+1} G_{e+1}>,
// e the segment's last token.
#include "common.cuh"
#include "linattn.cuh"

namespace kda {
namespace {

// One warp for each (token, key head): sums the value heads' gradients in head order.
template <typename TIn>
__global__ void __launch_bounds__(256) lin_share_kernel(const float *dqf, const float *dkf, const TIn *q, const TIn *k,
                                                        TIn *dq, TIn *dk, float *dot_q, float *dot_k, long long rows,
                                                        int Hk, int H, int d)
{
    const int lane = threadIdx.x & 31, group = H / Hk;
    const long long items = rows * Hk;
    for (long long it = blockIdx.x * 8ll + (threadIdx.x >> 5); it < items; it += gridDim.x * 8ll) {
        const long long row = it / Hk;
        const int hk = (int)(it % Hk);
        float sq[4] = {0.f, 0.f, 0.f, 0.f}, sk[4] = {0.f, 0.f, 0.f, 0.f}, qv[4], kv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = lane + 32 * e;
            qv[e] = i < d ? ld_f32(q + it * d + i) : 0.f;
            kv[e] = i < d ? ld_f32(k + it * d + i) : 0.f;
        }
        for (int m = 0; m < group; ++m) {
            const int h = hk * group + m;
            const float *gq = dqf + (row * H + h) * d, *gk = dkf + (row * H + h) * d;
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = lane + 32 * e;
                if (i < d) {
                    const float u = gq[i], w = gk[i];
                    sq[e] += u;
                    sk[e] += w;
                    a = fmaf(qv[e], u, a);
                    b = fmaf(kv[e], w, b);
                }
            }
#pragma unroll
            for (int off = 16; off; off >>= 1) {
                a += __shfl_xor_sync(0xffffffffu, a, off);
                b += __shfl_xor_sync(0xffffffffu, b, off);
            }
            if (lane == 0) {
                dot_q[(long long)h * rows + row] = a;
                dot_k[(long long)h * rows + row] = b;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = lane + 32 * e;
            if (i < d) {
                st_out(dq + it * d + i, sq[e]);
                st_out(dk + it * d + i, sk[e]);
            }
        }
    }
}

constexpr int GT = 128;              // threads of the gate-gradient kernel
constexpr int GV = LIN_SEG / GT;     // tokens of a thread

// One CTA for each (segment slot, head).
__global__ void __launch_bounds__(GT) lin_gate_grad_kernel(const LinGateGrad a)
{
    __shared__ float s_red[GT / 32];
    const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // sequence of the slot: the last one whose first slot is not behind it (first slots increase)
    int n = 0;
    {
        int lo = 0, hi = a.num_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            const int first = mid + (a.cu_seqlens ? a.cu_seqlens[mid] : mid * a.T) / LIN_SEG;
            if (first <= slot) lo = mid;
            else hi = mid - 1;
        }
        n = lo;
    }
    const int row0 = a.cu_seqlens ? a.cu_seqlens[n] : n * a.T;
    const int len = a.cu_seqlens ? a.cu_seqlens[n + 1] - row0 : a.T;
    const int t0 = (slot - n - row0 / LIN_SEG) * LIN_SEG;
    if (t0 < 0 || t0 >= len) {   // no segment has this slot
        if (a.partial && tid == 0) a.partial[(size_t)slot * a.H + h] = 0.f;
        return;
    }
    const int nt = min(LIN_SEG, len - t0);

    auto block_sum = [&](float v) {   // the same bits in every thread
#pragma unroll
        for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        __syncthreads();
        if (lane == 0) s_red[warp] = v;
        __syncthreads();
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < GT / 32; ++w) t += s_red[w];
        return t;
    };

    // what the pairs beyond the segment's end give
    float after = 0.f;
    if (t0 + nt < len || a.g_end) {
        const size_t at = ((size_t)slot * a.H + h) * a.dk * a.dv;
        const float4 *s = reinterpret_cast<const float4 *>(a.snap_s + at);
        const float4 *g = reinterpret_cast<const float4 *>(a.snap_g + at);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int e = tid; e < a.dk * a.dv / 4; e += GT) {
            const float4 u = __ldcs(s + e), w = __ldcs(g + e);
            acc.x = fmaf(u.x, w.x, acc.x); acc.y = fmaf(u.y, w.y, acc.y);
            acc.z = fmaf(u.z, w.z, acc.z); acc.w = fmaf(u.w, w.w, acc.w);
        }
        after = block_sum((acc.x + acc.y) + (acc.z + acc.w));
    }

    // inclusive sums from the segment's end: thread i has tokens GV*i .. GV*i+GV-1
    const float *dq = a.dot_q + (size_t)h * a.rows + row0 + t0, *dk = a.dot_k + (size_t)h * a.rows + row0 + t0;
    float d[GV], run = 0.f;
#pragma unroll
    for (int v = GV - 1; v >= 0; --v) {
        const int t = GV * tid + v;
        run += t < nt ? dq[t] - dk[t] : 0.f;
        d[v] = run;
    }
    float incl = run;   // of this thread and the lanes behind it
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float o = __shfl_down_sync(0xffffffffu, incl, off);
        if (lane + off < 32) incl += o;
    }
    __syncthreads();
    if (lane == 0) s_red[warp] = incl;
    __syncthreads();
    float behind = after;
#pragma unroll
    for (int w = GT / 32 - 1; w > 0; --w)
        if (w > warp) behind += s_red[w];
    behind += incl - run;
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < GV; ++v) {
        const int t = GV * tid + v;
        if (t < nt) {
            // e^g has slope 0 at -infinity; the difference of sums would leave its rounding there
            const float gt = a.g[((size_t)row0 + t0 + t) * a.g_ld + h];
            const float x = gt == -INFINITY ? 0.f : d[v] + behind;
            sum += x;
            if (a.dg) a.dg[((size_t)row0 + t0 + t) * a.H + h] = x;
        }
    }
    if (a.partial) {
        sum = block_sum(sum);
        if (tid == 0) a.partial[(size_t)slot * a.H + h] = sum;
    }
}

// dg of a head's own decay: the sum over its segments, in slot order and 64 bits
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

cudaError_t launch_lin_share(const float *dqf, const float *dkf, const void *q, const void *k, void *dq, void *dk,
                             float *dot_q, float *dot_k, long long rows, int Hk, int H, int d_k, bool bf16,
                             cudaStream_t st)
{
    const long long items = rows * Hk;
    if (items == 0) return cudaSuccess;
    const unsigned grid = (unsigned)min((items + 7) / 8, 148ll * 32);
    if (bf16)
        lin_share_kernel<<<grid, 256, 0, st>>>(dqf, dkf, (const __nv_bfloat16 *)q, (const __nv_bfloat16 *)k,
                                               (__nv_bfloat16 *)dq, (__nv_bfloat16 *)dk, dot_q, dot_k, rows, Hk, H, d_k);
    else
        lin_share_kernel<<<grid, 256, 0, st>>>(dqf, dkf, (const float *)q, (const float *)k, (float *)dq, (float *)dk,
                                               dot_q, dot_k, rows, Hk, H, d_k);
    return cudaGetLastError();
}

cudaError_t launch_lin_gate_grad(const LinGateGrad &a, cudaStream_t st)
{
    const long long ctas = (long long)a.slots * a.H;
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    lin_gate_grad_kernel<<<(unsigned)ctas, GT, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && a.dg_head) {
        lin_gate_head_kernel<<<a.H, 128, 0, st>>>(a.partial, a.slots, a.H, a.dg_head);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace kda
