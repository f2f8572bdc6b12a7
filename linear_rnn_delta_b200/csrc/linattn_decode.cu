// Single-token step of linear attention with one decay per head: the fp32 state is read, updated and
// written back once, in place,
//   S = e^g S + k v^T,   o = S^T q,
// which needs no value of S before the update, so every element is multiplied, added to, written and
// used for the readout as soon as it arrives.  Bound by HBM: 8 d_k d_v bytes for each (sequence, head).
//
// One CTA serves CB value columns of one (sequence, head); a thread owns 4 adjacent columns (16 bytes)
// of every RP-th row, so that a warp's accesses are whole 128-byte lines.  All of a thread's loads are
// issued before the first is used.  With few (sequence, head) pairs the columns are split over more
// CTAs (CB = 32): the step is then as long as one CTA's latency, and a quarter of the state is read in
// less time than all of it.
#include "common.cuh"
#include "linattn.cuh"

namespace kda {
namespace {

template <int DK, int CB> struct LinDecodeShape {
    static constexpr int THREADS = DK * CB / 4 >= 256 ? 256 : DK * CB / 4;
    static constexpr int CT = CB / 4;           // threads of a row
    static constexpr int RP = THREADS / CT;     // rows of a pass
    static constexpr int RPT = DK / RP;         // rows of a thread
    static_assert(RPT * RP == DK && THREADS % 32 == 0, "rows divide evenly into whole warps");
};

template <int DK, int DV, int CB, typename TIn>
__global__ void __launch_bounds__(LinDecodeShape<DK, CB>::THREADS) lin_decode_kernel(const LinDecode a)
{
    using SH = LinDecodeShape<DK, CB>;
    constexpr int CT = SH::CT, RP = SH::RP, RPT = SH::RPT, NW = SH::THREADS / 32, CTAS = DV / CB;
    __shared__ float s_q[DK], s_k[DK];
    __shared__ __align__(16) float s_red[NW][CB];
    const int pair = blockIdx.x / CTAS, col0 = blockIdx.x % CTAS * CB;
    const int n = pair / a.H, h = pair % a.H, hk = h / (a.H / a.Hk);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c4 = tid % CT, rg = tid / CT;
    float4 *S4 = reinterpret_cast<float4 *>(a.state + (size_t)pair * DK * DV + col0) + c4;

    float4 s[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) s[r] = __ldcs(S4 + (size_t)(rg + r * RP) * (DV / 4));

    const TIn *q = (const TIn *)a.q + ((size_t)n * a.Hk + hk) * DK, *k = (const TIn *)a.k + ((size_t)n * a.Hk + hk) * DK;
    for (int i = tid; i < DK; i += SH::THREADS) {
        s_q[i] = ld_f32(q + i);
        s_k[i] = ld_f32(k + i);
    }
    const TIn *v = (const TIn *)a.v + (size_t)pair * DV + col0 + 4 * c4;
    const float v0 = ld_f32(v), v1 = ld_f32(v + 1), v2 = ld_f32(v + 2), v3 = ld_f32(v + 3);
    const float al = expf(a.g[(size_t)n * a.g_ld + h]);
    __syncthreads();

    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const int i = rg + r * RP;
        const float ki = s_k[i], qi = s_q[i];
        float4 x = s[r];
        x.x = fmaf(ki, v0, x.x * al); x.y = fmaf(ki, v1, x.y * al);
        x.z = fmaf(ki, v2, x.z * al); x.w = fmaf(ki, v3, x.w * al);
        __stcs(S4 + (size_t)i * (DV / 4), x);
        o.x = fmaf(qi, x.x, o.x); o.y = fmaf(qi, x.y, o.y);
        o.z = fmaf(qi, x.z, o.z); o.w = fmaf(qi, x.w, o.w);
    }
#pragma unroll
    for (int off = 16; off >= CT; off >>= 1) {   // the warp's rows
        o.x += __shfl_xor_sync(0xffffffffu, o.x, off);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, off);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, off);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, off);
    }
    if (lane < CT) *reinterpret_cast<float4 *>(&s_red[warp][4 * c4]) = o;
    __syncthreads();
    if (tid < CB) {
        float acc = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) acc += s_red[w][tid];
        st_out((TIn *)a.o + (size_t)pair * DV + col0 + tid, acc);
    }
}

template <int DK, int DV, int CB>
cudaError_t launch_cols(const LinDecode &a, bool bf16, cudaStream_t st)
{
    const long long ctas = (long long)a.N * a.H * (DV / CB);
    if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    constexpr int NTH = LinDecodeShape<DK, CB>::THREADS;
    if (bf16) lin_decode_kernel<DK, DV, CB, __nv_bfloat16><<<(unsigned)ctas, NTH, 0, st>>>(a);
    else lin_decode_kernel<DK, DV, CB, float><<<(unsigned)ctas, NTH, 0, st>>>(a);
    return cudaGetLastError();
}
template <int DK, int DV>
cudaError_t launch_dims(const LinDecode &a, bool bf16, cudaStream_t st)
{
    if constexpr (DV > 32) {
        if ((long long)a.N * a.H <= 148) return launch_cols<DK, DV, 32>(a, bf16, st);
    }
    return launch_cols<DK, DV, DV>(a, bf16, st);
}
template <int DK>
cudaError_t launch_dv(const LinDecode &a, bool bf16, cudaStream_t st)
{
    switch (a.dv) {
    case 16: return launch_dims<DK, 16>(a, bf16, st);
    case 32: return launch_dims<DK, 32>(a, bf16, st);
    case 64: return launch_dims<DK, 64>(a, bf16, st);
    case 128: return launch_dims<DK, 128>(a, bf16, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_lin_decode(const LinDecode &a, bool bf16, cudaStream_t st)
{
    switch (a.dk) {
    case 16: return launch_dv<16>(a, bf16, st);
    case 32: return launch_dv<32>(a, bf16, st);
    case 64: return launch_dv<64>(a, bf16, st);
    case 128: return launch_dv<128>(a, bf16, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace kda
