// Linear attention with one decay per head: shared definitions of its kernels.
//
//   S_t = a_t S_{t-1} + k_t v_t^T,  a_t = e^{g_t},   o_t = S_t^T q_t
//
// Every gradient of this recurrence is the same recurrence with its arguments permuted:
//   dq_t = S_t do_t                                forward in time,  (q, k, v) := (do, v, k), state S^T
//   dv_t = G_t^T k_t, G_t = a_{t+1} G_{t+1} + q_t do_t^T   backward,  (q, k, v) := (k, q, do), state G
//   dk_t = G_t v_t                                 backward in time, (q, k, v) := (v, do, q), state G^T
// with G_t = dL/dS_t (G after the last token = dL/dS_final, dL/dS_initial = a_1 G_1).  One `LinRun`
// describes one such pass; the kernels know nothing of its role.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

struct LinRun {
    // query-, key- and value-like operands [B*T][heads][d], with the value heads per head of theirs
    const void *x, *y, *z;
    int gx, gy, gz;             // head of x for value head h: h / gx (x has H / gx heads)
    const float *g;             // log-decays [B*T][H] (g_ld = H) or [H] (g_ld = 0)
    int g_ld;
    const float *s_in;          // [N][H] states or NULL (zero)
    float *s_out;               // state after the last step (reverse: decayed by the first token too), or NULL
    int in_t;                   // s_in is [d_z][d_x] (transposed) instead of [d_x][d_z]
    float *snap;                // states at boundaries every `snap_tokens` tokens, [slot][H][d_x][d_z], or NULL
    int snap_tokens;            // (reverse: the state that enters the boundary token, decayed)
    void *out;                  // [B*T][H][d_z]
    int out_f32;                // out is fp32 whatever the inputs' type
    int reverse;                // backward in time
    int num_seqs, T, H;
    const int32_t *cu_seqlens;  // packed batch, or NULL (sequence n is rows n*T .. n*T+T-1)
    long long rows;             // tokens of the whole batch
    // token axis in segments: chunks of one (of 64 tokens, the scan's of 16; 0: not cut) and tokens, slots of all
    // sequences, and the state that enters each slot's segment [slot][H][d_x][d_z] with the decay over it [slot][H]
    int seg_chunks, seg_tokens, slots;
    float *seg_state, *seg_total;
    // segments in turn (tensor-core form): tickets given out [H] and state hand-overs done [slot][H], zero at the
    // launch; NULL: side by side
    int *tickets, *handed;
    int stall;                  // testing aid: (sequence 0, head 0)'s first segment in turn does not hand its state over
};

// Up to three passes of one shape, one cut of the token axis and one output type, side by side.
struct LinRuns {
    LinRun a[3];
};

__device__ __forceinline__ int lin_row0(const LinRun &a, int n) { return a.cu_seqlens ? a.cu_seqlens[n] : n * a.T; }
__device__ __forceinline__ int lin_len(const LinRun &a, int n)
{
    return a.cu_seqlens ? a.cu_seqlens[n + 1] - a.cu_seqlens[n] : a.T;
}

// Arguments of the gate gradient's kernels.
struct LinGateGrad {
    const void *q, *k, *v, *d_o;
    const float *snap_s, *snap_g;   // the dq and dk passes' states at boundaries of 64 tokens [slot][H][dv][dk]
    const float *s_init, *g_end;    // initial state and dL/dS_final, [N][H][dk][dv] or NULL
    const float *g;                 // log-decays as in LinRun
    int g_ld;
    float *dg;                      // [rows][H], or NULL with a decay of each head
    float *partial;                 // [slot][H] sums over a chunk's tokens (decay of each head), or NULL
    float *dg_head;                 // [H]
    long long rows;
    int Hk, H, dk, dv, num_seqs, T, slots;
    const int32_t *cu_seqlens;
    int stall;                      // testing aid (chunk form): slot 0 of head 0 does not load its tiles
};

cudaError_t launch_lin_scan(const LinRuns &r, int passes, int dx, int dz, bool bf16, cudaStream_t st);
constexpr int SCAN_CHUNK = 16;
int lin_scan_segment_chunks(int num_seqs, int H, int passes, int dx, int dz, long long rows);   // of SCAN_CHUNK, as below
// Turns what each segment adds (seg_state, seg_total) into the states that enter them.
cudaError_t launch_lin_segments(const LinRuns &r, int passes, int dx, int dz, cudaStream_t st);
// The tensor-core form's cut: chunks of a segment (0: sequences are left whole), and whether a sequence's segments
// are walked in turn; and the segments' slots (segment j of sequence n is slot n + floor(R_n / tokens) + j, R_n its
// first row).
struct LinCut {
    int chunks;
    bool turns;
};
LinCut lin_cut(int num_seqs, int T, int H, int passes, long long rows, bool packed);
inline int lin_segment_slots(int num_seqs, long long rows, int seg_tokens)
{
    return (int)(num_seqs + (rows + seg_tokens - 1) / seg_tokens);
}
// Tensor-core form, bf16 only.
bool lin_chunk_takes(int dx, int dz);
cudaError_t launch_lin_chunk(const LinRuns &r, int passes, int dx, int dz, cudaStream_t st);
// Sums the per-value-head fp32 gradients over the heads that share a key head and casts them: dqf, dkf
// [rows][H][dk]; dq, dk [rows][Hk][dk].
cudaError_t launch_lin_share(const float *dqf, const float *dkf, void *dq, void *dk, long long rows, int Hk, int H,
                             int d_k, bool bf16, cudaStream_t st);
// `chunk`: the chunk form's kernel (bf16 inputs, head sizes that lin_chunk_takes)
cudaError_t launch_lin_gate_grad(const LinGateGrad &a, bool bf16, bool chunk, cudaStream_t st);
cudaError_t launch_lin_gate_chunk(const LinGateGrad &a, cudaStream_t st);

struct LinDecode {
    const void *q, *k, *v;
    const float *g;
    int g_ld;
    float *state;
    void *o;
    int N, Hk, H, dk, dv;
};
cudaError_t launch_lin_decode(const LinDecode &a, bool bf16, cudaStream_t st);

// Counts log-decays that are positive or NaN and violations of the cu_seqlens contract (cu may be
// NULL), waiting for the verdict on `st` (check_gates.cu).
cudaError_t validate_decay(const float *g, long long n, const int32_t *cu, int num_seqs, long long total,
                           cudaStream_t st, int *bad_gates, int *bad_seqlens);

// Quantised state cache.
struct StateCache {
    const float *states;    // quantise: [M][H][dk][dv]
    float *out;             // dequantise: [n][H][dk][dv]
    uint8_t *codes;         // [S][H][dk][dv]
    float *scales;          // [S][H][dk]
    const int32_t *rows, *slots;
    int n, M, S, H, dk, dv;
    int format;
    unsigned *status;       // device failure word
};
cudaError_t launch_state_quantize(const StateCache &a, cudaStream_t st);
cudaError_t launch_state_dequantize(const StateCache &a, cudaStream_t st);

}  // namespace kda
