// C ABI of linear attention with one decay per head and of the quantised state cache: host-side
// argument checks and dispatch.  Declarations, layouts and error semantics: include/kda.h.
#include <climits>

#include "../../include/kda.h"
#include "api.cuh"
#include "common.cuh"
#include "linattn.cuh"

namespace {

using kda::LinRun;
using kda::api::aligned16;
using kda::api::cuda_fail;
using kda::api::fail;
using kda::api::head_dim_ok;

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

struct LinSizes {
    int dtype, B, T, Hk, H, dk, dv, N;
    bool packed;
    long long rows;
};

// Sizes shared by the calls; false with the detail set.
int lin_sizes(LinSizes &s, int dtype, int B, int T, int Hk, int H, int d_k, int d_v, bool packed, int num_seqs)
{
    if (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_F32)
        return fail(KDA_ERR_INVALID_ARG, "dtype %d is not BF16(0) or F32(1)", dtype);
    if (B < 1 || T < 0 || Hk < 1 || H < 1)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes B=%d T=%d Hk=%d H=%d (need B>=1, T>=0, Hk>=1, H>=1)", B, T, Hk, H);
    if (H % Hk)
        return fail(KDA_ERR_INVALID_ARG, "H=%d value heads are not a multiple of Hk=%d query and key heads", H, Hk);
    if (d_k < 1 || d_v < 1) return fail(KDA_ERR_INVALID_ARG, "head dims must be positive (d_k=%d, d_v=%d)", d_k, d_v);
    if (!head_dim_ok(d_k) || !head_dim_ok(d_v))
        return fail(KDA_ERR_UNSUPPORTED, "head dims d_k=%d, d_v=%d: supported are 16, 32, 64, 128", d_k, d_v);
    if (packed && B != 1) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens requires B == 1 (got B=%d)", B);
    if (packed && num_seqs < 1)
        return fail(KDA_ERR_INVALID_ARG, "num_seqs must be >= 1 with cu_seqlens (got %d)", num_seqs);
    s = LinSizes{dtype, B, T, Hk, H, d_k, d_v, packed ? num_seqs : B, packed, (long long)B * T};
    // row numbers and CTA counts are 32-bit
    if (s.rows > INT_MAX / 2 || (long long)s.N * H > INT_MAX / 64 || s.rows * H > (1ll << 39))
        return fail(KDA_ERR_INVALID_ARG, "problem too large (B*T=%lld, sequences*heads=%lld)", s.rows,
                    (long long)s.N * H);
    return KDA_OK;
}

int need_ptr(const void *p, const char *name)
{
    if (!p) return fail(KDA_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned16(p)) return fail(KDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
    return KDA_OK;
}
int opt_ptr(const void *p, const char *name)
{
    if (p && !aligned16(p)) return fail(KDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
    return KDA_OK;
}
int need_gate(const float *g)   // read as single floats
{
    if (!g) return fail(KDA_ERR_INVALID_ARG, "g is NULL");
    if (reinterpret_cast<uintptr_t>(g) & 3u) return fail(KDA_ERR_INVALID_ARG, "g is not 4-byte aligned");
    return KDA_OK;
}
#define CHECK(x) do { const int rc_ = (x); if (rc_ != KDA_OK) return rc_; } while (0)

int check_cu(const int32_t *cu)
{
    if (cu && (reinterpret_cast<uintptr_t>(cu) & 3u))
        return fail(KDA_ERR_INVALID_ARG, "cu_seqlens is not 4-byte aligned");
    return KDA_OK;
}

LinRun base_run(const LinSizes &s, const float *g, int g_per_token, const int32_t *cu)
{
    LinRun r{};
    r.gx = r.gy = r.gz = 1;
    r.g = g;
    r.g_ld = g_per_token ? s.H : 0;
    r.num_seqs = s.N;
    r.T = s.T;
    r.H = s.H;
    r.cu_seqlens = cu;
    r.rows = s.rows;
    return r;
}

// Tensor-core form for bf16 and the head sizes it takes, else the token scan.
bool chunk_form(const LinSizes &s, unsigned flags)
{
    return s.dtype == KDA_DTYPE_BF16 && !(flags & KDA_FLAG_FORCE_SCAN) && kda::lin_chunk_takes(s.dk, s.dv);
}
// Segments of the token axis: their length and the workspace of a pass's states and decays.
struct Segments {
    int chunks, tokens, slots;
    bool turns;
    size_t sync;            // bytes of all passes' tickets and hand-overs, first in the workspace
    size_t totals, total;   // a pass's offset and size in bytes
    size_t bytes;
};
Segments segments(const LinSizes &s, int passes, bool chunk)
{
    Segments g{};
    if (chunk) {
        const kda::LinCut cut = kda::lin_cut(s.N, s.T, s.H, passes, s.rows, s.packed);
        g.chunks = cut.chunks;
        g.turns = cut.turns;
    } else {
        g.chunks = kda::lin_scan_segment_chunks(s.N, s.H, passes, s.dk, s.dv, s.rows);
    }
    if (!g.chunks) return g;
    g.tokens = g.chunks * (chunk ? kda::SLOT_TOKENS : kda::SCAN_CHUNK);
    g.slots = kda::lin_segment_slots(s.N, s.rows, g.tokens);
    g.sync = g.turns ? up256((size_t)passes * (1 + g.slots) * s.H * 4) : 0;
    g.totals = up256((size_t)g.slots * s.H * s.dk * s.dv * 4);
    g.total = g.totals + (g.turns ? 0 : up256((size_t)g.slots * s.H * 4));
    g.bytes = g.sync + passes * g.total;
    return g;
}
// Passes of one shape; `seg_ws` holds a segments' workspace for each.
cudaError_t launch_runs(LinRun *r, int passes, int dx, int dz, bool chunk, bool bf16, const Segments &g, uint8_t *seg_ws,
                        cudaStream_t st)
{
    for (int i = 0; g.chunks && i < passes; ++i) {
        r[i].seg_chunks = g.chunks;
        r[i].seg_tokens = g.tokens;
        r[i].slots = g.slots;
        r[i].seg_state = reinterpret_cast<float *>(seg_ws + g.sync + i * g.total);
        if (g.turns) {
            r[i].tickets = reinterpret_cast<int *>(seg_ws) + (size_t)i * (1 + g.slots) * r[i].H;
            r[i].handed = r[i].tickets + r[i].H;
        } else {
            r[i].seg_total = reinterpret_cast<float *>(seg_ws + g.sync + i * g.total + g.totals);
        }
    }
    if (g.turns) {
        const cudaError_t e = cudaMemsetAsync(seg_ws, 0, g.sync, st);
        if (e != cudaSuccess) return e;
    }
    kda::LinRuns p{};
    for (int i = 0; i < passes; ++i) p.a[i] = r[i];
    return chunk ? kda::launch_lin_chunk(p, passes, dx, dz, st) : kda::launch_lin_scan(p, passes, dx, dz, bf16, st);
}

// Backward workspace regions.
struct BwdLayout {
    size_t dqf, dkf, snap_s, snap_g, partial, seg, total;
    int slots, together;   // passes of one launch
    Segments g;
};
BwdLayout bwd_layout(const LinSizes &s, bool chunk)
{
    BwdLayout L;
    // dq, dk and dv are passes of one shape where d_k = d_v and their outputs have one type; dq and dk always are
    const bool shared = s.H != s.Hk;
    L.together = s.dk == s.dv && !shared ? 3 : 2;
    L.g = segments(s, L.together, chunk);
    L.slots = (int)(s.N + (s.rows + kda::SLOT_TOKENS - 1) / kda::SLOT_TOKENS);
    const size_t grad = shared ? up256((size_t)s.rows * s.H * s.dk * 4) : 0;   // of each value head
    const size_t snap = up256((size_t)L.slots * s.H * s.dk * s.dv * 4);
    L.dqf = 0;
    L.dkf = L.dqf + grad;
    L.snap_s = L.dkf + grad;
    L.snap_g = L.snap_s + snap;
    L.partial = L.snap_g + snap;
    L.seg = L.partial + up256((size_t)L.slots * s.H * 4);
    L.total = L.seg + L.g.bytes;
    return L;
}

}  // namespace

extern "C" size_t kda_linattn_chunk_fwd_workspace_size(int dtype, int B, int T, int Hk, int H, int d_k, int d_v,
                                                       int has_cu_seqlens, int num_seqs, unsigned flags)
{
    LinSizes s;
    if (lin_sizes(s, dtype, B, T, Hk, H, d_k, d_v, has_cu_seqlens != 0, num_seqs) != KDA_OK) return 0;
    return segments(s, 1, chunk_form(s, flags)).bytes;
}

extern "C" int kda_linattn_chunk_fwd(int dtype, int B, int T, int Hk, int H, int d_k, int d_v,
                                     const void *q, const void *k, const void *v, const float *g, int g_per_token,
                                     const int32_t *cu_seqlens, int num_seqs, const float *initial_state,
                                     float *final_state, float *chunk_states, void *o, void *workspace,
                                     size_t workspace_bytes, unsigned flags, void *stream)
{
    LinSizes s;
    CHECK(lin_sizes(s, dtype, B, T, Hk, H, d_k, d_v, cu_seqlens != nullptr, num_seqs));
    if (flags & ~(KDA_FLAG_VALIDATE_RANGE | KDA_FLAG_FORCE_SCAN | KDA_FLAG_DEBUG_STALL))
        return fail(KDA_ERR_INVALID_ARG, "kda_linattn_chunk_fwd: unknown or unsupported flag bits 0x%x", flags);
    if (T > 0) {
        CHECK(need_ptr(q, "q"));
        CHECK(need_ptr(k, "k"));
        CHECK(need_ptr(v, "v"));
        CHECK(need_gate(g));
        CHECK(need_ptr(o, "o"));
    }
    CHECK(check_cu(cu_seqlens));
    CHECK(opt_ptr(initial_state, "initial_state"));
    CHECK(opt_ptr(final_state, "final_state"));
    CHECK(opt_ptr(chunk_states, "chunk_states"));
    CHECK(opt_ptr(workspace, "workspace"));
    const bool chunk = chunk_form(s, flags);
    const Segments segs = segments(s, 1, chunk);
    if ((flags & KDA_FLAG_DEBUG_STALL) && !segs.turns)
        return fail(KDA_ERR_INVALID_ARG, "KDA_FLAG_DEBUG_STALL needs segments in turn");
    if (segs.bytes && (!workspace || workspace_bytes < segs.bytes))
        return fail(KDA_ERR_INVALID_ARG, "kda_linattn_chunk_fwd needs a workspace of %zu bytes", segs.bytes);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (flags & KDA_FLAG_VALIDATE_RANGE) {
        int bad_g = 0, bad_cu = 0;
        const long long ng = s.rows == 0 ? 0 : (g_per_token ? s.rows * H : H);
        const cudaError_t e = kda::validate_decay(g, ng, cu_seqlens, s.N, s.rows, st, &bad_g, &bad_cu);
        if (e != cudaSuccess) return cuda_fail(e, "input validation");
        if (bad_cu)
            return fail(KDA_ERR_INVALID_ARG, "cu_seqlens violates cu[0] = 0, cu[n] <= cu[n+1], cu[N] = %lld "
                                             "(%d violations)", s.rows, bad_cu);
        if (bad_g) return fail(KDA_ERR_RANGE, "%d log-decays are positive or NaN", bad_g);
    }
    LinRun r = base_run(s, g, g_per_token, cu_seqlens);
    r.x = q;
    r.y = k;
    r.z = v;
    r.gx = r.gy = H / Hk;
    r.s_in = initial_state;
    r.s_out = final_state;
    r.snap = chunk_states;
    r.snap_tokens = kda::SLOT_TOKENS;
    r.out = o;
    r.stall = (flags & KDA_FLAG_DEBUG_STALL) != 0;
    const cudaError_t e = launch_runs(&r, 1, d_k, d_v, chunk, dtype == KDA_DTYPE_BF16, segs,
                                      static_cast<uint8_t *>(workspace), st);
    if (e != cudaSuccess) return cuda_fail(e, "kda_linattn_chunk_fwd launch");
    return KDA_OK;
}

extern "C" size_t kda_linattn_chunk_bwd_workspace_size(int dtype, int B, int T, int Hk, int H, int d_k, int d_v,
                                                       int has_cu_seqlens, int num_seqs)
{
    LinSizes s;
    if (lin_sizes(s, dtype, B, T, Hk, H, d_k, d_v, has_cu_seqlens != 0, num_seqs) != KDA_OK) return 0;
    // with KDA_FLAG_FORCE_SCAN or without
    const size_t scan = bwd_layout(s, false).total, chunk = bwd_layout(s, chunk_form(s, 0u)).total;
    return scan > chunk ? scan : chunk;
}

extern "C" int kda_linattn_chunk_bwd(int dtype, int B, int T, int Hk, int H, int d_k, int d_v,
                                     const void *q, const void *k, const void *v, const float *g, int g_per_token,
                                     const int32_t *cu_seqlens, int num_seqs, const float *initial_state,
                                     const void *d_o, const float *d_final_state,
                                     void *dq, void *dk, void *dv, float *dg, float *d_initial_state,
                                     void *workspace, size_t workspace_bytes, unsigned flags, void *stream)
{
    LinSizes s;
    CHECK(lin_sizes(s, dtype, B, T, Hk, H, d_k, d_v, cu_seqlens != nullptr, num_seqs));
    if (flags & ~(KDA_FLAG_FORCE_SCAN | KDA_FLAG_DEBUG_STALL))
        return fail(KDA_ERR_INVALID_ARG, "kda_linattn_chunk_bwd: unknown or unsupported flag bits 0x%x", flags);
    if ((flags & KDA_FLAG_DEBUG_STALL) && !chunk_form(s, flags))
        return fail(KDA_ERR_INVALID_ARG, "KDA_FLAG_DEBUG_STALL needs the tensor-core form");
    if (T > 0) {
        const void *ptrs[] = {q, k, v, d_o, dq, dk, dv};
        const char *names[] = {"q", "k", "v", "d_o", "dq", "dk", "dv"};
        for (int i = 0; i < 7; ++i) CHECK(need_ptr(ptrs[i], names[i]));
        CHECK(need_gate(g));
    }
    if (T > 0 || !g_per_token) {
        if (!dg) return fail(KDA_ERR_INVALID_ARG, "dg is NULL");
        if (reinterpret_cast<uintptr_t>(dg) & 3u) return fail(KDA_ERR_INVALID_ARG, "dg is not 4-byte aligned");
    }
    CHECK(check_cu(cu_seqlens));
    CHECK(opt_ptr(initial_state, "initial_state"));
    CHECK(opt_ptr(d_final_state, "d_final_state"));
    CHECK(opt_ptr(d_initial_state, "d_initial_state"));
    // both are read after d_initial_state is written
    if (d_initial_state && (d_initial_state == d_final_state || d_initial_state == initial_state))
        return fail(KDA_ERR_INVALID_ARG, "d_initial_state is d_final_state or initial_state");
    const bool chunk = chunk_form(s, flags);
    const BwdLayout L = bwd_layout(s, chunk);
    if (!workspace || !aligned16(workspace) || workspace_bytes < L.total)
        return fail(KDA_ERR_INVALID_ARG, "kda_linattn_chunk_bwd needs a 16-byte aligned workspace of %zu bytes", L.total);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const bool bf16 = dtype == KDA_DTYPE_BF16;
    const int group = H / Hk;
    auto f32 = [&](size_t off) { return reinterpret_cast<float *>(ws + off); };
    LinRun runs[3];
    // dq_t = S_t do_t: forward in time, the state transposed
    LinRun &rq = runs[0] = base_run(s, g, g_per_token, cu_seqlens);
    rq.x = d_o; rq.y = v; rq.z = k;
    rq.gz = group;
    rq.s_in = initial_state;
    rq.in_t = 1;
    rq.snap = f32(L.snap_s);
    rq.snap_tokens = kda::SLOT_TOKENS;
    rq.out = group > 1 ? f32(L.dqf) : dq;
    rq.out_f32 = group > 1;
    // dk_t = G_t v_t: backward in time, the state transposed
    LinRun &rk = runs[1] = base_run(s, g, g_per_token, cu_seqlens);
    rk.reverse = 1;
    rk.x = v; rk.y = d_o; rk.z = q;
    rk.gz = group;
    rk.s_in = d_final_state;
    rk.in_t = 1;
    rk.snap = f32(L.snap_g);
    rk.snap_tokens = kda::SLOT_TOKENS;
    rk.out = group > 1 ? f32(L.dkf) : dk;
    rk.out_f32 = group > 1;
    // dv_t = G_t^T k_t: backward in time
    LinRun &rv = runs[2] = base_run(s, g, g_per_token, cu_seqlens);
    rv.reverse = 1;
    rv.x = k; rv.y = q; rv.z = d_o;
    rv.gx = rv.gy = group;
    rv.s_in = d_final_state;
    rv.s_out = d_initial_state;
    rv.out = dv;
    cudaError_t e = launch_runs(runs, L.together, d_v, d_k, chunk, bf16, L.g, ws + L.seg, st);
    if (e == cudaSuccess && L.together < 3) e = launch_runs(runs + 2, 1, d_k, d_v, chunk, bf16, L.g, ws + L.seg, st);
    if (e != cudaSuccess) return cuda_fail(e, "kda_linattn_chunk_bwd passes");
    if (group > 1 && (e = kda::launch_lin_share(f32(L.dqf), f32(L.dkf), dq, dk, s.rows, Hk, H, d_k, bf16, st)) != cudaSuccess)
        return cuda_fail(e, "kda_linattn_chunk_bwd head sums");
    kda::LinGateGrad gg{};
    gg.q = q; gg.k = k; gg.v = v; gg.d_o = d_o;
    gg.s_init = initial_state;
    gg.snap_s = f32(L.snap_s); gg.snap_g = f32(L.snap_g);
    gg.g = g;
    gg.g_ld = g_per_token ? H : 0;
    gg.g_end = d_final_state;
    gg.dg = g_per_token ? dg : nullptr;
    gg.partial = g_per_token ? nullptr : f32(L.partial);
    gg.dg_head = g_per_token ? nullptr : dg;
    gg.rows = s.rows;
    gg.Hk = Hk; gg.H = H; gg.dk = d_k; gg.dv = d_v;
    gg.num_seqs = s.N; gg.T = T; gg.slots = L.slots;
    gg.cu_seqlens = cu_seqlens;
    gg.stall = (flags & KDA_FLAG_DEBUG_STALL) != 0;
    if ((e = kda::launch_lin_gate_grad(gg, bf16, chunk, st)) != cudaSuccess) return cuda_fail(e, "kda_linattn_chunk_bwd dg");
    return KDA_OK;
}

extern "C" int kda_linattn_decode_step(int dtype, int N, int Hk, int H, int d_k, int d_v,
                                       const void *q, const void *k, const void *v, const float *g, int g_per_token,
                                       float *state, void *o, unsigned flags, void *stream)
{
    LinSizes s;
    if (N < 1) return fail(KDA_ERR_INVALID_ARG, "bad size N=%d (need N>=1)", N);
    CHECK(lin_sizes(s, dtype, N, 1, Hk, H, d_k, d_v, false, 0));
    if (flags & ~KDA_FLAG_VALIDATE_RANGE)
        return fail(KDA_ERR_INVALID_ARG, "kda_linattn_decode_step: unknown or unsupported flag bits 0x%x", flags);
    const void *ptrs[] = {q, k, v, state, o};
    const char *names[] = {"q", "k", "v", "state", "o"};
    for (int i = 0; i < 5; ++i) CHECK(need_ptr(ptrs[i], names[i]));
    CHECK(need_gate(g));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (flags & KDA_FLAG_VALIDATE_RANGE) {
        int bad_g = 0, bad_cu = 0;
        const cudaError_t e = kda::validate_decay(g, g_per_token ? (long long)N * H : H, nullptr, 0, 0, st, &bad_g,
                                                  &bad_cu);
        if (e != cudaSuccess) return cuda_fail(e, "input validation");
        if (bad_g) return fail(KDA_ERR_RANGE, "%d log-decays are positive or NaN", bad_g);
    }
    const kda::LinDecode a{q, k, v, g, g_per_token ? H : 0, state, o, N, Hk, H, d_k, d_v};
    const cudaError_t e = kda::launch_lin_decode(a, dtype == KDA_DTYPE_BF16, st);
    if (e != cudaSuccess) return cuda_fail(e, "kda_linattn_decode_step launch");
    return KDA_OK;
}

namespace {

int cache_args(kda::StateCache &a, int format, int n, int num_slots, int H, int d_k, int d_v, const void *codes,
               const float *scales, const int32_t *slots)
{
    if (format != KDA_CACHE_INT8 && format != KDA_CACHE_E4M3)
        return fail(KDA_ERR_INVALID_ARG, "format %d is not INT8(0) or E4M3(1)", format);
    if (n < 0 || num_slots < 1 || H < 1)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes n=%d num_slots=%d H=%d (need n>=0, num_slots>=1, H>=1)", n,
                    num_slots, H);
    if (d_k < 1 || d_v < 1) return fail(KDA_ERR_INVALID_ARG, "head dims must be positive (d_k=%d, d_v=%d)", d_k, d_v);
    if (!head_dim_ok(d_k) || !head_dim_ok(d_v))
        return fail(KDA_ERR_UNSUPPORTED, "head dims d_k=%d, d_v=%d: supported are 16, 32, 64, 128", d_k, d_v);
    if ((long long)n * H > INT_MAX) return fail(KDA_ERR_INVALID_ARG, "problem too large (n*H=%lld)", (long long)n * H);
    if (!slots && n > num_slots)
        return fail(KDA_ERR_INVALID_ARG, "n=%d entries without slots exceed num_slots=%d", n, num_slots);
    CHECK(need_ptr(codes, "codes"));
    CHECK(need_ptr(scales, "scales"));
    if (slots && (reinterpret_cast<uintptr_t>(slots) & 3u))
        return fail(KDA_ERR_INVALID_ARG, "slots is not 4-byte aligned");
    a = kda::StateCache{};
    a.codes = static_cast<uint8_t *>(const_cast<void *>(codes));
    a.scales = const_cast<float *>(scales);
    a.slots = slots;
    a.n = n;
    a.S = num_slots;
    a.H = H;
    a.dk = d_k;
    a.dv = d_v;
    a.format = format;
    const cudaError_t e = n ? kda::device_status_word(&a.status) : cudaSuccess;
    if (e != cudaSuccess) return cuda_fail(e, "device failure word");
    return KDA_OK;
}

}  // namespace

extern "C" int kda_state_quantize(int format, int n, int num_states, int num_slots, int H, int d_k, int d_v,
                                  const float *states, const int32_t *rows, const int32_t *slots, void *codes,
                                  float *scales, void *stream)
{
    kda::StateCache a;
    if (num_states < 1) return fail(KDA_ERR_INVALID_ARG, "bad size num_states=%d (need num_states>=1)", num_states);
    if (!rows && n > num_states)
        return fail(KDA_ERR_INVALID_ARG, "n=%d entries without rows exceed num_states=%d", n, num_states);
    if (rows && (reinterpret_cast<uintptr_t>(rows) & 3u))
        return fail(KDA_ERR_INVALID_ARG, "rows is not 4-byte aligned");
    CHECK(need_ptr(states, "states"));
    CHECK(cache_args(a, format, n, num_slots, H, d_k, d_v, codes, scales, slots));
    if (n == 0) return KDA_OK;
    a.states = states;
    a.rows = rows;
    a.M = num_states;
    const cudaError_t e = kda::launch_state_quantize(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_state_quantize launch");
    return KDA_OK;
}

extern "C" int kda_state_dequantize(int format, int n, int num_slots, int H, int d_k, int d_v, const void *codes,
                                    const float *scales, const int32_t *slots, float *states, void *stream)
{
    kda::StateCache a;
    if (n > 0) CHECK(need_ptr(states, "states"));
    CHECK(cache_args(a, format, n, num_slots, H, d_k, d_v, codes, scales, slots));
    if (n == 0) return KDA_OK;
    a.out = states;
    const cudaError_t e = kda::launch_state_dequantize(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kda_state_dequantize launch");
    return KDA_OK;
}
