"""Cases that measure the per-head-decay linear attention operators and the quantised state cache.

Five operators of this package are called here, in four kinds of case:

  fwd     kda_linattn_chunk_fwd: S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = S_t^T q_t over whole prompts
  train   kda_linattn_chunk_fwd and kda_linattn_chunk_bwd: one layer's share of a training step
  decode  kda_linattn_decode_step: one token per (sequence, head), the fp32 state updated in place
  cache   kda_state_quantize and kda_state_dequantize: state snapshots written to 8-bit cache slots
          and read back as initial states

g is the logarithm of the decay, one value for each token and head or one for each head.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_C = 128  # tokens of a chunk of the plain form


# ---- cases --------------------------------------------------------------------------------------------------------

def _seq(kind, name, dtype, B, T, Hk, H, dk, dv, docs=0, init=False, per_head=False):
    """docs > 0: B is 1 and the T tokens are a packed batch of that many documents."""
    c = {"kind": kind, "dtype": dtype, "B": B, "T": T, "Hk": Hk, "H": H, "dk": dk, "dv": dv, "docs": docs,
         "init": init, "per_head": per_head}
    return dict(c, name=name) if name else c


def _decode(name, dtype, N, Hk, H, dk, dv, per_head=False):
    c = {"kind": "decode", "dtype": dtype, "N": N, "Hk": Hk, "H": H, "dk": dk, "dv": dv, "per_head": per_head}
    return dict(c, name=name) if name else c


def _cache(name, fmt, n, rows, slots, H, dk, dv):
    """n of `rows` states go to n of `slots` cache slots and come back."""
    c = {"kind": "cache", "fmt": fmt, "n": n, "rows": rows, "slots": slots, "H": H, "dk": dk, "dv": dv}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the repository's headline shape: a batch of long prompts, one CTA wave of (sequence, head) pairs
        _seq("fwd", "prompts 8x16x8192", "bf16", 8, 8192, 16, 16, 128, 128),
        # one very long prompt with shared query and key heads: few (sequence, head) pairs, a long token axis
        _seq("fwd", "long prompt 1x16x32768", "bf16", 1, 32768, 4, 16, 128, 128, init=True),
        # a packed serving batch: ragged documents with cached states
        _seq("fwd", "packed 16 docs x32", "bf16", 1, 36864, 32, 32, 128, 128, docs=16, init=True),
        # a short chat turn on a small model: latency counts
        _seq("fwd", "short turn 2x4x150", "bf16", 2, 150, 4, 4, 64, 64, init=True, per_head=True),
        # an fp32 evaluation run, an odd length
        _seq("fwd", "fp32 2x8x1001", "fp32", 2, 1001, 8, 8, 64, 128),
        # one layer of a training step at the repository's backward shape
        _seq("train", "train 4x16x4096", "bf16", 4, 4096, 16, 16, 128, 128),
        # training on packed documents, grouped heads, a narrow value
        _seq("train", "train packed 7 docs", "bf16", 1, 8191, 2, 16, 128, 64, docs=7, init=True),
        # a small fp32 training run (gradient checks, tiny models)
        _seq("train", "train fp32 2x2x300", "fp32", 2, 300, 2, 2, 32, 64, per_head=True),
        # decoding with the repository's serving shape: the state is the whole traffic
        _decode("decode 256x32", "bf16", 256, 32, 32, 128, 128),
        # a single user's decode step: the launch is the cost
        _decode("decode 1x16", "fp32", 1, 4, 16, 64, 64, per_head=True),
        # snapshots of a full serving batch parked in an int8 cache and taken up again
        _cache("cache int8 128x32", "int8", 128, 160, 512, 32, 128, 128),
        # a few states of a small model in e4m3
        _cache("cache e4m3 5x12", "e4m3", 5, 9, 16, 12, 64, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "fwd", "train", "train", "decode", "cache"])
    dim = lambda: rng.choice([128, 128, 128, 64, 64, 32, 16])  # noqa: E731
    dk, dv = dim(), dim()
    if kind == "cache":
        n = _log(rng, 1, 128)
        return _cache(None, rng.choice(["int8", "e4m3"]), n, n + rng.randint(0, 40), n + rng.randint(0, 300),
                      rng.randint(1, 32), dk, dv)
    Hk, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 4])
    H = Hk * group
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    per_head = rng.random() < 0.25
    if kind == "decode":
        return _decode(None, dtype, _log(rng, 1, 256), Hk, H, dk, dv, per_head)
    most = {"fwd": 1 << 20, "train": 1 << 18}[kind] // (16 if dtype == "fp32" else 1)  # tokens x heads
    total = _log(rng, 1, max(1, min(32768, most // H)))
    docs = rng.randint(1, 16) if rng.random() < 0.4 else 0
    B = 1 if docs else max(1, min(total, _log(rng, 1, 8)))
    return _seq(kind, None, dtype, B, max(1, total // B), Hk, H, dk, dv, docs, rng.random() < 0.5, per_head)


# ---- inputs -------------------------------------------------------------------------------------------------------

def _gates(gen, shape, H, per_head):
    """Log-decays as a model makes them: a rate of each head (half lives of one to some hundreds of tokens) times a
    softplus of the token's projection; with per_head, the rates alone."""
    rate = torch.exp2(-8 * torch.rand(H, generator=gen, device="cuda"))
    if per_head:
        return (-rate).contiguous()
    x = torch.randn(*shape, H, generator=gen, device="cuda")
    return (-rate * torch.nn.functional.softplus(x)).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    s = dict(case)
    dk, dv, H = case["dk"], case["dv"], case["H"]
    if case["kind"] == "cache":
        # each key channel of a state has its own size, as its decay and its keys have
        n, rows, slots = case["n"], case["rows"], case["slots"]
        s["states"] = rnd(rows, H, dk, dv) * torch.exp(rnd(rows, H, dk, 1))
        s["row_index"] = torch.randperm(rows, generator=gen, device="cuda")[:n].to(torch.int32)
        s["slot_index"] = torch.randperm(slots, generator=gen, device="cuda")[:n].to(torch.int32)
        dt = torch.int8 if case["fmt"] == "int8" else torch.float8_e4m3fn
        s["codes"] = torch.zeros(slots, H, dk, dv, dtype=torch.int8, device="cuda").view(dt)
        s["scales"] = torch.zeros(slots, H, dk, device="cuda")
        return s
    dt, Hk = _DTYPES[case["dtype"]], case["Hk"]
    lead = (case["N"],) if case["kind"] == "decode" else (case["B"], case["T"])
    # queries carry the 1/sqrt(d_k) of the softmax form, keys have unit length on average
    s["q"] = rnd(*lead, Hk, dk, scale=dk ** -0.5, dtype=dt)
    s["k"] = rnd(*lead, Hk, dk, scale=dk ** -0.5, dtype=dt)
    s["v"] = rnd(*lead, H, dv, dtype=dt)
    s["g"] = _gates(gen, lead, H, case["per_head"])
    if case["kind"] == "decode":
        s["state"] = rnd(case["N"], H, dk, dv)
        return s
    B, T, N = case["B"], case["T"], case["docs"] or case["B"]
    s["cu_seqlens"], s["longest"] = None, T
    if case["docs"]:  # documents of every length, the empty one among them
        cut = torch.randint(0, T + 1, (N - 1,), generator=gen, device="cuda").sort().values.tolist()
        cu = [0, *cut, T]
        s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["longest"] = max(b - a for a, b in zip(cu, cu[1:]))
    s["initial_state"] = rnd(N, H, dk, dv) if case["init"] else None
    if case["kind"] == "train":
        s["d_o"] = rnd(B, T, H, dv, dtype=dt)
        s["d_final_state"] = rnd(N, H, dk, dv) if case["init"] else None
    return s


# ---- one pass -----------------------------------------------------------------------------------------------------

def run(state):
    return {"fwd": _run_fwd, "train": _run_train, "decode": _run_decode, "cache": _run_cache}[state["kind"]](state)


def _run_fwd(s):
    if own:
        import linear_rnn_delta_b200 as kda
        o, sf = kda.kda_linattn_chunk_fwd(s["q"], s["k"], s["v"], s["g"], cu_seqlens=s["cu_seqlens"],
                                          initial_state=s["initial_state"])
    else:
        o, sf = _plain_fwd(s, s["q"].float(), s["k"].float(), s["v"].float(), s["g"], s["initial_state"])
        o = o.to(s["q"].dtype)
    return {"o": o, "final_state": sf}


def _run_train(s):
    if own:
        import linear_rnn_delta_b200 as kda
        o, sf = kda.kda_linattn_chunk_fwd(s["q"], s["k"], s["v"], s["g"], cu_seqlens=s["cu_seqlens"],
                                          initial_state=s["initial_state"])
        dq, dk, dv, dg, ds0 = kda.kda_linattn_chunk_bwd(
            s["q"], s["k"], s["v"], s["g"], s["d_o"], s["d_final_state"], cu_seqlens=s["cu_seqlens"],
            initial_state=s["initial_state"], d_initial_state=s["initial_state"] is not None)
    else:
        dt = s["q"].dtype
        ins = [None if s[n] is None else s[n].float().detach().requires_grad_()
               for n in ("q", "k", "v", "g", "initial_state")]
        with torch.enable_grad():
            o, sf = _plain_fwd(s, *ins)
            outs, douts = [o], [s["d_o"].float()]
            if s["d_final_state"] is not None:
                outs.append(sf)
                douts.append(s["d_final_state"])
            grads = iter(torch.autograd.grad(outs, [x for x in ins if x is not None], douts))
        dq, dk, dv, dg = next(grads).to(dt), next(grads).to(dt), next(grads).to(dt), next(grads)
        ds0 = next(grads, None)
        o, sf = o.detach().to(dt), sf.detach()
    out = {"o": o, "final_state": sf, "dq": dq, "dk": dk, "dv": dv, "dg": dg}
    if ds0 is not None:
        out["d_initial_state"] = ds0
    return out


def _run_decode(s):
    if own:
        import linear_rnn_delta_b200 as kda
        o = kda.kda_linattn_decode_step(s["q"], s["k"], s["v"], s["g"], s["state"])
    else:
        group = s["H"] // s["Hk"]
        q, k = (s[n].float().repeat_interleave(group, dim=1) for n in ("q", "k"))
        S = s["state"]
        S *= s["g"].exp()[..., None, None]
        S += k[..., :, None] * s["v"].float()[..., None, :]
        o = (q[..., None, :] @ S)[..., 0, :].to(s["q"].dtype)
    return {"o": o, "state": s["state"]}


def _run_cache(s):
    if own:
        import linear_rnn_delta_b200 as kda
        kda.kda_state_quantize(s["states"], s["codes"], s["scales"], s["slot_index"], rows=s["row_index"])
        restored = kda.kda_state_dequantize(s["codes"], s["scales"], s["slot_index"])
    else:
        at = s["slot_index"].long()
        x = s["states"][s["row_index"].long()]
        amax = x.abs().amax(-1)
        top = 127.0 if s["fmt"] == "int8" else 448.0
        # which code a value next to a border takes is decided in 64 bits
        y = x.double() * top / torch.where(amax > 0, amax, 1.0).double()[..., None]
        if s["fmt"] == "int8":
            codes = y.round().to(torch.int8)
        else:
            step = torch.exp2((torch.frexp(y).exponent - 1).clamp(min=-6).double() - 3)
            codes = ((y / step).round() * step).float().to(torch.float8_e4m3fn)
        s["codes"].view(torch.int8)[at] = codes.view(torch.int8)
        s["scales"][at] = (amax.double() / top).float()
        got = s["codes"].view(torch.int8)[at]
        got = got.float() if s["fmt"] == "int8" else got.view(torch.float8_e4m3fn).float()
        restored = got * s["scales"][at][..., None]
    return {"restored": restored, "scales": s["scales"]}


def _plain_fwd(s, q, k, v, g, s0):
    """The recurrence in chunks of 128 tokens: the quadratic form within a chunk, the states before each chunk as one
    product with the decays between chunks.  A packed batch is one row of chunks, the others have a row for each
    sequence.  Sums of log-decays and the decays between chunks in 64 bits, the rest in 32."""
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    docs, dev = s["docs"], q.device
    if docs:
        R, F, nc = 1, docs, T // _C + docs                                   # rows, sequences of a row, chunks of a row
        first, length = s["cu_seqlens"][None, :-1].long(), s["cu_seqlens"].long().diff()[None]
    else:
        R, F, nc = B, 1, max(1, -(-T // _C))
        first, length = torch.arange(B, device=dev)[:, None] * T, torch.full((B, 1), T, device=dev)
    upto = ((length + _C - 1) // _C).cumsum(-1)                              # [R,F]: chunks up to a sequence's end
    i = torch.arange(nc, device=dev).expand(R, nc)
    doc = torch.searchsorted(upto, i.contiguous(), right=True)               # [R,nc]; F: a chunk of no sequence
    of = doc.clamp(max=F - 1)
    begin = upto.gather(-1, of) - (length.gather(-1, of) + _C - 1) // _C     # first chunk of its sequence
    at = (i - begin)[..., None] * _C + torch.arange(_C, device=dev)          # [R,nc,C]: place in the sequence
    there = (doc < F)[..., None] & (at < length.gather(-1, of)[..., None])
    token = torch.where(there, first.gather(-1, of)[..., None] + at, B * T)

    def chunks(x):  # [B,T,H,...] -> [R,H,nc,C,...], zero where there is no token
        x = x.reshape(B * T, *x.shape[2:])
        return torch.cat([x, torch.zeros_like(x[:1])])[token].movedim(3, 1)

    q, k, v = chunks(q.repeat_interleave(H // Hk, dim=2)), chunks(k.repeat_interleave(H // Hk, dim=2)), chunks(v)
    c = chunks(g.double().expand(B, T, H).clamp(min=-1e4)).cumsum(-1)       # [R,H,nc,C]
    end = c[..., -1:]
    tri = torch.ones(_C, _C, dtype=torch.bool, device=dev).tril()
    lam = torch.where(tri, c[..., :, None] - c[..., None, :], -math.inf).exp().float()
    o = ((q @ k.transpose(-1, -2)) * lam) @ v
    kv = ((k * (end - c).exp().float()[..., None]).transpose(-1, -2) @ v).reshape(R, H, nc, dk * dv)
    # before chunk i: the sum over its sequence's chunks j < i of the decay over chunks j+1 .. i-1 times kv_j, and
    # the initial state decayed by all of them; after a sequence likewise
    E = torch.nn.functional.pad(end[..., 0].cumsum(-1), (1, 0))              # [R,H,nc+1]: decay up to chunk i
    E0 = E.gather(-1, begin[:, None].expand(R, H, nc))
    same = (doc[:, :, None] == doc[:, None, :]) & (i[:, :, None] > i[:, None, :])
    w = torch.where(same[:, None], E[..., :-1, None] - E[..., None, 1:], -math.inf).exp().float()
    before = w @ kv
    lastE = E.gather(-1, upto[:, None].expand(R, H, F))                      # [R,H,F]
    mine = doc[:, None, :] == torch.arange(F, device=dev)[:, None]           # [R,F,nc]
    final = torch.where(mine[:, None], lastE[..., None] - E[..., None, 1:], -math.inf).exp().float() @ kv
    if s0 is not None:
        s0 = s0.reshape(R, F, H, dk * dv).movedim(2, 1)                      # [R,H,F,..]
        since = (E[..., :-1] - E0).exp().float()
        before = before + since[..., None] * s0[torch.arange(R, device=dev)[:, None], :, of].movedim(2, 1)
        firstE = E.gather(-1, (upto - (length + _C - 1) // _C)[:, None].expand(R, H, F))
        final = final + (lastE - firstE).exp().float()[..., None] * s0
    o = o + (q * c.exp().float()[..., None]) @ before.reshape(R, H, nc, dk, dv)
    out = torch.zeros(B * T + 1, H, dv, device=dev).index_copy(0, token.reshape(-1), o.movedim(1, 3).reshape(-1, H, dv))
    return out[:-1].reshape(B, T, H, dv), final.movedim(1, 2).reshape(R * F, H, dk, dv)


# ---- the definition in 64 bits ------------------------------------------------------------------------------------

def _padded(s, x, N):
    """[N, longest, ...] in 64 bits, zeros behind each sequence's end."""
    if not s["docs"]:
        return x.double()
    cu = s["cu_seqlens"].tolist()
    out = torch.zeros(N, max(1, s["longest"]), *x.shape[2:], dtype=torch.float64, device=x.device)
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        out[n, :b - a] = x[0, a:b]
    return out


def _unpadded(s, x):
    if not s["docs"]:
        return x
    cu = s["cu_seqlens"].tolist()
    return torch.cat([x[n, :b - a] for n, (a, b) in enumerate(zip(cu, cu[1:]))])[None]


def _scan(q, k, v, a, S):
    """Token by token: S <- a_t S + k_t v_t^T, o_t = S^T q_t."""
    o = torch.empty_like(v)
    for t in range(v.shape[1]):
        S = torch.addcmul(S * a[:, t, :, None, None], k[:, t, :, :, None], v[:, t, :, None, :])
        o[:, t] = (q[:, t, :, None, :] @ S)[:, :, 0]
    return o, S


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "cache":
        return _exact_cache(s)
    group = case["H"] // case["Hk"]
    if case["kind"] == "decode":
        q, k = (s[n].double().repeat_interleave(group, dim=1) for n in ("q", "k"))
        S = s["g"].double().exp()[..., None, None] * s["state"].double() + torch.einsum("nhi,nhj->nhij", k, s["v"].double())
        return {"o": torch.einsum("nhij,nhi->nhj", S, q), "state": S}
    B, T, H, dk, dv = (case[n] for n in ("B", "T", "H", "dk", "dv"))
    N = case["docs"] or B
    q, k = (_padded(s, s[n], N).repeat_interleave(group, dim=2) for n in ("q", "k"))
    v = _padded(s, s["v"], N)
    a = _padded(s, s["g"].expand(B, T, H), N).exp()          # a padding token has g = 0: it leaves the state
    s0 = torch.zeros(N, H, dk, dv, dtype=torch.float64, device=q.device) if s["initial_state"] is None \
        else s["initial_state"].double()
    o, sf = _scan(q, k, v, a, s0)
    if case["kind"] == "fwd":
        return {"o": _unpadded(s, o), "final_state": sf}
    # dq_t = S_t do_t; with G_t the derivative by S_t: G_t = a_{t+1} G_{t+1} + q_t do_t^T, dk_t = G_t v_t,
    # dv_t = G_t^T k_t, and g_t enters through every pair of tokens that it stands between
    do = _padded(s, s["d_o"], N)
    dsf = torch.zeros_like(sf) if s["d_final_state"] is None else s["d_final_state"].double()
    dq, _ = _scan(do, v, k, a, s0.transpose(-1, -2))
    back = torch.cat([torch.ones_like(a[:, :1]), a.flip(1)[:, :-1]], 1)
    rev = [x.flip(1) for x in (q, k, v, do)]
    dvg, G = _scan(rev[1], rev[0], rev[3], back, dsf)
    dkg, _ = _scan(rev[2], rev[3], rev[0], back, dsf.transpose(-1, -2))
    dk_, dv_ = dkg.flip(1), dvg.flip(1)
    D = (q * dq - k * dk_).sum(-1)
    dg = D.flip(1).cumsum(1).flip(1) + (sf * dsf).sum((-1, -2))[:, None]
    share = lambda x: x.reshape(*x.shape[:2], case["Hk"], group, x.shape[-1]).sum(3)  # noqa: E731
    dg = _unpadded(s, dg)
    out = {"o": _unpadded(s, o), "final_state": sf, "dq": _unpadded(s, share(dq)), "dk": _unpadded(s, share(dk_)),
           "dv": _unpadded(s, dv_), "dg": dg.sum((0, 1)) if case["per_head"] else dg}
    if s["initial_state"] is not None:
        out["d_initial_state"] = G * a[:, 0, :, None, None]
    return out


def _exact_cache(s):
    """The nearest code to value / amax * top, found by search among all codes' values and the borders between them."""
    x = s["states"][s["row_index"].long()].double()
    if s["fmt"] == "int8":
        values = torch.arange(-127, 128, device=x.device).double()
    else:
        values = torch.arange(-126, 127, device=x.device)
        values = torch.sign(values) * values.abs().to(torch.uint8).view(torch.float8_e4m3fn).double()
        values = torch.unique(values)
    amax = x.abs().amax(-1, keepdim=True)
    top = values[-1]
    y = x * top / torch.where(amax > 0, amax, 1.0)
    border = (values[1:] + values[:-1]) / 2
    low = torch.searchsorted(border, y.reshape(-1).contiguous())              # y <= border: the lower one
    tie = border[low.clamp(max=border.numel() - 1)] == y.reshape(-1)
    odd = (values.numel() // 2 - low).abs() % 2 == 1                          # codes count from zero outwards
    code = values[low + (tie & odd)].reshape(y.shape)
    scales = s["scales"].double()
    scales[s["slot_index"].long()] = (amax / top)[..., 0]
    return {"restored": code * (amax / top), "scales": scales}


# ---- what a pass cannot do without --------------------------------------------------------------------------------

def work(case):
    dk, dv, H = case["dk"], case["dv"], case["H"]
    if case["kind"] == "cache":  # written: the state in, codes and scales out; read back: the other way round
        one = case["H"] * (dk * dv * 5 + dk * 4)
        return {"bytes": 2 * case["n"] * one, "flops": 4 * case["n"] * H * dk * dv}
    size, Hk = 2 if case["dtype"] == "bf16" else 4, case["Hk"]
    if case["kind"] == "decode":
        N = case["N"]
        return {"bytes": N * (8 * H * dk * dv + size * (2 * Hk * dk + 2 * H * dv) + 4 * H), "flops": 5 * N * H * dk * dv}
    tokens, N = case["B"] * case["T"], case["docs"] or case["B"]
    gate = 4 * H if case["per_head"] else 4 * tokens * H
    one_state = 4 * N * H * dk * dv
    fwd = tokens * size * (2 * Hk * dk + 2 * H * dv) + gate + one_state * (2 if case["init"] else 1)
    if case["kind"] == "fwd":
        return {"bytes": fwd, "flops": 4 * tokens * H * dk * dv}
    # backward: q, k, v, do and the gate in, four gradients out, the state gradients where there are any
    bwd = tokens * size * (4 * Hk * dk + 3 * H * dv) + 2 * gate + one_state * (3 if case["init"] else 0)
    return {"bytes": fwd + bwd, "flops": 14 * tokens * H * dk * dv}
