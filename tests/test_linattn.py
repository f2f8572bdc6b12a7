"""Linear attention with one decay per head against the float64 token-by-token form (linattn_ref.py).

Tolerances.  A value that is a sum of products is compared with an allowance of c * A, A the same sum over
magnitudes, plus half a step of its output type relative to itself (bf16 2^-8, fp32 2^-24):
  - the token scan rounds the state twice a token and adds d products: c = (2 T + d + 8) 2^-24;
  - the chunked form splits fp32 factors into bf16 parts.  Two parts leave 2^-16 of the value at most (a rounding
    is off by 2^-8 of the value, the second by 2^-8 of that): the state in the outputs (o, dq, dk, dv).  The
    pairs' weights within a chunk are rounded once there: 2^-8 of the sum over pairs of their magnitude, pair_size.
    In a chunk that decays by more than 2^-96 (`strong`) the query side is rounded once instead, too: 2^-8 of A.
    States have three parts (2^-24) and keep the scan's allowance: their own additions are fewer than the scan's.
Gradients of shared heads are sums over them (A is, too).  Gate gradients sum the pairs' shares in fp32, each of them
a product of sums over channels; gate_sum_size adds up their magnitudes (and those of the longer sums that they
are a part of).
"""
import math
import subprocess
import sys
import threading
from pathlib import Path
from types import SimpleNamespace

import pytest
import torch

import linattn_ref as ref

gpu = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module")
def kda():
    import linear_rnn_delta_b200 as k
    return k


def make(seed, dtype, B, T, Hk, H, dk, dv, cu=None, init=False, per_head=False, rate=1.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    N = B if cu is None else len(cu) - 1
    x = dict(q=r(B, T, Hk, dk).to(dtype), k=r(B, T, Hk, dk).to(dtype), v=r(B, T, H, dv).to(dtype))
    head = rate * torch.exp2(-6 * torch.rand(H, generator=gen))
    x["g"] = -head if per_head else -head * torch.nn.functional.softplus(r(B, T, H))
    x["do"] = r(B, T, H, dv).to(dtype)
    x["s0"] = r(N, H, dk, dv) if init else None
    x["dsf"] = r(N, H, dk, dv) if init else None
    x["cu"] = None if cu is None else torch.tensor(cu, dtype=torch.int32)
    return x


def dev(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def f64(x):
    return {n: None if t is None else (t if n == "cu" else t.to(F64)) for n, t in x.items()}


def near(got, want, size, c, step, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    allow = c * size + step * want.abs() + 1e-30
    worst = ((got - want).abs() / allow).max().item() if got.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the allowance"


STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def allowances(dtype, T, dk, dv):
    scan = (2 * T + max(dk, dv) + 8) * 2.0 ** -24
    return scan, scan + (2.0 ** -16 if dtype == torch.bfloat16 else 0.0)


def pairs(x, q, k, z, r, mag, strong, back=False):
    """Allowance for the weights that the chunked form rounds once."""
    if x["q"].dtype != torch.bfloat16:
        return 0.0
    size = ref.pair_size(q, k, z, r["g"], r["cu"], back)
    if mag.shape[2] != size.shape[2]:   # heads that share an output
        size = size.unflatten(2, (mag.shape[2], -1)).sum(3)
    return 2.0 ** -8 * (size + (mag if strong else 0.0))


def check_fwd(kda, x, flags=0, states=False, strong=False):
    T, dk, dv = x["q"].shape[1], x["q"].shape[3], x["v"].shape[3]
    d, r = dev(x), f64(x)
    got = kda.kda_linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], cu_seqlens=d["cu"], initial_state=d["s0"],
                                    flags=flags, chunk_states=states)
    torch.cuda.synchronize()
    o, sf, S = ref.forward(r["q"], r["k"], r["v"], r["g"], r["cu"], r["s0"])
    mo, msf, mS = ref.forward(r["q"].abs(), r["k"].abs(), r["v"].abs(), r["g"], r["cu"],
                              None if r["s0"] is None else r["s0"].abs())
    c, co = allowances(x["q"].dtype, T, dk, dv)
    near(got[0], o, mo + pairs(x, r["q"], r["k"], r["v"], r, mo, strong) / co, co, STEP[x["q"].dtype], "o")
    near(got[1], sf, msf, c, STEP[torch.float32], "final_state")
    if states:
        for n, (b, lo, hi) in enumerate(ref.spans(T, x["q"].shape[0], x["cu"])):
            row0 = b * T + lo
            for ch in range(-(-(hi - lo) // 64)):
                t = min(hi, lo + 64 * (ch + 1)) - 1
                near(got[2][kda.chunk_slot(n, ch, row0)], S[b, t], mS[b, t], c, STEP[torch.float32],
                     f"state {n} {ch}")
    return got


def check_bwd(kda, x, flags=0, strong=False):
    T, dk, dv = x["q"].shape[1], x["q"].shape[3], x["v"].shape[3]
    d, r = dev(x), f64(x)
    got = kda.kda_linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["dsf"], cu_seqlens=d["cu"],
                                    initial_state=d["s0"], flags=flags)
    torch.cuda.synchronize()
    ab = {n: None if t is None else (t if n in ("cu", "g") else t.abs()) for n, t in r.items()}
    want = ref.backward(r["q"], r["k"], r["v"], r["g"], r["do"], r["dsf"], r["cu"], r["s0"])
    mag = ref.backward(ab["q"], ab["k"], ab["v"], ab["g"], ab["do"], ab["dsf"], ab["cu"], ab["s0"])
    end = None
    if r["dsf"] is not None:
        _, msf, _ = ref.forward(ab["q"], ab["k"], ab["v"], ab["g"], ab["cu"], ab["s0"])
        end = (msf * ab["dsf"]).sum((-1, -2))
    size_g = ref.gate_sum_size(ab["q"], ab["k"], ab["g"], mag if r["g"].dim() > 1 else mag_tokens(mag, r), end, r["cu"])
    c, co = allowances(x["q"].dtype, T, dk, dv)
    step = STEP[x["q"].dtype]
    group = r["v"].shape[2] // r["q"].shape[2]
    qh, kh = (r[n].repeat_interleave(group, dim=2) for n in "qk")
    near(got[0], want.dq, mag.dq + pairs(x, r["do"], r["v"], kh, r, mag.dq, strong) / co, co, step, "dq")
    near(got[1], want.dk, mag.dk + pairs(x, r["do"], r["v"], qh, r, mag.dk, strong, back=True) / co, co, step, "dk")
    near(got[2], want.dv, mag.dv + pairs(x, r["q"], r["k"], r["do"], r, mag.dv, strong, back=True) / co, co, step, "dv")
    near(got[3], want.dg, size_g, c, STEP[torch.float32], "dg")
    near(got[4], want.ds0, mag.ds0, c, STEP[torch.float32], "d_initial_state")
    assert got[0].dtype == x["q"].dtype and got[3].dtype == torch.float32 and got[3].shape == x["g"].shape
    return got


def mag_tokens(mag, r):
    mag.dg = torch.zeros(*r["v"].shape[:3], dtype=F64)
    return mag


CU = [0, 0, 1, 65, 129, 129, 250, 251]
CASES = [  # dtype, B, T, Hk, H, dk, dv, cu, init, per_head
    ("bf16", 1, 1, 1, 1, 128, 128, None, False, False),
    ("bf16", 2, 1, 1, 2, 64, 128, None, True, False),
    ("bf16", 1, 63, 2, 2, 128, 64, None, False, True),
    ("bf16", 2, 64, 1, 3, 64, 64, None, True, False),
    ("bf16", 1, 65, 2, 4, 128, 128, None, True, False),
    ("bf16", 1, 251, 2, 2, 128, 128, CU, True, False),
    ("bf16", 1, 251, 1, 2, 64, 128, CU, False, False),
    ("bf16", 3, 200, 2, 2, 128, 64, None, True, True),
    ("bf16", 1, 130, 3, 3, 16, 32, None, True, False),
    ("bf16", 1, 251, 1, 2, 32, 16, CU, True, False),
    ("bf16", 1, 130, 1, 1, 32, 128, None, True, False),
    ("bf16", 1, 130, 1, 1, 128, 16, None, True, False),
    ("fp32", 1, 1, 1, 1, 16, 16, None, True, False),
    ("fp32", 2, 75, 2, 4, 64, 128, None, True, False),
    ("fp32", 1, 251, 1, 2, 128, 128, CU, True, True),
    ("fp32", 1, 130, 1, 1, 128, 32, None, False, False),
    ("fp32", 1, 70, 2, 2, 32, 64, None, True, False),
]
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def case(c, seed):
    dt, B, T, Hk, H, dk, dv, cu, init, per_head = c
    return make(seed, DT[dt], B, T, Hk, H, dk, dv, cu, init, per_head)


@gpu
@pytest.mark.parametrize("c", CASES, ids=str)
def test_forward(kda, c):
    check_fwd(kda, case(c, 1), states=True)


@gpu
@pytest.mark.parametrize("c", CASES, ids=str)
def test_backward(kda, c):
    check_bwd(kda, case(c, 2))


@gpu
@pytest.mark.parametrize("c", [CASES[4], CASES[5], CASES[7]], ids=str)
def test_token_scan(kda, c):
    check_fwd(kda, case(c, 3), flags=kda.FLAG_FORCE_SCAN, states=True)
    check_bwd(kda, case(c, 3), flags=kda.FLAG_FORCE_SCAN)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [511, 513, 1100])
def test_long_sequences_cross_the_gate_segments(kda, dtype, T):
    x = make(4, DT[dtype], 1, T, 1, 2, 64, 64, init=True, rate=0.2)
    check_fwd(kda, x, states=True)
    check_bwd(kda, x)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_packed_segments(kda, dtype):
    x = make(5, DT[dtype], 1, 1300, 1, 2, 64, 64, cu=[0, 3, 700, 700, 1300], init=True, rate=0.1)
    check_fwd(kda, x, states=True)
    check_bwd(kda, x)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_documents(kda, dtype):
    """1000 documents of 0 to 9 tokens, more than a block's threads and several to a tile."""
    gen = torch.Generator().manual_seed(29)
    cu = [0] + torch.randint(0, 10, (1000,), generator=gen).cumsum(0).tolist()
    x = make(29, DT[dtype], 1, cu[-1], 1, 1, 64, 64, cu=cu, init=True)
    check_fwd(kda, x, states=True)
    check_bwd(kda, x)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 128])
def test_resets_and_extreme_decays(kda, dtype, d):
    """g of -infinity (reset), the lowest number, strong and no decay, next to one another."""
    x = make(6, DT[dtype], 1, 150, 1, 2, d, d, init=True)
    g = x["g"]
    g[0, 0] = -math.inf
    g[0, 10] = -math.inf
    g[0, 11] = -math.inf
    g[0, 40] = torch.finfo(torch.float32).min
    g[0, 41:60] = 0.0
    g[0, 60:70] = -30.0
    g[0, 100] = -200.0
    g[0, 127:129] = -math.inf
    got = check_fwd(kda, x, states=True, strong=True)
    assert torch.isfinite(got[0]).all()
    dg = check_bwd(kda, x, strong=True)[3]
    assert (dg[0, [0, 10, 11, 127, 128]] == 0).all()


@gpu
def test_no_decay_and_total_decay(kda):
    """g = 0 is plain causal linear attention; g = -infinity everywhere leaves each token its own write."""
    for g in (0.0, -math.inf):
        x = make(7, torch.bfloat16, 1, 200, 1, 1, 128, 128, init=True)
        x["g"] = torch.full_like(x["g"], g)
        check_fwd(kda, x, strong=g < 0)
        check_bwd(kda, x, strong=g < 0)


@gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 16), ("fp32", 64)])
def test_values_behind_a_token_do_not_reach_it(kda, dtype, d):
    """NaN and infinities in the tokens behind one, and in the other documents of a batch, leave it as it is."""
    x = make(8, DT[dtype], 1, 300, 1, 2, d, d, cu=[0, 90, 200, 300], init=True)
    d0 = dev(x)
    want, sf = kda.kda_linattn_chunk_fwd(d0["q"], d0["k"], d0["v"], d0["g"], cu_seqlens=d0["cu"], initial_state=d0["s0"])
    for name, bad in (("v", math.nan), ("k", math.nan), ("q", math.nan), ("v", math.inf), ("k", -math.inf)):
        y = dev(x)
        y[name][0, 150:200] = bad
        o, s = kda.kda_linattn_chunk_fwd(y["q"], y["k"], y["v"], y["g"], cu_seqlens=y["cu"], initial_state=y["s0"])
        for part in (slice(0, 150), slice(200, 300)):
            assert torch.equal(o[0, part], want[0, part]), (name, bad, part)
        assert torch.equal(s[0], sf[0]) and torch.equal(s[2], sf[2])
        assert not torch.isfinite(o[0, 150:200].float()).any() or name == "q"
        if name == "q":
            assert torch.isnan(o[0, 150:200].float()).all() and torch.equal(s, sf)


@gpu
@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 128, 128), ("bf16", 64, 128), ("bf16", 32, 64), ("fp32", 64, 64)])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "do"])
def test_neighbours_in_a_tile_stay_apart(kda, dtype, dk, dv, name):
    """NaN in a document whose rows share 64-token tiles with the documents around it leaves their outputs, states
    and gradients as they are."""
    x = make(27, DT[dtype], 1, 300, 1, 2, dk, dv, cu=[0, 90, 190, 300], init=True)
    y = dict(x)
    y[name] = x[name].clone()
    y[name][0, 90:190] = math.nan

    def run(d):
        d = dev(d)
        return (kda.kda_linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], cu_seqlens=d["cu"], initial_state=d["s0"]) +
                kda.kda_linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["dsf"], cu_seqlens=d["cu"],
                                          initial_state=d["s0"]))

    for a, b in zip(run(x), run(y)):
        rows = a.shape[0] != 3
        for part in (slice(0, 90), slice(190, 300)) if rows else (slice(0, 1), slice(2, 3)):
            assert torch.equal(a[0, part], b[0, part]) if rows else torch.equal(a[part], b[part])


@gpu
def test_empty_calls(kda):
    for dtype in (torch.bfloat16, torch.float32):
        x = dev(make(9, dtype, 2, 0, 1, 2, 64, 64, init=True))
        o, sf, st = kda.kda_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["g"], initial_state=x["s0"], chunk_states=True)
        assert o.shape == (2, 0, 2, 64) and torch.equal(sf, x["s0"])
        _, sf = kda.kda_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["g"])
        assert (sf == 0).all()
        dq, dk, dv, dg, ds0 = kda.kda_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], x["dsf"])
        assert dg.shape == (2, 0, 2) and torch.equal(ds0, x["dsf"])
        g = torch.zeros(2, device="cuda") - 0.1
        assert (kda.kda_linattn_chunk_bwd(x["q"], x["k"], x["v"], g, x["do"], x["dsf"])[3] == 0).all()
        cu = torch.zeros(4, dtype=torch.int32, device="cuda")   # three empty documents
        x = dev(make(9, dtype, 1, 0, 1, 2, 64, 64, init=True))
        s0 = torch.randn(3, 2, 64, 64, device="cuda")
        o, sf = kda.kda_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, initial_state=s0)
        assert o.shape == (1, 0, 2, 64) and torch.equal(sf, s0)
        ds0 = kda.kda_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], s0, cu_seqlens=cu, initial_state=s0)[4]
        assert torch.equal(ds0, s0)


@gpu
def test_final_state_may_be_the_initial_state(kda):
    x = dev(make(10, torch.bfloat16, 1, 300, 2, 2, 128, 128, cu=[0, 100, 300], init=True))
    o, sf = kda.kda_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["g"], cu_seqlens=x["cu"], initial_state=x["s0"])
    state = x["s0"].clone()
    o2, s2 = kda.kda_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["g"], cu_seqlens=x["cu"], initial_state=state,
                                       final_state=state)
    assert s2 is state and torch.equal(o, o2) and torch.equal(sf, state)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompt_then_decode_equals_one_sequence(kda, dtype):
    """A prompt through the chunked form and tokens through the decode step give what the whole sequence gives."""
    x = make(11, DT[dtype], 2, 140, 2, 4, 64, 128)
    d, r = dev(x), f64(x)
    cut = 133
    o, state = kda.kda_linattn_chunk_fwd(*(d[n][:, :cut].contiguous() for n in "qkvg"))
    outs = [o]
    for t in range(cut, 140):
        outs.append(kda.kda_linattn_decode_step(*(d[n][:, t].contiguous() for n in "qkvg"), state)[:, None])
    got = torch.cat(outs, 1)
    want, sf, _ = ref.forward(r["q"], r["k"], r["v"], r["g"])
    mo, msf, _ = ref.forward(r["q"].abs(), r["k"].abs(), r["v"].abs(), r["g"])
    c, co = allowances(DT[dtype], 140, 64, 128)
    near(got, want, mo + pairs(x, r["q"], r["k"], r["v"], r, mo, False) / co, co, STEP[DT[dtype]], "o")
    near(state, sf, msf, c, 2.0 ** -24, "state")


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,Hk,H", [(1, 1, 1), (3, 2, 4), (40, 4, 4)])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (128, 16), (32, 64), (64, 32), (64, 64), (128, 128)])
def test_decode_step(kda, dtype, N, Hk, H, dk, dv):
    x = make(12, DT[dtype], N, 1, Hk, H, dk, dv, init=True, per_head=N == 3)
    d, r = dev(x), f64(x)
    state = d["s0"]
    g = d["g"] if N == 3 else d["g"][:, 0].contiguous()
    o = kda.kda_linattn_decode_step(d["q"][:, 0].contiguous(), d["k"][:, 0].contiguous(), d["v"][:, 0].contiguous(), g,
                                    state)
    torch.cuda.synchronize()
    want, sf, _ = ref.forward(r["q"], r["k"], r["v"], r["g"], None, r["s0"])
    mo, msf, _ = ref.forward(r["q"].abs(), r["k"].abs(), r["v"].abs(), r["g"], None, r["s0"].abs())
    c = (dk + 8) * 2.0 ** -24
    near(o, want[:, 0], mo[:, 0], c, STEP[DT[dtype]], "o")
    near(state, sf, msf, c, 2.0 ** -24, "state")


@gpu
def test_autograd_function(kda):
    x = make(13, torch.bfloat16, 1, 130, 1, 2, 64, 64, cu=[0, 50, 130], init=True)
    d = dev(x)
    want = kda.kda_linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["dsf"], cu_seqlens=d["cu"],
                                     initial_state=d["s0"])
    leaves = {n: d[n].requires_grad_() for n in ("q", "k", "v", "g", "s0")}
    o, sf = kda.KdaLinAttnFunction.apply(leaves["q"], leaves["k"], leaves["v"], leaves["g"], d["cu"], leaves["s0"])
    got = torch.autograd.grad([o, sf], list(leaves.values()), [d["do"], d["dsf"]])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    o, _ = kda.KdaLinAttnFunction.apply(leaves["q"], leaves["k"], leaves["v"], leaves["g"], d["cu"], None)
    (o.float() * d["do"].float()).sum().backward()
    want = kda.kda_linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], cu_seqlens=d["cu"])
    assert all(torch.equal(leaves[n].grad, w) for n, w in zip("qkvg", want))
    o, _ = kda.KdaLinAttnFunction.apply(leaves["q"], leaves["k"], leaves["v"], leaves["g"], d["cu"], None)
    first, = torch.autograd.grad((o.float() ** 2).sum(), leaves["q"], create_graph=True)
    with pytest.raises(RuntimeError):   # the gradients have none of their own
        first.float().sum().backward()


def test_reference_gradients_are_differences():
    """The reference's adjoint against central differences of its forward (float64)."""
    x = f64(make(14, torch.float32, 1, 7, 1, 2, 3, 4, cu=[0, 3, 3, 7], init=True))
    names = ("q", "k", "v", "g", "s0")
    loss = lambda y: (lambda o, sf, _: (o * x["do"]).sum() + (sf * x["dsf"]).sum())(  # noqa: E731
        *ref.forward(y["q"], y["k"], y["v"], y["g"], y["cu"], y["s0"]))
    want = ref.backward(x["q"], x["k"], x["v"], x["g"], x["do"], x["dsf"], x["cu"], x["s0"])
    for name, grad in zip(names, (want.dq, want.dk, want.dv, want.dg, want.ds0)):
        flat = x[name].reshape(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 25)):
            old, h = flat[i].item(), 1e-5
            flat[i] = old + h
            up = loss(x)
            flat[i] = old - h
            down = loss(x)
            flat[i] = old
            # the difference's own error: h^2 times a third derivative, and rounding 2^-53 |loss| / h
            assert abs((up - down) / (2 * h) - grad.reshape(-1)[i]) < 1e-7 * (1 + abs(grad.reshape(-1)[i]))


@gpu
def test_graph_replay(kda):
    """A captured forward, backward and decode step replayed on new inputs, twice."""
    x = dev(make(15, torch.bfloat16, 1, 200, 1, 2, 128, 128, init=True))
    y = dev(make(16, torch.bfloat16, 1, 200, 1, 2, 128, 128, init=True))

    def work(s):
        o, sf = kda.kda_linattn_chunk_fwd(s["q"], s["k"], s["v"], s["g"], initial_state=s["s0"])
        od = kda.kda_linattn_decode_step(s["q"][:, -1].contiguous(), s["k"][:, -1].contiguous(),
                                         s["v"][:, -1].contiguous(), s["g"][:, -1].contiguous(), sf)
        return (o, sf, od, *kda.kda_linattn_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], s["dsf"],
                                                      initial_state=s["s0"]))

    want = [t.clone() for t in work(y)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        work(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work(x)
    for _ in range(2):
        for n in x:
            if x[n] is not None:
                x[n].copy_(y[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


FIRST = """
import sys, torch, linear_rnn_delta_b200 as kda
torch.manual_seed(0)
dt, what = getattr(torch, sys.argv[1]), sys.argv[2]
q, k, v, do = [torch.randn(1, 300, 2, 128, device="cuda").to(dt) for _ in range(4)]
g = -0.1 * torch.rand(1, 300, 2, device="cuda")
calls = dict(fwd=lambda: kda.kda_linattn_chunk_fwd(q, k, v, g), bwd=lambda: kda.kda_linattn_chunk_bwd(q, k, v, g, do)[:4],
             step=lambda: [kda.kda_linattn_decode_step(q[0], k[0], v[0], g[0], torch.zeros(300, 2, 128, 128, device="cuda"))])
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls[what]()
graph.replay()
assert all(torch.equal(a, b) for a, b in zip(got, calls[what]()))
"""


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("what", ["fwd", "bwd", "step"])
def test_the_first_call_may_be_captured(dtype, what):
    """In a process that has launched nothing of the library yet."""
    run = subprocess.run([sys.executable, "-c", FIRST, dtype, what], cwd=Path(__file__).parents[1], capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


@gpu
def test_calls_from_threads(kda):
    x = dev(make(28, torch.bfloat16, 1, 300, 2, 2, 128, 128))
    args = (x["q"], x["k"], x["v"], x["g"])
    want = kda.kda_linattn_chunk_fwd(*args) + kda.kda_linattn_chunk_bwd(*args, x["do"])[:4]
    torch.cuda.synchronize()
    wrong = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                got = kda.kda_linattn_chunk_fwd(*args) + kda.kda_linattn_chunk_bwd(*args, x["do"])[:4]
            torch.cuda.current_stream().synchronize()
            wrong.extend(not torch.equal(a, b) for a, b in zip(got, want))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(wrong) == 4 * len(want) and not any(wrong)


@gpu
def test_side_stream(kda):
    x = dev(make(17, torch.bfloat16, 2, 300, 1, 2, 128, 128, init=True))
    want = kda.kda_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["g"], initial_state=x["s0"])
    wantb = kda.kda_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], x["dsf"], initial_state=x["s0"])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(3):   # two calls at once, each with its own workspace
        for s in (s1, s2):
            outs.append((kda.kda_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["g"], initial_state=x["s0"], stream=s),
                         kda.kda_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], x["dsf"],
                                                   initial_state=x["s0"], stream=s.cuda_stream)))
    torch.cuda.synchronize()
    for f, b in outs:
        assert all(torch.equal(p, q) for p, q in zip(f, want)) and all(torch.equal(p, q) for p, q in zip(b, wantb))


@gpu
def test_runs_repeat_bitwise(kda):
    x = dev(make(18, torch.bfloat16, 1, 700, 2, 4, 128, 128, cu=[0, 300, 700], init=True))
    args = (x["q"], x["k"], x["v"], x["g"])
    f = [kda.kda_linattn_chunk_fwd(*args, cu_seqlens=x["cu"], initial_state=x["s0"]) for _ in range(3)]
    b = [kda.kda_linattn_chunk_bwd(*args, x["do"], x["dsf"], cu_seqlens=x["cu"], initial_state=x["s0"])
         for _ in range(3)]
    for r in (f, b):
        assert all(torch.equal(p, q) for o in r[1:] for p, q in zip(o, r[0]))


@gpu
def test_validation_flag(kda):
    x = dev(make(19, torch.float32, 1, 20, 1, 2, 16, 16, cu=[0, 5, 20]))
    args = [x["q"], x["k"], x["v"], x["g"]]
    kda.kda_linattn_chunk_fwd(*args, cu_seqlens=x["cu"], flags=kda.FLAG_VALIDATE_RANGE)
    args[3] = x["g"].clone()
    args[3][0, 3, 1] = -math.inf
    kda.kda_linattn_chunk_fwd(*args, cu_seqlens=x["cu"], flags=kda.FLAG_VALIDATE_RANGE)
    for bad in (0.5, math.nan):
        args[3][0, 3, 1] = bad
        with pytest.raises(kda.KdaError) as e:
            kda.kda_linattn_chunk_fwd(*args, cu_seqlens=x["cu"], flags=kda.FLAG_VALIDATE_RANGE)
        assert e.value.code == 3
        with pytest.raises(kda.KdaError) as e:
            kda.kda_linattn_decode_step(*(t[0].contiguous() for t in args), torch.zeros(20, 2, 16, 16, device="cuda"),
                                        flags=kda.FLAG_VALIDATE_RANGE)
        assert e.value.code == 3
    for cu in ([1, 5, 20], [0, 6, 5, 20], [0, 5, 19]):
        with pytest.raises(kda.KdaError) as e:
            kda.kda_linattn_chunk_fwd(*args[:3], x["g"], flags=kda.FLAG_VALIDATE_RANGE,
                                      cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert e.value.code == 1


CUT = [  # few long sequences, walked in segments side by side: dtype, B, T, Hk, H, dk, dv, cu, init, per_head
    ("bf16", 1, 2177, 1, 2, 64, 64, None, True, False),
    ("bf16", 1, 2048, 1, 1, 128, 128, None, False, False),
    ("bf16", 1, 2049, 1, 1, 64, 128, None, True, True),
    ("bf16", 2, 2111, 1, 1, 128, 64, None, True, False),
    ("bf16", 1, 4500, 1, 2, 64, 64, [0, 3, 3, 2100, 4500], True, False),
    ("bf16", 1, 4500, 1, 1, 64, 64, [0, 4436, 4436, 4500], False, False),
    ("bf16", 1, 2177, 1, 1, 32, 64, None, True, False),
    ("fp32", 1, 2177, 1, 2, 64, 64, None, True, False),
    ("fp32", 1, 2500, 2, 2, 16, 32, [0, 1, 1, 1217, 1281, 2500], True, True),
]


def assert_cut(kda, c):
    dt, B, T, Hk, H, dk, dv, cu = c[:8]
    sizes = (0 if dt == "bf16" else 1, B, T, Hk, H, dk, dv, int(cu is not None), B if cu is None else len(cu) - 1, 0)
    assert kda.lib.kda_linattn_chunk_fwd_workspace_size(*sizes) > 0   # the segments' states


@pytest.mark.parametrize("c", CUT, ids=str)
def test_the_long_cases_are_cut(kda, c):
    assert_cut(kda, c)


@gpu
@pytest.mark.parametrize("c", CUT, ids=str)
def test_cut_sequences(kda, c):
    check_fwd(kda, make(21, *((DT[c[0]],) + c[1:]), rate=0.3), states=True)
    check_bwd(kda, make(22, *((DT[c[0]],) + c[1:]), rate=0.3))


TURNS = [  # segments walked in turn, where (sequence, head) pairs do not fill whole waves of CTAs: B, T, Hk, H, dk, dv,
    # cu, init; forward the first two and the third, backward the others
    (3, 2048, 50, 50, 64, 64, None, True),
    (3, 2047, 25, 50, 128, 64, None, False),
    (1, 10000, 64, 64, 64, 128, [0, 0, 6200, 10000], True),
    (1, 2500, 64, 64, 64, 64, None, True),
    (1, 2500, 40, 80, 64, 128, None, False),
    (1, 12000, 24, 24, 64, 64, [0, 7003, 12000], True),
]


def test_the_many_pairs_are_cut(kda):
    for c in TURNS[:3]:
        assert_cut(kda, ("bf16",) + c)


@gpu
@pytest.mark.parametrize("c", TURNS, ids=str)
def test_segments_in_turn(kda, c):
    """The last key head's value heads of a call with many."""
    B, T, Hk, H, dk, dv, cu, init = c
    x = make(25, torch.bfloat16, B, T, Hk, H, dk, dv, cu, init, rate=0.3)
    d = dev(x)
    fwd = lambda **kw: kda.kda_linattn_chunk_fwd(  # noqa: E731
        d["q"], d["k"], d["v"], d["g"], cu_seqlens=d["cu"], initial_state=d["s0"], chunk_states=True, **kw)
    bwd = lambda **kw: kda.kda_linattn_chunk_bwd(  # noqa: E731
        d["q"], d["k"], d["v"], d["g"], d["do"], d["dsf"], cu_seqlens=d["cu"], initial_state=d["s0"], **kw)
    f, b = fwd(), bwd()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    again = [(fwd(stream=s), bwd(stream=s)) for s in streams]   # three at once, each with its own workspace
    torch.cuda.synchronize()
    for f2, b2 in again:
        assert all(torch.equal(p, q) for p, q in zip(f[:2] + b, f2[:2] + b2))
    hv, hk = slice(H - H // Hk, H), slice(Hk - 1, Hk)
    y = {n: x[n] if x[n] is None or n == "cu" else x[n][:, :, hk] if n in "qk" else x[n][:, hv] if n in ("s0", "dsf")
         else x[n][:, :, hv] for n in x}
    part = (f[0][:, :, hv], f[1][:, hv], f[2][:, hv])
    check_fwd(SimpleNamespace(kda_linattn_chunk_fwd=lambda *a, **kw: part, chunk_slot=kda.chunk_slot), y, states=True)
    part = (b[0][:, :, hk], b[1][:, :, hk], b[2][:, :, hv], b[3][:, :, hv], b[4][:, hv])
    check_bwd(SimpleNamespace(kda_linattn_chunk_bwd=lambda *a, **kw: part), y)


@gpu
def test_segments_in_turn_replayed(kda):
    """Two graphs whose calls share nothing but the inputs, replayed in turn; the state written over in place."""
    x = dev(make(26, torch.bfloat16, 3, 2048, 50, 50, 64, 64, init=True))
    want, sf = kda.kda_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["g"], initial_state=x["s0"])
    state = x["s0"].clone()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, _ = kda.kda_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["g"], initial_state=state, final_state=state)
        graphs.append(graph), outs.append(o)
    for _ in range(2):
        for graph, o in zip(graphs, outs):
            state.copy_(x["s0"]), o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want) and torch.equal(state, sf)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_resets_in_cut_sequences(kda, dtype):
    """Resets at, before and behind the segments' borders (multiples of 64 here), and a whole segment of them."""
    x = make(23, DT[dtype], 1, 2200, 1, 1, 64, 64, init=True, rate=0.2)
    x["g"][0, [63, 64, 255, 256, 257, 1023, 1024, 2047, 2048, 2199]] = -math.inf
    x["g"][0, 512:900] = -math.inf
    x["g"][0, 1200:1500] = 0.0
    x["g"][0, 1600:1700] = -20.0
    check_fwd(kda, x, states=True, strong=True)
    check_bwd(kda, x, strong=True)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_cut_sequences_keep_what_is_behind_apart(kda, dtype):
    """NaN in a token leaves what is before it and the other sequences as they are; the final state may be the
    initial one; two streams and a replayed graph give the same bits."""
    x = make(24, DT[dtype], 1, 4500, 1, 2, 64, 64, cu=[0, 3, 2100, 4500], init=True, rate=0.2)
    d = dev(x)
    run = lambda y, **kw: kda.kda_linattn_chunk_fwd(  # noqa: E731
        y["q"], y["k"], y["v"], y["g"], cu_seqlens=y["cu"], **kw)
    want, sf = run(d, initial_state=d["s0"])
    for name in "kv":
        y = dev(x)
        y[name][0, 1500] = math.nan
        o, s = run(y, initial_state=y["s0"])
        for part in (slice(0, 1500), slice(2100, 4500)):
            assert torch.equal(o[0, part], want[0, part]), name
        assert torch.isnan(o[0, 1500:2100].float()).all() and torch.isnan(s[1]).all()
        assert torch.equal(s[0], sf[0]) and torch.equal(s[2], sf[2])
    state = d["s0"].clone()
    o, s = run(d, initial_state=state, final_state=state)
    assert s is state and torch.equal(o, want) and torch.equal(s, sf)
    torch.cuda.synchronize()
    outs = [run(d, initial_state=d["s0"], stream=st) for st in [torch.cuda.Stream() for _ in range(3)] for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, sf) for a, b in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, s = run(d, initial_state=d["s0"])
    for _ in range(2):
        o.zero_(), s.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(s, sf)


# ---- refusals (CPU) ------------------------------------------------------------------------------------------------

def test_binding_refuses(kda):
    x = make(20, torch.float32, 1, 8, 1, 2, 16, 16)
    args = [x["q"], x["k"], x["v"], x["g"]]
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_linattn_chunk_fwd(*args)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_linattn_chunk_bwd(*args, x["do"])
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_linattn_decode_step(*(t[0] for t in args), torch.zeros(8, 2, 16, 16))
    with pytest.raises(ValueError, match="unsupported"):
        kda.kda_linattn_chunk_fwd(*(t.half() for t in args))
    with pytest.raises(ValueError, match="must be"):
        kda.kda_linattn_chunk_fwd(*(t[0] for t in args))
    with pytest.raises(ValueError, match="multiple"):
        kda.kda_linattn_chunk_fwd(torch.zeros(1, 8, 3, 16), torch.zeros(1, 8, 3, 16), x["v"], x["g"])
    for name in ("kda_linattn_chunk_fwd", "kda_linattn_chunk_bwd", "KdaLinAttnFunction", "kda_linattn_decode_step"):
        assert name in kda.__all__


def test_abi_refuses(kda):
    import ctypes
    lib, P, BAD, ODD = kda.lib, ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)

    def fwd(**kw):
        a = dict(dtype=0, B=1, T=8, Hk=1, H=2, dk=128, dv=128, q=P, k=P, v=P, g=P, per=1, cu=None, n=0, s0=None, sf=None,
                 cs=None, o=P, ws=P, wsb=1 << 40, flags=0)
        a.update(kw)
        return lib.kda_linattn_chunk_fwd(*a.values(), None)

    def bwd(**kw):
        a = dict(dtype=0, B=1, T=8, Hk=1, H=2, dk=128, dv=128, q=P, k=P, v=P, g=P, per=1, cu=None, n=0, s0=None, do=P,
                 dsf=None, dq=P, dk_=P, dv_=P, dg=P, ds0=None, ws=P, wsb=1 << 40, flags=0)
        a.update(kw)
        return lib.kda_linattn_chunk_bwd(*a.values(), None)

    def dec(**kw):
        a = dict(dtype=0, N=4, Hk=1, H=2, dk=128, dv=128, q=P, k=P, v=P, g=P, per=1, state=P, o=P, flags=0)
        a.update(kw)
        return lib.kda_linattn_decode_step(*a.values(), None)

    for f in (fwd, bwd, dec):
        for bad in (dict(dtype=2), dict(Hk=0), dict(Hk=3, H=4), dict(H=0), dict(dk=0), dict(q=None), dict(k=BAD),
                    dict(v=None), dict(g=None), dict(g=ODD), dict(flags=1 << 9), dict(flags=16), dict(flags=32)):
            assert f(**bad) == 1, (f, bad)
        for bad in (dict(dk=48), dict(dv=256)):
            assert f(**bad) == 2, (f, bad)
    for f in (fwd, bwd):
        for bad in (dict(B=0), dict(T=-1), dict(cu=P, n=0), dict(cu=P, n=1, B=2), dict(cu=ctypes.c_void_p(0x10002), n=1),
                    dict(s0=BAD), dict(B=1 << 20, T=1 << 20), dict(ws=BAD)):
            assert f(**bad) == 1, (f, bad)
    assert fwd(o=None) == 1 and fwd(o=BAD) == 1 and fwd(sf=BAD) == 1 and fwd(cs=BAD) == 1
    for bad in (dict(do=None), dict(do=BAD), dict(dsf=BAD), dict(dq=None), dict(dk_=BAD), dict(dv_=None), dict(dg=None), dict(dg=ODD),
                dict(ds0=BAD), dict(ws=None), dict(wsb=64), dict(flags=1), dict(ds0=P, dsf=P), dict(ds0=P, s0=P)):
        assert bwd(**bad) == 1, bad
    assert dec(N=0) == 1 and dec(state=None) == 1 and dec(state=BAD) == 1 and dec(o=None) == 1 and dec(flags=2) == 1
    size = lib.kda_linattn_chunk_bwd_workspace_size
    assert size(0, 1, 8, 1, 2, 128, 128, 0, 0) > 0
    assert size(0, 0, 8, 1, 2, 128, 128, 0, 0) == 0 and size(0, 1, 8, 1, 2, 48, 128, 0, 0) == 0
