"""Linear attention at the edges of its kernels: hand-overs between a CTA's roles, ranges of values and decays,
long segments, waits that run out, gradients as autograd hands them over.

Tolerances and helpers are test_linattn.py's."""
import ctypes
import math
import re
import time

import pytest
import torch

from test_linattn import DT, TURNS, check_bwd, check_fwd, dev, make

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import linear_rnn_delta_b200 as k
    return k


# ---- a strong decay and a value that is not finite in one chunk ----------------------------------------------------

def both(kda, d):
    """Outputs by the name of the value-like operand of the pass that makes them, and which way it runs."""
    o, sf = kda.kda_linattn_chunk_fwd(d["q"], d["k"], d["v"], d["g"], initial_state=d["s0"])
    dq, dk, dv, _, ds0 = kda.kda_linattn_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["dsf"],
                                                   initial_state=d["s0"])
    return {"v": (o, sf, False), "k": (dq, None, False), "q": (dk, None, True), "do": (dv, ds0, True)}


@gpu
@pytest.mark.parametrize("T,chunk", [(64, 0), (128, 0), (128, 1), (150, 0), (150, 1), (192, 1), (192, 2), (640, 8), (640, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_reset_and_bad_value_in_one_chunk(kda, T, chunk, d, bad):
    """Every wait ends, and what does not depend on the bad value keeps its bits: the tokens before it (behind it in
    the passes backward in time) and the other head."""
    x = make(40, torch.bfloat16, 1, T, 2, 2, d, d, init=True)
    t = min(T - 1, 64 * chunk + 40)
    x["g"][0, 64 * chunk + 20] = -math.inf
    x["g"][0, 64 * chunk + 21:64 * chunk + 24] = -60.0
    kda.kda_device_status()
    want = both(kda, dev(x))
    for name in ("v", "k", "q", "do"):
        y = dict(x, **{name: x[name].clone()})
        y[name][0, t, 0] = bad
        out, state, back = both(kda, dev(y))[name]
        out0, state0, _ = want[name]
        keep = slice(t + 1, T) if back else slice(0, t)
        hit = slice(0, t + 1) if back else slice(t, T)
        assert torch.equal(out[0, keep, 0], out0[0, keep, 0]), name
        assert torch.equal(out[0, :, 1], out0[0, :, 1]), name
        assert not torch.isfinite(out[0, hit.stop - 1 if back else hit.start, 0].float()).any(), name
        if state is not None:
            assert torch.equal(state[0, 1], state0[0, 1]) and torch.isnan(state[0, 0]).all()
    assert kda.kda_device_status() == (0, 0)


# ---- waits that run out --------------------------------------------------------------------------------------------

STALLED = dict(B=3, T=4096, Hk=1, H=50, dk=64, dv=64)   # 50 heads of three sequences: four segments each, in turn


def refusal(kda, s, flags, bwd=False, cu=False):
    """Why a call without a workspace is refused (the pointers are never followed)."""
    P = ctypes.c_void_p(0x10000)
    sizes = [0, *s.values()]
    N = cu or s["B"]
    head = [*sizes, P, P, P, P, 1, P if cu else None, N, None]
    if bwd:
        rc = kda.lib.kda_linattn_chunk_bwd(*head, P, None, P, P, P, P, None, None, 0, flags, None)
    else:
        rc = kda.lib.kda_linattn_chunk_fwd(*head, None, None, P, None, 0, flags, None)
    assert rc == 1
    return kda.lib.kda_last_error_detail().decode()


def test_stall_flag_needs_a_wait_to_stall(kda):
    assert "workspace" in refusal(kda, STALLED, kda.FLAG_DEBUG_STALL)
    for s, flags in ((dict(STALLED, B=1, H=1), 0), (dict(STALLED, B=1, H=1, T=8192), 0), (STALLED, kda.FLAG_FORCE_SCAN)):
        assert "in turn" in refusal(kda, s, flags | kda.FLAG_DEBUG_STALL)
    assert "workspace" in refusal(kda, STALLED, kda.FLAG_DEBUG_STALL, bwd=True)
    assert "tensor-core" in refusal(kda, dict(STALLED, dk=32), kda.FLAG_DEBUG_STALL, bwd=True)
    assert "tensor-core" in refusal(kda, STALLED, kda.FLAG_DEBUG_STALL | kda.FLAG_FORCE_SCAN, bwd=True)


@gpu
def test_hand_over_that_never_comes(kda):
    """The segment that waits gives up, hands NaN on and ends; its successors end; nothing else notices."""
    s = STALLED
    x = dev(make(41, torch.bfloat16, s["B"], s["T"], s["Hk"], s["H"], s["dk"], s["dv"], init=True))
    run = lambda flags=0: kda.kda_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["g"], initial_state=x["s0"], flags=flags)  # noqa: E731
    kda.kda_device_status()
    want, sf = run()
    assert kda.kda_device_status() == (0, 0)
    t0 = time.time()
    o, st = run(kda.FLAG_DEBUG_STALL)
    assert kda.kda_device_status() == (5, kda.DEVICE_WAIT_TIMEOUT)
    assert time.time() - t0 < 1.0   # no further wait ran out (each about 2 s)
    assert torch.isnan(st[0, 0]).all() and torch.equal(st[0, 1:], sf[0, 1:]) and torch.equal(st[1:], sf[1:])
    assert torch.equal(o[0, :, 1:], want[0, :, 1:]) and torch.equal(o[1:], want[1:])
    # a segment has 16 or 17 chunks: the first is as it was, behind the second there is NaN
    assert torch.equal(o[0, :1024, 0], want[0, :1024, 0]) and torch.isnan(o[0, 2176:, 0].float()).all()
    o, st = run()
    assert torch.equal(o, want) and torch.equal(st, sf) and kda.kda_device_status() == (0, 0)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_gate_gradient_whose_inputs_never_come(kda, d):
    x = dev(make(42, torch.bfloat16, 2, 150, 1, 2, d, d, init=True))
    run = lambda flags=0: kda.kda_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], x["dsf"],  # noqa: E731
                                                    initial_state=x["s0"], flags=flags)
    kda.kda_device_status()
    want = run()
    assert kda.kda_device_status() == (0, 0)
    t0 = time.time()
    got = run(kda.FLAG_DEBUG_STALL)
    assert kda.kda_device_status() == (5, kda.DEVICE_WAIT_TIMEOUT) and time.time() - t0 < 1.0
    assert all(torch.equal(a, b) for i, (a, b) in enumerate(zip(got, want)) if i != 3)
    dg, dg0 = got[3], want[3]
    assert torch.isnan(dg[0, :64, 0]).all() and torch.equal(dg[0, 64:, 0], dg0[0, 64:, 0])
    assert torch.equal(dg[0, :, 1], dg0[0, :, 1]) and torch.equal(dg[1], dg0[1])
    assert all(torch.equal(a, b) for a, b in zip(run(), want)) and kda.kda_device_status() == (0, 0)


# ---- long segments -------------------------------------------------------------------------------------------------

RESETS = [  # T, H, d; d = 16 takes the token scan.  Segments of more than 148860 tokens
    (450000, 47, 64),
    (600000, 150, 16),
]


@pytest.mark.parametrize("T,H,d", RESETS)
def test_segments_are_long(kda, T, H, d):
    need = int(re.search(r"(\d+) bytes", refusal(kda, dict(B=1, T=T, Hk=1, H=H, dk=d, dv=d), 0)).group(1))
    assert "in turn" in refusal(kda, dict(B=1, T=T, Hk=1, H=H, dk=d, dv=d), kda.FLAG_DEBUG_STALL)
    slots = need // (H * d * d * 4)   # a state each, and one of the sequence: not cut into more than slots - 1
    assert 148860 * (slots - 1) < T


def small_ints(*shape, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)


@gpu
@pytest.mark.parametrize("T,H,d", RESETS)
def test_resets_all_along_a_long_segment(kda, T, H, d):
    """Every token resets: o_t = (q_t . k_t) v_t, in small whole numbers, which every format here holds."""
    q, k, v = small_ints(1, T, 1, d, seed=1), small_ints(1, T, 1, d, seed=2), small_ints(1, T, H, d, seed=3)
    g = torch.full((H,), -math.inf, device="cuda")
    o, sf = kda.kda_linattn_chunk_fwd(q, k, v, g, initial_state=torch.ones(1, H, d, d, device="cuda"))
    for t in range(0, T, 1 << 15):
        part = slice(t, t + (1 << 15))
        want = (q[:, part].float() * k[:, part].float()).sum(-1, keepdim=True) * v[:, part].float()
        assert torch.equal(o[:, part].float(), want), t
    assert torch.equal(sf[0], k[0, -1].float()[:, :, None] * v[0, -1].float()[:, None, :])


@gpu
def test_resets_all_along_a_long_segment_backward(kda):
    """dv_t = (q_t . k_t) do_t, dq_t the sum over the heads of (do_t . v_t) k_t, rounded once."""
    T, H, d = 600000, 75, 16   # two passes of a launch: cut like 150 heads
    q, k = small_ints(1, T, 1, d, seed=1), small_ints(1, T, 1, d, seed=2)
    v, do = small_ints(1, T, H, d, seed=3), small_ints(1, T, H, d, seed=4)
    g = torch.full((H,), -math.inf, device="cuda")
    dq, dk, dv, dg, _ = kda.kda_linattn_chunk_bwd(q, k, v, g, do)
    for t in range(0, T, 1 << 15):
        part = slice(t, t + (1 << 15))
        qk = (q[:, part].float() * k[:, part].float()).sum(-1, keepdim=True)
        dov = (do[:, part].float() * v[:, part].float()).sum((-1, -2))[..., None, None]
        assert torch.equal(dv[:, part].float(), qk * do[:, part].float()), t
        assert torch.equal(dq[:, part], (dov * k[:, part].float()).to(torch.bfloat16)), t
        assert torch.equal(dk[:, part], (dov * q[:, part].float()).to(torch.bfloat16)), t
    assert (dg == 0).all()


# ---- large and small values ----------------------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("fp32", 64)])
@pytest.mark.parametrize("size", [-24, 8, 12, 16])
@pytest.mark.parametrize("decay", ["limit", "little", "strong"])
def test_large_and_small_values(kda, dtype, d, size, decay):
    """Inputs of 2^size; chunks that decay by nearly the 2^-96 up to which the weights are divided by the decay to
    their token, hardly, or further."""
    x = make(43, DT[dtype], 1, 150, 1, 2, d, d, init=True)
    for n in ("q", "k", "v", "do", "s0", "dsf"):
        x[n] = x[n] * 2.0 ** size
    x["g"] = torch.full_like(x["g"], {"limit": -95.9 / 64 * math.log(2), "little": -0.01, "strong": -3.0}[decay])
    check_fwd(kda, x, strong=decay == "strong")
    check_bwd(kda, x, strong=decay == "strong")


# ---- steady decays -------------------------------------------------------------------------------------------------

@gpu
def test_steady_decay_over_a_chunk(kda):
    """A state that decays alone for 64 tokens.  The sum of their logarithms is off by less than 64 * 3 * 2^-33, the
    exponential by two units (2^-22), the product by half of one: at a token's 2^-26, the last place of a logarithm in
    fp32, the first would be 6.6e-7."""
    decays = [-0.9012105464935303, -0.9419410228729248, -0.8910042643547058, -0.9726753234863281,
              -0.9623535871505737, -0.870476245880127, -1.0030840635299683, -0.9521473050117493]
    g = torch.tensor(decays, device="cuda")
    x = torch.zeros(1, 64, 1, 64, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros(1, 64, 8, 64, device="cuda", dtype=torch.bfloat16)
    s0 = 1 + torch.rand(1, 8, 64, 64, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")
    _, sf = kda.kda_linattn_chunk_fwd(x, x, v, g, initial_state=s0)
    want = s0.double() * torch.exp(64 * g.double())[:, None, None]
    bound = 64 * 3 * 2.0 ** -33 * math.log(2) + 2.0 ** -22 + 2.0 ** -24
    assert ((sf.double() / want - 1).abs() <= bound).all()


# ---- autograd ------------------------------------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradients_that_are_parts_of_others(kda, dtype):
    """The gradients of o and of the final state behind an odd number of other values: contiguous, not aligned."""
    x = dev(make(44, DT[dtype], 1, 70, 1, 2, 64, 64, init=True))
    want = kda.kda_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], x["dsf"], initial_state=x["s0"])
    leaves = [x[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "s0")]
    o, sf = kda.KdaLinAttnFunction.apply(*leaves[:4], None, leaves[4])
    pad = lambda t: torch.cat([t.new_ones(1), t.flatten()])  # noqa: E731
    got = torch.autograd.grad([pad(o), pad(sf)], leaves, [pad(x["do"]), pad(x["dsf"])])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
@pytest.mark.parametrize("how", ["decode", "decode o", "prompt", "prompt o", "dequantize"])
def test_a_saved_tensor_that_a_call_writes(kda, how):
    """The backward of an earlier call refuses a state or a value that has been written since, as torch's own do."""
    x = dev(make(45, torch.bfloat16, 1, 1, 2, 2, 64, 64, init=True))
    one = [x[n][:, 0].contiguous() for n in "qkvg"]
    q = x["q"].clone().requires_grad_()
    o, _ = kda.KdaLinAttnFunction.apply(q, x["k"], x["v"], x["g"], None, x["s0"])
    if how == "decode":
        kda.kda_linattn_decode_step(*one, x["s0"])
    elif how == "decode o":
        kda.kda_linattn_decode_step(*one, x["s0"].clone(), o=x["v"][:, 0])
    elif how == "prompt":
        kda.kda_linattn_chunk_fwd(*(x[n] for n in "qkvg"), initial_state=x["s0"], final_state=x["s0"])
    elif how == "prompt o":
        kda.kda_linattn_chunk_fwd(*(x[n].clone() for n in "qkvg"), o=x["v"])
    else:
        codes = torch.zeros(1, 2, 64, 64, dtype=torch.int8, device="cuda")
        kda.kda_state_dequantize(codes, torch.ones(1, 2, 64, device="cuda"), out=x["s0"])
    with pytest.raises(RuntimeError, match="inplace"):
        o.float().sum().backward()


@gpu
def test_writes_in_inference_mode(kda):
    with torch.inference_mode():
        x = dev(make(46, torch.float32, 1, 3, 1, 2, 32, 32, init=True))
        o, st = kda.kda_linattn_chunk_fwd(*(x[n] for n in "qkvg"), initial_state=x["s0"], final_state=x["s0"])
        kda.kda_linattn_decode_step(*(x[n][:, 0].contiguous() for n in "qkvg"), st)
        codes, scales = torch.zeros(1, 2, 32, 32, dtype=torch.int8, device="cuda"), torch.zeros(1, 2, 32, device="cuda")
        kda.kda_state_quantize(st, codes, scales)
        assert kda.kda_state_dequantize(codes, scales, out=x["dsf"]) is x["dsf"]


# ---- which way long calls are cut ----------------------------------------------------------------------------------

def up256(x):
    return -(-x // 256) * 256


def backward_cuts(kda, s, cu):
    """The cuts that give the segments' share of a backward call's workspace: ("in turn" or "side by side", slots)."""
    B, T, Hk, H, dk, dv = s.values()
    rows, N = B * T, cu or B
    total = int(re.search(r"(\d+) bytes", refusal(kda, s, 0, bwd=True, cu=cu)).group(1))
    passes = 3 if dk == dv and H == Hk else 2
    slots = N + -(-rows // 64)
    fixed = 2 * (up256(rows * H * dk * 4) if H != Hk else 0) + 2 * up256(slots * H * dk * dv * 4) + up256(slots * H * 4)
    cuts = set()
    for n in range(N + 1, slots + 1):
        states = passes * up256(n * H * dk * dv * 4)
        if fixed + states + up256(passes * (1 + n) * H * 4) == total:
            cuts.add(("in turn", n))
        if fixed + states + passes * up256(n * H * 4) == total:
            cuts.add(("side by side", n))
    return cuts


@pytest.mark.parametrize("i", range(len(TURNS)))
def test_cases_in_turn_are_in_turn(kda, i):
    """The first three of test_segments_in_turn forward, the others backward."""
    B, T, Hk, H, dk, dv, cu, _ = TURNS[i]
    s, N = dict(B=B, T=T, Hk=Hk, H=H, dk=dk, dv=dv), 0 if cu is None else len(cu) - 1
    if i < 3:
        assert "workspace" in refusal(kda, s, kda.FLAG_DEBUG_STALL, cu=N)
    else:
        (how, slots), = backward_cuts(kda, s, N)
        assert how == "in turn" and slots > 2 * (N or B)


# ---- long waits ----------------------------------------------------------------------------------------------------

LONG_DOC = dict(B=1, T=600000, Hk=1, H=12, dk=64, dv=64)   # 32 documents, all but one of them short


def test_a_long_document_is_walked_in_turn(kda):
    assert "workspace" in refusal(kda, LONG_DOC, kda.FLAG_DEBUG_STALL, cu=32)


def test_no_walk_is_waited_for_longer_than_a_wait_lasts(kda):
    """5.5 us a chunk at the slowest measured: 2^23 tokens are 0.7 s of the 2 s after which a wait gives up."""
    for s, cu in ((LONG_DOC, 32), (STALLED, 0)):
        assert "workspace" in refusal(kda, dict(s, T=1 << 23), kda.FLAG_DEBUG_STALL, cu=cu)
        assert "in turn" in refusal(kda, dict(s, T=(1 << 23) + 1), kda.FLAG_DEBUG_STALL, cu=cu)


@gpu
def test_last_segment_waits_for_a_long_document(kda):
    """Its CTAs all start at once; the last waits for the whole walk before it, some 20 ms.  Every token resets, as
    in test_resets_all_along_a_long_segment."""
    T, H, d = LONG_DOC["T"], LONG_DOC["H"], LONG_DOC["dk"]
    cu = torch.cat([torch.arange(0, 31 * 30, 30), torch.tensor([31 * 30, T])]).to(torch.int32).cuda()
    q, k, v = small_ints(1, T, 1, d, seed=1), small_ints(1, T, 1, d, seed=2), small_ints(1, T, H, d, seed=3)
    g = torch.full((H,), -math.inf, device="cuda")
    kda.kda_device_status()
    o, sf = kda.kda_linattn_chunk_fwd(q, k, v, g, cu_seqlens=cu)
    assert kda.kda_device_status() == (0, 0)
    assert torch.equal(o.float(), (q.float() * k.float()).sum(-1, keepdim=True) * v.float())
    ends = cu[1:].long() - 1
    assert torch.equal(sf, k[0, ends].float()[..., None] * v[0, ends].float()[:, :, None, :])


# ---- streams -------------------------------------------------------------------------------------------------------

CALLS = {
    "prompt": lambda kda, x, s: kda.kda_linattn_chunk_fwd(x["q"], x["k"], x["v"], x["g"], initial_state=x["s0"], stream=s),
    "backward": lambda kda, x, s: kda.kda_linattn_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], x["dsf"],
                                                            initial_state=x["s0"], stream=s),
    "decode": lambda kda, x, s: (kda.kda_linattn_decode_step(x["q1"], x["k1"], x["v1"], x["g1"], x["s0"], stream=s),),
    "dequantize": lambda kda, x, s: (kda.kda_state_dequantize(x["codes"], x["scales"], x["slots"], stream=s),),
}


def stream_inputs():
    x = dev(make(47, torch.bfloat16, 2, 200, 1, 2, 64, 64, init=True))
    x.update({n + "1": x[n][:, 0].contiguous() for n in "qkvg"})
    x["codes"] = torch.randint(-127, 128, (4, 2, 64, 64), dtype=torch.int8, device="cuda")
    x["scales"], x["slots"] = torch.rand(4, 2, 64, device="cuda"), torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    return x


@gpu
@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("raw", [False, True])
def test_tensors_dropped_behind_a_call_on_another_stream(kda, name, raw):
    """Inputs that are dropped while the given stream has yet to come to the call, and outputs that are dropped while
    the current stream has yet to read them, keep their memory until then."""
    x = stream_inputs()
    copy = lambda: {n: t.clone() for n, t in x.items() if t is not None}  # noqa: E731
    want = [t.clone() for t in CALLS[name](kda, copy(), None) if t is not None]
    side = torch.cuda.Stream()
    s = side.cuda_stream if raw else side
    torch.cuda.synchronize()

    y = copy()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)   # some 25 ms
    got = [t for t in CALLS[name](kda, y, s) if t is not None]
    sizes = {t.numel() * t.element_size() for t in y.values()}
    del y
    junk = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)), "inputs"
    del junk, got

    y = copy()
    side.wait_stream(torch.cuda.current_stream())
    got = [t for t in CALLS[name](kda, y, s) if t is not None]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(50_000_000)
    read = [t.clone() for t in got]
    sizes = {t.numel() * t.element_size() for t in got}
    del got
    with torch.cuda.stream(side):
        junk = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(read, want)), "outputs"
    del junk


@gpu
def test_captured_on_a_given_stream(kda):
    x = stream_inputs()
    want = [t.clone() for t in CALLS["prompt"](kda, x, None)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = CALLS["prompt"](kda, x, side)
        torch.cuda.current_stream().wait_stream(side)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
