"""The quantised state cache: codes, scales and values against the definition in exact arithmetic.

A code is a whole number and has to be the exact quotient's nearest (ties to even); scales and values are fp32
results of one rounding each, 2^-24 relative."""
import ctypes
import math

import pytest
import torch

gpu = pytest.mark.gpu
FMT = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}


@pytest.fixture(scope="module")
def kda():
    import linear_rnn_delta_b200 as k
    return k


def code_values(fmt):
    """Magnitudes of the codes 0, 1, 2, ..."""
    if fmt == "int8":
        return torch.arange(128).double()
    return torch.arange(127).to(torch.uint8).view(torch.float8_e4m3fn).double()


def expected(x, fmt):
    """(signed code values, scales) of fp32 rows, in 64 bits; the products compared are exact there."""
    vals = code_values(fmt)
    top = vals[-1]
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    mid = (vals[1:] + vals[:-1]) / 2
    # number of borders below x top / amax; on a border the even code
    num, den = (x.abs() * top)[..., None], amax[..., None]
    below = (mid * den < num).sum(-1)
    on = (mid * den == num).any(-1) & (amax > 0)
    code = below + (on & (below % 2 == 1))
    code = torch.where(amax > 0, code, 0)
    return vals[code] * torch.sign(x), (amax / top)[..., 0]


def cache(S, H, dk, dv, fmt):
    codes = torch.full((S, H, dk, dv), 7, dtype=torch.int8, device="cuda").view(FMT[fmt][0])
    return codes, torch.full((S, H, dk), 0.5, device="cuda")


def check(kda, x, fmt, slots=None, S=None):
    M, H, dk, dv = x.shape
    S = S or M
    codes, scales = cache(S, H, dk, dv, fmt)
    kda.kda_state_quantize(x.cuda(), codes, scales, None if slots is None else slots.cuda())
    back = kda.kda_state_dequantize(codes, scales, None if slots is None else slots.cuda())
    at = torch.arange(M) if slots is None else slots.long()
    want, wscale = expected(x, fmt)
    got = codes.cpu().view(torch.int8)[at] if fmt == "int8" else codes.cpu().view(torch.int8)[at].view(codes.dtype)
    assert torch.equal(got.double(), want)
    s = scales.cpu()[at]
    assert ((s.double() - wscale).abs() <= 2.0 ** -24 * wscale + 2.0 ** -150).all()
    assert torch.equal(back.cpu(), (got.float() * s[..., None]))
    return codes, scales


@gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("M,H,dk,dv", [(1, 1, 16, 16), (3, 2, 32, 64), (5, 3, 64, 32), (2, 4, 128, 128), (7, 1, 16, 128)])
def test_round_trip(kda, fmt, M, H, dk, dv):
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(M, H, dk, dv, generator=gen) * torch.exp(3 * torch.randn(M, H, dk, 1, generator=gen))
    x[0, 0, 3] = 0
    slots = torch.randperm(M + 4, generator=gen)[:M].to(torch.int32)
    codes, scales = check(kda, x, fmt, slots, M + 4)
    rest = [s for s in range(M + 4) if s not in slots.tolist()]   # what no entry names stays
    assert (codes.view(torch.int8)[rest] == 7).all() and (scales[rest] == 0.5).all()
    check(kda, x, fmt)


@gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("amax", [1.0, 127.0, 448.0, 3.0, 1e-38, 1e-44, 3e38, 0.1])
def test_values_on_and_next_to_the_borders(kda, fmt, amax):
    """Every border of the format times amax / top, its neighbours in fp32, and the row's maximum."""
    vals = code_values(fmt)
    mid = (vals[1:] + vals[:-1]) / 2 * float(torch.tensor(amax)) / vals[-1]
    b = mid.float()
    up, down = torch.nextafter(b, torch.tensor(math.inf)), torch.nextafter(b, torch.tensor(-math.inf))
    x = torch.cat([b, up, down, -b, -up, -down])
    rows = -(-x.numel() // 15)
    pad = torch.zeros(rows * 15)
    pad[:x.numel()] = x
    pad = pad.clamp(-amax, amax).reshape(rows, 15)
    x = torch.cat([torch.full((rows, 1), amax), pad], 1)
    n = -(-rows // 16) * 16
    full = torch.zeros(n, 16)
    full[:rows] = x
    check(kda, full.reshape(1, n // 16, 16, 16), fmt)


@gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_up_to_the_largest_value(kda, fmt):
    """They read back finite, within a unit of the scale's last place and half a code (the smallest code of e4m3 is
    TOP / 229376, its largest step TOP / 14)."""
    most = torch.finfo(torch.float32).max
    x = torch.randn(1, 1, 32, 16, generator=torch.Generator().manual_seed(5)).clamp(-1, 1) * most
    x[0, 0, :, 3] = most
    x[0, 0, 1, 3] = -most
    x[0, 0, 2, 3] = torch.nextafter(torch.tensor(most), torch.tensor(0.0))
    x[0, 0, 3] = most
    codes, scales = cache(1, 1, 32, 16, fmt)
    kda.kda_state_quantize(x.cuda(), codes, scales)
    back = kda.kda_state_dequantize(codes, scales).cpu().double()
    assert torch.isfinite(back).all() and torch.isfinite(scales).all()
    half = most / 254 if fmt == "int8" else x.double().abs() * 2.0 ** -4 + most / 448 * 2.0 ** -10
    assert ((back - x.double()).abs() <= half * (1 + 2.0 ** -20) + 2.0 ** -22 * x.double().abs()).all()


@gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_that_are_not_finite(kda, fmt):
    x = torch.randn(2, 2, 16, 32, generator=torch.Generator().manual_seed(2))
    x[0, 0, 1, 5] = math.nan
    x[0, 1, 2, 31] = math.inf
    x[1, 1, 15, 0] = -math.inf
    codes, scales = cache(2, 2, 16, 32, fmt)
    kda.kda_state_quantize(x.cuda(), codes, scales)
    back = kda.kda_state_dequantize(codes, scales).cpu()
    bad = ~torch.isfinite(x).all(-1)
    assert torch.isnan(back[bad]).all() and torch.isfinite(back[~bad]).all()
    assert torch.isnan(scales.cpu()[bad]).all()


@gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_indices(kda, fmt):
    """Skipped entries, several entries for one slot (the last one wins), indices that are too large."""
    x = torch.randn(6, 2, 16, 64, generator=torch.Generator().manual_seed(3))
    codes, scales = cache(5, 2, 16, 64, fmt)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    assert kda.kda_device_status()[0] == 0
    kda.kda_state_quantize(x.cuda(), codes, scales, i32(2, -1, 0, 2, 2, 0), rows=i32(0, 1, 2, 3, 4, -7))
    assert kda.kda_device_status() == (0, 0)
    back = kda.kda_state_dequantize(codes, scales, i32(2, 0, -3)).cpu()
    for got, row in ((back[0], x[4]), (back[1], x[2])):
        want, s = expected(row[None], fmt)
        assert ((got.double() - (want * s[..., None])[0]).abs() <= 2.0 ** -22 * row.abs().max()).all()
    assert (back[2] == 0).all()
    assert (codes.view(torch.int8)[[1, 3, 4]] == 7).all() and (scales[[1, 3, 4]] == 0.5).all()
    before = codes.clone().view(torch.int8), scales.clone()
    kda.kda_state_quantize(x.cuda(), codes, scales, i32(5, 3), rows=i32(0, 6))
    code, bits = kda.kda_device_status()
    assert code == 5 and bits == kda.DEVICE_BAD_INDEX
    assert torch.equal(codes.view(torch.int8), before[0]) and torch.equal(scales, before[1])
    back = kda.kda_state_dequantize(codes, scales, i32(5, 2))
    assert torch.isnan(back[0]).all() and torch.isfinite(back[1]).all()
    assert kda.kda_device_status() == (5, kda.DEVICE_BAD_INDEX) and kda.kda_device_status() == (0, 0)


@gpu
def test_empty_index(kda):
    x = torch.randn(2, 1, 16, 16).cuda()
    codes, scales = cache(2, 1, 16, 16, "int8")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    kda.kda_state_quantize(x, codes, scales, none)
    assert kda.kda_state_dequantize(codes, scales, none).shape == (0, 1, 16, 16)
    assert (codes == 7).all()


@gpu
def test_offsets_beyond_32_bits(kda):
    """A cache of more than 2^32 codes: the last slots are reached."""
    S, H, dk, dv = 8200, 32, 128, 128
    codes = torch.zeros(S, H, dk, dv, dtype=torch.int8, device="cuda")
    scales = torch.zeros(S, H, dk, device="cuda")
    x = torch.randn(2, H, dk, dv, generator=torch.Generator().manual_seed(4))
    slots = torch.tensor([S - 1, 4], dtype=torch.int32, device="cuda")
    kda.kda_state_quantize(x.cuda(), codes, scales, slots)
    back = kda.kda_state_dequantize(codes, scales, slots).cpu()
    want, s = expected(x[:, :2], "int8")
    assert ((back[:, :2].double() - want * s[..., None]).abs() <= 2.0 ** -22 * x.abs().max()).all()
    assert int((codes[5:S - 1] != 0).any()) == 0


@gpu
def test_prompt_snapshots_through_the_cache(kda):
    """Used together: a prompt's snapshots are parked, one is taken up again, the rest of the prompt and a decode
    step run from it.  The int8 step is amax / 254 of each row at most, and what follows is linear in the state:
    the outputs may be off by what that much state gives, found by running the magnitudes."""
    gen = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    B, T, H, d = 1, 192, 2, 64
    q, k, v = r(B, T, H, d), r(B, T, H, d), r(B, T, H, d)
    g = -0.05 * r(B, T, H).abs()
    o, sf, snaps = kda.kda_linattn_chunk_fwd(q, k, v, g, chunk_states=True)
    codes = torch.zeros(4, H, d, d, dtype=torch.int8, device="cuda")
    scales = torch.zeros(4, H, d, device="cuda")
    row = kda.chunk_slot(0, 1, 0)   # after 128 tokens
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kda.kda_state_quantize(snaps, codes, scales, i32(3), rows=i32(row))
    s0 = kda.kda_state_dequantize(codes, scales, i32(3))
    off = (s0 - snaps[row][None]).abs()
    assert (off <= snaps[row].abs().amax(-1)[None, ..., None] / 254 * (1 + 2.0 ** -20)).all()
    rest = [x[:, 128:].contiguous() for x in (q, k, v, g)]
    o2, sf2 = kda.kda_linattn_chunk_fwd(*rest, initial_state=s0)
    zero = torch.zeros_like(rest[2])
    allow, allow_s = kda.kda_linattn_chunk_fwd(rest[0].abs(), rest[1], zero, rest[3], initial_state=off)
    slack = 1e-4 * (1 + o[:, 128:].abs().max())
    assert ((o2 - o[:, 128:]).abs() <= allow + slack).all()
    assert ((sf2 - sf).abs() <= allow_s + slack).all()
    # the same snapshot resumes the delta-rule forward as well
    od, _ = kda.kda_chunk_fwd("kda", "standard", rest[0], torch.nn.functional.normalize(rest[1], dim=-1), rest[2],
                              torch.full_like(rest[0], 0.9), torch.full_like(rest[3], 0.5), initial_state=s0)
    assert torch.isfinite(od).all()


# ---- refusals (CPU) ------------------------------------------------------------------------------------------------

def test_binding_refuses(kda):
    x, codes, scales = torch.zeros(2, 1, 16, 16), torch.zeros(2, 1, 16, 16, dtype=torch.int8), torch.zeros(2, 1, 16)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_state_quantize(x, codes, scales)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_state_dequantize(codes, scales)
    with pytest.raises(ValueError, match="int8 or float8"):
        kda.kda_state_dequantize(codes.float(), scales)
    with pytest.raises(ValueError, match="must be"):
        kda.kda_state_quantize(x[0], codes, scales)
    for name in ("kda_state_quantize", "kda_state_dequantize", "CACHE_FORMATS"):
        assert name in kda.__all__


def test_abi_refuses(kda):
    lib, P, BAD, ODD = kda.lib, ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)

    def quant(**kw):
        a = dict(fmt=0, n=2, M=2, S=2, H=1, dk=16, dv=16, states=P, rows=None, slots=None, codes=P, scales=P)
        a.update(kw)
        return lib.kda_state_quantize(*a.values(), None)

    def dequant(**kw):
        a = dict(fmt=0, n=2, S=2, H=1, dk=16, dv=16, codes=P, scales=P, slots=None, states=P)
        a.update(kw)
        return lib.kda_state_dequantize(*a.values(), None)

    for f in (quant, dequant):
        for bad in (dict(fmt=2), dict(n=-1), dict(S=0), dict(H=0), dict(dk=0), dict(n=3), dict(codes=None),
                    dict(codes=BAD), dict(scales=None), dict(states=None), dict(states=BAD), dict(slots=ODD),
                    dict(n=1 << 20, H=1 << 20, slots=P, rows=P) if f is quant else dict(n=1 << 20, H=1 << 20, slots=P)):
            assert f(**bad) == 1, (f, bad)
        assert f(dk=48) == 2 and f(dv=256) == 2
    assert quant(M=0) == 1 and quant(rows=ODD) == 1 and quant(n=3, S=9) == 1
