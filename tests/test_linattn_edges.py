"""Linear attention at the edges of its kernels: hand-overs between a CTA's roles, ranges of values and decays,
long segments, waits that run out, gradients as autograd hands them over.

Tolerances and helpers are test_linattn.py's."""
import math

import pytest
import torch

from test_linattn import dev, make

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
