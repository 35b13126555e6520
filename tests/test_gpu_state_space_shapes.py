"""The state-space layer at sizes whose loops turn more than once: rows of the scan cut into runs that remember, the
convolution's long runs of tokens, and the norm's CTAs with several slices.  The scan against the fp64 oracle; the other two,
too large for it, against the same formulas in fp64 torch.  Tolerances as in test_gpu_state_space.py."""
from __future__ import annotations

import numpy as np
import pytest

from tests.test_gpu_state_space import DT, FORMS, FP32, W, _ssm_case, _ssm_check, _t   # noqa: F401

pytestmark = pytest.mark.gpu


def _close64(got, ref, dtype, what):
    """As _close, on the device: the largest error beyond the half step of storing, relative to the reference's RMS."""
    import torch
    assert got.shape == ref.shape and bool(got.isfinite().all()), what
    got = got.double()
    d = (got - ref).abs()
    if dtype != "f32":
        top = torch.maximum(got.abs(), ref.abs())
        step = torch.ldexp(torch.ones_like(top), torch.floor(torch.log2(top.clamp(min=1e-300))).int() - (7 if dtype == "bf16" else 10) - 1)
        d = (d - torch.where(top > 0, step, torch.zeros_like(step))).clamp(min=0)
    err = (d.max() / ref.square().mean().sqrt()).item()
    assert err <= FP32, (what, err)


# ------------------------------------------------------------------ scan
@pytest.mark.parametrize("dtype,algo", FORMS)
@pytest.mark.parametrize("reset", (None, "one"))
@pytest.mark.parametrize("H,T,N", ((2, 900, 64), (1, 1021, 128), (3, 769, 128)))
def test_cut_rows_remember(W, monkeypatch, dtype, algo, reset, H, T, N):   # noqa: F811
    """A row cut into runs whose decays leave a good part of the state from end to end, so that s0 reaches the last token and
    dsT the first; or with one reset in a run in the middle.

    The fp32 tolerance counts 512 operations in a chain.  In token order a state that is remembered for T tokens is the end
    of 3 T of them (a decay, its product, a sum), so there the same formula takes 3 T: 3 T * 2^-24 * 3."""
    import torch
    from tests import test_gpu_state_space as base
    if algo == "scan":
        monkeypatch.setattr(base, "FP32", 3 * T * 2.0 ** -24 * 3)
    rng = np.random.default_rng(600 + T)
    dev, ref = _ssm_case(rng, dtype, 1, T, H, 1, N, reset=None, A_scale=1e-3)
    states = 4 * H * (-(-T // 128) + 1) * 64 * N
    desc = W.make_desc(1, T, H, _t(dtype), algo, N=N)
    assert W.lib().wkv7_ssm_workspace_bytes(desc, W.Ssm(1, None, None, None, 1, 0, 0, 0, 0)) >= states + 3 * 4 * H * 64 * N   # three runs at least
    if reset:
        ref["reset"] = np.zeros((1, T), np.uint8)
        ref["reset"][0, T // 2 + 5] = 1
        dev["reset"] = torch.from_numpy(ref["reset"]).cuda()
    else:   # what is left at the end of what the row starts from
        step = np.logaddexp(0.0, ref["dt"] + ref["dt_bias"])
        assert np.exp((step * ref["A"]).sum(1)).min() > 0.05
    _ssm_check(W, rng, dtype, algo, dev, ref)
