"""The chunked scan's bf16 outputs are off by their own rounding and no more than fp32 arithmetic beside it.

Bound of an element, beyond the half step (2^-8 of the value) that storing it costs, relative to the sum of its terms'
absolute values (the oracle on absolute values): an operand in two bf16 parts leaves 2^-18, and a term has two such factors at
most; its fp32 factors (the step, the decay as one or two exponentials, their products) are at most eight roundings of
2^-22; the tensor core adds at most 32 steps of 16 terms, each cut at 2^-22 of what it has so far: 2 * 2^-18 + 8 * 2^-22 +
32 * 2^-22 = 1.8e-5, and twice that for what the states carry in from earlier chunks by the same sums: 2^-14 covers it.
An operand in one bf16 part is off by 2^-9 of each term.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import state_space as S
from tests.test_gpu_state_space import W, _dev, _f64, _sizes, _ssm_case   # noqa: F401

pytestmark = pytest.mark.gpu

BOUND = 2.0 ** -14
CASES = {"plain": dict(B=2, T=300, H=4, G=2, N=64), "wide": dict(B=1, T=391, H=6, G=2, N=128),
         "long_memory": dict(B=2, T=260, H=3, G=1, N=128, A_scale=1e-2, reset=None), "one_head": dict(B=1, T=900, H=1, G=1, N=64, A_scale=0.1),
         "many_heads": dict(B=1, T=200, H=24, G=2, N=128)}


def _check(got, ref, size, what):
    got = _f64(got)
    assert np.isfinite(got).all(), what
    worst = np.max((np.abs(got - ref) - np.abs(ref) * 2.0 ** -8) / (np.abs(size) + 1e-30))
    assert worst <= BOUND, (what, worst)


def _case(case):
    rng = np.random.default_rng(400)
    kw = dict(CASES[case])
    dev, ref = _ssm_case(rng, "bf16", **kw)
    return rng, dev, ref


@pytest.mark.parametrize("case", CASES)
def test_outputs_are_rounded_once(W, case):   # noqa: F811
    _, dev, ref = _case(case)
    y, _, _ = W.ssm_forward(**dev, algo="chunked")
    _check(y, S.ssm_forward(**ref)[0], _sizes(ref, True), "y")


@pytest.mark.parametrize("case", CASES)
def test_gradients_are_rounded_once(W, case):   # noqa: F811
    """dx, ddt, and db, dc, whose sums run over the group's heads as well (more steps, each cut alike)."""
    rng, dev, ref = _case(case)
    dy, dy64 = _dev(rng.standard_normal(ref["x"].shape), "bf16")
    ds, ds64 = _dev(rng.standard_normal(ref["s0"].shape).astype(np.float32))
    _, _, ws = W.ssm_forward(**dev, algo="chunked")
    g = W.ssm_backward(dy=dy, workspace=ws, dsT=ds, algo="chunked", **dev)
    go = S.ssm_backward(dy=dy64, dsT=ds64, **ref)
    size = _sizes(ref, True, dy64, ds64)
    for n in ("dx", "ddt", "db", "dc"):
        _check(g[n], go[n], size[n], n)
