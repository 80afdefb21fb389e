"""CPU checks of the rounded chunk form that the GPU prefill's error is held against."""
import numpy as np
import pytest

from oracle import gdn as orc
from oracle.mamba2 import round_to
from recurrent_state_update_amd import synth
from tests import gdn_roundings


def case(shape, T):
    rng = np.random.default_rng(1)
    Hk, Hv, dk, dv = shape
    cd = 2 * Hk * dk + Hv * dv
    ex = lambda v, t="f32": synth.cast_exact(v, t).astype(np.float64)
    params = dict(A=ex(-np.exp(rng.uniform(0, np.log(16), Hv))), dt_bias=ex(rng.uniform(-4, -2, Hv)),
                  conv_w=ex(rng.uniform(-0.5, 0.5, (cd, 4))), conv_b=ex(rng.uniform(-0.5, 0.5, cd)))
    rows = [ex(rng.normal(0, 1, (T, n)), "bf16") for n in (cd, Hv, Hv)]
    ssm = np.zeros((1, Hv, dv, dk))
    ref = orc.prefill(shape, ssm, np.zeros((1, cd, 3)), params, np.array([0, T]), [0], [0], None, *rows)
    return params, rows, ref, ssm[0]


def test_without_roundings_it_is_the_recurrence():
    shape = (1, 2, 32, 16)
    params, rows, ref, state = case(shape, 150)
    o, S = gdn_roundings.prefill(shape, params, *rows, operand=lambda x: x)
    assert np.allclose(o, ref, rtol=0, atol=1e-12 * np.abs(ref).max())
    assert np.array_equal(round_to(S, "bf16"), state) or gdn_roundings.norm_of_error(S, state) <= 2.0 ** -8


@pytest.mark.parametrize("shape", [(2, 4, 128, 64), (2, 4, 64, 48), (1, 2, 256, 48)], ids=str)
def test_a_coarser_operand_shows(shape):
    """What 5% above the fp16 form's error lets through: none of the operands that weigh, in bf16."""
    params, rows, ref, state = case(shape, 500)
    error = lambda x: [gdn_roundings.norm_of_error(round_to(y, "bf16"), want) for y, want in zip(x, (ref, state))]
    fine = error(gdn_roundings.prefill(shape, params, *rows))
    assert 1.6e-3 < fine[0] < 1.05 * gdn_roundings.norm_of_error(round_to(ref, "bf16"), ref) and fine[1] < 1.3e-3
    for name, out in (("K", 0), ("Q", 0), ("A", 0), ("U", 0), ("K", 1), ("R", 1), ("W", 1)):
        coarse = error(gdn_roundings.prefill(shape, params, *rows, coarse=(name,)))
        assert coarse[out] > 1.1 * fine[out], (name, out, coarse, fine)
