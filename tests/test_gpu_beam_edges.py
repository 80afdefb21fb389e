"""GPU checks of the beam step at the edges of what its call allows: ties between rows at every alignment, selections of
many candidates, pools of every family.  Tokens, parents, slots and states exactly; scores as in the parity tests unless
a test says otherwise."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import log
from tests.test_gpu_beam import draw, make_pool, run

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("V,pitch", [(32003, 32003), (9001, 9001), (9001, 9007), (20000, 20001), (8192, 8193), (8191, 8191),
                                     (77, 77), (5, 5)])
def test_equal_rows_tie_at_every_alignment(V, pitch, dt):
    """Equal rows with equal scores have equal candidates, whatever their distance from 16 bytes: the lowest beams come
    first.  An odd row pitch puts the beams of a request at all the offsets that the type has."""
    log(f"case: beam equal rows V={V} pitch={pitch} {dt}")
    B, K = 3, 9
    for seed in range(3):
        _, x, scores, slots = draw(200 + seed, B, K, V, dt)
        buf = torch.full((B * K, pitch), 60.0, dtype=dt, device="cuda")     # what lies between rows is not read
        rows = buf[:, :V].unflatten(0, (B, K))
        rows.copy_(x[:, :1].expand(B, K, V))
        run(rows, np.full((B, K), -1.25), slots)
        run(rows, np.repeat(scores[:, :1], K, axis=1).astype(np.float32), slots)


def test_log_sum_exp_of_usual_rows():
    """The log-sum-exp to 2e-8.  A score that the best logit brings back to about 0 shows it with many more digits than
    fp32 has there.  Roundings of a term's argument (|arg| of 4 to 8: half a step is 2^-22, times ln 2 and 1/sqrt(3):
    1e-7), of its exponential (rms 3e-8) and of its sums (6e-8) are independent from term to term: 1.2e-7 over the root of
    the about 131072 e^-4 = 2400 terms that count is 2.5e-9, six times that 1.5e-8; the exponential's mean error is 3e-9.
    A constant log2 e rounded to fp32 would push every term the same way: 1.3e-8 |x - max| of it, 5e-8 here."""
    log("case: beam log-sum-exp")
    n, V = 24, 131072
    g = torch.Generator(device="cuda")
    g.manual_seed(300)
    x = 2.0 * torch.randn((n, 1, V), generator=g, device="cuda")
    wide = x[:, 0].double()
    top = wide.max(dim=1).values
    lse = top + torch.log(torch.exp(wide - top[:, None]).sum(dim=1))
    scores = (lse - top).float()
    i32 = lambda: torch.zeros(n, dtype=torch.int32, device="cuda")
    out, slots = torch.zeros(n, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    make_pool(n).beam_step(x, scores, slots, i32(), i32(), out, i32())
    err = (out.double() - (scores.double() + (top - lse))).abs().max().item()
    log(f"  log-sum-exp off by {err:.1e}")
    assert err <= 2e-8
