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
