"""GPU checks of the beam step at the edges of what its call allows: ties between rows at every alignment, selections of
many candidates, pools of every family.  Tokens, parents, slots and states exactly; scores as in the parity tests unless
a test says otherwise."""
import numpy as np
import pytest
import torch

from recurrent_state_update_amd.pool import Pool
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


@pytest.mark.parametrize("dt", DTYPES, ids=str)
@pytest.mark.parametrize("B,K,V", [(1, 32, 40001), (2, 32, 131072), (1, 20, 100003), (1, 32, 32768)])
def test_more_candidates_than_are_held(B, K, V, dt):
    """ceil(V / 8192) K^2 candidates of a request: above 4096 their scores are worked out twice."""
    log(f"case: beam candidates {B}x{K} vocab {V} {dt}")
    _, logits, scores, slots = draw(400 + K + V, B, K, V, dt)
    run(logits, scores, slots)
    fin = np.zeros((B, K), np.uint8)
    fin[:, 1::3] = 1
    run(logits, scores, slots, finished=fin, eos=V - 1, in_place=True)


@pytest.mark.parametrize("V", [9000, 32768, 40001], ids=lambda v: f"V{v}")
def test_more_ties_than_the_list_holds(V):
    """Constant rows and equal scores: all candidates tie (2048, 4096 and 5120 of them, held or not)."""
    log(f"case: beam ties of all candidates V={V}")
    K = 32
    for dt in DTYPES:
        logits, scores = torch.zeros((2, K, V), dtype=dt, device="cuda"), np.full((2, K), -1.25)
        logits[1] = 7.0
        slots = np.arange(2 * K).reshape(2, K)
        run(logits, scores, slots)
        scores[:, :5] = -9.0                          # the lowest beams are not the best
        logits[:, 7] = -torch.inf                     # nor has every beam a candidate
        run(logits, scores, slots, finished=(np.arange(2 * K).reshape(2, K) == 9).astype(np.uint8), eos=3)


@pytest.mark.parametrize("V", [9000, 40001], ids=lambda v: f"V{v}")
def test_ties_of_several_scores_within_the_threshold(V):
    """Over 1024 candidates whose scores share their upper 32 bits but are not all equal: beam 20 has three tokens a
    little above the ties of beams 2 and up, which come next, the lowest first; beams 0 and 1 lie a little below."""
    log(f"case: beam nearly equal candidates V={V}")
    K, dt = 32, torch.float32
    logits = torch.zeros((1, K, V), dtype=dt, device="cuda")
    scores = np.full((1, K), np.float32(-1.25), np.float32)
    scores[0, :2] = np.nextafter(np.float32(-1.25), np.float32(-2))
    logits[0, 20] = -torch.inf
    logits[0, 20, [5, V // 2, V - 1]] = 3.0
    tie = np.float64(scores[0, 2]) - np.log(V)
    upper = lambda v: int(np.float64(v).view(np.uint64)) >> 32
    s = np.float32(tie + np.log(3.0))
    while np.float64(s) - np.log(3.0) <= tie:
        s = np.nextafter(s, np.float32(0))
    scores[0, 20] = s
    assert upper(np.float64(s) - np.log(3.0)) == upper(tie) == upper(np.float64(scores[0, 0]) - np.log(V))
    tok, par = run(logits, scores, np.arange(K).reshape(1, K))
    assert par.tolist() == [20] * 3 + [2] * (K - 3) and tok.tolist() == [5, V // 2, V - 1] + list(range(K - 3))


@pytest.mark.parametrize("family", ["mamba2 f32", "mamba2 bf16", "mamba1", "kda"])
def test_pools_of_every_family(family):
    """Selection and copies on the other families' pools, on a stream of its own."""
    log(f"case: beam pool {family}")
    f32, bf16 = torch.float32, torch.bfloat16
    pool = {"mamba2 f32": lambda: Pool.allocate(3, 14, 4, 16, 32, 2, 4, f32, f32),
            "mamba2 bf16": lambda: Pool.allocate(1, 14, 4, 16, 32, 2, 4, bf16, bf16),
            "mamba1": lambda: Pool.allocate_mamba1(2, 14, 64, 16, 4),
            "kda": lambda: Pool.allocate_kda(2, 14, 2, 32, 4)}[family]()
    g = torch.Generator(device="cuda")
    g.manual_seed(14)
    for t in (pool.ssm, pool.conv):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    _, logits, scores, slots = draw(500, 3, 4, 3001, f32)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        run(logits, scores, slots, pool=pool)
        run(logits, scores, slots, pool=pool, in_place=True)


def test_logits_past_32_bit_offsets():
    """16400 rows of 131075 bf16 logits, over 2^31 elements: the last requests as in a call of their own."""
    log("case: beam far logits")
    B, K, V, tail = 2050, 8, 131075, 3
    n, m = B * K, tail * K
    g = torch.Generator(device="cuda")
    g.manual_seed(600)
    logits = torch.empty((B, K, V), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    scores = -3.0 * torch.rand(n, generator=g, device="cuda")
    i32 = lambda c: torch.zeros(c, dtype=torch.int32, device="cuda")
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    pool = Pool.allocate_gdn(1, n, 1, 16, 32, 1, 4)
    got = [i32(n), i32(n), torch.zeros(n, device="cuda"), i32(n)]
    want = [i32(m), i32(m), torch.zeros(m, device="cuda"), i32(m)]
    pool.beam_step(logits, scores, slots, *got)
    pool.beam_step(logits[-tail:], scores[-m:].clone(), slots[-m:].clone(), *want)
    torch.cuda.synchronize()
    assert all(torch.equal(x[-m:], y) for x, y in zip(got, want))
    best = logits[-1].double().log_softmax(-1) + scores[-K:].double()[:, None]
    assert [int(got[1][n - K]), int(got[0][n - K])] == list(divmod(int(best.argmax()), V))
