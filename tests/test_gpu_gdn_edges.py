"""GPU checks of the gated delta rule at the edges of what its calls allow: rows that are not finite, forms and sizes
that the parity tests do not reach, views of one row.  Tolerances are those of the parity tests unless a test says
otherwise."""
import numpy as np
import pytest
import torch

from oracle import gdn as orc
from oracle.mamba2 import round_to
from recurrent_state_update_amd.pool import Pool
from tests import gdn_roundings
from tests.gpu_helpers import dev, host, log
from tests.test_gpu_gdn import LENS, SHAPES, Layer, near, run_prefill

pytestmark = pytest.mark.gpu


def same(got, want):
    """Bit for bit (one NaN is as good as another)."""
    kind = torch.int16 if got.element_size() == 2 else torch.int32
    return torch.equal(got.contiguous().view(kind), want.contiguous().view(kind))


@pytest.mark.parametrize("shape,io", [((2, 4, 64, 48), "bf16"), ((2, 4, 64, 48), "f32"), ((1, 2, 256, 32), "bf16"),
                                      ((1, 2, 256, 32), "f32")], ids=str)
@pytest.mark.parametrize("what", ["q", "k", "v", "a", "b"])
def test_rows_behind_a_checkpoint_leave_it_as_it_is(shape, io, what):
    """A NaN or an infinity in the row right behind a checkpoint that ends a chunk early: the checkpoint's state and
    window and the outputs up to it are those of a clean prompt, bit for bit; the next checkpoint's are not."""
    log(f"case: gdn rows behind a checkpoint {shape} io={io} {what}")
    T, iv = 100, 37                                   # checkpoints behind rows 36 and 73; chunks end at 37, 64, 74, 100
    for bad in (float("nan"), float("inf")):
        kept = []
        for spoil in (False, True):
            L = Layer(shape, 4, 4, 161)
            L.seed_slots([1])
            u, a, b = (dev(x, io) for x in L.rows(T, io))
            q, k, v = L.pool.split_qkv(u)
            if spoil:
                dict(q=q, k=k, v=v, a=a, b=b)[what][iv:iv + 2] = bad
            o = L.out(T, io)
            L.pool.gdn_prefill(0, L.w, [0, T], [1], [1], q, k, v, a, b, o, ckpt_interval=iv, ckpt_slots=[[2, 3]])
            torch.cuda.synchronize()
            kept.append((o, L.pool.ssm[0, 2].clone(), L.pool.conv[0, 2].clone(), L.pool.ssm[0, 3].clone()))
        clean, spoiled = kept
        assert same(spoiled[0][:iv], clean[0][:iv])
        assert same(spoiled[1], clean[1]) and same(spoiled[2], clean[2])
        assert torch.isfinite(clean[3].float()).all()
        if what in "kv":                              # what a row writes into the state
            assert not torch.isfinite(spoiled[3].float()).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_a_single_row_may_have_any_pitch(io):
    """One row of a projection [q | k | v | a | b] whose pitch is no multiple of 16 bytes: its stride is never used."""
    log(f"case: gdn single row of an odd pitch io={io}")
    shape = (1, 3, 32, 16)
    for call in ("decode", "multi", "prefill"):
        kept = []
        for packed in (False, True):
            L = Layer(shape, 4, 4, 171)
            L.seed_slots([1])
            u, a, b = (dev(x, io) for x in L.rows(1, io))
            if packed:
                wide = torch.cat([u, a, b], dim=1)                       # cd + 6 values
                assert wide.stride(0) * wide.element_size() % 16 != 0 and wide.data_ptr() % 16 == 0
                u, a, b = wide[:, :L.cd], wide[:, L.cd:L.cd + 3], wide[:, L.cd + 3:]
            q, k, v = L.pool.split_qkv(u)
            o = L.out(1, io)
            slot = torch.tensor([1], dtype=torch.int32, device="cuda")
            if call == "decode":
                L.pool.gdn_decode_step(0, L.w, slot, q, k, v, a, b, o)
            elif call == "multi":
                L.pool.gdn_decode_multi(0, L.w, slot, slot.view(1, 1) + 1, q, k, v, a, b, o)
            else:
                L.pool.gdn_prefill(0, L.w, [0, 1], [1], [1], q, k, v, a, b, o)
            torch.cuda.synchronize()
            kept.append((o, L.pool.ssm.clone(), L.pool.conv.clone()))
        assert all(same(x, y) for x, y in zip(*kept)), call


def test_calls_without_rows():
    """No sequence, or only empty ones: taken, and nothing is touched."""
    log("case: gdn calls without rows")
    L = Layer((1, 3, 32, 16), 4, 4, 181)
    L.seed_slots([1, 2])
    u, a, b = (dev(x, "bf16") for x in L.rows(0, "bf16"))
    q, k, v = L.pool.split_qkv(u)
    o, none = L.out(0, "bf16"), torch.zeros(0, dtype=torch.int32, device="cuda")
    before = L.pool.ssm.clone(), L.pool.conv.clone()
    L.pool.gdn_decode_step(0, L.w, none, q, k, v, a, b, o, slots_host=[])
    L.pool.gdn_decode_multi(0, L.w, none, none.view(0, 3), q, k, v, a, b, o, slots_in_host=[], slots_out_host=[])
    L.pool.gdn_prefill(0, L.w, [0], [], [], q, k, v, a, b, o)
    L.pool.gdn_prefill(0, L.w, [0], [], [], q, k, v, a, b, o, start_pos=[], ckpt_interval=8,
                       ckpt_slots=np.zeros((0, 2), np.int32))
    L.pool.gdn_prefill(0, L.w, [0, 0, 0], [1, 2], [1, 0], q, k, v, a, b, o, ckpt_interval=8, ckpt_slots=[[3], [-1]])
    f = torch.zeros(0, device="cuda")
    L.pool.beam_step(torch.zeros((0, 4, 50), device="cuda"), f, none, none, none, f, none)
    torch.cuda.synchronize()
    assert same(L.pool.ssm, before[0]) and same(L.pool.conv, before[1])


def test_gates_of_one_head_may_be_a_transposed_row():
    """[rows, 1] gates out of a [1, rows] tensor: the rows lie one element apart."""
    log("case: gdn transposed gates of one head")
    L = Layer((1, 1, 32, 16), 4, 8, 191)
    L.seed_slots(range(5))
    u, a, b = (dev(x, "bf16") for x in L.rows(5, "bf16"))
    q, k, v = L.pool.split_qkv(u)
    slots = torch.arange(5, dtype=torch.int32, device="cuda")
    start = L.pool.ssm.clone(), L.pool.conv.clone()
    kept = []
    for x, y in ((a, b), (a.t().contiguous().t(), b.t().contiguous().t())):
        L.pool.ssm.copy_(start[0]), L.pool.conv.copy_(start[1])
        o, op = L.out(5, "bf16"), L.out(5, "bf16")
        L.pool.gdn_decode_step(0, L.w, slots, q, k, v, x, y, o)
        L.pool.gdn_prefill(0, L.w, [0, 5], [7], [0], q, k, v, x, y, op)
        torch.cuda.synchronize()
        kept.append((o, op, L.pool.ssm.clone()))
    assert all(same(x, y) for x, y in zip(*kept))


def multi_against_single_steps(shape, W, K, io, odt):
    """K tokens of three rows (one is padding, one snapshot dropped, one row ends in its own slot) and the same tokens as
    single steps on a copy of the pool: outputs, states and windows bit for bit; the first tokens against the oracle."""
    n = 3
    L = Layer(shape, W, 40, 191)
    L.seed_slots([5, 9])
    slots_in = np.array([5, -1, 9], np.int32)
    out = (10 + np.arange(n * K, dtype=np.int32)).reshape(n, K)
    out[0, K - 1], out[2, 0] = 5, -1
    rows = L.rows(n * K, io)
    u, a, b = (dev(x, io) for x in rows)
    q, k, v = L.pool.split_qkv(u)
    single = Pool(L.pool.ssm.clone(), L.pool.conv.clone(), shape[1], shape[3], shape[2], shape[0], W, family=2)
    want_s, want_c = L.pool.ssm.clone(), L.pool.conv.clone()
    o, o1 = L.out(n * K, odt), L.out(n * K, odt)
    sl = torch.from_numpy(slots_in).cuda()
    L.pool.gdn_decode_multi(0, L.w, sl, torch.from_numpy(out).cuda(), q, k, v, a, b, o)
    for t in range(K):
        pick = torch.arange(n, device="cuda") * K + t
        ot = L.out(n, odt)
        single.gdn_decode_step(0, L.w, sl, q[pick], k[pick], v[pick], a[pick], b[pick], ot)
        o1[pick] = ot
        for i in (0, 2):
            if out[i, t] >= 0:
                want_s[0, out[i, t]], want_c[0, out[i, t]] = single.ssm[0, slots_in[i]], single.conv[0, slots_in[i]]
    torch.cuda.synchronize()
    assert same(o, o1) and same(L.pool.ssm, want_s) and same(L.pool.conv, want_c)
    ref = orc.decode_multi(shape, L.ssm, L.conv, L.params, slots_in, out, *rows)
    near(host(o)[0::K], ref[0::K], odt, "first tokens")
    assert np.array_equal(host(L.pool.conv[0, out[0].tolist()]), L.conv[out[0]])


@pytest.mark.parametrize("io,odt", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_decode_multi_of_other_types(shape, io, odt):
    """fp32 rows enter the window rounded to bf16, for the next token of the same call too."""
    log(f"case: gdn multi decode {shape} io={io} o={odt}")
    multi_against_single_steps(shape, 4, 4, io, odt)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3])
def test_decode_multi_conv_widths(W, io):
    log(f"case: gdn multi decode W={W} io={io}")
    multi_against_single_steps((1, 3, 64, 16), W, 5, io, io)


def test_decode_multi_in_all_of_lds():
    """42 value heads of 320 on one key head of 64, 3 tokens: 163836 bytes a workgroup."""
    log("case: gdn multi decode, all of LDS")
    multi_against_single_steps((1, 42, 64, 320), 4, 3, "bf16", "bf16")


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("shape", SHAPES[:4], ids=str)
def test_prefill_fp32_rows_bf16_output(shape, lens):
    """fp32 rows: a bf16 output is the fp32 one rounded, bit for bit, and the slots are the same."""
    log(f"case: gdn prefill {shape} lens={lens} io=f32 o=bf16")
    n, T = len(lens), sum(lens)
    L = Layer(shape, 4, 2 * n + 3, 31)
    L.seed_slots(range(n))
    u, a, b = (dev(x, "f32") for x in L.rows(T, "f32"))
    q, k, v = L.pool.split_qkv(u)
    start = L.pool.ssm.clone(), L.pool.conv.clone()
    kept = []
    for odt in ("f32", "bf16"):
        L.pool.ssm.copy_(start[0]), L.pool.conv.copy_(start[1])
        o = L.out(T, odt, 2)
        L.pool.gdn_prefill(0, L.w, np.concatenate([[0], np.cumsum(lens)]), np.arange(n), np.arange(n) % 2, q, k, v, a, b, o)
        torch.cuda.synchronize()
        kept.append((o.bfloat16(), L.pool.ssm.clone(), L.pool.conv.clone()))
    assert all(same(x, y) for x, y in zip(*kept))
    assert (kept[1][0][T:] == 7).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prefill_wide_at_dk_256(io):
    """Several chunks and parts of dv at the largest key width, with initial states and checkpoints."""
    log(f"case: gdn prefill wide dk 256 io={io}")
    run_prefill(Layer((2, 4, 256, 256), 4, 30, 201), [500, 77, 130], io, io, seeded=True, interval=96,
                starts=np.array([0, 31, 95], np.int32))


def test_decode_of_more_rows_than_one_launch_takes():
    """70001 rows in one call (launches of 65535), in shuffled slots: as two calls of fewer, bit for bit."""
    log("case: gdn decode 70001 rows")
    shape, n, cut = (1, 1, 32, 16), 70001, 40000
    L = Layer(shape, 4, n + 5, 211)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    for t in (L.pool.ssm, L.pool.conv):
        t.copy_(0.5 * torch.randn(t.shape, generator=g, device="cuda"))
    u = torch.randn((n, L.cd + 2), generator=g, device="cuda")
    rows = u[:, :L.cd].bfloat16()
    a, b = u[:, L.cd:-1].bfloat16(), u[:, -1:].bfloat16()
    slots = torch.randperm(n + 5, generator=g, device="cuda")[:n].to(torch.int32)
    slots[[7, 65534, 65535, 70000]] = -1
    other = Pool(L.pool.ssm.clone(), L.pool.conv.clone(), 1, 16, 32, 1, 4, family=2)
    got, want = L.out(n, "bf16"), L.out(n, "bf16")
    q, k, v = L.pool.split_qkv(rows)
    L.pool.gdn_decode_step(0, L.w, slots, q, k, v, a, b, got)
    for r in (slice(0, cut), slice(cut, n)):
        other.gdn_decode_step(0, L.w, slots[r].clone(), q[r], k[r], v[r], a[r], b[r], want[r])
    torch.cuda.synchronize()
    assert same(got, want) and same(L.pool.ssm, other.ssm) and same(L.pool.conv, other.conv)
    assert not got[[7, 65534, 65535, 70000]].any() and got[69999].any()


@pytest.mark.parametrize("shape", [(2, 4, 128, 64), (2, 4, 64, 48), (1, 2, 256, 48)], ids=str)
def test_prefill_rounds_where_it_says_and_nowhere_else(shape):
    """bf16 rows: the 2-norm error of o and of the state against that of a CPU form in fp64 with roundings at the same
    places of the same values.  fp32 arithmetic takes a value over a rounding border now and then, which changes single
    errors and not their size: of the n > 3000 elements each norm is one of n errors that are independent in the main, so
    it varies by 1/sqrt(2 n) < 1.3%, and 5% is four times that.  A bf16 operand in the place of an fp16 one adds 10% at
    least, for K, Q, R, the masked Q K^T, U or e^(G-g) U (test_gdn_cpu_roundings.py)."""
    log(f"case: gdn prefill roundings {shape}")
    T = 500
    L = Layer(shape, 4, 3, 221)
    rows = L.rows(T, "bf16")
    u, a, b = (dev(x, "bf16") for x in rows)
    o = L.out(T, "bf16")
    L.pool.gdn_prefill(0, L.w, [0, T], [1], [0], *L.pool.split_qkv(u), a, b, o)
    torch.cuda.synchronize()
    ref = orc.prefill(shape, L.ssm, L.conv, L.params, np.array([0, T]), [1], [0], None, *rows)
    sim_o, sim_s = gdn_roundings.prefill(shape, L.params, *rows)
    for what, got, sim, want in (("o", host(o), sim_o, ref), ("state", host(L.pool.ssm[0, 1]), sim_s, L.ssm[1])):
        err, bound = (gdn_roundings.norm_of_error(x, want) for x in (got, round_to(sim, "bf16")))
        log(f"  {what}: error {err:.3e}, of the rounded form {bound:.3e}")
        assert err <= 1.05 * bound, what


def test_drafts_whose_first_state_replaces_the_rows_own():
    """The state after the first of four tokens goes back into the row's slot, which is read for it, the rest elsewhere."""
    log("case: gdn multi decode, first state in place")
    shape, K = (2, 4, 128, 80), 4
    L = Layer(shape, 4, 12, 231)
    L.seed_slots([3, 6])
    slots_in = np.array([3, 6], np.int32)
    apart, own = np.array([[0, 1, 2, 4], [5, 7, 8, 9]], np.int32), np.array([[3, 1, 2, 4], [6, 7, 8, 9]], np.int32)
    u, a, b = (dev(x, "bf16") for x in L.rows(2 * K, "bf16"))
    start = L.pool.ssm.clone(), L.pool.conv.clone()
    kept = []
    for out in (apart, own):
        L.pool.ssm.copy_(start[0]), L.pool.conv.copy_(start[1])
        o = L.out(2 * K, "bf16")
        L.pool.gdn_decode_multi(0, L.w, torch.from_numpy(slots_in).cuda(), torch.from_numpy(out).cuda(), *L.pool.split_qkv(u),
                                a, b, o, slots_in_host=slots_in, slots_out_host=out)
        torch.cuda.synchronize()
        at = out.ravel().tolist()
        kept.append((o, L.pool.ssm[0, at], L.pool.conv[0, at]))
    assert all(same(x, y) for x, y in zip(*kept))


@pytest.mark.parametrize("io,first,second", [("bf16", 100032, 50001), ("f32", 60000, 20001)])
def test_prefill_past_32_bit_offsets(io, first, second):
    """Rows and a workspace of more than 2^31 bytes: a sequence behind a very long one is what it is alone, bit for bit."""
    log(f"case: gdn prefill {first} + {second} wide rows io={io}")
    L = Layer(SHAPES[-1], 4, 4, 241)
    T = first + second
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    rows = lambda n: torch.empty((T, n), dtype=torch.bfloat16 if io == "bf16" else torch.float32, device="cuda").normal_(generator=g)
    u, a, b = rows(L.cd), rows(32), rows(32)
    q, k, v = L.pool.split_qkv(u)
    o, alone = L.out(T, io), L.out(second, io)
    assert L.pool.gdn_workspace_size([0, first, T], io_dtype=o.dtype, o_dtype=o.dtype) > 2 ** 31
    L.pool.gdn_prefill(0, L.w, [0, first, T], [0, 1], [0, 0], q, k, v, a, b, o)
    L.pool.gdn_prefill(0, L.w, [0, second], [2], [0], q[first:], k[first:], v[first:], a[first:], b[first:], alone)
    torch.cuda.synchronize()
    assert torch.isfinite(alone).all() and alone.float().abs().max() > 0.01
    assert same(o[first:], alone) and same(L.pool.ssm[0, 1], L.pool.ssm[0, 2]) and same(L.pool.conv[0, 1], L.pool.conv[0, 2])


def test_prefill_of_66001_sequences():
    """One row each; the last ones as in a call of their own, bit for bit, and no slot but theirs is touched."""
    log("case: gdn prefill 66001 sequences")
    n, shape = 66001, (1, 1, 32, 16)
    L = Layer(shape, 4, n + 6, 251)
    L.pool.ssm.normal_(), L.pool.conv.normal_()
    u = torch.randn((n, L.cd + 2), device="cuda").bfloat16()
    q, k, v = L.pool.split_qkv(u[:, :L.cd].contiguous())
    a, b = u[:, L.cd:L.cd + 1], u[:, L.cd + 1:]
    for t in (L.pool.ssm, L.pool.conv):
        t[0, n + 1:] = t[0, n - 5:n]
    kept = L.pool.ssm[0, n].clone()
    o, last = L.out(n, "bf16"), L.out(5, "bf16")
    L.pool.gdn_prefill(0, L.w, np.arange(n + 1), np.arange(n), np.ones(n), q, k, v, a, b, o)
    L.pool.gdn_prefill(0, L.w, np.arange(6), np.arange(n + 1, n + 6), np.ones(5), q[-5:], k[-5:], v[-5:], a[-5:], b[-5:], last)
    torch.cuda.synchronize()
    assert same(o[-5:], last) and same(L.pool.ssm[0, n - 5:n], L.pool.ssm[0, n + 1:]) and same(L.pool.ssm[0, n], kept)
    assert same(L.pool.conv[0, n - 5:n], L.pool.conv[0, n + 1:])


def scaled_columns(shape, T, seed, column, row):
    """A layer whose v reaches the recurrence as SiLU(u) (a conv of one tap), with column c of it times column[c] and row
    t times row[t]; one sequence from a random state, scaled by column too."""
    Hk, Hv, dk, dv = shape
    L = Layer(shape, 4, 3, seed, bias=False)
    qk = 2 * Hk * dk
    L.params["conv_w"][qk:] = [0, 0, 0, 1]
    L.w.conv_w[qk:] = torch.tensor([0.0, 0.0, 0.0, 1.0], device="cuda")
    L.ssm[1] = round_to(L.rng.normal(0, 0.1, L.ssm[1].shape) * column.reshape(Hv, dv, 1), "bf16")
    L.conv[1] = 0
    L.pool.ssm[0, 1], L.pool.conv[0, 1] = torch.from_numpy(L.ssm[1]).to(torch.bfloat16).cuda(), 0
    u, a, b = L.rows(T, "bf16")
    u[:, qk:] = round_to(u[:, qk:] * column * row[:, None], "bf16")
    o = L.out(T, "bf16")
    q, k, v = L.pool.split_qkv(dev(u, "bf16"))
    L.pool.gdn_prefill(0, L.w, [0, T], [1], [1], q, k, v, dev(a, "bf16"), dev(b, "bf16"), o)
    torch.cuda.synchronize()
    ref = orc.prefill(shape, L.ssm, L.conv, L.params, np.array([0, T]), [1], [1], None, u, a, b)
    return host(o), ref, host(L.pool.ssm[0, 1]), L.ssm[1]


# One element's own rounding is off by 2^-8 at most; the fp16 operands add 3e-4 of the 2-norm on usual rows, and 2e-3 is
# what the worst conditioned ones (keys that repeat) come to.
COLUMN_2NORM = 2.0 ** -8 + 2e-3


def rel(got, ref, axis):
    return np.sqrt(((got - ref) ** 2).sum(axis) / np.maximum((ref ** 2).sum(axis), 1e-300))


@pytest.mark.parametrize("shape", [(1, 2, 64, 48), (2, 2, 128, 32), (1, 1, 256, 32)], ids=str)
def test_prefill_columns_of_any_magnitude(shape):
    """Columns of v and of the state from 1e-25 to 1e30, one of zeros among them: each as exact as the others."""
    log(f"case: gdn prefill columns of many magnitudes {shape}")
    n = shape[1] * shape[3]
    column = 10.0 ** np.linspace(-25, 30, n)
    column[n // 2] = 0.0
    o, ref, s, want = scaled_columns(shape, 150, 261, column, np.ones(150))
    live = np.arange(n) != n // 2
    assert not o[:, ~live].any() and not s.reshape(n, -1)[~live].any() and np.isfinite(o).all()
    assert rel(o, ref, 0)[live].max() <= COLUMN_2NORM
    assert rel(s, want, -1).reshape(-1)[live].max() <= COLUMN_2NORM


@pytest.mark.parametrize("shape", [(1, 2, 64, 48), (1, 1, 256, 32)], ids=str)
def test_prefill_rows_of_many_magnitudes(shape):
    """v that grows by 1e5 inside a chunk, shrinks by 1e5 in the next, and goes on from there: every row is as exact as
    its own size asks, also next to rows that set the unit of its chunk."""
    log(f"case: gdn prefill rows of many magnitudes {shape}")
    T = 260
    row = np.ones(T)
    row[:40] = 1e-5
    row[40:90] = 1.0
    row[90:] = 1e-5
    o, ref, s, want = scaled_columns(shape, T, 271, np.full(shape[1] * shape[3], 1e-3), row)
    assert rel(o, ref, 1).max() <= COLUMN_2NORM and rel(s.ravel(), want.ravel(), 0) <= COLUMN_2NORM


def test_prefill_goes_on_from_a_wiped_state():
    """Huge rows, then a state that alpha = 0 wipes to exactly nothing, then tiny rows: the unit falls by 2^100."""
    log("case: gdn prefill wiped state")
    for shape in ((1, 1, 64, 32), (1, 1, 256, 32)):
        Hk, Hv, dk, dv = shape
        L = Layer(shape, 4, 3, 281, bias=False)
        T = 200
        L.params["conv_w"][2 * dk:] = [0, 0, 0, 1]
        L.w.conv_w[2 * dk:] = torch.tensor([0.0, 0.0, 0.0, 1.0], device="cuda")
        u, a, b = L.rows(T, "bf16")
        u[:64, 2 * dk:] = round_to(u[:64, 2 * dk:] * 1e15, "bf16")
        u[64:, 2 * dk:] = round_to(u[64:, 2 * dk:] * 1e-15, "bf16")
        u[100:140, 2 * dk:] = 0.0
        a[64:72] = 3e4
        b[64:68] = -200.0                             # beta is 0: nothing is written either
        o = L.out(T, "bf16")
        L.pool.gdn_prefill(0, L.w, [0, T], [1], [0], *L.pool.split_qkv(dev(u, "bf16")), dev(a, "bf16"), dev(b, "bf16"), o)
        torch.cuda.synchronize()
        ref = orc.prefill(shape, L.ssm, L.conv, L.params, np.array([0, T]), [1], [0], None, u, a, b)
        got = host(o)
        assert not got[64:68].any()
        for part in (slice(0, 64), slice(68, T)):
            assert rel(got[part].ravel(), ref[part].ravel(), 0) <= COLUMN_2NORM
        assert rel(host(L.pool.ssm[0, 1]).ravel(), L.ssm[1].ravel(), 0) <= COLUMN_2NORM


@pytest.mark.parametrize("shape", [(1, 1, 64, 32), (1, 1, 256, 32)], ids=str)
def test_prefill_of_a_huge_state_that_nothing_is_written_to(shape):
    """A state of 1e28 that two rows read with beta = 0, then wiped inside the chunk, then v of 1e-8 (a factor of 2^120):
    the outputs of the first two rows are the state's, those of the rest v's, and all are finite."""
    log(f"case: gdn prefill huge state, tiny rows {shape}")
    Hk, Hv, dk, dv = shape
    L = Layer(shape, 4, 3, 291, bias=False)
    T = 70
    L.params["conv_w"][2 * dk:] = [0, 0, 0, 1]
    L.w.conv_w[2 * dk:] = torch.tensor([0.0, 0.0, 0.0, 1.0], device="cuda")
    L.ssm[1], L.conv[1] = round_to(L.rng.normal(0, 1e28, L.ssm[1].shape), "bf16"), 0
    L.pool.ssm[0, 1], L.pool.conv[0, 1] = torch.from_numpy(L.ssm[1]).to(torch.bfloat16).cuda(), 0
    u, a, b = L.rows(T, "bf16")
    u[:, 2 * dk:] = round_to(u[:, 2 * dk:] * 1e-8, "bf16")
    b[:3], a[2] = -200.0, 3e4
    o = L.out(T, "bf16")
    L.pool.gdn_prefill(0, L.w, [0, T], [1], [1], *L.pool.split_qkv(dev(u, "bf16")), dev(a, "bf16"), dev(b, "bf16"), o)
    torch.cuda.synchronize()
    ref = orc.prefill(shape, L.ssm, L.conv, L.params, np.array([0, T]), [1], [1], None, u, a, b)
    got = host(o)
    assert np.isfinite(got).all()
    for part in (slice(0, 2), slice(3, 64), slice(64, T)):
        assert rel(got[part].ravel(), ref[part].ravel(), 0) <= COLUMN_2NORM, part
    assert rel(host(L.pool.ssm[0, 1]).ravel(), L.ssm[1].ravel(), 0) <= COLUMN_2NORM
