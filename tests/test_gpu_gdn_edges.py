"""GPU checks of the gated delta rule at the edges of what its calls allow: rows that are not finite, forms and sizes
that the parity tests do not reach, views of one row.  Tolerances are those of the parity tests unless a test says
otherwise."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import dev, log
from tests.test_gpu_gdn import Layer

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
