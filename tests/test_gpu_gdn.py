"""GPU parity of the gated delta rule (decode, multi-token decode, chunked prefill) with the fp64 oracle.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value.  Decode computes in fp32: an
element of o is off by that rounding (fp32 outputs: none), one of the stored state by twice that
(the oracle's is rounded too), plus fp32 rounding, whose
sums over dk <= 256 products and few-ulp exp, reciprocal and root stay below 2^-24 * 300 < 2e-5 of the
largest value.  The prefill's contractions take operands of fewer bits: with one rounding to bf16 each, whose relative
rms is 2^-8 / sqrt(3) * 0.72 = 1.6e-3, about 25 independent contributions of weight one would give 5 * 1.6e-3 = 8e-3 of
the 2-norm, the bound here; they are fp16, an eighth of that each, and test_gpu_gdn_edges.py holds the error to that of
these roundings alone, about 1.7e-3 with the output's own.  With fp32 rows or
outputs an operand is three planes, off by 2^-24, as are products: the fp32 rule holds, of the 2-norm.
Single elements: six times the 2-norm bound, taken of the largest value.
"""
import numpy as np
import pytest
import torch

from oracle import gdn as orc
from oracle.mamba2 import round_to
from recurrent_state_update_amd import synth
from recurrent_state_update_amd.pool import LayerWeights, Mamba2Error, Pool
from tests.gpu_helpers import TORCH_DT, dev, host, log, raw_bytes, untouched

pytestmark = pytest.mark.gpu

F32_ABS = 2e-5
PREFILL_2NORM = {"bf16": 8e-3, "f32": 2e-5}


class Layer:
    """Seeded parameters and a sentinel-filled pool of one gated-delta shape (Hk, Hv, dk, dv)."""

    def __init__(self, shape, W, slots, seed, bias=True, layers=1):
        Hk, Hv, dk, dv = self.shape = shape
        self.W, self.cd = W, 2 * Hk * dk + Hv * dv
        self.rng = rng = np.random.default_rng(seed)
        ex = lambda v: synth.cast_exact(v, "f32").astype(np.float64)
        self.params = dict(A=ex(-np.exp(rng.uniform(0, np.log(16), Hv))), dt_bias=ex(rng.uniform(-4, -2, Hv)),
                           conv_w=ex(rng.uniform(-0.5, 0.5, (self.cd, W))),
                           conv_b=ex(rng.uniform(-0.5, 0.5, self.cd)) if bias else None)
        f = lambda k: None if self.params[k] is None else torch.as_tensor(self.params[k].astype(np.float32), device="cuda")
        self.w = LayerWeights(f("A"), None, f("dt_bias"), f("conv_w"), f("conv_b"))
        self.pool = Pool.allocate_gdn(layers, slots, Hv, dv, dk, Hk, W)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        for t in (self.pool.ssm, self.pool.conv):
            b = t.view(torch.uint8)
            b.copy_(torch.randint(0, 256, b.shape, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8))
        self.ssm = np.zeros((slots, Hv, dv, dk))
        self.conv = np.zeros((slots, self.cd, W - 1))

    def seed_slots(self, slots):
        for s in slots:
            self.ssm[s] = synth.cast_exact(self.rng.normal(0, 0.1, self.ssm[s].shape), "bf16")
            self.conv[s] = synth.cast_exact(self.rng.normal(0, 1, self.conv[s].shape), "bf16")
            self.pool.ssm[0, s] = torch.from_numpy(self.ssm[s]).to(torch.bfloat16).cuda()
            self.pool.conv[0, s] = torch.from_numpy(self.conv[s]).to(torch.bfloat16).cuda()

    def rows(self, n, io):
        ex = lambda v: synth.cast_exact(v, io).astype(np.float64)
        Hv = self.shape[1]
        return ex(self.rng.normal(0, 1, (n, self.cd))), ex(self.rng.normal(0, 1, (n, Hv))), ex(self.rng.normal(0, 1, (n, Hv)))

    def out(self, n, dt, extra=0):
        return torch.full((n + extra, self.shape[1] * self.shape[3]), 7.0, dtype=TORCH_DT[dt], device="cuda")


def near(got, ref, dt, what, halves=1):
    """Element by element: half steps of the type's rounding (two where ref is rounded too) plus fp32 rounding."""
    tol = (halves * 2.0 ** -8 if dt == "bf16" else 0.0) * np.abs(ref) + F32_ABS * np.abs(ref).max()
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - ref).max()))


def near2(got, ref, tol, what):
    err = got - ref
    rel = np.sqrt((err ** 2).sum() / max((ref ** 2).sum(), 1e-300))
    log(f"  {what}: 2-norm {rel:.2e} (bound {tol:.0e}), max {np.abs(err).max() / np.abs(ref).max():.2e}")
    assert np.isfinite(got).all() and rel <= tol, (what, rel)
    assert np.abs(err).max() <= 6 * tol * np.abs(ref).max(), what


WIDE = (16, 32, 128, 128)
SHAPES = [(2, 8, 32, 64), (1, 3, 64, 16), (3, 3, 128, 80), (2, 4, 256, 48), WIDE]


@pytest.mark.parametrize("io,odt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_decode(shape, io, odt):
    log(f"case: gdn decode {shape} io={io} o={odt}")
    L = Layer(shape, 4, 12, 11, bias=shape != WIDE)
    slots = np.array([3, -1, 0, 11, 7, 12], np.int32)     # a padding row and a slot out of range
    L.seed_slots([0, 3, 7, 11])
    bs, bc = raw_bytes(L.pool.ssm), raw_bytes(L.pool.conv)
    for step in range(3):
        u, a, b = L.rows(len(slots), io)
        o = L.out(len(slots), odt)
        q, k, v = L.pool.split_qkv(dev(u, io))
        L.pool.gdn_decode_step(0, L.w, torch.from_numpy(slots).cuda(), q, k, v, dev(a, io), dev(b, io), o)
        torch.cuda.synchronize()
        live = [3, 0, 11, 7]
        ref = orc.decode_step(shape, L.ssm, L.conv, L.params, slots, u, a, b)
        near(host(o), ref, odt, f"o {step}")
        assert not host(o)[[1, 5]].any()
        near(host(L.pool.ssm[0, live]), L.ssm[live], "bf16", "state", 2)
        assert np.array_equal(host(L.pool.conv[0, live]), L.conv[live])
        # go on from what the slots hold: a state element next to a rounding border may go either way
        L.ssm[live] = host(L.pool.ssm[0, live])
    assert untouched(bs, L.pool.ssm, live) and untouched(bc, L.pool.conv, live)


@pytest.mark.parametrize("W", [2, 3])
def test_decode_conv_widths_and_strides(W):
    log(f"case: gdn decode W={W}, rows inside wider ones")
    shape = (2, 4, 64, 32)
    L = Layer(shape, W, 5, 12)
    L.seed_slots([1, 4])
    u, a, b = L.rows(2, "bf16")
    wide = torch.full((2, L.cd + 24), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + L.cd] = dev(u, "bf16")
    q, k, v = L.pool.split_qkv(wide[:, 8:8 + L.cd])
    ab = torch.cat([dev(a, "bf16"), dev(b, "bf16")], dim=1)
    big = torch.full((2, shape[1] * shape[3] + 3), 5.0, dtype=torch.float32, device="cuda")
    slots = np.array([4, 1], np.int32)
    L.pool.gdn_decode_step(0, L.w, torch.from_numpy(slots).cuda(), q, k, v, ab[:, :4], ab[:, 4:], big[:, 1:-2],
                           slots_host=slots)
    torch.cuda.synchronize()
    ref = orc.decode_step(shape, L.ssm, L.conv, L.params, slots, u, a, b)
    near(host(big[:, 1:-2]), ref, "f32", "o")
    near(host(L.pool.ssm[0, [1, 4]]), L.ssm[[1, 4]], "bf16", "state", 2)
    assert np.array_equal(host(L.pool.conv[0, [1, 4]]), L.conv[[1, 4]])
    assert (big[:, 0] == 5).all() and (big[:, -2:] == 5).all()


@pytest.mark.parametrize("K", [1, 3, 8])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_decode_multi_equals_single_steps_bit_for_bit(shape, K):
    log(f"case: gdn multi decode {shape} K={K}")
    n, S = 3, 40
    L = Layer(shape, 4, S, 21)
    L.seed_slots([5, 9, 2])
    slots_in = np.array([5, -1, 9], np.int32)
    out = (10 + np.arange(n * K, dtype=np.int32)).reshape(n, K)
    out[0, K - 1] = 5            # the last state back into the row's own slot
    if K > 1:
        out[2, 0] = -1           # one snapshot dropped
    u, a, b = L.rows(n * K, "bf16")
    q, k, v = L.pool.split_qkv(dev(u, "bf16"))
    ad, bd = dev(a, "bf16"), dev(b, "bf16")
    ssm0, conv0 = L.pool.ssm.clone(), L.pool.conv.clone()
    o = L.out(n * K, "bf16")
    L.pool.gdn_decode_multi(0, L.w, torch.from_numpy(slots_in).cuda(), torch.from_numpy(out).cuda(), q, k, v, ad, bd, o,
                            slots_in_host=slots_in, slots_out_host=out)
    torch.cuda.synchronize()
    # the same tokens as single steps on a copy
    other = Pool(ssm0.clone(), conv0.clone(), shape[1], shape[3], shape[2], shape[0], 4, family=2)
    want_s, want_c = ssm0.clone(), conv0.clone()
    o1 = L.out(n * K, "bf16")
    sl = torch.from_numpy(slots_in).cuda()
    for t in range(K):
        pick = torch.arange(n, device="cuda") * K + t
        ot = L.out(n, "bf16")
        other.gdn_decode_step(0, L.w, sl, q[pick], k[pick], v[pick], ad[pick], bd[pick], ot)
        o1[pick] = ot
        for i in (0, 2):
            if out[i, t] >= 0:
                want_s[0, out[i, t]], want_c[0, out[i, t]] = other.ssm[0, slots_in[i]], other.conv[0, slots_in[i]]
    torch.cuda.synchronize()
    assert torch.equal(o.view(torch.int16), o1.view(torch.int16))
    assert torch.equal(L.pool.ssm.view(torch.int16), want_s.view(torch.int16))
    assert torch.equal(L.pool.conv.view(torch.int16), want_c.view(torch.int16))
    # and the first token against the oracle
    ref = orc.decode_multi(shape, L.ssm, L.conv, L.params, slots_in, out, u, a, b)
    near(host(o)[0::K], ref[0::K], "bf16", "first tokens")


def run_prefill(L, lens, io, odt, seeded=False, interval=0, starts=None, seed_all=False):
    n = len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    slots = (np.arange(n, dtype=np.int32) * 2 + 1)
    has = (np.arange(n) % 2 == 0).astype(np.uint8) if seeded else np.zeros(n, np.uint8)
    L.seed_slots([s for s, h in zip(slots, has) if h])
    ck = None
    if interval:
        st = starts if starts is not None else [0] * n
        counts = [(p + m) // interval - p // interval for p, m in zip(st, lens)]
        ck = np.full((n, max(1, max(counts))), -1, np.int32)
        free = iter(range(2 * n + 1, L.pool.num_slots))
        for i, m in enumerate(counts):
            for j in range(m):
                if (i + j) % 4 != 3:          # some are skipped
                    ck[i, j] = next(free)
    T = int(cu[-1])
    u, a, b = L.rows(T, io)
    extra = 3
    pad = lambda t: torch.cat([t, torch.full((extra, t.shape[1]), float("nan"), dtype=t.dtype, device="cuda")])
    o = L.out(T, odt, extra)
    q, k, v = L.pool.split_qkv(pad(dev(u, io)))
    bs, bc = raw_bytes(L.pool.ssm), raw_bytes(L.pool.conv)
    L.pool.gdn_prefill(0, L.w, cu, slots, has, q, k, v, pad(dev(a, io)), pad(dev(b, io)), o, start_pos=starts,
                       ckpt_interval=interval, ckpt_slots=ck)
    torch.cuda.synchronize()
    ref = orc.prefill(L.shape, L.ssm, L.conv, L.params, cu, slots, has, starts, u, a, b, interval, ck)
    assert (o[T:] == 7).all()                  # rows behind the last sequence
    live = [int(s) for s, m in zip(slots, lens) if m] + ([int(s) for s in ck.ravel() if s >= 0] if ck is not None else [])
    assert untouched(bs, L.pool.ssm, live) and untouched(bc, L.pool.conv, live)
    kind = "bf16" if io == "bf16" and odt == "bf16" else "f32"
    tol = PREFILL_2NORM[kind]
    rnd = 1.7e-3 if odt == "bf16" else 0.0     # the output's own rounding
    near2(host(o[:T]), ref, tol + rnd, "o")
    near2(host(L.pool.ssm[0, live]), L.ssm[live], tol + 1.7e-3, "states")
    assert np.array_equal(host(L.pool.conv[0, live]), L.conv[live])


LENS = [[1], [63, 64, 65], [130, 0, 1, 2, 3, 200]]


@pytest.mark.parametrize("io,odt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("shape", SHAPES[:4], ids=str)
def test_prefill(shape, lens, io, odt):
    log(f"case: gdn prefill {shape} lens={lens} io={io} o={odt}")
    run_prefill(Layer(shape, 4, 2 * len(lens) + 3, 31), lens, io, odt, seeded=len(lens) > 1)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_prefill_checkpoints(W, io):
    log(f"case: gdn prefill checkpoints W={W} io={io}")
    L = Layer((2, 4, 64, 48), W, 80, 41, bias=W != 3)
    run_prefill(L, [97, 5, 300, 1, 0, 66], io, io, seeded=True, interval=23, starts=np.array([0, 21, 7, 22, 3, 0], np.int32))


def test_prefill_wide_long():
    log("case: gdn prefill wide 500 + 77 rows")
    run_prefill(Layer(WIDE, 4, 8, 51), [500, 77], "bf16", "bf16", seeded=True)


def test_prefill_many_sequences_uses_upload_launches():
    """More tables than the first launch's arguments hold."""
    log("case: gdn prefill 120 sequences")
    rng = np.random.default_rng(3)
    run_prefill(Layer((1, 2, 32, 16), 4, 250, 61), [int(v) for v in rng.integers(0, 90, 120)], "f32", "f32", seeded=True)


@pytest.mark.parametrize("kind", ["strong decay", "no decay", "repeated keys", "reset"])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prefill_extremes(kind, io):
    """Gates at their ends and keys that repeat exactly (the worst conditioned T)."""
    log(f"case: gdn prefill {kind} io={io}")
    shape = (1, 2, 64, 32)
    L = Layer(shape, 4, 4, 71)
    T = 150
    u, a, b = L.rows(T, io)
    if kind == "strong decay":
        a[:] = 40.0
    elif kind == "no decay":
        a[:], b[:] = -60.0, 30.0
    elif kind == "repeated keys":
        u[:, 64:128] = u[:1, 64:128]
        a[:], b[:] = -60.0, 30.0
    else:
        a[:] = -20.0
        a[[10, 50, 64, 100]] = 3e4          # the state is wiped: alpha is 0
    L.seed_slots([2])
    o = L.out(T, io)
    q, k, v = L.pool.split_qkv(dev(u, io))
    L.pool.gdn_prefill(0, L.w, [0, T], [2], [1], q, k, v, dev(a, io), dev(b, io), o)
    torch.cuda.synchronize()
    ref = orc.prefill(shape, L.ssm, L.conv, L.params, np.array([0, T]), [2], [1], None, u, a, b)
    extra = 1.7e-3 if io == "bf16" else 0.0
    near2(host(o), ref, PREFILL_2NORM[io] + extra, "o")
    near2(host(L.pool.ssm[0, 2]), L.ssm[2], PREFILL_2NORM[io] + 1.7e-3, "state")


def test_prefill_then_drafts_then_decode_run_together():
    """A prompt, a draft step of which two tokens are accepted, then single tokens, as a server runs them, on a
    stream of its own; against the oracle from the same slots."""
    log("case: gdn prefill + multi + decode")
    shape, io = (2, 4, 128, 64), "bf16"
    L = Layer(shape, 4, 16, 81)
    cu, slots = np.array([0, 70, 75], np.int32), np.array([4, 9], np.int32)
    u, a, b = L.rows(75, io)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o = L.out(75, io)
        q, k, v = L.pool.split_qkv(dev(u, io))
        L.pool.gdn_prefill(0, L.w, cu, slots, [0, 0], q, k, v, dev(a, io), dev(b, io), o)
    s.synchronize()
    ref = orc.prefill(shape, L.ssm, L.conv, L.params, cu, slots, [0, 0], None, u, a, b)
    near2(host(o), ref, 8e-3 + 1.7e-3, "prompt")
    L.ssm[slots] = host(L.pool.ssm[0, slots.tolist()])
    with torch.cuda.stream(s):
        u, a, b = L.rows(6, io)
        snap = np.array([[0, 1, 2], [5, 6, 7]], np.int32)
        o = L.out(6, io)
        q, k, v = L.pool.split_qkv(dev(u, io))
        L.pool.gdn_decode_multi(0, L.w, torch.from_numpy(slots).cuda(), torch.from_numpy(snap).cuda(), q, k, v,
                                dev(a, io), dev(b, io), o)
    s.synchronize()
    near(host(o)[[0, 3]], orc.decode_multi(shape, L.ssm, L.conv, L.params, slots, snap, u, a, b)[[0, 3]], io, "drafts")
    now = snap[:, 1].copy()                     # two tokens accepted: the sequences live there now
    L.ssm[now], L.conv[now] = host(L.pool.ssm[0, now.tolist()]), host(L.pool.conv[0, now.tolist()])
    with torch.cuda.stream(s):
        u, a, b = L.rows(2, io)
        o = L.out(2, io)
        q, k, v = L.pool.split_qkv(dev(u, io))
        L.pool.gdn_decode_step(0, L.w, torch.from_numpy(now).cuda(), q, k, v, dev(a, io), dev(b, io), o)
    s.synchronize()
    near(host(o), orc.decode_step(shape, L.ssm, L.conv, L.params, now, u, a, b), io, "decode")


def test_prefill_and_decode_in_a_graph():
    """A prefill and a decode step captured together and replayed on changing rows equal the eager calls."""
    log("case: gdn graph")
    shape, io = (2, 4, 64, 64), "bf16"
    L = Layer(shape, 4, 6, 91)
    cu = np.array([0, 66, 99], np.int32)
    ins = [dev(L.rows(101, io)[0], io) for _ in range(3)]
    gates = [tuple(dev(x, io) for x in L.rows(101, io)[1:]) for _ in range(3)]
    u, a, b = ins[0].clone(), gates[0][0].clone(), gates[0][1].clone()
    o = L.out(101, io)
    sl = torch.tensor([1, 3], dtype=torch.int32, device="cuda")
    ws = torch.empty(L.pool.gdn_workspace_size(cu), dtype=torch.uint8, device="cuda")

    def step():
        q, k, v = L.pool.split_qkv(u)
        L.pool.gdn_prefill(0, L.w, cu, [1, 3], [0, 0], q, k, v, a, b, o, workspace=ws)
        q, k, v = L.pool.split_qkv(u[99:])
        L.pool.gdn_decode_step(0, L.w, sl, q, k, v, a[99:], b[99:], o[99:])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x, (ga, gb) in zip(ins, gates):
        u.copy_(x), a.copy_(ga), b.copy_(gb)
        step()
        want = o.clone(), L.pool.ssm[0, [1, 3]].clone(), L.pool.conv[0, [1, 3]].clone()
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((o, L.pool.ssm[0, [1, 3]], L.pool.conv[0, [1, 3]]), want):
            assert torch.equal(got.view(torch.int16), w.view(torch.int16))


def test_bindings_refuse_mismatched_rows():
    L = Layer((2, 4, 32, 16), 4, 4, 1)
    u, a, b = (dev(x, "bf16") for x in L.rows(2, "bf16"))
    q, k, v = L.pool.split_qkv(u)
    o = L.out(2, "bf16")
    sl = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        L.pool.gdn_decode_step(0, L.w, sl, q, k, v[:1], a, b, o)
    with pytest.raises(ValueError):
        L.pool.gdn_decode_step(0, L.w, sl, q.cpu(), k, v, a, b, o)
    with pytest.raises(TypeError):
        L.pool.gdn_decode_step(0, L.w, sl, q, k, v, a.float(), b, o)
    with pytest.raises(Mamba2Error):
        L.pool.gdn_decode_step(0, L.w, sl, q, k, v, a, b, o, slots_host=[0, 0])
    with pytest.raises(ValueError):
        L.pool.gdn_prefill(0, L.w, [0, 3], [1], [0], q, k, v, a, b, o)


def test_slots_beyond_32_bit_offsets():
    """State elements past 2^31 (a slot of the wide layer holds 2^19): decode, drafts, prefill and checkpoints there."""
    log("case: gdn far slots")
    Hk, Hv, dk, dv = WIDE
    S = 4100
    pool = Pool(torch.empty((1, S, Hv, dv, dk), dtype=torch.bfloat16, device="cuda"),
                torch.empty((1, S, 2 * Hk * dk + Hv * dv, 3), dtype=torch.bfloat16, device="cuda"), Hv, dv, dk, Hk, 4, family=2)
    L = Layer(WIDE, 4, 6, 101)
    L.seed_slots([0, 1])
    far = {0: 4099, 1: 4097, 2: 4098, 3: 4096, 4: 7}
    for s in (0, 1):
        pool.ssm[0, far[s]], pool.conv[0, far[s]] = L.pool.ssm[0, s], L.pool.conv[0, s]
    u, a, b = L.rows(70, "bf16")
    q, k, v = L.pool.split_qkv(dev(u, "bf16"))
    ad, bd = dev(a, "bf16"), dev(b, "bf16")
    got, want = L.out(70, "bf16"), L.out(70, "bf16")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for P, m, o in ((L.pool, lambda s: s, want), (pool, lambda s: far[s], got)):
        P.gdn_prefill(0, L.w, [0, 66], [m(0)], [1], q, k, v, ad, bd, o, ckpt_interval=40, ckpt_slots=[[m(2)]])
        P.gdn_decode_multi(0, L.w, i32(m(0)), i32(m(3), m(4)).view(1, 2), q[66:68], k[66:68], v[66:68], ad[66:68],
                           bd[66:68], o[66:68])
        P.gdn_decode_step(0, L.w, i32(m(4), m(1)), q[68:], k[68:], v[68:], ad[68:], bd[68:], o[68:])
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    for s, f in far.items():
        assert torch.equal(pool.ssm[0, f].view(torch.int16), L.pool.ssm[0, s].view(torch.int16)), s
        assert torch.equal(pool.conv[0, f].view(torch.int16), L.pool.conv[0, s].view(torch.int16)), s


@pytest.mark.parametrize("dk", [64, 256])
def test_prefill_output_at_any_alignment_and_stride(dk):
    log(f"case: gdn prefill odd output rows dk={dk}")
    L = Layer((1, 2, dk, 48), 4, 4, 111)
    T = 67
    u, a, b = L.rows(T, "bf16")
    q, k, v = L.pool.split_qkv(dev(u, "bf16"))
    ad, bd = dev(a, "bf16"), dev(b, "bf16")
    want = L.out(T, "bf16")
    L.pool.gdn_prefill(0, L.w, [0, T], [1], [0], q, k, v, ad, bd, want)
    for width, off in ((97, 0), (98, 1), (104, 3)):
        buf = torch.full((T, width), 5.0, dtype=torch.bfloat16, device="cuda")
        L.pool.gdn_prefill(0, L.w, [0, T], [1], [0], q, k, v, ad, bd, buf[:, off:off + 96])
        torch.cuda.synchronize()
        assert torch.equal(buf[:, off:off + 96], want)
        assert (buf[:, :off] == 5).all() and (buf[:, off + 96:] == 5).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prefill_checkpoint_after_every_row(io):
    log(f"case: gdn prefill checkpoint after every row io={io}")
    run_prefill(Layer((1, 2, 32, 32), 4, 60, 121), [9, 1, 5], io, io, seeded=True, interval=1,
                starts=np.array([2, 0, 7], np.int32))


def test_prefill_does_not_depend_on_its_batch():
    """Bit for bit the same alone, beside others, and on a second run."""
    log("case: gdn prefill batch independence")
    L = Layer((2, 4, 128, 64), 4, 8, 131)
    T = 200
    u, a, b = L.rows(T, "bf16")
    q, k, v = L.pool.split_qkv(dev(u, "bf16"))
    ad, bd = dev(a, "bf16"), dev(b, "bf16")
    outs = []
    for cu, slots in (([0, 90, T], [1, 2]), ([0, 90, T], [1, 2])):
        o = L.out(T, "bf16")
        L.pool.gdn_prefill(0, L.w, cu, slots, [0] * len(slots), q, k, v, ad, bd, o)
        outs.append((o.clone(), L.pool.ssm[0, 2].clone()))
    o = L.out(T - 90, "bf16")
    L.pool.gdn_prefill(0, L.w, [0, T - 90], [5], [0], q[90:], k[90:], v[90:], ad[90:], bd[90:], o)
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.equal(o, outs[0][0][90:]) and torch.equal(L.pool.ssm[0, 5], outs[0][1])


def test_prefill_of_a_long_sequence():
    """More chunks than the first launch's arguments hold, in one sequence."""
    log("case: gdn prefill 13001 rows")
    run_prefill(Layer((1, 1, 32, 16), 4, 4, 141), [13001], "bf16", "bf16")


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace and slots, equal the same calls one after the other."""
    log("case: gdn two streams")
    L = Layer((2, 4, 64, 64), 4, 8, 151)
    T = 400
    u, a, b = L.rows(T, "bf16")
    q, k, v = L.pool.split_qkv(dev(u, "bf16"))
    ad, bd = dev(a, "bf16"), dev(b, "bf16")
    ws = [torch.empty(L.pool.gdn_workspace_size([0, T]), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [L.out(T, "bf16") for _ in range(4)]
    for i in range(2):
        L.pool.gdn_prefill(0, L.w, [0, T], [i], [0], q, k, v, ad, bd, outs[i], workspace=ws[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            L.pool.gdn_prefill(0, L.w, [0, T], [4 + i], [0], q, k, v, ad, bd, outs[2 + i], workspace=ws[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], outs[2 + i]) and torch.equal(L.pool.ssm[0, i], L.pool.ssm[0, 4 + i])
