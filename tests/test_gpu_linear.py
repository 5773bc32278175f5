"""Linear attention with a fixed decay for each head on the GPU, against the recurrence in 64 bits.

Tolerances, from the arithmetic (A: the sum of the absolute values of a result's terms; a rounding to bf16 is 2^-8 relative at most):

* steps (decode, verify, commit) and prompts outside the tensor-core kernel compute in fp32: sums of at most a few hundred terms, 2^-24
  each and some on the powers of the decay, are good to 2^-15 A; a bf16 result adds 2^-8 of itself;
* the tensor-core kernel takes P and S as bf16 into o: 2^-8 A + 2^-15 A, and o's own rounding; its state takes v g^e in two bf16 parts
  (2^-16) for a bf16 pool and in three (2^-24) for an fp32 one.
"""
import math

import pytest
import torch

import gated_deltanet_linear_mtp_gb300 as gdn
import linear_ref
from test_gpu_timeout import run_with, timeout_lib  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
I32 = dict(dtype=torch.int32, device="cuda")
CANARY = 7.25


def near(x, ref, A, extra, what):
    x, ref = x.detach().cpu(), ref.cpu()
    tol = (2.0 ** -15 + extra) * A.cpu() + (2.0 ** -8 * ref.abs() if x.dtype == torch.bfloat16 else 0) + 1e-30
    bad = (x.double() - ref).abs() > tol
    assert bool(torch.isfinite(x).all()), what
    assert not bool(bad.any()), (what, float(((x.double() - ref).abs() / tol).max()))


def written(o):
    """Whether every row of o was written (a single number may be the canary's by chance)."""
    return not bool((o == CANARY).all(-1).any())


class Case:
    """A pool, lanes and tokens; the lanes' slots differ, and so do the slots they write."""

    def __init__(self, lead, B, HK, HV, DK, DV, io="bf16", state="bf16", seed=0, slots=None, log_decay=None):
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.B, self.HK, self.HV, self.DK, self.DV = B, HK, HV, DK, DV
        self.slots = slots or 2 * B + 2
        self.pool = r(self.slots, HV, DV, DK).to(TYPES[state])
        self.q, self.k = r(*lead, HK, DK).to(TYPES[io]), r(*lead, HK, DK).to(TYPES[io])
        self.v = r(*lead, HV, DV).to(TYPES[io])
        ld = -torch.exp2(-8.0 * (torch.arange(HV) + 1) / HV) if log_decay is None else torch.tensor(log_decay)
        self.ld = ld.float().cuda()
        order = torch.randperm(self.slots, generator=torch.Generator().manual_seed(seed))
        self.read, self.write = order[:B].to(**I32), order[B:2 * B].to(**I32)
        self.o = torch.full((*lead, HV, DV), CANARY, dtype=TYPES[io], device="cuda")
        self.scale = DK ** -0.5
        self.err = torch.zeros(1, **I32)

    def ref(self, S, rows, index=()):
        q, k, v = (x[rows].cpu() for x in (self.q, self.k, self.v))
        return linear_ref.steps(S.cpu(), q, k, v, self.ld.cpu(), self.scale)


STEPS = [  # T, HK, HV, DK, DV, io, state
    (1, 1, 1, 128, 128, "bf16", "bf16"), (1, 2, 4, 128, 64, "bf16", "f32"), (4, 1, 2, 128, 33, "bf16", "bf16"),
    (8, 2, 2, 64, 40, "bf16", "f32"), (9, 1, 3, 128, 128, "bf16", "bf16"), (16, 1, 2, 64, 17, "bf16", "f32"),
    (16, 1, 1, 128, 96, "bf16", "f32"), (3, 1, 2, 32, 1, "bf16", "bf16"), (12, 2, 4, 256, 20, "bf16", "bf16"),
    (5, 1, 2, 256, 64, "bf16", "f32"), (2, 2, 2, 16, 48, "bf16", "bf16"), (1, 1, 2, 64, 65, "f32", "f32"),
    (16, 2, 4, 128, 31, "f32", "bf16"), (7, 1, 1, 16, 7, "f32", "f32"), (1, 1, 1, 32, 130, "bf16", "f32"), (15, 1, 2, 256, 66, "f32", "f32")]


@pytest.mark.parametrize("T,HK,HV,DK,DV,io,state", STEPS)
def test_steps(T, HK, HV, DK, DV, io, state):
    c = Case((4, T), 4, HK, HV, DK, DV, io, state, seed=T)
    c.read[2], c.write[2] = -1, -1  # a padded lane
    before = c.pool.clone()
    lanes = [0, 1, 3]
    # verify: nothing of the pool changes, lanes may share a slot
    read = c.read.clone()
    read[1] = read[0]
    gdn.gdn_linear_verify(c.q, c.k, c.v, c.ld, c.pool, read, c.o, None, c.err, scale=c.scale)
    states = torch.full((4, T, HV, DV, DK), CANARY, dtype=c.pool.dtype, device="cuda")
    o2 = torch.full_like(c.o, CANARY)
    gdn.gdn_linear_verify(c.q, c.k, c.v, c.ld, c.pool, read, o2, states, c.err, scale=c.scale)
    assert torch.equal(c.pool, before)
    assert bool((c.o[2] == CANARY).all()) and bool((o2[2] == CANARY).all()) and bool((states[2] == CANARY).all())
    for b in lanes:
        o, s, oa, sa = c.ref(before[read[b]], b)
        near(c.o[b], o, oa, 0, "o")
        near(o2[b], o, oa, 0, "o beside states")
        for t in range(T):
            near(states[b, t], s[t], sa[t], 0, f"state {t}")
    # decode into other slots, and none for lane 3
    write = c.write.clone()
    write[3] = -1
    o3 = torch.full_like(c.o, CANARY)
    gdn.gdn_linear_decode(c.q, c.k, c.v, c.ld, c.pool, c.read, o3, c.err, out_indices=write, scale=c.scale)
    touched = torch.zeros(c.slots, dtype=torch.bool)
    for b in lanes:
        o, s, oa, sa = c.ref(before[c.read[b]], b)
        near(o3[b], o, oa, 0, "decode o")
        if b != 3:
            touched[int(write[b])] = True
            near(c.pool[write[b]], s[-1], sa[-1], 0, "decode state")
    assert torch.equal(c.pool[~touched], before[~touched])
    # commit of prefixes in place: 0 leaves the slot
    c.pool.copy_(before)
    n = torch.tensor([0, max(1, T // 2), 1, T], **I32)
    gdn.gdn_linear_commit(c.k, c.v, c.ld, c.pool, c.read, n, c.err)
    assert torch.equal(c.pool[c.read[0]], before[c.read[0]])
    for b in (1, 3):
        _, s, _, sa = c.ref(before[c.read[b]], b)
        near(c.pool[c.read[b]], s[int(n[b]) - 1], sa[int(n[b]) - 1], 0, "commit")
    # and of none into another slot: a copy
    c.pool.copy_(before)
    gdn.gdn_linear_commit(c.k, c.v, c.ld, c.pool, c.read, torch.zeros(4, **I32), c.err, out_indices=c.write)
    assert torch.equal(c.pool[c.write[0]], before[c.read[0]]) and torch.equal(c.pool[c.read[0]], before[c.read[0]])
    assert int(c.err) == 0


def prompts(lens, HK, HV, DK, DV, io, state, seed=0, has=None, in_place=False, tail=3, log_decay=None, poison=True):
    B, N = len(lens), sum(lens) + tail
    c = Case((N,), B, HK, HV, DK, DV, io, state, seed, log_decay=log_decay)
    cu = torch.zeros(B + 1, dtype=torch.int64)
    cu[1:] = torch.cumsum(torch.tensor(lens), 0)
    if tail and poison:  # what lies behind the last prompt may be anything
        for x in (c.q, c.k, c.v):
            x[-tail:] = float("nan")
    has = torch.tensor([b % 3 != 1 for b in range(B)] if has is None else has).to(**I32)
    before = c.pool.clone()
    write = c.read if in_place else c.write
    ws = gdn.linear_prefill_workspace(N, B, HV, DK, DV)
    ws.fill_(255)
    gdn.gdn_linear_prefill(c.q, c.k, c.v, c.ld, c.pool, c.read, cu.to(**I32), c.o, ws, has, c.err,
                           out_indices=None if in_place else write, scale=c.scale)
    tensor = io == "bf16" and DK in (64, 128) and DV % 8 == 0
    touched = torch.zeros(c.slots, dtype=torch.bool)
    for b in range(B):
        S0 = before[c.read[b]] if int(has[b]) else torch.zeros_like(before[0])
        o, s, oa, sa = c.ref(S0, slice(int(cu[b]), int(cu[b + 1])))
        if lens[b] or not in_place:
            touched[int(write[b])] = True
        if lens[b]:
            near(c.o[cu[b]:cu[b + 1]], o, oa, 2.0 ** -8 if tensor else 0, f"o of prompt {b}")
            near(c.pool[write[b]], s[-1], sa[-1], (2.0 ** -16 if state == "bf16" else 2.0 ** -24) if tensor else 0, f"state {b}")
        elif not in_place:
            assert torch.equal(c.pool[write[b]], S0)
    assert torch.equal(c.pool[~touched], before[~touched])
    assert tail == 0 or bool((c.o[-tail:] == CANARY).all())
    assert int(c.err) == 0
    return c, cu, has, ws


@pytest.mark.parametrize("DK,DV,io,state", [(128, 128, "bf16", "bf16"), (128, 72, "bf16", "f32"), (64, 64, "bf16", "f32"), (64, 8, "bf16", "bf16"),
                                            (128, 200, "bf16", "f32"), (64, 33, "bf16", "bf16"), (32, 40, "bf16", "f32"), (256, 48, "bf16", "bf16"),
                                            (16, 16, "f32", "f32"), (128, 64, "f32", "bf16"), (64, 96, "f32", "f32")])
@pytest.mark.parametrize("in_place", [False, True])
def test_prompts(DK, DV, io, state, in_place):
    prompts([0, 1, 127, 128, 129, 5, 300], 2, 4, DK, DV, io, state, seed=DK + DV, in_place=in_place)


# few lanes and heads: prompts in pieces (of at least 512 tokens), whose states a first launch forms
@pytest.mark.parametrize("lens", [[1500], [1024], [700, 1900], [0, 2500], [1025, 3, 1400]])
@pytest.mark.parametrize("DK,state", [(128, "f32"), (64, "bf16")])
@pytest.mark.parametrize("in_place", [False, True])
def test_prompts_in_pieces(lens, DK, state, in_place):
    c, cu, has, ws = prompts(lens, 1, 1, DK, 64, "bf16", state, seed=sum(lens), in_place=in_place)
    assert ws.numel() > 0


@pytest.mark.parametrize("log_decay", [[0.0, -30.0], [-math.inf, -1e-3], [-200.0, 0.0]])
@pytest.mark.parametrize("lens", [[200, 64], [1300]])
def test_decays_of_all_sizes(log_decay, lens):
    prompts(lens, 1, 2, 64, 64, "bf16", "f32", seed=9, log_decay=log_decay)
    T = 10
    c = Case((2, T), 2, 1, 2, 64, 24, "bf16", "f32", seed=3, log_decay=log_decay)
    before = c.pool.clone()
    gdn.gdn_linear_decode(c.q, c.k, c.v, c.ld, c.pool, c.read, c.o, c.err, scale=c.scale)
    for b in range(2):
        o, s, oa, sa = c.ref(before[c.read[b]], b)
        near(c.o[b], o, oa, 0, "o")
        near(c.pool[c.read[b]], s[-1], sa[-1], 0, "state")


@pytest.mark.parametrize("what", ["v", "k", "q"])
@pytest.mark.parametrize("value", [math.inf, math.nan])
@pytest.mark.parametrize("kind", ["tensor", "fp32", "T5", "T14", "states", "old"])
def test_what_is_not_finite_does_not_reach_earlier_tokens(what, value, kind):
    """From token `at` on anything goes (for q: at that token alone); before it, and in the other prompt, nothing changes."""
    if kind in ("tensor", "fp32"):
        io, at, lens = ("bf16" if kind == "tensor" else "f32"), 150, [260, 140]
        c = Case((400,), 2, 1, 2, 64, 64, io, "f32", seed=5)
        cu = torch.tensor([0, 260, 400], **I32)
        ws = gdn.linear_prefill_workspace(400, 2, 2, 64, 64)

        def call():
            gdn.gdn_linear_prefill(c.q, c.k, c.v, c.ld, c.pool, c.read, cu, c.o, ws, None, c.err, out_indices=c.write, scale=c.scale)
            return c.o.clone()
        clean = call()
        getattr(c, what)[at, :, 3] = value
        got = call()
        assert torch.equal(got[260:], clean[260:])
        before, after = slice(0, at), slice(at + 1, 260)
    else:
        T = 14 if kind == "T14" else 5
        c = Case((1, T), 1, 1, 2, 16 if kind == "old" else 64, 24, "bf16", "f32", seed=6)
        states = torch.zeros((1, T, 2, 24, c.DK), device="cuda") if kind == "states" else None

        def call():
            gdn.gdn_linear_verify(c.q, c.k, c.v, c.ld, c.pool, c.read, c.o, states, c.err, scale=c.scale)
            return c.o[0].clone()
        clean, at = call(), 3
        getattr(c, what)[0, at, :, 3] = value
        got = call()
        before, after = slice(0, at), slice(at + 1, T)
    # the sums of a chunk with such a v are formed in another order, P rounded as before
    assert torch.allclose(got[before].float(), clean[before].float(), rtol=2.0 ** -7, atol=2.0 ** -6 if kind == "tensor" else 1e-5)
    assert bool(torch.isfinite(got[before]).all())
    if what == "q":
        assert torch.equal(got[after], clean[after])
    else:
        assert not bool(torch.isfinite(got[after]).all())


def test_errors_skip_the_lane():
    c = Case((5, 3), 5, 1, 2, 64, 32, seed=1)
    before = c.pool.clone()
    c.read[0], c.read[1] = c.slots, -2
    c.write[2] = c.slots
    gdn.gdn_linear_decode(c.q, c.k, c.v, c.ld, c.pool, c.read, c.o, c.err, out_indices=c.write)
    assert int(c.err) == gdn.ERRBIT_INDEX
    assert bool((c.o[:3] == CANARY).all()) and written(c.o[3:])
    assert int((c.pool != before).flatten(1).any(1).sum()) == 2
    for DK in (64, 16):
        c = Case((3, 3), 3, 1, 2, DK, 32, seed=1)
        before = c.pool.clone()
        gdn.gdn_linear_commit(c.k, c.v, c.ld, c.pool, c.read, torch.tensor([4, -1, 2], **I32), c.err)
        assert int(c.err) == gdn.ERRBIT_ACCEPT_LEN
        assert int((c.pool != before).flatten(1).any(1).sum()) == 1
        N = 40
        c = Case((N,), 4, 1, 2, DK, 32, seed=2)
        before = c.pool.clone()
        ws = gdn.linear_prefill_workspace(N, 4, 2, DK, 32)
        gdn.gdn_linear_prefill(c.q, c.k, c.v, c.ld, c.pool, c.read, torch.tensor([0, 10, 5, 20, N + 1], **I32), c.o, ws, None, c.err)
        assert int(c.err) == gdn.ERRBIT_SEQLEN  # prompts 1 (decreasing) and 3 (beyond N)
        assert bool((c.o[20:] == CANARY).all()) and written(c.o[:20])
        assert int((c.pool != before).flatten(1).any(1).sum()) == 2
        c.err.zero_()
        gdn.gdn_linear_prefill(c.q, c.k, c.v, c.ld, c.pool, torch.tensor([-1, c.slots, -5, -1], **I32), torch.tensor([0, 10, 15, 20, N], **I32), c.o, ws,
                               None, c.err)
        assert int(c.err) == gdn.ERRBIT_INDEX


def test_no_lanes_and_no_tokens():
    c = Case((0, 2), 0, 1, 2, 64, 32)
    gdn.gdn_linear_decode(c.q, c.k, c.v, c.ld, c.pool, c.read, c.o, c.err)
    gdn.gdn_linear_verify(c.q, c.k, c.v, c.ld, c.pool, c.read, c.o, None, c.err)
    gdn.gdn_linear_commit(c.k, c.v, c.ld, c.pool, c.read, torch.zeros(0, **I32), c.err)
    c = Case((0,), 2, 1, 2, 64, 32)
    before = c.pool.clone()
    ws = gdn.linear_prefill_workspace(0, 2, 2, 64, 32)
    cu, has = torch.zeros(3, **I32), torch.tensor([1, 0], **I32)
    gdn.gdn_linear_prefill(c.q, c.k, c.v, c.ld, c.pool, c.read, cu, c.o, ws, has, c.err)
    assert torch.equal(c.pool, before)
    gdn.gdn_linear_prefill(c.q, c.k, c.v, c.ld, c.pool, c.read, cu, c.o, ws, has, c.err, out_indices=c.write)
    assert torch.equal(c.pool[c.write[0]], before[c.read[0]]) and not bool(c.pool[c.write[1]].any())
    assert int(c.err) == 0


def test_offsets_beyond_32_bits():
    slots = 2200  # of 2^20 elements each
    c = Case((2, 2), 2, 8, 64, 128, 128, seed=4, slots=slots)
    c.read = torch.tensor([slots - 1, 2049], **I32)
    c.write = torch.tensor([2100, slots - 2], **I32)
    gdn.gdn_linear_decode(c.q, c.k, c.v, c.ld, c.pool, c.read, c.o, c.err, out_indices=c.write, scale=c.scale)
    for b in range(2):
        o, s, oa, sa = c.ref(c.pool[c.read[b]], b)
        near(c.o[b], o, oa, 0, "o")
        near(c.pool[c.write[b]], s[-1], sa[-1], 0, "state")
    q, k, v = c.q.flatten(0, 1), c.k.flatten(0, 1), c.v.flatten(0, 1)
    o = torch.zeros_like(v)
    ws = gdn.linear_prefill_workspace(4, 2, 64, 128, 128)
    gdn.gdn_linear_prefill(q, k, v, c.ld, c.pool, c.read, torch.tensor([0, 2, 4], **I32), o, ws, None, c.err, out_indices=c.write, scale=c.scale)
    for b in range(2):
        ro, s, oa, sa = c.ref(c.pool[c.read[b]], b)
        near(o[2 * b:2 * b + 2], ro, oa, 2.0 ** -8, "o")
        near(c.pool[c.write[b]], s[-1], sa[-1], 2.0 ** -16, "state")
    assert int(c.err) == 0


def test_verify_then_either_commit_and_steps_one_by_one():
    T = 6
    c = Case((3, T), 3, 2, 4, 128, 128, "bf16", "f32", seed=11)
    start = c.pool.clone()
    states = torch.zeros((3, T, 4, 128, 128), device="cuda")
    gdn.gdn_linear_verify(c.q, c.k, c.v, c.ld, c.pool, c.read, c.o, states, c.err, scale=c.scale)
    n = torch.tensor([2, 6, 1], **I32)
    gdn.gdn_commit(c.pool, c.read, states, n, c.err)
    kept = c.pool.clone()
    c.pool.copy_(start)
    gdn.gdn_linear_commit(c.k, c.v, c.ld, c.pool, c.read, n, c.err)
    assert torch.allclose(c.pool, kept, rtol=1e-5, atol=1e-5)
    c.pool.copy_(start)
    for t in range(T):
        o1 = torch.zeros((3, 1, 4, 128), dtype=torch.bfloat16, device="cuda")
        gdn.gdn_linear_decode(c.q[:, t:t + 1].contiguous(), c.k[:, t:t + 1].contiguous(), c.v[:, t:t + 1].contiguous(), c.ld, c.pool, c.read, o1,
                              c.err, scale=c.scale)
        assert torch.allclose(o1[:, 0].float(), c.o[:, t].float(), rtol=2.0 ** -7, atol=1e-4)
    assert torch.allclose(c.pool[c.read.long()], states[:, -1], rtol=1e-5, atol=1e-5)
    assert int(c.err) == 0


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_captured_replayed_and_on_another_stream(kind):
    if kind == "decode":
        c = Case((4, 3), 4, 1, 2, 128, 64, seed=8)

        def call(**kw):
            gdn.gdn_linear_decode(c.q, c.k, c.v, c.ld, c.pool, c.read, c.o, c.err, out_indices=c.write, scale=c.scale, **kw)
    else:
        c = Case((1500,), 1, 1, 1, 128, 64, seed=8)
        ws, cu = gdn.linear_prefill_workspace(1500, 1, 1, 128, 64), torch.tensor([0, 1500], **I32)

        def call(**kw):
            gdn.gdn_linear_prefill(c.q, c.k, c.v, c.ld, c.pool, c.read, cu, c.o, ws, None, c.err, out_indices=c.write, scale=c.scale, **kw)
    call()
    torch.cuda.synchronize()
    o, pool = c.o.clone(), c.pool.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    c.o.zero_()
    c.pool[c.write.long()] = 0
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.o, o) and torch.equal(c.pool, pool)
    side = torch.cuda.Stream()
    c.o.zero_()
    torch.cuda.synchronize()
    call(stream=side)
    side.synchronize()
    assert torch.equal(c.o, o) and int(c.err) == 0


@pytest.mark.parametrize("lens,in_pieces", [([500, 300], False), ([1500], True)])
def test_a_tile_that_never_lands(timeout_lib, monkeypatch, lens, in_pieces):  # noqa: F811
    """A test build leaves the first tiles unasked for: the waits run out, the call says so, and the library's own runs on."""
    N, B = sum(lens), len(lens)
    c = Case((N,), B, 1, 1 if in_pieces else 8, 128, 128, seed=2)
    cu = torch.zeros(B + 1, **I32)
    cu[1:] = torch.cumsum(torch.tensor(lens), 0)
    ws = gdn.linear_prefill_workspace(N, B, c.HV, 128, 128)

    def call():
        gdn.gdn_linear_prefill(c.q, c.k, c.v, c.ld, c.pool, c.read, cu, c.o, ws, None, c.err, out_indices=c.write, scale=c.scale)
        torch.cuda.synchronize()

    call()
    assert int(c.err) == 0
    good = c.o.clone()
    run_with(timeout_lib, monkeypatch, call)
    assert int(c.err) & gdn.ERRBIT_TIMEOUT
    c.err.zero_()
    call()
    assert int(c.err) == 0 and torch.equal(c.o, good)


STREAMED = [  # B, T, HK, HV, DK, DV, state: enough lanes for the streaming kernel
    (90, 8, 4, 8, 128, 128, "bf16"), (200, 1, 2, 6, 128, 72, "bf16"), (100, 3, 7, 7, 64, 136, "bf16"), (170, 5, 1, 4, 256, 48, "bf16"),
    (90, 7, 8, 8, 128, 128, "f32"), (156, 2, 2, 4, 64, 200, "f32"), (1000, 8, 1, 1, 64, 80, "bf16"), (40, 4, 16, 32, 128, 128, "bf16")]


def lanes_in_64_bits(c, S, T):
    """States and o's after 0 .. T tokens of all lanes at once, with the sums of absolute values."""
    rep = c.HV // c.HK
    q, k = c.q.double().repeat_interleave(rep, 2), c.k.double().repeat_interleave(rep, 2)
    v, g = c.v.double(), torch.exp(c.ld.double())[None, :, None, None]
    S, A = S.double(), S.double().abs()
    states, o = [(S, A)], []
    for t in range(T):
        S = g * S + v[:, t, :, :, None] * k[:, t, :, None, :]
        A = g * A + v[:, t, :, :, None].abs() * k[:, t, :, None, :].abs()
        states.append((S, A))
        o.append((c.scale * torch.einsum("bhij,bhj->bhi", S, q[:, t]), c.scale * torch.einsum("bhij,bhj->bhi", A, q[:, t].abs())))
    return states, [torch.stack(x, 1) for x in zip(*o)]


@pytest.mark.parametrize("B,T,HK,HV,DK,DV,state", STREAMED)
def test_steps_of_many_lanes(B, T, HK, HV, DK, DV, state):
    c = Case((B, T), B, HK, HV, DK, DV, "bf16", state, seed=B)
    g = torch.Generator().manual_seed(B)
    padded = (torch.rand(B, generator=g) < 0.2).cuda()
    padded[1], padded[-1] = True, False
    read, write = c.read.clone(), c.write.clone()
    read[padded] = -1
    before, live = c.pool.clone(), ~padded
    states, (o, oa) = lanes_in_64_bits(c, before[c.read.long()], T)
    gdn.gdn_linear_verify(c.q, c.k, c.v, c.ld, c.pool, read, c.o, None, c.err, scale=c.scale)
    assert torch.equal(c.pool, before) and bool((c.o[padded] == CANARY).all())
    near(c.o[live], o[live], oa[live], 0, "o")
    # decode into other slots, some lanes into none
    write[::7] = -1
    o2 = torch.full_like(c.o, CANARY)
    gdn.gdn_linear_decode(c.q, c.k, c.v, c.ld, c.pool, read, o2, c.err, out_indices=write, scale=c.scale)
    near(o2[live], o[live], oa[live], 0, "decode o")
    to = live & (write >= 0)
    touched = torch.zeros(c.slots, dtype=torch.bool, device="cuda")
    touched[write[to].long()] = True
    near(c.pool[write[to].long()], states[T][0][to], states[T][1][to], 0, "decode state")
    assert torch.equal(c.pool[~touched], before[~touched]) and bool((o2[padded] == CANARY).all())
    # commit of 0 .. T tokens in place
    c.pool.copy_(before)
    n = torch.randint(0, T + 1, (B,), generator=g).to(**I32)
    n[0], n[-1] = 0, T
    gdn.gdn_linear_commit(c.k, c.v, c.ld, c.pool, read, n, c.err)
    S = torch.stack([x[0] for x in states])[n.long(), torch.arange(B, device="cuda")]
    A = torch.stack([x[1] for x in states])[n.long(), torch.arange(B, device="cuda")]
    near(c.pool[c.read[live].long()], S[live], A[live], 0, "commit")
    still = torch.ones(c.slots, dtype=torch.bool, device="cuda")
    still[read[live & (n > 0)].long()] = False
    assert torch.equal(c.pool[still], before[still])
    # of none into other slots: copies
    c.pool.copy_(before)
    gdn.gdn_linear_commit(c.k, c.v, c.ld, c.pool, read, torch.zeros(B, **I32), c.err, out_indices=c.write)
    assert torch.equal(c.pool[c.write[live].long()], before[c.read[live].long()])
    assert int(c.err) == 0


def test_many_lanes_with_bad_indices_lengths_and_values():
    """Bad lanes are skipped and counted, good ones beside them get their results; what is not finite stays in its own rows and
    tokens, and behind a lane's accepted tokens it is not read."""
    B, T, HK, HV, DK, DV = 90, 6, 4, 8, 128, 128
    c = Case((B, T), B, HK, HV, DK, DV, seed=5)
    before = c.pool.clone()
    n = torch.full((B,), 3, **I32)
    c.k[7, 3:], c.v[7, 4:] = float("nan"), float("inf")  # behind the accepted tokens
    c.v[8, 2, 1, 5] = float("inf")
    c.k[9, 1, 0, 3] = float("-inf")
    states, (o, oa) = lanes_in_64_bits(c, before[c.read.long()], T)
    read = c.read.clone()
    read[3], read[4], n[5], n[6] = -2, c.slots, T + 1, -1
    gdn.gdn_linear_commit(c.k, c.v, c.ld, c.pool, read, n, c.err)
    assert int(c.err) == gdn.ERRBIT_INDEX | gdn.ERRBIT_ACCEPT_LEN
    got, (S, A) = c.pool[c.read.long()], states[3]
    for b in range(B):
        if b in (3, 4, 5, 6):
            assert torch.equal(got[b], before[c.read[b].long()])
        elif b in (8, 9):
            fine = torch.isfinite(S[b])
            assert torch.equal(torch.isfinite(got[b]), fine) and torch.equal(got[b][~fine].isnan(), S[b][~fine].isnan())
            assert torch.equal(got[b][~fine & ~S[b].isnan()].double(), S[b][~fine & ~S[b].isnan()])
            near(got[b][fine], S[b][fine], A[b][fine], 0, "beside what is not finite")
        else:
            near(got[b], S[b], A[b], 0, "commit")
    # verify: tokens before the one with an infinity are not touched by it, nor are the other rows
    c.err.zero_()
    c.pool.copy_(before)
    gdn.gdn_linear_verify(c.q, c.k, c.v, c.ld, c.pool, read, c.o, None, c.err, scale=c.scale)
    assert int(c.err) == gdn.ERRBIT_INDEX and bool((c.o[3:5] == CANARY).all())
    keep = torch.isfinite(o)
    keep[3:5] = False
    keep[[7, 9]] = False
    near(c.o[keep], o[keep], oa[keep], 0, "o")
    near(c.o[7, :3], o[7, :3], oa[7, :3], 0, "o in front of what is not finite")
    near(c.o[9, :1], o[9, :1], oa[9, :1], 0, "o in front of an infinite k")
    assert not bool(torch.isfinite(c.o[8, 2:, 1, 5]).any())


def test_many_lanes_twice_at_once_and_replayed():
    """Two streams at once, and a captured call whose pool changes between replays."""
    cases = [Case((128, 4), 128, 4, 8, 128, 128, seed=s) for s in (1, 2)]
    alone = []
    for c in cases:
        gdn.gdn_linear_verify(c.q, c.k, c.v, c.ld, c.pool, c.read, c.o, None, c.err, scale=c.scale)
        alone.append(c.o.clone())
        c.o.fill_(CANARY)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for c, s in zip(cases, streams):
            gdn.gdn_linear_verify(c.q, c.k, c.v, c.ld, c.pool, c.read, c.o, None, c.err, scale=c.scale, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(c.o, a) for c, a in zip(cases, alone))
    c = cases[0]
    start = c.pool.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_linear_decode(c.q, c.k, c.v, c.ld, c.pool, c.read, c.o, c.err, scale=c.scale)
    c.pool.copy_(start)
    for _ in range(3):
        graph.replay()
    replayed, o = c.pool.clone(), c.o.clone()
    c.pool.copy_(start)
    for _ in range(3):
        gdn.gdn_linear_decode(c.q, c.k, c.v, c.ld, c.pool, c.read, c.o, c.err, scale=c.scale)
    assert torch.equal(replayed, c.pool) and torch.equal(o, c.o) and int(c.err) == 0


def test_a_state_that_never_lands(timeout_lib, monkeypatch):  # noqa: F811
    c = Case((128, 4), 128, 4, 8, 128, 128, seed=3)

    def call():
        gdn.gdn_linear_verify(c.q, c.k, c.v, c.ld, c.pool, c.read, c.o, None, c.err, scale=c.scale)
        torch.cuda.synchronize()

    call()
    assert int(c.err) == 0
    good = c.o.clone()
    run_with(timeout_lib, monkeypatch, call)
    assert int(c.err) & gdn.ERRBIT_TIMEOUT
    c.err.zero_()
    call()
    assert int(c.err) == 0 and torch.equal(c.o, good)


def test_tensors_that_the_binding_refuses():
    c = Case((2, 2), 2, 1, 2, 64, 32)
    ok = (c.q, c.k, c.v, c.ld, c.pool, c.read, c.o)
    for at, bad in ((0, c.q.float()), (0, c.q[:, :, :, :32]), (1, c.k.transpose(0, 1)), (2, c.v[:, :1]), (3, c.ld.double()), (4, c.pool[0]),
                    (5, c.read.long()), (5, c.read[:1]), (6, c.o[:1]), (2, c.v.cpu())):
        args = list(ok)
        args[at] = bad
        with pytest.raises((ValueError, TypeError, gdn.GdnError)):
            gdn.gdn_linear_decode(*args)
    with pytest.raises((ValueError, TypeError)):
        gdn.gdn_linear_verify(*ok, torch.zeros((2, 2, 2, 32, 64), device="cuda"))
    with pytest.raises((ValueError, TypeError)):
        gdn.gdn_linear_decode(*ok, out_indices=c.read[:1])
    with pytest.raises(gdn.GdnError):
        gdn.gdn_linear_decode(*ok, scale=math.inf)


@pytest.mark.parametrize("B", [2, 31, 32, 33])
def test_prompts_of_many_lengths(B):
    """Up to 32 prompts are taken from the longest to the shortest: each is served once, equal and empty ones among them."""
    lens = [(b * 37) % 150 for b in range(B - 1)] + [260]
    if B > 4:
        lens[3] = lens[2] = 0
        lens[-2] = lens[0] = lens[1]
    prompts(lens, 1, 2, 64, 72, "bf16", "f32", seed=B)
    prompts([130] * B, 1, 1, 128, 64, "bf16", "bf16", seed=B)


def test_bad_prompts_between_good_ones_of_many_lengths():
    """Padded lanes and bad bounds keep their place in the order: the prompts beside them get their results."""
    lens = [100, 5, 300, 40, 129]
    c = Case((sum(lens),), 5, 1, 2, 64, 64, seed=9)
    cu = torch.zeros(6, dtype=torch.int64)
    cu[1:] = torch.cumsum(torch.tensor(lens), 0)
    ws = gdn.linear_prefill_workspace(sum(lens), 5, 2, 64, 64)
    before = c.pool.clone()
    c.read[1], c.read[3] = -1, c.slots
    gdn.gdn_linear_prefill(c.q, c.k, c.v, c.ld, c.pool, c.read, cu.to(**I32), c.o, ws, None, c.err, out_indices=c.write, scale=c.scale)
    assert int(c.err) == gdn.ERRBIT_INDEX
    for b in range(5):
        at = slice(int(cu[b]), int(cu[b + 1]))
        if b in (1, 3):
            assert bool((c.o[at] == CANARY).all()) and torch.equal(c.pool[c.write[b]], before[c.write[b]])
            continue
        o, s, oa, sa = c.ref(before[c.read[b]], at)
        near(c.o[at], o, oa, 2.0 ** -8, "o")
        near(c.pool[c.write[b]], s[-1], sa[-1], 2.0 ** -16, "state")
    # a bound beyond the tokens, and one that goes back
    c.err.zero_()
    c.read[1], c.read[3] = 0, 1
    cu[5], cu[1] = sum(lens) + 7, 200
    before = c.pool.clone()
    gdn.gdn_linear_prefill(c.q, c.k, c.v, c.ld, c.pool, torch.arange(5, **I32), cu.to(**I32), c.o, ws, None, c.err,
                           out_indices=torch.arange(5, 10, **I32), scale=c.scale)
    assert int(c.err) == gdn.ERRBIT_SEQLEN
    for b in (2, 3):
        o, s, oa, sa = c.ref(before[b], slice(int(cu[b]), int(cu[b + 1])))
        alone = max(0, 200 - int(cu[b]))  # by these bounds the first prompt has tokens 0 .. 199 too, so o there is of either
        near(c.o[int(cu[b]) + alone:int(cu[b + 1])], o[alone:], oa[alone:], 2.0 ** -8, "o")
        near(c.pool[5 + b], s[-1], sa[-1], 2.0 ** -16, "state")
    for b in (1, 4):
        assert torch.equal(c.pool[5 + b], before[5 + b])
