"""Linear attention where tokens or states are not finite, against the recurrence in 64 bits.  Tolerances are those of test_gpu_linear."""
import math

import pytest
import torch

import gated_deltanet_linear_mtp_gb300 as gdn
import linear_ref
from test_gpu_linear import I32, Case, near

pytestmark = pytest.mark.gpu
INF = math.inf


def where_finite(x, ref, A, extra, what):
    """x is finite where the recurrence's result is, and near it there."""
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(x), fine), what
    near(x[fine], ref[fine], A[fine], extra, what)


def recurrence(c, S0, tokens):
    """linear_ref.steps for some of the tokens, on the GPU (hundreds of steps take minutes on a host)."""
    return linear_ref.steps(S0, c.q[tokens], c.k[tokens], c.v[tokens], c.ld, c.scale)


def run_prompts(c, cu, has=None):
    ws = gdn.linear_prefill_workspace(c.q.shape[0], c.B, c.HV, c.DK, c.DV)
    ws.fill_(255)
    gdn.gdn_linear_prefill(c.q, c.k, c.v, c.ld, c.pool, c.read, torch.tensor(cu).to(**I32), c.o, ws, has, c.err, out_indices=c.write, scale=c.scale)
    assert int(c.err) == 0
    return ws


@pytest.mark.parametrize("DK,state", [(128, "bf16"), (128, "f32"), (64, "f32")])
@pytest.mark.parametrize("lens", [[200], [384], [946], [140, 300]])
def test_products_that_wait_long_for_the_chunk_before(DK, state, lens):
    """A chunk whose V is not finite takes a hundred microseconds for o, so that the products of the next wait beyond their first try: they and
    their arrivals are issued once all the same, and the call ends by itself, not by its waits' limit of some seconds."""
    N = sum(lens)
    cu = [sum(lens[:b]) for b in range(len(lens) + 1)]
    c = Case((N,), len(lens), 1, 2, DK, 64, "bf16", state, seed=N, log_decay=[-0.02, -0.3])
    before = c.pool.clone()
    for b in range(len(lens)):
        for first in range(cu[b], cu[b + 1], 256):  # every other chunk
            c.v[first + 5, :, (first - cu[b]) // 128] = INF
    run_prompts(c, cu)
    times = []
    for _ in range(3):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        c.pool.copy_(before)
        start.record()
        run_prompts(c, cu)
        end.record()
        end.synchronize()
        times.append(start.elapsed_time(end))
    assert max(times) < 500, times  # ms; the limit of one wait alone is about 16 s
    for b in range(len(lens)):
        o, s, oa, sa = recurrence(c, before[c.read[b]], slice(cu[b], cu[b + 1]))
        where_finite(c.o[cu[b]:cu[b + 1]], o, oa, 2.0 ** -8, f"o of prompt {b}")
        where_finite(c.pool[c.write[b]], s[-1], sa[-1], 2.0 ** -16 if state == "bf16" else 2.0 ** -24, f"state {b}")


@pytest.mark.parametrize("DK,state", [(128, "bf16"), (128, "f32"), (64, "bf16"), (64, "f32")])
@pytest.mark.parametrize("chunks", [(0, 1, 2, 3, 4, 5, 6), (0, 2, 4, 6), (1, 2, 4, 5), (0, 3, 4)])
def test_infinite_values_in_chunk_after_chunk(DK, state, chunks):
    """Each of these chunks has an infinity in a value dimension of its own: o of the others is served, of whole chunks by the copy out of shared
    memory, of these by the sum over their tokens."""
    L = 7 * 128 + 50
    for seed in range(2):
        c = Case((L,), 1, 1, 2, DK, 64, "bf16", state, seed=seed, log_decay=[-0.02, -0.3])
        before = c.pool.clone()
        for n in chunks:
            c.v[128 * n + 37 * (seed + 1), :, n] = INF
        run_prompts(c, [0, L])
        o, s, oa, sa = recurrence(c, before[c.read[0]], slice(0, L))
        where_finite(c.o, o, oa, 2.0 ** -8, "o")
        where_finite(c.pool[c.write[0]], s[-1], sa[-1], 2.0 ** -16 if state == "bf16" else 2.0 ** -24, "state")


def as_the_recurrence(x, ref, A, extra, what):
    """Infinities and NaN of a state are those of the recurrence, what is finite is near it."""
    assert torch.equal(x.isnan(), ref.isnan()), what
    assert torch.equal(torch.where(x.isinf(), x.double(), 0), torch.where(ref.isinf(), ref, 0)), what
    fine = torch.isfinite(ref)
    near(x[fine], ref[fine], A[fine], extra, what)


def put(c, what, at, before):
    """An infinity of each sign in v, in k (with a 0 of v beside it: NaN) or in a state."""
    if what == "v":
        c.v[at, :, 3], c.v[at + 1, :, 9] = INF, -INF
    elif what == "k":
        c.k[at, :, 5], c.v[at, :, 2] = -INF, 0.0
    elif what == "both":
        c.v[at, :, 3], c.k[at + 2, :, 7] = INF, INF
        c.v[at + 1, :, 3] = -INF  # meets the first: NaN where k has the same sign
    else:
        before[c.read.long(), :, 6, 4], before[c.read.long(), :, 7, 1] = INF, -INF
        c.pool.copy_(before)


@pytest.mark.parametrize("what", ["v", "k", "both", "state"])
@pytest.mark.parametrize("DK,state,io", [(128, "f32", "bf16"), (128, "bf16", "bf16"), (64, "f32", "bf16"), (64, "bf16", "bf16"), (32, "f32", "bf16"), (64, "f32", "f32")])
@pytest.mark.parametrize("lens,at", [([300], 20), ([300], 140), ([129, 260], 150), ([1400], 1100), ([1400], 200), ([1400], 1390), ([40], 37)])
def test_states_of_prompts_keep_infinities(what, DK, state, io, lens, at):
    """Whole prompts and prompts in pieces; heads that forget slowly, and at once (outside the tensor-core kernel not so soon that v times a
    power of g underflows beside an infinite k)."""
    N = sum(lens) + 3
    cu = [sum(lens[:b]) for b in range(len(lens) + 1)]
    tensor = io == "bf16" and DK >= 64
    c = Case((N,), len(lens), 1, 3, DK, 64, io, state, seed=at, log_decay=[-0.002, -0.9, -30.0 if tensor or what in ("v", "state") else -4.0])
    before = c.pool.clone()
    put(c, what, at, before)
    run_prompts(c, cu)
    for b in range(len(lens)):
        o, s, oa, sa = recurrence(c, before[c.read[b]], slice(cu[b], cu[b + 1]))
        as_the_recurrence(c.pool[c.write[b]], s[-1], sa[-1], (2.0 ** -16 if state == "bf16" else 2.0 ** -24) if tensor else 0, f"state {b}")
        where_finite(c.o[cu[b]:cu[b + 1]], o, oa, 2.0 ** -8 if tensor else 0, f"o of prompt {b}")


@pytest.mark.parametrize("what", ["v", "k", "both", "state"])
@pytest.mark.parametrize("B,T,DK,DV,state,io", [(2, 8, 128, 64, "f32", "bf16"), (2, 16, 128, 64, "bf16", "bf16"), (2, 7, 64, 24, "f32", "bf16"),
                                                (2, 9, 256, 32, "f32", "f32"), (300, 8, 128, 128, "bf16", "bf16"), (300, 5, 64, 128, "f32", "bf16")])
def test_states_of_steps_keep_infinities(what, B, T, DK, DV, state, io):
    c = Case((B, T), B, 1, 3, DK, DV, io, state, seed=T, log_decay=[-0.002, -0.9, -8.0 if what in ("v", "state") else -4.0])
    before, lane = c.pool.clone(), B // 2
    slots = c.read.clone()
    c.read = c.read[lane:lane + 1]
    flat = Case.__new__(Case)
    flat.__dict__.update(c.__dict__, q=c.q[lane], k=c.k[lane], v=c.v[lane])
    put(flat, what, 1, before)
    o, s, oa, sa = recurrence(flat, before[slots[lane]], slice(0, T))
    gdn.gdn_linear_verify(c.q, c.k, c.v, c.ld, c.pool, slots, c.o, None, c.err, scale=c.scale)
    where_finite(c.o[lane], o, oa, 0, "o of verify")
    states = torch.zeros((B, T, 3, DV, DK), dtype=c.pool.dtype, device="cuda")
    gdn.gdn_linear_verify(c.q, c.k, c.v, c.ld, c.pool, slots, c.o, states, c.err, scale=c.scale)
    where_finite(c.o[lane], o, oa, 0, "o beside states")
    for t in range(T):
        as_the_recurrence(states[lane, t], s[t], sa[t], 0, f"state after {t}")
    gdn.gdn_linear_decode(c.q, c.k, c.v, c.ld, c.pool, slots, c.o, c.err, out_indices=c.write, scale=c.scale)
    where_finite(c.o[lane], o, oa, 0, "o of decode")
    as_the_recurrence(c.pool[c.write[lane]], s[-1], sa[-1], 0, "state of decode")
    n = torch.full((B,), T - 1, **I32)
    gdn.gdn_linear_commit(c.k, c.v, c.ld, c.pool, slots, n, c.err, out_indices=c.write)
    as_the_recurrence(c.pool[c.write[lane]], s[T - 2], sa[T - 2], 0, "state of commit")
    others = torch.arange(B, device="cuda") != lane
    assert bool(torch.isfinite(c.pool[c.write[others].long()]).all()) and bool(torch.isfinite(c.o[others]).all()) and int(c.err) == 0


@pytest.mark.parametrize("kind", ["prompts", "pieces", "verify", "commit"])
def test_beside_streams_that_take_the_memory(kind):
    """Copies on other streams make tiles come late, beyond a wait's first try: results are those of a call alone, bit by bit."""
    if kind in ("prompts", "pieces"):
        lens = [2048, 130, 777, 1500] if kind == "prompts" else [6000]
        N = sum(lens)
        cu = torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)]).to(**I32)
        c = Case((N,), len(lens), 8 if kind == "prompts" else 1, 16 if kind == "prompts" else 2, 128, 128, "bf16", "bf16", seed=7)
        ws = gdn.linear_prefill_workspace(N, c.B, c.HV, c.DK, c.DV)

        def call():
            gdn.gdn_linear_prefill(c.q, c.k, c.v, c.ld, c.pool, c.read, cu, c.o, ws, None, c.err, out_indices=c.write, scale=c.scale)
    else:
        c = Case((128, 8), 128, 8, 16, 128, 128, seed=7)
        n = torch.full((128,), 5, **I32)

        def call():
            if kind == "verify":
                gdn.gdn_linear_verify(c.q, c.k, c.v, c.ld, c.pool, c.read, c.o, None, c.err, scale=c.scale)
            else:
                gdn.gdn_linear_commit(c.k, c.v, c.ld, c.pool, c.read, n, c.err, out_indices=c.write)
    call()
    torch.cuda.synchronize()
    o, pool = c.o.clone(), c.pool.clone()
    big = [torch.ones(1 << 28, device="cuda") for _ in range(4)]
    others = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, s in enumerate(others):
            with torch.cuda.stream(s):
                for _ in range(3):
                    big[2 * i].copy_(big[2 * i + 1])
        c.o.fill_(7.25)
        for _ in range(3):
            call()
        torch.cuda.current_stream().synchronize()
        assert torch.equal(c.pool, pool) and (kind == "commit" or torch.equal(c.o, o))
    torch.cuda.synchronize()
    assert int(c.err) == 0
