"""Token probabilities and draft acceptance on the GPU, against 64-bit arithmetic, and a speculative step of a linear-attention layer
through all of them.

Tolerance of a probability, from the arithmetic: the exponent e (in powers of two) of a weight is rounded with its constant to 2^-23 |e|, which
is 2^-23 |e| ln 2 of the weight; the exponential adds 2^-22, a sum of up to 2^18 terms (512 threads a run, at most 64 additions of 8 or 16
a thread, then trees) 2^-17: 2^-16 + 2^-22 |e| relative, and what is below 2^-126 may be 0.  Accepted drafts and tokens are equal."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_linear_mtp_gb300 as gdn
import linear_ref

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")
CANARY = -3.0


def check_probs(x, temp, bits=0, out=None):
    """One call on logits x [B, T, V] (any strides a call takes); the error word it leaves."""
    B, T, V = x.shape
    wide = torch.full((B, T, V + 5), CANARY, device="cuda") if out is None else out
    y, err = wide[..., :V], torch.zeros(1, **I32)
    gdn.gdn_token_probs(x, temp, y, err)
    assert int(err) == bits
    got, xs, ts = y.double().cpu().numpy(), x.double().cpu().numpy(), temp.double().cpu().numpy()
    for b in range(B):
        for t in range(T):
            ref, e = linear_ref.softmax(xs[b, t], ts[b])
            tol = ref * (2.0 ** -16 + 2.0 ** -22 * e) + 2.0 ** -126
            assert np.all(np.abs(got[b, t] - ref) <= tol), (b, t, float(np.max(np.abs(got[b, t] - ref) / tol)))
    assert out is not None or bool((wide[..., V:] == CANARY).all())
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (2, 3, 2), (3, 1, 7), (2, 2, 1000), (1, 4, 4097), (5, 2, 8192), (1, 1, 50001), (40, 4, 33000), (1, 2, 131075),
                                   (1, 1, 300000)])
def test_probs(dtype, B, T, V):
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (3 * torch.randn((B, T, V + 3), generator=g, device="cuda")).to(dtype)
    temp = torch.linspace(0.2, 1.5, B, device="cuda")
    if B > 2:
        temp[1] = 0.0
    for first in (0, 1):  # rows on and off 16 bytes
        check_probs(x[..., first:first + V], temp)
    check_probs(x[..., :V].contiguous(), temp, out=torch.zeros((B, T, V), device="cuda"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [9, 5000, 70001])
def test_probs_of_masked_and_strange_rows(dtype, V):
    g = torch.Generator(device="cuda").manual_seed(V + 1)
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    rows = torch.randn((12, V), generator=g, device="cuda")
    at = V // 2
    rows[0, torch.rand(V, generator=g, device="cuda") < 0.9] = -math.inf
    rows[1] = -math.inf                  # nothing is allowed: zeros
    rows[2, :at], rows[2, at:] = -math.inf, low   # the rest is the type's lowest: even
    rows[3] = low
    rows[3, at] = 1.0                    # one real logit among the lowest
    rows[4] = 0.0                        # all equal
    rows[5] = 1e30 * torch.sign(rows[5])  # beyond the fast path's offsets
    rows[6] = high
    rows[7] = -1e7 + rows[7]
    rows[8] = -math.inf
    rows[8, V - 1] = -5.0                # a single token
    rows[9] = rows[9] * 1e4
    rows[10], rows[11] = low, rows[11] - 60.0
    rows[10, 0] = -math.inf
    x = rows.to(dtype)[:, None]
    for T in (0.7, 0.0, 2.0, 1e-3):
        check_probs(x, torch.full((12,), T, device="cuda"))
    # the first of the largest
    y = torch.zeros((1, 1, V), dtype=dtype, device="cuda")
    y[0, 0, [3, V - 2]] = 2.0
    assert int(check_probs(y, torch.zeros(1, device="cuda")).argmax()) == 3


@pytest.mark.parametrize("V", [5, 40000])
def test_probs_that_cannot_be(V):
    x = torch.randn((6, 1, V), device="cuda")
    x[0, 0, 1], x[1, 0, V - 1], x[2] = math.nan, math.inf, -math.inf
    x[2, 0, 2] = math.nan
    temp = torch.tensor([1.0, 1.0, 1.0, -1.0, math.nan, math.inf], device="cuda")
    assert not check_probs(x, temp, bits=gdn.ERRBIT_NONFINITE).any()
    temp = torch.tensor([0.0, 0.0, 0.0, 1e-39, 1e-37, 3e38], device="cuda")
    got = check_probs(x, temp, bits=gdn.ERRBIT_NONFINITE)
    assert not got[:3].any() and abs(got[3:].sum() - 3) < 1e-3


class Lanes:
    def __init__(self, B, T, V, probs, seed=0, peak=2.0, pad=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        x = peak * r(B, T, V)
        y = x[:, :T - 1] + 0.8 * r(B, T - 1, V)
        wide = torch.full((B, T, V + pad), math.nan, device="cuda")
        wide[..., :V] = torch.softmax(x, -1)
        self.p, self.q = wide[..., :V], torch.softmax(y, -1)
        race = torch.rand((B, T - 1, V), generator=g, device="cuda").clamp(min=1e-6).log().neg()
        self.drafts = ((self.q / race) if probs else y).argmax(-1).to(torch.int32) if T > 1 else torch.zeros((B, 0), **I32)
        if not probs:
            self.q = None
        self.u = torch.rand((B, T), generator=g, device="cuda")
        self.index = torch.arange(B, **I32)
        self.len, self.tokens, self.err = torch.full((B,), 99, **I32), torch.full((B, T), 99, **I32), torch.zeros(1, **I32)
        self.B, self.T, self.V = B, T, V

    def call(self, **kw):
        gdn.gdn_draft_accept(self.p, self.drafts, self.u, self.index, self.len, self.tokens, self.q, self.err, **kw)

    def check(self, bits=0):
        self.call()
        assert int(self.err) == bits
        p, d, u = self.p.cpu().numpy(), self.drafts.cpu().numpy(), self.u.cpu().numpy()
        q = None if self.q is None else self.q.cpu().numpy()
        for b in range(self.B):
            if self.index is not None and int(self.index[b]) < 0:
                assert int(self.len[b]) == 99 and bool((self.tokens[b] == 99).all())
                continue
            n, tokens = linear_ref.accept(p[b], None if q is None else q[b], d[b], u[b])
            assert int(self.len[b]) == n and self.tokens[b].tolist() == tokens, (b, n, tokens, int(self.len[b]), self.tokens[b].tolist())


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("B,T,V", [(3, 1, 1), (4, 2, 2), (5, 4, 31), (8, 16, 257), (20, 3, 2049), (9, 5, 10007), (2, 4, 131073), (300, 2, 5000), (1, 2, 2200001)])
def test_accept(B, T, V, probs):
    for seed in range(3 if V < 1e5 else 1):
        x = Lanes(B, T, V, probs, seed, pad=seed)
        if B > 2:
            x.index[1] = -1
        x.check()
        x.index = None
        x.check()


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("B,T,V", [(151, 2, 9001), (160, 3, 40000), (512, 2, 20001), (1100, 1, 9000)])
def test_accept_of_many_lanes(B, T, V, probs):
    """Lanes that fill the GPU: smaller CTAs, one, two or four a lane."""
    test_accept(B, T, V, probs)


def test_accept_flat_and_peaked():
    """Flat probabilities put every threshold next to a border; a row of one token has one."""
    for seed in range(4):
        Lanes(64, 2, 65536, True, seed, peak=0.0).check()
    x = Lanes(6, 3, 1000, True, 1, peak=300.0)
    x.check()


def test_numbers_at_the_ends():
    for u in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, math.nan):
        x = Lanes(6, 3, 4000, True, 5)
        x.u[:, -1] = u
        if u == u and u < 1:
            x.u[0, 0] = u
        x.p[2, :, 3990:] = 0.0  # the last tokens have nothing
        x.p[3, :, :10] = 0.0    # nor the first
        x.check()


def test_fewer_drafts_and_wrong_ones():
    x = Lanes(5, 4, 300, True, 2)
    x.u[:, :3] = 0.0  # every draft that may be is accepted
    x.drafts[0, 0], x.drafts[1, 1], x.drafts[2, 2] = -1, -1, -1
    x.check()
    assert x.len.tolist()[:3] == [1, 2, 3]
    x.drafts[3, 1], x.drafts[4, 0] = 300, -7
    x.check(bits=gdn.ERRBIT_INDEX)
    assert x.len.tolist() == [1, 2, 3, 2, 1]
    x = Lanes(3, 2, 300, False, 2)
    x.index[0], x.index[2] = -4, -1
    x.check(bits=gdn.ERRBIT_INDEX)


def test_rows_without_anything_left():
    x = Lanes(5, 3, 5000, True, 3)
    x.u[:, 0] = 1.0
    x.q[0, 0] = x.p[0, 0]   # p - q is nothing: the token comes from p
    x.q[1, 0] = 2 * x.p[1, 0]
    x.p[2, 0] = 0.0         # the row itself is nothing
    x.p[3, 0, 7], x.q[3, 0, 9] = math.nan, math.inf
    x.p[4, 0, ::2] = 0.0
    x.check(bits=gdn.ERRBIT_NONFINITE)
    assert int(x.tokens[2, 0]) == -1
    y = Lanes(2, 2, 50, False, 3)
    y.u[:, 0] = 1.0
    y.p[0, 0] = 0.0
    y.p[0, 0, int(y.drafts[0, 0])] = 1.0  # certain of the draft, which u = 1 refuses all the same
    y.check()
    assert int(y.tokens[0, 0]) == int(y.drafts[0, 0])


def test_shapes_that_the_binding_refuses():
    x = Lanes(2, 3, 40, True)
    ok = [x.p, x.drafts, x.u, x.index, x.len, x.tokens, x.q]
    for at, bad in ((0, x.p.double()), (0, x.p.transpose(1, 2)), (0, x.p[:, ::2]), (1, x.drafts[:, :1]), (1, x.drafts.long()), (2, x.u[:, :2]),
                    (3, x.index[:1]), (4, x.len[:1]), (5, x.tokens[:, :2]), (6, x.q[:, :1])):
        args = list(ok)
        args[at] = bad
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_draft_accept(*args)
    y = torch.zeros((2, 3, 40), device="cuda")
    for args in ((y.half(), x.u[:, 0], y), (y, x.u[:, 0].double(), y), (y, x.u[:1, 0], y), (y, x.u[:, 0].contiguous(), y[:, :1]), (y[0], x.u[:, 0], y)):
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_token_probs(*args)


def test_no_lanes():
    gdn.gdn_token_probs(torch.zeros((0, 2, 9), device="cuda"), torch.zeros(0, device="cuda"), torch.zeros((0, 2, 9), device="cuda"))
    Lanes(0, 2, 9, True).call()


@pytest.mark.parametrize("captured", [False, True])
def test_a_speculative_step(captured):
    """Drafts through a linear-attention layer, logits of its outputs, probabilities, acceptance, and the commit of what was accepted:
    the states are those of the accepted tokens."""
    B, T, HK, HV, D, V = 6, 4, 1, 2, 64, 997
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, k, v = r(B, T, HK, D).bfloat16(), r(B, T, HK, D).bfloat16(), r(B, T, HV, D).bfloat16()
    ld, pool = -torch.tensor([0.5, 0.05], device="cuda"), r(B + 2, HV, D, D)
    head = (r(HV * D, V) / 8).bfloat16()
    index = torch.tensor([3, 1, -1, 0, 6, 5], **I32)
    temp = torch.tensor([0.8, 0.0, 1.0, 1.2, 0.5, 0.0], device="cuda")
    drafts, u = torch.randint(0, V, (B, T - 1), generator=g, device="cuda").to(torch.int32), torch.rand((B, T), generator=g, device="cuda")
    o, probs = torch.zeros((B, T, HV, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((B, T, V), device="cuda")
    n, tokens, err = torch.zeros(B, **I32), torch.zeros((B, T), **I32), torch.zeros(1, **I32)
    start = pool.clone()

    def step():
        gdn.gdn_linear_verify(q, k, v, ld, pool, index, o, None, err, scale=D ** -0.5)
        gdn.gdn_token_probs(o.flatten(2) @ head, temp, probs, err)
        gdn.gdn_draft_accept(probs, drafts, u, index, n, tokens, None, err)
        gdn.gdn_linear_commit(k, v, ld, pool, index, n, err)

    step()
    # half of the drafts become what the target would take, so that some are accepted
    best = probs[:, :T - 1].argmax(-1).to(torch.int32)
    drafts.copy_(torch.where(torch.rand((B, T - 1), generator=g, device="cuda") < 0.7, best, drafts))
    pool.copy_(start)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        pool.copy_(start)
        graph.replay()
    else:
        step()
    torch.cuda.synchronize()
    assert int(err) == 0
    p, d, un = probs.cpu().numpy(), drafts.cpu().numpy(), u.cpu().numpy()
    for b in range(B):
        if int(index[b]) < 0:
            assert int(n[b]) == 0
            continue
        want, tk = linear_ref.accept(p[b], None, d[b], un[b])
        assert int(n[b]) == want and tokens[b].tolist() == tk
        _, s, _, sa = linear_ref.steps(start[index[b]].cpu(), q[b, :want].cpu(), k[b, :want].cpu(), v[b, :want].cpu(), ld.cpu(), 1.0)
        assert bool(((pool[index[b]].double().cpu() - s[-1]).abs() <= 2.0 ** -15 * sa[-1]).all())


def test_clusters_captured_replayed_and_on_another_stream():
    """Rows that several CTAs share, in a graph and on a side stream."""
    x, te = 3 * torch.randn((3, 2, 60001), device="cuda"), torch.tensor([0.7, 0.0, 1.1], device="cuda")
    y = torch.zeros_like(x)
    lanes = Lanes(3, 3, 60001, True, 4)
    gdn.gdn_token_probs(x, te, y)
    lanes.check()
    want, n, tokens = y.clone(), lanes.len.clone(), lanes.tokens.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_token_probs(x, te, y)
        lanes.call()
    for side in (None, torch.cuda.Stream()):
        y.zero_()
        lanes.len.zero_()
        lanes.tokens.zero_()
        torch.cuda.synchronize()
        if side is None:
            graph.replay()
            graph.replay()
        else:
            gdn.gdn_token_probs(x, te, y, stream=side)
            lanes.call(stream=side)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(lanes.len, n) and torch.equal(lanes.tokens, tokens)


def test_from_other_threads():
    """As a thread's first CUDA call, and from two at once."""
    import threading

    from test_gpu_threads import in_thread

    lanes = [Lanes(4, 3, 30011, True, s) for s in range(2)]
    xs = [torch.randn((2, 2, 9000 + s), device="cuda") for s in range(2)]
    ys, te = [torch.zeros_like(x) for x in xs], torch.ones(2, device="cuda")
    q, k, v = (torch.randn((300, 1, 64), device="cuda").bfloat16() for _ in range(3))
    ld, pools, cu = torch.tensor([-0.1], device="cuda"), [torch.zeros((1, 1, 64, 64), device="cuda") for _ in range(3)], torch.tensor([0, 300], **I32)
    os_ = [torch.zeros_like(v) for _ in range(3)]
    index = torch.zeros(1, **I32)

    def work(i):
        ws = gdn.linear_prefill_workspace(300, 1, 1, 64, 64)
        gdn.gdn_linear_prefill(q, k, v, ld, pools[i], index, cu, os_[i], ws)
        gdn.gdn_token_probs(xs[i % 2], te, ys[i % 2])
        lanes[i % 2].call()

    in_thread(lambda: work(2))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(os_[i], os_[2]) and torch.equal(pools[i], pools[2]) and bool(os_[i].any())
        check_probs(xs[i], te)
        lanes[i].check()
