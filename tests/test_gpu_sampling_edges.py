"""Token probabilities and draft acceptance where one row is not sound: every such row in a call and with an error word of its own, so that no
other row can hide it.  Tolerances are those of test_gpu_sampling."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_linear_mtp_gb300 as gdn
import linear_ref
from test_gpu_sampling import Lanes, check_probs

pytestmark = pytest.mark.gpu
NAN, INF = math.nan, math.inf


def bad_rows(V):
    """Rows of V logits that hold NaN where what lies around it has no maximum of its own, by name."""
    g = torch.Generator().manual_seed(V)
    normal, last = torch.randn(V, generator=g), V - 1
    rows = {"NaN throughout": torch.full((V,), NAN)}
    for at in sorted({0, 1, V // 2, V - 2, last}):
        row = torch.full((V,), -INF)
        row[at] = NAN
        rows[f"NaN at {at} among -inf"] = row
        row = row.clone()
        row[(at + V // 3) % V] = 0.5  # V >= 3: another place
        rows[f"NaN at {at}, one logit elsewhere"] = row
        row = normal.clone()
        row[at] = NAN
        rows[f"NaN at {at} among logits"] = row
        row = normal.clone()
        row[max(0, at - 40):at + 41] = -INF  # whole pieces of 16 bytes, and the neighbouring threads'
        row[at] = NAN
        rows[f"NaN at {at} in a masked run"] = row
        row = torch.where(torch.rand(V, generator=g) < 0.999, torch.full((V,), -INF), normal)
        row[at] = NAN
        rows[f"NaN at {at}, nearly all masked"] = row
        row = normal.clone()
        row[at] = INF
        rows[f"inf at {at}"] = row
    return rows


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [3, 5, 19, 1000, 5000, 40003])
def test_a_row_that_holds_nan_is_zeros_and_told(dtype, V):
    for name, row in bad_rows(V).items():
        for first in (0, 1, 3):  # rows on and off 16 bytes: numbers in front of the first piece and behind the last are a thread's own
            x = torch.zeros((1, 1, V + 3), dtype=dtype, device="cuda")
            x[0, 0, first:first + V] = row.to(dtype)
            for T in (1.0, 0.0):
                try:
                    got = check_probs(x[..., first:first + V], torch.full((1,), T, device="cuda"), bits=gdn.ERRBIT_NONFINITE)
                except AssertionError as e:
                    raise AssertionError(f"{name}, first {first}, T {T}") from e
                assert not got.any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [20000, 40003])
def test_one_such_row_among_many(dtype, V):
    """Rows enough for one CTA each, or a few: a thread has more pieces than it has in flight.  Beside the bad row the others get their results."""
    B, at = 160, 77
    x = torch.randn((B, 1, V), generator=torch.Generator(device="cuda").manual_seed(V), device="cuda").to(dtype)
    temp = torch.full((B,), 0.8, device="cuda")
    temp[at + 1] = 0.0
    for places in ([0], [V - 1], [9000], range(0, V, 4096)):  # the first, the last, a middle piece of a thread, and its first in each round
        x[at, 0] = 1.0
        for p in places:
            x[at, 0, p // 8 * 8:p // 8 * 8 + 8] = -INF  # the piece around it
            x[at, 0, p] = NAN
        y, err = torch.full((B, 1, V), -3.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.gdn_token_probs(x, temp, y, err)
        assert int(err) == gdn.ERRBIT_NONFINITE
        assert not bool(y[at].any())  # NaN counts as anything
        sums = y.double().sum(-1).flatten()
        sums[at] = 1.0
        assert bool(((sums - 1).abs() <= 2.0 ** -16 + 2.0 ** -22 * 32).all())


@pytest.mark.parametrize("V", [7, 300, 5000, 40003])
@pytest.mark.parametrize("lanes", [1, 160])
def test_what_is_not_finite_in_a_row_of_acceptance_is_told(V, lanes):
    """One bad number in the row that the token comes from, of p or of q: it counts as nothing, and the bit says so."""
    for at in sorted({0, 1, V // 2, V - 1}):
        for value in (NAN, INF, -INF):
            for of in ("p", "q", "p after the last draft", "p alone"):
                x = Lanes(lanes, 1 if of == "p alone" else 2, V, True, 3)
                lane, row = lanes // 2, 0
                if of == "p after the last draft":
                    x.u[:, 0], row = 0.0, 1
                    x.p[lane, 0, int(x.drafts[lane, 0])] = 0.5  # 0 q < p: accepted
                elif of != "p alone":
                    x.u[lane, 0] = 1.0
                    x.p[lane, 0, int(x.drafts[lane, 0])] = 0.0  # refused
                (x.q if of == "q" else x.p)[lane, row, at] = value
                # u q(x) < p(x) holds for an infinite p(x) and for q(x) = -inf: accepted, and that row is not read
                accepted = at == int(x.drafts[lane, 0]) if x.T == 2 and (of, value) in (("p", INF), ("q", -INF)) else False
                x.check(bits=0 if accepted else gdn.ERRBIT_NONFINITE)


@pytest.mark.parametrize("V", [7, 5000, 40003])
def test_a_row_of_nothing_is_told(V):
    for T in (1, 2):
        x = Lanes(1, T, V, True, 2)
        x.p.zero_()
        x.check(bits=gdn.ERRBIT_NONFINITE)
        assert x.len.tolist() == [1] and int(x.tokens[0, 0]) == -1
    x = Lanes(1, 2, V, False, 2)
    x.p[0, 0] = NAN
    x.check(bits=gdn.ERRBIT_NONFINITE)
    assert int(x.tokens[0, 0]) == -1


@pytest.mark.parametrize("V", [7, 5000, 40003])
def test_what_is_not_read_is_not_told(V):
    """Rows in front of the token's own and behind it may hold anything but at the drafts."""
    x = Lanes(1, 4, V, True, 4)
    x.u[:, :2] = 0.0  # accepted while p(x) > 0
    x.u[:, 2] = 1.0
    d = x.drafts[0].tolist()
    keep = [float(x.p[0, t, d[t]]) for t in range(2)]
    x.p[0, :2] = NAN
    x.q[0, :2] = INF
    x.p[0, 3] = NAN
    for t in range(2):
        x.p[0, t, d[t]], x.q[0, t, d[t]] = keep[t], 0.5
    x.p[0, 2, d[2]] = 0.0  # refused
    x.check()
    assert x.len.tolist() == [3]


def test_the_oracle_of_acceptance_by_hand():
    p = np.array([[0.5, np.nan, 0.25], [0.2, 0.3, 0.5]], np.float32)
    q = np.array([[0.125, 0.5, np.inf]], np.float32)
    assert linear_ref.accept(p, q, [1], [0.5, 0.0]) == (1, [0, -1])  # NaN is refused, 1 and 2 count as nothing
