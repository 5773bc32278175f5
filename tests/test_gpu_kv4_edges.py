"""The attention-layer calls over the 4-bit cache at the edges of their ranges: tiles of rows that whole tokens do not fill,
launch limits of the page plan, intervals of the store's rounding around zero, values at the ends of the types, and
long contexts.  References and bounds are those of tests/kv4_ref.py unless a test derives its own."""
from __future__ import annotations

import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import gated_deltanet_linear_mtp_gb300 as gdn
import kv4_ref as ref
from test_gpu_kv4 import I32, attend, check_attend, check_rotated, check_store, err_word, f64, pool

pytestmark = pytest.mark.gpu


# ---- tiles of rows ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [3, 5, 6, 7, 12, 40])
def test_attention_row_tiles_that_whole_tokens_do_not_fill(D, G):
    """G heads a key head where G does not divide a tile of 128 or 256 rows.  Lane b's first row tile (b even; its second, b odd)
    ends with a token whose keys fill its tiles of 64 or 128 keys, so that the next token's own key lies in a further one."""
    rng = np.random.default_rng(D * 100 + G)
    tt = (128 if D == 256 else 256) // G
    qlens = [2 * tt + 1, 3 * tt, 2 * tt + max(1, tt // 2)]
    kvlens = [n + (-(1 + b % 2) * tt) % 128 + 128 * b for b, n in enumerate(qlens)]
    r = attend(rng, qlens, kvlens, G, 1, D, 32)
    check_attend(r)
    o, lse = r["o"].clone(), r["lse"].clone()
    for _ in range(4):
        r["o"].fill_(5.0)
        r["lse"].fill_(5.0)
        r["call"]()
        assert torch.equal(r["o"], o) and torch.equal(r["lse"], lse)


# ---- page plan -----------------------------------------------------------------------------------------------------
def plan_of_ones(B):
    """A plan of B lanes without a token that bring one each, its call's arguments, and the slots that it gives."""
    plan = gdn.PagePlan(*(torch.full((n,), -9, **I32) for n in (B + 1, B, B, B, B, 1)))
    args = (torch.zeros(B, **I32), torch.ones(B, **I32), 16, torch.full((B, 2), -1, **I32), torch.zeros(B, **I32),
            torch.arange(B, **I32), torch.zeros(1, **I32), plan, torch.zeros(1, **I32))
    return plan, args, torch.arange(0, 16 * B, 16, **I32)


def test_page_plan_on_the_stream_of_another_thread():
    """A stream that a second thread makes (its handle lies beyond 32 bits), as the current one and as an argument, and a graph."""
    failed = []

    def work():
        try:
            s = torch.cuda.Stream()
            for given in (None, s):
                with torch.cuda.stream(s if given is None else torch.cuda.default_stream()):
                    plan, args, want = plan_of_ones(300)
                torch.cuda.synchronize()
                with torch.cuda.stream(s if given is None else torch.cuda.default_stream()):
                    gdn.gdn_page_plan(*args, stream=given)
                s.synchronize()
                assert torch.equal(plan.slot_map, want)
            plan, args, want = plan_of_ones(40)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                gdn.gdn_page_plan(*args)
            assert (plan.slot_map == -9).all()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(plan.slot_map, want)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not failed, failed


PLAN_SIZES = """
import sys
sys.path.insert(0, "tests")
import torch
import gated_deltanet_linear_mtp_gb300 as gdn
from test_gpu_kv4_edges import plan_of_ones
for B in range(2440, 2462):  # ascending, in a process that has made no larger call
    plan, args, want = plan_of_ones(B)
    gdn.gdn_page_plan(*args)
    assert torch.equal(plan.slot_map, want), B
print("sizes ok")
"""


def test_page_plan_sizes_around_the_default_shared_memory():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", PLAN_SIZES], capture_output=True, text=True, cwd=root, timeout=300)
    assert p.returncode == 0 and "sizes ok" in p.stdout, p.stdout + p.stderr


def test_page_plan_of_two_sizes_from_two_threads():
    """Each thread plans on its own stream and buffers, one with little shared memory and one with much; the library is called
    directly, so that the calls meet."""
    failed, start = [], threading.Barrier(2)

    def work(B):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            plan, a, want = plan_of_ones(B)
        s.synchronize()
        args = (B, B, 16, 2, B, *(x.data_ptr() for x in (a[0], a[1], a[3], a[4], a[5], a[6])), plan.ref, a[8].data_ptr(), None, s.cuda_stream)
        call = gdn.lib().gdn_page_plan
        start.wait()
        for _ in range(20000):
            status = call(*args)
            if status != 0:
                failed.append((B, status))
                break
        s.synchronize()
        if not torch.equal(plan.slot_map, want):
            failed.append((B, "slots"))

    threads = [threading.Thread(target=work, args=(B,)) for B in (2600, 8192)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("N", [0, 1, 5000])
@pytest.mark.parametrize("inplace", [False, True])
def test_page_plan_of_no_lanes(N, inplace):
    """A step without lanes leaves nothing of an earlier step in its buffers."""
    taken = torch.full((1,), 2, **I32)
    plan = gdn.PagePlan(torch.full((1,), 9, **I32), torch.full((N,), 9, **I32), torch.full((N,), 9, **I32), torch.zeros(0, **I32),
                        torch.zeros(0, **I32), taken if inplace else torch.full((1,), 9, **I32))
    ticket, err, none = torch.zeros(1, **I32), err_word(), torch.zeros(0, **I32)
    gdn.gdn_page_plan(none, none, 16, torch.zeros((0, 4), **I32), none, torch.arange(7, **I32), taken, plan, ticket, err)
    assert plan.cu_seqlens.tolist() == [0] and not plan.positions.any() and (plan.slot_map == -1).all()
    assert int(plan.taken) == 2 and int(ticket) == 0 and int(err) == 0


# ---- the store's codes -----------------------------------------------------------------------------------------
def store_keys(k, kw, pos, freq, k_scale=1.0, eps=1e-6, inter=False, v=None, v_scale=1.0):
    """The keys (and values) of k [N, HK, D] stored at slots 0 .. N - 1 -> (cache, slots, error bits)."""
    N, HK, D = k.shape
    cache, slots, err = pool(-(-N // 16), HK, 16, D, k_scale, v_scale), np.arange(N, dtype=np.int32), err_word()
    q = torch.ones((N, 1, D), dtype=k.dtype, device="cuda")
    gdn.gdn_qk_norm_rope(q, k, kw, kw, pos, freq, torch.empty_like(q), v=k if v is None else v, cache=cache,
                         slot_map=torch.tensor(slots, **I32), err_word=err, eps=eps, interleaved=inter)
    return cache, slots, int(err)


@pytest.mark.parametrize("exponent", [-8, -7])
def test_keys_whose_interval_of_rounding_holds_zero(exponent):
    """A number that is 0 but for the rounding of its far larger partner, which lies in another group, beside numbers so small
    that this rounding passes their group's borders."""
    small = np.geomspace(1e-6, 3e-5, 64)
    x = np.zeros((len(small), 1, 128), np.float32)
    x[:, 0, 0] = small
    x[:, 0, 65] = x[:, 0, 70] = 1.0
    k = torch.tensor(x).cuda()
    w, freq = torch.ones(128, device="cuda"), torch.tensor(1e4 ** (-np.arange(0, 128, 2) / 128), dtype=torch.float32).cuda()
    for at in (0, 12345):
        pos = torch.full((len(small),), at, **I32)
        cache, slots, bits = store_keys(k, w, pos, freq, 2.0 ** exponent)
        want = ref.norm_rope(f64(k), f64(w), pos.cpu().numpy(), f64(freq), float(np.float32(1e-6)), False)[0]
        check_store(cache, slots, 0, want, 2.0 ** exponent)
        assert bits == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
def test_keys_of_many_magnitudes(dtype, inter):
    """Numbers of one row over eight decades, a third of them 0, at cache scales down to their smallest."""
    rng = np.random.default_rng(21)
    for D, R in ((64, 64), (128, 64), (256, 256)):
        x = rng.normal(size=(300, 2, D)) * 10.0 ** rng.uniform(-8, 0, size=(300, 2, D)) * (rng.random((300, 2, D)) > 0.33)
        k = torch.tensor(x, dtype=torch.float32).to(dtype).cuda()
        w = torch.tensor(1 + 0.2 * rng.normal(size=D), dtype=torch.float32).cuda()
        freq = torch.tensor(1e4 ** (-np.arange(0, R, 2) / R), dtype=torch.float32).cuda()
        pos = torch.tensor(rng.integers(0, 100000, 300) * (rng.random(300) > 0.3), **I32)
        for e in (0, -6, -10, -16):
            cache, slots, bits = store_keys(k, w, pos, freq, 2.0 ** e, inter=inter)
            want = ref.norm_rope(f64(k), f64(w), pos.cpu().numpy(), f64(freq), float(np.float32(1e-6)), inter)[0]
            check_store(cache, slots, 0, want, 2.0 ** e)
            assert bits == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("exponent", [-32, -20, -9, -8, 0, 32])
def test_values_beyond_the_cache_keep_their_sign(dtype, exponent):
    """Infinities, and finite numbers whose quotient by the scale passes the type, are held as the largest number of their sign."""
    v = torch.zeros((4, 1, 64), dtype=dtype, device="cuda")
    v[0, 0, :4] = torch.tensor([float("-inf"), float("inf"), -3e38, 1.0])
    v[1, 0, :4] = torch.tensor([-3e38, 3e38, -1e30, -1.0])
    v[2, 0, 16:20] = torch.tensor([-1e10, 1e10, 5.0, float("-inf")])
    v[3, 0, 40:44] = torch.tensor([-1e10, 3e10, -2e10, -2.5])
    k, w = torch.ones((4, 1, 64), dtype=dtype, device="cuda"), torch.ones(64, device="cuda")
    cache, slots, bits = store_keys(k, w, torch.zeros(4, **I32), torch.zeros(0, device="cuda"), v=v, v_scale=2.0 ** exponent)
    with np.errstate(over="ignore"):
        check_store(cache, slots, 1, f64(v), 2.0 ** exponent)
    assert bits == gdn.ERRBIT_NONFINITE


# ---- rows whose squares leave fp32 -----------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-33, 1e-6])
@pytest.mark.parametrize("D,R,inter", [(64, 32, False), (128, 128, True), (256, 64, False)])
def test_rows_whose_squares_leave_the_type(dtype, eps, D, R, inter):
    """Rows whose sum of squares is beyond fp32 or below its normal numbers are normed, rotated and stored like others."""
    rng = np.random.default_rng(D)
    size = np.array([3e37, 1e30, 2e19, 1e10, 1.0, 1e-15, 1e-19, 1e-23, 1e-30, 1e-37, 4e-40])
    x = rng.normal(size=(len(size), 2, D)) * size[:, None, None]
    x[2, 1] *= rng.random(D) > 0.9  # beside numbers of another size
    x[2, 1, 5] = 1e38
    x[8, 1, ::3] = 1e-38
    k = torch.tensor(x, dtype=torch.float32).to(dtype).cuda()
    w = torch.tensor(1 + 0.2 * rng.normal(size=D), dtype=torch.float32).cuda()
    freq = torch.tensor(1e4 ** (-np.arange(0, R, 2) / R), dtype=torch.float32).cuda()
    pos = torch.tensor(rng.integers(0, 10000, len(size)), **I32)
    q_out, k_out = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    e32 = float(np.float32(eps))
    gdn.gdn_qk_norm_rope(k, k, w, w, pos, freq, q_out, k_out, eps=eps, interleaved=inter)
    want = check_rotated(q_out, k, w, pos, freq, e32, inter, dtype, "q")
    check_rotated(k_out, k, w, pos, freq, e32, inter, dtype, "k")
    for e in (0, -12):
        cache, slots, bits = store_keys(k, w, pos, freq, 2.0 ** e, eps, inter, v=torch.zeros_like(k))
        check_store(cache, slots, 0, want, 2.0 ** e)
        assert bits == 0


def test_rows_of_zeros_without_epsilon_and_infinite_rows():
    """0 / 0 is no number, whatever the path: such keys are held as 0 with their bit; so is what stands beside an infinity."""
    k = torch.ones((3, 1, 64), device="cuda")
    k[0] = 0.0
    k[1, 0, 7] = float("inf")
    w, pos, freq = torch.ones(64, device="cuda"), torch.zeros(3, **I32), torch.zeros(0, device="cuda")
    out = torch.empty_like(k)
    gdn.gdn_qk_norm_rope(k, k, w, w, pos, freq, out, torch.empty_like(k), eps=0.0)
    assert out[0].isnan().all() and out[1, 0, 7].isnan() and not out[1, 0, :7].any() and (out[2] == 1.0).all()
    cache, _, bits = store_keys(k, w, pos, freq, eps=0.0)
    assert bits == gdn.ERRBIT_NONFINITE and not cache.codes[0, 0, 0, :2].any() and not cache.scales[0, 0, 0, :2].any()


# ---- long contexts -----------------------------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 12, 20, 40])  # with one head: each size of item of either kernel
@pytest.mark.parametrize("L,gap", [(131072, 18.0), (1000003, 19.0), (65536, 12.0)])
def test_attention_many_small_weights_beside_large_ones(D, T, L, gap):
    """Every 16th of the first 256 keys has score `gap` and value 0, the others score 0 and value 1: o = n e^-gap / (16 + n e^-gap)
    for the n of these that a token sees; lanes enough for each CTA to hold a whole one.  P is held in f16 at 2^7 times (at
    least) its share of the row's largest, so a weight is off by 2^-11 of itself or by 2^-25 2^-7; the exponentials are off
    by 2^-18 at most, and the sums, in L / 16 steps at most, by 2^-23 a step."""
    B, page = 304, 256
    codes = torch.zeros((2, 2, 1, page, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((2, 2, 1, page, D // 16), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    codes[0, 0, 0, ::16, 0] = 0x02  # 1.0 in the first dimension
    codes[:, 1] = 0x22              # the values: 1.0
    codes[0, 1, 0, ::16] = 0
    table = torch.ones((B, -(-L // page)), **I32)
    table[:, 0] = 0
    q = torch.zeros((B * T, 1, D), dtype=torch.bfloat16, device="cuda")
    q[:, 0, 0] = gap  # exact in bf16
    o, lse, err = torch.full_like(q, 9.0), torch.full((B * T, 1), 9.0, device="cuda"), err_word()
    gdn.gdn_kv4_attention(q, gdn.Kv4Cache(codes, scales), table, torch.full((B,), L, **I32), o,
                          gdn.kv4_attention_workspace(B, T, 1, 1, D), lse=lse, scale=1.0, err_word=err)
    n = L - T + np.arange(T, dtype=np.float64) - 15
    l = 16 + n * np.exp(-gap)
    want = (l - 16) / l
    sums = L / 16 * 2.0 ** -23
    bound = 2.0 ** -8 * want + (want * (2.0 ** -11 + 2.0 ** -18 + sums) + n * 2.0 ** -32 / l) * (1 + 2.0 ** -8)
    d = np.abs(f64(o).reshape(B, T, D) - want[:, None])
    assert (d <= bound[:, None]).all(), (float(d.max()), float(want.max()), float(bound.max()))
    assert (np.abs(f64(lse).reshape(B, T) - gap - np.log(l)) <= 2.0 ** -21 * (gap + 4) + 2.0 ** -18 + sums).all()
    assert int(err) == 0


# ---- what a cache may hold -----------------------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,HQ", [(3, 2), (4, 4), (8, 4), (40, 2), (150, 2)])
def test_attention_values_with_a_nan_scale(D, T, HQ):
    """A scale byte of NaN, which no store writes, in the values: its 16 numbers count as 0, so that the tokens which do not see
    them keep their bits."""
    rng = np.random.default_rng(D + T)
    r = attend(rng, [T, 1], [T + 61, 30], HQ, 1, D, 64, spoil=False)
    base = r["o"].clone()
    L = T + 61
    for j, groups in ((L - 1, slice(None)), (L - 2, slice(1, 2)), (5, slice(0, 1))):
        page, row = int(r["tables"][0, j // 64]), j % 64
        r["cache"].scales[page, 1, 0, row, groups] = 0x7F if j != L - 2 else 0xFF
        view = r["num"][page, 1, 0, row].reshape(-1, 16)
        view[groups] = 0.0
        if j == L - 2:
            r["call"]()
            assert torch.equal(r["o"][:T - 2], base[:T - 2]) and torch.equal(r["o"][T:], base[T:])
    r["call"]()
    check_attend(r)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,HQ", [(4, 4), (40, 2)])
def test_attention_keys_with_a_nan_scale(D, T, HQ):
    """In the keys it makes NaN of the tokens that see it, and of no other."""
    rng = np.random.default_rng(D + T)
    r = attend(rng, [T, 1], [T + 61, 30], HQ, 1, D, 64, spoil=False)
    base = r["o"].clone()
    j = T + 61 - 2
    r["cache"].scales[int(r["tables"][0, j // 64]), 0, 0, j % 64, 1] = 0x7F
    r["call"]()
    assert torch.equal(r["o"][:T - 2], base[:T - 2]) and torch.equal(r["o"][T:], base[T:])
    assert r["o"][T - 2:T].isnan().all() and r["lse"][T - 2:T].isnan().all() and not r["lse"][:T - 2].isnan().any()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("exponent", [120, 100, -100, -115])
def test_attention_queries_of_any_size(D, T, exponent):
    """Queries times a power of two, and the scale by its reciprocal: the same scores."""
    rng = np.random.default_rng(D + T)
    r = attend(rng, [T, T], [T + 200, T], 4, 2, D, 64)
    r["q"][r["q"].abs() < 2.0 ** -9] = 0.0  # what is left is a normal number after the smallest factor too
    r["call"]()
    check_attend(r, rows_per_lane=4)
    base = r["o"].clone(), r["lse"].clone()
    q = (r["q"].float() * 2.0 ** exponent).bfloat16()
    assert torch.equal(q.float() * 2.0 ** -exponent, r["q"].float())
    o, lse, err = torch.full_like(q, 9.0), torch.full_like(r["lse"], 9.0), err_word()
    gdn.gdn_kv4_attention(q, r["cache"], torch.tensor(r["tables"], **I32), torch.tensor(r["kvlens"], **I32), o,
                          gdn.kv4_attention_workspace(2, T, 4, 2, D), cu_seqlens=torch.tensor(r["cu"], **I32), max_q=T, lse=lse,
                          scale=r["scale"] * 2.0 ** -exponent, err_word=err)
    assert torch.equal(o, base[0]) and torch.equal(lse, base[1]) and int(err) == 0
