"""The attention-layer calls on the GPU against the 64-bit reference (tests/kv4_ref.py): page plan, norm + rotation, the
store into the 4-bit cache and its read-back, and attention over the cache.

Tolerances, from the arithmetic: whole numbers, stored codes and scales and the numbers read back are equal; norm +
rotation is off by half a step of its type (bf16 2^-8, fp32 2^-24 of the value) and by 2^-19 of the two numbers that a
rotation mixes (fp32 sum, root, products and angle); attention by bf16's half step and the bounds that
kv4_ref.attention derives."""
from __future__ import annotations

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import gated_deltanet_linear_mtp_gb300 as gdn
import kv4_ref as ref

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def err_word():
    return torch.zeros(1, **I32)


# ---- page plan ---------------------------------------------------------------------------------------------
def plan_inputs(rng, B, page, width, new_hi, ctx, spare=3, over_held=True):
    kv = rng.integers(0, ctx + 1, B).astype(np.int32)
    new = rng.integers(0, new_hi + 1, B).astype(np.int32)
    held = -(-kv // page)
    if over_held:  # pages of rejected drafts
        held = np.minimum(held + rng.integers(0, 2, B), width)
    num = int((-(-(kv.astype(np.int64) + new) // page)).sum() + held.sum()) + spare
    order = rng.permutation(num).astype(np.int32)
    tables = np.full((B, width), -7, np.int32)
    at = 0
    for b in range(B):
        tables[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    return kv, new, held.astype(np.int32), tables, order, at


def check_plan(kv, new, page, tables, held, free, taken, N, inplace=False):
    B = len(kv)
    want = ref.page_plan(kv, new, page, tables, held, free, taken, N)
    t = [torch.tensor(np.ascontiguousarray(x), **I32) for x in (kv, new, tables, held, free, [taken])]
    held_out = t[3] if inplace else torch.full((B,), -9, **I32)
    taken_out = t[5] if inplace else torch.full((1,), -9, **I32)
    plan = gdn.PagePlan(torch.full((B + 1,), -9, **I32), torch.full((N,), -9, **I32), torch.full((N,), -9, **I32),
                        torch.full((B,), -9, **I32), held_out, taken_out)
    ticket, err = torch.zeros(1, **I32), err_word()
    gdn.gdn_page_plan(t[0], t[1], page, t[2], t[3], t[4], t[5], plan, ticket, err)
    got = [t[2], plan.cu_seqlens, plan.positions, plan.slot_map, plan.total_lens, plan.held, plan.taken]
    for name, g, w in zip(("tables", "cu", "positions", "slots", "total", "held", "taken"), got, want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name
    assert int(err) == want[7] and int(ticket) == 0
    return want


@pytest.mark.parametrize("B,page,new_hi,ctx", [(1, 16, 1, 0), (1, 64, 1, 63), (1, 64, 1, 64), (3, 16, 40, 50), (5, 256, 8, 2000),
                                               (37, 32, 300, 700), (200, 64, 8, 5000), (513, 128, 4, 900),
                                               (1500, 16, 2, 100), (8192, 16, 1, 40)])
@pytest.mark.parametrize("inplace", [False, True])
def test_page_plan(B, page, new_hi, ctx, inplace):
    rng = np.random.default_rng(B * 7 + page + new_hi)
    width = -(-(ctx + new_hi) // page) + 2
    kv, new, held, tables, free, taken = plan_inputs(rng, B, page, width, new_hi, ctx)
    check_plan(kv, new, page, tables, held, free, taken, int(new.sum()) + 5, inplace)


def test_page_plan_more_ctas():
    rng = np.random.default_rng(3)
    kv, new, held, tables, free, taken = plan_inputs(rng, 300, 16, 600, 900, 5000)
    check_plan(kv, new, 16, tables, held, free, taken, int(new.sum()) + 3000, True)
    check_plan(kv, new, 16, tables, held, free, taken, max(1, int(new.sum()) // 2))  # fewer places than tokens: bit, no overrun


@pytest.mark.parametrize("short", [1, 5, 40, 10 ** 6])
def test_page_plan_short_of_pages(short):
    rng = np.random.default_rng(5)
    kv, new, held, tables, free, taken = plan_inputs(rng, 60, 16, 30, 60, 200, spare=0, over_held=False)
    need = int((-(-(kv + new) // 16) - held).sum())
    taken = max(taken, len(free) - max(0, need - short))
    want = check_plan(kv, new, 16, tables, held, free, taken, int(new.sum()))
    assert want[7] & gdn.ERRBIT_PAGES


def test_page_plan_bad_lengths_and_pages():
    rng = np.random.default_rng(6)
    kv, new, held, tables, free, taken = plan_inputs(rng, 40, 16, 30, 60, 200, over_held=False)
    kv[3], new[5], held[7], held[9] = -4, -2, -1, 31
    kv[11] = 30 * 16
    held[13] = 0
    kv[13] = max(kv[13], 1)
    free = free.copy()
    free[taken + 2] = -5
    free[taken + 4] = len(free)
    check_plan(kv, new, 16, tables, held, free, taken, int(np.maximum(new, 0).sum()) + 2)
    check_plan(kv, new, 16, tables, held, free, -3, int(np.maximum(new, 0).sum()) + 2)
    check_plan(kv, new, 16, tables, held, free, len(free) + 1, int(np.maximum(new, 0).sum()) + 2)


# ---- norm + rotation, store, read ------------------------------------------------------------------------------
def qk_inputs(rng, N, HQ, HK, D, R, dtype, far=100000, spread=1.0):
    x = rng.normal(size=(N, HQ + 2 * HK, D)) * np.exp(rng.normal(size=(N, HQ + 2 * HK, 1)) * spread)
    t = torch.tensor(x, dtype=torch.float32).to(dtype).cuda()  # fused rows: q, k, v are views with a token stride
    w = [torch.tensor(1 + 0.2 * rng.normal(size=D), dtype=torch.float32, device="cuda") for _ in range(2)]
    pos = torch.tensor(rng.integers(0, far, N), **I32)
    freq = torch.tensor(1e4 ** (-np.arange(0, R, 2) / max(R, 1)), dtype=torch.float32, device="cuda")
    return (*t.split((HQ, HK, HK), 1), *w, pos, freq)


def f64(t):
    return t.detach().cpu().double().numpy()


def check_rotated(got, x, w, pos, freq, eps, inter, dtype, what):
    want, size = ref.norm_rope(f64(x), f64(w), pos.cpu().numpy(), f64(freq), eps, inter)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    bad = np.abs(f64(got) - want) > half * np.abs(want) + 2.0 ** -19 * (1 + 2 * half) * size + 1e-37
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}"
    return want


SHAPES = [(1, 1, 1, 64, 64), (1, 16, 2, 256, 64), (3, 4, 4, 128, 128), (7, 5, 1, 64, 32), (33, 32, 8, 128, 128),
          (130, 16, 2, 256, 256), (517, 8, 2, 128, 64), (64, 6, 3, 64, 0), (2000, 24, 8, 128, 16), (9, 130, 2, 256, 0)]


@pytest.mark.parametrize("N,HQ,HK,D,R", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope(N, HQ, HK, D, R, dtype, inter):
    rng = np.random.default_rng(N + HQ + D)
    q, k, _, qw, kw, pos, freq = qk_inputs(rng, N, HQ, HK, D, R, dtype)
    qo, ko = torch.full((N, HQ, D), 7.0, dtype=dtype, device="cuda"), torch.full((N, HK, D), 7.0, dtype=dtype, device="cuda")
    gdn.gdn_qk_norm_rope(q, k, qw, kw, pos, freq, qo, ko, eps=1e-5, interleaved=inter)
    check_rotated(qo, q, qw, pos, freq, 1e-5, inter, dtype, "q")
    check_rotated(ko, k, kw, pos, freq, 1e-5, inter, dtype, "k")


def test_norm_rope_in_place_and_far_and_special_rows():
    rng = np.random.default_rng(1)
    q, k, _, qw, kw, _, freq = qk_inputs(rng, 6, 4, 2, 128, 128, torch.float32)
    q, k = q.clone(), k.clone()
    q[1, 1] = 0.0
    q[2, 2] *= 1e-18  # its mean square is lost beside eps
    q0, k0 = q.clone(), k.clone()
    pos = torch.tensor([0, 1, 2 ** 20 + 7, 2 ** 30 + 1, 2 ** 31 - 1, -5], **I32)
    gdn.gdn_qk_norm_rope(q, k, qw, kw, pos, freq, q, k)
    # beyond 2^20 the reference's own angle, in fp64, is right to 2^31 * 2^-53 turns only: far less than the bound
    check_rotated(q, q0, qw, pos, freq, 1e-6, False, torch.float32, "q")
    check_rotated(k, k0, kw, pos, freq, 1e-6, False, torch.float32, "k")
    assert not q[1, 1].any()


def pool(pages, HK, page, D, k_scale=1.0, v_scale=1.0, fill=0xA5):
    codes = torch.full((pages, 2, HK, page, D // 2), fill, dtype=torch.uint8, device="cuda")
    scales = torch.full((pages, 2, HK, page, D // 16), fill, dtype=torch.uint8, device="cuda")
    return gdn.Kv4Cache(codes, scales, k_scale, v_scale)


def slots_for(rng, N, pages, page, skip=0):
    s = rng.permutation(pages * page)[:N].astype(np.int32)
    s[rng.permutation(N)[:skip]] = -1
    return s


def check_store(cache, slots, which, x, unit):
    """The stored bytes of every slot, and that no other byte of the pool changed."""
    codes, scales = ref.quantise(x, unit)
    page = cache.page_size
    gc, gs = cache.codes.cpu().numpy()[:, which], cache.scales.cpu().numpy()[:, which]
    wc, ws = np.full_like(gc, 0xA5), np.full_like(gs, 0xA5)
    for n in np.flatnonzero(slots >= 0):
        wc[slots[n] // page, :, slots[n] % page] = codes[n]
        ws[slots[n] // page, :, slots[n] % page] = scales[n]
    assert np.array_equal(gs, ws), f"scales: {(gs != ws).sum()}"
    # a zero may carry either sign
    both = lambda c: np.stack((c & 15, c >> 4))  # noqa: E731
    a, b = both(gc), both(wc)
    assert np.array_equal(np.where(a == 8, 0, a), np.where(b == 8, 0, b)), f"codes: {(a != b).sum()}"


@pytest.mark.parametrize("N,HQ,HK,D,R,page", [(1, 1, 1, 64, 64, 16), (5, 16, 2, 256, 64, 64), (130, 8, 8, 128, 128, 32),
                                              (517, 4, 2, 64, 32, 256), (1200, 16, 4, 128, 0, 128), (64, 12, 3, 256, 256, 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter,units", [(False, (1.0, 1.0)), (True, (0.25, 4.0))])
def test_store_and_read(N, HQ, HK, D, R, page, dtype, inter, units):
    rng = np.random.default_rng(N + D + page)
    q, k, v, qw, kw, pos, freq = qk_inputs(rng, N, HQ, HK, D, R, dtype)
    pages = -(-N // page) + 2
    cache = pool(pages, HK, page, D, *units)
    slots = slots_for(rng, N, pages, page, N // 10)
    st, err = torch.tensor(slots, **I32), err_word()
    qo = torch.zeros((N, HQ, D), dtype=dtype, device="cuda")
    ko = torch.zeros((N, HK, D), dtype=dtype, device="cuda") if inter else None
    gdn.gdn_qk_norm_rope(q, k, qw, kw, pos, freq, qo, ko, v=v, cache=cache, slot_map=st, err_word=err, interleaved=inter)
    check_rotated(qo, q, qw, pos, freq, 1e-6, inter, dtype, "q")
    kx = ref.norm_rope(f64(k), f64(kw), pos.cpu().numpy(), f64(freq), float(np.float32(1e-6)), inter)[0]
    if ko is not None:
        check_rotated(ko, k, kw, pos, freq, 1e-6, inter, dtype, "k")
    check_store(cache, slots, 0, kx, units[0])
    check_store(cache, slots, 1, f64(v), units[1])
    kr = torch.full((N, HK, D), 7.0, dtype=torch.bfloat16, device="cuda")
    vr = torch.full((N, HK, D), 7.0, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_kv4_read(cache, st, kr, vr, err)
    for got, x, unit in ((kr, kx, units[0]), (vr, f64(v), units[1])):
        want = ref.numbers(*ref.quantise(x, unit), unit)
        want[slots < 0] = 7.0
        assert np.array_equal(f64(got), want)
    assert int(err) == 0


def test_store_ties_zeros_and_nonfinite_values():
    N, HK, D, page = 8, 1, 64, 16
    v = torch.zeros((N, HK, D), dtype=torch.float32, device="cuda")
    grid = torch.tensor([6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5.0, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25, 0.0])
    v[1, 0, :16] = grid.cuda()                                       # every tie
    v[1, 0, 16:32] = torch.nextafter(grid, grid * 9).cuda()          # just beyond: fp32 has to see it
    v[1, 0, 32:48] = torch.nextafter(grid, grid * 0).cuda()
    v[2] = 1e30                                                      # saturates
    v[3] = 1e-9                                                      # below the least scale
    v[4, 0, 0] = 6.375                                               # the scale's tie
    v[4, 0, 16] = float(np.nextafter(np.float32(6.375), np.float32(9)))
    v[4, 0, 32] = float(np.nextafter(np.float32(6.375), np.float32(0)))
    v[5, 0, 3], v[5, 0, 5] = float("nan"), 2.0
    v[6, 0, 3], v[6, 0, 5] = float("inf"), 2.0
    k = torch.randn((N, HK, D), device="cuda")
    k[7, 0, 9] = float("nan")
    one, freq = torch.ones(D, device="cuda"), torch.zeros(0, device="cuda")
    cache, slots, err = pool(1, HK, page, D), np.arange(N, dtype=np.int32), err_word()
    qo = torch.zeros((N, 1, D), device="cuda")
    args = (torch.randn((N, 1, D), device="cuda"), k, one, one, torch.zeros(N, **I32), freq, qo)
    gdn.gdn_qk_norm_rope(*args, v=v, cache=cache, slot_map=torch.tensor(slots, **I32), err_word=err)
    check_store(cache, slots, 1, f64(v), 1.0)
    assert int(err) == gdn.ERRBIT_NONFINITE
    assert not cache.codes[0, 0, 0, 7].any() and not cache.scales[0, 0, 0, 7].any()  # a key row of NaN is stored as zeros


def test_store_bad_slots():
    N, HK, D, page = 6, 2, 128, 32
    cache, err = pool(2, HK, page, D), err_word()
    slots = np.array([-2, 64, 5, -1, 2 ** 31 - 1, -2 ** 31], np.int32)
    st = torch.tensor(slots, **I32)
    rng = np.random.default_rng(9)
    q, k, v, qw, kw, pos, freq = qk_inputs(rng, N, 2, HK, D, 64, torch.bfloat16)
    gdn.gdn_qk_norm_rope(q, k, qw, kw, pos, freq, torch.zeros((N, 2, D), dtype=torch.bfloat16, device="cuda"), v=v, cache=cache,
                         slot_map=st, err_word=err)
    ok = np.where((slots >= 0) & (slots < 64), slots, -1)
    check_store(cache, ok, 1, f64(v), 1.0)
    assert int(err) == gdn.ERRBIT_INDEX
    err.zero_()
    out = torch.full((N, HK, D), 3.0, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_kv4_read(cache, st, out, out.clone(), err)
    assert int(err) == gdn.ERRBIT_INDEX and (out[ok < 0] == 3.0).all() and not (out[2] == 3.0).all()


# ---- attention --------------------------------------------------------------------------------------------------
def filled(rng, pages, HK, page, D, junk=True):
    """A pool of quantised normal rows; with `junk`, pages * page rows are followed by nothing that may be relied on."""
    x = rng.normal(size=(pages, 2, HK, page, D)) * (1 + 2 * (np.arange(D) % 29 == 3))
    codes, scales = ref.quantise(x)
    return gdn.Kv4Cache(torch.tensor(codes).cuda(), torch.tensor(scales).cuda()), ref.numbers(codes, scales)


def attend(rng, qlens, kvlens, HQ, HK, D, page, cu=True, scale=None, lse=True, max_q=None, spoil=True):
    B, width = len(qlens), max(1, max(-(-max(n, 0) // page) for n in kvlens)) + 1
    need = [-(-max(n, 0) // page) for n in kvlens]
    pages = sum(need) + 2
    cache, num = filled(rng, pages, HK, page, D)
    order = rng.permutation(pages).astype(np.int32)
    tables, at = np.full((B, width), -1, np.int32), 0
    for b in range(B):
        tables[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    if spoil:  # what lies behind a lane's last token is NaN scales and full codes
        for b in range(B):
            if kvlens[b] > 0 and kvlens[b] % page:
                cache.codes[int(tables[b, need[b] - 1]), :, :, kvlens[b] % page:] = 0x77
                cache.scales[int(tables[b, need[b] - 1]), :, :, kvlens[b] % page:] = 0x7F
        for p in order[at:]:
            cache.scales[int(p)] = 0x7F
    cus = np.concatenate(([0], np.cumsum(qlens))).astype(np.int32)
    N = int(cus[-1])
    q = torch.tensor(rng.normal(size=(N, HQ, D)) * 1.5, dtype=torch.float32).bfloat16().cuda()
    o = torch.full((N, HQ, D), 9.0, dtype=torch.bfloat16, device="cuda")
    ls = torch.full((N, HQ), 9.0, device="cuda") if lse else None
    mq = max_q or max(1, max(qlens))
    ws = gdn.kv4_attention_workspace(B, mq, HQ, HK, D)
    ws.fill_(0xFF)  # its contents need not be kept
    err = err_word()
    call = lambda: gdn.gdn_kv4_attention(q, cache, torch.tensor(tables, **I32), torch.tensor(kvlens, **I32), o, ws,  # noqa: E731
                                         cu_seqlens=torch.tensor(cus, **I32) if cu else None, max_q=mq if cu else None, lse=ls,
                                         scale=scale, err_word=err)
    call()
    return dict(q=q, o=o, lse=ls, cache=cache, num=num, tables=tables, cu=cus, err=err, call=call, qlens=qlens, kvlens=kvlens,
                page=page, HQ=HQ, HK=HK, D=D, scale=D ** -0.5 if scale is None else scale)


def check_attend(r, rows_per_lane=None):
    q, o = f64(r["q"]), f64(r["o"])
    lse = f64(r["lse"]) if r["lse"] is not None else None
    G, page = r["HQ"] // r["HK"], r["page"]
    for b, (n, L) in enumerate(zip(r["qlens"], r["kvlens"])):
        pick = range(n) if rows_per_lane is None or n <= rows_per_lane else sorted({0, 1, n // 3, n // 2, n - 2, n - 1})
        if not n:
            continue
        pick = list(pick)
        j = np.arange(max(L, 0))
        rows = r["num"][r["tables"][b, j // page], :, :, j % page] if L > 0 else np.zeros((0, 2, r["HK"], r["D"]))
        for h in range(r["HQ"]):
            at = r["cu"][b] + np.array(pick)
            want, wl, be, bl = ref.attention(q[at, h], rows[:, 0, h // G], rows[:, 1, h // G], [L - n + t + 1 for t in pick], r["scale"])
            d = np.abs(o[at, h] - want)
            bad = ~(d <= 2.0 ** -8 * np.abs(want) + be * (1 + 2.0 ** -8) + 1e-37)
            assert not bad.any(), (b, h, n, L, int(bad.sum()), float(d.max()), float(np.abs(want).max()))
            if lse is not None:
                got = lse[at, h]
                none = wl == -math.inf
                assert np.array_equal(got == -math.inf, none), (b, h)
                assert (np.abs(got - np.where(none, 0, wl))[~none] <= bl[~none]).all(), (b, h, got, wl)
    assert int(r["err"]) == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("HQ,HK", [(1, 1), (8, 1), (6, 2), (20, 4)])
@pytest.mark.parametrize("T", [1, 3, 4])
def test_attention_shapes(D, HQ, HK, T):
    rng = np.random.default_rng(D + HQ + T)
    lens = [T, 16, 127, 128, 129, 300]
    check_attend(attend(rng, [T] * 6, lens, HQ, HK, D, 16 if T == 3 else 64, cu=T == 4))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_pages_ending_inside_a_tile(page, D):
    rng = np.random.default_rng(page + D)
    check_attend(attend(rng, [1, 2, 1, 2, 1], [1, 2, page - 1, page + 1, 3 * page + 5], 4, 2, D, page))


@pytest.mark.parametrize("T,HQ,HK,D", [(8, 16, 2, 64), (8, 16, 2, 128), (16, 8, 1, 256), (16, 16, 1, 128), (5, 7, 1, 128), (2, 64, 1, 64),
                                       (13, 24, 8, 256)])
def test_attention_many_rows(T, HQ, HK, D):
    rng = np.random.default_rng(T + D)
    check_attend(attend(rng, [T, T, T], [T, 200, 777], HQ, HK, D, 32, cu=False))


@pytest.mark.parametrize("D,HQ,HK,T", [(128, 8, 2, 1), (64, 8, 1, 8), (256, 4, 1, 2)])
def test_attention_one_long_lane(D, HQ, HK, T):
    """One lane over every CTA: its parts are joined, also beside a lane of one tile."""
    rng = np.random.default_rng(D)
    check_attend(attend(rng, [T, T], [40000, 17], HQ, HK, D, 64))


def test_attention_rows_without_keys_and_empty_lanes():
    rng = np.random.default_rng(11)
    r = attend(rng, [4, 0, 3, 2, 0, 1], [0, 0, 1, 70, 9, 0], 6, 2, 128, 16)
    check_attend(r)
    assert not r["o"][:4].any() and (r["lse"][:4] == -math.inf).all()
    assert not r["o"][4:6].any() and r["o"][6].any()


@pytest.mark.parametrize("D,HQ,HK", [(64, 4, 2), (128, 8, 1), (128, 6, 2), (256, 4, 1)])
def test_attention_prompts(D, HQ, HK):
    rng = np.random.default_rng(D + HQ)
    check_attend(attend(rng, [17, 130, 1, 257, 0, 40], [17, 130, 300, 500, 8, 39], HQ, HK, D, 32), rows_per_lane=20)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_long_prompt(D):
    rng = np.random.default_rng(D)
    check_attend(attend(rng, [1500, 3], [2100, 2000], 4, 1, D, 64), rows_per_lane=8)


def test_attention_large_and_small_scores():
    for scale in (0.0, -0.2, 3.0, 1e-4):
        rng = np.random.default_rng(12)
        check_attend(attend(rng, [2, 2], [200, 40], 4, 2, 128, 64, scale=scale))


def test_attention_more_lanes_than_threads():
    rng = np.random.default_rng(13)
    lens = rng.integers(0, 90, 300).tolist()
    qlens = [int(min(3, n)) for n in lens]
    check_attend(attend(rng, qlens, lens, 4, 2, 64, 16))


def test_attention_masked_values_do_not_leak():
    """A draft's NaN value (a scale byte no store writes) or infinite query stays in the rows that see it."""
    rng = np.random.default_rng(14)
    r = attend(rng, [2, 1], [50, 30], 2, 1, 128, 64, spoil=False)
    base = r["o"].clone()
    r["q"][1, 1, 5] = float("nan")
    r["q"][0, 1, 5] = float("inf")
    r["call"]()
    keep = [(0, 0), (1, 0), (2, 0), (2, 1)]
    assert all(torch.equal(r["o"][t, h], base[t, h]) for t, h in keep)
    assert r["o"][1, 1].isnan().all()


def test_attention_bad_lanes_and_pages():
    rng = np.random.default_rng(15)
    r = attend(rng, [2, 2, 2, 2], [40, 40, 40, 40], 4, 2, 64, 16, spoil=False)
    good = r["o"].clone()
    tables, cu = torch.tensor(r["tables"], **I32), torch.tensor(r["cu"], **I32)
    ws = gdn.kv4_attention_workspace(4, 2, 4, 2, 64)

    def go(kv=(40, 40, 40, 40), cu=cu, tables=tables):
        o, err = torch.full_like(good, 9.0), err_word()
        gdn.gdn_kv4_attention(r["q"], r["cache"], tables, torch.tensor(kv, **I32), o, ws, cu_seqlens=cu, max_q=2, err_word=err)
        return o, int(err)

    o, bits = go(kv=(40, -1, 10 ** 6, 40))
    assert bits == gdn.ERRBIT_SEQLEN and (o[2:6] == 9.0).all() and torch.equal(o[:2], good[:2]) and torch.equal(o[6:], good[6:])
    for bad in ([0, 2, 1, 6, 8], [0, 2, 5, 6, 8], [0, 2, 4, 6, 9], [-1, 1, 4, 6, 8]):
        _, bits = go(cu=torch.tensor(bad, **I32))
        assert bits == gdn.ERRBIT_SEQLEN
    t2 = tables.clone()
    t2[1, 1], t2[2, 0] = r["cache"].num_pages, -3
    o, bits = go(tables=t2)
    assert bits == gdn.ERRBIT_INDEX and torch.equal(o[:2], good[:2]) and torch.equal(o[6:], good[6:]) and torch.isfinite(o).all()


def test_attention_needs_no_lse_and_repeats_bit_for_bit():
    rng = np.random.default_rng(16)
    r = attend(rng, [4] * 5, [3000, 1, 700, 64, 2049], 8, 2, 128, 64, lse=False)
    first = r["o"].clone()
    for _ in range(3):
        r["o"].fill_(5.0)
        r["call"]()
        assert torch.equal(r["o"], first)
    check_attend(r)


def test_attention_reads_pages_beyond_two_gigabytes():
    """A slot whose byte offset in the pool passes 32 bits."""
    HK, page, D = 8, 256, 256
    pages = (1 << 32) // (2 * HK * page * D // 2) + 40
    codes = torch.zeros((pages, 2, HK, page, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((pages, 2, HK, page, D // 16), dtype=torch.uint8, device="cuda")
    cache = gdn.Kv4Cache(codes, scales)
    rng = np.random.default_rng(17)
    N, HQ = 20, 8
    q, k, v, qw, kw, pos, freq = qk_inputs(rng, N, HQ, HK, D, 64, torch.bfloat16)
    last = pages - 1
    slots = np.arange(N, dtype=np.int32) + last * page
    qo = torch.zeros((N, HQ, D), dtype=torch.bfloat16, device="cuda")
    gdn.gdn_qk_norm_rope(q, k, qw, kw, pos, freq, qo, v=v, cache=cache, slot_map=torch.tensor(slots, **I32))
    kx = ref.norm_rope(f64(k), f64(kw), pos.cpu().numpy(), f64(freq), float(np.float32(1e-6)), False)[0]
    kq, vq = ref.numbers(*ref.quantise(kx)), ref.numbers(*ref.quantise(f64(v)))
    kr, vr = torch.zeros((N, HK, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((N, HK, D), dtype=torch.bfloat16, device="cuda")
    gdn.gdn_kv4_read(cache, torch.tensor(slots, **I32), kr, vr)
    assert np.array_equal(f64(kr), kq) and np.array_equal(f64(vr), vq)
    o = torch.zeros_like(qo[:1])
    gdn.gdn_kv4_attention(qo[:1], cache, torch.tensor([[last]], **I32), torch.tensor([N], **I32), o,
                          gdn.kv4_attention_workspace(1, 1, HQ, HK, D))
    for h in range(HQ):
        want, _, be, _ = ref.attention(f64(qo)[:1, h], kq[:, h], vq[:, h], [N], D ** -0.5)
        assert (np.abs(f64(o)[:, h] - want) <= 2.0 ** -8 * np.abs(want) + be * 1.01).all()


# ---- streams, graphs, the set together -----------------------------------------------------------------------
def test_streams_and_graph_replay():
    """The calls on a stream of their own, then captured into a graph and replayed on changed inputs."""
    rng = np.random.default_rng(18)
    r = attend(rng, [2] * 3, [500, 77, 200], 8, 2, 128, 64, cu=False)
    tables, kv = torch.tensor(r["tables"], **I32), torch.tensor(r["kvlens"], **I32)
    ws = gdn.kv4_attention_workspace(3, 2, 8, 2, 128)
    o = torch.zeros_like(r["o"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gdn.gdn_kv4_attention(r["q"], r["cache"], tables, kv, o, ws, stream=s)
    s.synchronize()
    assert torch.equal(o, r["o"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_kv4_attention(r["q"], r["cache"], tables, kv, o, ws)
    kv.copy_(torch.tensor([130, 9, 2], **I32))
    o.zero_()
    g.replay()
    torch.cuda.synchronize()
    want = torch.zeros_like(o)
    gdn.gdn_kv4_attention(r["q"], r["cache"], tables, kv, want, ws)
    assert torch.equal(o, want)


def test_the_example_runs():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, os.path.join(root, "examples", "attention_step.py")], capture_output=True, text=True,
                       cwd=root, timeout=300)
    assert p.returncode == 0 and "ok" in p.stdout, p.stdout + p.stderr


@pytest.mark.parametrize("D,HQ,HK,T", [(64, 8, 2, 10), (64, 16, 2, 8), (128, 8, 2, 20), (128, 16, 2, 16), (256, 8, 2, 12), (256, 8, 2, 33)])
def test_attention_runs_of_many_tiles(D, HQ, HK, T):
    """Every CTA of the kernel for many rows takes a run of several items and of several tiles of each, of few rows and of
    many in turn."""
    rng = np.random.default_rng(D + T)
    lens = [int(n) for n in rng.integers(1500, 2600, size=40)]
    check_attend(attend(rng, [(T, 3 * T, 1, 7 * T // 2)[b % 4] for b in range(40)], lens, HQ, HK, D, 64), rows_per_lane=2)
