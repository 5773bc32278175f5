"""Refusals of the attention-layer calls on the host, before anything reaches the GPU, and the 64-bit reference's own
format against hand-made values (no GPU needed)."""
import ctypes
import os

import numpy as np
import pytest

import gated_deltanet_linear_mtp_gb300 as gdn
import kv4_ref
from gated_deltanet_linear_mtp_gb300 import build as gbuild

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
BAD4 = ctypes.c_void_p(0x10002)
OK, NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, VALUE = 0, 1, 2, 3, 4, 5, 7


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gbuild.LIB_PATH):
        gbuild.build()
    return gdn.lib()


def cache(**kw):
    base = dict(codes=0x10000, scales=0x20000, num_pages=8, page_size=64, HK=2, D=128, k_scale=1.0, v_scale=1.0)
    base.update(kw)
    return gdn._Kv4CacheC(**base)


BAD_CACHES = [(dict(num_pages=0), SHAPE), (dict(page_size=48), SHAPE), (dict(page_size=8), SHAPE),
              (dict(page_size=512), SHAPE), (dict(HK=0), SHAPE), (dict(HK=1025), SHAPE), (dict(D=96), UNSUPPORTED),
              (dict(num_pages=1 << 27, page_size=16), SHAPE), (dict(codes=None), NULL), (dict(scales=None), NULL),
              (dict(codes=0x10008), ALIGN), (dict(scales=0x10004), ALIGN), (dict(k_scale=0.3), VALUE),
              (dict(v_scale=0.0), VALUE), (dict(k_scale=-1.0), VALUE), (dict(v_scale=float("inf")), VALUE),
              (dict(k_scale=float("nan")), VALUE), (dict(v_scale=2.0 ** 40), VALUE)]


def plan(L, B=4, N=16, page=64, width=8, pages=32, out=True, **ptr):
    a = dict(kv=P, new=P, table=P, held=P, free=P, taken=P, ticket=P, err=None)
    a.update({k: v for k, v in ptr.items() if k in a})
    o = gdn._PagePlanC(**{n: ptr.get(n, P) for n, _ in gdn._PagePlanC._fields_})
    return L.gdn_page_plan(B, N, page, width, pages, a["kv"], a["new"], a["table"], a["held"], a["free"], a["taken"],
                           ctypes.byref(o) if out else None, a["ticket"], a["err"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), SHAPE), (dict(B=8193), SHAPE), (dict(N=-1), SHAPE), (dict(page=24), SHAPE), (dict(page=0), SHAPE),
    (dict(width=0), SHAPE), (dict(pages=0), SHAPE), (dict(pages=1 << 26), SHAPE), (dict(width=1 << 26), SHAPE),
    (dict(kv=None), NULL), (dict(new=None), NULL), (dict(table=None), NULL), (dict(held=None), NULL),
    (dict(free=None), NULL), (dict(taken=None), NULL), (dict(ticket=None), NULL), (dict(out=False), NULL),
    (dict(cu_seqlens=None), NULL), (dict(positions=None), NULL), (dict(slot_map=None), NULL), (dict(kv=BAD4), ALIGN),
    (dict(taken=BAD4), ALIGN), (dict(slot_map=BAD4), ALIGN), (dict(err=BAD4), ALIGN), (dict(B=0, kv=None), OK)])
def test_page_plan_refusals(L, kw, status):
    assert plan(L, **kw) == status


def norm_rope(L, d=None, c=None, store=True, **ptr):
    base = dict(N=4, HQ=8, HK=2, D=128, R=64, interleaved=0, dtype=1, q_stride=1024, k_stride=256, v_stride=256, eps=1e-6)
    base.update(d or {})
    dims = gdn._QkDimsC(**base)
    a = dict(q=P, k=P, qw=P, kw=P, pos=P, freq=P, qo=P, ko=ctypes.c_void_p(0x20000), v=P if store else None, slots=P if store else None, err=None)
    a.update(ptr)
    cc = cache(**(c or {})) if store else None
    return L.gdn_qk_norm_rope(ctypes.byref(dims), a["q"], a["k"], a["qw"], a["kw"], a["pos"], a["freq"], a["qo"], a["ko"],
                              a["v"], ctypes.byref(cc) if cc is not None else None, a["slots"], a["err"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), SHAPE), (dict(HQ=0), SHAPE), (dict(HK=0), SHAPE), (dict(HQ=1025), SHAPE), (dict(D=32), UNSUPPORTED),
    (dict(R=24), SHAPE), (dict(R=144), SHAPE), (dict(R=-16), SHAPE), (dict(interleaved=2), VALUE), (dict(dtype=2), DTYPE),
    (dict(eps=-1.0), VALUE), (dict(eps=float("nan")), VALUE), (dict(q_stride=1023), SHAPE), (dict(k_stride=128), SHAPE),
    (dict(v_stride=0), SHAPE), (dict(q_stride=1028), ALIGN), (dict(v_stride=257), ALIGN), (dict(HK=1), SHAPE),
    (dict(N=0), OK)])
def test_norm_rope_refusals(L, kw, status):
    assert norm_rope(L, kw) == status


@pytest.mark.parametrize("ptr,status", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(qw=None), NULL), (dict(kw=None), NULL), (dict(pos=None), NULL),
    (dict(freq=None), NULL), (dict(qo=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(q=ODD), ALIGN),
    (dict(k=ODD), ALIGN), (dict(qo=ODD), ALIGN), (dict(ko=ODD), ALIGN), (dict(v=ODD), ALIGN), (dict(qw=ODD), ALIGN),
    (dict(pos=BAD4), ALIGN), (dict(slots=BAD4), ALIGN), (dict(err=BAD4), ALIGN)])
def test_norm_rope_pointers(L, ptr, status):
    assert norm_rope(L, **ptr) == status


def test_norm_rope_without_a_cache(L):
    assert norm_rope(L, store=False, ko=None) == NULL
    assert norm_rope(L, store=False, v=P) == NULL
    assert norm_rope(L, dict(N=0), store=False) == OK


def test_keys_are_not_stored_from_where_they_are_overwritten(L):
    other = ctypes.c_void_p(0x30000)
    assert norm_rope(L, k=other, ko=other) == VALUE


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(L, kw, status):
    c = cache(**kw)
    assert L.gdn_kv4_read(ctypes.byref(c), 4, P, P, P, None, None) == status
    assert attention(L, c=kw) == status
    if "HK" not in kw and "D" not in kw:
        assert norm_rope(L, c=kw) == status


@pytest.mark.parametrize("a,status", [((-1, P, P, P, None), SHAPE), ((4, None, P, P, None), NULL), ((4, P, None, P, None), NULL),
                                      ((4, P, P, None, None), NULL), ((4, P, ODD, P, None), ALIGN),
                                      ((4, BAD4, P, P, None), ALIGN), ((4, P, P, P, BAD4), ALIGN), ((0, None, None, None, None), OK)])
def test_read_refusals(L, a, status):
    c = cache()
    assert L.gdn_kv4_read(ctypes.byref(c), *a, None) == status


def attention(L, d=None, c=None, bytes_=1 << 40, **ptr):
    base = dict(B=2, N=8, max_q=4, HQ=8, max_pages=4, scale=0.1)
    base.update(d or {})
    dims, cc = gdn._Kv4AttentionDimsC(**base), cache(**(c or {}))
    a = dict(q=P, cu=None, table=P, kv=P, o=P, lse=None, ws=P, err=None)
    a.update(ptr)
    return L.gdn_kv4_attention(ctypes.byref(dims), ctypes.byref(cc), a["q"], a["cu"], a["table"], a["kv"], a["o"], a["lse"],
                               a["ws"], bytes_, a["err"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(N=-1), SHAPE), (dict(max_q=0), SHAPE), (dict(HQ=7), SHAPE),
    (dict(HQ=1), SHAPE), (dict(HQ=130), SHAPE), (dict(max_pages=0), SHAPE), (dict(max_pages=1 << 26), SHAPE),
    (dict(N=7), SHAPE), (dict(scale=float("nan")), VALUE), (dict(B=0, N=0), OK)])
def test_attention_refusals(L, kw, status):
    assert attention(L, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), NULL), (dict(table=None), NULL), (dict(kv=None), NULL), (dict(o=None), NULL), (dict(ws=None), NULL),
    (dict(q=ODD), ALIGN), (dict(o=ODD), ALIGN), (dict(ws=ODD), ALIGN), (dict(cu=BAD4), ALIGN), (dict(lse=BAD4), ALIGN),
    (dict(kv=BAD4), ALIGN), (dict(bytes_=100), SHAPE)])
def test_attention_pointers(L, kw, status):
    assert attention(L, **kw) == status


@pytest.mark.parametrize("a", [(-1, 1, 8, 2, 128), (4, 0, 8, 2, 128), (4, 1, 7, 2, 128), (4, 1, 8, 2, 96), (4, 1, 130, 2, 64)])
def test_workspace_refusals(L, a):
    assert L.gdn_kv4_attention_workspace(*a) == -1


def test_workspace_grows_with_the_rows(L):
    small = L.gdn_kv4_attention_workspace(4, 1, 8, 2, 128)
    assert 0 < small <= L.gdn_kv4_attention_workspace(4, 8, 8, 2, 128)


def test_cpu_tensors_are_refused():
    import torch

    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.Kv4Cache(torch.zeros((2, 2, 1, 16, 32), dtype=torch.uint8), torch.zeros((2, 2, 1, 16, 4), dtype=torch.uint8))
    with pytest.raises(ValueError):
        gdn.PagePlan(torch.zeros(5, dtype=torch.int32), z, z, z, z, z[:1])
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope(torch.zeros(1, 2, 64), torch.zeros(1, 1, 64), *[None] * 5)


# ---- the reference's format --------------------------------------------------------------------------------
def test_reference_codes_by_hand():
    x = np.zeros(16)
    x[:9] = [6.0, -6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]  # scale 1; the ties go to the even code
    codes, scales = kv4_ref.quantise(x)
    assert kv4_ref.E4M3[scales[0]] == 1.0
    assert kv4_ref.numbers(codes, scales)[:9].tolist() == [6.0, -6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]


def test_reference_scales_match_torch():
    import torch

    x = np.abs(np.random.default_rng(0).normal(size=4000)) * np.exp(np.random.default_rng(1).normal(size=4000) * 3)
    mine = kv4_ref.E4M3[kv4_ref.nearest(np.minimum(x, 448.0), kv4_ref.E4M3)]
    theirs = torch.tensor(np.minimum(x, 448.0), dtype=torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(mine, theirs)
    assert kv4_ref.E4M3[-1] == 448.0


def test_reference_attention_in_closed_form():
    k = np.zeros((3, 64))
    k[1, 0] = 2.0
    v = np.eye(3, 64)
    o, lse, _, _ = kv4_ref.attention(np.eye(1, 64), k, v, [2], 0.5)
    e = np.exp(1.0)
    assert np.allclose(o[0, :3], [1 / (1 + e), e / (1 + e), 0.0]) and np.isclose(lse[0], np.log(1 + e))
    o, lse, _, _ = kv4_ref.attention(np.eye(1, 64), k, v, [0], 0.5)
    assert not o.any() and lse[0] == -np.inf


def test_reference_rotation_keeps_lengths_and_turns_by_the_angle():
    x = np.random.default_rng(2).normal(size=(3, 2, 64))
    f = np.array([1.0, 0.5, 0.25, 0.1, 0.01, 0.02, 0.03, 0.04], np.float32)
    for inter in (False, True):
        y, _ = kv4_ref.norm_rope(x, np.ones(64), np.array([0, 1, 7]), f, 0.0, inter)
        assert np.allclose((y ** 2).mean(-1), 1.0) and np.allclose(y[0], x[0] / np.sqrt((x[0] ** 2).mean(-1, keepdims=True)))
        a, b = (0, 1) if inter else (0, 8)
        z0 = kv4_ref.norm_rope(x, np.ones(64), np.zeros(3), f, 0.0, inter)[0]
        turn = np.angle((y[1, 0, a] + 1j * y[1, 0, b]) / (z0[1, 0, a] + 1j * z0[1, 0, b]))
        assert np.isclose(turn, 1.0)
