"""Refusals of the linear-attention and sampling calls on the host, before anything reaches the GPU (no GPU needed)."""
import ctypes
import os

import numpy as np
import pytest

import gated_deltanet_linear_mtp_gb300 as gdn
import linear_ref
from gated_deltanet_linear_mtp_gb300 import build as gbuild

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
BAD4 = ctypes.c_void_p(0x10002)
BAD1 = ctypes.c_void_p(0x10001)
OK, NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, VALUE = 0, 1, 2, 3, 4, 5, 7


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gbuild.LIB_PATH):
        gbuild.build()
    return gdn.lib()


def dims(**kw):
    base = dict(B=4, T=2, HK=2, HV=4, DK=64, DV=32, num_slots=8, qkv_dtype=1, state_dtype=1, out_dtype=1, scale=1.0, l2_eps=float("nan"))
    base.update(kw)
    return gdn.GdnDims(**base)


def call(L, name, d=True, n_bytes=1 << 40, **kw):
    ptr = dict(q=P, k=P, v=P, ld=P, pool=P, idx=P, out=P, o=P, acc=P, cu=P, has=P, ws=P, states=P, err=P)
    ptr.update({k: v for k, v in kw.items() if k in ptr})
    dd = ctypes.byref(dims(**{k: v for k, v in kw.items() if k not in ptr})) if d else None
    a = ptr
    if name == "decode":
        return L.gdn_linear_decode(dd, a["q"], a["k"], a["v"], a["ld"], a["pool"], a["idx"], a["out"], a["o"], a["err"], None)
    if name == "verify":
        return L.gdn_linear_verify(dd, a["q"], a["k"], a["v"], a["ld"], a["pool"], a["idx"], a["o"], a["states"], a["err"], None)
    if name == "commit":
        return L.gdn_linear_commit(dd, a["k"], a["v"], a["ld"], a["pool"], a["idx"], a["out"], a["acc"], a["err"], None)
    return L.gdn_linear_prefill(dd, a["cu"], a["q"], a["k"], a["v"], a["ld"], a["pool"], a["idx"], a["out"], a["has"], a["o"], a["ws"], n_bytes, a["err"],
                                None)


ALL = ("decode", "verify", "commit", "prefill")
COMMON = [(dict(d=False), NULL), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(HK=0), SHAPE), (dict(HK=3), SHAPE), (dict(HV=0), SHAPE),
          (dict(DV=0), SHAPE), (dict(DK=0), SHAPE), (dict(DK=48), UNSUPPORTED), (dict(DK=512), UNSUPPORTED), (dict(num_slots=0), SHAPE),
          (dict(qkv_dtype=2), DTYPE), (dict(state_dtype=-1), DTYPE), (dict(out_dtype=7), DTYPE), (dict(scale=float("inf")), VALUE),
          (dict(k=None), NULL), (dict(v=None), NULL), (dict(ld=None), NULL), (dict(pool=None), NULL), (dict(idx=None), NULL),
          (dict(k=ODD), ALIGN), (dict(pool=ODD), ALIGN), (dict(v=BAD1), ALIGN), (dict(ld=BAD4), ALIGN), (dict(idx=BAD4), ALIGN),
          (dict(err=BAD4), ALIGN), (dict(B=0, k=None, q=None), OK)]


@pytest.mark.parametrize("name", ALL)
@pytest.mark.parametrize("kw,status", COMMON)
def test_refusals_of_all(L, name, kw, status):
    assert call(L, name, **kw) == status


@pytest.mark.parametrize("name,kw,status", [
    ("decode", dict(T=0), SHAPE), ("verify", dict(T=17), SHAPE), ("commit", dict(T=0), SHAPE), ("prefill", dict(T=-1), SHAPE),
    ("decode", dict(q=None), NULL), ("verify", dict(o=None), NULL), ("prefill", dict(q=None), NULL), ("decode", dict(q=ODD), ALIGN),
    ("decode", dict(o=BAD1), ALIGN), ("decode", dict(out=BAD4), ALIGN), ("verify", dict(states=ODD), ALIGN), ("commit", dict(acc=None), NULL),
    ("commit", dict(acc=BAD4), ALIGN), ("commit", dict(out=BAD4), ALIGN), ("prefill", dict(cu=None), NULL), ("prefill", dict(cu=BAD4), ALIGN),
    ("prefill", dict(has=BAD4), ALIGN), ("prefill", dict(ws=ODD), ALIGN), ("prefill", dict(T=0, out=None), OK),
    ("prefill", dict(B=1, T=4096, HV=2, ws=None), NULL), ("prefill", dict(B=1, T=4096, HV=2, n_bytes=64), SHAPE)])
def test_refusals_of_each(L, name, kw, status):
    assert call(L, name, **kw) == status


def test_workspace_sizes(L):
    f = L.gdn_linear_prefill_workspace
    for bad in ((-1, 8, 2, 64, 64), (65536, 8, 2, 64, 64), (1, -1, 2, 64, 64), (1, 8, 0, 64, 64), (1, 8, 2, 48, 64), (1, 8, 2, 64, 0)):
        assert f(*bad) == -1
    assert f(0, 0, 2, 64, 64) == 0 and f(1, 100, 2, 128, 128) == 0 and f(64, 65536, 32, 128, 128) == 0
    assert f(1, 16384, 16, 128, 128) > 0 and f(1, 16384, 16, 32, 128) == 0
    assert f(1, 2 ** 31 - 1, 1, 128, 64) > 0


def probs(L, d=True, **kw):
    base = dict(B=2, T=3, V=100, dtype=1, logits_stride=100, probs_stride=128)
    ptr = dict(x=P, t=P, y=P, err=P)
    base.update({k: v for k, v in kw.items() if k in base})
    ptr.update({k: v for k, v in kw.items() if k in ptr})
    return L.gdn_token_probs(ctypes.byref(gdn._TokenDimsC(**base)) if d else None, ptr["x"], ptr["t"], ptr["y"], ptr["err"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=False), NULL), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(T=0), SHAPE), (dict(V=0), SHAPE), (dict(V=2 ** 30 + 1), SHAPE),
    (dict(B=65535, T=32769), SHAPE), (dict(dtype=3), DTYPE), (dict(logits_stride=99), SHAPE), (dict(probs_stride=99), SHAPE),
    (dict(probs_stride=2 ** 31 + 1), SHAPE), (dict(x=None), NULL), (dict(t=None), NULL), (dict(y=None), NULL), (dict(x=BAD1), ALIGN),
    (dict(x=BAD4, dtype=0), ALIGN), (dict(y=BAD4), ALIGN), (dict(t=BAD4), ALIGN), (dict(err=BAD4), ALIGN), (dict(B=0, x=None), OK)])
def test_probs_refusals(L, kw, status):
    assert probs(L, **kw) == status


def accept(L, d=True, **kw):
    base = dict(B=2, T=3, V=100, target_stride=100, draft_stride=100)
    ptr = dict(p=P, x=P, q=P, u=P, idx=P, n=P, tok=P, err=P)
    base.update({k: v for k, v in kw.items() if k in base})
    ptr.update({k: v for k, v in kw.items() if k in ptr})
    return L.gdn_draft_accept(ctypes.byref(gdn._AcceptDimsC(**base)) if d else None, ptr["p"], ptr["x"], ptr["q"], ptr["u"], ptr["idx"], ptr["n"], ptr["tok"],
                              ptr["err"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=False), NULL), (dict(B=-1), SHAPE), (dict(T=0), SHAPE), (dict(T=17), SHAPE), (dict(V=0), SHAPE), (dict(V=2 ** 30 + 1), SHAPE),
    (dict(target_stride=99), SHAPE), (dict(draft_stride=99), SHAPE), (dict(p=None), NULL), (dict(x=None), NULL), (dict(u=None), NULL),
    (dict(n=None), NULL), (dict(tok=None), NULL), (dict(p=BAD4), ALIGN), (dict(q=BAD4), ALIGN), (dict(idx=BAD4), ALIGN), (dict(tok=BAD4), ALIGN),
    (dict(err=BAD4), ALIGN), (dict(B=0, p=None), OK), (dict(q=None, draft_stride=0, p=BAD4), ALIGN)])
def test_accept_refusals(L, kw, status):
    assert accept(L, **kw) == status


def test_the_plain_forms_by_hand():
    p, _ = linear_ref.softmax(np.array([0.0, np.log(3.0), -np.inf]), 1.0)
    assert np.allclose(p, [0.25, 0.75, 0])
    assert linear_ref.softmax(np.array([1.0, 2.0, 2.0]), 0.0)[0].tolist() == [0, 1, 0]
    p, q = np.array([[0.5, 0.5], [0.25, 0.75]], np.float32), np.array([[0.9, 0.1]], np.float32)
    assert linear_ref.accept(p, q, [0], [0.6, 0.3]) == (1, [1, -1])  # 0.54 >= 0.5: refused, r = (0, 0.4)
    assert linear_ref.accept(p, q, [0], [0.5, 0.3]) == (2, [0, 1])   # 0.45 < 0.5: accepted, 0.3 > 0.25
    assert linear_ref.accept(p, None, [1], [0.6, 0.0]) == (1, [0, -1])
