"""The Python binding against the header: every call's parameters, one by one (no GPU needed).  ctypes converts what its argtypes
do not name by itself, a pointer to 32 bits."""
import ctypes
import os
import re

import pytest

import gated_deltanet_linear_mtp_gb300 as gdn
from gated_deltanet_linear_mtp_gb300 import build as gbuild

HEADER = os.path.join(gbuild.INCLUDE, "gdn.h")


def prototypes():
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    out = {}
    for name, args in re.findall(r"GDN_API\s+[\w\s*]+?\b(gdn_\w+)\(([^)]*)\)\s*;", text):
        out[name] = [] if args.strip() in ("", "void") else [" ".join(a.split()) for a in args.split(",")]
    return out


def kind_of_parameter(a):
    if "*" in a or "gdn_stream_t" in a:
        return "pointer"
    return next(k for k in ("int64_t", "int32_t", "float", "gdn_status") if k in a)


def kind_of_ctype(t):
    if t is ctypes.c_void_p or t is ctypes.c_char_p or issubclass(t, ctypes._Pointer):
        return "pointer"
    return {ctypes.c_int64: "int64_t", ctypes.c_int32: "int32_t", ctypes.c_float: "float"}[t]


def test_the_header_names_every_export():
    assert sorted(prototypes()) == sorted(gdn.EXPORTS)


@pytest.mark.parametrize("name", gdn.EXPORTS)
def test_argument_types_are_the_headers(name):
    if not os.path.exists(gbuild.LIB_PATH):
        gbuild.build()
    want = ["int32_t" if k == "gdn_status" else k for k in map(kind_of_parameter, prototypes()[name])]
    got = [kind_of_ctype(t) for t in getattr(gdn.lib(), name).argtypes or ()]
    assert got == want
