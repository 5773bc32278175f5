"""Register spills of the kernels of the attention layer over the 4-bit cache, from ptxas's own report (no GPU needed), held to what
they were when the kernels were timed; most of them lie outside the loops.  A kernel that is not named spills nothing."""
from concurrent.futures import ThreadPoolExecutor

import pytest

from gated_deltanet_linear_mtp_gb300 import build as gbuild
from test_build_host import ptxas_spills

# substring of the mangled kernel name: spill-store ceiling in bytes
CEILINGS = {
    "gdn_kv4_attention.cu": {"CfgILi128ELi4E": 24, "CfgILi128ELi1E": 28, "CfgILi64ELi2E": 58},  # 32 rows D 128, 8 rows D 128, 16 rows D 64
    "gdn_kv4_attention_wide.cu": {"WideILi64E": 24},
    "gdn_qk_norm_rope.cu": {  # type, D, with the store, neighbouring pairs
        "I13__nv_bfloat16Li256ELb0ELb0E": 24, "I13__nv_bfloat16Li256ELb0ELb1E": 12, "I13__nv_bfloat16Li256ELb1ELb0E": 108,
        "I13__nv_bfloat16Li256ELb1ELb1E": 72, "I13__nv_bfloat16Li128ELb0ELb0E": 24, "I13__nv_bfloat16Li128ELb0ELb1E": 4,
        "I13__nv_bfloat16Li128ELb1ELb0E": 132, "I13__nv_bfloat16Li128ELb1ELb1E": 68, "I13__nv_bfloat16Li64ELb0ELb0E": 24,
        "I13__nv_bfloat16Li64ELb0ELb1E": 4, "I13__nv_bfloat16Li64ELb1ELb0E": 132, "I13__nv_bfloat16Li64ELb1ELb1E": 68,
        "IfLi256ELb0ELb0E": 56, "IfLi256ELb0ELb1E": 32, "IfLi256ELb1ELb0E": 172, "IfLi256ELb1ELb1E": 240, "IfLi128ELb0ELb0E": 48,
        "IfLi128ELb0ELb1E": 24, "IfLi128ELb1ELb0E": 216, "IfLi128ELb1ELb1E": 244, "IfLi64ELb0ELb0E": 48, "IfLi64ELb0ELb1E": 36,
        "IfLi64ELb1ELb0E": 216, "IfLi64ELb1ELb1E": 244},
    "gdn_page_plan.cu": {},
}


@pytest.fixture(scope="module")
def spills():
    try:
        gbuild.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    with ThreadPoolExecutor(len(CEILINGS)) as ex:
        return dict(zip(CEILINGS, ex.map(ptxas_spills, CEILINGS)))


@pytest.mark.parametrize("src", CEILINGS)
def test_spills_stay_below_their_ceilings(spills, src):
    seen = set()
    for name, got in spills[src].items():
        keys = [k for k in CEILINGS[src] if k in name]
        assert len(keys) < 2, name
        seen.update(keys)
        assert got <= (CEILINGS[src][keys[0]] if keys else 0), (name, got)
    assert seen == set(CEILINGS[src])
