"""Register spills of the linear-attention and sampling kernels, from ptxas's own report (no GPU needed), held to what they were when the
kernels were timed.  A kernel that is not named spills nothing."""
from concurrent.futures import ThreadPoolExecutor

import pytest

from gated_deltanet_linear_mtp_gb300 import build as gbuild
from test_build_host import ptxas_spills

# substring of the mangled kernel name: spill-store ceiling in bytes
CEILINGS = {
    "gdn_linear_f32.cu": {
        "gdn_linear_kernelILi256EffLb0EEEvNS": 64,
        "gdn_linear_kernelILi256EffLb1EEEvNS": 80,
        "gdn_linear_kernelILi256E13__nv_bfloat16fLb0EEEvNS": 64,
        "gdn_linear_kernelILi256E13__nv_bfloat16fLb1EEEvNS": 96,
        "gdn_linear_kernelILi128EffLb0EEEvNS": 64,
        "gdn_linear_kernelILi128EffLb1EEEvNS": 96,
        "gdn_linear_kernelILi128E13__nv_bfloat16fLb0EEEvNS": 64,
        "gdn_linear_kernelILi128E13__nv_bfloat16fLb1EEEvNS": 96,
        "gdn_linear_kernelILi64EffLb0EEEvNS": 64,
        "gdn_linear_kernelILi64EffLb1EEEvNS": 96,
        "gdn_linear_kernelILi64E13__nv_bfloat16fLb0EEEvNS": 64,
        "gdn_linear_kernelILi64E13__nv_bfloat16fLb1EEEvNS": 96,
        "gdn_linear_mma_kernelILi64EfLi2ELi0EEEvNS": 16,
        "gdn_linear_mma_kernelILi64EfLi2ELi1EEEvNS": 4,
        "gdn_linear_mma_kernelILi64EfLi2ELi2EEEvNS": 4,
        "gdn_linear_mma_kernelILi64EfLi1ELi2EEEvNS": 16,
        "gdn_linear_kernelILi32EffLb0EEEvNS": 64,
        "gdn_linear_kernelILi32EffLb1EEEvNS": 96,
        "gdn_linear_kernelILi32E13__nv_bfloat16fLb0EEEvNS": 64,
        "gdn_linear_kernelILi32E13__nv_bfloat16fLb1EEEvNS": 96,
        "gdn_linear_kernelILi16EffLb0EEEvNS": 8,
        "gdn_linear_kernelILi16E13__nv_bfloat16fLb0EEEvNS": 40,
    },
    "gdn_linear_bf16.cu": {
        "gdn_linear_kernelILi256Ef13__nv_bfloat16Lb1EEEvNS": 16,
        "gdn_linear_kernelILi256E13__nv_bfloat16S1_Lb0EEEvNS": 32,
        "gdn_linear_kernelILi256E13__nv_bfloat16S1_Lb1EEEvNS": 32,
        "gdn_linear_kernelILi128Ef13__nv_bfloat16Lb1EEEvNS": 16,
        "gdn_linear_kernelILi128E13__nv_bfloat16S1_Lb0EEEvNS": 32,
        "gdn_linear_kernelILi128E13__nv_bfloat16S1_Lb1EEEvNS": 32,
        "gdn_linear_mma_kernelILi128E13__nv_bfloat16Li2ELi0EEEvNS": 112,
        "gdn_linear_mma_kernelILi128E13__nv_bfloat16Li2ELi1EEEvNS": 128,
        "gdn_linear_mma_kernelILi128E13__nv_bfloat16Li2ELi2EEEvNS": 144,
        "gdn_linear_mma_kernelILi128E13__nv_bfloat16Li1ELi0EEEvNS": 64,
        "gdn_linear_mma_kernelILi128E13__nv_bfloat16Li1ELi1EEEvNS": 48,
        "gdn_linear_mma_kernelILi128E13__nv_bfloat16Li1ELi2EEEvNS": 48,
        "gdn_linear_kernelILi64Ef13__nv_bfloat16Lb1EEEvNS": 16,
        "gdn_linear_kernelILi64E13__nv_bfloat16S1_Lb0EEEvNS": 32,
        "gdn_linear_kernelILi64E13__nv_bfloat16S1_Lb1EEEvNS": 32,
        "gdn_linear_kernelILi32Ef13__nv_bfloat16Lb1EEEvNS": 32,
        "gdn_linear_kernelILi32E13__nv_bfloat16S1_Lb0EEEvNS": 32,
        "gdn_linear_kernelILi32E13__nv_bfloat16S1_Lb1EEEvNS": 32,
        "gdn_linear_kernelILi16E13__nv_bfloat16S1_Lb0EEEvNS": 4,
    },
    "gdn_linear_prefill.cu": {},
    "gdn_token_probs.cu": {},
    "gdn_draft_accept.cu": {},
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
    for name, got in spills[src].items():
        keys = [k for k in CEILINGS[src] if k in name]
        assert len(keys) < 2, name
        assert got <= (CEILINGS[src][keys[0]] if keys else 0), (name, got)
