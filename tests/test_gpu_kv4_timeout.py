"""The bounded waits of the attention kernels over the 4-bit cache, made to run out without a fault: a test build leaves the
copy of the first keys of the first lane unissued, so that the wait for it can only run out.  The kernel reports
GDN_ERRBIT_TIMEOUT, drains the copies it did issue and ends; the product library then runs the same call correctly."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_mtp_gb300 as gdn
from test_gpu_kv4 import attend, check_attend
from test_gpu_timeout import run_with, timeout_lib  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


# rows a key head: the decode kernel with 8 and with 32, the one for prompts with one tile of rows and with two
@pytest.mark.parametrize("T,HQ,HK,D", [(1, 8, 1, 128), (4, 8, 1, 128), (2, 4, 1, 256), (8, 8, 1, 64), (40, 8, 1, 128), (20, 4, 1, 256)])
def test_a_copy_that_never_lands(timeout_lib, monkeypatch, T, HQ, HK, D):  # noqa: F811
    rng = np.random.default_rng(T + D)
    r = attend(rng, [T, T], [300, 500], HQ, HK, D, 64)
    good = r["o"].clone()

    def call():
        r["call"]()
        torch.cuda.synchronize()

    run_with(timeout_lib, monkeypatch, call)
    assert int(r["err"]) & gdn.ERRBIT_TIMEOUT, "the wait did not report running out"
    r["err"].zero_()
    call()
    assert torch.equal(r["o"], good)
    check_attend(r, rows_per_lane=8)
