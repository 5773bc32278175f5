"""The attention-layer calls over the 4-bit cache at the edges of their ranges: tiles of rows that whole tokens do not fill,
launch limits of the page plan, intervals of the store's rounding around zero, values at the ends of the types, and
long contexts.  References and bounds are those of tests/kv4_ref.py unless a test derives its own."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gated_deltanet_linear_mtp_gb300 as gdn
import kv4_ref as ref
from test_gpu_kv4 import I32, attend, check_attend, err_word, f64

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
