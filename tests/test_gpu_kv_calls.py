"""Calls of the key/value cache's operators at the edges of what they take."""
import numpy as np
import pytest
import torch

import kv_exact
import kv_ref
import ternary_weight_fwd_b200 as tw
from kv_util import DEV, dev, make_batch, make_cache, rows, same_bits, to_dev

pytestmark = pytest.mark.gpu

MARK = 0.0078125


@pytest.fixture(autouse=True)
def _clean_status():
    tw.bitnet_device_status()
    tw.bitnet_batch_status()
    yield
    assert tw.bitnet_device_status() == 0
    assert tw.bitnet_batch_status() == 0


def meta(b):
    return dev(b["table"]), dev(b["lens"]), dev(b["q_start"])


def test_sequences_that_claim_the_same_rows_over_and_over():
    """Row starts that fall back again and again: sequences that are sound one by one claim three times the rows
    there are.  Their tiles could outnumber what the workspace has room for, so the kernel for prompts takes none."""
    n = 40
    b = make_batch([n] * 5, [n + 7] * 5, 16, 901)
    b["q_start"] = np.array([0, n, 0, n, 0, n], np.int32)
    cache = make_cache(b["pages"], 2, 16, 64, 902, b["free"])
    q, _ = rows((n, 4, 64), 903)
    out = torch.full(q.shape, MARK, dtype=torch.bfloat16, device=DEV)
    tw.bitnet_attention(to_dev(cache), *meta(b), q, n, out=out)
    assert tw.bitnet_batch_status() == tw.BITNET_ERR_INVALID_ARG
    assert (out == MARK).all()
