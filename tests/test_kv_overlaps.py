"""What a cache call writes may not be what it reads, beyond the cases that the header allows: refused on the host,
before anything is launched (no GPU needed)."""
import pytest
import torch

import ternary_weight_fwd_b200 as tw
from test_kv_host import C, INVALID, P, structs

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is not refused would launch on made-up addresses")

M = 1 << 20
ROPE, Q_OUT, OUT, WS = P + 5 * M, P + 4 * M, P + 4 * M, P + 6 * M
TABLE, LENS, STARTS = P + 9 * M, P + 10 * M, P + 11 * M
# 8 pages, 2 kv heads, 32 tokens of 64: 32768 bytes of codes, 64 bytes of steps


def append(**case):
    a = dict(q=P, k_rows=P + M, v_rows=P + 2 * M, rope=ROPE, q_out=Q_OUT, page_table=TABLE, seq_lens=LENS, q_start=STARTS)
    a.update(case)
    c, b = structs(**a)
    return tw.load_library().bitnet_kv_append(c, b, a["q"], a["k_rows"], a["v_rows"], 0, 4, 256, 128, 128, a["rope"], 64,
                                              a["q_out"], 256, None)


def attention(**case):
    need = tw.bitnet_attention_workspace_size(3, 5, 4, 2, 64, 2)
    a = dict(q=P, out=OUT, ws=WS, page_table=TABLE, seq_lens=LENS, q_start=STARTS)
    a.update(case)
    c, b = structs(**a)
    return tw.load_library().bitnet_attention(c, b, a["q"], 256, 4, 2, 0.125, a["out"], 256, a["ws"], need, None)


@pytest.mark.parametrize("case", [
    # q_out over the rotation table, the page table, the lengths, the row starts
    dict(q_out=ROPE), dict(q_out=TABLE), dict(q_out=LENS), dict(q_out=STARTS),
    # the cache's arrays over one another
    dict(v=C), dict(v=C + 16384), dict(k_step=C + 1024), dict(v_step=C + 2 * M), dict(v_step=C + 2 * M + 60),
    # new rows, the rotation table or the batch inside the cache
    dict(q=C), dict(k_rows=C + 32752), dict(v_rows=C + M), dict(rope=C), dict(page_table=C), dict(seq_lens=C + 2 * M),
    dict(q_start=C + 3 * M + 60),
])
def test_append_refuses_what_it_would_read_back(case):
    assert append(**case) == INVALID


@pytest.mark.parametrize("case", [
    dict(out=TABLE), dict(out=LENS), dict(out=STARTS), dict(ws=TABLE), dict(ws=LENS), dict(ws=STARTS),
])
def test_attention_refuses_what_it_would_read_back(case):
    assert attention(**case) == INVALID


@pytest.mark.parametrize("case", [
    dict(q_out=P), dict(v=C + 32768), dict(k_rows=C + 32768), dict(q_out=LENS + 16), dict(q_start=LENS),
    dict(rope=None), dict(k_rows=P + M, v_rows=P + M),
])
def test_append_takes_neighbours_and_shared_inputs(case):
    """Not refused for its arguments: without a GPU the launch fails."""
    assert append(**case) == tw.BITNET_ERR_CUDA


def test_attention_takes_keys_that_are_the_values():
    """It only reads the cache; out may be q."""
    assert attention(v=C) == tw.BITNET_ERR_CUDA
    assert attention(out=P) == tw.BITNET_ERR_CUDA
