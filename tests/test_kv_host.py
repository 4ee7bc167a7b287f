"""The key/value cache's entry points refuse bad arguments on the host, before anything is launched, and
its host-only sizes (no GPU needed)."""
import ctypes

import pytest
import torch

import ternary_weight_fwd_b200 as tw

P = 1 << 40  # a 16-byte aligned non-null address; never dereferenced
INVALID, SHAPE, MISALIGNED, WORKSPACE = (tw.BITNET_ERR_INVALID_ARG, tw.BITNET_ERR_UNSUPPORTED_SHAPE,
                                         tw.BITNET_ERR_MISALIGNED, tw.BITNET_ERR_WORKSPACE)


C = 1 << 41  # the cache


def structs(**kw):
    a = dict(k=C, v=C + (1 << 20), k_step=C + (2 << 20), v_step=C + (3 << 20), num_pages=8, n_kv_heads=2, page_size=32, head_dim=64, page_table=P,
             seq_lens=P, q_start=P, table_width=4, n_seqs=3, T=5)
    a.update({x: y for x, y in kw.items() if x in a})
    c = tw.bitnet_kv_cache_t(*(a[x] for x in ("k", "v", "k_step", "v_step", "num_pages", "n_kv_heads", "page_size",
                                              "head_dim")))
    b = tw.bitnet_kv_batch_t(*(a[x] for x in ("page_table", "seq_lens", "q_start", "table_width", "n_seqs", "T")))
    return c, b


COMMON = [
    (dict(k=None), INVALID), (dict(v_step=None), INVALID), (dict(page_table=None), INVALID),
    (dict(num_pages=0), INVALID), (dict(n_kv_heads=0), INVALID), (dict(n_seqs=0), INVALID), (dict(T=0), INVALID),
    (dict(table_width=0), INVALID), (dict(page_size=48), SHAPE), (dict(page_size=256), SHAPE),
    (dict(head_dim=96), SHAPE), (dict(n_kv_heads=2000), SHAPE), (dict(num_pages=1 << 31), SHAPE),
    (dict(n_seqs=70000), SHAPE), (dict(T=(1 << 24) + 1), SHAPE), (dict(table_width=1 << 27), SHAPE),
    (dict(k=C + 8), MISALIGNED), (dict(k_step=C + 2), MISALIGNED), (dict(q_start=P + 1), MISALIGNED),
]


@pytest.mark.parametrize("case,expect", COMMON + [
    (dict(k_rows=None), INVALID), (dict(v_rows=None), INVALID), (dict(dtype=2), INVALID),
    (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(heads=0), INVALID), (dict(heads=3), SHAPE),
    (dict(heads=512), SHAPE), (dict(q_stride=64 * 3), SHAPE), (dict(k_stride=120), SHAPE),
    (dict(q_stride=64 * 4 + 4), MISALIGNED), (dict(k_rows=P + (1 << 20) + 8), MISALIGNED), (dict(rope=P + 4), MISALIGNED),
    (dict(rope_len=0), INVALID),
    # q_out over the new keys' rows; over q shifted by one row; over q of another type
    (dict(q_out=P + (1 << 20)), INVALID), (dict(q_out=P + 512), INVALID), (dict(q_out=P, dtype=1), INVALID),
    (dict(q_out=C), INVALID), (dict(q_out=C + (3 << 20)), INVALID),  # over the cache
])
def test_append_refuses(case, expect):
    a = dict(q=P, k_rows=P + (1 << 20), v_rows=P + (2 << 20), dtype=0, heads=4, q_stride=256, k_stride=128, v_stride=128,
             rope=P, rope_len=64, q_out=P + (3 << 20), q_out_stride=256)
    a.update(case)
    c, b = structs(**case)
    st = tw.load_library().bitnet_kv_append(c, b, a["q"], a["k_rows"], a["v_rows"], a["dtype"], a["heads"],
                                            a["q_stride"], a["k_stride"], a["v_stride"], a["rope"], a["rope_len"],
                                            a["q_out"], a["q_out_stride"], None)
    assert st == expect


@pytest.mark.parametrize("case,expect", COMMON + [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(heads=0), INVALID), (dict(heads=3), SHAPE),
    (dict(max_new=0), INVALID), (dict(max_new=6), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(q_stride=200), SHAPE),
    (dict(out_stride=260), MISALIGNED), (dict(q=P + 8), MISALIGNED), (dict(out=P + 512), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE), (dict(ws=P + (4 << 20) + 4), MISALIGNED),
    (dict(scale=3e38), INVALID), (dict(out=C + 256), INVALID), (dict(ws=C), INVALID), (dict(ws=P), INVALID),
    (dict(ws=P + (1 << 20)), INVALID),  # over the cache, q, out
])
def test_attention_refuses(case, expect):
    need = tw.bitnet_attention_workspace_size(3, 5, 4, 2, 64, 2)
    assert need > 0
    a = dict(q=P, q_stride=256, heads=4, max_new=2, scale=0.125, out=P + (1 << 20), out_stride=256, ws=P + (4 << 20),
             ws_bytes=need)
    a.update(case)
    c, b = structs(**case)
    st = tw.load_library().bitnet_attention(c, b, a["q"], a["q_stride"], a["heads"], a["max_new"], a["scale"], a["out"],
                                            a["out_stride"], a["ws"], a["ws_bytes"], None)
    assert st == expect


def test_structs_are_required():
    lib = tw.load_library()
    c, b = structs()
    assert lib.bitnet_attention(None, b, P, 256, 4, 1, 0.1, P, 256, P, 1 << 30, None) == INVALID
    assert lib.bitnet_kv_append(c, None, None, P, P, 0, 0, 0, 128, 128, None, 0, None, 0, None) == INVALID


def test_rope_table_refuses():
    f = tw.load_library().bitnet_rope_table
    assert f(0.0, 8, 64, P, None) == INVALID
    assert f(float("inf"), 8, 64, P, None) == INVALID
    assert f(1e4, 0, 64, P, None) == INVALID
    assert f(1e4, 8, 64, None, None) == INVALID
    assert f(1e4, 8, 80, P, None) == SHAPE
    assert f(1e4, (1 << 24) + 1, 64, P, None) == SHAPE
    assert f(1e4, 8, 64, P + 8, None) == MISALIGNED


def test_workspace_sizes():
    size = tw.bitnet_attention_workspace_size
    assert size(1, 1, 20, 5, 128, 1) > 0
    assert size(1, 1, 20, 5, 128, 1) <= size(64, 64, 20, 5, 128, 1) <= size(64, 512, 20, 5, 128, 8)
    for bad in ((0, 1, 4, 2, 64, 1), (1, 0, 4, 2, 64, 1), (1, 1, 3, 2, 64, 1), (1, 1, 4, 2, 96, 1), (1, 1, 4, 2, 64, 2),
                (1, 1, 4, 0, 64, 1), (1, 4, 4, 2, 64, 0), (1, 1, 258, 2, 64, 1)):
        assert size(*bad) == 0


def cpu_args():
    cache = (torch.zeros((4, 2, 16, 64), dtype=torch.int8), torch.zeros((4, 2, 16, 64), dtype=torch.int8),
             torch.zeros((4, 2)), torch.zeros((4, 2)))
    meta = (torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    return cache, meta


def test_wrappers_refuse_wrong_tensors():
    """Types, shapes, strides and devices, before the library is called."""
    (k, v, ks, vs), (table, lens, starts) = cpu_args()
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    kv = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    for cache in ((k.float(), v, ks, vs), (k, v, ks.double(), vs)):
        with pytest.raises(TypeError):
            tw.bitnet_attention(cache, table, lens, starts, q, 1)
    with pytest.raises(TypeError):
        tw.bitnet_attention((k, v, ks, vs), table.long(), lens, starts, q, 1)
    with pytest.raises(TypeError):
        tw.bitnet_attention((k, v, ks, vs), table, lens, starts, q.float(), 1)
    with pytest.raises(TypeError):
        tw.bitnet_kv_append((k, v, ks, vs), table, lens, starts, kv, kv.float())
    with pytest.raises(ValueError, match="GPU"):
        tw.bitnet_attention((k, v, ks, vs), table, lens, starts, q, 1)
    for bad in (dict(q=q[:, :, :32]), dict(q=q.transpose(1, 2)), dict(starts=starts[:1]), dict(table=table.t()),
                dict(v=v[:2]), dict(ks=ks[:2])):
        a = dict(k=k, v=v, ks=ks, vs=vs, table=table, lens=lens, starts=starts, q=q)
        a.update(bad)
        with pytest.raises(ValueError):
            tw.bitnet_attention((a["k"], a["v"], a["ks"], a["vs"]), a["table"], a["lens"], a["starts"], a["q"], 1)
    with pytest.raises(ValueError):
        tw.bitnet_kv_append((k, v, ks, vs), table, lens, starts, kv, kv[:2])
    with pytest.raises(ValueError):
        tw.bitnet_kv_append((k, v, ks, vs), table, lens, starts, kv[:, :1], kv[:, :1])
    with pytest.raises(ValueError, match="GPU"):
        tw.bitnet_rope_table(4, 64, device="cpu")


def test_struct_layouts():
    assert ctypes.sizeof(tw.bitnet_kv_cache_t) == 56
    assert ctypes.sizeof(tw.bitnet_kv_batch_t) == 40
