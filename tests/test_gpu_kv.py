"""The paged 8-bit key/value cache and its attention on the GPU, against the plain forms of kv_ref.

The append is compared bit for bit (codes, steps, rotated queries); attention with the bound that its
documented roundings give for each output element."""
import numpy as np
import pytest
import torch

import kv_ref
import ternary_weight_fwd_b200 as tw
from kv_util import DEV, dev, make_batch, make_cache, rows, same_bits, to_dev

pytestmark = pytest.mark.gpu

MARK = 0.0078125  # a bf16 value that rows of no sequence keep


@pytest.fixture(autouse=True)
def _clean_status():
    tw.bitnet_device_status()
    tw.bitnet_batch_status()
    yield
    assert tw.bitnet_device_status() == 0
    assert tw.bitnet_batch_status() == 0


def marked(shape):
    return torch.full(shape, MARK, dtype=torch.bfloat16, device=DEV)


def check_append(b, cache, hq, hk, d, dtype, seed, rope=True, with_q=True, scale=1.0, fused=False):
    t = b["rows"]
    dc = to_dev(cache)
    if fused:
        x, xf = rows((t, (hq + 2 * hk) * d), seed, dtype, scale)
        cut = [slice(0, hq * d), slice(hq * d, (hq + hk) * d), slice((hq + hk) * d, None)]
        (q, k, v), (qf, kf, vf) = ([y[:, c].reshape(t, -1, d) if isinstance(y, np.ndarray) else y[:, c].unflatten(1, (-1, d))
                                    for c in cut] for y in (x, xf))
    else:
        (q, qf), (k, kf), (v, vf) = (rows((t, n, d), seed + i, dtype, scale) for i, n in enumerate((hq, hk, hk)))
    tab = kv_ref.rope_table(int(b["lens"].max()) if len(b["lens"]) else 1, d) if rope else None
    ref = [np.array(x) for x in cache]
    qr = kv_ref.append(ref, b["table"], b["lens"], b["q_start"], kf, vf, qf if with_q else None, tab)
    out = marked((t, hq, d)) if with_q else None
    got = tw.bitnet_kv_append(dc, dev(b["table"]), dev(b["lens"]), dev(b["q_start"]), k, v, q=q if with_q else None,
                              rope=None if tab is None else dev(tab), q_out=out)
    torch.cuda.synchronize()
    for x, y, name in zip(dc, ref, ("k", "v", "k_step", "v_step")):
        assert same_bits(x.cpu().numpy(), y), name
    if with_q:
        assert got is out
        end = int(b["q_start"][-1])
        assert same_bits(out[:end].float().cpu().numpy(), qr[:end])
        assert (out[end:] == MARK).all()
    else:
        assert got is None
    return dc


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_shapes(page, d, dtype):
    """Empty sequences, single tokens, page borders, whole pages, several pages; padding behind."""
    new = [1, 0, page, 3, 2 * page + 5, 1, page - 1, 7]
    lens = [1, 9, page, page + 2, 3 * page + 4, 5 * page + 1, 2 * page, page + 3]
    b = make_batch(new, lens, page, page + d, behind=3)
    cache = make_cache(b["pages"], 3, page, d, page * d, b["free"])
    check_append(b, cache, 6, 3, d, dtype, 11)


@pytest.mark.parametrize("hq,hk", [(20, 5), (1, 1), (8, 1), (7, 7), (5, 1), (32, 2)])
def test_append_heads_and_fused_rows(hq, hk):
    """q, k and v as parts of one projection's rows."""
    b = make_batch([1, 70, 2], [200, 70, 33], 32, 3, behind=1)
    cache = make_cache(b["pages"], hk, 32, 128, 5, b["free"])
    check_append(b, cache, hq, hk, 128, "bf16", 21, fused=True)


@pytest.mark.parametrize("rope,with_q", [(False, True), (True, False), (False, False)])
def test_append_without_rotation_or_queries(rope, with_q):
    b = make_batch([4, 40], [20, 41], 16, 4)
    cache = make_cache(b["pages"], 2, 16, 64, 6, b["free"])
    check_append(b, cache, 4, 2, 64, "f32", 31, rope=rope, with_q=with_q)


def test_append_steps_grow_and_stay():
    """Token by token with growing and shrinking values: earlier codes follow a growing step, and a
    smaller token leaves it."""
    page, d, hk = 32, 128, 2
    cache = make_cache(3, hk, page, d, 7)
    for i, scale in enumerate([1.0, 0.01, 3.0, 2.0, 100.0, 0.0, 1e-3, 101.0]):
        n = 1 + i % 3
        done = sum(1 + j % 3 for j in range(i))
        b = dict(table=np.array([[2, 0]], np.int32), lens=np.array([done + n], np.int32),
                 q_start=np.array([0, n], np.int32), pages=3, rows=n)
        cache = [x.cpu().numpy() for x in check_append(b, cache, 4, hk, d, "bf16", 40 + i, scale=scale)]


def test_append_extreme_values():
    """Zeros, subnormals and the largest bf16 values: steps of 0, subnormal steps, codes clamped."""
    for i, scale in enumerate([0.0, 1e-44, 1e-39, 1e-30, 1e37]):
        b = make_batch([3, 17], [3, 40], 16, 50 + i)
        cache = make_cache(b["pages"], 1, 16, 64, 60 + i, b["free"])
        check_append(b, cache, 1, 1, 64, "f32", 70 + i, rope=False, scale=scale)


def test_append_again_changes_nothing():
    b = make_batch([5, 33], [21, 33], 32, 8)
    cache = make_cache(b["pages"], 2, 32, 128, 9, b["free"])
    once = [x.cpu().numpy() for x in check_append(b, cache, 2, 2, 128, "bf16", 80)]
    twice = [x.cpu().numpy() for x in check_append(b, once, 2, 2, 128, "bf16", 80)]
    assert all(same_bits(x, y) for x, y in zip(once, twice))


def test_append_queries_in_place():
    b = make_batch([6, 1], [6, 50], 16, 10)
    cache = make_cache(b["pages"], 2, 16, 128, 11, b["free"])
    x, xf = rows((7, (8 + 4) * 128), 90)
    q, k, v = x[:, :1024].unflatten(1, (8, 128)), x[:, 1024:1280].unflatten(1, (2, 128)), x[:, 1280:].unflatten(1, (2, 128))
    tab = kv_ref.rope_table(50, 128)
    ref = [np.array(y) for y in cache]
    qr = kv_ref.append(ref, b["table"], b["lens"], b["q_start"], xf[:, 1024:1280].reshape(7, 2, 128),
                       xf[:, 1280:].reshape(7, 2, 128), xf[:, :1024].reshape(7, 8, 128), tab)
    dc = to_dev(cache)
    tw.bitnet_kv_append(dc, dev(b["table"]), dev(b["lens"]), dev(b["q_start"]), k, v, q=q, rope=dev(tab), q_out=q)
    torch.cuda.synchronize()
    assert same_bits(q.float().cpu().numpy(), qr)
    assert all(same_bits(a.cpu().numpy(), c) for a, c in zip(dc, ref))


def test_append_many_sequences():
    """More sequences than threads of a CTA."""
    r = np.random.default_rng(12)
    new = r.integers(0, 3, 700).tolist()
    lens = [n + int(r.integers(0, 40)) for n in new]
    b = make_batch(new, lens, 16, 13)
    cache = make_cache(b["pages"], 1, 16, 64, 14, b["free"])
    check_append(b, cache, 2, 1, 64, "bf16", 91)


def test_rope_table():
    """Angles in fp64, so far positions keep their bits: each entry within a rounding of fp32 (2^-24, and
    2^-52 times the angle before it)."""
    n, d = 200001, 128
    t = tw.bitnet_rope_table(n, d).cpu().numpy()
    w = 500000.0 ** (-2.0 * np.arange(d // 2) / d)
    for p in (0, 1, 77, 4095, 131071, 200000):
        ref = np.concatenate([np.cos(p * w), np.sin(p * w)])
        assert np.abs(t[p] - ref).max() <= 2.0 ** -24 + 4 * p * 2.0 ** -52


def check_attention(b, cache, hq, d, seed, max_new=None, scale=None, qscale=1.5, dc=None):
    hk = cache[0].shape[1]
    q, qf = rows((b["rows"], hq, d), seed, scale=qscale)
    new = np.diff(b["q_start"])
    out = marked(q.shape)
    got = tw.bitnet_attention(dc or to_dev(cache), dev(b["table"]), dev(b["lens"]), dev(b["q_start"]), q,
                              max_new or max(1, int(new.max())), scale=scale, out=out)
    torch.cuda.synchronize()
    assert got is out
    ref = kv_ref.attention(cache, b["table"], b["lens"], b["q_start"], qf, scale)
    bound = kv_ref.attention_bound(cache, b["table"], b["lens"], b["q_start"], qf, ref, scale)
    end = int(b["q_start"][-1])
    o = out.float().cpu().numpy()
    assert (o[end:] == MARK).all()
    err = np.abs(o[:end] - ref[:end])
    bad = ~(err <= bound[:end])
    assert not bad.any(), (np.argwhere(bad)[:5], err[bad][:5], bound[:end][bad][:5])
    return o


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_tokens_lengths(page, d):
    """One new token per sequence; contexts of one token, group, chunk and page borders, empty sequences,
    sequences without new tokens."""
    lens = [1, 2, 15, 16, 17, 0, 31, 33, 127, 128, 129, 255, 257, 64, 500, 1000]
    new = [1] * len(lens)
    new[13] = 0
    b = make_batch(new, lens, page, page + d, behind=2)
    cache = make_cache(b["pages"], 2, page, d, page * d + 1, b["free"])
    check_attention(b, cache, 8, d, 101)


@pytest.mark.parametrize("hq,hk,n", [(20, 5, 1), (1, 1, 1), (16, 1, 1), (5, 1, 3), (32, 1, 1), (7, 1, 4), (12, 4, 8),
                                     (6, 6, 16), (3, 3, 32)])
@pytest.mark.parametrize("d", [64, 128])
def test_tokens_heads_and_drafts(hq, hk, n, d):
    """Groups of any size, several new tokens (each sees itself and what came before), some sequences
    shorter than their new tokens."""
    lens = [n, n + 1, max(1, n - 1), 130, 300 + n]
    b = make_batch([n, max(1, n - 1), n, n, n], lens, 32, hq + n, behind=1)
    cache = make_cache(b["pages"], hk, 32, d, hq * n, b["free"])
    check_attention(b, cache, hq, d, 111, max_new=n)


def test_tokens_long_and_many():
    """One long sequence cut over all CTAs; then many short ones."""
    b = make_batch([1], [20011], 64, 15)
    check_attention(b, make_cache(b["pages"], 2, 64, 128, 16, b["free"]), 4, 128, 121)
    r = np.random.default_rng(17)
    lens = r.integers(0, 300, 400).tolist()
    b = make_batch([1] * 400, lens, 16, 18)
    check_attention(b, make_cache(b["pages"], 1, 16, 64, 19, b["free"]), 2, 64, 122)


@pytest.mark.parametrize("qscale", [0.0, 1e-30, 1e-3, 30.0, 1e4])
def test_tokens_query_range(qscale):
    """Queries far below and above fp16's range."""
    b = make_batch([2, 2], [200, 77], 16, 20)
    check_attention(b, make_cache(b["pages"], 1, 16, 128, 21, b["free"]), 4, 128, 131, qscale=qscale, scale=0.01)


def test_tokens_steps_of_any_size():
    """Steps of neighbouring pages many orders of magnitude apart, pages of zeros."""
    b = make_batch([1, 1, 1], [400, 400, 90], 16, 22)
    cache = make_cache(b["pages"], 1, 16, 128, 23, b["free"])
    r = np.random.default_rng(24)
    cache[3][:] = (10.0 ** r.uniform(-12, 6, cache[3].shape)).astype(np.float32)
    cache[3][b["table"][0, :3]] = 0.0
    cache[2][b["table"][1, 2:5]] = 0.0
    check_attention(b, cache, 4, 128, 132)


def test_tokens_same_bits_every_time():
    b = make_batch([1] * 9, [3000, 1, 700, 64, 5000, 129, 12, 2048, 999], 32, 25)
    cache = make_cache(b["pages"], 3, 32, 128, 26, b["free"])
    a = check_attention(b, cache, 12, 128, 141)
    for _ in range(3):
        assert same_bits(a, check_attention(b, cache, 12, 128, 141))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_lengths(page, d):
    """Whole prompts and chunks of lengths around rows, tiles, blocks and pages; sequences without new
    tokens, with fewer cached than new tokens, with none."""
    new = [40, 1, 0, 63, 64, 65, 130, 200, 5, 3, 33]
    lens = [40, 300, 7, 63, 64, 200, 130, 333, 3, 0, 128]
    b = make_batch(new, lens, page, page + d + 1, behind=2)
    cache = make_cache(b["pages"], 2, page, d, page * d + 2, b["free"])
    check_attention(b, cache, 8, d, 151)


@pytest.mark.parametrize("hq,hk", [(20, 5), (1, 1), (3, 3), (7, 1), (32, 1), (12, 4), (128, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_heads(hq, hk, d):
    """Groups of any size, those that do not divide a row tile among them."""
    new, lens = [37, 150, 2], [37, 190, 500]
    b = make_batch(new, lens, 64, hq)
    check_attention(b, make_cache(b["pages"], hk, 64, d, hq, b["free"]), hq, d, 161, max_new=150)


@pytest.mark.parametrize("n,length,hq,hk", [(1000, 1000, 4, 1), (64, 5000, 4, 2), (700, 2111, 5, 5)])
def test_prompt_long(n, length, hq, hk):
    """Tiles shared by several CTAs."""
    b = make_batch([n], [length], 32, n)
    check_attention(b, make_cache(b["pages"], hk, 32, 128, n + 1, b["free"]), hq, 128, 171)


def test_prompt_many_sequences():
    r = np.random.default_rng(31)
    new = r.integers(0, 60, 300).tolist()
    lens = [n + int(r.integers(0, 90)) for n in new]
    b = make_batch(new, lens, 16, 32, behind=1)
    check_attention(b, make_cache(b["pages"], 1, 16, 64, 33, b["free"]), 1, 64, 172)


@pytest.mark.parametrize("qscale", [0.0, 1e-30, 1e-3, 30.0, 1e4])
def test_prompt_query_range(qscale):
    b = make_batch([50, 20], [200, 20], 16, 34)
    check_attention(b, make_cache(b["pages"], 1, 16, 128, 35, b["free"]), 4, 128, 181, qscale=qscale, scale=0.01)


def test_prompt_steps_of_any_size():
    """Steps of neighbouring pages up to nine orders of magnitude apart, pages of zeros."""
    b = make_batch([90, 60], [400, 290], 16, 36)
    cache = make_cache(b["pages"], 1, 16, 128, 37, b["free"])
    r = np.random.default_rng(38)
    cache[3][:] = (10.0 ** r.uniform(-6, 3, cache[3].shape)).astype(np.float32)
    cache[3][b["table"][0, :3]] = 0.0
    cache[2][b["table"][1, 2:5]] = 0.0
    cache[3][b["table"][1, :8]] = 0.0  # a whole first block of zeros
    check_attention(b, cache, 4, 128, 182)


def test_prompt_same_bits_every_time():
    b = make_batch([300, 1, 77, 512], [900, 1, 77, 2048], 32, 39)
    cache = make_cache(b["pages"], 3, 32, 128, 40, b["free"])
    a = check_attention(b, cache, 12, 128, 191)
    for _ in range(3):
        assert same_bits(a, check_attention(b, cache, 12, 128, 191))
