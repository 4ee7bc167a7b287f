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


# Batches that the kernel for prompts takes tile by tile, with tiles of both halves and up to 32 blocks
WHOLE = [([4096], [4096], 20, 5, 128, 64), ([700, 1024, 1, 1000, 1024, 33], [700, 1300, 900, 1000, 2048, 40], 20, 5, 128, 32),
         ([1024, 1000, 1024, 333, 900], [1024, 1000, 1024, 400, 1000], 16, 16, 64, 128),
         ([1999, 1500], [1999, 1500], 28, 14, 128, 16)]


@pytest.mark.parametrize("new,lens,hq,hk,d,page", WHOLE)
def test_prompt_by_whole_tiles(new, lens, hq, hk, d, page):
    """Right, the same bits every time, with the result over the queries, and rows of no sequence left alone."""
    b = make_batch(new, lens, page, 911, behind=3)
    assert kv_exact.whole_tiles(b, hq // hk, hk)
    cache = make_cache(b["pages"], hk, page, d, 912, b["free"])
    q, qf = rows((b["rows"], hq, d), 913)
    ref, bound = kv_exact.attention(cache, b, qf)
    args = (to_dev(cache), *meta(b))
    end = int(b["q_start"][-1])
    outs = []
    for _ in range(4):
        out = torch.full(q.shape, MARK, dtype=torch.bfloat16, device=DEV)
        outs.append(tw.bitnet_attention(args[0], *args[1:], q, max(new), out=out))
    tw.bitnet_attention(args[0], *args[1:], q, max(new), out=q)
    torch.cuda.synchronize()
    o = outs[0].float().cpu().numpy()
    assert (np.abs(o - ref) <= bound)[:end].all()
    assert (outs[0][end:] == MARK).all()
    assert all(torch.equal(x, outs[0]) for x in outs[1:])
    assert torch.equal(q[:end], outs[0][:end])


STRIDED = [([1, 1, 1], [300, 17, 1000], 1, 128), ([3, 1, 2], [300, 17, 1000], 3, 64), ([200, 70], [900, 70], 200, 128),
           ([65, 500], [65, 501], 500, 64)]


@pytest.mark.parametrize("new,lens,max_new,d", STRIDED)
@pytest.mark.parametrize("whole", [False, True])
def test_rows_within_wider_rows(new, lens, max_new, d, whole):
    """Queries rotated in place inside a fused projection's rows, the result written into wider rows: the same as from
    and to rows of their own, and what lies between is left alone."""
    hq, hk, page = 8, 2, 32
    if whole:
        new, lens = new * 40, lens * 40
    b = make_batch(new, lens, page, 921, behind=2)
    if whole and max_new > 12:
        assert kv_exact.whole_tiles(b, hq // hk, hk)
    t = b["rows"]
    cache = make_cache(b["pages"], hk, page, d, 922, b["free"])
    fused, ff = rows((t, (hq + 2 * hk) * d), 923)
    q, k, v = (fused[:, i * d:j * d].unflatten(1, (-1, d)) for i, j in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
    rope = dev(kv_ref.rope_table(max(lens), d))
    apart = to_dev(cache)
    together = to_dev(cache)
    qr = tw.bitnet_kv_append(apart, *meta(b), k.contiguous(), v.contiguous(), q=q.contiguous(), rope=rope)
    want = tw.bitnet_attention(apart, *meta(b), qr, max_new)
    wide = torch.full((t, hq + 3, d), MARK, dtype=torch.bfloat16, device=DEV)
    out = wide[:, 2:2 + hq]
    kv_before = fused[:, hq * d:].clone()
    tw.bitnet_kv_append(together, *meta(b), k, v, q=q, rope=rope, q_out=q)
    tw.bitnet_attention(together, *meta(b), q, max_new, out=out)
    torch.cuda.synchronize()
    end = int(b["q_start"][-1])
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(apart, together))
    assert torch.equal(q[:end], qr[:end]) and torch.equal(fused[:, hq * d:], kv_before)
    assert torch.equal(out[:end], want[:end]) and (out[end:] == MARK).all()
    assert (wide[:, :2] == MARK).all() and (wide[:, 2 + hq:] == MARK).all()
    host = [x.cpu().numpy() for x in apart]
    ref, bound = kv_exact.attention(host, b, qr.float().cpu().numpy())
    assert (np.abs(want.float().cpu().numpy()[:end] - ref[:end]) <= bound[:end]).all()


@pytest.mark.parametrize("n", [1, 70])
def test_pages_beyond_32_bits(n):
    """Codes more than 4 GiB behind the cache's start: the same as in a small cache."""
    hq, hk, page, d = 16, 8, 128, 128
    b = make_batch([n, n], [500, 140], page, 931)
    cache = make_cache(b["pages"], hk, page, d, 932)
    (q, _), (k, _), (v, _) = (rows((b["rows"], h, d), 933 + i) for i, h in enumerate((hq, hk, hk)))
    small = to_dev(cache)
    pages = 2 ** 32 // (hk * page * d) + b["pages"]
    far = pages - b["pages"]
    big = tw.kv_cache(pages, hk, d, page)
    for x, y in zip(big, small):
        x[far:].copy_(y)
    moved = dict(b, table=np.where(b["table"] >= 0, b["table"] + far, b["table"]).astype(np.int32))
    outs = []
    for c, bt in ((small, b), (big, moved)):
        qr = tw.bitnet_kv_append(c, *meta(bt), k, v, q=q)
        outs.append(tw.bitnet_attention(c, *meta(bt), qr, n))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    assert all(torch.equal(x[far:].view(torch.uint8), y.view(torch.uint8)) for x, y in zip(big, small))
    assert not any(x[:far].any() for x in big)


def test_more_sequences_than_the_kernels_have_threads():
    """3000 sequences, some without new or cached tokens: the append, then both attention kernels."""
    r = np.random.default_rng(941)
    new = r.integers(0, 3, 3000).tolist()
    lens = [x + int(r.integers(0, 60)) for x in new]
    b = make_batch(new, lens, 16, 942, behind=1)
    hq, hk, d = 2, 1, 64
    cache = make_cache(b["pages"], hk, 16, d, 943, b["free"])
    (q, qf), (k, kf), (v, vf) = (rows((b["rows"], h, d), 944 + i) for i, h in enumerate((hq, hk, hk)))
    ref = [np.array(x) for x in cache]
    want = kv_ref.append(ref, b["table"], b["lens"], b["q_start"], kf, vf, qf)
    dc = to_dev(cache)
    qr = tw.bitnet_kv_append(dc, *meta(b), k, v, q=q)
    few = tw.bitnet_attention(dc, *meta(b), qr, 2)
    many = tw.bitnet_attention(dc, *meta(b), qr, 60)
    torch.cuda.synchronize()
    end = int(b["q_start"][-1])
    assert all(same_bits(x.cpu().numpy(), y) for x, y in zip(dc, ref))
    exact, bound = kv_ref_batch(ref, b, want)
    for o in (few, many):
        assert (np.abs(o.float().cpu().numpy() - exact) <= bound)[:end].all()


def kv_ref_batch(cache, b, q):
    exact = kv_ref.attention(cache, b["table"], b["lens"], b["q_start"], q)
    return exact, kv_ref.attention_bound(cache, b["table"], b["lens"], b["q_start"], q, exact)
