"""Attention over contexts whose later tokens move the running maxima, sums and units of a row again and again."""
import numpy as np
import pytest
import torch

import kv_exact
import ternary_weight_fwd_b200 as tw
from kv_util import DEV, dev, make_batch, make_cache, rows, same_bits, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    tw.bitnet_device_status()
    tw.bitnet_batch_status()
    yield
    assert tw.bitnet_device_status() == 0
    assert tw.bitnet_batch_status() == 0


def check(b, cache, hq, seed, max_new=None, scale=None, qscale=1.5, repeat=1):
    d = cache[0].shape[3]
    q, qf = rows((b["rows"], hq, d), seed, scale=qscale)
    ref, bound = kv_exact.attention(cache, b, qf, scale)
    args = (to_dev(cache), dev(b["table"]), dev(b["lens"]), dev(b["q_start"]), q,
            max_new or max(1, int(np.diff(b["q_start"]).max())))
    first = None
    for _ in range(repeat):
        out = tw.bitnet_attention(*args, scale=scale)
        torch.cuda.synchronize()
        o = out.float().cpu().numpy()
        bad = ~(np.abs(o - ref) <= bound)
        assert not bad.any(), (np.argwhere(bad)[:5], o[bad][:5], ref[bad][:5], bound[bad][:5])
        assert first is None or same_bits(o, first)
        first = o
    return first


def along(b, cache, which, f):
    """Steps `which` (2: keys, 3: values) of the page j of every sequence become f(j)."""
    for s, length in enumerate(b["lens"].tolist()):
        for j in range(-(-length // cache[0].shape[2])):
            cache[which][b["table"][s, j]] = f(j)


def grow(b, cache, kind, every):
    """Pages in runs of `every`.  keys: key steps that grow by 0.05 a run; the largest of 16 or more scores lies about
    60 * 1.44 * 2 * step in powers of two above 0, so a row's maximum rises by more than 2^8 in most runs.  values:
    value steps that alternate by 2^7, so the sums change their unit with every run."""
    if kind == "keys":
        along(b, cache, 2, lambda j: 0.05 * (1 + j // every))
    else:
        along(b, cache, 3, lambda j: 0.02 * (1.0 if j // every % 2 else 2.0 ** -7))


WHOLE = ([512, 500, 512, 490, 512, 333], [2048, 1500, 512, 1999, 1024, 2040])
SHARED = ([150, 77], [4000, 1333])


@pytest.mark.parametrize("kind", ["keys", "values"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [WHOLE, SHARED], ids=["whole", "shared"])
def test_prompt_sums_that_are_rescaled_in_every_block(lengths, d, kind):
    """A row's two softmax threads rescale a half of its sums each, and the products of either half of a block's
    tokens add to all of them: neither may begin before both are done."""
    hq, hk, page = 20, 5, 64
    b = make_batch(*lengths, page, 801)
    assert kv_exact.whole_tiles(b, hq // hk, hk) == (lengths is WHOLE)
    cache = make_cache(b["pages"], hk, page, d, 802, b["free"])
    grow(b, cache, kind, 128 // page)
    check(b, cache, hq, 803, repeat=5)


TINY = [1e-20, 1e-30, 1e-34, 1e-35, 1e-37]


@pytest.mark.parametrize("tiny", TINY)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 4])
def test_tokens_values_of_tiny_steps_behind_ordinary_ones(n, d, tiny):
    """Ordinary pages, many groups of 16 tokens on pages of tiny values, ordinary ones again: what the sums hold stays
    finite while their unit follows the pages' steps."""
    b = make_batch([n] * 3, [300, 64, 2000], 32, 811)
    cache = make_cache(b["pages"], 2, 32, d, 812, b["free"])
    along(b, cache, 3, lambda j: tiny if 0 < j % 7 < 6 else 1.0)
    check(b, cache, 8, 813, max_new=n)


@pytest.mark.parametrize("tiny", TINY)
@pytest.mark.parametrize("n", [1, 4])
def test_tokens_tiny_steps_within_a_warps_share(n, tiny):
    """As above with so many tokens that a warp adds up groups of ordinary and of tiny pages itself (148 CTAs of 12
    warps, 16384 groups of one row tile, or 32768 of two)."""
    b = make_batch([n] * 64, [2048] * 64, 32, 816)
    cache = make_cache(b["pages"], 2, 32, 128, 817, b["free"])
    along(b, cache, 3, lambda j: tiny if 0 < j % 5 < 4 else 1.0)
    check(b, cache, 8, 818, max_new=n)


@pytest.mark.parametrize("tiny", TINY)
@pytest.mark.parametrize("n", [1, 4])
def test_tokens_all_weight_on_tiny_values(n, tiny):
    """The first page's scores are 0, those behind have maxima of hundreds: what the ordinary page left vanishes and
    the results are as small as the tiny values, with the same relative precision.  The step of the first page is
    smaller than e^127 times the tiny one, so its part of the result is below the bound's."""
    b = make_batch([n] * 2, [400, 90], 16, 821)
    cache = make_cache(b["pages"], 1, 16, 128, 822, b["free"])
    along(b, cache, 2, lambda j: 0.0 if j == 0 else 5.0)
    along(b, cache, 3, lambda j: 1.0 if j == 0 else tiny)
    check(b, cache, 4, 823, max_new=n)


@pytest.mark.parametrize("n", [1, 4])
def test_tokens_sums_that_are_rescaled_in_every_group(n):
    for kind in ("keys", "values"):
        b = make_batch([n] * 4, [1000, 300, 3000, 17], 16, 831)
        cache = make_cache(b["pages"], 2, 16, 128, 832, b["free"])
        grow(b, cache, kind, 1)
        check(b, cache, 8, 833, max_new=n, repeat=3)


@pytest.mark.parametrize("tiny", TINY)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [WHOLE, SHARED], ids=["whole", "shared"])
def test_prompt_values_of_tiny_steps_behind_ordinary_ones(lengths, d, tiny):
    """As for few tokens, by blocks of 128 tokens."""
    hq, hk, page = 20, 5, 128
    b = make_batch(*lengths, page, 841)
    assert kv_exact.whole_tiles(b, hq // hk, hk) == (lengths is WHOLE)
    cache = make_cache(b["pages"], hk, page, d, 842, b["free"])
    along(b, cache, 3, lambda j: tiny if 0 < j % 7 < 6 else 1.0)
    check(b, cache, hq, 843)


@pytest.mark.parametrize("tiny", [1e-20, 1e-25])
def test_prompt_all_weight_on_tiny_values(tiny):
    b = make_batch([150, 60], [900, 290], 128, 851)
    cache = make_cache(b["pages"], 1, 128, 128, 852, b["free"])
    along(b, cache, 2, lambda j: 0.0 if j == 0 else 5.0)
    along(b, cache, 3, lambda j: 1.0 if j == 0 else tiny)
    check(b, cache, 4, 853)


@pytest.mark.parametrize("n,length", [(1, 400), (100, 400)])
def test_pages_of_key_step_zero_have_scores_of_zero(n, length):
    """However large the queries: with a scale that brings the other pages' scores to the order of 1."""
    b = make_batch([n], [length], 16, 861)
    cache = make_cache(b["pages"], 1, 16, 128, 862, b["free"])
    along(b, cache, 2, lambda j: 0.0 if j % 3 else 0.02)
    check(b, cache, 2, 863, qscale=1e33, scale=1e-34)
