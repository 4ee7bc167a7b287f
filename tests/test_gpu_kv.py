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
                                     (6, 6, 16), (3, 3, 32), (12, 1, 4), (2, 2, 47)])
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


# ---- calls as they are used: together, captured, on streams, refused on the device -----------------------
def layer_inputs(seed, hq=4, hk=2, d=64, width=256):
    from gpu_util import make_weights
    return {n: make_weights(o, i, seed + k) for k, (n, o, i) in
            enumerate((("q", hq * d, width), ("k", hk * d, width), ("v", hk * d, width), ("o", width, hq * d)))}


def test_decoder_attention_run():
    """A prompt and three decode steps of one layer's attention as a user chains it: BitLinear q, k, v,
    append, attention, output BitLinear.  Every stage is checked on what the stage before really gave."""
    import oracle
    from gpu_util import assert_rel_close, make_x
    hq, hk, d, page, width = 4, 2, 64, 16, 256
    W = layer_inputs(500, hq, hk, d, width)
    rope = tw.bitnet_rope_table(256, d)
    tab = rope.cpu().numpy()
    cache = tw.kv_cache(12, hk, d, page)
    ref = [x.cpu().numpy() for x in cache]
    table = np.array([[7, 2, 9, 0], [4, 11, 1, 5]], np.int32)
    lens = np.zeros(2, np.int32)
    for step, new in enumerate([(37, 20), (1, 1), (1, 3), (2, 0)]):
        t = sum(new)
        lens = lens + np.array(new, np.int32)
        starts = np.array([0, new[0], t], np.int32)
        x, xf = make_x(t, width, 510 + step)
        q, k, v = (tw.bitnet_linear_ex(x, W[n]["p"], W[n]["g"], y_dtype=torch.bfloat16).view(t, -1, d)
                   for n in ("q", "k", "v"))
        qr = tw.bitnet_kv_append(cache, dev(table), dev(lens), dev(starts), k, v, q=q, rope=rope)
        out = tw.bitnet_attention(cache, dev(table), dev(lens), dev(starts), qr, max(new))
        y = tw.bitnet_linear_norm(out.view(t, -1), torch.ones(hq * d, device=DEV), W["o"]["p"], W["o"]["g"])
        torch.cuda.synchronize()
        host = [z.float().cpu().numpy() for z in (q, k, v)]
        want = kv_ref.append(ref, table, lens, starts, host[1], host[2], host[0], tab)
        assert all(same_bits(a.cpu().numpy(), b) for a, b in zip(cache, ref))
        assert same_bits(qr.float().cpu().numpy(), want)
        o = out.float().cpu().numpy()
        exact = kv_ref.attention(ref, table, lens, starts, want)
        assert (np.abs(o - exact) <= kv_ref.attention_bound(ref, table, lens, starts, want, exact)).all()
        y_ref = oracle.bitlinear_norm(o.reshape(t, -1), np.ones(hq * d, np.float32), W["o"]["p_ref"], W["o"]["g_ref"],
                                      hq * d)[0]
        assert_rel_close(y.cpu().numpy(), y_ref)


def batch_on_device(b):
    return dev(b["table"]), dev(b["lens"]), dev(b["q_start"])


@pytest.mark.parametrize("new,max_new", [([1, 1, 1, 0], 1), ([70, 1, 33, 2], 70)])
def test_captured_and_replayed(new, max_new):
    """Append and attention captured once and replayed with other lengths, pages and values in the same
    buffers; a second graph shares the workspace, replayed in turn."""
    hq, hk, d, page = 8, 2, 128, 32
    lens = [130, 1, 40, 9]
    a = make_batch(new, lens, page, 601, width=8)
    b = make_batch(new[::-1], [n + 50 for n in new[::-1]], page, 602, width=8, spare=2)
    t = a["rows"]
    assert b["rows"] == t
    pages = max(a["pages"], b["pages"])
    caches = [make_cache(pages, hk, page, d, 603 + i) for i in range(2)]
    state = [torch.zeros_like(x) for x in to_dev(caches[0])]
    table, seq, starts = (torch.zeros_like(x) for x in batch_on_device(a))
    x = [rows((t, n, d), 610 + i) for i, n in enumerate((hq, hk, hk))]
    y = [rows((t, n, d), 620 + i) for i, n in enumerate((hq, hk, hk))]
    q, k, v = (z[0].clone() for z in x)
    rope_np = kv_ref.rope_table(256, d)
    rope = dev(rope_np)
    need = tw.bitnet_attention_workspace_size(4, t, hq, hk, d, max_new)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV)
    outs = [torch.zeros((t, hq, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    qr = torch.zeros((t, hq, d), dtype=torch.bfloat16, device=DEV)
    graphs = []
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tw.bitnet_kv_append(state, table, seq, starts, k, v, q=q, rope=rope, q_out=qr)
            tw.bitnet_attention(state, table, seq, starts, qr, max_new, out=out, workspace=ws)
        graphs.append(g)
    for turn, (bt, cache, z) in enumerate(((a, caches[0], x), (b, caches[1], y), (a, caches[1], y))):
        for dst, src in zip((table, seq, starts), batch_on_device(bt)):
            dst.copy_(src)
        for dst, src in zip(state, to_dev(cache)):
            dst.copy_(src)
        for dst, src in zip((q, k, v), z):
            dst.copy_(src[0])
        graphs[turn % 2].replay()
        graphs[(turn + 1) % 2].replay()  # again with the same tokens: nothing changes
        torch.cuda.synchronize()
        ref = [np.array(c) for c in cache]
        want = kv_ref.append(ref, bt["table"], bt["lens"], bt["q_start"], z[1][1], z[2][1], z[0][1], rope_np)
        assert all(same_bits(s.cpu().numpy(), c) for s, c in zip(state, ref))
        exact = kv_ref.attention(ref, bt["table"], bt["lens"], bt["q_start"], want)
        bound = kv_ref.attention_bound(ref, bt["table"], bt["lens"], bt["q_start"], want, exact)
        o = [out.float().cpu().numpy() for out in outs]
        assert same_bits(o[0], o[1])
        assert (np.abs(o[0] - exact) <= bound).all()


@pytest.mark.parametrize("n", [1, 40])
def test_two_calls_at_once(n):
    """Two streams, two batches over one cache, each call with its own workspace (made by the call)."""
    hq, hk, d, page = 8, 2, 128, 32
    bs = [make_batch([n] * 6, [300 + 40 * i for i in range(6)], page, 631 + s) for s in range(2)]
    pages = max(b["pages"] for b in bs)
    cache = make_cache(pages, hk, page, d, 633)
    dc = to_dev(cache)
    qs = [rows((b["rows"], hq, d), 635 + i) for i, b in enumerate(bs)]
    meta = [batch_on_device(b) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i in range(2):
            outs[i].append(tw.bitnet_attention(dc, *meta[i], qs[i][0], n, stream=streams[i]))
    torch.cuda.synchronize()
    for i, b in enumerate(bs):
        exact = kv_ref.attention(cache, b["table"], b["lens"], b["q_start"], qs[i][1])
        bound = kv_ref.attention_bound(cache, b["table"], b["lens"], b["q_start"], qs[i][1], exact)
        for o in outs[i]:
            assert (np.abs(o.float().cpu().numpy() - exact) <= bound).all()


@pytest.mark.parametrize("n", [1, 40])
def test_output_over_the_queries(n):
    b = make_batch([n, n], [90, n], 32, 641)
    cache = make_cache(b["pages"], 2, 32, 128, 642, b["free"])
    q, _ = rows((b["rows"], 4, 128), 643)
    args = (to_dev(cache), *batch_on_device(b))
    want = tw.bitnet_attention(*args, q, n)
    got = tw.bitnet_attention(*args, q, n, out=q)
    torch.cuda.synchronize()
    assert got is q and torch.equal(q, want)


@pytest.mark.parametrize("n", [1, 40])
def test_padding_and_free_memory_have_no_effect(n):
    """Infinities and NaN in rows of no sequence, in steps of free pages, in table entries behind a
    sequence's last page; any bytes in slots behind its last token."""
    b = make_batch([n, n], [n + 3, 77], 16, 651, behind=4, width=9)
    cache = make_cache(b["pages"], 2, 16, 64, 652, b["free"])
    q, _ = rows((b["rows"], 4, 64), 653)
    out = [marked(q.shape), marked(q.shape)]
    tw.bitnet_attention(to_dev(cache), *batch_on_device(b), q, n, out=out[0])
    q[2 * n:] = float("nan")
    cache[2][b["free"]] = np.inf
    cache[3][b["free"]] = -np.inf
    for s in range(2):
        last = int(b["lens"][s]) - 1
        for c in cache[:2]:
            c[b["table"][s, last // 16], :, last % 16 + 1:] = -128
    b["table"][b["table"] < 0] = 2 ** 31 - 1
    tw.bitnet_attention(to_dev(cache), *batch_on_device(b), q, n, out=out[1])
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and (out[0][2 * n:] == MARK).all()


BAD = [("page", lambda b: b["table"].__setitem__(1, 10 ** 6)),
       ("negative page", lambda b: b["table"].__setitem__(1, -1)),
       ("length beyond the table", lambda b: b["lens"].__setitem__(1, 10 ** 6)),
       ("negative length", lambda b: b["lens"].__setitem__(1, -5)),
       ("rows beyond T", lambda b: b["q_start"].__setitem__(3, 10 ** 6)),
       ("decreasing rows", lambda b: b["q_start"].__setitem__(2, 0))]


@pytest.mark.parametrize("what,spoil", BAD, ids=[w for w, _ in BAD])
@pytest.mark.parametrize("n", [2, 40])
def test_bad_batches_are_refused_on_the_device(what, spoil, n):
    """Contradictory batches set the status word and touch nothing outside the sequences concerned (shown on
    the CPU: every access of the kernels lies behind the checks of seq_info / attn_seq / page_of)."""
    b = make_batch([n, n, n], [n + 20, n + 30, n + 9], 16, 661)
    cache = make_cache(b["pages"], 2, 16, 64, 662)
    q, _ = rows((b["rows"], 4, 64), 663)
    k, _ = rows((b["rows"], 2, 64), 664)
    good = to_dev(cache)
    first = tw.bitnet_attention(good, *batch_on_device(b), q, n)
    tw.bitnet_kv_append(good, *batch_on_device(b), k, k)
    assert tw.bitnet_batch_status() == 0
    spoil(b)
    args = batch_on_device(b)
    dc = to_dev(cache)
    got = tw.bitnet_attention(dc, *args, q, n)
    assert tw.bitnet_batch_status() == tw.BITNET_ERR_INVALID_ARG
    assert tw.bitnet_batch_status() == 0
    tw.bitnet_kv_append(dc, *args, k, k)
    assert tw.bitnet_batch_status() == tw.BITNET_ERR_INVALID_ARG
    if what == "decreasing rows":
        return  # the last sequence then claims the first one's rows too
    assert torch.equal(got[:n], first[:n])  # the sound first sequence
    page = int(b["table"][0, (n + 20 - 1) // 16])
    assert torch.equal(dc.k[page], good.k[page]) and torch.equal(dc.v_step[page], good.v_step[page])


def test_more_new_tokens_than_said_and_short_rotation_tables():
    b = make_batch([3, 1], [30, 20], 16, 671)
    cache = make_cache(b["pages"], 2, 16, 64, 672)
    q, qf = rows((4, 4, 64), 673)
    out = tw.bitnet_attention(to_dev(cache), *batch_on_device(b), q, 2)
    assert tw.bitnet_batch_status() == tw.BITNET_ERR_INVALID_ARG
    exact = kv_ref.attention(cache, b["table"], b["lens"], b["q_start"], qf)
    assert np.allclose(out[3].float().cpu().numpy(), exact[3], rtol=0.02, atol=0.02)
    k, _ = rows((4, 2, 64), 674)
    dc = to_dev(cache)
    tw.bitnet_kv_append(dc, *batch_on_device(b), k, k, rope=dev(kv_ref.rope_table(25, 64)))
    assert tw.bitnet_batch_status() == tw.BITNET_ERR_INVALID_ARG
    assert same_bits(dc.k[int(b["table"][0, 1])].cpu().numpy(), cache[0][int(b["table"][0, 1])])


def test_append_with_fewer_cached_than_new_tokens_is_refused():
    b = make_batch([5], [5], 16, 681)
    cache = make_cache(b["pages"], 1, 16, 64, 682)
    b["lens"][0] = 3
    k, _ = rows((5, 1, 64), 683)
    dc = to_dev(cache)
    tw.bitnet_kv_append(dc, *batch_on_device(b), k, k)
    assert tw.bitnet_batch_status() == tw.BITNET_ERR_INVALID_ARG
    assert all(same_bits(x.cpu().numpy(), y) for x, y in zip(dc, cache))


def test_a_bad_batch_leaves_later_calls_alone():
    """The batch status is a word of its own: the BitLinear calls' waits do not give up over it."""
    from gpu_util import make_weights, make_x
    b = make_batch([1], [20], 16, 691)
    cache = make_cache(b["pages"], 1, 16, 64, 692)
    b["table"][:] = 10 ** 6
    q, _ = rows((1, 1, 64), 693)
    tw.bitnet_attention(to_dev(cache), *batch_on_device(b), q, 1)
    W = make_weights(512, 256, 694)
    x, _ = make_x(300, 256, 695)
    y = tw.bitnet_linear(x, W["p"], W["g"])
    assert tw.bitnet_device_status() == 0
    assert tw.bitnet_batch_status() == tw.BITNET_ERR_INVALID_ARG
    assert torch.equal(y, tw.bitnet_linear(x, W["p"], W["g"]))


@pytest.mark.parametrize("n", [1, 40])
def test_rows_in_front_of_the_first_sequence(n):
    """q_start need not begin at 0: rows in front of it are padding like those behind."""
    b = make_batch([n, n], [n + 30, n], 16, 701)
    b["q_start"] = b["q_start"] + 5
    b["rows"] += 5
    cache = make_cache(b["pages"], 2, 16, 64, 702)
    (q, qf), (k, kf) = rows((b["rows"], 4, 64), 703), rows((b["rows"], 2, 64), 704)
    dc, ref = to_dev(cache), [np.array(c) for c in cache]
    rot = marked(q.shape)
    tw.bitnet_kv_append(dc, *batch_on_device(b), k, k, q=q, q_out=rot)
    want = kv_ref.append(ref, b["table"], b["lens"], b["q_start"], kf, kf, qf)
    out = marked(q.shape)
    tw.bitnet_attention(dc, *batch_on_device(b), q, n, out=out)
    torch.cuda.synchronize()
    assert all(same_bits(x.cpu().numpy(), y) for x, y in zip(dc, ref))
    assert (rot[:5] == MARK).all() and (out[:5] == MARK).all()
    assert same_bits(rot[5:].float().cpu().numpy(), want[5:])
    exact = kv_ref.attention(ref, b["table"], b["lens"], b["q_start"], qf)
    bound = kv_ref.attention_bound(ref, b["table"], b["lens"], b["q_start"], qf, exact)
    assert (np.abs(out.float().cpu().numpy() - exact)[5:] <= bound[5:]).all()


def test_memory_made_for_another_stream():
    """What a call makes for itself on a given stream is not memory that the current stream still works on."""
    b = make_batch([40, 40], [400, 40], 32, 711)
    cache = make_cache(b["pages"], 2, 32, 128, 712)
    q, _ = rows((80, 8, 128), 713)
    args = (to_dev(cache), *batch_on_device(b))
    want = tw.bitnet_attention(*args, q, 40)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(5):
        busy = torch.randn(4096, 4096, device=DEV)
        for _ in range(4):
            busy = busy @ busy * 1e-2  # frees memory that is still being read on the current stream
        del busy
        got = tw.bitnet_attention(*args, q, 40, stream=other)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
