"""What the cache's kernels access for batches that contradict themselves, restated on the CPU: every row, table entry,
page and workspace entry lies inside its buffer, whatever the page table, the lengths and the row starts hold.  The
restatement follows seq_info, attn_seq, page_of, ka_base, the unit list of the kernel for few tokens and the plan of the
one for prompts, line by line."""
import random

import pytest

GROUP, BLOCK = 16, 128  # tokens of a unit (few tokens), of a block (prompts)


def make(rng, sound):
    page = rng.choice([16, 32, 64, 128])
    n_seqs, width, pages = rng.randint(1, 12), rng.randint(1, 6), rng.randint(1, 40)
    if sound:
        new = [rng.choice([0, 1, 2, rng.randint(0, width * page)]) for _ in range(n_seqs)]
        lens = [rng.randint(n, width * page) for n in new]
        starts = [rng.randint(0, 3)]
        for n in new:
            starts.append(starts[-1] + n)
        rows = max(1, starts[-1] + rng.randint(0, 3))
        table = [[rng.randrange(pages) for _ in range(width)] for _ in range(n_seqs)]
    else:
        rows = rng.randint(1, 400)
        wild = lambda lo, hi: rng.choice([rng.randint(lo, hi), lo - 1, hi + 1, -2 ** 31, 2 ** 31 - 1, 0])
        starts = [wild(0, rows) for _ in range(n_seqs + 1)]
        if rng.random() < 0.4:
            starts = [0, rows] * n_seqs
            starts = starts[:n_seqs + 1]
        lens = [wild(0, width * page) for _ in range(n_seqs)]
        table = [[wild(0, pages - 1) for _ in range(width)] for _ in range(n_seqs)]
    return dict(page=page, shift=page.bit_length() - 1, n_seqs=n_seqs, width=width, pages=pages, rows=rows, starts=starts,
                lens=lens, table=table, group=rng.choice([1, 2, 3, 4, 8, 16, 128]), hk=rng.randint(1, 3))


def page_of(c, b, j):
    assert 0 <= b < c["n_seqs"] and 0 <= j < c["width"]
    p = c["table"][b][j]
    return p if 0 <= p < c["pages"] else -1


def attn_seq(c, b, max_new):
    q0, q1, length = c["starts"][b], c["starts"][b + 1], c["lens"][b]
    if q0 < 0 or q1 < q0 or q1 > c["rows"] or length < 0 or length > c["width"] * c["page"] or q1 - q0 > max_new:
        return q0, 0, 0
    return q0, q1 - q0, length


def tokens_accesses(c, max_new):
    """Few tokens: units (sequence, kv head, row tile, 16 tokens)."""
    for b in range(c["n_seqs"]):
        q0, n, length = attn_seq(c, b, max_new)
        for r in range(n):
            assert 0 <= q0 + r < c["rows"]  # queries read, results written
        for u in range(-(-length // GROUP) if n > 0 else 0):
            key0 = u * GROUP
            p = page_of(c, b, key0 >> c["shift"])
            slot = key0 & (c["page"] - 1)
            if p >= 0:
                assert p < c["pages"] and slot + GROUP <= c["page"]


def prompt_accesses(c, max_new):
    """Prompts: the plan's tiles against the workspace, the blocks' pages, the rows."""
    t = 2 * (128 // c["group"])
    seqs = [attn_seq(c, b, max_new) for b in range(c["n_seqs"])]
    if sum(n for _, n, _ in seqs) > c["rows"]:
        return False
    tiles = 0
    for b, (q0, n, length) in enumerate(seqs):
        for qt in range(-(-n // t)):
            last = min(n, (qt + 1) * t) - 1
            assert 0 <= q0 + qt * t and q0 + last < c["rows"]
            limit = length - n + last
            blocks = 0 if limit < 0 else limit // BLOCK + 1
            assert blocks == 0 or (blocks - 1) * BLOCK < length
            tiles += blocks > 0
            for j in range(blocks):
                for key0 in range(j * BLOCK, (j + 1) * BLOCK, GROUP):
                    if key0 < length:
                        page_of(c, b, key0 >> c["shift"])
    assert tiles * c["hk"] <= (c["rows"] // t + c["n_seqs"]) * c["hk"]  # attn_plan's room
    return True


def ka_base(q0, b, shift):
    return min(q0, (q0 >> shift) + 2 * b)


def append_accesses(c):
    """The items of the append; yields (sequence, position) of every token that is written."""
    shift, page = c["shift"], c["page"]
    for item in range(ka_base(c["rows"], c["n_seqs"], shift)):
        owners = []
        for b in range(c["n_seqs"]):
            lo, hi = c["starts"][b], c["starts"][b + 1]
            if lo < 0 or hi < lo or hi > c["rows"]:
                continue
            if ka_base(lo, b, shift) <= item < ka_base(hi, b + 1, shift):
                owners.append(b)
        for b in owners:  # any of them may be taken
            q0, n, length = c["starts"][b], c["starts"][b + 1] - c["starts"][b], c["lens"][b]
            if length < 0 or length > c["width"] * page or n > length or n == 0:
                continue
            first = length - n
            j = (first >> shift) + item - ka_base(q0, b, shift)
            if j > (length - 1) >> shift:
                continue
            assert j >= 0
            lo, hi = max(first, j << shift), min(length, (j + 1) << shift)
            assert lo < hi and 0 <= q0 + lo - first and q0 + hi - first <= c["rows"]
            assert 0 <= lo - (j << shift) and hi - (j << shift) <= page
            page_of(c, b, j)
            for pos in range(lo, hi):
                yield b, pos


@pytest.mark.parametrize("seed", range(0, 300, 30))
def test_contradictory_batches_stay_inside_their_buffers(seed):
    for i in range(30):
        c = make(random.Random(seed + i), sound=False)
        for max_new in (1, 40, c["rows"]):
            tokens_accesses(c, min(max_new, c["rows"]))
            prompt_accesses(c, min(max_new, c["rows"]))
        for _ in append_accesses(c):
            pass


@pytest.mark.parametrize("seed", range(1000, 1300, 30))
def test_sound_batches_are_done_once_and_whole(seed):
    for i in range(30):
        c = make(random.Random(seed + i), sound=True)
        tokens_accesses(c, c["rows"])
        assert prompt_accesses(c, c["rows"])
        want = [(b, p) for b in range(c["n_seqs"])
                for p in range(c["lens"][b] - (c["starts"][b + 1] - c["starts"][b]), c["lens"][b])]
        assert sorted(append_accesses(c)) == want


def test_claims_that_32_bits_cannot_count():
    """Row starts 0, T, 0, T, ... over all sequences that a call takes: with 128 query heads per kv head and T = 2^18 the
    tiles are exactly 2^32, which a 32-bit count takes for none; their rows, in 64 bits, exceed T."""
    rows, seqs, group = 1 << 18, 65536, 128
    per = rows // (2 * (128 // group))
    claimants = seqs // 2
    assert (per * claimants) % (1 << 32) == 0
    # as the plan adds them up: a thread's sequences in 64 bits, at most 2^25 a thread, 32 threads in 32 bits
    thread = [0] * 1024
    for b in range(0, seqs, 2):
        thread[b % 1024] += rows
    capped = [min(x, 1 << 25) for x in thread]
    warps = [sum(capped[w * 32:w * 32 + 32]) for w in range(32)]
    assert max(warps) < 1 << 31 and sum(warps) > rows
