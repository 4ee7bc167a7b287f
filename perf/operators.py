"""The paged 8-bit key/value cache and the attention that reads it: what is measured of them.

Three operators around the BitLinear projections of a decoder layer:

* ``bitnet_kv_append`` rotates the new queries and keys by their positions, quantises the new keys and
  values to int8 with one step per (page, kv head) and writes them into the pages of their sequences;
* ``bitnet_attention`` over few new tokens per sequence (decoding, drafts to be verified);
* ``bitnet_attention`` over prompts (whole ones and chunks).

Cache: codes int8 ``[pages][kv heads][page size][head dim]``, steps fp32 ``[pages][kv heads]``, a key or
value is ``code * step``.  A batch is ``page_table [seqs][width]``, ``seq_lens [seqs]`` (tokens in the
cache, the new ones included) and ``q_start [seqs + 1]`` (the new tokens of sequence b are rows
``q_start[b] .. q_start[b + 1]`` of q, k, v).

Heads and widths are those of BitNetConfig (20 query and 5 kv heads of 128, context 4096) beside generic ones.
"""
import torch

own = False

DEV = "cuda"
THETA = 500000.0


# ---- cases --------------------------------------------------------------------------------------------
def listed():
    return [
        # one user decoding: one token into the cache of one sequence, the smallest call there is
        dict(name="append_token_1", op="append", seqs=1, new=1, ctx=260, ragged=False, heads=20, kv_heads=5, dim=128,
             page=64, dtype="bf16", behind=0),
        # a decode step of a full batch; the projections hand over fp32
        dict(name="append_tokens_64", op="append", seqs=64, new=1, ctx=4096, ragged=True, heads=20, kv_heads=5,
             dim=128, page=64, dtype="f32", behind=0),
        # a prompt of the model's whole context
        dict(name="append_prompt_4096", op="append", seqs=1, new=4096, ctx=4096, ragged=False, heads=20, kv_heads=5,
             dim=128, page=64, dtype="bf16", behind=0),
        # many prompts and chunks of odd lengths on short pages, a few rows of padding behind them
        dict(name="append_ragged_32", op="append", seqs=32, new=1000, ctx=2000, ragged=True, heads=16, kv_heads=16,
             dim=64, page=16, dtype="f32", behind=5),
        # one user early in an answer: latency
        dict(name="token_1_short", op="tokens", seqs=1, new=1, ctx=257, ragged=False, heads=20, kv_heads=5, dim=128,
             page=64, behind=0),
        # a full decode batch with contexts of every length up to the model's
        dict(name="tokens_64", op="tokens", seqs=64, new=1, ctx=4096, ragged=True, heads=20, kv_heads=5, dim=128,
             page=64, behind=0),
        # one user far into a long document: one long axis, few rows
        dict(name="token_1_long", op="tokens", seqs=1, new=1, ctx=131071, ragged=False, heads=20, kv_heads=5, dim=128,
             page=128, behind=0),
        # drafts of four tokens verified at once, a larger group of query heads, short pages
        dict(name="drafts_16x4", op="tokens", seqs=16, new=4, ctx=8000, ragged=True, heads=32, kv_heads=4, dim=128,
             page=16, behind=0),
        # a prompt of the model's whole context
        dict(name="prompt_4096", op="prompt", seqs=1, new=4096, ctx=4096, ragged=False, heads=20, kv_heads=5, dim=128,
             page=64, behind=0),
        # a chunk of a long prompt: few rows of tiles, a long context
        dict(name="chunk_512_of_16384", op="prompt", seqs=1, new=512, ctx=16384, ragged=False, heads=20, kv_heads=5,
             dim=128, page=64, behind=0),
        # prompts of odd lengths batched together, padded behind
        dict(name="prompts_ragged_8", op="prompt", seqs=8, new=2001, ctx=2001, ragged=True, heads=20, kv_heads=5,
             dim=128, page=32, behind=3),
        # narrow heads that share nothing, chunks behind a cached prefix
        dict(name="prompts_narrow_4", op="prompt", seqs=4, new=1001, ctx=1500, ragged=True, heads=16, kv_heads=16,
             dim=64, page=128, behind=0),
    ]


def _log(rng, lo, hi):
    return min(hi, int(lo * (hi / lo) ** rng.random()))


def draw(rng):
    heads, kv_heads = rng.choice([(20, 5), (16, 16), (32, 4), (8, 8), (12, 4), (8, 1), (28, 4), (6, 2), (32, 2)])
    c = dict(op=rng.choice(["append", "tokens", "prompt"]), heads=heads, kv_heads=kv_heads, dim=rng.choice([64, 128]),
             page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.7, behind=rng.choice([0, 0, 1, 7]))
    if c["op"] == "append":
        c["dtype"] = rng.choice(["bf16", "f32"])
        if rng.random() < 0.5:
            c.update(seqs=_log(rng, 1, 64), new=_log(rng, 1, 8), ctx=_log(rng, 16, 4096))
        else:
            c.update(seqs=_log(rng, 1, 16), new=_log(rng, 9, 1000))
            c["ctx"] = c["new"] + rng.choice([0, _log(rng, 1, 1000)])
    elif c["op"] == "tokens":
        c.update(seqs=_log(rng, 1, 64), new=_log(rng, 1, 4))
        c["ctx"] = _log(rng, 16, min(65536, 98304 // c["seqs"]))
        if kv_heads == 16:
            c["ctx"] = max(16, c["ctx"] // 4)
    else:
        c["seqs"] = _log(rng, 1, 6)
        c["new"] = _log(rng, 33, 4096 // c["seqs"])
        c["ctx"] = c["new"] + rng.choice([0, _log(rng, 1, 3 * c["new"])])
        while work(c)["flops"] > 8e10:
            c.update(new=c["new"] * 3 // 4, ctx=c["ctx"] * 3 // 4)
    return c


def _lengths(case, seed):
    """New tokens and cached tokens (the new ones included) of every sequence, on the host."""
    g = torch.Generator().manual_seed(seed * 7919 + 17)
    b, new, ctx = case["seqs"], case["new"], max(case["ctx"], case["new"])
    if not case["ragged"]:
        return [new] * b, [ctx] * b
    if case["op"] == "prompt" or new > 8:
        # the same total for every seed: shares between a sixteenth and the whole of the longest, in a drawn order
        share = [1 + 15 * i / max(1, b - 1) for i in range(b)] if b > 1 else [16.0]
        n = [max(1, round(new * s / 16)) for s in share]
        pre = [round((ctx - new) * (i % 5) / 4) for i in range(b)]
    else:
        n = [new] * b
        share = [1 + 31 * i / max(1, b - 1) for i in range(b)] if b > 1 else [32.0]
        pre = [max(0, round(ctx * s / 32) - new) for s in share]
    order = torch.randperm(b, generator=g).tolist()
    return [n[i] for i in order], [n[i] + pre[i] for i in order]


# ---- inputs -------------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n, lens = _lengths(case, seed)
    b, hq, hk, d, page = case["seqs"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    # pages in a drawn order, a few of them belonging to nobody; their steps are not numbers
    used = [-(-x // page) for x in lens]
    total = sum(used) + 3
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed + 1)).to(torch.int32)
    table = torch.full((b, max(used) + 1), -1, dtype=torch.int32)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = perm[at:at + u]
        at += u
    step_k = 0.02 * torch.exp(0.3 * torch.randn(total, hk, generator=g, device=DEV))
    step_v = 0.02 * torch.exp(0.3 * torch.randn(total, hk, generator=g, device=DEV))
    free = perm[at:].long().to(DEV)
    step_k[free] = float("nan")
    step_v[free] = float("nan")

    def codes():
        out = torch.empty((total, hk, page, d), dtype=torch.int8, device=DEV)
        for i in range(0, total, 512):
            part = out[i:i + 512]
            part.copy_(torch.randn(part.shape, generator=g, device=DEV).mul_(40).round_().clamp_(-127, 127))
        return out

    t, rows = sum(n), sum(n) + case["behind"]
    state = dict(op=case["op"], dim=d, rows=t, max_new=max(n), table=table.to(DEV),
                 lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 q_start=torch.tensor([0] + n, dtype=torch.int32).cumsum(0).to(torch.int32).to(DEV))
    if case["op"] == "append":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # one fused projection's output; q, k and v are views of it
        qkv = torch.randn((rows, (hq + 2 * hk) * d), generator=g, device=DEV)
        qkv[:, ::37] *= 6  # a few strong channels
        qkv = qkv.to(dt)
        state["q"] = qkv[:, :hq * d].view(rows, hq, d)
        state["k"] = qkv[:, hq * d:(hq + hk) * d].view(rows, hk, d)
        state["v"] = qkv[:, (hq + hk) * d:].view(rows, hk, d)
        inv = THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device=DEV) / d)
        ang = torch.arange(max(lens), dtype=torch.float64, device=DEV)[:, None] * inv
        state["rope"] = torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32)
        state["cache"] = (codes(), codes(), step_k * 2, step_v * 2)
        state["out"] = torch.full((rows, hq, d), 0.01, dtype=torch.bfloat16, device=DEV)
    else:
        state["cache"] = (codes(), codes(), step_k, step_v)
        state["q"] = (1.5 * torch.randn((rows, hq, d), generator=g, device=DEV)).to(torch.bfloat16)
        state["out"] = torch.full((rows, hq, d), 0.01, dtype=torch.bfloat16, device=DEV)
    return state


# ---- plain forms ----------------------------------------------------------------------------------------
def _owners(state):
    """Sequence and index within its new tokens of every row that belongs to a sequence."""
    row = torch.arange(state["rows"], device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(state["q_start"], row, right=True) - 1
    return seq, row - state["q_start"][seq]


def _rotate(x, cos, sin):
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_store(x, codes, step, page_of, slot, old_page, old_slots):
    """Codes and steps after rows x [T][kv heads][D] went to (page_of, slot)."""
    size = codes.shape[2]
    amax = x.abs().amax(-1)
    peak = torch.zeros_like(step)
    peak.scatter_reduce_(0, page_of[:, None].expand_as(amax), amax, "amax")
    touched = torch.zeros(step.shape[0], dtype=torch.bool, device=DEV)
    touched[page_of] = True
    keeps = torch.zeros_like(touched)
    keeps[old_page] = True
    old = torch.where(keeps[:, None], step, torch.zeros_like(step))
    grown = torch.maximum(old, peak / 127)
    # what the pages held before, in the new steps
    ratio = torch.where(grown[old_page] > old[old_page], old[old_page] / grown[old_page], torch.ones_like(old[old_page]))
    held = codes[old_page]
    again = torch.round(held.float() * ratio[..., None, None]).to(torch.int8)
    below = torch.arange(size, device=DEV)[None, :] < old_slots[:, None]
    codes[old_page] = torch.where(below[:, None, :, None], again, held)
    s = grown[page_of][..., None]
    q = torch.where(s > 0, torch.round(x / s), torch.zeros_like(x)).clamp(-127, 127).to(torch.int8)
    codes[page_of, :, slot] = q
    step.copy_(torch.where(touched[:, None], grown, step))


def _plain_append(state):
    k, v, step_k, step_v = state["cache"]
    size, t = k.shape[2], state["rows"]
    seq, i = _owners(state)
    n = state["q_start"][1:] - state["q_start"][:-1]
    first = state["lens"] - n
    pos = (first[seq] + i).long()
    page_of = state["table"][seq, pos // size].long()
    slot = pos % size
    # the only page of a sequence that can hold older tokens is the one its first new token goes to
    has = (n > 0) & (first % size > 0)
    old_page = state["table"][has, (first[has] // size).long()].long()
    old_slots = (first % size)[has]
    h = state["dim"] // 2
    cos, sin = state["rope"][pos, None, :h], state["rope"][pos, None, h:]
    state["out"][:t] = _rotate(state["q"][:t].float(), cos, sin).to(torch.bfloat16)
    _plain_store(_rotate(state["k"][:t].float(), cos, sin), k, step_k, page_of, slot, old_page, old_slots)
    _plain_store(state["v"][:t].float(), v, step_v, page_of, slot, old_page, old_slots)
    return {"q": state["out"], "k": k, "v": v, "k_step": step_k, "v_step": step_v}


def _values(codes, step, pages):
    b, w = pages.shape
    x = codes[pages].float() * step[pages][..., None, None]
    return x.transpose(1, 2).reshape(b, codes.shape[1], w * codes.shape[2], codes.shape[3])


def _plain_attention(state):
    k, v, step_k, step_v = state["cache"]
    q, t, n = state["q"], state["rows"], state["max_new"]
    b, hq, hk, d = state["table"].shape[0], q.shape[1], k.shape[1], state["dim"]
    table = state["table"]
    pages = torch.where(table < 0, table[:, :1], table).long()  # behind a sequence's last page: any of its own
    i = torch.arange(n, device=DEV)
    rows = (state["q_start"][:-1, None] + i).clamp(max=q.shape[0] - 1).long()
    qf = q[rows].float().view(b, n, hk, hq // hk, d).transpose(1, 2).reshape(b, hk, n * (hq // hk), d)
    s = torch.matmul(qf, _values(k, step_k, pages).transpose(-1, -2)) * d ** -0.5
    new = state["q_start"][1:] - state["q_start"][:-1]
    last = (state["lens"] - new)[:, None] + i  # the last position that new token i sees: its own
    seen = torch.arange(s.shape[-1], device=DEV) <= last[..., None]
    seen = (seen & (i < new[:, None])[..., None]).repeat_interleave(hq // hk, 1)[:, None]
    s = s.masked_fill_(~seen, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(torch.isfinite(m), m, torch.zeros_like(m))).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _values(v, step_v, pages)) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(b, hk, n, hq // hk, d).transpose(1, 2).reshape(b, n, hq, d)
    seq, at = _owners(state)
    state["out"][:t] = o[seq, at.long()].to(torch.bfloat16)
    return state["out"]


def run(state):
    if own:
        import ternary_weight_fwd_b200 as tw

        if state["op"] == "append":
            out = tw.bitnet_kv_append(state["cache"], state["table"], state["lens"], state["q_start"], state["k"],
                                      state["v"], q=state["q"], rope=state["rope"], q_out=state["out"])
            k, v, step_k, step_v = state["cache"]
            return {"q": out, "k": k, "v": v, "k_step": step_k, "v_step": step_v}
        return tw.bitnet_attention(state["cache"], state["table"], state["lens"], state["q_start"], state["q"],
                                   state["max_new"], out=state["out"])
    return _plain_append(state) if state["op"] == "append" else _plain_attention(state)


# ---- what a pass cannot do without -------------------------------------------------------------------------
def work(case):
    n, lens = _lengths(case, 0)
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    t = sum(n)
    pages = sum(-(-x // page) for x in lens)
    if case["op"] == "append":
        e = 2 if case["dtype"] == "bf16" else 4
        touched = sum((x - 1) // page - (x - m) // page + 1 for x, m in zip(lens, n))
        moved = t * (hq + 2 * hk) * d * e + t * hq * d * 2 + t * 2 * hk * d + t * d * 4 + 2 * touched * hk * 4
        return {"bytes": moved, "flops": t * ((hq + hk) * d * 3 + 2 * hk * d * 2)}
    seen = sum(m * (x - m) + m * (m + 1) // 2 for x, m in zip(lens, n))
    moved = 2 * t * hq * d * 2 + sum(lens) * 2 * hk * d + 2 * pages * hk * 4 + pages * 4
    return {"bytes": moved, "flops": 4 * seen * hq * d}


# ---- the definition in 64 bits ---------------------------------------------------------------------------
def exact(case, seed):
    """Sequence by sequence, token by token where the cache's steps need it, in 64 bits."""
    s = prepare(case, seed)
    n, lens = _lengths(case, seed)
    k, v, step_k, step_v = s["cache"]
    page, d = case["page"], case["dim"]
    table = s["table"].tolist()
    if case["op"] == "append":
        inv = THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device=DEV) / d)
        out = s["out"].double()
        sk, sv = step_k.double(), step_v.double()
        at = 0
        for i in range(len(n)):
            pos = torch.arange(lens[i] - n[i], lens[i], dtype=torch.float64, device=DEV)
            turn = torch.polar(torch.ones((n[i], 1, d // 2), dtype=torch.float64, device=DEV), pos[:, None, None] * inv)

            def turned(x):
                z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * turn
                return torch.cat([z.real, z.imag], -1)

            mine = slice(at, at + n[i])
            out[mine] = turned(s["q"][mine].double())
            kd, vd = turned(s["k"][mine].double()), s["v"][mine].double()
            start = lens[i] - n[i]
            for j in range(start // page, (lens[i] - 1) // page + 1):
                lo, hi = max(start, j * page) - start, min(lens[i], (j + 1) * page) - start
                for steps, x in ((sk, kd), (sv, vd)):
                    new = x[lo:hi].abs().amax((0, 2)) / 127
                    p = table[i][j]
                    steps[p] = torch.maximum(steps[p], new) if start > j * page else new
            at += n[i]
        return {"q": out, "k": None, "v": None, "k_step": sk, "v_step": sv}
    if work(case)["flops"] > 4e11:
        return None
    hq, hk = case["heads"], case["kv_heads"]
    out, at = s["out"].double(), 0
    for i in range(len(n)):
        p = torch.tensor(table[i][:-(-lens[i] // page)], device=DEV)
        for h in range(hk):
            kd = (k[p, h].double() * step_k[p, h].double()[:, None, None]).reshape(-1, d)[:lens[i]]
            vd = (v[p, h].double() * step_v[p, h].double()[:, None, None]).reshape(-1, d)[:lens[i]]
            last = torch.arange(lens[i] - n[i], lens[i], device=DEV)
            hidden = torch.arange(lens[i], device=DEV)[None] > last[:, None]
            for g in range(h * (hq // hk), (h + 1) * (hq // hk)):
                logits = (s["q"][at:at + n[i], g].double() @ kd.T) / d ** 0.5
                out[at:at + n[i], g] = torch.softmax(logits.masked_fill_(hidden, float("-inf")), -1) @ vd
        at += n[i]
    return out
