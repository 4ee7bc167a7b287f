"""The forms of kv_ref.attention and kv_ref.attention_bound for long contexts: the same 64-bit arithmetic, a kv head
of a sequence at a time, by torch on the GPU."""
import numpy as np
import torch

DEV = "cuda"


def attention(cache, b, q, scale=None):
    """(result, largest error that the documented roundings allow) of every row of a sequence, NaN elsewhere.
    cache: four numpy arrays; b: a batch of kv_util.make_batch; q [rows][heads][D] fp32 numpy."""
    kc, vc, ks, vs = (torch.from_numpy(np.ascontiguousarray(x)).to(DEV) for x in cache)
    qd = torch.from_numpy(np.ascontiguousarray(q)).to(DEV).double()
    hk, d = kc.shape[1], kc.shape[3]
    hq = q.shape[1]
    g = hq // hk
    scale = d ** -0.5 if scale is None else scale
    out = torch.full(qd.shape, float("nan"), dtype=torch.float64, device=DEV)
    bound = out.clone()
    for s, length in enumerate(b["lens"].tolist()):
        q0, n = int(b["q_start"][s]), int(b["q_start"][s + 1] - b["q_start"][s])
        if n == 0:
            continue
        pages = torch.from_numpy(b["table"][s, :-(-length // kc.shape[2])].astype(np.int64)).to(DEV)
        limit = (length - n + torch.arange(n, device=DEV)).repeat_interleave(g)
        hidden = torch.arange(length, device=DEV)[None] > limit[:, None]
        for h in range(hk):
            kd = (kc[pages, h].double() * ks[pages, h].double()[:, None, None]).reshape(-1, d)[:length]
            vd = (vc[pages, h].double() * vs[pages, h].double()[:, None, None]).reshape(-1, d)[:length]
            rows = qd[q0:q0 + n, h * g:(h + 1) * g].reshape(n * g, d)
            if length == 0:
                o = e = torch.zeros_like(rows)
            else:
                x = (rows @ kd.T * scale).masked_fill_(hidden, float("-inf"))
                m = x.amax(-1, keepdim=True)
                p = torch.exp(x - torch.where(m.isinf(), torch.zeros_like(m), m))
                p /= p.sum(-1, keepdim=True).clamp(min=1e-300)
                o = p @ vd
                ds = (rows.abs() @ kd.abs().T).masked_fill_(hidden, 0.0).amax(-1, keepdim=True)
                ds *= scale * (d + 8) * 2.0 ** -24
                seen = (limit + 1).clamp(min=0).double()[:, None]
                rel = 2 * 2.0 ** -11 + 2 * 2.0 ** -18 + 2 * seen * 2.0 ** -24 + 2 * ds
                # the result's rounding: half a step of bf16, 2^-8 of a normal value; below 2^-126 steps are
                # 2^(-126 - 7) wide whatever the value, half of one 2^-134
                half_step = (o.abs() * 2.0 ** -8).clamp(min=2.0 ** -134)
                e = (rel * p + p.clamp(max=2.0 ** -21)) @ vd.abs() + half_step
            out[q0:q0 + n, h * g:(h + 1) * g] = o.view(n, g, d)
            bound[q0:q0 + n, h * g:(h + 1) * g] = e.view(n, g, d)
    return out.cpu().numpy(), bound.cpu().numpy()


def whole_tiles(b, group, hk):
    """Whether the kernel for prompts takes this batch tile by tile (no tile dearer than a CTA's even share of the
    work) or in equal shares of the whole."""
    tokens = 2 * (128 // group)
    most = total = 0
    for s, length in enumerate(b["lens"].tolist()):
        n = int(b["q_start"][s + 1] - b["q_start"][s])
        for t in range(-(-n // tokens)):
            last = length - n + min(n, (t + 1) * tokens) - 1
            blocks = last // 128 + 1 if last >= 0 else 0
            most = max(most, blocks)
            total += hk * (blocks + 2 if blocks else 0)
    ctas = min(torch.cuda.get_device_properties(0).multi_processor_count, 160)
    return (most + 2) * ctas <= total
