"""Plain numpy forms of the paged 8-bit key/value cache, written from the definitions: the append in
fp32 operation by operation (its codes are defined so), attention in 64 bits, one row at a time."""
import numpy as np

F = np.float32


def bf16_round(x):
    """fp32 values rounded to the nearest bf16 (ties to even), as fp32."""
    u = np.ascontiguousarray(x, F).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(F)


def rope_table(max_pos, d, theta=500000.0):
    w = theta ** (-2.0 * np.arange(d // 2) / d)
    ang = np.arange(max_pos)[:, None] * w
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(F)


def rotate(x, row):
    """x [heads][D] fp32 by one row of the table; every product and sum rounded to fp32."""
    h = x.shape[-1] // 2
    c, s = row[:h], row[h:]
    a, b = x[..., :h], x[..., h:]
    return np.concatenate([F(a * c) - F(b * s), F(b * c) + F(a * s)], -1).astype(F)


def append(cache, table, lens, q_start, k, v, q=None, rope=None):
    """In place on cache = [k, v, k_step, v_step] (numpy); returns rotated queries (bf16 values, fp32)."""
    size = cache[0].shape[2]
    out = None if q is None else np.array(q, F)
    for b in range(len(lens)):
        q0, n = int(q_start[b]), int(q_start[b + 1] - q_start[b])
        first = int(lens[b]) - n
        rows = range(q0, q0 + n)
        kr = [np.array(k[t], F) if rope is None else rotate(k[t], rope[first + t - q0]) for t in rows]
        if q is not None:
            for t in rows:
                out[t] = bf16_round(q[t] if rope is None else rotate(q[t], rope[first + t - q0]))
        if n == 0:
            continue
        for j in range(first // size, (first + n - 1) // size + 1):
            lo, hi = max(first, j * size), min(first + n, (j + 1) * size)
            p = int(table[b, j])
            for codes, steps, x in ((cache[0], cache[2], np.stack(kr[lo - first:hi - first])),
                                    (cache[1], cache[3], np.asarray(v[q0 + lo - first:q0 + hi - first], F))):
                for h in range(codes.shape[1]):
                    t = F(np.abs(x[:, h]).max()) * (F(1) / F(127))
                    old = steps[p, h] if lo > j * size else F(0)
                    step = max(old, t)
                    if lo > j * size and step > old:
                        ratio = F(old / step)
                        was = codes[p, h, :lo - j * size].astype(F)
                        codes[p, h, :lo - j * size] = np.rint(F(was * ratio)).astype(np.int8)
                    with np.errstate(divide="ignore", invalid="ignore"):
                        new = np.clip(np.rint(x[:, h] / step), -127, 127) if step > 0 else np.zeros_like(x[:, h])
                    codes[p, h, lo - j * size:hi - j * size] = new.astype(np.int8)
                    steps[p, h] = step
    return out


def attention(cache, table, lens, q_start, q, scale=None):
    """64-bit result for every row of a sequence; other rows NaN."""
    kc, vc, ks, vs = cache
    size, d = kc.shape[2], kc.shape[3]
    hq, hk = q.shape[1], kc.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out = np.full(q.shape, np.nan)
    for b in range(len(lens)):
        q0, n, length = int(q_start[b]), int(q_start[b + 1] - q_start[b]), int(lens[b])
        if n == 0:
            continue
        pages = table[b, :-(-length // size)].astype(np.int64)
        for h in range(hk):
            kd = (kc[pages, h].astype(np.float64) * ks[pages, h, None, None].astype(np.float64)).reshape(-1, d)
            vd = (vc[pages, h].astype(np.float64) * vs[pages, h, None, None].astype(np.float64)).reshape(-1, d)
            for i in range(n):
                seen = max(0, length - n + i + 1)
                for g in range(h * (hq // hk), (h + 1) * (hq // hk)):
                    if seen == 0:
                        out[q0 + i, g] = 0.0
                        continue
                    s = (kd[:seen] @ q[q0 + i, g].astype(np.float64)) * scale
                    p = np.exp(s - s.max())
                    out[q0 + i, g] = (p / p.sum()) @ vd[:seen]
    return out


def attention_bound(cache, table, lens, q_start, q, ref, scale=None):
    """Largest error that the kernels' documented roundings allow, per output element, from the inputs:

    * the result is rounded to bf16 once: half a step, 2^-8 |o|;
    * weights enter the products in fp16, relative to the running maximum and times a factor of at least 2^-4
      (v_step in units of a power of two near it): each is off by 2^-11 of itself, twice that for the rounding of
      the factor, or, where weight times factor is below fp16's normal range, by half of the spacing 2^-24 there,
      2^-25 / 2^-4 = 2^-21 of the largest weight, and never by more than itself (it becomes 0 at worst).  So by
      sum_j (2 2^-11 p_j + min(p_j, 2^-21)) |v_j|, p normalised (the sum is at least the largest weight);
    * a score is a sum of D products of codes (exact in fp16) and queries (bf16, exact in fp16 after scaling),
      in fp32: off by (D + 8) 2^-24 sum_d |q_d k_d| scale at most, which moves p by as much of itself, in the
      numerator and in the sum; exp2 (2.7e-6 of p where a polynomial gives it) and the remaining fp32 operations
      add less than 2^-18 of p each way;
    * fp32 sums over L tokens: L 2^-24 of sum p |v|, numerator and denominator.
    """
    kc, vc, ks, vs = cache
    size, d = kc.shape[2], kc.shape[3]
    hq, hk = q.shape[1], kc.shape[1]
    scale = d ** -0.5 if scale is None else scale
    bound = np.full(q.shape, np.nan)
    for b in range(len(lens)):
        q0, n, length = int(q_start[b]), int(q_start[b + 1] - q_start[b]), int(lens[b])
        pages = table[b, :-(-length // size)].astype(np.int64)
        for h in range(hk):
            kd = np.abs(kc[pages, h].astype(np.float64) * ks[pages, h, None, None]).reshape(-1, d)
            kd_s = (kc[pages, h].astype(np.float64) * ks[pages, h, None, None]).reshape(-1, d)
            vd = np.abs(vc[pages, h].astype(np.float64) * vs[pages, h, None, None]).reshape(-1, d)
            for i in range(n):
                seen = max(0, length - n + i + 1)
                for g in range(h * (hq // hk), (h + 1) * (hq // hk)):
                    if seen == 0:
                        bound[q0 + i, g] = 0.0
                        continue
                    qq = q[q0 + i, g].astype(np.float64)
                    s = (kd_s[:seen] @ qq) * scale
                    ds = (kd[:seen] @ np.abs(qq)) * scale * (d + 8) * 2.0 ** -24
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    rel = 2 * 2.0 ** -11 + 2 * 2.0 ** -18 + 2 * seen * 2.0 ** -24 + 2 * ds.max()
                    bound[q0 + i, g] = (rel * p + np.minimum(p, 2.0 ** -21)) @ vd[:seen]
    return bound + np.abs(ref) * 2.0 ** -8
