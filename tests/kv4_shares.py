"""A restatement in Python of how the attention over the 4-bit cache shares its tiles out to thread blocks when there
are many rows per KV head: 256 query rows of one KV head are a tile, and a block's share is a list of works, each a
tile over key blocks j0 .. j1 - 1. For tests that need a certain order of works in a share."""

from collections import namedtuple

Work = namedtuple("Work", "request head tile j0 j1 starts ends")

SMS = 148
START = 4          # what starting a tile costs, in blocks of keys


def block_keys(d):
    return 96 if d == 64 else 48


def cut_cost(parts, d):
    return 2 + parts * d // 2600


def _ceil(a, b):
    return -(-a // b)


def uses_tiles(max_q, group, d):
    """Whether a call of these sizes goes to the kernel that works on tiles."""
    return max_q * group > (16 if d == 176 else 32)


def shares(d, h, hk, queries, keys, causal, max_q=None, max_kv=None):
    """[block] -> works in their order, for good requests over `keys` positions each."""
    group, B, T = h // hk, len(queries), sum(queries)
    max_q, max_kv, bk = max_q or max(queries), max_kv or max(keys), block_keys(d)
    assert uses_tiles(max_q, group, d)
    bound = hk * min(B * _ceil(max_q * group, 256), T * group // 256 + B)
    assert bound * (8 + _ceil(max_kv, 48)) < 2 ** 31        # else costs are counted in coarser units
    may_cut = _ceil(bound, SMS) * (START + _ceil(max_kv, bk)) > cut_cost(SMS, d) + 2

    def blocks(b, tile):
        last = min(queries[b] * group, 256 * (tile + 1)) - 1
        limit = keys[b] if not causal else max(0, min(keys[b], keys[b] - queries[b] + last // group + 1))
        return _ceil(limit, bk)

    # request by request, head by head, from the last tile to the first
    tiles = [(b, g, i, blocks(b, i)) for b in range(B) for g in range(hk)
             for i in reversed(range(_ceil(queries[b] * group, 256)))]
    costs = [START + t[3] for t in tiles]
    count = len(tiles)
    if count == 0:
        return [[] for _ in range(SMS)]
    parts = count if count < SMS else 2 * SMS
    cut = may_cut and _ceil(count, SMS) * max(costs) > sum(costs) // SMS + cut_cost(parts, d)
    if not cut:
        costs = [1] * count
    total = sum(costs)
    n = min(total, SMS)
    if count < n:
        n = n // count * count
    each, more = total // n, total % n
    out, at, x = [], 0, 0
    for k in range(SMS):
        left = 0
        if k < n:
            left = each * (k + 1) + more * (k + 1) // n - (each * k + more * k // n)
        works = []
        while left > 0:
            b, g, i, all_ = tiles[at]
            take = min(left, costs[at] - x)
            j0 = max(0, x - START) if cut else 0
            j1 = min(all_, max(0, x + take - START)) if cut else all_
            if j1 > j0 or (all_ == 0 and x == 0):
                works.append(Work(b, g, i, j0, j1, j0 == 0, j1 == all_))
            left -= take
            x += take
            if x == costs[at]:
                at, x = at + 1, 0
        out.append(works)
    assert at == count and x == 0
    return out


def keyless_before_keys(share, rows_of, half):
    """Works of a share with keys, in this half of the tile's rows, right behind one or more without any key."""
    found, waiting = [], False
    for w in share:
        if rows_of(w.request) - 256 * w.tile <= 128 * half:
            continue                                            # the half has no row
        if w.j1 == w.j0:
            waiting = True
        else:
            if waiting:
                found.append(w)
            waiting = False
    return found


def attend64(q, k, v, scale, limits):
    """oracle.kv4.attend for many rows: q [n][H][d], k and v [keys][Hkv][d] in 64 bits, query i sees keys below limits[i].
    Returns out, lse, and what bounds of the error need: the sum of weight * |v|, and the largest sum over dims of
    |q k| * scale that a row sees."""
    import torch
    n, H, d = q.shape
    group = H // k.shape[1]
    out, mass = q.new_zeros((n, H, d)), q.new_zeros((n, H, d))
    lse, size = q.new_full((n, H), -float("inf")), q.new_zeros((n, H))
    if len(k) == 0:
        return out, lse, mass, size
    unseen = torch.arange(len(k), device=q.device)[None] >= limits[:, None]
    none = unseen.all(-1)
    for h in range(H):
        kk, vv = k[:, h // group], v[:, h // group]
        s = (q[:, h] @ kk.T * scale).masked_fill(unseen, -float("inf"))
        lse[:, h] = torch.logsumexp(s, -1)
        w = torch.exp(s - torch.where(none, 0.0, lse[:, h])[:, None])
        out[:, h], mass[:, h] = w @ vv, w @ vv.abs()
        size[:, h] = (q[:, h].abs() @ kk.abs().T * scale).masked_fill(unseen, 0.0).amax(-1)
    return out, lse, mass, size


def off_by(out, lse, q, k, v, scale, limits):
    """How far a request's results lie from the definition, as multiples of what roundings explain (out, lse). The
    bounds are those of the other tests of attention: a score is a sum of d products in fp32, off by at most
    e = (d + 4) 2^-23 sum|q k| scale plus its scaling's rounding; a weight is then off by a factor e^(2 e), by half an
    fp16 step and by 2^-20 for exp2 and the sums, or by 2^-30 of the largest where it is tiny; the result is rounded to
    bf16. Rows without a key have to be 0 and -inf exactly."""
    import torch
    want, want_lse, mass, size = attend64(q, k, v, scale, limits)
    seen = (limits > 0) & (len(k) > 0)
    e = (q.shape[-1] + 4) * 2.0 ** -23 * size + 2.0 ** -22 * torch.where(seen[:, None], want_lse, 0.0).abs()
    weight = (2.02 * e + 1.01 * 2.0 ** -11 + 2.0 ** -20)[..., None]
    tiny = len(k) * 2.0 ** -30 * (float(v.abs().max()) if len(k) else 0.0)
    bound = 2.0 ** -8 * want.abs() * 1.01 + 1.01 * weight * mass + tiny + 1e-37
    # NaN counts as off
    far = lambda got, exact, b: float(((got - exact).abs() / b).nan_to_num(float("inf")).max()) if got.numel() else 0.0  # noqa: E731
    assert bool((out[~seen] == 0).all()) and bool((lse[~seen] == -float("inf")).all())
    return far(out[seen], want[seen], bound[seen]), far(lse[seen], want_lse[seen], (e + 2.0 ** -20)[seen])
