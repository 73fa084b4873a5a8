"""The rule by which attention over the 4-bit cache shares tiles out, and that the batches used on the GPU to test works
without keys contain them where they matter (no GPU)."""

import numpy as np
import pytest
import torch

from kv4_shares import attend64, block_keys, keyless_before_keys, off_by, shares
from oracle import kv4 as ref

# batches in which some thread block takes a tile without keys and then one with keys: idle slots of a batch of fixed
# size that keep their query rows, and causal pieces that are longer than what they see
# (name, d, heads, KV heads, queries, keys, causal)
IDLE_BATCHES = [
    ("one of 16 canvases idle", 176, 16, 8, [256] * 16, [0 if b == 3 else 4352 for b in range(16)], False),
    ("every fourth of 32 canvases idle", 64, 16, 4, [256] * 32, [0 if b % 4 == 0 else 2000 for b in range(32)], False),
    ("every fourth of 32 canvases idle, d 128", 128, 16, 4, [256] * 32, [0 if b % 4 == 3 else 2000 for b in range(32)], False),
    ("pieces longer than their keys", 64, 16, 4, [1024] * 8, [512 + 64 * b for b in range(8)], True),
    ("pieces longer than their keys, d 176", 176, 16, 4, [1024] * 8, [512 + 64 * b for b in range(8)], True),
    ("two idle of many short ones", 128, 8, 4, [70 + b % 5 for b in range(90)], [0 if b in (20, 51) else 100 + 7 * b for b in range(90)], False),
]
IDS = [c[0] for c in IDLE_BATCHES]


@pytest.mark.parametrize("case", IDLE_BATCHES, ids=IDS)
def test_the_batches_with_idle_requests_have_keyless_works_before_others(case):
    _, d, h, hk, queries, keys, causal = case
    works = shares(d, h, hk, queries, keys, causal)
    for half in (0, 1):
        if half == 1 and max(queries) * (h // hk) <= 128 + 256 * (max(queries) * (h // hk) // 256):
            continue
        assert sum(len(keyless_before_keys(s, lambda b: queries[b] * (h // hk), half)) for s in works) >= 1


@pytest.mark.parametrize("d,h,hk", [(64, 8, 2), (128, 16, 8), (176, 6, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_shares_cover_every_block_of_keys_once(d, h, hk, causal):
    rng = np.random.default_rng(d)
    for B, most in ((1, 4000), (5, 9000), (40, 700), (300, 200)):
        queries = [int(n) for n in rng.integers(0, 300, B)]
        keys = [int(n) for n in rng.integers(0, most, B)]
        queries[0], keys[-1] = 300, 0
        works = shares(d, h, hk, queries, keys, causal)
        seen = {}
        for block, share in enumerate(works):
            for i, w in enumerate(share):
                # a part that does not end its tile is a block's last work, one that does not begin it its first
                assert w.ends or i == len(share) - 1
                assert w.starts or i == 0
                seen.setdefault((w.request, w.head, w.tile), []).append((block, w))
        group = h // hk
        assert len(seen) == sum(hk * -(-n * group // 256) for n in queries)
        for (b, _, tile), parts in seen.items():
            last = (min(queries[b] * group, 256 * (tile + 1)) - 1) // group
            limit = keys[b] if not causal else max(0, min(keys[b], keys[b] - queries[b] + last + 1))
            assert [w.j0 for _, w in parts] == [0] + [w.j1 for _, w in parts[:-1]]
            assert parts[-1][1].j1 == -(-limit // block_keys(d)) and parts[0][1].starts and parts[-1][1].ends
            assert [k for k, _ in parts] == list(range(parts[0][0], parts[0][0] + len(parts)))


def _request(seed, n, H, hk, d, keys):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((n, H, d), generator=g, dtype=torch.float64) * 4
    k, v = (torch.randint(-7, 8, (keys, hk, d), generator=g).double() * 0.125 for _ in range(2))
    return q.bfloat16().double(), k, v


def test_the_definition_for_many_rows_is_the_oracle():
    q, k, v = _request(1, 9, 4, 2, 64, 30)
    limits = torch.tensor([0, 1, 5, 29, 30, 30, 2, 0, 7])
    for got, want in zip(attend64(q, k, v, 0.125, limits), ref.attend(q.numpy(), k.numpy(), v.numpy(), 0.125, limits)):
        assert np.allclose(got.numpy(), want, rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("d,keys", [(64, 2000), (128, 2000), (176, 4352)])
def test_scores_of_another_works_queries_lie_outside_the_bounds(d, keys):
    """The first block of keys scored with other queries: outputs and sums leave the bounds by far; rounded exact
    results lie within."""
    q, k, v = _request(d, 8, 2, 1, d, keys)
    other = _request(d + 1, 8, 2, 1, d, 1)[0]
    limits = torch.full((8,), keys)
    out, lse, _, _ = attend64(q, k, v, d ** -0.5, limits)
    assert max(off_by(out.bfloat16().double(), lse.float().double(), q, k, v, d ** -0.5, limits)) <= 1.0
    s = torch.einsum("nhd,kd->nhk", q, k[:, 0]) * d ** -0.5
    s[..., :48] = torch.einsum("nhd,kd->nhk", other, k[:48, 0]) * d ** -0.5
    wrong = torch.softmax(s, -1) @ v[:, 0]
    off = off_by(wrong.bfloat16().double(), torch.logsumexp(s, -1).float().double(), q, k, v, d ** -0.5, limits)
    assert min(off) > 4.0
