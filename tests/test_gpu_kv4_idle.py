"""Attention over the 4-bit cache where some works have query rows but no key: the other requests' results are theirs."""

import pytest
import torch

from kv4_shares import off_by
from masked_block_diffusion_b200 import KVCache4, binding, build
from test_kv4_shares import IDLE_BATCHES, IDS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_all()
    binding.load()


def make(d, h, hk, page, queries, room, seed):
    """A cache of random codes and scales over two octaves with room for `room` positions per request, pages in random
    order, and bf16 queries large enough that the softmax is far from flat."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = [max(1, -(-n // page)) for n in room]
    cache = KVCache4(sum(per), page, hk, d)
    u = torch.randint(1, 16, (2, *cache.codes.shape), generator=g, device="cuda", dtype=torch.uint8)
    cache.codes.copy_(u[0] | (u[1] << 4))
    cache.scales.copy_(torch.randint(88, 104, cache.scales.shape, generator=g, device="cuda", dtype=torch.uint8))
    order = torch.randperm(sum(per), generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(per), max(per)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    q = (4 * torch.randn((sum(queries), h, d), generator=g, device="cuda")).bfloat16()
    start = torch.tensor([0] + queries, device="cuda").cumsum(0).to(torch.int32)
    return cache, table, q, start


def check(cache, table, q, out, lse, queries, keys, causal):
    """Every row of every request against the definition in 64 bits."""
    t = 0
    for b, (n, m) in enumerate(zip(queries, keys)):
        pos = torch.arange(m, dtype=torch.int32, device="cuda")
        k, v = (x.double() for x in cache.read(torch.full_like(pos, b), pos, table))
        i = torch.arange(n, device="cuda")
        limits = (m - n + i + 1).clamp(min=0, max=m) if causal else torch.full_like(i, m)
        rows = slice(t, t + n)
        off = off_by(out[rows].double(), lse[rows].double(), q[rows].double(), k, v, q.shape[-1] ** -0.5, limits)
        assert max(off) <= 1.0, (b, off)
        t += n


@pytest.mark.parametrize("case", IDLE_BATCHES, ids=IDS)
def test_requests_without_keys_do_not_touch_the_others(case):
    _, d, h, hk, queries, keys, causal = case
    cache, table, q, start = make(d, h, hk, 64, queries, keys, seed=d + len(keys))
    lens = torch.tensor(keys, dtype=torch.int32, device="cuda")
    out, lse = cache.attend(q, start, lens, table, max_q=max(queries), max_kv=max(keys), causal=causal, return_lse=True)
    check(cache, table, q, out, lse, queries, keys, causal)


def test_idle_slots_of_a_captured_batch_come_and_go():
    """One graph of a batch of fixed size, replayed as slots fall idle and come back."""
    B, d, h, hk, n, most = 32, 64, 16, 4, 256, 2000
    queries = [n] * B
    cache, table, q, start = make(d, h, hk, 64, queries, [most] * B, seed=5)
    lens = torch.full((B,), most, dtype=torch.int32, device="cuda")
    cache.attend(q, start, lens, table, max_q=n, max_kv=most, return_lse=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = cache.attend(q, start, lens, table, max_q=n, max_kv=most, return_lse=True)
    for idle in ([], [0], [5, 6, 7, 20], list(range(0, B, 4)), list(range(B - 1)), list(range(B))):
        keys = [0 if b in idle else most - 31 * b for b in range(B)]
        lens.copy_(torch.tensor(keys, dtype=torch.int32))
        graph.replay()
        check(cache, table, q, out, lse, queries, keys, False)
