"""Attention over the 4-bit cache at the ends of its range: very large scores, long caches, large offsets."""

import numpy as np
import pytest
import torch

from masked_block_diffusion_b200 import KVCache4, Rope, binding, build, rope
from oracle import kv4 as ref
from test_gpu_kv4 import filled, i32
from test_gpu_kv4_idle import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_all()
    binding.load()


@pytest.mark.parametrize("d", [64, 128, 176])
@pytest.mark.parametrize("queries,keys", [(1, 300), (3, 3000), (40, 300), (40, 3000), (300, 700)])
def test_very_large_scores_give_the_largest_ones_value(d, queries, keys):
    """Scores far above what fp32 resolves in steps of one: the key of the largest score takes all the weight. Products
    q k are multiples of 1/64 here and below 2^14 in size, so they are exact, and the largest leads by 1 at least."""
    rng = np.random.default_rng(d + queries + keys)
    h, hk, page = 4, 2, 64
    cache, table, held = filled(rng, [keys], page, hk, d)
    k = rng.integers(-7, 8, (keys, hk, d)) * 0.125
    k[:, :, ::16] = 0.875                                             # every group's scale is 1/8
    q = rng.integers(-8, 9, (queries, h, d)) * 0.125
    best = np.empty((queries, h), int)
    for i in range(queries):
        for g in range(h):
            s = k[:, g // 2] @ q[i, g]
            best[i, g] = s.argmax()
            while np.sort(s)[-1] - np.sort(s)[-2] < 1.0:              # pull the leader ahead
                q[i, g] += np.sign(k[best[i, g], g // 2]) * 0.125
                s = k[:, g // 2] @ q[i, g]
                best[i, g] = s.argmax()
    assert np.abs(q).max() < 16
    u, byte = ref.quantise(k)
    assert np.array_equal(ref.unpack(ref.pack(u), byte), k)
    p = np.arange(keys)
    codes, scales = cache.codes.cpu().numpy(), cache.scales.cpu().numpy()
    codes[table[0, p // page], 0, :, p % page] = ref.pack(u)
    scales[table[0, p // page], 0, :, p % page] = byte
    cache.codes.copy_(torch.tensor(codes))
    cache.scales.copy_(torch.tensor(scales))
    qt = torch.tensor(q, device="cuda").bfloat16()
    assert np.array_equal(qt.double().cpu().numpy(), q)
    top = np.array([[k[best[i, g], g // 2] @ q[i, g] for g in range(h)] for i in range(queries)])
    want = np.array([[held[0][1][best[i, g], g // 2] for g in range(h)] for i in range(queries)])
    for scale in (1.1e3, 2.0 ** 20, 3.3e7, 7.7e8, 2.0 ** 36, 1.3e15, 3.1e30):
        out, lse = cache.attend(qt, i32([0, queries]), i32([keys]), i32(table), queries, keys, scale=scale, return_lse=True)
        got = out.double().cpu().numpy()
        assert np.array_equal(got, want), (scale, np.abs(got - want).max())
        # the score's product with scale and log2 e, log2 of the sum and the way back: a few roundings
        z = lse.double().cpu().numpy()
        assert np.all(np.abs(z - top * scale) <= 8 * 2.0 ** -24 * np.abs(top * scale) + 1e-6)


@pytest.mark.parametrize("d", [64, 128, 176])
@pytest.mark.parametrize("queries", [1, 40])
@pytest.mark.parametrize("keys,ahead", [(256, 200), (600, 500)])
def test_scores_one_step_of_fp32_apart(d, queries, keys, ahead):
    """Scores of 1.9e8 octaves, where fp32 numbers are 16 apart, first all equal, then one 16 octaves above the others:
    it weighs 65536 times as much as each of them. 256 keys go through one block. Results over 600 keys are joined from
    parts, each with the log of its sum in fp32: that is off by up to 8 octaves, and with it the parts' weights, so
    that all there is to say is that the result lies between the least and the largest value."""
    page, scale = 64, 16.0 / 1.4426950408889634
    rng = np.random.default_rng(d)
    cache, table, held = filled(rng, [keys], page, 1, d)
    k = np.zeros((keys, 1, d))
    k[:, 0, 0] = 448.0
    k[:, 0, 17] = 7.0                                                 # the group's scale is 1; no query looks at it
    k[ahead, 0, 16] = 1.0
    u, byte = ref.quantise(k)
    assert np.array_equal(ref.unpack(ref.pack(u), byte), k)
    p = np.arange(keys)
    codes, scales = cache.codes.cpu().numpy(), cache.scales.cpu().numpy()
    codes[table[0, p // page], 0, :, p % page] = ref.pack(u)
    scales[table[0, p // page], 0, :, p % page] = byte
    cache.codes.copy_(torch.tensor(codes))
    cache.scales.copy_(torch.tensor(scales))
    q = torch.zeros((queries, 2, d), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0], q[:, :, 16] = 26496.0, 1.0                            # 26496 * 448 = 11870208, and one more for the key ahead
    assert float(q[0, 0, 0]) == 26496.0
    out, lse = cache.attend(q, i32([0, queries]), i32([keys]), i32(table), queries, keys, scale=scale, return_lse=True)
    v = held[0][1][:, 0]
    w = np.full(keys, 2.0 ** -16)
    w[ahead] = 1.0
    want = (w[:, None] * v).sum(0) / w.sum()
    mass = (w[:, None] * np.abs(v)).sum(0) / w.sum()
    # bf16's half step, and fp16's of the weights
    bound = 2.0 ** -8 * 1.01 * np.abs(want) + 1.01 * 2.0 ** -11 * mass
    got = out.double().cpu().numpy()
    if keys == 256:
        assert np.all(np.abs(got - want) <= bound)
    else:
        room = 2.0 ** -8 * np.abs(v).max(0)
        assert np.all(got >= v.min(0) - room) and np.all(got <= v.max(0) + room)
    assert np.all(np.abs(lse.double().cpu().numpy() / (11870209 * scale) - 1) <= 8 * 2.0 ** -24)


@pytest.mark.parametrize("queries", [2, 40])
def test_pages_beyond_4_gb_of_codes(queries):
    """The same requests in a small cache and in the last pages of one whose offsets do not fit 32 bits."""
    d, h, hk, page, B, keys = 176, 16, 8, 64, 2, 300
    torch.manual_seed(queries)
    per = -(-keys // page)
    small, large = KVCache4(B * per, page, hk, d), KVCache4(60000, page, hk, d)
    assert large.codes.numel() > 1 << 32
    first = torch.arange(B * per, dtype=torch.int32, device="cuda").view(B, per)
    last = first + (large.n_pages - B * per)
    req = torch.arange(B, dtype=torch.int32, device="cuda").repeat_interleave(keys)
    pos = torch.arange(keys, dtype=torch.int32, device="cuda").repeat(B)
    k, v = (torch.randn(B * keys, hk, d, device="cuda") for _ in range(2))
    q = torch.randn(B * queries, h, d, device="cuda").bfloat16()
    start, lens = i32(np.arange(B + 1) * queries), i32([keys] * B)
    for cache, table in ((small, first), (large, last)):
        cache.append(k, v, req, pos, table, rope=Rope(d))
    a, b = ((*cache.read(req, pos, table), *cache.attend(q, start, lens, table, queries, keys, causal=True, return_lse=True))
            for cache, table in ((small, first), (large, last)))
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and a[0].any()
    assert not large.codes[:large.n_pages - B * per].any()


def test_rows_beyond_2_to_the_31_elements():
    """Tensors of more elements than 32 bits count: what lies at their end, against the same rows by themselves."""
    d, h, page, keys = 176, 8, 64, 200
    T = (1 << 31) // (h * d) + 1000
    plan, cache = Rope(d), KVCache4(8, page, h, d)
    big = torch.empty(T, h, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(600, h, d, device="cuda").bfloat16()
    big[-600:] = tail
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    assert torch.equal(rope(big, pos, plan, out=big)[-600:], rope(tail, pos[-600:].contiguous(), plan))
    big[-600:] = tail
    # append and read: all padding but the last tokens
    req = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    req[-keys:] = 0
    at = torch.zeros(T, dtype=torch.int32, device="cuda")
    at[-keys:] = torch.arange(keys, dtype=torch.int32, device="cuda")
    table = i32([[5, 2, 7, 0]])
    cache.append(big, big, req, at, table, rope=plan)
    other = KVCache4(8, page, h, d)
    other.append(tail[-keys:], tail[-keys:], req[-keys:].contiguous(), at[-keys:].contiguous(), table, rope=plan)
    assert torch.equal(cache.codes, other.codes) and torch.equal(cache.scales, other.scales) and cache.codes.any()
    k, v = (torch.empty_like(big) for _ in range(2))
    cache.read(req, at, table, k_out=k, v_out=v)
    for got, want in zip((k, v), cache.read(req[-keys:].contiguous(), at[-keys:].contiguous(), table)):
        assert torch.equal(got[-keys:], want)
    del v
    for n in (1, 257):
        start = [T - 2 * n, T - n, T]
        lens = i32([keys, keys - 31])
        two = i32([[5, 2, 7, 0]] * 2)
        out, lse = cache.attend(big, i32(start), lens, two, n, keys, causal=True, out=k, return_lse=True)
        want = cache.attend(tail[600 - 2 * n:], i32([0, n, 2 * n]), lens, two, n, keys, causal=True, return_lse=True)
        assert torch.equal(out[-2 * n:], want[0]) and torch.equal(lse[-2 * n:], want[1]), n


@pytest.mark.parametrize("d,h,hk,queries,keys", [(64, 4, 2, 256, 131072), (176, 2, 1, 200, 100001), (64, 2, 1, 1, 1 << 20), (128, 4, 1, 7, 300007)])
def test_caches_of_many_keys(d, h, hk, queries, keys):
    cache, table, q, start = make(d, h, hk, 64, [queries], [keys], seed=d)
    out, lse = cache.attend(q, start, i32([keys]), table, queries, keys, causal=True, return_lse=True)
    check(cache, table, q, out, lse, [queries], [keys], True)


@pytest.mark.parametrize("d", [64, 176])
@pytest.mark.parametrize("queries", [1, 36])
def test_queries_of_any_magnitude(d, queries):
    """From bf16's subnormal numbers to 2^108, a magnitude per request; within a row too."""
    exps = list(range(-130, 110, 6))
    B, keys = len(exps), 200
    cache, table, q, start = make(d, 4, 2, 32, [queries] * B, [keys] * B, seed=3)
    size = torch.tensor([2.0 ** e for e in exps], dtype=torch.float64, device="cuda").repeat_interleave(queries)
    spread = torch.exp2(torch.randint(-12, 1, q.shape, device="cuda").double())
    q = (q.double() * size[:, None, None] * spread).bfloat16()
    assert torch.isfinite(q).all()
    out, lse = cache.attend(q, start, i32([keys] * B), table, queries, keys, return_lse=True)
    check(cache, table, q, out, lse, [queries] * B, [keys] * B, False)


@pytest.mark.parametrize("queries", [1, 17])
def test_as_many_requests_as_a_call_takes(queries):
    B, d, h, keys = 65535, 64, 2, 16
    cache, table, q, start = make(d, h, 1, 16, [queries] * B, [keys] * B, seed=4)
    out, lse = cache.attend(q, start, i32([keys] * B), table, queries, keys, return_lse=True)
    pos = torch.arange(keys, dtype=torch.int32, device="cuda").repeat(B)
    k, v = (t.view(B, keys, d) for t in cache.read(torch.arange(B, dtype=torch.int32, device="cuda").repeat_interleave(keys), pos, table))
    s = q.view(B, queries * h, d).double() @ k.double().transpose(1, 2) * d ** -0.5
    w = torch.softmax(s, -1)
    want, mass = w @ v.double(), w @ v.double().abs()
    # scores below 64 in size, sums of 64 products: e = 68 2^-23 sum|q k| scale < 2^-10
    e = 68 * 2.0 ** -23 * (q.view(B, queries * h, d).double().abs() @ k.double().abs().transpose(1, 2) * d ** -0.5).amax(-1)
    assert float(e.max()) < 2.0 ** -10
    bound = 2.0 ** -8 * 1.01 * want.abs() + (2.02 * e[..., None] + 1.01 * 2.0 ** -11 + 2.0 ** -20) * mass + 1e-37
    assert bool(((out.view_as(want).double() - want).abs() <= bound).all())
    assert bool(((lse.view(B, -1).double() - torch.logsumexp(s, -1)).abs() <= e + 2.0 ** -17).all())
