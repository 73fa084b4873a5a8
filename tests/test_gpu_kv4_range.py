"""Attention over the 4-bit cache at the ends of its range: very large scores, long caches, large offsets."""

import numpy as np
import pytest
import torch

from masked_block_diffusion_b200 import KVCache4, binding, build
from oracle import kv4 as ref
from test_gpu_kv4 import filled, i32

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
