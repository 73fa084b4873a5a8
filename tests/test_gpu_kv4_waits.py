"""Attention over the 4-bit cache when waits inside its kernels run out."""

import pytest
import torch

from kv4_shares import shares
from masked_block_diffusion_b200 import Denoiser, binding, build
from synth import WORKLOADS, blob_from_weights, gen_weights
from test_gpu_kv4_idle import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    build.build_all()
    cfg = WORKLOADS["c1-tiny-dense"].model
    den = Denoiser(cfg, blob_from_weights(cfg, gen_weights(cfg)), max_ctx=256, max_batch=1)
    yield den.h
    den.close()


@pytest.mark.parametrize("d", [64, 128, 176])
def test_a_wait_of_the_tile_kernel_that_runs_out_loses_rows_and_nothing_else(handle, d):
    """The first request has a bad length and 60 000 rows, which its thread block fills with NaN for milliseconds while
    the warps that issue products wait for the next tile's queries: longer than a limit of 1 ns and a suspended try."""
    h, hk, n, B, keys, many = 8, 4, 256, 100, 500, 60000
    cache, table, q, start = make(d, h, hk, 64, [many] + [n] * B, [1] + [keys] * B, seed=d)
    lens = torch.full((B + 1,), keys, dtype=torch.int32, device="cuda")
    lens[0] = -1
    # to the sharing rule a bad request is one tile per head without keys
    first = shares(d, h, hk, [1] + [n] * B, [0] + [keys] * B, False)[0]
    assert any(w.request == 0 for w in first) and first[-1].request > 0

    def call():
        return cache.attend(q, start, lens, table, n, keys, return_lse=True)

    out, lse = call()
    assert torch.isnan(out[:many]).all() and torch.isnan(lse[:many]).all()
    check(cache, table[1:], q[many:], out[many:], lse[many:], [n] * B, [keys] * B, False)
    torch.cuda.synchronize()
    binding.dllm_set_wait_limit(handle, 1)
    try:
        o, z = call()
        torch.cuda.synchronize()
    finally:
        binding.dllm_set_wait_limit(handle, 0)
    lost = torch.isnan(z)
    assert torch.equal(lost, torch.isnan(o).all(-1)) and torch.equal(lost, torch.isnan(o).any(-1)) and lost[:many].all()
    assert torch.equal(o[~lost], out[~lost]) and torch.equal(z[~lost], lse[~lost])
    group = h // hk
    for w in first:                                                  # what the block took up after the bad tiles
        if w.request > 0:
            R = torch.arange(256 * w.tile, min(n * group, 256 * (w.tile + 1)), device="cuda")
            assert lost[many + (w.request - 1) * n + R // group, w.head * group + R % group].all()
    o, z = call()
    assert torch.equal(o[many:], out[many:]) and torch.equal(z[many:], lse[many:])


def test_waits_of_the_few_row_kernel_that_run_out_lose_rows_and_nothing_else(handle):
    """Requests with pages of their own, which come from memory while another stream fills memory. How long a copy
    takes is not in the test's hands; where every wait was short enough it says so."""
    B, d, h, hk, queries, keys = 64, 176, 16, 8, 1, 4352
    cache, table, q, start = make(d, h, hk, 64, [queries] * B, [keys] * B, seed=d + queries)
    lens = torch.full((B,), keys, dtype=torch.int32, device="cuda")
    big = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    out, lse = cache.attend(q, start, lens, table, queries, keys, return_lse=True)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    most = 0
    torch.cuda.synchronize()
    binding.dllm_set_wait_limit(handle, 1)
    try:
        for i in range(5):
            with torch.cuda.stream(side):
                big.fill_(i)
            o, z = cache.attend(q, start, lens, table, queries, keys, return_lse=True)
            torch.cuda.synchronize()
            lost = torch.isnan(z)
            most = max(most, int(lost.sum()))
            assert torch.equal(lost, torch.isnan(o).all(-1)) and torch.equal(lost, torch.isnan(o).any(-1))
            assert torch.equal(o[~lost], out[~lost]) and torch.equal(z[~lost], lse[~lost])
    finally:
        torch.cuda.synchronize()
        binding.dllm_set_wait_limit(handle, 0)
    o, z = cache.attend(q, start, lens, table, queries, keys, return_lse=True)
    assert torch.equal(o, out) and torch.equal(z, lse)
    if most == 0:
        pytest.skip("no wait ran out in five calls: the path that loses rows was not taken")


@pytest.mark.parametrize("d,h,hk,B", [(176, 4, 2, 150), (64, 16, 1, 37)])
def test_answering_a_large_bad_request_does_not_keep_the_next_tile_waiting_for_long(handle, d, h, hk, B):
    """60 000 rows of NaN for two KV heads with 2 heads of 176 each are 84 MB, for one with 16 heads of 64 123 MB. The limit
    of 10 ms for them, 12 GB/s from one thread block, stands for the default of 2 s for 200 times as many."""
    n, keys, many = 256, 500, 60000
    cache, table, q, start = make(d, h, hk, 64, [many] + [n] * B, [1] + [keys] * B, seed=d)
    lens = torch.full((B + 1,), keys, dtype=torch.int32, device="cuda")
    lens[0] = -1
    first = shares(d, h, hk, [1] + [n] * B, [0] + [keys] * B, False)[0]
    assert [w.request for w in first[:hk]] == [0] * hk and first[hk].request == 1
    torch.cuda.synchronize()
    binding.dllm_set_wait_limit(handle, 10_000_000)
    try:
        out, lse = cache.attend(q, start, lens, table, n, keys, return_lse=True)
        torch.cuda.synchronize()
    finally:
        binding.dllm_set_wait_limit(handle, 0)
    assert torch.isnan(out[:many]).all() and torch.isnan(lse[:many]).all()
    assert torch.isfinite(out[many:]).all() and torch.isfinite(lse[many:]).all()
