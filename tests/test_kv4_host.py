"""Rotation plans, the packed format and argument checks of the paged 4-bit KV cache (no GPU)."""

import ctypes

import numpy as np
import pytest

from masked_block_diffusion_b200 import DllmError, Rope, binding, build
from oracle import kv4 as ref


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build_dllm()
    return binding.load()


@pytest.mark.parametrize("rotary", [2, 30, 64, 128, 176, 256])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 32.0), ("yarn", 1.0)])
def test_rotation_plan_matches_the_definition(rotary, scaling, factor):
    if scaling == "ntk" and rotary < 4:
        with pytest.raises(DllmError):
            Rope(rotary, scaling=scaling, factor=factor)
        return
    plan = Rope(rotary, "interleaved", 10000.0, scaling, factor, 4096)
    f, m = ref.rope_frequencies(rotary, 10000.0, scaling, factor, 4096)
    got = np.array(plan.c.turns[:])
    # pow, a product and a quotient in 64 bits on either side
    assert np.allclose(got[:rotary // 2] * 2 * np.pi, f, rtol=1e-14, atol=0)
    assert not got[rotary // 2:].any()
    assert abs(plan.c.magnitude - m) < 1e-15 * 8
    assert plan.c.layout == binding.DLLM_ROPE_INTERLEAVED and plan.c.rotary_dim == rotary


def test_rotation_by_parts_keeps_fast_pairs_and_divides_slow_ones():
    f0, _ = ref.rope_frequencies(128)
    got = np.array(Rope(128, scaling="yarn", factor=16.0, original_ctx=4096).c.turns[:64]) * 2 * np.pi
    turns = f0 * 4096 / (2 * np.pi)
    assert np.allclose(got[turns > 40], f0[turns > 40], rtol=1e-14)
    assert np.allclose(got[turns < 0.8], f0[turns < 0.8] / 16, rtol=1e-14)
    assert np.all(got <= f0 * (1 + 1e-14)) and np.all(got >= f0 / 16 * (1 - 1e-14))


@pytest.mark.parametrize("args", [
    dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=258), dict(rotary_dim=64, theta=1.0),
    dict(rotary_dim=64, theta=float("inf")), dict(rotary_dim=64, scaling="linear", factor=0.5),
    dict(rotary_dim=64, scaling="linear", factor=float("nan")),
    dict(rotary_dim=64, scaling="yarn", factor=2.0, beta_fast=1.0, beta_slow=2.0),
    dict(rotary_dim=64, scaling="yarn", factor=2.0, beta_slow=0.0),
    dict(rotary_dim=64, scaling="yarn", factor=2.0, original_ctx=0)])
def test_rotation_plan_refuses(args):
    with pytest.raises(DllmError) as e:
        Rope(**args)
    assert e.value.code == binding.DLLM_E_INVAL


def test_rotation_plan_refuses_unknown_names():
    with pytest.raises(ValueError):
        Rope(64, layout="quarter")
    with pytest.raises(ValueError):
        Rope(64, scaling="longer")


def test_oracle_packing_round_trip_and_scale_rule():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(50, 176)) * np.exp(rng.normal(size=(50, 1)) * 4)
    x[3, 16:32] = 0.0
    x[4, :16] = 1e9
    x[5, 0] = np.nan
    codes, byte = ref.quantise(x)
    held = ref.unpack(ref.pack(codes), byte)
    s = np.repeat(ref.scale_values()[byte], 16, -1)
    assert np.array_equal(held, (codes.astype(float) - 8) * s)
    fine = (np.abs(x) < 7 * 2560) & ~np.isnan(x)
    assert np.all(np.abs(held - np.where(fine, x, 0))[fine] <= s[fine] / 2)
    assert not held[3, 16:32].any() and np.all(held[4, :16] == 17920.0) and held[5, 0] == 0.0
    # the least sufficient scale: the next smaller one would not do
    top = np.nanmax(np.abs(x).reshape(50, 11, 16), -1)
    inner = (byte > 0) & (byte < ref.MAX_SCALE_BYTE)
    assert np.all(7 * ref.scale_values()[byte - 1 * (byte > 0)][inner] < top[inner])
    assert np.all(7 * ref.scale_values()[byte][inner] >= top[inner])


def _cache(**kw):
    a = dict(codes=1 << 20, scales=1 << 21, n_pages=8, page=64, n_kv_heads=2, head_dim=64)
    a.update(kw)
    return binding.dllm_kv4(a["codes"], a["scales"], a["n_pages"], a["page"], a["n_kv_heads"], a["head_dim"])


BAD_CACHES = [dict(codes=None), dict(scales=None), dict(codes=(1 << 20) + 8), dict(scales=(1 << 21) + 1), dict(n_pages=0),
              dict(n_pages=-1), dict(page=8), dict(page=48), dict(page=512), dict(n_kv_heads=0), dict(head_dim=80),
              dict(head_dim=0), dict(n_pages=1 << 25, page=64)]
P = 1 << 22   # stands for a device address: a refused call never reads it


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_every_operation_refuses_a_bad_cache(lib, bad):
    c = _cache(**bad)
    assert lib.dllm_op_append_kv4(c, P, 128, 64, P, 128, 64, 0, P, P, None, 4, P, 1, 1, None, None) == binding.DLLM_E_INVAL
    assert lib.dllm_op_read_kv4(c, P, P, 4, P, 1, 1, P, P, 0, None) == binding.DLLM_E_INVAL
    assert lib.dllm_op_attn_kv4_workspace(c, 1, 1, 1, 64, 2) == binding.DLLM_E_INVAL
    assert lib.dllm_op_attn_kv4(c, P, 128, 64, P, 128, 64, None, P, P, 1, 1, 1, 64, 2, P, 1, 0, 1.0, None, 0,
                                None) == binding.DLLM_E_INVAL


def test_append_and_read_refuse(lib):
    c = _cache()
    ok = dict(k=P, v=P, type=0, req=P, pos=P, T=4, table=P, n_req=1, stride=1, rope=None)
    bad_rope = Rope(128).c                       # wider than the head
    for bad in (dict(k=None), dict(v=None), dict(type=2), dict(type=-1), dict(req=None), dict(pos=None), dict(T=-1),
                dict(table=None), dict(n_req=0), dict(stride=0), dict(rope=bad_rope)):
        a = {**ok, **bad}
        assert lib.dllm_op_append_kv4(c, a["k"], 128, 64, a["v"], 128, 64, a["type"], a["req"], a["pos"], None, a["T"],
                                      a["table"], a["n_req"], a["stride"], a["rope"], None) == binding.DLLM_E_INVAL, bad
    for bad in (dict(req=None), dict(pos=None), dict(T=-1), dict(table=None), dict(n_req=0), dict(stride=0), dict(k=P + 2),
                dict(v=P + 8)):
        a = {**ok, **bad}
        assert lib.dllm_op_read_kv4(c, a["req"], a["pos"], a["T"], a["table"], a["n_req"], a["stride"], a["k"], a["v"],
                                    0, None) == binding.DLLM_E_INVAL, bad
    # nothing to do is not an error, and queues nothing
    assert lib.dllm_op_append_kv4(c, None, 0, 0, None, 0, 0, 0, None, None, None, 0, None, 0, 0, None, None) == 0
    assert lib.dllm_op_read_kv4(c, None, None, 0, None, 0, 0, None, None, 0, None) == 0


def test_rope_refuses(lib):
    ok = dict(rope=Rope(64).c, x=P, xt=0, pos=P, T=4, H=2, hd=64, y=2 * P, yt=0, ys=64)
    for bad in (dict(rope=None), dict(x=None), dict(y=None), dict(pos=None), dict(xt=2), dict(yt=-1), dict(T=-1), dict(H=0), dict(H=32769),
                dict(H=16385), dict(hd=62), dict(hd=2048), dict(y=P, yt=1), dict(y=P, ys=128)):
        a = {**ok, **bad}
        assert lib.dllm_op_rope(a["rope"], a["x"], a["xt"], 128, 64, a["pos"], a["T"], a["H"], a["hd"], a["y"], a["yt"], 128,
                                a["ys"], 0, None) == binding.DLLM_E_INVAL, bad
    broken = Rope(64).c
    broken.rotary_dim = 63
    assert lib.dllm_op_rope(broken, P, 0, 128, 64, P, 4, 2, 64, 2 * P, 0, 128, 64, 0, None) == binding.DLLM_E_INVAL
    broken = Rope(64).c
    broken.layout = 5
    assert lib.dllm_op_rope(broken, P, 0, 128, 64, P, 4, 2, 64, 2 * P, 0, 128, 64, 0, None) == binding.DLLM_E_INVAL
    assert lib.dllm_op_rope(Rope(64).c, None, 0, 0, 0, None, 0, 2, 64, None, 0, 0, 0, 0, None) == 0


def test_attention_refuses(lib):
    c = _cache()
    ok = dict(q=P, qs=64, out=P, os=64, q_start=P, kv_len=P, B=1, T=1, max_q=1, max_kv=64, H=2, table=P, stride=1, scale=0.125,
              ws=None, wb=0)
    for bad in (dict(q=None), dict(out=None), dict(q_start=None), dict(kv_len=None), dict(table=None), dict(stride=0),
                dict(B=-1), dict(T=-1), dict(max_q=-1), dict(max_q=2), dict(max_kv=-1), dict(max_kv=1 << 29), dict(H=0),
                dict(H=3), dict(H=2 * 129), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(q=P + 2), dict(qs=60), dict(out=P + 4), dict(os=4), dict(B=65536),
                dict(ws=P + 4, wb=1 << 20),
                dict(max_kv=1 << 20)):            # needs a workspace, none given
        a = {**ok, **bad}
        assert lib.dllm_op_attn_kv4(c, a["q"], 128, a["qs"], a["out"], 128, a["os"], None, a["q_start"], a["kv_len"], a["B"],
                                    a["T"], a["max_q"], a["max_kv"], a["H"], a["table"], a["stride"], 0, a["scale"], a["ws"],
                                    a["wb"], None) == binding.DLLM_E_INVAL, bad
    need = lib.dllm_op_attn_kv4_workspace(c, 1, 1, 1, 1 << 20, 2)
    assert need > 0
    assert lib.dllm_op_attn_kv4(c, P, 128, 64, P, 128, 64, None, P, P, 1, 1, 1, 1 << 20, 2, P, 1, 0, 0.125, P, need - 1,
                                None) == binding.DLLM_E_INVAL
    # no request, or none with a query
    assert lib.dllm_op_attn_kv4(c, None, 0, 0, None, 0, 0, None, None, None, 0, 0, 0, 0, 2, None, 0, 0, 1.0, None, 0, None) == 0
    assert lib.dllm_op_attn_kv4_workspace(c, 3, 0, 0, 64, 2) == 0


def test_torch_wrappers_refuse_cpu_tensors():
    torch = pytest.importorskip("torch")
    from masked_block_diffusion_b200 import KVCache4, rope
    x = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError):
        rope(x, torch.zeros(2, dtype=torch.int32), Rope(64))
    with pytest.raises(ValueError):
        rope(x[0], torch.zeros(3, dtype=torch.int32), Rope(64))
    with pytest.raises(ValueError):
        KVCache4(4, 32, 1, 64, device="cpu")
    for bad in (dict(page=24), dict(head_dim=96), dict(n_pages=0)):
        with pytest.raises(ValueError):
            KVCache4(**{**dict(n_pages=2, page=32, n_kv_heads=1, head_dim=64, device="cpu"), **bad})
    assert ctypes.sizeof(binding.dllm_rope) == 8 + 8 + 8 * binding.DLLM_ROPE_MAX_PAIRS
