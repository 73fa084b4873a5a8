"""Rotary positions and the paged 4-bit KV cache on the GPU against plain 64-bit definitions."""

import numpy as np
import pytest
import torch

from masked_block_diffusion_b200 import DllmError, KVCache4, Rope, binding, build, rope
from oracle import kv4 as ref

pytestmark = pytest.mark.gpu

HALF_BF16, HALF_F32, HALF_F16 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -11


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_all()
    binding.load()


def i32(v):
    return torch.tensor(np.asarray(v, np.int32), device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


# ---------------------------------------------------------------- rope


def rope_bound(x, pos, y, out, rotary, layout, **scaling):
    """Elementwise bound of |y - exact|: cos and sin off by half a step, two products and a sum rounded (and the
    two errors' products), then the output's rounding. |angle error| < 2^-50 turns * 2^20 positions is far below."""
    f, m = ref.rope_frequencies(rotary, **scaling)
    i = np.arange(rotary // 2)
    p, q = (i, i + rotary // 2) if layout == "half" else (2 * i, 2 * i + 1)
    size = np.zeros_like(x)
    size[..., p] = size[..., q] = m * (np.abs(x[..., p]) + np.abs(x[..., q]))
    return 4 * HALF_F32 * size + (HALF_BF16 if out == torch.bfloat16 else 0) * np.abs(y) * 1.0001 + 1e-37


@pytest.mark.parametrize("T,H,d,rotary", [(1, 1, 64, 64), (3, 5, 176, 176), (70, 2, 176, 60), (17, 3, 128, 64), (5, 1, 10, 6),
                                          (513, 4, 64, 32), (2, 33, 200, 16), (1, 16, 256, 256), (4, 2, 66, 66)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tin,tout", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16),
                                      (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16)])
def test_rope_matches_the_definition(T, H, d, rotary, layout, tin, tout):
    rng = np.random.default_rng(T * 1000 + d + rotary)
    x = torch.tensor(rng.normal(size=(T, H, d)), device="cuda").to(tin)
    pos = rng.integers(0, 1 << 20, T)
    got = rope(x, i32(pos), Rope(rotary, layout), out_dtype=tout)
    want = ref.rotate(f64(x), pos, rotary, layout)
    assert got.dtype == tout and got.shape == x.shape
    assert np.all(np.abs(f64(got) - want) <= rope_bound(f64(x), pos, want, tout, rotary, layout))
    assert torch.equal(got[..., rotary:], x[..., rotary:].to(tout))


@pytest.mark.parametrize("scaling,factor", [("linear", 4.0), ("ntk", 8.0), ("yarn", 32.0)])
def test_rope_scaled_for_long_contexts(scaling, factor):
    rng = np.random.default_rng(5)
    x = torch.tensor(rng.normal(size=(200, 2, 64)), device="cuda").float()
    pos = rng.integers(0, 2 ** 31 - 1, 200)
    pos[:3] = [0, 1, 2 ** 31 - 1]
    args = dict(scaling=scaling, factor=factor, original_ctx=4096)
    got = f64(rope(x, i32(pos), Rope(64, "half", **args)))
    want = ref.rotate(f64(x), pos, 64, **args)
    # at 2^31 positions the 64-bit angle itself (a product of relative error 2^-53, up to 2^31 radians) is off by 2^-22
    bound = rope_bound(f64(x), pos, want, torch.float32, 64, "half", **args) + 2 * 2.0 ** -21 * np.abs(f64(x)).max()
    assert np.all(np.abs(got - want) <= bound)
    near = pos < 2 ** 20
    assert near.sum() >= 2


def test_rope_negative_positions_turn_back():
    x = torch.randn(4, 2, 64, device="cuda")
    plan = Rope(64)
    a = rope(x, i32([5, 6, 7, 8]), plan)
    b = rope(x, i32([-5, -6, -7, -8]), plan, transposed=True)
    assert torch.equal(a, b)


def test_rope_strided_in_place_and_misaligned():
    torch.manual_seed(0)
    plan = Rope(48, "half")
    pos = i32(np.arange(7) * 1000)
    wide = torch.randn(7, 9, 80, device="cuda")
    want = rope(wide[:, 2:6, 5:69].contiguous(), pos, plan)
    sliced = wide.clone()
    out = rope(sliced[:, 2:6, 5:69], pos, plan)                      # rows that start anywhere: the scalar path
    assert torch.equal(out, want)
    rope(sliced[:, 2:6, 5:69], pos, plan, out=sliced[:, 2:6, 5:69])  # in place, between other data
    assert torch.equal(sliced[:, 2:6, 5:69], want)
    keep = torch.ones_like(wide, dtype=torch.bool)
    keep[:, 2:6, 5:69] = False
    assert torch.equal(sliced[keep], wide[keep])
    into = torch.zeros(7, 4, 96, dtype=torch.bfloat16, device="cuda")
    rope(wide[:, 2:6, 5:69], pos, plan, out=into[..., 16:80])
    assert torch.equal(into[..., 16:80], want.bfloat16()) and not into[..., :16].any() and not into[..., 80:].any()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_transposed_is_the_gradient(layout):
    """Against the formula's gradient, and against differences of the map itself (it is linear)."""
    rng = np.random.default_rng(9)
    args = dict(scaling="yarn", factor=8.0, original_ctx=64)
    plan = Rope(32, layout, **args)
    x, dy = (torch.tensor(rng.normal(size=(6, 2, 64)), device="cuda").float() for _ in range(2))
    pos = rng.integers(0, 500, 6)
    dx = rope(dy, i32(pos), plan, transposed=True)
    want = ref.rotate(f64(dy), pos, 32, layout, transposed=True, **args)
    assert np.all(np.abs(f64(dx) - want) <= rope_bound(f64(dy), pos, want, torch.float32, 32, layout, **args))
    e = torch.randn_like(x)
    change = f64(rope(x + e, i32(pos), plan)) - f64(rope(x - e, i32(pos), plan))
    lhs, rhs = (change * f64(dy)).sum(), 2 * (f64(e) * f64(dx)).sum()
    # every term carries a few fp32 roundings of values below 8 in size
    assert abs(lhs - rhs) <= 8 * 8 * 8 * HALF_F32 * x.numel()


def test_rope_empty_and_refusals():
    plan = Rope(64)
    x = torch.randn(4, 2, 64, device="cuda")
    pos = i32(np.arange(4))
    assert rope(x[:0], pos[:0], plan).shape == (0, 2, 64)
    for bad in (lambda: rope(x, pos[:3], plan), lambda: rope(x, pos.long(), plan), lambda: rope(x.half(), pos, plan),
                lambda: rope(x, pos.cpu(), plan), lambda: rope(x.transpose(1, 2), pos, plan),
                lambda: rope(x, pos, plan, out=torch.empty(4, 2, 32, device="cuda")),
                lambda: rope(x, pos, plan, out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(DllmError):
        rope(x, pos, Rope(128))
    with pytest.raises(RuntimeError):
        rope(x.requires_grad_(), pos, plan)


# ---------------------------------------------------------------- append and read


def fresh(n_pages, page, hk, d, fill=0xFF):
    """A cache whose every byte is garbage: scale bytes 0xFF would be NaN as fp16."""
    c = KVCache4(n_pages, page, hk, d)
    c.codes.fill_(fill)
    c.scales.fill_(fill)
    return c


def tables(rng, lengths, page, spare=2):
    """A table over pages in random order; entries that no position uses are no page at all."""
    per = [-(-n // page) for n in lengths]
    total = sum(per) + spare
    order = rng.permutation(total)
    t = np.full((len(lengths), max(1, max(per))), -7, np.int32)
    at = 0
    for b, n in enumerate(per):
        t[b, :n] = order[at:at + n]
        at += n
    return t, total


@pytest.mark.parametrize("d,hk,page,tin", [(64, 4, 16, torch.float32), (176, 8, 64, torch.float32), (176, 1, 32, torch.bfloat16),
                                           (128, 2, 256, torch.bfloat16), (64, 3, 128, torch.bfloat16)])
@pytest.mark.parametrize("aligned", [True, False])
def test_append_stores_the_defined_bytes(d, hk, page, tin, aligned):
    rng = np.random.default_rng(d + hk + page)
    lengths = [1, page, 2 * page + 5, 37]
    table, total = tables(rng, lengths, page)
    T = sum(lengths)
    x = rng.normal(size=(2, T, hk, d)) * np.exp(2 * rng.normal(size=(2, T, hk, 1)))
    x[0, 0, 0, :16] = 0.0
    x[0, 1, 0, 3] = 1e30
    x[1, 2, 0, 5] = np.nan
    x[1, 3, 0, 5] = -np.inf
    x[1, 4, 0, :16] = np.arange(16) * 2.0 ** -17            # the smallest scales
    x[1, 5, 0, :16] = np.arange(16) * 2.0 ** -22
    x[0, 6, 0, :16] = 7.0 * ref.scale_values()[100]         # exactly seven scales
    x[0, 7, 0, :16] = ref.scale_values()[100] * (np.arange(16) - 6.5)   # ties between codes
    x[0, 7, 0, 15] = 7.0 * ref.scale_values()[100]
    pad = 0 if aligned else 3
    buf = torch.zeros((2, T, hk, d + 2 * pad), device="cuda", dtype=tin)
    kv = buf[..., pad:pad + d]
    kv.copy_(torch.tensor(x))
    req = np.repeat(np.arange(4), lengths)
    pos = np.concatenate([np.arange(n) for n in lengths])
    order = rng.permutation(T)                              # tokens in any order
    c = fresh(total, page, hk, d)
    c.append(kv[0][order] if aligned else kv[0], kv[1][order] if aligned else kv[1], i32(req[order] if aligned else req),
             i32(pos[order] if aligned else pos), i32(table))
    codes, byte = ref.quantise(f64(kv))
    want = ref.pack(codes)
    pages = table[req, pos // page]
    for part in (0, 1):
        assert np.array_equal(c.codes.cpu().numpy()[pages, part, :, pos % page], want[part])
        assert np.array_equal(c.scales.cpu().numpy()[pages, part, :, pos % page], byte[part])
    # everything else is as it was
    used = np.zeros((total, page), bool)
    used[pages, pos % page] = True
    assert (c.codes.cpu().numpy().transpose(0, 3, 1, 2, 4)[~used] == 0xFF).all()
    assert (c.scales.cpu().numpy().transpose(0, 3, 1, 2, 4)[~used] == 0xFF).all()
    k, v = c.read(i32(req), i32(pos), i32(table))
    held = ref.unpack(want, byte)
    assert np.array_equal(f64(k), held[0]) and np.array_equal(f64(v), held[1])


@pytest.mark.parametrize("tin", [torch.float32, torch.bfloat16])
def test_append_at_every_scale(tin):
    """Values at, just above and just below the ties between codes, and largest values just above and below
    what a scale holds, for every scale: the nearest code of the exact quotient."""
    s = ref.scale_values()[1:ref.MAX_SCALE_BYTE + 1].astype(np.float32)
    ties = np.append(np.arange(-7, 8) + 0.5, 7.0).astype(np.float32)[None] * s[:, None]    
    ties[:, 14] = 0.0                                                # in place of 7.5, which no group holds
    up, down = np.nextafter(ties, np.float32(np.inf)), np.nextafter(ties, np.float32(-np.inf))
    up[:, 15] = down[:, 15] = ties[:, 15]
    over = down.copy()
    over[:, 15] = np.nextafter(ties[:, 15], np.float32(np.inf))       # the next scale is due (the last one saturates)
    k = np.stack([ties, up, down, over], 1).reshape(-1, 1, 64)
    rng = np.random.default_rng(3)
    v = (rng.uniform(-7, 7, (len(s), 4, 16)) * s[:, None, None]).astype(np.float32)
    v[:, 0, 0] = np.nextafter(7 * s, np.float32(0))
    v = v.reshape(-1, 1, 64)
    kv = torch.tensor(np.stack([k, v]), device="cuda").to(tin)
    n = len(s)
    c = fresh(-(-n // 16), 16, 1, 64)
    table = np.arange(c.n_pages)[None]
    pos = np.arange(n)
    c.append(kv[0], kv[1], i32(np.zeros(n)), i32(pos), i32(table))
    codes, byte = ref.quantise(f64(kv))
    want = ref.pack(codes)
    for part in (0, 1):
        assert np.array_equal(c.scales.cpu().numpy()[pos // 16, part, :, pos % 16], byte[part])
        assert np.array_equal(c.codes.cpu().numpy()[pos // 16, part, :, pos % 16], want[part])


@pytest.mark.parametrize("layout,rotary,scaling", [("half", 176, {}), ("interleaved", 64, {}), ("half", 60, {}),
                                                   ("interleaved", 6, dict(scaling="yarn", factor=8.0, original_ctx=512))])
@pytest.mark.parametrize("tin", [torch.float32, torch.bfloat16])
def test_append_rotates_on_the_way(layout, rotary, scaling, tin):
    """The cache holds what rope and a plain append hold, bit for bit, and the nearest values of the exact rotation."""
    rng = np.random.default_rng(rotary)
    d, hk, h, page, T = 176, 2, 4, 32, 61
    table, total = tables(rng, [200], page)
    qkv = torch.tensor(rng.normal(size=(T, h + 2 * hk, d)), device="cuda").to(tin)   # a fused projection's slices
    k, v = qkv[:, h:h + hk], qkv[:, h + hk:]
    pos = rng.permutation(200)[:T]
    rope_pos = pos + 100000
    plan = Rope(rotary, layout, **scaling)
    one, two, req = fresh(total, page, hk, d), fresh(total, page, hk, d), i32(np.zeros(T))
    one.append(k, v, req, i32(pos), i32(table), rope=plan, rope_pos=i32(rope_pos))
    two.append(rope(k, i32(rope_pos), plan, out_dtype=torch.float32), v.float(), req, i32(pos), i32(table))
    assert torch.equal(one.codes, two.codes) and torch.equal(one.scales, two.scales)
    held = f64(one.read(req, i32(pos), i32(table))[0])
    want = ref.rotate(f64(k), rope_pos, rotary, layout, **scaling)
    pages = table[0, pos // page]
    scale = np.repeat(ref.scale_values()[one.scales.cpu().numpy()[pages, 0, :, pos % page]], 16, -1)
    off = rope_bound(f64(k), rope_pos, want, torch.float32, rotary, layout, **scaling)
    assert np.all(np.abs(held - want) <= scale / 2 * (1 + 2.0 ** -20) + off)
    one.append(k, v, req, i32(pos), i32(table), rope=plan)           # written anew, at the cache's own positions
    two.append(k, v, req, i32(pos), i32(table), rope=plan, rope_pos=i32(pos))
    assert torch.equal(one.codes, two.codes) and torch.equal(one.scales, two.scales)


def test_append_and_read_skip_padding_and_what_does_not_exist():
    d, hk, page = 64, 2, 16
    c = fresh(4, page, hk, d)
    table = i32([[1, 3, 99], [2, -5, 0]])                            # 99 and -5 are no pages
    req = [0, -1, 0, 1, 1, 2, 0, 0, -2 ** 31, 0]
    pos = [0, 5, 33, 17, 3, 0, -1, 48, 0, 2 ** 31 - 1]
    good = [0, 4]
    T = len(req)
    x = torch.randn(2, T, hk, d, device="cuda")
    x[:, 1] = float("nan")                                           # padding holds anything
    before = c.codes.clone(), c.scales.clone()
    c.append(x[0], x[1], i32(req), i32(pos), table, rope=Rope(64))
    changed = (c.scales != before[1]).any(-1).any(1).any(1).nonzero().cpu().tolist()   # (page, offset)
    assert changed == [[1, 0], [2, 3]]
    k = torch.full((T, hk, d), 5.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    c.read(i32(req), i32(pos), table, k_out=k, v_out=v)
    for out in (k, v):
        for t in range(T):
            if req[t] < 0:
                assert (out[t] == 5.0).all()
            elif t in good:
                assert torch.isfinite(out[t]).all() and not (out[t] == 5.0).all()
            else:
                assert torch.isnan(out[t]).all(), t
    made, _ = c.read(i32(req), i32(pos), table)
    assert not made[1].any()


def test_every_scale_byte_and_code_reads_back():
    c = KVCache4(256, 16, 1, 64)
    c.codes.copy_(torch.randint(0, 256, c.codes.shape, dtype=torch.uint8, device="cuda"))
    byte = torch.arange(256, device="cuda").to(torch.uint8) % 0xF8       # beyond are infinities and NaN
    c.scales.copy_(byte[:, None, None, None, None].expand_as(c.scales))
    req = np.repeat(np.arange(256), 16)
    pos = np.tile(np.arange(16), 256)
    k, v = c.read(i32(req), i32(pos), i32(np.arange(256)[:, None]))
    for part, got in ((0, k), (1, v)):
        want = ref.unpack(c.codes.cpu().numpy()[req, part, :, pos], c.scales.cpu().numpy()[req, part, :, pos])
        assert np.array_equal(f64(got), want)


# ---------------------------------------------------------------- attention


def filled(rng, lengths, page, hk, d, peak=1.0):
    """A cache of known values: the arrays, the table and each request's (k, v) in 64 bits. Garbage everywhere else."""
    table, total = tables(rng, lengths, page)
    codes = np.full((total, 2, hk, page, d // 2), 0xFF, np.uint8)
    scales = np.full((total, 2, hk, page, d // 16), 0xFF, np.uint8)
    held = []
    for b, n in enumerate(lengths):
        x = rng.normal(size=(2, n, hk, d)) * np.exp(0.5 * rng.normal(size=(2, n, hk, 1)))
        x[0] *= peak
        u, byte = ref.quantise(x)
        p = np.arange(n)
        codes[table[b, p // page], :, :, p % page] = ref.pack(u).transpose(1, 0, 2, 3)
        scales[table[b, p // page], :, :, p % page] = byte.transpose(1, 0, 2, 3)
        held.append(ref.unpack(ref.pack(u), byte))
    cache = KVCache4.from_tensors(torch.tensor(codes, device="cuda"), torch.tensor(scales, device="cuda"))
    return cache, table, held


def check_attention(got, lse, q, held, queries, keys, causal, scale):
    """Elementwise bounds. A score is a sum of d products in fp32: off by at most e = (d + 4) 2^-23 sum|q k| scale (each
    step of the sum truncated at worst) plus its scaling's rounding. A weight is then off by a factor e^(2 e), by half
    an fp16 step and by 2^-20 for exp2 and the sums, or by 2^-30 of the largest where it is tiny; the result is rounded
    to bf16."""
    t = 0
    for (k, v), n, m in zip(held, queries, keys):
        limits = np.full(n, m) if not causal else np.arange(n) + m - n + 1
        want, want_lse, mass, size = ref.attend(f64(q[t:t + n]), k[:m], v[:m], scale, limits)
        o, z = f64(got[t:t + n]), f64(lse[t:t + n])
        e = (q.shape[-1] + 4) * 2.0 ** -23 * size + 2.0 ** -22 * np.abs(np.where(np.isinf(want_lse), 0, want_lse))
        weight = (2.02 * e + 1.01 * HALF_F16 + 2.0 ** -20)[..., None]
        tiny = m * 2.0 ** -30 * (np.abs(v[:m]).max() if m else 0.0)
        bound = HALF_BF16 * np.abs(want) * 1.01 + 1.01 * weight * mass + tiny + 1e-37
        assert np.all(np.abs(o - want) <= bound), (np.abs(o - want) / bound).max()
        seen = limits > 0
        assert np.all(z[~seen] == -np.inf) and np.all(o[~seen] == 0)
        assert np.all(np.abs(z[seen] - want_lse[seen]) <= (e + 2.0 ** -20)[seen])
        t += n


def attend_case(d, h, hk, page, queries, keys, causal, seed, peak=1.0, lengths=None, scale=None):
    rng = np.random.default_rng(seed)
    cache, table, held = filled(rng, lengths or keys, page, hk, d, peak)
    T = sum(queries)
    q = torch.tensor(2.0 * rng.normal(size=(T, h, d)), device="cuda").bfloat16()
    starts = np.concatenate([[0], np.cumsum(queries)])
    out, lse = cache.attend(q, i32(starts), i32(keys), i32(table), max_q=max(queries), max_kv=max(keys), causal=causal,
                            return_lse=True, scale=scale)
    check_attention(out, lse, q, held, queries, keys, causal, d ** -0.5 if scale is None else scale)
    return cache, table, held, q, out, lse


@pytest.mark.parametrize("d,h,hk,page", [(64, 4, 4, 16), (64, 16, 4, 32), (128, 6, 2, 64), (128, 8, 1, 16), (176, 16, 8, 64),
                                         (176, 3, 1, 256), (64, 40, 2, 128)])
def test_attention_of_single_tokens(d, h, hk, page):
    attend_case(d, h, hk, page, [1] * 8, [1, 2, 15, 16, 17, 63, 300, 129], True, seed=d + h)


@pytest.mark.parametrize("d,h,hk,page", [(64, 4, 2, 16), (176, 16, 8, 64), (128, 12, 4, 32)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_of_few_tokens_ragged_with_empty_requests(d, h, hk, page, causal):
    attend_case(d, h, hk, page, [3, 0, 8, 5, 1, 7], [200, 40, 4, 0, 77, 7], causal, seed=d + 1)


@pytest.mark.parametrize("d,h,hk,page", [(64, 4, 2, 32), (176, 4, 2, 64), (128, 4, 1, 16)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_of_canvases_and_prompt_pieces(d, h, hk, page, causal):
    attend_case(d, h, hk, page, [33, 1, 130, 64], [333, 1, 130, 20], causal, seed=d + 2)


def test_attention_groups_that_do_not_divide_a_tile():
    attend_case(64, 15, 3, 32, [70, 9], [150, 333], True, seed=11)
    attend_case(176, 7, 1, 64, [40], [90], False, seed=12)


@pytest.mark.parametrize("d,h,hk", [(176, 16, 8), (64, 16, 4), (128, 2, 1)])
def test_attention_split_over_a_long_cache(d, h, hk):
    attend_case(d, h, hk, 64, [1, 2], [9001, 4097], True, seed=d + 4)


def test_attention_split_canvas():
    attend_case(176, 4, 2, 64, [40, 17], [3001, 1290], False, seed=21)


@pytest.mark.parametrize("d", [64, 128, 176])
@pytest.mark.parametrize("queries", [8, 9])
def test_attention_around_the_kernels_border(d, queries):
    """32 and 36 rows per KV head, of which some requests fill one tile and a part of another, or none."""
    attend_case(d, 8, 2, 32, [queries, 5, 3, 0, 1, queries], [700, 1500, 3, 9, 40, 2], True, seed=31)
    attend_case(d, 8, 2, 32, [queries, 4, queries], [90, 2600, 0], False, seed=32)


@pytest.mark.parametrize("d,keys", [(64, 10000), (128, 5000), (176, 7000)])
def test_attention_of_one_tile_in_many_splits(d, keys):
    """One KV head and few rows: more splits than a warp has lanes."""
    attend_case(d, 2, 1, 64, [20], [keys], True, seed=22)


@pytest.mark.parametrize("d,h,hk", [(64, 8, 2), (128, 2, 2), (176, 4, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_of_many_tiles_in_equal_shares(d, h, hk, causal):
    """Tiles that start and end anywhere in a block's share: ragged requests, some without queries or keys."""
    rng = np.random.default_rng(d + causal)
    queries = [int(n) for n in rng.integers(0, 150, 40)]
    keys = [int(n) for n in rng.integers(0, 700, 40)]
    queries[:6], keys[:6] = [150, 0, 130, 64, 129, 1], [700, 300, 0, 64, 96, 1]
    queries[-3:], keys[-3:] = [140, 0, 0], [0, 5, 0]
    attend_case(d, h, hk, 32, queries, keys, causal, seed=25)


@pytest.mark.parametrize("d,keys,n", [(64, 9000, 1), (176, 5000, 2), (128, 40, 1)])
def test_attention_of_one_tile_among_many_empty_requests(d, keys, n):
    """The batch is sized for more requests than there are: one tile's keys over all blocks, or a block per tile."""
    B = 90
    queries, lens = [0] * B, [0] * B
    for i in range(n):
        queries[60 * i + 5], lens[60 * i + 5] = 20, keys - 700 * i
    attend_case(d, 2, 1, 64, queries, lens, True, seed=26)


@pytest.mark.parametrize("queries", [1, 8, 40])
def test_attention_with_the_widest_bounds(queries):
    """Bounds far above the lengths: the work is shared out in coarser units, and splits are mostly empty."""
    rng = np.random.default_rng(30)
    B, h, hk, d = 100, 8, 4, 64
    keys = [int(n) for n in rng.integers(1, 300, B)]
    keys[3], keys[70] = 2000, 1500
    cache, table, held = filled(rng, keys, 32, hk, d)
    q = torch.tensor(rng.normal(size=(B * queries, h, d)), device="cuda").bfloat16()
    out, lse = cache.attend(q, i32(np.arange(B + 1) * queries), i32(keys), i32(table), max_q=queries, max_kv=(1 << 29) - 1,
                            causal=False, return_lse=True)
    check_attention(out, lse, q, held, [queries] * B, keys, False, d ** -0.5)


def test_attention_of_requests_far_apart_in_a_padded_batch():
    B = 300
    queries, lens = [0] * B, [3] * B
    for i, n, m in ((0, 40, 900), (31, 1, 1), (32, 70, 2500), (170, 33, 700), (299, 150, 1200)):
        queries[i], lens[i] = n, m
    attend_case(176, 4, 2, 32, queries, lens, True, seed=28)
    attend_case(64, 4, 2, 32, queries, lens, False, seed=29)


def test_attention_of_many_tiles_answers_bad_requests_with_nan():
    rng = np.random.default_rng(27)
    B, queries, keys, page, h, hk, d = 40, 70, 300, 32, 4, 2, 64
    cache, table, held = filled(rng, [keys] * B, page, hk, d)
    q = torch.tensor(rng.normal(size=(B * queries, h, d)), device="cuda").bfloat16()
    starts = np.arange(B + 1) * queries
    lens = np.full(B, keys)
    lens[[0, 7, 39]] = [-1, keys + page + 5, keys + 1000]
    table[12, 3] = cache.n_pages
    table[30, (keys - 1) // page] = -1
    out, lse = cache.attend(q, i32(starts), i32(lens), i32(table), max_q=queries, max_kv=keys + 500, causal=True, return_lse=True)
    for b in range(B):
        rows = slice(b * queries, (b + 1) * queries)
        if b in (0, 7, 39):
            assert torch.isnan(out[rows]).all() and torch.isnan(lse[rows]).all(), b
        elif b in (12, 30):                                           # the rows that see the page
            lost = torch.isnan(lse[rows]).all(-1).cpu().numpy()
            assert lost[np.arange(queries) + keys - queries >= 32 * (3 if b == 12 else (keys - 1) // page)].all()
            assert torch.equal(torch.isnan(out[rows]).all(-1), torch.isnan(lse[rows]))
        else:
            check_attention(out[rows], lse[rows], q[rows], [held[b]], [queries], [keys], True, d ** -0.5)


@pytest.mark.parametrize("queries", [1, 30])
def test_attention_without_a_key_and_in_place(queries):
    cache, table, held = filled(np.random.default_rng(23), [70], 16, 2, 64)
    q = torch.randn(queries, 8, 64, device="cuda").bfloat16()
    out, lse = cache.attend(q, i32([0, queries]), i32([0]), i32(table), max_q=queries, max_kv=0, return_lse=True)
    assert not out.any() and (lse == -np.inf).all()
    want = cache.attend(q, i32([0, queries]), i32([70]), i32(table), max_q=queries, max_kv=70)
    assert cache.attend(q, i32([0, queries]), i32([70]), i32(table), max_q=queries, max_kv=70, out=q) is q
    assert torch.equal(q, want)


def test_attention_with_scores_that_climb_and_with_one_that_stands_out():
    """Rising scores move the softmax's reference block after block; then one key takes all the weight."""
    rng = np.random.default_rng(6)
    d, page, n = 64, 32, 400
    cache, table, held = filled(rng, [n], page, 1, d)
    k = np.zeros((n, 1, d))
    k[:, 0, 0] = np.linspace(-20, 20, n)
    k[200, 0, 0] = 60.0
    u, byte = ref.quantise(k)
    p = np.arange(n)
    codes, scales = cache.codes.cpu().numpy(), cache.scales.cpu().numpy()
    codes[table[0, p // page], 0, :, p % page] = ref.pack(u)
    scales[table[0, p // page], 0, :, p % page] = byte
    cache.codes.copy_(torch.tensor(codes))
    cache.scales.copy_(torch.tensor(scales))
    held[0][0] = ref.unpack(ref.pack(u), byte)
    for queries in (2, 40):
        q = torch.zeros((queries, 2, d), device="cuda", dtype=torch.bfloat16)
        q[:, 0, 0] = 30.0
        q[:, 1, 0] = -30.0
        for m in (n, 190):
            out, lse = cache.attend(q, i32([0, queries]), i32([m]), i32(table), max_q=queries, max_kv=n, return_lse=True, scale=1.0)
            check_attention(out, lse, q, held, [queries], [m], False, 1.0)


@pytest.mark.parametrize("queries", [1, 40])
def test_attention_strided_and_rows_of_no_request_stay(queries):
    rng = np.random.default_rng(13)
    d, h, hk, page = 64, 4, 2, 32
    cache, table, held = filled(rng, [90, 50], page, hk, d)
    T = 2 * queries + 9
    big = torch.randn(T, 3 * h, d, device="cuda").bfloat16()
    q = big[:, h:2 * h]
    starts = [4, 4 + queries, 4 + 2 * queries]                        # rows before and behind belong to nobody
    room = torch.full((T, h, 2 * d), 3.0, dtype=torch.bfloat16, device="cuda")
    out = room[..., d // 2:d // 2 + d]
    same, lse = cache.attend(q, i32(starts), i32([90, 50]), i32(table), max_q=queries, max_kv=90, out=out, return_lse=True)
    assert same is out
    check_attention(out[4:], lse[4:], q[4:], held, [queries, queries], [90, 50], False, d ** -0.5)
    assert (room[:4] == 3.0).all() and (room[4 + 2 * queries:] == 3.0).all()
    assert (room[..., :d // 2] == 3.0).all() and (room[..., d // 2 + d:] == 3.0).all()


@pytest.mark.parametrize("queries,keys", [(1, 100), (1, 5000), (40, 100), (40, 3000)])
def test_attention_answers_bad_lengths_and_pages_with_nan(queries, keys):
    rng = np.random.default_rng(14)
    d, h, hk, page = 64, 4, 2, 64
    B = 6
    cache, table, held = filled(rng, [keys] * B, page, hk, d)
    starts = np.arange(B + 1) * queries
    q = torch.tensor(rng.normal(size=(B * queries, h, d)), device="cuda").bfloat16()
    lens = np.array([keys, -1, table.shape[1] * page + 1, keys, keys, keys])
    table[3, 0] = cache.n_pages                                       # no page
    table[4, (keys - 1) // page] = -1
    out, lse = cache.attend(q, i32(starts), i32(lens), i32(table), max_q=queries, max_kv=table.shape[1] * page + 64,
                            return_lse=True)
    for b in range(B):
        rows = slice(b * queries, (b + 1) * queries)
        if b in (0, 5):
            check_attention(out[rows], lse[rows], q[rows], [held[b]], [queries], [keys], False, d ** -0.5)
        else:
            assert torch.isnan(out[rows]).all() and torch.isnan(lse[rows]).all(), b
    # a request longer than max_kv or max_q says; row ranges that are none are skipped
    out, lse = cache.attend(q, i32(starts), i32([keys] * B), i32(table), max_q=queries, max_kv=keys - 1, return_lse=True)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    if queries > 1:
        out, lse = cache.attend(q, i32(starts), i32([keys] * B), i32(table), max_q=queries - 1, max_kv=keys, return_lse=True)
        assert torch.isnan(out).all() and torch.isnan(lse).all()
    out = torch.full_like(q, 2.0)
    bad = np.array([-3, queries, 0, B * queries + 1, 5 * queries, 6 * queries, 6 * queries])
    cache.attend(q, i32(bad), i32([keys] * B), i32(table), max_q=queries, max_kv=keys, out=out)
    assert (out[:5 * queries] == 2.0).all() and torch.isnan(out[5 * queries:]).all()   # the one left has a bad page


@pytest.mark.parametrize("queries", [2, 40])
def test_attention_nan_and_infinite_queries_stay_in_their_rows(queries):
    rng = np.random.default_rng(15)
    cache, table, held = filled(rng, [100], 32, 1, 64)
    q = torch.tensor(rng.normal(size=(queries, 2, 64)), device="cuda").bfloat16()
    q[0, 1] = float("nan")
    q[1, 0, 3] = float("inf")
    out, lse = cache.attend(q, i32([0, queries]), i32([100]), i32(table), max_q=queries, max_kv=100, return_lse=True)
    bad = torch.zeros(queries, 2, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 0] = True
    assert torch.equal(torch.isnan(out).all(-1), bad) and torch.equal(torch.isnan(lse), bad)


def test_attention_pages_shared_by_requests():
    """Two requests over one prefix: the same pages in both rows."""
    rng = np.random.default_rng(16)
    cache, table, held = filled(rng, [128, 64], 32, 2, 64)
    table[1, :2] = table[0, :2]
    q = torch.tensor(rng.normal(size=(2, 4, 64)), device="cuda").bfloat16()
    q[1] = q[0]
    out = cache.attend(q, i32([0, 1, 2]), i32([64, 64]), i32(table), max_q=1, max_kv=64)
    assert torch.equal(out[0], out[1])


def test_results_do_not_change_from_call_to_call():
    for queries, keys in ((1, 6000), (64, 2000)):
        cache, table, held, q, out, lse = attend_case(64, 4, 2, 32, [queries], [keys], True, seed=17)
        for _ in range(3):
            o, z = cache.attend(q, i32([0, queries]), i32([keys]), i32(table), max_q=queries, max_kv=keys, causal=True,
                                return_lse=True)
            assert torch.equal(o, out) and torch.equal(z, lse)


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("d,h,hk", [(64, 16, 4), (176, 16, 8)])
def test_prompt_then_canvas_passes_then_tokens(d, h, hk):
    """As a program uses them: GEMM -> rotate and append -> attend, a prompt in two pieces, a canvas written anew
    in a second pass at the same positions, then single tokens; requests of different lengths."""
    rng = np.random.default_rng(31)
    page, width, canvas = 32, 256, 32
    prompts = [70, 45]
    cap = [n + canvas + 3 for n in prompts]
    table, total = tables(rng, cap, page)
    cache, tab = fresh(total, page, hk, d), i32(table)
    plan = Rope(d)
    rows = (h + 2 * hk) * d
    w = torch.tensor(rng.normal(size=(rows, width)) * width ** -0.5, device="cuda").bfloat16()
    held = [np.zeros((2, n, hk, d)) for n in cap]
    length = [0, 0]

    def step(new, causal):
        T = sum(new)
        x = torch.tensor(rng.normal(size=(T, width)), device="cuda").bfloat16()
        qkv = torch.empty((T, rows), device="cuda")
        binding.dllm_op_gemm_bf16(x.data_ptr(), w.data_ptr(), qkv.data_ptr(), T, rows, width,
                                  torch.cuda.current_stream().cuda_stream)
        qkv = qkv.view(T, h + 2 * hk, d)
        req = np.repeat([0, 1], new)
        pos = np.concatenate([length[b] + np.arange(new[b]) for b in (0, 1)])
        q = rope(qkv[:, :h], i32(pos), plan, out_dtype=torch.bfloat16)
        cache.append(qkv[:, h:h + hk], qkv[:, h + hk:], i32(req), i32(pos), tab, rope=plan)
        keys = [length[b] + new[b] for b in (0, 1)]
        out, lse = cache.attend(q, i32([0, new[0], T]), i32(keys), tab, max_q=max(new), max_kv=max(keys), causal=causal,
                                return_lse=True)
        got = np.stack([f64(t) for t in cache.read(i32(req), i32(pos), tab)])
        k64 = ref.rotate(f64(qkv[:, h:h + hk]), pos, d)
        top = np.repeat(np.abs(np.stack([k64, f64(qkv[:, h + hk:])])).reshape(2, T, hk, -1, 16).max(-1), 16, -1)
        # the scale is at most 9/8 of a seventh of the largest magnitude, and a value half a scale off
        assert np.all(np.abs(got - np.stack([k64, f64(qkv[:, h + hk:])])) <= top * (9 / 8 / 7 / 2 + 1e-5))
        for b in (0, 1):
            held[b][:, length[b]:keys[b]] = got[:, req == b]
        check_attention(out, lse, q, held, new, keys, causal, d ** -0.5)
        return keys

    length = step([40, 45], True)
    length = step([30, 0], True)
    step([canvas, canvas], False)                     # a pass over the canvas
    length = step([canvas, canvas], False)            # the next pass writes the same positions anew
    for _ in range(3):
        length = step([1, 1], True)


@pytest.mark.parametrize("queries", [1, 64])
def test_capture_replay_and_two_graphs(queries):
    """Captured calls read lengths and tables when they are replayed; two graphs with a workspace each may overlap."""
    rng = np.random.default_rng(32)
    d, h, hk, page, keys = 64, 8, 2, 32, 2500
    cache, table, held = filled(rng, [keys], page, hk, d)
    q = torch.tensor(rng.normal(size=(queries, h, d)), device="cuda").bfloat16()
    start, lens, tab = i32([0, queries]), i32([keys]), i32(table)
    graphs, outs = [], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(cache.attend(q, start, lens, tab, max_q=queries, max_kv=keys, causal=True, return_lse=True))
        graphs.append(g)
    for m in (keys, 700, 1):
        lens.fill_(m)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for out, lse in outs:
            check_attention(out, lse, q, held, [queries], [m], True, d ** -0.5)


def test_a_step_captured_in_a_graph_matches_the_eager_one():
    rng = np.random.default_rng(33)
    d, h, hk, page = 176, 16, 8, 64
    cache, table, _ = filled(rng, [200, 130], page, hk, d)
    tab, plan = i32(table), Rope(d)
    qkv = torch.tensor(rng.normal(size=(2, h + 2 * hk, d)), device="cuda").float()
    pos, req, lens, start = i32([199, 129]), i32([0, 1]), i32([200, 130]), i32([0, 1, 2])

    def step():
        q = rope(qkv[:, :h], pos, plan, out_dtype=torch.bfloat16)
        cache.append(qkv[:, h:h + hk], qkv[:, h + hk:], req, pos, tab, rope=plan)
        return cache.attend(q, start, lens, tab, max_q=1, max_kv=200, causal=True)

    eager = step().clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    cache.codes[table[0, 3], 0, :, 7] = 0x88                          # the replay writes position 199 again
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, eager)


def test_calls_on_another_stream_and_with_the_callers_workspace():
    rng = np.random.default_rng(34)
    d, h, hk, keys = 128, 8, 2, 4000
    cache, table, held = filled(rng, [keys], 64, hk, d)
    q = torch.tensor(rng.normal(size=(1, h, d)), device="cuda").bfloat16()
    start, lens, tab = i32([0, 1]), i32([keys]), i32(table)
    need = cache.workspace_bytes(1, 1, 1, keys, h)
    assert need > 0
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = cache.attend(q, start, lens, tab, max_q=1, max_kv=keys, return_lse=True, workspace=ws)
    s.synchronize()
    check_attention(out, lse, q, held, [1], [keys], False, d ** -0.5)
    assert (ws[need:] == 255).all()                                   # and nothing behind what was asked for
    with pytest.raises(DllmError):
        cache.attend(q, start, lens, tab, max_q=1, max_kv=keys, workspace=ws[:need - 16])
    with pytest.raises(ValueError):
        cache.attend(q, start, lens, tab, max_q=1, max_kv=keys, workspace=ws.cpu())


def test_torch_refusals():
    c = KVCache4(4, 32, 2, 64)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    start, lens, tab = i32([0, 3]), i32([10]), i32([[0]])
    k = torch.zeros(3, 2, 64, device="cuda")
    req, pos = i32([0, 0, 0]), i32([0, 1, 2])
    for bad in (lambda: c.attend(q.float(), start, lens, tab, 3, 10), lambda: c.attend(q[..., :32], start, lens, tab, 3, 10),
                lambda: c.attend(q, start[:1], lens, tab, 3, 10), lambda: c.attend(q, start, lens.long(), tab, 3, 10),
                lambda: c.attend(q, start, lens, tab[0], 3, 10), lambda: c.attend(q, start, lens, tab.expand(2, 1), 3, 10),
                lambda: c.attend(q, start, lens, i32([[0, 1], [2, 3]])[:, :1], 3, 10), lambda: c.attend(q, i32([0, 1, 3]), i32([5, 5]), tab, 3, 10),
                lambda: c.attend(q, start, lens, tab, 3, 10, out=torch.zeros_like(q, dtype=torch.float32)),
                lambda: c.append(k, k.bfloat16(), req, pos, tab), lambda: c.append(k[:, :1], k, req, pos, tab),
                lambda: c.append(k, k, req[:2], pos, tab), lambda: c.append(k, k, req, pos.float(), tab),
                lambda: c.read(req, pos, tab, k_out=k), lambda: c.read(req, pos[:1], tab),
                lambda: KVCache4.from_tensors(c.codes, c.scales[..., :2]), lambda: KVCache4.from_tensors(c.codes[1:, :, :1], c.scales)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: c.attend(q[:, :3], start, lens, tab, 3, 10),          # heads that do not divide
                lambda: c.attend(q, start, lens, tab, 4, 10),                 # more than T queries
                lambda: c.attend(q, start, lens, tab, 3, 10, scale=0.0)):
        with pytest.raises(DllmError):
            bad()
    assert c.attend(q[:0], i32([0, 0]), lens, tab, 0, 10).shape == (0, 4, 64)
    assert c.read(req[:0], pos[:0], tab)[0].shape == (0, 2, 64)
    c.append(k[:0], k[:0], req[:0], pos[:0], tab)


@pytest.mark.parametrize("d,queries", [(64, 1), (176, 1), (64, 40), (176, 256)])
def test_a_wait_that_runs_out_answers_nan_and_the_next_call_is_right(d, queries):
    """Waits limited to 1 ns, a first wait of up to 256 ns aside: rows are lost as a whole or right. How many are lost
    depends on how the blocks' roles happen to meet (many blocks at once, out of the L2 cache)."""
    from masked_block_diffusion_b200 import Denoiser
    from synth import WORKLOADS, blob_from_weights, gen_weights

    cfg = WORKLOADS["c1-tiny-dense"].model
    den = Denoiser(cfg, blob_from_weights(cfg, gen_weights(cfg)), max_ctx=256, max_batch=1)
    n, keys, page = 80, 3000, 64
    rng = np.random.default_rng(24)
    cache, table, held = filled(rng, [keys] * 4, page, 2, d)
    q = torch.tensor(2.0 * rng.normal(size=(n * queries, 4, d)), device="cuda").bfloat16()
    args = (q, i32(np.arange(n + 1) * queries), i32([keys] * n), i32(np.tile(table, (n // 4, 1))), queries, keys)
    out, lse = cache.attend(*args, return_lse=True)
    check_attention(out[:queries], lse[:queries], q, held, [queries], [keys], False, d ** -0.5)
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    try:
        binding.dllm_set_wait_limit(den.h, 1)
        try:
            for i in range(10):
                big.fill_(i)
                o, z = cache.attend(*args, return_lse=True)
                lost = torch.isnan(z)
                assert torch.equal(lost, torch.isnan(o).all(-1)) and torch.equal(lost, torch.isnan(o).any(-1))
                assert torch.equal(o[~lost], out[~lost]) and torch.equal(z[~lost], lse[~lost])
        finally:
            torch.cuda.synchronize()
            binding.dllm_set_wait_limit(den.h, 0)
        o, z = cache.attend(*args, return_lse=True)
        assert torch.equal(o, out) and torch.equal(z, lse)
    finally:
        den.close()
