"""Calls on rotary positions and the paged 4-bit KV cache that other tests do not make: which tensors are taken and
which are refused, on the GPU."""

import itertools

import numpy as np
import pytest
import torch

from masked_block_diffusion_b200 import DllmError, KVCache4, Rope, binding, build, rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_all()
    binding.load()


def i32(v):
    return torch.tensor(np.asarray(v, np.int32), device="cuda")


@pytest.mark.parametrize("T,H,d", [(2, 2, 4), (3, 4, 6), (5, 2, 2), (1, 3, 4), (3, 1, 4)])
def test_rope_takes_outputs_of_any_strides_whose_rows_are_apart(T, H, d):
    x, pos, plan = torch.randn(T, H, d, device="cuda"), i32(range(T)), Rope(2)
    want = rope(x, pos, plan)
    for tok, head in itertools.product(range(0, 14), repeat=2):
        room = torch.full((T * tok + H * head + d,), 7.0, device="cuda")
        out = room.as_strided((T, H, d), (tok, head, 1))
        cells = {t * tok + h * head + e for t in range(T) for h in range(H) for e in range(d)}
        if len(cells) < T * H * d:
            with pytest.raises(DllmError):
                rope(x, pos, plan, out=out)
            assert (room == 7.0).all()
        else:
            rope(x, pos, plan, out=out)
            assert torch.equal(out, want), (tok, head)


@pytest.mark.parametrize("queries", [1, 40])
def test_attend_refuses_an_expanded_output_and_takes_heads_first(queries):
    cache = KVCache4(4, 32, 2, 64)
    q = torch.randn(queries, 4, 64, device="cuda").bfloat16()
    args = (i32([0, queries]), i32([70]), i32([[2, 0, 1]]), queries, 70)
    want = cache.attend(q, *args)
    for shape in ((queries, 1, 64), (1, 4, 64)):
        if queries == 1 and shape[0] == 1:
            continue
        with pytest.raises(DllmError):
            cache.attend(q, *args, out=torch.zeros(shape, dtype=torch.bfloat16, device="cuda").expand(queries, 4, 64))
    turned = torch.zeros(4, queries, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    assert torch.equal(cache.attend(q, *args, out=turned), want)


@pytest.mark.parametrize("queries", [1, 40])
def test_slices_of_one_buffer_are_taken_and_shifted_views_are_not(queries):
    cache = KVCache4(4, 32, 2, 64)
    cache.codes.random_(0, 256)
    cache.scales.fill_(100)
    args = (i32([0, queries]), i32([70]), i32([[2, 0, 1]]), queries, 70)
    buf = torch.randn(queries, 12, 64, device="cuda").bfloat16()
    want = cache.attend(buf[:, 4:8].contiguous(), *args)
    assert torch.equal(cache.attend(buf[:, 4:8], *args, out=buf[:, 8:]), want)    # side by side
    assert torch.equal(cache.attend(buf[:, 4:8], *args, out=buf[:, 4:8]), want)   # in place
    flat = torch.randn((queries + 1) * 256, device="cuda").bfloat16()
    q, shifted = flat[:-256].view(queries, 4, 64), flat[64:64 - 256].view(queries, 4, 64)
    with pytest.raises(DllmError):
        cache.attend(q, *args, out=shifted)
    pos = i32(range(queries))
    with pytest.raises(DllmError):
        rope(q, pos, Rope(64), out=shifted)
    req, pos, table = i32([0] * 5), i32(range(5)), i32([[2, 0, 1]])
    both = torch.zeros(7, 2, 64, dtype=torch.bfloat16, device="cuda")
    for k, v in ((both[:5], both[:5]), (both[:5], both[2:])):
        with pytest.raises(DllmError):
            cache.read(req, pos, table, k_out=k, v_out=v)
    assert not both.any()
    pair = torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16, device="cuda")          # next to each other
    cache.read(req, pos, table, k_out=pair[0], v_out=pair[1])
    assert all(torch.equal(a, b) for a, b in zip(pair, cache.read(req, pos, table)))


def _dual(t):
    return torch.autograd.forward_ad.make_dual(t, torch.ones_like(t))


def test_dual_tensors_are_refused_and_plain_ones_within_their_level_are_not():
    cache, plan = KVCache4(4, 32, 2, 64), Rope(64)
    x, pos, req, table = torch.randn(3, 2, 64, device="cuda"), i32(range(3)), i32([0] * 3), i32([[2, 0, 1]])
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    args = (i32([0, 3]), i32([3]), table, 3, 3)
    held = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    with torch.autograd.forward_ad.dual_level(), torch.no_grad():
        for bad in (lambda: rope(_dual(x), pos, plan), lambda: rope(x, pos, plan, out=_dual(x.clone())),
                    lambda: cache.append(_dual(x), x, req, pos, table), lambda: cache.append(x, _dual(x), req, pos, table),
                    lambda: cache.read(req, pos, table, k_out=held[0], v_out=_dual(held[1])),
                    lambda: cache.attend(_dual(q), *args), lambda: cache.attend(q, *args, out=_dual(q.clone()))):
            with pytest.raises(RuntimeError, match="tangent"):
                bad()
        assert not cache.codes.any()
        # the way that the message names
        dual = _dual(x)
        y, dy = (rope(t, pos, plan) for t in torch.autograd.forward_ad.unpack_dual(dual))
        cache.append(x, x, req, pos, table)
        cache.read(req, pos, table)
        cache.attend(q, *args)
    assert torch.equal(y, rope(x, pos, plan)) and torch.equal(dy, rope(torch.ones_like(x), pos, plan))


def test_outputs_that_require_a_gradient_are_refused():
    """As torch refuses to write to them in place; without gradients being recorded both may."""
    cache, plan = KVCache4(4, 32, 2, 64), Rope(64)
    x, pos, req, table = torch.randn(3, 2, 64, device="cuda"), i32(range(3)), i32([0] * 3), i32([[2, 0, 1]])
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    args = (i32([0, 3]), i32([3]), table, 3, 3)
    leaf = [torch.full(t.shape, 5.0, dtype=t.dtype, device="cuda", requires_grad=True) for t in (x, q, x.bfloat16(), x.bfloat16())]
    plain = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    calls = (lambda: rope(x, pos, plan, out=leaf[0]), lambda: cache.attend(q, *args, out=leaf[1]),
             lambda: cache.read(req, pos, table, k_out=leaf[2], v_out=plain), lambda: cache.read(req, pos, table, k_out=plain, v_out=leaf[3]))
    for call in calls:
        with pytest.raises(RuntimeError, match="gradient"):
            call()
    assert all((t == 5.0).all() for t in leaf)
    with torch.no_grad():
        for call in calls:
            call()
    assert not any((t == 5.0).any() for t in leaf)


def test_a_backward_pass_notices_that_a_saved_tensor_was_written_to():
    cache, plan = KVCache4(4, 32, 2, 64), Rope(64)
    pos, req, table = i32(range(3)), i32([0] * 3), i32([[2, 0, 1]])
    args = (i32([0, 3]), i32([3]), table, 3, 3)
    spare = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    x, q = (torch.randn(3, h, 64, device="cuda").bfloat16() for h in (2, 4))
    for shape, write in ((x, lambda y: rope(x, pos, plan, out=y)), (x, lambda y: rope(y, pos, plan, out=y)),
                         (q, lambda y: cache.attend(q, *args, out=y)), (x, lambda y: cache.read(req, pos, table, k_out=y, v_out=spare)),
                         (x, lambda y: cache.read(req, pos, table, k_out=spare, v_out=y))):
        leaf = torch.randn_like(shape).requires_grad_()
        y = leaf.exp()                                               # its gradient is made of y itself
        write(y.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
    with torch.inference_mode():                                     # where nothing counts writes
        y = torch.empty_like(x)
        assert rope(x, pos, plan, out=y) is y
        cache.read(req, pos, table, k_out=y, v_out=torch.empty_like(y))


@pytest.mark.parametrize("columns", [0, 3])
def test_a_batch_of_no_requests_has_a_table_without_rows(columns):
    cache = KVCache4(4, 32, 2, 64)
    table = torch.zeros((0, columns), dtype=torch.int32, device="cuda")
    none = i32([])
    k = torch.zeros((0, 2, 64), device="cuda")
    cache.append(k, k, none, none, table, rope=Rope(64))
    assert all(t.shape == (0, 2, 64) for t in cache.read(none, none, table))
    for T, max_q, max_kv in ((0, 0, 0), (5, 2, 70)):
        q = torch.zeros((T, 4, 64), dtype=torch.bfloat16, device="cuda")
        out, lse = cache.attend(q, i32([0]), none, table, max_q, max_kv, return_lse=True, out=torch.full_like(q, 3.0))
        assert out.shape == q.shape and lse.shape == (T, 4) and (out == 3.0).all()
    x = torch.zeros((1, 2, 64), device="cuda")                        # with a token or a request a row is needed
    for bad in (lambda: cache.append(x, x, i32([0]), i32([0]), table), lambda: cache.read(i32([0]), i32([0]), table),
                lambda: cache.attend(torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda"), i32([0, 1]), i32([1]), table, 1, 1)):
        with pytest.raises(ValueError):
            bad()
