"""Calls on rotary positions and the paged 4-bit KV cache that are refused before anything is queued (no GPU)."""

import pytest

from masked_block_diffusion_b200 import Rope, binding, build

P = 1 << 24      # stands for a device address: a refused call never reads it


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build_dllm()
    return binding.load()


def call_rope(lib, T=4, H=2, d=64, tok=128, head=64, y=2 * P, x=P, x_type=0, y_type=0, x_tok=128, x_head=64):
    return lib.dllm_op_rope(Rope(2).c, x, x_type, x_tok, x_head, P, T, H, d, y, y_type, tok, head, 0, None)


def call_attend(lib, T=4, H=2, tok=128, head=64, out=2 * P, q=P, q_tok=128, q_head=64):
    c = binding.dllm_kv4(P, P, 8, 64, 2, 64)
    return lib.dllm_op_attn_kv4(c, q, q_tok, q_head, out, tok, head, None, P, P, 1, T, 1, 64, H, P, 1, 0, 0.125, None, 0, None)


@pytest.mark.parametrize("tok,head", [(0, 64), (128, 0), (0, 0), (64, 64), (120, 64), (128, 56), (-64, 64), (96, 192), (64, 96)])
def test_outputs_whose_rows_overlap_are_refused(lib, tok, head):
    assert call_rope(lib, tok=tok, head=head) == binding.DLLM_E_INVAL
    if tok % 8 == 0 and head % 8 == 0:
        assert call_attend(lib, tok=tok, head=head) == binding.DLLM_E_INVAL


def test_outputs_that_share_memory_with_an_input_are_refused(lib):
    n = 4 * 2 * 64
    for off in (4, 64 * 4, n * 4 - 4):                               # x fp32, y fp32, ahead and behind
        assert call_rope(lib, y=P + off) == binding.DLLM_E_INVAL
        assert call_rope(lib, x=P + off, y=P) == binding.DLLM_E_INVAL
    assert call_rope(lib, x_type=1, y=P + n * 2 - 4) == binding.DLLM_E_INVAL
    assert call_rope(lib, x_type=1, x=P + n * 4 - 2, y=P) == binding.DLLM_E_INVAL
    assert call_rope(lib, T=1, tok=0, x_tok=7, y=P + 8) == binding.DLLM_E_INVAL
    for off in (16, 256, n * 2 - 16):
        assert call_attend(lib, out=P + off) == binding.DLLM_E_INVAL
        assert call_attend(lib, q=P + off, out=P) == binding.DLLM_E_INVAL
    assert call_attend(lib, out=P, tok=256) == binding.DLLM_E_INVAL    # q itself, with other strides
    assert call_attend(lib, out=P, tok=64, head=256) == binding.DLLM_E_INVAL


def test_reading_keys_and_values_into_one_place_is_refused(lib):
    c = binding.dllm_kv4(P, P, 8, 64, 2, 64)
    n = 3 * 2 * 64 * 2
    for k, v in ((P, P), (P, P + n - 16), (P + n - 16, P)):
        assert lib.dllm_op_read_kv4(c, P, P, 3, P, 1, 1, k, v, 0, None) == binding.DLLM_E_INVAL


def test_tangents_are_seen_where_requires_grad_is_not_set():
    torch = pytest.importorskip("torch")
    from masked_block_diffusion_b200 import kv4
    x = torch.ones(3)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, x)
        assert torch.autograd.forward_ad._current_level >= 0 and not dual.requires_grad
        with pytest.raises(RuntimeError):
            kv4._refuse_tangent(x, dual)
        kv4._refuse_tangent(x, x)
    assert torch.autograd.forward_ad._current_level < 0


WIDE = 1 << 32                                                       # an int of 32 bits would take this as 0


def test_sizes_beyond_32_bits_are_refused():
    """Not taken modulo 2^32 on their way to the library."""
    c, plan = binding.dllm_kv4(P, P, 8, 64, 2, 64), Rope(64).c
    rope = dict(T=4, H=2, head_dim=64)
    page = dict(T=4, n_req=1, table_stride=1)
    attn = dict(B=1, T=4, max_q=1, max_kv=64, H=2)
    calls = [(binding.dllm_op_rope, rope, lambda a: (plan, P, 0, 128, 64, P, a["T"], a["H"], a["head_dim"], 2 * P, 0, 128, 64, 0, None)),
             (binding.dllm_op_append_kv4, page, lambda a: (c, P, 128, 64, P, 128, 64, 0, P, P, None, a["T"], P, a["n_req"], a["table_stride"],
                                                           None, None)),
             (binding.dllm_op_read_kv4, page, lambda a: (c, P, P, a["T"], P, a["n_req"], a["table_stride"], P, 2 * P, 0, None)),
             (binding.dllm_op_attn_kv4, {**attn, "table_stride": 1},
              lambda a: (c, P, 128, 64, 2 * P, 128, 64, None, P, P, a["B"], a["T"], a["max_q"], a["max_kv"], a["H"], P, a["table_stride"],
                         0, 0.125, None, 0, None)),
             (binding.dllm_op_attn_kv4_workspace, attn, lambda a: (c, a["B"], a["T"], a["max_q"], a["max_kv"], a["H"]))]
    for f, sizes, args in calls:
        for name in sizes:
            for off in (WIDE, -WIDE if name in ("T", "B") else WIDE * 3):
                with pytest.raises(binding.DllmError) as e:
                    f(*args({**sizes, name: sizes[name] * (off > 0) + off}))
                assert e.value.code == binding.DLLM_E_INVAL, (f.__name__, name)
    for n in (WIDE + 64, 64 - WIDE):
        with pytest.raises(binding.DllmError):
            Rope(n)
