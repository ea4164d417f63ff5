"""Refusals and workspace sizes of the attention and head-norm calls: no GPU needed
(argument errors are returned before the device is looked at)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def B():
    from linear_cross_entropy_logit_gb300 import binding, build
    build.build()
    binding.lib()
    return binding


def attention_desc(B, **changes):
    d = B.FlceAttentionDesc(ctypes.sizeof(B.FlceAttentionDesc), 10, 2, 4, 2, 64, B.FLCE_BF16, 0.125,
                            512, 64, 512, 64, 512, 64)
    for name, value in changes.items():
        setattr(d, name, value)
    return d


def norm_desc(B, **changes):
    d = B.FlceQkNormRopeDesc(ctypes.sizeof(B.FlceQkNormRopeDesc), 10, 4, 2, 64, 64, 32, B.FLCE_BF16,
                             1e-6, 0, 512, 64, 512, 64)
    for name, value in changes.items():
        setattr(d, name, value)
    return d


P = 4096  # an address that is aligned; never read: every call below is refused
ATTENTION_BAD = [
    {"struct_size": 8}, {"tokens": -1}, {"sequences": -1}, {"q_heads": 3}, {"q_heads": 0},
    {"kv_heads": 0}, {"head_dim": 12}, {"head_dim": 136}, {"head_dim": 0}, {"dtype": 9},
    {"scale": 0.0}, {"scale": -1.0}, {"scale": float("nan")}, {"scale": float("inf")},
    {"q_row": 4}, {"k_head": 60}, {"v_head": 0}, {"v_row": 0}, {"tokens": 2**31},
]


@pytest.mark.parametrize("bad", ATTENTION_BAD, ids=str)
def test_attention_refuses_bad_descriptions(B, bad):
    d = ctypes.byref(attention_desc(B, **bad))
    assert B.lib().flce_attention_forward(d, P, P, P, P, P, P, P, None) == B.FLCE_ERR_ARG
    assert B.lib().flce_attention_backward(d, P, P, P, P, P, P, P, P, P, P, P, 1 << 30, P,
                                           None) == B.FLCE_ERR_ARG


def test_attention_refuses_fp32(B):
    d = ctypes.byref(attention_desc(B, dtype=B.FLCE_FP32))
    assert B.lib().flce_attention_forward(d, P, P, P, P, P, P, P, None) == B.FLCE_ERR_UNSUPPORTED


def test_attention_refuses_bad_pointers(B):
    d = ctypes.byref(attention_desc(B))
    good = [P] * 7
    for i in range(7):
        for bad in (None, P + 2):
            args = list(good)
            args[i] = bad
            assert B.lib().flce_attention_forward(d, *args, None) == B.FLCE_ERR_ARG, (i, bad)
    good = [P] * 10
    need = B.lib().flce_attention_workspace_size(d)
    for i in range(10):
        for bad in (None, P + 2):
            args = list(good)
            args[i] = bad
            assert B.lib().flce_attention_backward(d, *args, P, need, P, None) == B.FLCE_ERR_ARG
    for ws, n in ((None, need), (P + 16, need), (P, need - 1)):
        assert B.lib().flce_attention_backward(d, *good, ws, n, P, None) == B.FLCE_ERR_WORKSPACE


NORM_BAD = [
    {"struct_size": 8}, {"tokens": -1}, {"q_heads": 0}, {"kv_heads": 0}, {"head_dim": 20},
    {"head_dim": 264}, {"rot_dim": 4}, {"rot_dim": 72}, {"rot_dim": -8}, {"dtype": 3},
    {"eps": -1.0}, {"eps": float("nan")}, {"table_rows": 0}, {"q_row": 12}, {"k_head": 32},
]


@pytest.mark.parametrize("bad", NORM_BAD, ids=str)
def test_norm_refuses_bad_descriptions(B, bad):
    d = ctypes.byref(norm_desc(B, **bad))
    assert B.lib().flce_qk_norm_rope_forward(d, *[P] * 10, None) == B.FLCE_ERR_ARG
    assert B.lib().flce_qk_norm_rope_backward(d, *[P] * 14, 1 << 30, P, None) == B.FLCE_ERR_ARG


def test_norm_refuses_bad_pointers(B):
    d = ctypes.byref(norm_desc(B))
    # q, k, weights, tables, positions, outputs, err_word
    for i, nulls in enumerate([1, 1, 0, 0, 1, 1, 0, 1, 1, 1]):
        for bad in ([None] if nulls else []) + [P + 2]:
            args = [P] * 10
            args[i] = bad
            assert B.lib().flce_qk_norm_rope_forward(d, *args, None) == B.FLCE_ERR_ARG, (i, bad)


def test_workspace_sizes(B):
    L = B.lib()
    assert L.flce_attention_workspace_size(ctypes.byref(attention_desc(B, head_dim=12))) == 0
    small = L.flce_attention_workspace_size(ctypes.byref(attention_desc(B)))
    large = L.flce_attention_workspace_size(ctypes.byref(attention_desc(B, tokens=100000)))
    assert 0 < small < large
    assert L.flce_qk_norm_rope_workspace_size(ctypes.byref(norm_desc(B, rot_dim=4))) == 0
    assert L.flce_qk_norm_rope_workspace_size(ctypes.byref(norm_desc(B))) > 0


def test_binding_refuses_mismatched_tensors(B):
    import torch
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # not on a GPU
        B.flce_attention_forward(q, q, q, cu)
    with pytest.raises(ValueError):
        B.flce_qk_norm_rope_forward(q, q, None, None, None, None)


def test_exports(B):
    for name in B.EXPORTED:
        assert hasattr(B.lib(), name), name
