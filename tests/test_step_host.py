"""Refusals and workspace sizes of the distillation, the layer norm and the rotary positions:
no GPU needed (argument errors are returned before the device is looked at)."""
import ctypes
import math

import pytest

from tests.test_attention_host import B  # noqa: F401

P = 4096  # an address that is aligned; never read: every call below is refused
NAN, INF = float("nan"), float("inf")


def distill(B, **changes):  # noqa: F811
    d = B.FlceDistillDesc(ctypes.sizeof(B.FlceDistillDesc), 10, 64, 300, 5, B.FLCE_BF16, B.FLCE_FP32, B.FLCE_BF16,
                          1.0, B.FLCE_MEAN)
    for name, value in changes.items():
        setattr(d, name, value)
    return d


def norm(B, **changes):  # noqa: F811
    d = B.FlceLayerNormDesc(ctypes.sizeof(B.FlceLayerNormDesc), 10, 64, B.FLCE_BF16, 1e-5, 0, 64, 64)
    for name, value in changes.items():
        setattr(d, name, value)
    return d


def rope(B, **changes):  # noqa: F811
    d = B.FlceRopeDesc(ctypes.sizeof(B.FlceRopeDesc), 10, 4, 2, 64, 32, B.FLCE_BF16, 1.0, 0, 256, 64, 128, 64)
    for name, value in changes.items():
        setattr(d, name, value)
    return d


def calls(B, kind, d):  # noqa: F811
    """(forward, backward), each a function of its pointers by place."""
    L, d = B.lib(), ctypes.byref(d)
    if kind == "distill":
        return (lambda a: L.flce_distill_forward(d, *a, P, 1 << 40, P, None),
                lambda a: L.flce_distill_backward(d, *a, 0, P, 1 << 40, P, None))
    if kind == "norm":
        return (lambda a: L.flce_layer_norm_forward(d, *a, None),
                lambda a: L.flce_layer_norm_backward(d, *a, P, 1 << 40, None))
    return lambda a: L.flce_rope_forward(d, *a, None), lambda a: L.flce_rope_backward(d, *a, None)


POINTERS = {"distill": (10, 11), "norm": (8, 9), "rope": (6, 6)}
OPTIONAL = {"distill": ({4, 6}, {4, 8, 9, 10}), "norm": ({1, 2, 3, 5}, {2, 5, 8}), "rope": ({3}, {3})}
MAKE = {"distill": distill, "norm": norm, "rope": rope}
BAD = [("distill", c) for c in (
    {"struct_size": 8}, {"N": -1}, {"N": 2**31}, {"H": 12}, {"H": 0}, {"V": 0}, {"V": 2**31}, {"K": 0}, {"K": 1025},
    {"dtype": 9}, {"teacher_dtype": 9}, {"dw_dtype": 9}, {"temperature": 0.0}, {"temperature": -1.0},
    {"temperature": NAN}, {"temperature": INF}, {"reduction": 7})]
BAD += [("norm", c) for c in (
    {"struct_size": 8}, {"rows": -1}, {"rows": 2**31}, {"cols": 12}, {"cols": 0}, {"cols": 16392}, {"dtype": 9},
    {"eps": -1.0}, {"eps": NAN}, {"eps": INF}, {"rms": 2}, {"x_row": 60}, {"x_row": 56}, {"x_row": 0})]
BAD += [("rope", c) for c in (
    {"struct_size": 8}, {"tokens": -1}, {"tokens": 2**31}, {"q_heads": 0}, {"kv_heads": 0}, {"head_dim": 12},
    {"head_dim": 264}, {"rot_dim": 0}, {"rot_dim": 12}, {"rot_dim": 72}, {"dtype": 9}, {"magnitude": NAN},
    {"magnitude": INF}, {"q_row": 4}, {"q_row": 0}, {"k_head": 56}, {"k_head": 60})]


@pytest.mark.parametrize("kind,bad", BAD, ids=str)
def test_bad_descriptions_are_refused(B, kind, bad):  # noqa: F811
    for call, n in zip(calls(B, kind, MAKE[kind](B, **bad)), POINTERS[kind]):
        assert call([P] * n) == B.FLCE_ERR_ARG


@pytest.mark.parametrize("kind", MAKE)
def test_bad_pointers_are_refused(B, kind):  # noqa: F811
    for call, n, optional in zip(calls(B, kind, MAKE[kind](B)), POINTERS[kind], OPTIONAL[kind]):
        for i in range(n):
            for bad in (P + 1,) if i in optional else (None, P + 1):
                args = [P] * n
                args[i] = bad
                assert call(args) == B.FLCE_ERR_ARG, (i, bad)


def test_a_residual_needs_its_sum_and_its_stride(B):  # noqa: F811
    forward, _ = calls(B, "norm", norm(B))
    assert forward([P, P, P, P, P, None, P, P]) == B.FLCE_ERR_ARG
    for row in (60, 56):
        forward, _ = calls(B, "norm", norm(B, residual_row=row))
        assert forward([P] * 8) == B.FLCE_ERR_ARG


def test_fp32_distillation_and_accumulating_into_bf16_are_refused(B):  # noqa: F811
    forward, backward = calls(B, "distill", distill(B, dtype=B.FLCE_FP32))
    assert forward([P] * 10) == backward([P] * 11) == B.FLCE_ERR_UNSUPPORTED
    d = ctypes.byref(distill(B))
    assert B.lib().flce_distill_backward(d, *[P] * 11, 1, P, 1 << 40, P, None) == B.FLCE_ERR_ARG


def test_a_distillation_without_any_gradient_is_refused(B):  # noqa: F811
    _, backward = calls(B, "distill", distill(B))
    assert backward([P] * 9 + [None, None]) == B.FLCE_ERR_ARG


def test_workspaces(B):  # noqa: F811
    """Too small or misaligned ones are refused; their sizes have room for the entries and
    no N x V array, and are 0 for what is refused."""
    L = B.lib()
    for mode, args in ((B.MODE_FWD, 10), (B.MODE_BWD, 11)):
        need = L.flce_distill_workspace_size(distill(B), mode)
        call = L.flce_distill_forward if mode == B.MODE_FWD else L.flce_distill_backward
        extra = () if mode == B.MODE_FWD else (0,)
        for ws, size in ((None, need), (P + 64, need), (P, need - 1)):
            assert call(ctypes.byref(distill(B)), *[P] * args, *extra, ws, size, P, None) == B.FLCE_ERR_WORKSPACE
    assert L.flce_distill_workspace_size(distill(B, H=12), B.MODE_FWD) == 0
    assert L.flce_layer_norm_workspace_size(norm(B, cols=12)) == 0
    N, V, K = 8192, 128256, 64
    loss = B.flce_workspace_size(N, 4096, V, B.FLCE_BF16, B.MODE_FWD_BWD)
    size = B.flce_distill_workspace_size(N, 4096, V, K)
    assert loss < size <= loss + N * (K * 6 + 33 + 2 * 4096) + 10 * 256


def test_frequencies():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    def f(*a, **k):
        inv, m = B.rope_frequencies(*a, device="cpu", **k)
        return inv.tolist(), m
    plain, one = f(64, 10000.0)
    assert one == 1.0 and plain[0] == 1.0 and abs(plain[16] - 0.01) < 1e-15 and len(plain) == 32
    assert f(64, 10000.0, "linear", factor=4.0)[0] == [p / 4.0 for p in plain]
    ntk, _ = f(64, 10000.0, "ntk", factor=4.0)
    assert ntk[0] == 1.0 and abs(ntk[31] * 4.0 / plain[31] - 1) < 1e-12
    for kind, high, m in (("llama3", 4.0, 1.0), ("yarn", 32.0, 1.0 + 0.1 * math.log(4.0))):
        inv, got = f(64, 10000.0, kind, factor=4.0, trained_length=2048)
        assert got == m
        turns = [2048 * p / (2 * math.pi) for p in plain]
        for p, q, n in zip(plain, inv, turns):
            assert p / 4.0 * (1 - 1e-12) <= q <= p * (1 + 1e-12)
            if n > 1.5 * high:
                assert q == p
            if n < 0.6:
                assert abs(q * 4.0 / p - 1) < 1e-12
        assert all(a > b for a, b in zip(inv, inv[1:]))
    assert f(2, 10000.0, "yarn", factor=2.0)[0][0] <= 1.0
    for bad in ((63,), (0,), (64, 1.0), (64, 10.0, "other")):
        with pytest.raises(ValueError):
            f(*bad)
    with pytest.raises(ValueError):
        f(64, 10.0, "linear", factor=0.5)
    with pytest.raises(ValueError):
        f(64, 10.0, "yarn", low=40.0)
    assert B.rope_frequencies(8, device="cpu")[0].dtype == torch.float64


class Elsewhere:
    """A tensor of another GPU than the current one, as far as the checks before a launch look."""
    device, is_cuda = "cuda:1", True

    def get_device(self):
        return 1

    def __getattr__(self, name):
        if name == "dtype":
            import torch
            return torch.bfloat16
        raise AssertionError(f"{name} was looked at before the device")


def test_tensors_of_another_gpu_or_the_host_are_refused(B, monkeypatch):  # noqa: F811
    import torch
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    for t, match in ((Elsewhere(), "current device"), (torch.zeros(8, 8), "CUDA tensor")):
        for call in (lambda: B.flce_distill_forward(t, t, t, t), lambda: B.flce_distill_backward(t, t, t, t, t, t, t),
                     lambda: B.flce_layer_norm_forward(t, t), lambda: B.flce_layer_norm_backward(t, t, t, t, t),
                     lambda: B.flce_rope_forward(t, t, t), lambda: B.flce_rope_backward(t, t, t)):
            with pytest.raises(ValueError, match=match):
                call()
