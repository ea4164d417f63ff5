"""The attention kernels' index arithmetic at the ends of its range: on the host, compiled from
the kernels' own headers, and offsets that no sequence can have on the GPU."""
import os
import subprocess

import pytest

from linear_cross_entropy_logit_gb300 import build

LOW, HIGH = -2**31, 2**31 - 1
# tokens, offsets, whether they ascend within [0, tokens]
OFFSETS = [
    (300, [0, 300], True), (300, [5, 5], True), (300, [300, 300], True), (0, [0, 0], True),
    (HIGH - 1024, [0, HIGH - 1024], True),
    (300, [0, 301], False), (300, [-1, 300], False), (300, [10, 9], False), (300, [301, 301], False),
    # differences that pass 32 bits
    (300, [5, LOW], False), (300, [300, LOW], False), (300, [0, LOW], False), (300, [1, LOW + 1], False),
    (300, [HIGH, LOW], False), (300, [LOW, HIGH], False), (300, [LOW, 300], False), (300, [LOW, LOW], False),
    (HIGH - 1024, [HIGH - 1024, LOW], False),
]


def host_program(tmp_path, header, body):
    """Output lines of a host program made of `body` with one of the kernels' headers."""
    src, exe = tmp_path / "t.cu", tmp_path / "t"
    src.write_text(f'#include "{header}"\n#include <cstdio>\nint main() {{\n{body}\n}}\n')
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-I", build.CSRC, "-I", build.INCLUDE,
                    str(src), "-o", str(exe)], check=True, capture_output=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()


def test_offsets_are_compared_not_subtracted(tmp_path):
    calls = "".join(f'printf("%d\\n", flce::sequence_ok({a[0]}, {a[1]}, {t}));\n' for t, a, _ in OFFSETS)
    got = host_program(tmp_path, "attn_common.cuh", calls)
    assert [x == "1" for x in got] == [ok for *_, ok in OFFSETS]


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [a for t, a, ok in OFFSETS if t == 300 and not ok]
                         + [[0, 100, LOW], [0, HIGH, 300], [LOW, 0, 300], [0, 300, LOW, 300], [HIGH], [LOW]], ids=str)
def test_offsets_that_no_sequence_has(cu):
    """Reported, and every row then counts as one of no sequence."""
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    from tests.test_gpu_attention import make, run
    q, k, v, g = make(300, 2, 1, 64, seed=22)
    out, lse, dq, dk, dv, err = run(q, k, v, g, cu)
    assert err == B.FLCE_ERR_INDEX
    assert torch.isneginf(lse).all() and not any(t.any() for t in (out, dq, dk, dv))


# splits, tokens, key / value heads, head size: the second and third pass 32 bits in the product
# of splits and tokens alone
PARTIALS = [(2, 100, 8, 128), (65521, 17000, 1, 8), (4096, 2**20, 2, 128)]


def test_partial_sums_lie_where_the_workspace_has_them(tmp_path):
    """Offsets of the backward's partial sums of dk and dv of each split, in 64 bits."""
    body = "".join(
        f'{{ flce::AttnBwdParams p{{}}; p.splits = {s}; p.tokens = {t}; p.kv_heads = {h}; p.head_dim = {d};\n'
        f'  printf("%lld %lld %lld\\n", (long long)p.partial_at(false, 0), (long long)p.partial_at(false, {s - 1}),\n'
        f'         (long long)p.partial_at(true, {s - 1})); }}\n' for s, t, h, d in PARTIALS)
    got = [int(x) for x in host_program(tmp_path, "attn_bwd.cuh", body)]
    assert got == [part * t * h * d for s, t, h, d in PARTIALS for part in (0, s - 1, 2 * s - 1)]
