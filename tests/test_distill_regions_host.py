"""The debug library lays a distillation's workspace out as the release library does and finds
its regions in order: it answers 0 for a layout that overlaps or overruns (no GPU needed)."""
import ctypes

import pytest

from tests.test_attention_host import B  # noqa: F401


@pytest.mark.parametrize("chunk", [0, 256, 2048, 100000])
def test_the_debug_library_accepts_every_layout(B, chunk):  # noqa: F811
    sizes = []
    for path in (B.LIB_PATH, B.DEBUG_LIB_PATH):
        L = B.load(path)
        L.flce_set_vocab_chunk(chunk)
        try:
            sizes.append([
                L.flce_distill_workspace_size(
                    B.FlceDistillDesc(ctypes.sizeof(B.FlceDistillDesc), N, H, V, K, B.FLCE_BF16, B.FLCE_FP32,
                                      B.FLCE_BF16, 1.0, B.FLCE_MEAN), mode)
                for N in (0, 1, 63, 64, 257, 2001, 8192, 100000) for H in (8, 520, 4096)
                for V in (1, 255, 257, 4099, 32003, 128256) for K in (1, 33, 1024)
                for mode in (B.MODE_FWD, B.MODE_BWD, B.MODE_FWD_BWD)])
        finally:
            L.flce_set_vocab_chunk(0)
    assert all(sizes[0]) and sizes[0] == sizes[1]
