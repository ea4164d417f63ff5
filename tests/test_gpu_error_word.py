"""What went wrong on the device reaches the user of the autograd entries."""
import pytest

pytestmark = pytest.mark.gpu


def test_attention_reports_bad_offsets():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q = torch.randn(40, 2, 64, device="cuda").bfloat16().requires_grad_()
    err = B.new_err_word("cuda")
    good, bad = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in ([0, 10, 40], [0, 30, 20, 40]))
    B.packed_attention(q, q, q, good, err_word=err).sum().backward()
    assert int(err.item()) == 0
    out = B.packed_attention(q, q, q, bad, err_word=err)
    assert int(err.item()) == B.FLCE_ERR_INDEX
    err.zero_()  # the backward's own report, into the same word
    out.sum().backward()
    assert int(err.item()) == B.FLCE_ERR_INDEX


def test_head_norm_reports_positions_outside_the_tables():
    import torch
    from linear_cross_entropy_logit_gb300 import binding as B
    q = torch.randn(8, 2, 64, device="cuda").requires_grad_()
    cos, sin = torch.ones(8, 32, device="cuda"), torch.zeros(8, 32, device="cuda")
    err = B.new_err_word("cuda")
    B.qk_norm_rope(q, q, None, None, cos, sin, err_word=err)[0].sum().backward()
    assert int(err.item()) == 0
    pos = torch.arange(8, device="cuda") + 1
    out, _ = B.qk_norm_rope(q, q, None, None, cos, sin, pos, err_word=err)
    assert int(err.item()) == B.FLCE_ERR_INDEX
    err.zero_()
    out.sum().backward()
    assert int(err.item()) == B.FLCE_ERR_INDEX


def test_block_passes_its_error_word_on():
    import os
    import sys
    import torch
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    from linear_cross_entropy_logit_gb300 import binding as B
    from packed_training_step import Block, packed_batch
    block = Block(256, 4, 2, 64, 1000, 100)
    x, cu, positions, labels = packed_batch(100, 3, 256, 1000)
    err = B.new_err_word("cuda")
    block(x, cu, positions, labels, err).backward()
    assert int(err.item()) == 0
    block(x, cu, positions + 100, labels, err)
    assert int(err.item()) == B.FLCE_ERR_INDEX
