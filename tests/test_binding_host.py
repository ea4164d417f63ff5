"""Refusals of the Python calls that need no GPU: tensors that only claim to be on one."""
import pytest


@pytest.fixture(scope="module")
def B():
    from linear_cross_entropy_logit_gb300 import binding, build
    build.build()
    binding.lib()
    return binding


class Elsewhere:
    """A tensor of another GPU than the current one, as far as the checks before a launch look."""
    device, is_cuda = "cuda:1", True

    def get_device(self):
        return 1

    def is_contiguous(self):
        return True

    def __getattr__(self, name):
        raise AssertionError(f"{name} was looked at before the device")


def test_attention_and_norm_refuse_tensors_of_another_gpu(B, monkeypatch):
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    t = Elsewhere()
    for call in (lambda: B.flce_attention_forward(t, t, t, t),
                 lambda: B.flce_attention_backward(t, t, t, t, t, t, t),
                 lambda: B.packed_attention(t, t, t, t),
                 lambda: B.flce_qk_norm_rope_forward(t, t, None, None, None, None),
                 lambda: B.flce_qk_norm_rope_backward(t, t, t, t, None, None, None, None),
                 lambda: B.qk_norm_rope(t, t, None, None, None, None)):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_loss_refuses_tensors_of_another_gpu(B, monkeypatch):
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    t = Elsewhere()
    for call in (lambda: B.flce_forward(t, t, t), lambda: B.flce_forward_ex(t, t, t, B.make_options()),
                 lambda: B.flce_backward(t, t, t, t, t), lambda: B.flce_fwd_bwd(t, t, t),
                 lambda: B.flce_forward_vocab_shard(t, t, t, 0, 10), lambda: B.flce_combine_vocab_shards(t, t, 10),
                 lambda: B.flce_backward_vocab_shard(t, t, t, 0, 10, t, t),
                 lambda: B.flce_forward_noalloc(t, t, t, loss=t, lse=t, valid_count=t, err_word=t)):
        with pytest.raises(ValueError, match="current device"):
            call()
