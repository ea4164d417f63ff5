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


def test_error_words_and_workspaces_are_checked(B):
    import torch
    for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64, device="meta"),
                torch.zeros(0, dtype=torch.int32, device="meta")):
        with pytest.raises(ValueError, match="err_word"):
            B._error_word(bad, None, bad.get_device() if bad.is_meta else 0)
    host = torch.zeros(4096, dtype=torch.uint8)
    for bad, dev in ((host, 0), (host.expand(2, 4096), -1), (host[::2], -1)):
        with pytest.raises(ValueError, match="workspace_buf"):
            B._scratch(bad, 256, None, dev)


@pytest.mark.gpu
def test_error_words_and_workspaces_on_the_host_are_refused(B):
    import torch
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    lse = torch.zeros(2, 4, device="cuda")
    err, ws = torch.zeros(1, dtype=torch.int32), torch.zeros(1 << 20, dtype=torch.uint8)
    forward = (lambda **kw: B.flce_attention_forward(q, q, q, cu, **kw),
               lambda **kw: B.flce_qk_norm_rope_forward(q, q, None, None, None, None, **kw))
    backward = (lambda **kw: B.flce_attention_backward(q, q, q, q, q, lse, cu, **kw),
                lambda **kw: B.flce_qk_norm_rope_backward(q, q, q, q, None, None, None, None, **kw))
    for call in forward + backward:
        with pytest.raises(ValueError, match="err_word"):
            call(err_word=err)
    one = torch.zeros(1, dtype=torch.uint8, device="cuda")
    for call in backward:
        for bad in (ws, one.expand(1 << 20)):
            with pytest.raises(ValueError, match="workspace_buf"):
                call(workspace_buf=bad)
        with pytest.raises(B.FlceError):  # too small
            call(workspace_buf=one)
        call(workspace_buf=ws.cuda(), err_word=err.cuda())
