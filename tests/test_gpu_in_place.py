"""GPU checks that an output given by the caller counts as a change in place: what
autograd saved of it before is not used afterwards."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    import logits_sampling_gb300 as ls
    ls.load_library()


def _writers():
    import logits_sampling_gb300 as ls
    return {
        "process_logits": lambda x, ids, lp: ls.process_logits(x, out=x),
        "process_logits view": lambda x, ids, lp: ls.process_logits(x[:2], out=x[:2]),
        "distill_loss_grad": lambda x, ids, lp: ls.distill_loss_grad(x, ids, lp, out_grad=x),
        "distill_loss_backward": lambda x, ids, lp: ls.distill_loss_backward(x, ids, lp, ls.distill_loss(x, ids, lp)[1],
                                                                             out=x),
        "out_ids": lambda x, ids, lp: ls.top_log_probs(x, 5, out_ids=ids),
        "out_log_probs": lambda x, ids, lp: ls.top_log_probs(x, 5, out_log_probs=lp),
    }


@pytest.mark.parametrize("which", ["process_logits", "process_logits view", "distill_loss_grad", "distill_loss_backward",
                                   "out_ids", "out_log_probs"])
def test_backward_refuses_what_a_call_has_overwritten(which):
    import torch
    import logits_sampling_gb300 as ls
    leaf = torch.randn(4, 1000, device="cuda").requires_grad_()
    x = leaf * 1.0
    ids, lp, _ = ls.top_log_probs(x.detach(), 5)
    loss = ls.distill(x, ids, lp).sum()
    _writers()[which](x.detach(), ids, lp)  # detached, and views of it: one version for all
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_each_given_output_counts_once_and_nothing_else_does():
    import torch
    import logits_sampling_gb300 as ls
    x = torch.randn(4, 1000, device="cuda")
    ids, lp, lse = ls.top_log_probs(x, 5)
    loss, stats = ls.distill_loss(x, ids, lp)
    tensors = (x, ids, lp, lse, loss, stats)
    assert [t._version for t in tensors] == [0] * 6
    ls.top_log_probs(x, 5, out_ids=ids, out_log_probs=lp, out_lse=lse)
    ls.distill_loss(x, ids, lp, out=loss, out_stats=stats)
    assert [t._version for t in tensors] == [0, 1, 1, 1, 1, 1]
    with pytest.raises(ls.LSError):
        ls.process_logits(x, 5, out=torch.empty(5, 1000, device="cuda"))
    with torch.inference_mode():
        y = torch.randn(4, 1000, device="cuda")
        ls.process_logits(y, out=y)
    ls.process_logits(y, out=y)  # has no version, and no graph can have saved it


def test_a_gradient_over_the_logits_after_its_own_forward():
    """The calls without autograd work in place as before."""
    import torch
    import logits_sampling_gb300 as ls
    x = torch.randn(4, 1000, device="cuda")
    ids, lp, _ = ls.top_log_probs(torch.randn_like(x), 5)
    loss, stats = ls.distill_loss(x, ids, lp)
    want = ls.distill_loss_backward(x, ids, lp, stats)
    assert torch.equal(ls.distill_loss_backward(x, ids, lp, stats, out=x), want)
