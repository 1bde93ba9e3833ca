"""GPU checks of rows of weight 0 in the distillation calls: loss 0 and gradient 0
whatever arrives from the layers above."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tail", ["drop", "renorm", "bucket"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_weight_zero_under_any_gradient_of_the_loss(dtype, tail):
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    import logits_sampling_gb300 as ls
    n, V = 8, 3001
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(n, V, device="cuda", generator=gen).to(getattr(torch, dtype))
    ids, lp, _ = ls.top_log_probs(torch.randn(n, V, device="cuda", generator=gen), 9)
    w = torch.tensor([0.0, 0.0, -0.0, 0.0, 1.0, 1.0, 2.0, 1.0], device="cuda")
    up = torch.tensor([float("inf"), float("nan"), -float("inf"), 3.0, 1.0, 0.0, 0.5, 1.0], device="cuda")
    loss, stats = ls.distill_loss(x, ids, lp, tail=tail, weights=w)
    grad = ls.distill_loss_backward(x, ids, lp, stats, grad_loss=up, tail=tail, weights=w)
    assert bool((loss[:4] == 0).all()) and bool((grad[:4] == 0).all())
    assert bool((grad[5] == 0).all()) and bool((grad[[4, 6, 7]] != 0).any(1).all()) and bool(torch.isfinite(grad).all())
    leaf = x.clone().requires_grad_()
    (ls.distill(leaf, ids, lp, tail=tail, weights=w)).backward(up)
    assert torch.equal(leaf.grad, grad)
