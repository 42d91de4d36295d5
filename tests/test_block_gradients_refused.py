"""linattn, add_norm and gated_norm record no graph: a tensor that requires a gradient
is refused where one would be recorded, and taken under torch.no_grad().  The refusal
comes before any other check, so most of this runs without a GPU."""
import pytest
import torch

import mamba_ssd_chunked_fwd_amd as ssd

T, H, G, K, V, D = 20, 4, 2, 64, 64, 96


def tensors(device="cpu"):
    g = torch.Generator().manual_seed(3)

    def rows(*shape):
        return torch.randn(*shape, generator=g).to(device)

    return {"linattn": {"q": rows(1, T, G, K), "k": rows(1, T, G, K), "v": rows(1, T, H, V),
                        "log_decay": -rows(H).abs(), "init_state": rows(1, H, K, V)},
            "add_norm": {"x": rows(T, D), "residual": rows(T, D), "res_scale": rows(D),
                         "weight": rows(D)},
            "gated_norm": {"x": rows(T, D), "z": rows(T, D), "weight": rows(D)}}


CALLS = [(f, n) for f, t in tensors().items() for n in t]


@pytest.mark.parametrize("call,name", CALLS)
def test_a_lost_gradient_is_refused(call, name):
    args = tensors()[call]
    args[name].requires_grad_()
    with pytest.raises(ValueError, match=f"{call} records no graph.*{name}.*{call}_backward"):
        getattr(ssd, call)(**args)
    # where no graph is recorded the next check speaks: the tensors are not on a GPU
    for mode in (torch.no_grad, torch.inference_mode):
        with mode(), pytest.raises(ValueError, match="must be a GPU tensor"):
            getattr(ssd, call)(**args)
    args[name] = args[name].detach()
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        getattr(ssd, call)(**args)


@pytest.mark.gpu
@pytest.mark.parametrize("call,name", CALLS)
def test_without_a_graph_the_results_are_the_same(call, name):
    args = tensors("cuda:0")[call]
    want = getattr(ssd, call)(**args)
    args[name].requires_grad_()
    with pytest.raises(ValueError):
        getattr(ssd, call)(**args)
    with torch.no_grad():
        got = getattr(ssd, call)(**args)
    if isinstance(want, torch.Tensor):
        got, want = (got,), (want,)
    for a, b in zip(got, want):
        assert not a.requires_grad and torch.equal(a, b)


@pytest.mark.gpu
def test_inside_an_autograd_function():
    """A function of the user's own, whose forward and backward record no graph: its
    gradients are those of the call."""
    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, z, weight):
            ctx.save_for_backward(x, z, weight)
            return ssd.gated_norm(x, z, weight)

        @staticmethod
        def backward(ctx, dy):
            return ssd.gated_norm_backward(*ctx.saved_tensors, dy.contiguous())

    args = tensors("cuda:0")["gated_norm"]
    dy = torch.randn(T, D, device="cuda:0")
    want = ssd.gated_norm_backward(*args.values(), dy)
    leaves = [t.requires_grad_() for t in args.values()]
    Norm.apply(*leaves).backward(dy)
    for t, w in zip(leaves, want):
        assert torch.equal(t.grad, w)
