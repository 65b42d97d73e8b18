"""The 64-bit definitions behind the training and adapter tests: their gradients against central differences."""
import torch

import train_reference as ref


def rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def differences(f, x, h=1e-6):
    """Central differences of the scalar function f at x, element by element."""
    out = torch.empty_like(x)
    flat, grad = x.reshape(-1), out.reshape(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + h
        hi = f()
        flat[i] = keep - h
        grad[i] = (hi - f()) / (2 * h)
        flat[i] = keep
    return out


def test_layer_norm_gradient_against_differences():
    K, T = 7, 4
    x, g, b, dy = rand(K, T, seed=1), rand(K, seed=2), rand(K, seed=3), rand(K, T, seed=4)
    loss = lambda: (ref.layer_norm(x, g, b)[0] * dy).sum()  # noqa: E731
    got = ref.layer_norm_grad(dy, x, g, b)
    for grad, at in zip(got, (x, g, b)):
        # the differences carry h^2 f''' and 1e-16 / h: about 1e-9 here
        assert torch.allclose(grad, differences(loss, at), rtol=1e-6, atol=1e-7)


def test_layer_norm_gradient_against_the_closed_form():
    x, g, dy = rand(9, 5, seed=5) + 3, rand(9, seed=6), rand(9, 5, seed=7)
    _, mean, rstd = ref.layer_norm(x, g)
    h, gy = (x - mean) * rstd, g[:, None] * dy
    dx = rstd * (gy - (gy.sum(0) + h * (gy * h).sum(0)) / 9)
    got = ref.layer_norm_grad(dy, x, g)
    assert torch.allclose(got[0], dx, rtol=1e-12, atol=1e-12)
    assert torch.allclose(got[1], (dy * h).sum(1), rtol=1e-12, atol=1e-12)
    assert torch.allclose(got[2], dy.sum(1), rtol=1e-12, atol=1e-12)


def test_cross_entropy_gradient_against_differences():
    w, x = rand(6, 5, seed=8), rand(5, 4, seed=9)
    target, dloss = torch.tensor([3, -100, 5, 6]), rand(4, seed=10)
    loss = lambda: (ref.cross_entropy(w @ x, target)[0] * dloss).sum()  # noqa: E731
    G, dX, dW = ref.cross_entropy_grad(w, x, target, dloss)
    assert torch.allclose(dX, differences(loss, x), rtol=1e-6, atol=1e-7)
    assert torch.allclose(dW, differences(loss, w), rtol=1e-6, atol=1e-7)
    p = torch.softmax(w @ x, 0)
    want = p.clone()
    want[3, 0] -= 1
    want[5, 2] -= 1
    want *= torch.where((target >= 0) & (target < 6), dloss, 0.0)
    assert torch.allclose(G, want, rtol=1e-12, atol=1e-14)


def test_adapter_gradients_against_differences():
    w, x, dy = rand(5, 6, seed=11), rand(6, 4, seed=12), rand(5, 4, seed=13)
    A, B, scale = rand(3, 2, 6, seed=14), rand(3, 5, 2, seed=15), rand(3, seed=16)
    adapter, idx = torch.tensor([2, 0, -1, 2]), torch.tensor([3, 0, 5, 1, 2, 4])
    f = lambda: (ref.lora(w, x[idx], A, B, adapter, scale, x) * dy).sum()  # noqa: E731
    for grad, at in zip(ref.lora_grad(dy, w, x, A, B, adapter, scale, idx), (x, A, B)):
        assert torch.allclose(grad, differences(f, at), rtol=1e-6, atol=1e-7)
    t = 0  # one token written out
    want = w @ x[idx][:, t] + scale[2] * B[2] @ (A[2] @ x[:, t])
    assert torch.allclose(ref.lora(w, x[idx], A, B, adapter, scale, x)[:, t], want, rtol=1e-13, atol=1e-13)
