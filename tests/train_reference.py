"""64-bit definitions of the operators around a pruned projection, for the GPU parity tests.

Plain torch.float64 on the CPU, written from the formulas; gradients come from
autograd on these definitions, so that a gradient kernel is checked against
the derivative of the forward formula and not against a copy of its own.
"""
import torch

U32 = 2.0 ** -24    # half a step of float32
UBF16 = 2.0 ** -8   # half a step of bf16


def layer_norm(x, gamma=None, beta=None, eps=1e-5):
    """(y, mean, rstd) over dim 0 of x (features x tokens, float64)."""
    mean = x.mean(0)
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(0) + eps)
    y = (x - mean) * rstd
    if gamma is not None:
        y = y * gamma[:, None]
    if beta is not None:
        y = y + beta[:, None]
    return y, mean, rstd


def layer_norm_grad(dy, x, gamma=None, beta=None, eps=1e-5):
    """(dx, dgamma, dbeta) by autograd; gamma and beta default to ones and zeros."""
    K = x.shape[0]
    x = x.detach().clone().requires_grad_()
    g = (torch.ones(K, dtype=torch.float64) if gamma is None else gamma.detach().clone()).requires_grad_()
    b = (torch.zeros(K, dtype=torch.float64) if beta is None else beta.detach().clone()).requires_grad_()
    return torch.autograd.grad(layer_norm(x, g, b, eps)[0], (x, g, b), dy)


def chain(n):
    """Relative bound of a float32 sum whose longest chain has n additions: n u / (1 - n u)."""
    return n * U32 / (1 - n * U32)


def cross_entropy(z, target):
    """(loss, lse) per column of the logits z (R x T, float64); a target outside [0, R) gives a loss of 0."""
    lse = torch.logsumexp(z, 0)
    has = (target >= 0) & (target < z.shape[0])
    at = torch.where(has, target, 0).long()
    return torch.where(has, lse - z.gather(0, at[None, :])[0], torch.zeros_like(lse)), lse


def cross_entropy_grad(w, x, target, dloss):
    """(G, dX, dW) of sum(dloss * loss) with z = w x, by autograd."""
    w, x = w.detach().clone().requires_grad_(), x.detach().clone().requires_grad_()
    z = w @ x
    loss, _ = cross_entropy(z, target)
    return torch.autograd.grad((loss * dloss).sum(), (z, x, w))


def lora(w, x, A, B, adapter, scale=None, low_x=None):
    """w x + scale_a B_a A_a low_x column by column (float64); low_x: the adapters' input, x by default."""
    y, z = w @ x, x if low_x is None else low_x
    for a in range(A.shape[0]):
        serves = (adapter == a).to(torch.float64)
        y = y + (1.0 if scale is None else scale[a]) * (B[a] @ (A[a] @ z)) * serves
    return y


def lora_grad(dy, w, x, A, B, adapter, scale=None, idx=None):
    """(dX, dA, dB) of <dy, lora> by autograd, x before the index map."""
    x, A, B = (v.detach().clone().requires_grad_() for v in (x, A, B))
    y = lora(w, x if idx is None else x[idx], A, B, adapter, scale, x)
    return torch.autograd.grad((y * dy).sum(), (x, A, B), allow_unused=True, materialize_grads=True)
