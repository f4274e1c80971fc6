"""Definition in 64 bits of the softmax cross entropy over a vocabulary, for the
tests; on whatever device its inputs are.

Bounds.  A logit z is a sum of K products in fp32: off by 1e-5 of the sum over
magnitudes at most (as the ragged products' tests take it).  With e that error,
largest over a token's words, and s = max |z| log2(e) + log2(V) + 1:
  lse   e + 2^-21 (an exponential) + 4 s 2^-24 (the scaled logits' roundings and the
        sums of 32, of tiles and of parts: V <= 2^17 words in chunks of 32 in order,
        V / 64 2^-24 at most) + 2^-23 |lse|
  p     relative: twice the error of z - lse, 2^-21, and one rounding to bf16 (2^-8)
"""
import torch

F64 = torch.float64
U = 2.0 ** -24
BF16_ROUND = 2.0 ** -8


def logits(X, W):
    return X.to(F64) @ W.to(F64).t()


def magnitudes(X, W):
    return X.to(F64).abs() @ W.to(F64).abs().t()


def there(targets, V):
    return (targets >= 0) & (targets < V)


def loss(X, W, targets):
    z = logits(X, W)
    lse = torch.logsumexp(z, 1)
    on = there(targets, W.shape[0])
    y = torch.where(on, targets, 0).long()
    return torch.where(on, lse - z.gather(1, y[:, None])[:, 0], 0.0), lse


def probabilities(X, W, targets, lse, d_loss):
    """p [T, V]."""
    V = W.shape[0]
    on = there(targets, V)
    p = torch.exp(logits(X, W) - lse.to(F64)[:, None])
    at = on.nonzero()[:, 0]
    p[at, targets[at].long()] -= 1.0
    return p * torch.where(on, d_loss.to(F64), 0.0)[:, None]


def gradients(X, W, targets, lse, d_loss):
    p = probabilities(X, W, targets, lse, d_loss)
    return p @ W.to(F64), p.t() @ X.to(F64)


def slack(X, W):
    """Error of a token's logits, and of its lse."""
    z, V = logits(X, W), W.shape[0]
    e = 1e-5 * magnitudes(X, W).amax(1)
    s = z.abs().amax(1) * 1.4427 + V ** 0.5 / 8 + 20
    return e, e + 2.0 ** -21 + (4 * s + V / 64) * U + 2 * U * torch.logsumexp(z, 1).abs()
