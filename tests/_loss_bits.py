"""Inputs whose float32 vocabulary loss has one product of two numbers in each value that counts, so that its bits can be seen.

A float32 value is three parts of 8 bits, a product six pairs of parts.  Truncated
parts of v, 2^e <= |v| < 2^(e+1), are below 2^(e+1), 2^(e-7) and 2^(e-15); rounded ones
are 2^(e+1), 2^(e-8), 2^(e-16) at most.  Relative errors of a product, U = 2^-24:
  left out   two truncated factors: 2 * 2^-7 * 2^-15 = 8 U;  one of them rounded: 2^-8 * 2^-15 + 2^-16 * 2^-7 = 4 U
  added up   six times cut off to fp32 (2 U each), three chains added in fp32 (U each): 15 U
The smallest pairs that are used are up to 2^-15 of the product: one that is missing
shows in the worst of some hundred values by more than three times these bounds.
"""
import torch

U = 2.0 ** -24
FORWARD = 8 * U + 15 * U + 3 * U  # and expf, logf of 1, the last sum
# dz of probability 1 / V: exp of a difference near log V < 8, off by some 2^-20 of p and so 2^-20 / V of dz; its two roundings
BACKWARD = 4 * U + 15 * U + 4 * U


def mantissas(*shape, g):
    """Values of 1 to 2 and either sign whose 24 bits are all used."""
    m = 1 + torch.randint(0, 1 << 23, shape, generator=g).double() * 2.0 ** -23
    return (m * (1 - 2 * torch.randint(0, 2, shape, generator=g))).float()


def forward_case(T, d, V, seed):
    """(x, W, labels, lse in 64 bits): a token has one element, its largest logit is far above the others."""
    g = torch.Generator().manual_seed(seed)
    at, word = torch.randint(0, d, (T,), generator=g), torch.randint(0, V, (d,), generator=g)
    x, W = torch.zeros(T, d), 0.25 * mantissas(V, d, g=g)
    x[torch.arange(T), at] = mantissas(T, g=g)
    W[word, torch.arange(d)] = 64 * mantissas(d, g=g).abs()
    x = x.abs()
    labels = torch.randint(0, V, (T,), generator=g).int()
    return x, W, labels, x[torch.arange(T), at].double() * W[word[at], at].double()


def backward_case(T, d, V, seed, word, token=None):
    """(x, W, labels, lse, dloss): logits of nearly 0, one word of W that is not 0, the label of all tokens; and of x one
    token (or every one).  dx of a token is its dz times that word, dW of the word that token's dz times its x."""
    g = torch.Generator().manual_seed(seed)
    x, W = mantissas(T, d, g=g) * 2.0 ** -60, torch.zeros(V, d)
    W[word] = mantissas(d, g=g)
    if token is not None:
        x[torch.arange(T) != token] = 0
    lse = torch.full((T,), float(V)).log()
    # of some thousand gradients those whose dz has the largest second and third parts
    some = mantissas(4096, g=g).abs()
    _, mid, lo = parts((some.double() * (torch.exp(-lse[:1].double()) - 1)).float(), True)
    best = torch.minimum(mid.abs() * 2.0 ** 8, lo.abs() * 2.0 ** 16).argsort(descending=True)
    return x, W, torch.full((T,), word, dtype=torch.int32), lse, some[best[:T]]


def parts(v, rounded=False):
    """The three bf16 parts of float32 values, in 64 bits."""
    p, rest = [], v.float()
    for _ in range(3):
        top = rest.bfloat16().float() if rounded else (rest.view(torch.int32) & -65536).view(torch.float32)
        p.append(top.double())
        rest = rest - top
    return p


def product(a, b, without=None):
    """The sum of the six pairs of parts, one of them left out."""
    return sum(a[i] * b[j] for i in range(3) for j in range(3 - i) if (i, j) != without)
