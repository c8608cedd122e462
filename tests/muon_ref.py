"""Newton-Schulz steps in 64 bits, and what the library's arithmetic may be off by.

What it rounds: an operand kept as two fp16 limbs of 1024 times its value is off by
at most 2^-22 of its value, or, where the second limb is subnormal (a multiple of
2^-24), by half of that over 1024, 2^-35; a product of two leaves out lo lo (2^-22 of each term) and adds its K terms
in fp32, in K/16 chunks of the tensor cores whose sums may be truncated, each by
2^-23 of the sum of magnitudes so far, together (K/16 + 8) 2^-23 of it at most.
`spread` carries errors of that size through the steps, once with random signs and
once all of one sign, and returns twice the largest difference that either makes."""
import torch

NS = (3.4445, -4.7750, 2.0315)


def triples(coeffs, steps):
    return list(coeffs) if coeffs and hasattr(coeffs[0], "__len__") else [coeffs] * steps


def steps64(x, coeffs, steps, eps=1e-7, noise=None):
    """x: fp64 [rows, cols]; noise(value, magnitudes) -> value with an error, or None."""
    off = noise or (lambda v, mag, K: v)
    stored = lambda v: off(v, v.abs() * 2.0 ** -22 + 2.0 ** -35, 0)  # noqa: E731
    x = x / (torch.linalg.matrix_norm(x) + eps)
    flip = x.shape[0] > x.shape[1]
    x = stored(x.T if flip else x)
    for a, b, c in triples(coeffs, steps):
        if noise is None:
            g = x @ x.T
            x = a * x + (b * g + c * g @ g) @ x
            continue
        err = lambda K: 2.0 ** -22 + (K / 16 + 8) * 2.0 ** -23  # noqa: E731
        g = x @ x.T
        g = stored(off(g, err(x.shape[1]) * (x.abs() @ x.abs().T), 1))
        p = a * torch.eye(len(g), dtype=g.dtype) + b * g + c * off(g @ g, err(len(g)) * (g.abs() @ g.abs()), 1)
        p = stored(p)
        x = stored(off(p @ x, err(len(g)) * (p.abs() @ x.abs()), 1))
    return x.T if flip else x


def by_singular_values(x, coeffs, steps, eps=1e-7):
    """The same from the definition: the polynomial of every singular value."""
    u, s, v = torch.linalg.svd(x / (torch.linalg.matrix_norm(x) + eps), full_matrices=False)
    for a, b, c in triples(coeffs, steps):
        s = a * s + b * s ** 3 + c * s ** 5
    return (u * s) @ v


def spread(x, coeffs, steps, eps=1e-7):
    want = steps64(x, coeffs, steps, eps)
    g = torch.Generator().manual_seed(7)
    rand = steps64(x, coeffs, steps, eps, lambda v, mag, K: v + mag * (torch.randint(0, 2, v.shape, generator=g) * 2 - 1))
    down = steps64(x, coeffs, steps, eps, lambda v, mag, K: v - mag if K else v + mag)
    return want, 2 * max(float((rand - want).abs().max()), float((down - want).abs().max())) + 2.0 ** -40


def plain_steps(x, coeffs=NS, steps=5, eps=1e-7, stored=lambda v: v):
    """The steps in x's own type; stored: what keeping an operand does to it."""
    x = x / (x.double().norm() + eps).to(x.dtype)
    flip = x.shape[0] > x.shape[1]
    x = stored(x.mT if flip else x)
    for a, b, c in triples(coeffs, steps):
        g = stored(x @ x.mT)
        p = stored(a * torch.eye(len(g), dtype=g.dtype, device=g.device) + b * g + c * (g @ g))
        x = stored(p @ x)
    return x.mT if flip else x


def in_limbs(v, t, count):
    """v as `count` limbs of type t hold 1024 times it."""
    total, rest = torch.zeros_like(v), v * 1024
    for _ in range(count):
        limb = rest.to(t).to(v.dtype)
        total, rest = total + limb, rest - limb
    return total / 1024
