"""Plain forms of the new-token calls in 64 bits (or more): rotation by position, int8 cells."""
import numpy as np
import torch


def rotate(x, positions, freqs, axis=None, interleaved=False, inverse=False):
    """x [ntok, nheads, 128] rotated, in 64 bits on the CPU; whole turns are taken off in numpy's longest type, as a
    position of 2^31 times a 24-bit frequency has 55 bits."""
    n = freqs.numel()
    pos = positions.cpu().numpy().astype(np.longdouble)
    pos = pos[None] if pos.ndim == 1 else pos
    f = freqs.cpu().numpy().astype(np.longdouble)
    which = np.zeros(n, dtype=int) if axis is None else axis.cpu().numpy()
    turned = (which >= 0) & (which < pos.shape[0])
    angle = pos[np.where(turned, which, 0)].T * np.where(turned, f, 0)
    two_pi = np.longdouble("6.28318530717958647692528676655900577")
    angle = torch.from_numpy((angle - np.rint(angle / two_pi) * two_pi).astype(np.float64))
    if inverse:
        angle = -angle
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    x = x.detach().cpu().to(torch.float64)
    y = x.clone()
    i = torch.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def inv_two_pi(bits):
    """2^bits / (2 pi), cut off, by Machin's formula in whole numbers."""
    unit = 1 << (bits + 64)

    def arctan_of_one_over(n):
        term, total, k = unit // n, 0, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term, k = term // (n * n), k + 2
        return total

    return (unit << bits) // (8 * (4 * arctan_of_one_over(5) - arctan_of_one_over(239)))


def far_angles(positions, freqs):
    """position x frequency less its whole turns [ntok, pairs], in 64 bits: worked out in whole numbers of 2^-400 turns."""
    unit, inv = 1 << 400, inv_two_pi(400)
    rows = []
    for p in positions.tolist():
        row = []
        for f in freqs.tolist():
            n, d = float(f).as_integer_ratio()
            turns = p * n * inv // d % unit
            row.append((turns - unit if 2 * turns > unit else turns) / unit * 2 * np.pi)
        rows.append(row)
    return torch.tensor(rows, dtype=torch.float64)


def rotate_tol(x, want, dtype, pairs, interleaved=False):
    """sincospif is off by one unit in the last place (2^-24 below 1), its argument by 2^-24 of at most pi/4 and the
    angle by 2^-32 turns and 2^-33 of the factor's: below 1.9 x 2^-24 for each sine and cosine; a product and a fused
    product and sum round twice by 2^-24. In all below 4 x 2^-24 of |a| + |b|. Then half a step of the type."""
    x = x.detach().cpu().to(torch.float64).abs()
    both = torch.zeros_like(x)
    i = torch.arange(pairs)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    both[..., a] = both[..., b] = x[..., a] + x[..., b]
    tol = both * 4 * 2.0 ** -24
    if dtype != torch.float32:
        tol = tol + (want.abs() + tol) * torch.finfo(dtype).eps / 2 + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    return tol


def codes(x):
    """int8 codes and binary16 scales of rows x [..., 128] of fp32 values, by single IEEE operations."""
    x = x.detach().cpu().float()
    finite = torch.isfinite(x).all(-1)
    x0 = torch.where(finite[..., None], x, 0.0)
    scale = (x0.abs().amax(-1) / torch.tensor(127.0)).clamp(max=65504.0).to(torch.float16)
    f = scale.float()[..., None]
    q = torch.where(f > 0, torch.round(x0 / torch.where(f > 0, f, 1.0)), 0.0).clamp(-127, 127).to(torch.int8)
    return q, torch.where(finite, scale, torch.tensor(float("nan"), dtype=torch.float16))
