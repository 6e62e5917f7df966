"""Plain 64-bit forms of the bounded-cache operators and the error bounds of
the kernels' arithmetic (u = 2^-24, S = scale * sum_d |q_d k_d| of a cell).

A logit is a 128-term dot product in fp32, in any order and with the tensor
cores' truncating adds: at most 256 u S off, and each weight then at most
twice that, relative. Sums over n cells in any order: (n + 256) u of the sum
of absolute terms. Results and the weights that enter a product in a 16-bit
type are off by half a step of that type."""
import math

import torch

U = 2.0 ** -24
D = 128


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def attend(q, k, v, seen, scale):
    """q [g, m, D], k, v [n, D], seen [m, n] -> out, lse, weights, sum of
    |weight * value|, largest S over the visible cells (all float64)."""
    q, k, v = q.double(), k.double(), v.double()
    if k.shape[0] == 0:
        z = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        return z, torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device), z[..., :0], z, z[..., 0]
    # what is not seen takes no part, whatever it holds
    some = seen.any(0)
    k, v = torch.where(some[:, None], k, 0.0), torch.where(some[:, None], v, 0.0)
    x = (q @ k.T * scale).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None]).masked_fill(~seen, 0.0)
    S = ((q.abs() @ k.abs().T) * scale).masked_fill(~seen, 0.0).amax(-1)
    return p @ v, lse, p, p @ v.abs(), S


def bounds(out, lse, size, S, n, dtype, p_half):
    """(tolerance of out, tolerance of lse). n: cells summed; p_half: half
    step of the weights in the product with the values."""
    w = 2 * 256 * U * S + (n + 256) * U
    tiny = 2.0 ** -24 * size.amax() if dtype == torch.float16 and size.numel() else 0.0   # binary16 weights below its normal range
    sub = 2.0 ** -25 if dtype == torch.float16 else 0.0                      # half a subnormal step of the result
    tol = out.abs() * half_step(dtype) + size * (p_half + w[..., None]) * 2 + tiny + sub
    return tol, w + 8 * U * torch.where(lse == -math.inf, 0.0, lse.abs()) + 8 * U


def check(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol) & ~((got.double() == want))
    assert not bad.any(), (what, int(bad.sum()), float((err / tol)[bad].max()), float(err[bad].max()))


def paged_cells(pages, scale, table, n, head, page):
    """Cells 0 .. n-1 of one sequence and head in 64 bits, and whether their page exists."""
    j = torch.arange(n, device=pages.device)
    p = table.long()[j // page]
    ok = (p >= 0) & (p < pages.shape[0])
    x = pages[p.clamp(0, max(pages.shape[0] - 1, 0)), j % page, head].double()
    if scale is not None:
        x = x * scale[p.clamp(0, pages.shape[0] - 1), j % page, head].view(torch.float16).double()[:, None]
    return x, ok


def evict(mass, n, budget, sinks, recent):
    """The kept cells of one sequence, by a plain sort (python numbers)."""
    if n <= budget:
        return list(range(n))
    key = lambda j: (-(mass[j] if mass[j] == mass[j] else -math.inf), j)  # noqa: E731
    mid = sorted(range(sinks, n - recent), key=key)[:budget - sinks - recent]
    return list(range(sinks)) + sorted(mid) + list(range(n - recent, n))
