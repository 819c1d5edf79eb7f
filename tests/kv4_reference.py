"""The 4-bit cache, its attention and the rotary positions from their definitions, in 64 bits
(no code shared with the library)."""
import math

import torch

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
EVEN_FIRST = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7])   # codes of equal distance: the even one is found first


def quantised(x, unit=1.0):
    """The values that rows x [.., D] have in the cache, in float64."""
    y = (x.detach().cpu().float() / torch.tensor(unit, dtype=torch.float32)).unflatten(-1, (-1, 16))
    finite = torch.isfinite(y).all(-1, keepdim=True)
    most = torch.where(finite, y, 0.0).abs().amax(-1, keepdim=True)
    scale = (most / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).double()
    ratio = torch.where(scale > 0, y.double().abs() / scale, 0.0)
    ratio = torch.where(finite, ratio, 0.0)
    code = EVEN_FIRST[(ratio.unsqueeze(-1) - LEVELS[EVEN_FIRST]).abs().argmin(-1)]
    v = (torch.sign(y.double()) * LEVELS[code] * scale).float() * torch.tensor(unit, dtype=torch.float32)
    return torch.where(finite, v, math.nan).flatten(-2).double()


def attention(q, k, v, scale, window=0):
    """q [n, Hq, D], the newest n of the cached k, v [ctx, Hkv, D]; float64.  NaN counts where it is seen."""
    n, Hq, D = q.shape
    ctx, Hkv = k.shape[:2]
    out = torch.zeros(n, Hq, D, dtype=torch.float64)
    for i in range(n):
        hi = ctx - n + 1 + i
        lo = max(0, hi - window) if window else 0
        if hi <= 0 or hi <= lo:
            continue
        for h in range(Hkv):
            g = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            w = torch.softmax(q[i, g].double() @ k[lo:hi, h].T * scale, -1)
            out[i, g] = w @ v[lo:hi, h]
    return out


def tolerance(ref, q, k, v, scale, dtype):
    """What the kernel's roundings come to.  Weights enter P . V in f16: 2^-11 of each.  A score is a sum of D
    products that are exact in 32 bits, each addition off by at most 2^-23 of the sum of magnitudes S, and a
    relative error of a weight counts in the sum above and below: 2 (D 2^-23 S + 2^-20).  One rounding of the output."""
    k, v = torch.nan_to_num(k, 0, 0, 0), torch.nan_to_num(v, 0, 0, 0)
    if k.shape[0] == 0:
        return torch.zeros_like(ref)
    D = q.shape[-1]
    S = abs(scale) * float(q.double().abs().amax() * k.abs().sum(-1).amax())
    return (2.0 ** -11 + 2 * (D * 2.0 ** -23 * S + 2.0 ** -20)) * float(v.abs().amax()) + \
        torch.finfo(dtype).eps / 2 * ref.abs() + torch.finfo(dtype).tiny


def rotated(x, positions, frequencies, magnitude=1.0, interleaved=False):
    """Rows x [T, H, D] turned, in float64 (angles by exact integer positions)."""
    half = len(frequencies)
    angle = positions.cpu().double()[:, None] * torch.as_tensor(frequencies, dtype=torch.float64)
    c, s = (magnitude * torch.cos(angle))[:, None], (magnitude * torch.sin(angle))[:, None]
    y = x.detach().cpu().double()
    r, rest = y[..., :2 * half], y[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    a, b = a * c - b * s, b * c + a * s
    return torch.cat((torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1), rest), -1)
