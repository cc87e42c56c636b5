"""64-bit references of the experts' products and the activations in blocks of
128, and exact inputs.

Exact inputs: codes of whole numbers up to 4 in magnitude and factors of 1/4
to 4.  Every product of two with its factors is a multiple of 2^-4, and a sum
of 2^12 such terms stays below 2^4 2^4 2^12 = 2^20, 2^24 units: FP32 holds each partial sum
exactly, in whatever order, so results are compared bit for bit."""
import torch

F64 = torch.float64
TOP = {0: 448.0, 1: 57344.0}
TYPE = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}


def held(off, M):
    """Offsets as the calls take them: within 0..M, never falling."""
    out, top = [], 0
    for o in off:
        top = max(top, min(max(o, 0), M))
        out.append(top)
    return out


def values(q, fmt):
    return q.cpu().view(TYPE[fmt]).to(F64)


def by_rows(q, inv, fmt):
    """What codes with 1x128 factors stand for."""
    return values(q, fmt) * inv.cpu().to(F64).repeat_interleave(128, dim=1)


def by_tiles(q, inv, fmt):
    """The same of [E, N, K] with 128x128 factors."""
    return values(q, fmt) * inv.cpu().to(F64).repeat_interleave(128, dim=1).repeat_interleave(128, dim=2)


def exact_codes(g, fmt, *shape):
    return torch.randint(-4, 5, shape, generator=g).float().to(TYPE[fmt]).view(torch.uint8)


def exact_factors(g, *shape):
    return 2.0 ** torch.randint(-2, 3, shape, generator=g).float()


def any_codes(g, fmt, *shape):
    """Codes over the whole range, none of them NaN or infinite."""
    top = 0x7F if fmt == 0 else 0x7C
    return (torch.randint(0, top, shape, generator=g) | torch.randint(0, 2, shape, generator=g) * 0x80).to(torch.uint8)


def products(a, b, off):
    """(rows by expert of a . b_e^T, sums of magnitudes, the rows that are experts')."""
    at = held(off, a.shape[0])
    d = torch.zeros(a.shape[0], b.shape[1], dtype=F64)
    mag = torch.zeros_like(d)
    live = torch.zeros(a.shape[0], dtype=torch.bool)
    for e, (x, y) in enumerate(zip(at, at[1:])):
        d[x:y], mag[x:y] = a[x:y] @ b[e].t(), a[x:y].abs() @ b[e].abs().t()
        live[x:y] = True
    return d, mag, live


def cast(v, fmt, pow2):
    """FP32 v [rows, cols] in 1x128 blocks by the casts' rule: (codes, factors)."""
    b = v.unflatten(1, (-1, 128))
    top = b.abs().amax(2)
    # divided by a tensor: a number over a tensor would be rounded twice
    s = torch.where((top > 0) & torch.isfinite(top), torch.full_like(top, TOP[fmt]) / top, torch.ones_like(top))
    s = s.clamp(2.0 ** -126, torch.finfo(torch.float32).max)
    if pow2:
        s = (s.view(torch.int32) & 0x7F800000).view(torch.float32)
    c = (b * s[..., None]).flatten(1)
    nan = torch.isnan(c)
    q = c.clamp(-TOP[fmt], TOP[fmt]).to(TYPE[fmt]).view(torch.uint8)
    return torch.where(nan, torch.full_like(q, 0x7F), q), 1.0 / s
