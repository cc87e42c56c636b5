"""64-bit references of the operators between the linears, and the bounds
their kernels are held to.

Bounds: a bf16 output is one rounding to nearest even (2^-8 of the value).
Everything before it is fp32 (unit roundoff 2^-24); a row's statistics are
sums of at most 2^14 terms in a tree (32 terms a thread, two shuffle trees:
under 64 roundings), and an element sees fewer than 16 further operations, so
its error is below 2^-17 of the sum of the magnitudes that make it up, which
every reference returns beside the value."""
import math

import torch

F64 = torch.float64
U_BF16, U_F32 = 2.0 ** -8, 2.0 ** -17


def check(got, ref, mag, what, extra=None):
    """|got - ref| <= u |ref| + 2^-17 mag (+ extra), u by got's type."""
    g = got.detach().to(F64).cpu()
    ref, mag = ref.cpu(), mag.cpu()
    tol = U_F32 * mag
    if got.dtype == torch.bfloat16:
        tol = tol + U_BF16 * (ref.abs() + tol)
    if extra is not None:
        tol = tol + extra.cpu()
    bad = ~((g - ref).abs() <= tol)
    assert g.shape == ref.shape, f"{what}: shape {tuple(g.shape)}, expected {tuple(ref.shape)}"
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {i}: got "
                             f"{g[i]}, want {ref[i]}, tolerance {tol[i]}")


def check_codes(q, fmt, v, tol, what):
    """FP8 codes q of values v that are known to within tol: half a step of
    the format, saturating."""
    dt, top, mant, low = ((torch.float8_e4m3fn, 448.0, 3, -6) if fmt == 0 else
                          (torch.float8_e5m2, 57344.0, 2, -14))
    got = q.view(dt).to(F64).cpu()
    v, tol = v.cpu().clamp(-top, top), tol.cpu()
    half = 2.0 ** (torch.floor(torch.log2(v.abs().clamp_min(2.0 ** low))) - mant - 1)
    # a step doubles at a power of two, which v may reach within tol
    ok = (got - v).abs() <= 2 * half * ((v.abs() + tol) >= 2 ** (mant + 2) * half) + half + tol
    assert ok.all(), f"{what}: {int((~ok).sum())} codes of {ok.numel()} off"


def norm(v, kind, w, b, eps, mag):
    """N(v; w, b), its magnitude (v known to within 2^-24-ish of mag), mean, rstd."""
    mean = v.mean(dim=1, keepdim=True) if kind == 1 else torch.zeros_like(v[:, :1])
    r = 1.0 / torch.sqrt(((v - mean) ** 2).mean(dim=1, keepdim=True) + eps)
    n, u = (v - mean) * r, (mag + mean.abs() + mag.mean(dim=1, keepdim=True)) * r
    # an error of v's elements moves the statistics as well
    u = u + n.abs() * (1 + (u * n.abs()).mean(dim=1, keepdim=True))
    if w is not None:
        n, u = n * w, u * w.abs()
    if b is not None:
        n, u = n + b, u + b.abs()
    return n, u, mean[:, 0], r[:, 0]


def spread(gate, T):
    return gate.repeat_interleave(T // gate.shape[0], dim=0)


def norm_fwd(x, h, gate, kind, eps, alpha, post, w_post, b_post, w_pre, b_pre):
    ref = x if x is not None else h
    T = ref.shape[0]
    z = torch.zeros(ref.shape, dtype=F64)
    p, pm = (z, z) if h is None else (h, h.abs())
    mp = rp = torch.zeros(T, dtype=F64)
    if post:
        p, pm, mp, rp = norm(p, kind, w_post, b_post, eps, pm)
    if gate is not None:
        p, pm = p * spread(gate, T), pm * spread(gate, T).abs()
    xo, xm = p, pm
    if x is not None:
        xo, xm = alpha * x + p, abs(alpha) * x.abs() + pm
    y, ym, m, r = norm(xo, kind, w_pre, b_pre, eps, xm)
    return xo, xm, y, ym, torch.stack([mp, rp, m, r])


def _through(g, gm, u, um, r, kind):
    """The norm's own gradient and its magnitude."""
    c1, c2 = (g * u).mean(1, keepdim=True), (gm * um).mean(1, keepdim=True)
    c0, c3 = ((g.mean(1, keepdim=True), gm.mean(1, keepdim=True)) if kind == 1 else (0.0, 0.0))
    return r * (g - c0 - u * c1), r.abs() * (gm + c3 + um * c2)


def norm_bwd(dy, x_out, dx_out, h, gate, stats, kind, alpha, post, w_post, b_post, w_pre):
    """{name: (gradient, magnitude)}, from the statistics as stored."""
    T = x_out.shape[0]
    mp, rp, m, r = (s[:, None] for s in stats)
    out = {}
    dX = torch.zeros_like(x_out) if dx_out is None else dx_out
    dM = dX.abs()
    if dy is not None:
        u, um = (x_out - m) * r, (x_out.abs() + m.abs()) * r
        out["dw_pre"] = ((dy * u).sum(0), (dy.abs() * um).sum(0))
        out["db_pre"] = (dy.sum(0), dy.abs().sum(0))
        w = torch.ones_like(x_out[0]) if w_pre is None else w_pre
        d, dm = _through(dy * w, dy.abs() * w.abs(), u, um, r, kind)
        dX, dM = dX + d, dM + dm
    out["dx"] = (alpha * dX, abs(alpha) * dM)
    if h is None:
        return out
    hh, hm = (h, h.abs()) if not post else ((h - mp) * rp, (h.abs() + mp.abs()) * rp)
    w = torch.ones_like(h[0]) if w_post is None else w_post
    p, pm = (hh * w, hm * w.abs()) if post else (hh, hm)
    if b_post is not None:
        p, pm = p + b_post, pm + b_post.abs()
    if gate is not None:
        G = gate.shape[0]
        out["dgate"] = ((dX * p).view(G, -1, h.shape[1]).sum(1), (dM * pm).view(G, -1, h.shape[1]).sum(1))
        dX, dM = dX * spread(gate, T), dM * spread(gate, T).abs()
    if post:
        out["dw_post"] = ((dX * hh).sum(0), (dM * hm).sum(0))
        out["db_post"] = (dX.sum(0), dM.sum(0))
        dX, dM = _through(dX * w, dM * w.abs(), hh, hm, rp, kind)
    out["dh"] = (dX, dM)
    return out


def act(z, a):
    if a == 1:
        return z.clamp_min(0)
    if a == 2:
        return z * torch.sigmoid(z)
    if a == 3:
        return z * 0.5 * torch.erfc(-z * math.sqrt(0.5))
    if a == 4:
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def act_grad(z, a):
    if a == 1:
        return (z > 0).to(z.dtype)
    if a == 2:
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if a == 3:
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if a == 4:
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def plan(ids, experts, align, rows):
    """The plan by a walk over the slots."""
    T, k = ids.shape
    places = [[] for _ in range(experts)]
    for i, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < experts:
            places[e].append(i)
    offsets, src = [0], []
    for p in places:
        src += p + [-1] * (-len(p) % align)
        offsets.append(len(src))
    src += [-1] * (rows - len(src))
    row_of = [-1] * (T * k)
    for r, i in enumerate(src):
        if i >= 0:
            row_of[i] = r
    i32 = torch.int32
    return (torch.tensor(offsets, dtype=i32), torch.tensor([len(p) for p in places], dtype=i32),
            torch.tensor(row_of, dtype=i32).view(T, k), torch.tensor(src, dtype=i32))
