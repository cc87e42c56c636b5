"""The operators of an expert (or dense) feed-forward block in blocks of 128, measured.

Each case is one pass through one operator, in one of two forms: plain
(elementary torch operations in 32 bits, rounded once at the end), or, with
`own`, the calls that a user makes of this package.

  gemm_experts      D = sum over blocks of K of  s_a s_b (A . B_e^T),  rows by expert
  wgrad_experts     dW_e = sum over blocks of tokens of  s_dy s_x (dY^T . X),  tokens by expert
  act_block         h = act(z) [* z_up] as codes in 1x128 blocks, z kept as codes
  act_block_bwd     its gradient from the kept codes, along rows and along tokens; h^T again
  block_transpose   kept codes of x -> codes of x^T in blocks along the tokens
"""
import math
import random

import torch

own = False

DEV = "cuda"
B = 128                                   # the block of every scale
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
TYPE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ------------------------------------------------------------------ the cases

def gemm_case(name, rows, experts, active, out_features, in_features, align=1, fmt="e4m3", pow2=False,
              out="bf16"):
    """rows: in all, over `active` of the experts (each a multiple of align)."""
    return dict(name=name, op="gemm_experts", rows=rows, experts=experts, active=active,
                out_features=out_features, in_features=in_features, align=align, fmt=fmt, pow2=pow2,
                out=out)


def wgrad_case(name, rows, experts, active, out_features, in_features, pow2=False):
    return dict(name=name, op="wgrad_experts", rows=rows, experts=experts, active=active,
                out_features=out_features, in_features=in_features, align=B, pow2=pow2)


def act_case(name, rows, features, act="silu", gated=True, keep=True):
    return dict(name=name, op="act_block", rows=rows, features=features, act=act, gated=gated, keep=keep)


def act_bwd_case(name, rows, features, act="silu", gated=True, tokens=True, h=True):
    return dict(name=name, op="act_block_bwd", rows=rows, features=features, act=act, gated=gated,
                tokens=tokens, h=h)


def transpose_case(name, rows, features, fmt="e4m3", pow2=False):
    return dict(name=name, op="block_transpose", rows=rows, features=features, fmt=fmt, pow2=pow2)


def listed():
    return [
        # decoding: 16 tokens to 4 of 32 experts, gate and up of 2048 from a width of 7168; the
        # weights' bytes are the floor
        gemm_case("gemm_experts_decode", 64, 32, 28, 4096, 7168),
        # a chunk of a prompt: some 64 rows an expert, ragged
        gemm_case("gemm_experts_chunk", 2043, 32, 31, 4096, 4096),
        # a training batch's gate and up products
        gemm_case("gemm_experts_train", 32768, 32, 31, 4096, 4096, align=B),
        # a training batch's input gradient, E5M2 against E4M3, factors powers of two
        gemm_case("gemm_experts_dgrad_pow2", 16384, 64, 60, 7168, 2048, align=B, fmt="e5m2", pow2=True),
        # weight gradients of a training batch, some 2000 tokens an expert
        wgrad_case("wgrad_experts_train", 32768, 16, 15, 4096, 4096),
        # the same with few tokens an expert, where writing the gradients is the floor
        wgrad_case("wgrad_experts_few_pow2", 8192, 64, 40, 2048, 2048, pow2=True),
        # decoding: the activation between the two products, nothing kept
        act_case("act_block_decode", 64, 2048, keep=False),
        # training: the same with the checkpoint
        act_case("act_block_train", 32768, 2048),
        # a dense block without a gate, row codes only (no weight gradient: frozen weights)
        act_bwd_case("act_block_bwd_dense", 4099, 11008, act="gelu_tanh", gated=False, tokens=False,
                     h=False),
        # training: everything the two dgrads and wgrads read
        act_bwd_case("act_block_bwd_train", 32768, 2048),
        # a small layer's kept input, 256 tokens: latency
        transpose_case("block_transpose_small", 256, 512),
        # the kept input of a training batch
        transpose_case("block_transpose_train", 32768, 7168, pow2=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm_experts", "gemm_experts", "wgrad_experts", "act_block", "act_block_bwd",
                     "block_transpose"])
    if op == "gemm_experts":
        e, n, k = _log(rng, 1, 64), B * _log(rng, 1, 56), B * _log(rng, 1, 56)
        while e > 1 and e * n * k > 1 << 30:
            e //= 2
        align = rng.choice([1, 1, 16, B])
        rows = _log(rng, 1, 32768)
        while rows > 1 and rows * n * k > 32768 * 4096 * 4096:
            rows //= 2
        rows = (rows + align - 1) // align * align
        active = max(1, min(rows // align, int(e * rng.uniform(0.3, 1.0))))
        c = gemm_case("", rows, e, active, n, k, align=align, fmt=rng.choice(["e4m3", "e4m3", "e5m2"]),
                      pow2=rng.random() < 0.4, out=rng.choice(["bf16", "bf16", "f32"]))
    elif op == "wgrad_experts":
        e, n, k = _log(rng, 1, 64), B * _log(rng, 1, 56), B * _log(rng, 1, 56)
        while e > 1 and e * n * k > 1 << 28:
            e //= 2
        blocks = _log(rng, 1, 256)
        while blocks > 1 and blocks * B * n * k > 32768 * 4096 * 4096:
            blocks //= 2
        active = max(1, min(blocks, int(e * rng.uniform(0.3, 1.0))))
        c = wgrad_case("", blocks * B, e, active, n, k, pow2=rng.random() < 0.4)
    else:
        n = B * _log(rng, 1, 86)
        rows = _log(rng, 1, 32768)
        while rows > 1 and rows * n > 32768 * 2048:
            rows //= 2
        act, gated = rng.choice(["silu", "gelu_tanh", "gelu", "relu"]), rng.random() < 0.6
        if op == "act_block":
            c = act_case("", rows, n, act=act, gated=gated, keep=rng.random() < 0.6)
        elif op == "act_block_bwd":
            tokens = rng.random() < 0.7
            if tokens:
                rows = (rows + B - 1) // B * B
            c = act_bwd_case("", rows, n, act=act, gated=gated, tokens=tokens,
                             h=tokens and rng.random() < 0.7)
        else:
            c = transpose_case("", (rows + B - 1) // B * B, n, fmt=rng.choice(["e4m3", "e5m2"]),
                               pow2=rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1013 + 7)
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(std)


def _activations(g, rows, cols):
    """Rows of unequal size, one column in 256 an outlier channel."""
    x = _normal(g, rows, cols)
    x *= 0.5 + torch.rand(rows, 1, generator=g, device=DEV)
    x[:, torch.randperm(cols, generator=g, device=DEV)[:cols // 256]] *= 20.0
    return x


def _offsets(case, seed):
    """Segment starts of the sorted rows: unequal shares over the experts that
    have any, in units of align rows."""
    r = random.Random(seed * 31 + case["experts"])
    unit, active = case["align"], sorted(r.sample(range(case["experts"]), case["active"]))
    share = {e: r.expovariate(1.0) + 0.05 for e in active}
    spare, total, count = case["rows"] // unit - len(active), sum(share.values()), {}
    for e in active:
        count[e] = 1 + int(spare * share[e] / total)
    for e in r.sample(active, len(active)):
        if sum(count.values()) < case["rows"] // unit:
            count[e] += 1
    off = [0]
    for e in range(case["experts"]):
        off.append(off[-1] + unit * count.get(e, 0))
    return off


def _scale(amax, top, pow2):
    """top / amax, of a block of zeros 1; rounded down to a power of two."""
    # (a number over a tensor would be a reciprocal and a product: two roundings)
    s = torch.where(amax > 0, torch.full_like(amax, top) / amax, torch.ones_like(amax))
    return torch.ldexp(torch.ones_like(s), torch.frexp(s).exponent - 1) if pow2 else s


def _rows_1x128(x, fmt, pow2=False):
    """Codes of x in blocks of 128 of each row, as a view of 8-bit floats, and
    the factors that take them back."""
    v = x.view(x.shape[0], -1, B)
    s = _scale(v.abs().amax(dim=2), TOP[fmt], pow2)
    q = (v * s[:, :, None]).clamp_(-TOP[fmt], TOP[fmt]).view(x.shape).to(TYPE[fmt])
    return q, 1.0 / s


def _tiles_128x128(w, fmt, pow2=False):
    """The same of each 128 x 128 tile of w [E, N, K]."""
    e, n, k = w.shape
    v = w.view(e, n // B, B, k // B, B)
    s = _scale(v.abs().amax(dim=(2, 4)), TOP[fmt], pow2)
    q = (v * s[:, :, None, :, None]).clamp_(-TOP[fmt], TOP[fmt]).view(e, n, k).to(TYPE[fmt])
    return q, 1.0 / s


def _codes(pair):
    return pair[0].view(torch.uint8), pair[1].contiguous()


def prepare(case, seed):
    g, op, s = _gen(seed), case["op"], dict(case)
    if op in ("gemm_experts", "wgrad_experts"):
        m, e, n, k, p2 = case["rows"], case["experts"], case["out_features"], case["in_features"], case["pow2"]
        off = _offsets(case, seed)
        s["most"] = max(b - a for a, b in zip(off, off[1:]))
        s["offsets"] = torch.tensor(off, dtype=torch.int32, device=DEV)
        if op == "gemm_experts":
            s["a"], s["sa"] = _codes(_rows_1x128(_activations(g, m, k), case["fmt"], p2))
            s["b"] = torch.empty(e, n, k, dtype=torch.uint8, device=DEV)
            s["sb"] = torch.empty(e, n // B, k // B, device=DEV)
            for i in range(e):
                w = _normal(g, 1, n, k, std=1.0 / math.sqrt(k))
                q, f = _codes(_tiles_128x128(w, "e4m3", p2))
                s["b"][i], s["sb"][i] = q[0], f[0]
        else:
            s["dy_t"], s["s_dy"] = _codes(_rows_1x128(_activations(g, m, n).mul_(1e-3).t().contiguous(), "e5m2", p2))
            s["x_t"], s["s_x"] = _codes(_rows_1x128(_activations(g, m, k).t().contiguous(), "e4m3", p2))
        return s
    m, n = case["rows"], case["features"]
    if op == "block_transpose":
        s["q"], s["inv"] = _codes(_rows_1x128(_activations(g, m, n), case["fmt"], case["pow2"]))
        return s
    z = _normal(g, m, 2 * n if case["gated"] else n, std=1.5)
    z *= 0.5 + torch.rand(m, 1, generator=g, device=DEV)
    if op == "act_block":
        s["z"] = z.to(torch.bfloat16)
    else:
        s["zq"], s["z_inv"] = _codes(_rows_1x128(z.to(torch.bfloat16).float(), "e4m3"))
        s["d"] = _activations(g, m, n).mul_(1e-3).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ plain forms

def _values(q, inv, fmt):
    """The numbers that codes in blocks of 128 of each row stand for."""
    v = q.view(TYPE[fmt]).float()
    return (v.view(v.shape[0], -1, B) * inv[:, :, None]).view(v.shape)


def _places(s, rows):
    """Where each sorted row stands in a block of `most` rows an expert."""
    off = s["offsets"].long()
    at = torch.arange(rows, device=DEV)
    e = torch.searchsorted(off, at, right=True) - 1
    return e * s["most"] + at - off[e]


def _plain_gemm(s):
    e, n, k = s["b"].shape
    a = _values(s["a"], s["sa"], s["fmt"])
    b = s["b"].view(TYPE["e4m3"]).float().view(e, n // B, B, k // B, B)
    b = (b * s["sb"][:, :, None, :, None]).view(e, n, k)
    at = _places(s, a.shape[0])
    full = a.new_zeros(e * s["most"], k)
    full[at] = a
    d = torch.bmm(full.view(e, s["most"], k), b.transpose(1, 2)).view(-1, n)[at]
    return {"d": d if s["out"] == "f32" else d.to(torch.bfloat16)}


def _plain_wgrad(s):
    e, most = s["experts"], s["most"]
    dy, x = _values(s["dy_t"], s["s_dy"], "e5m2"), _values(s["x_t"], s["s_x"], "e4m3")
    at = _places(s, dy.shape[1])
    full_dy, full_x = dy.new_zeros(dy.shape[0], e * most), x.new_zeros(x.shape[0], e * most)
    full_dy[:, at], full_x[:, at] = dy, x
    return {"dw": torch.bmm(full_dy.view(-1, e, most).transpose(0, 1),
                            full_x.view(-1, e, most).permute(1, 2, 0))}


def _act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_grad(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _plain_act(s):
    z, n = s["z"].float(), s["features"]
    h = _act(z[:, :n], s["act"])
    if s["gated"]:
        h = h * z[:, n:]
    r = {}
    r["q"], r["inv"] = _rows_1x128(h, "e4m3")
    if s["keep"]:
        r["zq"], r["z_inv"] = _rows_1x128(z, "e4m3")
    return r


def _plain_act_bwd(s):
    z, d, n = _values(s["zq"], s["z_inv"], "e4m3"), s["d"].float(), s["features"]
    g, h = _act_grad(z[:, :n], s["act"]), _act(z[:, :n], s["act"])
    if s["gated"]:
        dz = torch.cat([d * z[:, n:] * g, d * h], dim=1)
        h = h * z[:, n:]
    else:
        dz = d * g
    r = {}
    r["q"], r["inv"] = _rows_1x128(dz, "e5m2")
    if s["tokens"]:
        r["q_t"], r["inv_t"] = _rows_1x128(dz.t().contiguous(), "e5m2")
    if s["h"]:
        r["h_t"], r["h_inv_t"] = _rows_1x128(h.t().contiguous(), "e4m3")
    return r


def _plain_transpose(s):
    x = _values(s["q"], s["inv"], s["fmt"])
    q, inv = _rows_1x128(x.t().contiguous(), s["fmt"], s["pow2"])
    return {"q_t": q, "inv_t": inv}


PLAIN = {"gemm_experts": _plain_gemm, "wgrad_experts": _plain_wgrad, "act_block": _plain_act,
         "act_block_bwd": _plain_act_bwd, "block_transpose": _plain_transpose}


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import scaled_fp8_linear_gb300 as F
    op = s["op"]
    f = {"e4m3": F.E4M3, "e5m2": F.E5M2}
    if op == "gemm_experts":
        return {"d": F.fp8_gemm_experts(s["a"], f[s["fmt"]], s["b"], F.E4M3, s["sa"], s["sb"], s["offsets"],
                                        out=F.OUT_F32 if s["out"] == "f32" else F.OUT_BF16, pow2=s["pow2"])}
    if op == "wgrad_experts":
        return {"dw": F.fp8_wgrad_experts(s["dy_t"], F.E5M2, s["x_t"], F.E4M3, s["s_dy"], s["s_x"],
                                          s["offsets"], pow2=s["pow2"])}
    if op == "block_transpose":
        q, inv = F.fp8_block_transpose(s["q"], f[s["fmt"]], s["inv"], pow2=s["pow2"])
        return {"q_t": q.view(TYPE[s["fmt"]]), "inv_t": inv}
    act = {"relu": F.ACT_RELU, "silu": F.ACT_SILU, "gelu": F.ACT_GELU, "gelu_tanh": F.ACT_GELU_TANH}[s["act"]]
    if op == "act_block":
        o = F.fp8_act_block(s["z"], act, gated=s["gated"], keep=s["keep"])
        r = {"q": o.q.view(TYPE["e4m3"]), "inv": o.scale_inv}
        if s["keep"]:
            r["zq"], r["z_inv"] = o.z_q.view(TYPE["e4m3"]), o.z_scale_inv
        return r
    o = F.fp8_act_block_bwd(s["d"], s["zq"], s["z_inv"], act, gated=s["gated"], want_t=s["tokens"],
                            want_h_t=s["h"])
    r = {"q": o.q.view(TYPE["e5m2"]), "inv": o.scale_inv}
    if s["tokens"]:
        r["q_t"], r["inv_t"] = o.q_t.view(TYPE["e5m2"]), o.scale_inv_t
    if s["h"]:
        r["h_t"], r["h_inv_t"] = o.h_t.view(TYPE["e4m3"]), o.h_scale_inv_t
    return r


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ------------------------------------------------------------------ what a pass has to do

def work(case):
    op, m = case["op"], case["rows"]
    if op in ("gemm_experts", "wgrad_experts"):
        n, k, e = case["out_features"], case["in_features"], case["experts"]
        if op == "gemm_experts":   # the weights of the experts that have rows
            b = m * k + case["active"] * n * k + m * n * (4 if case["out"] == "f32" else 2)
            b += (m + case["active"] * n // B) * k // B * 4
        else:
            b = m * (n + k) + (n + k) * m // B * 4 + e * n * k * 4
        return {"bytes": b + (e + 1) * 4, "flops": 2 * m * n * k}
    n = case["features"]
    if op == "block_transpose":
        return {"bytes": 2 * m * n + 8 * m * n // B, "flops": 3 * m * n}
    w = 2 * n if case["gated"] else n
    if op == "act_block":
        b = 2 * m * w + m * n + 4 * m * n // B + (m * w + 4 * m * w // B if case["keep"] else 0)
        return {"bytes": b, "flops": 12 * m * n}
    b = 2 * m * n + (m * w + 4 * m * w // B) * (2 + case["tokens"]) + (m * n + 4 * m * n // B) * case["h"]
    return {"bytes": b, "flops": 25 * m * n}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_values(q, inv, fmt):
    return q.view(TYPE[fmt]).double() * inv.double().repeat_interleave(B, dim=1)


def _exact_cast(x, fmt, pow2=False):
    """The 8-bit number next to x over its block's factor, and the factors."""
    top = x.unflatten(1, (-1, B)).abs().amax(2)
    inv = torch.where(top > 0, top / TOP[fmt], torch.ones_like(top))
    if pow2:
        part, power = torch.frexp(inv)   # the least power of two that is not below
        inv = torch.ldexp(torch.ones_like(inv), power - (part == 0.5).int())
    v = x / inv.repeat_interleave(B, dim=1)
    mantissa, least = {"e4m3": (3, -6), "e5m2": (2, -14)}[fmt]
    power = (torch.frexp(v).exponent - 1).clamp_min(least) - mantissa
    step = torch.ldexp(torch.ones_like(v), power)   # between neighbours; ties go to even
    return (torch.round(v / step) * step).clamp(-TOP[fmt], TOP[fmt]), inv


def _exact_act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "gemm_experts":
        off = s["offsets"].tolist()
        d = torch.zeros(case["rows"], case["out_features"], dtype=torch.float64, device=DEV)
        for e, (a, b) in enumerate(zip(off, off[1:])):
            if b > a:
                x = _exact_values(s["a"][a:b], s["sa"][a:b], case["fmt"])
                w = _exact_values(s["b"][e], s["sb"][e].repeat_interleave(B, dim=0), "e4m3")
                d[a:b] = x @ w.t()
        return {"d": d}
    if op == "wgrad_experts":
        off = s["offsets"].tolist()
        dw = torch.zeros(case["experts"], case["out_features"], case["in_features"], dtype=torch.float64, device=DEV)
        dy, x = _exact_values(s["dy_t"], s["s_dy"], "e5m2"), _exact_values(s["x_t"], s["s_x"], "e4m3")
        for e, (a, b) in enumerate(zip(off, off[1:])):
            if b > a:
                dw[e] = dy[:, a:b] @ x[:, a:b].t()
        return {"dw": dw}
    if op == "block_transpose":
        q, inv = _exact_cast(_exact_values(s["q"], s["inv"], case["fmt"]).t().contiguous(), case["fmt"], case["pow2"])
        return {"q_t": q, "inv_t": inv}
    n = case["features"]
    z = s["z"].double() if op == "act_block" else _exact_values(s["zq"], s["z_inv"], "e4m3")
    zg = z[:, :n].clone()
    if op == "act_block":
        h = _exact_act(zg, case["act"])
        r = {}
        r["q"], r["inv"] = _exact_cast(h * z[:, n:] if case["gated"] else h, "e4m3")
        if case["keep"]:
            r["zq"], r["z_inv"] = _exact_cast(z, "e4m3")
        return r
    zg.requires_grad_(True)
    with torch.enable_grad():
        h = _exact_act(zg, case["act"])
    grad, = torch.autograd.grad(h, zg, torch.ones_like(h))
    h, d = h.detach(), s["d"].double()
    dz = torch.cat([d * z[:, n:] * grad, d * h], 1) if case["gated"] else d * grad
    r = {}
    r["q"], r["inv"] = _exact_cast(dz, "e5m2")
    if case["tokens"]:
        r["q_t"], r["inv_t"] = _exact_cast(dz.t().contiguous(), "e5m2")
    if case["h"]:
        r["h_t"], r["h_inv_t"] = _exact_cast((h * z[:, n:] if case["gated"] else h).t().contiguous(), "e4m3")
    return r
