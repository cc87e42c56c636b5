"""The operators between the FP8 linears of a feed-forward block, measured.

Each case is one pass through one operator, in one of two forms: plain
(elementary torch operations in 32 bits, rounded once at the end), or, with
`own`, the calls that a user makes of this package.

  norm_fwd / norm_bwd   x' = alpha x + gate * N_post(h),  y = N_pre(x')
  gemm_act / act_bwd    z = s_a s_b A B^T + bias,  D = act(z) [* z_up] + residual
  moe_dispatch          tokens sorted by expert (stable), rows copied
  moe_combine[_bwd]     the weighted sum back per token, and its gradient
"""
import math

import torch

own = False

E4M3_MAX, E5M2_MAX = 448.0, 57344.0
EPS = 1e-5
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def norm_case(name, op, tokens, width, kind="rms", stream="bf16", post=False, gate_rows=0,
              alpha=1.0, out="bf16"):
    return dict(name=name, op=op, tokens=tokens, width=width, kind=kind, stream=stream, post=post,
                gate_rows=gate_rows, alpha=alpha, out=out)


def gemm_case(name, tokens, out_features, in_features, act="none", gated=False, bias=False,
              residual=False, save_z=False, gran="tensor", out="bf16", experts=0):
    return dict(name=name, op="gemm_act", tokens=tokens, out_features=out_features,
                in_features=in_features, act=act, gated=gated, bias=bias, residual=residual,
                save_z=save_z, gran=gran, out=out, experts=experts)


def act_case(name, tokens, features, act="silu", gated=True, out="bf16", bias=False):
    return dict(name=name, op="act_bwd", tokens=tokens, features=features, act=act, gated=gated,
                out=out, bias=bias)


def moe_case(name, op, tokens, k, experts, width, dtype="bf16", align=16, dropped=0.0):
    return dict(name=name, op=op, tokens=tokens, k=k, experts=experts, width=width, dtype=dtype,
                align=align, dropped=dropped)


def listed():
    return [
        # a decoding step's residual add and pre-norm: latency
        norm_case("norm_fwd_decode", "norm_fwd", 8, 4096),
        # a training step's sandwich norm with a learned per-channel gate, hidden size of the
        # benchmark's larger linears
        norm_case("norm_fwd_sandwich", "norm_fwd", 8192, 8192, post=True, gate_rows=1),
        # an FP32 residual stream, layer norm, codes for the next per-token-scaled linear; a
        # ragged token count
        norm_case("norm_fwd_fp8", "norm_fwd", 4099, 7168, kind="layer", stream="f32", alpha=0.81,
                  out="fp8_row"),
        # its backward: norms' weights, a gate per sequence
        norm_case("norm_bwd_sandwich", "norm_bwd", 8192, 4096, post=True, gate_rows=4),
        # the benchmark's small layer with everything in the epilogue
        gemm_case("gemm_small_gelu", 256, 512, 512, act="gelu_tanh", bias=True, residual=True),
        # the benchmark's gate and up linears as one gated product, training (z is kept)
        gemm_case("gemm_gated_train", 4096, 28672, 8192, act="silu", gated=True, save_z=True),
        # the benchmark's down linear onto the residual stream; ragged tokens, per-row factors
        gemm_case("gemm_down_residual", 4099, 8192, 28672, residual=True, gran="row"),
        # one gated product per expert over sorted rows, codes for the experts' second product
        gemm_case("gemm_experts_fp8", 8192, 2048, 4096, act="silu", gated=True, out="fp8",
                  experts=32),
        # gradient of a gated product, E5M2 codes for its dgrad and wgrad
        act_case("act_bwd_gated_fp8", 8192, 11008, out="fp8"),
        # routing of a few decoded tokens: latency
        moe_case("moe_dispatch_decode", "moe_dispatch", 16, 2, 8, 4096),
        # routing of a training batch, some tokens over capacity
        moe_case("moe_dispatch_train", "moe_dispatch", 8192, 8, 64, 4096, align=32, dropped=0.01),
        # the weighted sum's gradient, wide rows
        moe_case("moe_combine_bwd", "moe_combine_bwd", 8191, 8, 256, 7168, align=32, dropped=0.01),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "gemm_act", "act_bwd", "moe_dispatch", "moe_combine",
                     "moe_combine_bwd"])
    if op in ("norm_fwd", "norm_bwd"):
        width = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            width = (width + 63) // 64 * 64
        groups = rng.choice([0, 0, 1, 2, 4, 8])
        tokens = _log(rng, 1, 8192)
        if groups > 1:
            tokens = max(1, tokens // groups) * groups
        c = norm_case("", op, tokens, width, kind=rng.choice(["rms", "layer"]),
                      stream=rng.choice(["bf16", "f32"]), post=rng.random() < 0.5,
                      gate_rows=groups, alpha=rng.choice([1.0, round(rng.uniform(0.3, 2.0), 3)]),
                      out=rng.choice(["bf16", "fp8", "fp8_row"]) if op == "norm_fwd" else "bf16")
    elif op == "gemm_act":
        gated = rng.random() < 0.5
        experts = rng.choice([0, 0, _log(rng, 2, 64)])
        n = 16 * _log(rng, 4, 512)
        k = 16 * _log(rng, 4, 512)
        c = gemm_case("", _log(rng, 1, 8192), n, k,
                      act=rng.choice(["silu", "gelu_tanh", "gelu", "relu"] + ([] if gated else ["none"])),
                      gated=gated, bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                      save_z=rng.random() < 0.5, gran=rng.choice(["tensor", "row"]),
                      out=rng.choice(["bf16", "fp8"]), experts=experts)
        if experts and 2 * n * k * experts > 1 << 30:
            c["experts"] = 2
    elif op == "act_bwd":
        c = act_case("", _log(rng, 1, 8192), 16 * _log(rng, 4, 688),
                     act=rng.choice(["silu", "gelu_tanh", "gelu", "relu"]),
                     gated=rng.random() < 0.5, out=rng.choice(["bf16", "fp8"]),
                     bias=rng.random() < 0.5)
    else:
        experts = _log(rng, 4, 256)
        width = _log(rng, 64, 7168)
        if rng.random() < 0.7:
            width = (width + 63) // 64 * 64
        c = moe_case("", op, _log(rng, 1, 8192), rng.randint(1, min(8, experts)), experts, width,
                     dtype=rng.choice(["bf16", "f32", "fp8"]) if op == "moe_dispatch" else
                     rng.choice(["bf16", "f32"]), align=rng.choice([1, 16, 32, 128]),
                     dropped=rng.choice([0.0, 0.02]))
        while c["tokens"] * c["k"] * c["width"] * (4 if c["dtype"] == "f32" else 2) > 1 << 30:
            c["tokens"] = c["tokens"] // 2
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs

def _gen(seed, salt=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1009 + salt)
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(std)


def _activations(g, rows, cols):
    """Rows of unequal size, one column in 256 an outlier channel."""
    x = _normal(g, rows, cols)
    x *= 0.5 + torch.rand(rows, 1, generator=g, device=DEV)
    ch = torch.randperm(cols, generator=g, device=DEV)[:cols // 256]
    x[:, ch] *= 20.0
    return x


def _e4m3(x, gran):
    """Codes of x and the factors to take them back with."""
    amax = x.abs().amax(dim=1) if gran == "row" else x.abs().amax().reshape(1)
    inv = (amax / E4M3_MAX).clamp_min(1e-30)
    q = (x / (inv[:, None] if gran == "row" else inv)).clamp_(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn).view(torch.uint8), inv


def _stream_type(case):
    return torch.float32 if case["stream"] == "f32" else torch.bfloat16


def _offsets(seed, tokens, experts):
    """Segment starts of the sorted rows, each a multiple of 32: unequal
    shares, one expert in eight without rows."""
    import random
    r = random.Random(seed * 31 + experts)
    share = [0.0 if r.random() < 0.125 else r.expovariate(1.0) + 0.05 for _ in range(experts)]
    if not any(share):
        share[0] = 1.0
    off = [0]
    for s in share:
        off.append(off[-1] + (int(tokens * s / sum(share)) + 31) // 32 * 32)
    if off[-1] == 0:
        off = [0] + [32] * experts
    return off


def _routing(case, g):
    t, k, e = case["tokens"], case["k"], case["experts"]
    # unequal popularity, k different experts a token
    logits = torch.rand(t, e, generator=g, device=DEV).clamp_min_(1e-9).log_().neg_()
    logits /= 0.25 + torch.rand(e, generator=g, device=DEV)
    w, ids = logits.neg_().softmax(dim=1).topk(k, dim=1)
    ids = ids.to(torch.int32)
    if case["dropped"]:
        ids[torch.rand(t, k, generator=g, device=DEV) < case["dropped"]] = -1
    return ids, (w / w.sum(dim=1, keepdim=True)).contiguous()


def _capacity(case):
    n = case["tokens"] * case["k"]
    return n + min(n, case["experts"]) * (case["align"] - 1)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op in ("norm_fwd", "norm_bwd"):
        t, c, gr = case["tokens"], case["width"], case["gate_rows"]
        st = _stream_type(case)
        layer = case["kind"] == "layer"
        s["x"] = _activations(g, t, c).to(st)
        s["h"] = _activations(g, t, c).mul_(0.7).to(torch.bfloat16)
        s["gate"] = _normal(g, gr, c, std=0.3).to(torch.bfloat16) if gr else None
        s["w_pre"] = (1 + _normal(g, c, std=0.1))
        s["b_pre"] = _normal(g, c, std=0.1) if layer else None
        s["w_post"] = (1 + _normal(g, c, std=0.1)) if case["post"] else None
        s["b_post"] = _normal(g, c, std=0.1) if case["post"] and layer else None
        s["y_scale"] = torch.full((1,), 24.0, device=DEV)
        if op == "norm_bwd":
            x_out, stats = _norm_stats(s)
            s["x_out"], s["stats"] = x_out.to(st), stats
            s["x"] = None
            s["dy"] = _activations(g, t, c).mul_(1e-3).to(torch.bfloat16)
            s["dx_out"] = _normal(g, t, c, std=1e-3).to(st)
    elif op == "gemm_act":
        m, n, k, e = case["tokens"], case["out_features"], case["in_features"], case["experts"]
        s["offsets"] = None
        if e:
            off = _offsets(seed, m, e)
            m = off[-1]
            s["most"] = max(b - a for a, b in zip(off, off[1:]))
            s["offsets"] = torch.tensor(off, dtype=torch.int32, device=DEV)
        rows = n * (2 if case["gated"] else 1)
        s["a"], s["sa"] = _e4m3(_activations(g, m, k), case["gran"])
        b = _normal(g, max(1, e) * rows, k, std=1.0 / math.sqrt(k))
        s["b"], s["sb"] = _e4m3(b, case["gran"])
        del b
        if e:
            s["b"] = s["b"].view(e, rows, k)
            s["sb"] = s["sb"].view(e, rows) if case["gran"] == "row" else s["sb"].repeat(e)
        s["bias_v"] = (_normal(g, max(1, e), rows, std=0.2).to(torch.bfloat16)
                       if case["bias"] else None)
        if case["bias"] and not e:
            s["bias_v"] = s["bias_v"].view(rows)
        s["res"] = _activations(g, m, n).to(torch.bfloat16) if case["residual"] else None
        s["q_scale"] = torch.full((1,), 30.0, device=DEV)
    elif op == "act_bwd":
        m, n = case["tokens"], case["features"]
        s["d"] = _activations(g, m, n).mul_(1e-3).to(torch.bfloat16)
        s["z"] = _normal(g, m, 2 * n if case["gated"] else n, std=1.5).to(torch.bfloat16)
        s["q_scale"] = torch.full((1,), 2e5, device=DEV)
    else:
        t, c = case["tokens"], case["width"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["ids"], s["w"] = _routing(case, g)
        if op == "moe_dispatch":
            x = _activations(g, t, c)
            s["scale"] = None
            if case["dtype"] == "fp8":
                s["x"], s["scale"] = _e4m3(x, "row")
            else:
                s["x"] = x.to(dt)
        else:
            _, _, s["row_of"], s["src"], _ = _plain_plan(s["ids"], case["experts"], case["align"],
                                                         _capacity(case))
            s["ys"] = _activations(g, s["src"].numel(), c).to(dt)
            s["dy"] = _activations(g, t, c).mul_(1e-3).to(dt)
    return s


# ------------------------------------------------------------------ plain forms

def _norm(v, kind, w, b):
    if kind == "layer":
        mean = v.mean(dim=1, keepdim=True)
        c = v - mean
    else:
        mean = torch.zeros_like(v[:, :1])
        c = v
    r = 1.0 / torch.sqrt((c * c).mean(dim=1, keepdim=True) + EPS)
    n = c * r
    if w is not None:
        n = n * w.to(v.dtype)
    if b is not None:
        n = n + b.to(v.dtype)
    return n, mean[:, 0], r[:, 0]


def _gate_rows(gate, tokens, dtype):
    if gate is None:
        return None
    g = gate.to(dtype)
    return g if g.shape[0] == 1 else g.repeat_interleave(tokens // g.shape[0], dim=0)


def _norm_stats(s):
    """x' (unrounded) and the rows' statistics: mean_post, rstd_post, mean_pre, rstd_pre."""
    h = s["h"].float()
    zero = torch.zeros(h.shape[0], device=h.device)
    p, mp, rp = h, zero, zero
    if s["post"]:
        p, mp, rp = _norm(h, s["kind"], s["w_post"], s["b_post"])
    g = _gate_rows(s["gate"], h.shape[0], torch.float32)
    x_out = s["alpha"] * s["x"].float() + (p if g is None else g * p)
    _, m, r = _norm(x_out, s["kind"], None, None)
    return x_out, torch.stack([mp, rp, m, r])


def _to_fp8(v, fmt):
    top, dt = (E5M2_MAX, torch.float8_e5m2) if fmt == "e5m2" else (E4M3_MAX, torch.float8_e4m3fn)
    return v.clamp(-top, top).to(dt)


def _plain_norm_fwd(s):
    x_out, stats = _norm_stats(s)
    y, _, _ = _norm(x_out, s["kind"], s["w_pre"], s["b_pre"])
    r = {"x_out": x_out.to(s["x"].dtype), "stats": stats}
    if s["out"] == "bf16":
        r["y"] = y.to(torch.bfloat16)
    elif s["out"] == "fp8":
        r["y"] = _to_fp8(y * s["y_scale"], "e4m3")
        r["amax"] = y.abs().amax().reshape(1)
    else:
        scale = E4M3_MAX / y.abs().amax(dim=1, keepdim=True)
        r["y"] = _to_fp8(y * scale, "e4m3")
        r["scale_inv"] = (1.0 / scale)[:, 0]
    return r


def _norm_grad(g, xh, r, kind):
    """Gradient of the normalised vector's input from that of its output."""
    d = g - xh * (g * xh).mean(dim=1, keepdim=True)
    if kind == "layer":
        d = d - g.mean(dim=1, keepdim=True)
    return d * r


def _norm_bwd_of(s, dt):
    t, kind = s["x_out"].shape[0], s["kind"]
    mp, rp, m, r = (v[:, None].to(dt) for v in s["stats"])
    dy, h = s["dy"].to(dt), s["h"].to(dt)
    xh = (s["x_out"].to(dt) - m) * r
    out = {"dw_pre": (dy * xh).sum(dim=0)}
    if kind == "layer":
        out["db_pre"] = dy.sum(dim=0)
    dx = s["dx_out"].to(dt) + _norm_grad(dy * s["w_pre"].to(dt), xh, r, kind)
    out["dx"] = s["alpha"] * dx
    hh = p = h
    if s["post"]:
        hh = (h - mp) * rp
        p = hh * s["w_post"].to(dt)
        if kind == "layer":
            p = p + s["b_post"].to(dt)
    dp = dx
    if s["gate"] is not None:
        dp = dx * _gate_rows(s["gate"], t, dt)
        out["dgate"] = (dx * p).view(s["gate"].shape[0], -1, h.shape[1]).sum(dim=1)
    if s["post"]:
        out["dw_post"] = (dp * hh).sum(dim=0)
        if kind == "layer":
            out["db_post"] = dp.sum(dim=0)
        dp = _norm_grad(dp * s["w_post"].to(dt), hh, rp, kind)
    out["dh"] = dp
    return out


def _plain_norm_bwd(s):
    out = _norm_bwd_of(s, torch.float32)
    out["dx"] = out["dx"].to(s["x_out"].dtype)
    out["dh"] = out["dh"].to(torch.bfloat16)
    return out


def _act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    if name == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _factors(v, inv, dt):
    return v * (inv.to(dt)[..., None] if inv.numel() > 1 else inv.to(dt))


def _plain_gemm_act(s):
    f32 = torch.float32
    a = _factors(s["a"].view(torch.float8_e4m3fn).to(f32), s["sa"], f32)
    b = s["b"].view(torch.float8_e4m3fn).to(f32)
    n = s["out_features"]
    if s["experts"]:
        e = s["experts"]
        sb = s["sb"].view(e, -1, 1) if s["sb"].numel() == e else s["sb"][..., None]
        b = b * sb
        # each row's expert and place there, in a block of `most` rows an expert
        off = s["offsets"].long()
        rows = torch.arange(a.shape[0], device=a.device)
        ex = torch.searchsorted(off, rows, right=True) - 1
        at = ex * s["most"] + rows - off[ex]
        full = a.new_zeros(e * s["most"], a.shape[1])
        full[at] = a
        z = torch.bmm(full.view(e, s["most"], -1), b.transpose(1, 2)).view(e * s["most"], -1)[at]
        if s["bias_v"] is not None:
            z = z + s["bias_v"].to(f32)[ex]
    else:
        z = a @ _factors(b, s["sb"], f32).t()
        if s["bias_v"] is not None:
            z = z + s["bias_v"].to(f32)
    v = _act(z[:, :n], s["act"]) * z[:, n:] if s["gated"] else _act(z, s["act"])
    if s["res"] is not None:
        v = v + s["res"].to(f32)
    r = {}
    if s["save_z"]:
        r["z"] = z.to(torch.bfloat16)
    if s["out"] == "bf16":
        r["d"] = v.to(torch.bfloat16)
    else:
        r["d"] = _to_fp8(v * s["q_scale"], "e4m3")
        r["amax"] = v.abs().amax().reshape(1)
    return r


def _act_bwd_of(s, dt):
    d, z, n = s["d"].to(dt), s["z"].to(dt), s["features"]
    if s["gated"]:
        zg, zu = z[:, :n], z[:, n:]
        return torch.cat([d * zu * _act_grad(zg, s["act"]), d * _act(zg, s["act"])], dim=1)
    return d * _act_grad(z, s["act"])


def _plain_act_bwd(s):
    dz = _act_bwd_of(s, torch.float32)
    r = {"dbias": dz.sum(dim=0)} if s["bias"] else {}
    if s["out"] == "bf16":
        r["dz"] = dz.to(torch.bfloat16)
    else:
        r["dz"] = _to_fp8(dz * s["q_scale"], "e5m2")
        r["amax"] = dz.abs().amax().reshape(1)
    return r


def _plain_plan(ids, experts, align, capacity):
    """offsets [E + 1], counts [E], row of each (token, slot) or -1, and the
    (token, slot) of each row or -1; and the flat rows with a place for the
    dropped ones at the end."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    ones = torch.ones_like(key)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, ones)
    starts = torch.cumsum(counts, 0) - counts
    padded = (counts[:experts] + align - 1) // align * align
    offsets = torch.cat([padded.new_zeros(1), torch.cumsum(padded, 0)])
    order = torch.argsort(key, stable=True)
    ks = key[order]
    rank = torch.arange(key.numel(), device=ids.device) - starts[ks]
    row = torch.where(ks < experts, offsets[ks] + rank, torch.full_like(ks, capacity))
    flat_row = torch.empty_like(row)
    flat_row[order] = row
    src = torch.full((capacity + 1,), -1, dtype=torch.int32, device=ids.device)
    src[row] = order.to(torch.int32)
    row_of = torch.where(flat_row < capacity, flat_row, torch.full_like(flat_row, -1))
    return (offsets.to(torch.int32), counts[:experts].to(torch.int32),
            row_of.to(torch.int32).view(ids.shape), src[:capacity], flat_row)


def _plain_moe_dispatch(s):
    cap = _capacity(s)
    offsets, counts, row_of, src, flat_row = _plain_plan(s["ids"], s["experts"], s["align"], cap)
    x, k = s["x"], s["k"]
    xs = x.new_zeros(cap + 1, x.shape[1])
    xs[flat_row] = x.repeat_interleave(k, dim=0)
    xs = xs[:cap]
    r = {"offsets": offsets, "counts": counts, "row_of": row_of, "src": src,
         "xs": xs.view(torch.float8_e4m3fn) if s["dtype"] == "fp8" else xs}
    if s["scale"] is not None:
        sc = s["scale"].new_zeros(cap + 1)
        sc[flat_row] = s["scale"].repeat_interleave(k)
        r["scale"] = sc[:cap]
    return r


def _plain_moe_combine(s):
    row = s["row_of"].long()
    v = s["ys"][row.clamp_min(0)].to(torch.float32)
    v = torch.where((row >= 0)[..., None], v * s["w"][..., None], torch.zeros_like(v))
    return {"y": v.sum(dim=1).to(s["ys"].dtype)}


def _plain_moe_combine_bwd(s):
    row, t, k = s["row_of"].long(), s["tokens"], s["k"]
    here = row >= 0
    dy = s["dy"].to(torch.float32)
    v = s["ys"][row.clamp_min(0)].to(torch.float32)
    dw = torch.where(here, (v * dy[:, None, :]).sum(dim=2), torch.zeros_like(s["w"]))
    del v
    src = s["src"].long()
    at = src.clamp_min(0)
    dys = dy[at // k] * s["w"].view(-1)[at][:, None]
    dys = torch.where((src >= 0)[:, None], dys, torch.zeros_like(dys))
    return {"dys": dys.to(s["ys"].dtype), "dw": dw}


PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "gemm_act": _plain_gemm_act,
         "act_bwd": _plain_act_bwd, "moe_dispatch": _plain_moe_dispatch,
         "moe_combine": _plain_moe_combine, "moe_combine_bwd": _plain_moe_combine_bwd}


# ------------------------------------------------------------------ this package

def _own(s):
    import scaled_fp8_linear_gb300 as F
    op = s["op"]
    kind = F.NORM_LAYER if s.get("kind") == "layer" else F.NORM_RMS
    act = {"none": F.ACT_NONE, "relu": F.ACT_RELU, "silu": F.ACT_SILU, "gelu": F.ACT_GELU,
           "gelu_tanh": F.ACT_GELU_TANH}[s.get("act", "none")]
    if op == "norm_fwd":
        fp8 = s["out"] != "bf16"
        o = F.fp8_norm_fwd(s["x"], s["h"], kind=kind, eps=EPS, alpha=s["alpha"], gate=s["gate"],
                           post_norm=s["post"], w_post=s["w_post"], b_post=s["b_post"],
                           w_pre=s["w_pre"], b_pre=s["b_pre"], want_y=not fp8, want_stats=True,
                           q_fmt=F.E4M3 if fp8 else None,
                           q_gran=F.GRAN_ROW if s["out"] == "fp8_row" else F.GRAN_TENSOR,
                           q_scale=s["y_scale"] if s["out"] == "fp8" else None,
                           want_amax=s["out"] == "fp8")
        r = {"x_out": o.x_out, "stats": o.stats,
             "y": o.q.view(torch.float8_e4m3fn) if fp8 else o.y}
        if s["out"] == "fp8":
            r["amax"] = o.amax
        if s["out"] == "fp8_row":
            r["scale_inv"] = o.q_scale_inv
        return r
    if op == "norm_bwd":
        o = F.fp8_norm_bwd(s["dy"], s["x_out"], s["stats"], dx_out=s["dx_out"], h=s["h"],
                           kind=kind, alpha=s["alpha"], gate=s["gate"], post_norm=s["post"],
                           w_post=s["w_post"], b_post=s["b_post"], w_pre=s["w_pre"],
                           b_pre=s["b_pre"])
        return {k: v for k, v in o._asdict().items() if v is not None}
    if op == "gemm_act":
        fp8 = s["out"] != "bf16"
        gran = F.GRAN_ROW if s["gran"] == "row" else F.GRAN_TENSOR
        o = F.fp8_gemm_act(s["a"], F.E4M3, s["b"], F.E4M3, s["sa"], s["sb"], ga=gran, gb=gran,
                           act=act, gated=s["gated"], bias=s["bias_v"], residual=s["res"],
                           want_z=s["save_z"], want_d=not fp8, q_fmt=F.E4M3 if fp8 else None,
                           q_scale=s["q_scale"] if fp8 else None, want_amax=fp8,
                           offsets=s["offsets"])
        r = {"d": o.q.view(torch.float8_e4m3fn) if fp8 else o.d}
        if s["save_z"]:
            r["z"] = o.z
        if fp8:
            r["amax"] = o.amax
        return r
    if op == "act_bwd":
        fp8 = s["out"] != "bf16"
        o = F.fp8_act_bwd(s["d"], s["z"], act, gated=s["gated"], want_dz=not fp8,
                          q_fmt=F.E5M2 if fp8 else None, q_scale=s["q_scale"] if fp8 else None,
                          want_amax=fp8, want_dbias=s["bias"])
        r = {"dz": o.q.view(torch.float8_e5m2) if fp8 else o.dz}
        if fp8:
            r["amax"] = o.amax
        if s["bias"]:
            r["dbias"] = o.dbias
        return r
    if op == "moe_dispatch":
        p = F.fp8_moe_plan(s["ids"], s["experts"], align=s["align"])
        xs, sc = F.fp8_moe_permute(s["x"], p.row_of, p.src, scale=s["scale"])
        r = {"offsets": p.offsets, "counts": p.counts, "row_of": p.row_of, "src": p.src,
             "xs": xs.view(torch.float8_e4m3fn) if s["dtype"] == "fp8" else xs}
        if sc is not None:
            r["scale"] = sc
        return r
    if op == "moe_combine":
        return {"y": F.fp8_moe_unpermute(s["ys"], s["row_of"], weights=s["w"])}
    dys, dw = F.fp8_moe_unpermute_bwd(s["dy"], s["ys"], s["row_of"], s["src"], s["w"])
    return {"dys": dys, "dw": dw}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ------------------------------------------------------------------ what a pass has to do

def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        t, c, gr = case["tokens"], case["width"], case["gate_rows"]
        st = 4 if case["stream"] == "f32" else 2
        n = t * c
        small = (gr * 2 + 8 + 8 * case["post"]) * c
        if op == "norm_fwd":
            return {"bytes": n * (2 * st + 2 + (2 if case["out"] == "bf16" else 1)) + 16 * t + small,
                    "flops": n * 12}
        return {"bytes": n * (3 * st + 6) + 16 * t + small + (gr + 4) * c * 4, "flops": n * 30}
    if op == "gemm_act":
        m, n, k, e = case["tokens"], case["out_features"], case["in_features"], max(1, case["experts"])
        rows = n * (2 if case["gated"] else 1)
        b = m * k + e * rows * k + m * n * (2 if case["out"] == "bf16" else 1)
        b += m * n * 2 * case["residual"] + m * rows * 2 * case["save_z"] + e * rows * 2 * case["bias"]
        b += (m + e * rows) * 4 * (case["gran"] == "row")
        return {"bytes": b, "flops": 2 * m * rows * k}
    if op == "act_bwd":
        n = case["tokens"] * case["features"]
        rows = 2 if case["gated"] else 1
        return {"bytes": n * (2 + 2 * rows + (2 if case["out"] == "bf16" else 1) * rows)
                + case["features"] * rows * 4 * case["bias"], "flops": n * 20}
    t, c, k = case["tokens"], case["width"], case["k"]
    size = {"bf16": 2, "f32": 4, "fp8": 1}[case["dtype"]]
    rows = _capacity(case)
    if op == "moe_dispatch":
        return {"bytes": t * c * size + rows * c * size + t * k * 8 + rows * 4 + case["experts"] * 8,
                "flops": t * k * 4}
    if op == "moe_combine":
        return {"bytes": t * k * c * size + t * c * size + t * k * 8, "flops": 2 * t * k * c}
    return {"bytes": t * c * size + (t * k + rows) * c * size + t * k * 12, "flops": 3 * t * k * c}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "norm_fwd":
        def norm64(v, w, b):
            mean = v.sum(1, keepdim=True) / v.shape[1] if case["kind"] == "layer" else 0 * v[:, :1]
            var = ((v - mean) ** 2).sum(1, keepdim=True) / v.shape[1]
            rstd = (var + EPS) ** -0.5
            n = (v - mean) * rstd
            n = n if w is None else n * w.to(f64)
            return (n if b is None else n + b.to(f64)), mean[:, 0], rstd[:, 0]
        p = s["h"].to(f64)
        st = torch.zeros(4, case["tokens"], dtype=f64, device=DEV)
        if case["post"]:
            p, st[0], st[1] = norm64(p, s["w_post"], s["b_post"])
        if case["gate_rows"]:
            gr = case["gate_rows"]
            p = (p.view(gr, -1, case["width"]) * s["gate"].to(f64)[:, None, :]).view_as(p)
        x = case["alpha"] * s["x"].to(f64) + p
        y, st[2], st[3] = norm64(x, s["w_pre"], s["b_pre"])
        r = {"x_out": x, "stats": st}
        if case["out"] == "bf16":
            r["y"] = y
        elif case["out"] == "fp8":
            r["y"] = (y * s["y_scale"].to(f64)).clamp(-E4M3_MAX, E4M3_MAX)
            r["amax"] = y.abs().max().reshape(1)
        else:
            inv = y.abs().amax(1, keepdim=True) / E4M3_MAX
            r["y"], r["scale_inv"] = y / inv, inv[:, 0]
        return r
    if op == "norm_bwd":
        return _exact_norm_bwd(case, s)
    if op == "gemm_act":
        return _exact_gemm_act(case, s)
    if op == "act_bwd":
        z = s["z"].to(f64)
        n = case["features"]
        zg = z[:, :n].clone().requires_grad_(True)
        with torch.enable_grad():
            a = _exact_act(zg, case["act"])
        grad, = torch.autograd.grad(a, zg, torch.ones_like(a))
        d = s["d"].to(f64)
        dz = torch.cat([d * z[:, n:] * grad, d * a.detach()], 1) if case["gated"] else d * grad
        r = {"dbias": dz.sum(0)} if case["bias"] else {}
        if case["out"] == "bf16":
            r["dz"] = dz
        else:
            r["dz"] = (dz * s["q_scale"].to(f64)).clamp(-E5M2_MAX, E5M2_MAX)
            r["amax"] = dz.abs().max().reshape(1)
        return r
    t, k = case["tokens"], case["k"]
    if op == "moe_dispatch":
        ids = s["ids"].cpu().numpy().reshape(-1)
        places = [[] for _ in range(case["experts"])]
        for i, e in enumerate(ids):
            if 0 <= e < case["experts"]:
                places[e].append(i)
        src = []
        for p in places:
            src += p + [-1] * (-len(p) % case["align"])
        src = torch.tensor(src + [-1] * (_capacity(case) - len(src)), device=DEV)
        x = s["x"].view(torch.float8_e4m3fn) if case["dtype"] == "fp8" else s["x"]
        xs = x.to(f64)[src.clamp_min(0) // k] * (src >= 0)[:, None]
        r = {"offsets": None, "counts": None, "row_of": None, "src": None, "xs": xs}
        if s["scale"] is not None:
            r["scale"] = s["scale"].to(f64)[src.clamp_min(0) // k] * (src >= 0)
        return r
    row = s["row_of"].long()
    here = (row >= 0).to(f64)
    if op == "moe_combine":
        y = torch.zeros(t, case["width"], dtype=f64, device=DEV)
        for j in range(k):
            y += s["ys"][row[:, j].clamp_min(0)].to(f64) * (s["w"][:, j].to(f64) * here[:, j])[:, None]
        return {"y": y}
    dy = s["dy"].to(f64)
    dw = torch.zeros(t, k, dtype=f64, device=DEV)
    dys = torch.zeros(s["ys"].shape, dtype=f64, device=DEV)
    for j in range(k):
        live = row[:, j] >= 0
        r = row[live, j]
        dw[live, j] = (s["ys"][r].to(f64) * dy[live]).sum(1)
        dys[r] = dy[live] * s["w"][live, j].to(f64)[:, None]
    return {"dys": dys, "dw": dw}


def _exact_norm_bwd(case, s):
    """Written out per row from the chain rule, with the rows' stored statistics."""
    f64 = torch.float64
    c, kind = case["width"], case["kind"]
    mp, rp, m, r = s["stats"].to(f64)[:, :, None]
    dy = s["dy"].to(f64)
    u = (s["x_out"].to(f64) - m) * r
    v = dy * s["w_pre"].to(f64)
    centre = v.sum(1, keepdim=True) / c if kind == "layer" else 0.0
    dx = s["dx_out"].to(f64) + r * (v - centre - u * ((v * u).sum(1, keepdim=True) / c))
    out = {"dx": case["alpha"] * dx, "dw_pre": (dy * u).sum(0)}
    if kind == "layer":
        out["db_pre"] = dy.sum(0)
    p = s["h"].to(f64)
    if case["post"]:
        hh = (p - mp) * rp
        p = hh * s["w_post"].to(f64)
        if kind == "layer":
            p = p + s["b_post"].to(f64)
    gr = case["gate_rows"]
    if gr:
        out["dgate"] = torch.stack([q.sum(0) for q in (dx * p).chunk(gr)])
        dx = (dx.view(gr, -1, c) * s["gate"].to(f64)[:, None, :]).view_as(dx)
    if case["post"]:
        out["dw_post"] = (dx * hh).sum(0)
        if kind == "layer":
            out["db_post"] = dx.sum(0)
        v = dx * s["w_post"].to(f64)
        centre = v.sum(1, keepdim=True) / c if kind == "layer" else 0.0
        dx = rp * (v - centre - hh * ((v * hh).sum(1, keepdim=True) / c))
    out["dh"] = dx
    return out


def _exact_act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        return z * torch.sigmoid(2 * u)
    return z * 1.0


def _exact_gemm_act(case, s):
    f64 = torch.float64
    n, e = case["out_features"], case["experts"]
    rows = n * (2 if case["gated"] else 1)
    a = s["a"].view(torch.float8_e4m3fn).to(f64)
    b = s["b"].view(torch.float8_e4m3fn).view(max(1, e), rows, -1)
    sb = s["sb"].to(f64).view(max(1, e), -1)
    a = a * (s["sa"].to(f64)[:, None] if case["gran"] == "row" else s["sa"].to(f64))
    bias = None if s["bias_v"] is None else s["bias_v"].to(f64).view(max(1, e), rows)
    off = s["offsets"].tolist() if e else [0, a.shape[0]]
    z = torch.empty(a.shape[0], rows, dtype=f64, device=DEV)
    for i in range(max(1, e)):
        part = a[off[i]:off[i + 1]] @ b[i].to(f64).t() * sb[i]
        z[off[i]:off[i + 1]] = part if bias is None else part + bias[i]
    v = _exact_act(z[:, :n], case["act"])
    if case["gated"]:
        v = v * z[:, n:]
    if s["res"] is not None:
        v = v + s["res"].to(f64)
    r = {"z": z} if case["save_z"] else {}
    if case["out"] == "bf16":
        r["d"] = v
    else:
        r["d"] = (v * s["q_scale"].to(f64)).clamp(-E4M3_MAX, E4M3_MAX)
        r["amax"] = v.abs().max().reshape(1)
    return r
