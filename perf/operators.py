"""Cases and plain forms of the feed-forward operators.

The operators are the ones around the parameters that the optimizer step
updates: the bf16 model copies that it writes feed them, and the fp32
main_grad buffers that it reads come out of them.

  norm           h = x + residual;  y = h / rms(h) * gamma  in bf16, and in
                 e4m3 with one fp32 scale per row
  norm_grad      gradient of the norm and of the addition; dgamma in fp32
  quantize       rows of a weight in e4m3 with one fp32 scale per row
  linear         y = act(x w^T + bias) + residual, bf16 operands or e4m3
                 operands with a scale per row of each
  linear_grad    dx = (dz w) * act'(z_prev), dw = dz^T x (+ main_grad),
                 dbias = column sums of dz (+ main_grad)

`own` selects between the plain form (elementary torch operations in 32 bits)
and the library's entry points.  A case is a dict of plain values; `prepare`
makes its tensors on the GPU from a seed, `run` is one pass, `work` what a
pass has to move and compute, `exact` the result in 64 bits.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 1e-30          # smallest row maximum that a scale is made from
EPS = 1e-6

# Model widths that a drawn case may take come from 64 up to the widest matrix
# of the repository's 16-layer workload.
MAX_WIDTH = 14336
MAX_TOKENS = 16384


def listed():
    return [
        # one token of a residual stream: a launch's latency
        dict(name="norm 1 token", op="norm", rows=1, cols=4096, dtype="bf16", residual=True, q=True),
        # a batch of sequences between two blocks: addition, norm, bf16 for the
        # gradient's product and e4m3 for the forward product
        dict(name="norm 16384 tokens", op="norm", rows=16384, cols=4096, dtype="bf16", residual=True, q=True),
        # the same block on the way back, with the residual stream's gradient
        dict(name="norm_grad 8192 tokens", op="norm_grad", rows=8192, cols=4096, dtype="bf16", residual=True),
        # fp32 residual stream, odd width, ragged token count
        dict(name="norm_grad 1031x1023", op="norm_grad", rows=1031, cols=1023, dtype="fp32", residual=False),
        # a model copy laid out in 8 bits after an optimizer step
        dict(name="quantize 14336x4096", op="quantize", rows=14336, cols=4096, dtype="bf16"),
        # an fp32 master of odd width
        dict(name="quantize 777x1111", op="quantize", rows=777, cols=1111, dtype="fp32"),
        # one token through an up projection: the weights' bytes
        dict(name="linear 1 token", op="linear", m=1, n=14336, k=4096, dtype="bf16", act="silu", bias=True,
             residual=False, save_z=False, strided=False),
        # training forward of an up projection, pre-activation kept
        dict(name="linear 8192 bf16", op="linear", m=8192, n=14336, k=4096, dtype="bf16", act="gelu", bias=True,
             residual=False, save_z=True, strided=False),
        # 8-bit down projection that ends in the residual stream
        dict(name="linear 8192 e4m3", op="linear", m=8192, n=4096, k=14336, dtype="e4m3", act="none", bias=False,
             residual=True, save_z=False, strided=False),
        # odd widths, rows that are slices of wider ones
        dict(name="linear 331 odd", op="linear", m=331, n=2049, k=1023, dtype="bf16", act="relu", bias=True,
             residual=True, save_z=False, strided=True),
        # training backward of a down projection: the gradient passes the up
        # projection's activation on its way
        dict(name="linear_grad 8192", op="linear_grad", m=8192, n=4096, k=14336, act="gelu", bias=True,
             accumulate=False, strided=False),
        # a short ragged micro-batch, added to what main_grad holds
        dict(name="linear_grad 100 odd", op="linear_grad", m=100, n=777, k=1000, act="silu", bias=True,
             accumulate=True, strided=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, hi):
    w = _log_int(rng, 64, hi)
    how = rng.random()
    if how < 0.5:
        return max(64, w // 64 * 64)
    if how < 0.75:
        return max(64, w // 8 * 8)
    return w | 1


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quantize", "linear", "linear", "linear_grad", "linear_grad"])
    rows = _log_int(rng, 1, MAX_TOKENS)
    if op in ("norm", "norm_grad", "quantize"):
        cols = _width(rng, MAX_WIDTH)
        rows = max(1, min(rows, 16384 * 4096 // cols))
        c = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "fp32"]))
        if op != "quantize":
            c["residual"] = rng.random() < 0.5
        if op == "norm":
            c["q"] = rng.random() < 0.5
        return c
    n, k = _width(rng, MAX_WIDTH), _width(rng, MAX_WIDTH)
    rows = max(1, min(rows, 8192 * 4096 * 14336 // (n * k)))
    if op == "linear":
        return dict(op=op, m=rows, n=n, k=k, dtype=rng.choice(["bf16", "bf16", "e4m3"]),
                    act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, save_z=rng.random() < 0.3, strided=rng.random() < 0.2)
    return dict(op=op, m=rows, n=n, k=k, act=rng.choice(["none", "relu", "gelu", "silu"]), bias=rng.random() < 0.5,
                accumulate=rng.random() < 0.3, strided=rng.random() < 0.2)


# ------------------------------------------------------------------ inputs --


class State:
    """The tensors of one case, by name."""


DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _normal(gen, shape, dtype=torch.bfloat16, std=1.0, mean=0.0, strided=False):
    """Normal values; `strided`: a slice of rows that are 24 elements wider."""
    wide = list(shape)
    wide[-1] += 24 if strided else 0
    t = torch.randn(wide, generator=gen, device="cuda", dtype=torch.float32).mul_(std).add_(mean).to(dtype)
    return t[..., 8:8 + shape[-1]] if strided else t


def _e4m3_rows(t):
    scale = t.float().abs().amax(dim=1).clamp_min(AMAX_FLOOR) / E4M3_MAX
    return (t.float() / scale[:, None]).to(torch.float8_e4m3fn), scale


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = State()
    s.op = case["op"]
    if s.op in ("norm", "norm_grad", "quantize"):
        rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        if s.op == "quantize":
            s.x = _normal(gen, (rows, cols), dt, std=0.02)
            s.q, s.scale = _empty((rows, cols), torch.float8_e4m3fn), _empty((rows,), torch.float32)
            return s
        # a residual stream has a few channels far larger than the others
        s.gamma = _normal(gen, (cols,), torch.bfloat16, std=0.1, mean=1.0)
        s.x = _normal(gen, (rows, cols), dt)
        s.x[:, :: max(1, cols // 4)] *= 8
        s.residual = s.q = s.q_scale = s.h = s.dh = None
        if s.op == "norm":
            s.y, s.rstd = _empty((rows, cols), torch.bfloat16), _empty((rows,), torch.float32)
            if case["residual"]:
                s.residual = _normal(gen, (rows, cols), dt, std=2.0)
                s.h = _empty((rows, cols), dt)
            if case["q"]:
                s.q, s.q_scale = _empty((rows, cols), torch.float8_e4m3fn), _empty((rows,), torch.float32)
            return s
        s.rstd = torch.rsqrt(s.x.float().square().mean(dim=1) + EPS)
        s.dy = _normal(gen, (rows, cols), torch.bfloat16, std=1e-2)
        if case["residual"]:
            s.dh = _normal(gen, (rows, cols), dt, std=1e-2)
        s.dx, s.dgamma = _empty((rows, cols), dt), _empty((cols,), torch.float32)
        if own:      # a program keeps its workspace beside its buffers
            import mixed_precision_optimizer_gb300 as mp
            s.workspace = mp.rmsnorm_workspace(rows, cols)
        return s
    m, n, k = case["m"], case["n"], case["k"]
    strided = case["strided"]
    s.act = case["act"]
    s.w = _normal(gen, (n, k), std=0.02)
    s.bias = s.residual = s.z = s.x_scale = s.w_scale = None
    if s.op == "linear":
        s.x = _normal(gen, (m, k), strided=strided)
        if case["dtype"] == "e4m3":
            s.x, s.x_scale = _e4m3_rows(s.x)
            s.w, s.w_scale = _e4m3_rows(s.w)
        if case["bias"]:
            s.bias = _normal(gen, (n,), std=0.1)
        if case["residual"]:
            s.residual = _normal(gen, (m, n), std=2.0, strided=strided)
        if case["save_z"]:
            s.z = _empty((m, n), torch.bfloat16)
        s.y = _empty((m, n), torch.bfloat16)
    else:
        s.dz = _normal(gen, (m, n), std=1e-2, strided=strided)
        s.x = _normal(gen, (m, k), strided=strided)
        s.z_prev = _normal(gen, (m, k)) if s.act != "none" else None
        s.dx = _empty((m, k), torch.bfloat16)
        s.accumulate = case["accumulate"]
        s.dw = _normal(gen, (n, k), torch.float32, std=1e-2)
        s.dbias = _normal(gen, (n,), torch.float32, std=1e-2) if case["bias"] else None
    if own:
        import mixed_precision_optimizer_gb300 as mp
        s.workspace = mp.linear_workspace(m, n, k)
    return s


# --------------------------------------------------------------- one pass --


def _act(z, act):
    if act == "relu":
        return torch.clamp_min(z, 0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        t = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * 0.7978845608028654 * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _quantize_plain(y):
    scale = y.abs().amax(dim=1).clamp_min(AMAX_FLOOR) / E4M3_MAX
    return (y / scale[:, None]).to(torch.float8_e4m3fn), scale


def _plain(s):
    if s.op == "quantize":
        q, scale = _quantize_plain(s.x.float())
        return {"q": q, "scale": scale}
    if s.op == "norm":
        h = s.x.float() if s.residual is None else s.x.float() + s.residual.float()
        rstd = torch.rsqrt(h.square().mean(dim=1) + EPS)
        y = h * rstd[:, None] * s.gamma.float()
        out = {"y": y.to(torch.bfloat16), "rstd": rstd}
        if s.residual is not None:
            out["h"] = h.to(s.x.dtype)
        if s.q is not None:
            out["q"], out["q_scale"] = _quantize_plain(y)
        return out
    if s.op == "norm_grad":
        n = s.x.float() * s.rstd[:, None]
        dy = s.dy.float()
        g = dy * s.gamma.float()
        dx = s.rstd[:, None] * (g - n * (g * n).mean(dim=1, keepdim=True))
        if s.dh is not None:
            dx = dx + s.dh.float()
        return {"dx": dx.to(s.x.dtype), "dgamma": (dy * n).sum(dim=0)}
    if s.op == "linear":
        x, w = s.x.float(), s.w.float()
        if s.x_scale is not None:
            x, w = x * s.x_scale[:, None], w * s.w_scale[:, None]
        z = x @ w.t()
        if s.bias is not None:
            z = z + s.bias.float()
        y = _act(z, s.act)
        if s.residual is not None:
            y = y + s.residual.float()
        out = {"y": y.to(torch.bfloat16)}
        if s.z is not None:
            out["z"] = z.to(torch.bfloat16)
        return out
    dz = s.dz.float()
    dx = dz @ s.w.float()
    if s.z_prev is not None:
        dx = dx * _act_grad(s.z_prev.float(), s.act)
    dw = dz.t() @ s.x.float()
    out = {"dx": dx.to(torch.bfloat16), "dw": dw + s.dw if s.accumulate else dw}
    if s.dbias is not None:
        db = dz.sum(dim=0)
        out["dbias"] = db + s.dbias if s.accumulate else db
    return out


def _own(s):
    import mixed_precision_optimizer_gb300 as mp
    if s.op == "quantize":
        mp.quantize_rows(s.x, s.q, s.scale)
        return {"q": s.q, "scale": s.scale}
    if s.op == "norm":
        mp.rmsnorm(s.x, s.gamma, EPS, residual=s.residual, h=s.h, y=s.y, q=s.q, q_scale=s.q_scale, rstd=s.rstd)
        out = {"y": s.y, "rstd": s.rstd}
        if s.residual is not None:
            out["h"] = s.h
        if s.q is not None:
            out["q"], out["q_scale"] = s.q, s.q_scale
        return out
    if s.op == "norm_grad":
        mp.rmsnorm_backward(s.dy, s.x, s.gamma, s.rstd, s.dx, dh=s.dh, dgamma=s.dgamma, accumulate=False,
                            workspace=s.workspace)
        return {"dx": s.dx, "dgamma": s.dgamma}
    if s.op == "linear":
        mp.linear(s.x, s.w, s.y, bias=s.bias, act=s.act, residual=s.residual, z=s.z, x_scale=s.x_scale,
                  w_scale=s.w_scale, workspace=s.workspace)
        out = {"y": s.y}
        if s.z is not None:
            out["z"] = s.z
        return out
    dw, dbias = s.dw, s.dbias
    if s.accumulate:      # the sums of the micro-batches before this one stay as they are for the next pass
        dw, dbias = dw.clone(), dbias if dbias is None else dbias.clone()
    mp.linear_backward(s.dz, s.x, s.w, dx=s.dx, z_prev=s.z_prev, act_prev=s.act, dw=dw, dbias=dbias,
                       accumulate=s.accumulate, workspace=s.workspace)
    out = {"dx": s.dx, "dw": dw}
    if dbias is not None:
        out["dbias"] = dbias
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------- bytes and flops --


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad", "quantize"):
        r, c = case["rows"], case["cols"]
        e = 2 if case["dtype"] == "bf16" else 4
        if op == "quantize":
            return {"bytes": r * c * (e + 1) + 4 * r, "flops": 2 * r * c}
        if op == "norm":
            b = r * c * (e + 2) + 2 * c + 4 * r
            b += r * c * 2 * e if case["residual"] else 0
            b += r * c + 4 * r if case["q"] else 0
            return {"bytes": b, "flops": 6 * r * c}
        b = r * c * (2 + 2 * e) + 6 * c + 4 * r + (r * c * e if case["residual"] else 0)
        return {"bytes": b, "flops": 10 * r * c}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "linear":
        e = 1 if case["dtype"] == "e4m3" else 2
        b = e * (m * k + n * k) + 2 * m * n
        b += 2 * n if case["bias"] else 0
        b += 2 * m * n if case["residual"] else 0
        b += 2 * m * n if case["save_z"] else 0
        b += 4 * (m + n) if e == 1 else 0
        return {"bytes": b, "flops": 2 * m * n * k}
    b = 2 * (m * n + m * k + n * k) + 2 * m * k + 4 * n * k
    b += 2 * m * k if case["act"] != "none" else 0
    b += 4 * n * k if case["accumulate"] else 0
    b += 4 * n * (2 if case["accumulate"] else 1) if case["bias"] else 0
    return {"bytes": b, "flops": 4 * m * n * k}


# ------------------------------------------------------------- in 64 bits --


def _exact_sigmoid(z):
    e = torch.exp(-z.abs())
    return torch.where(z >= 0, 1 / (1 + e), e / (1 + e))


def exact(case, seed):
    """The definitions in fp64, nothing rounded: an 8-bit value is the
    quotient that it stands in for."""
    s = prepare(case, seed)
    f = torch.float64
    if s.op == "quantize":
        x = s.x.to(f)
        amax = torch.maximum(x.max(dim=1).values, -x.min(dim=1).values)
        return {"q": x * (E4M3_MAX / amax)[:, None], "scale": amax / E4M3_MAX}
    if s.op == "norm":
        h = s.x.to(f) + (0 if s.residual is None else s.residual.to(f))
        rms = ((h * h).sum(dim=1) / case["cols"] + EPS).sqrt()
        y = h * s.gamma.to(f) / rms[:, None]
        out = {"y": y, "rstd": 1 / rms}
        if s.residual is not None:
            out["h"] = h
        if s.q is not None:
            amax = torch.maximum(y.max(dim=1).values, -y.min(dim=1).values)
            out["q"], out["q_scale"] = y * (E4M3_MAX / amax)[:, None], amax / E4M3_MAX
        return out
    if s.op == "norm_grad":
        h, dy, r = s.x.to(f), s.dy.to(f), s.rstd.to(f)
        g = dy * s.gamma.to(f)
        dot = (g * h).sum(dim=1)
        dx = g * r[:, None] - h * (r ** 3 * dot / case["cols"])[:, None]
        return {"dx": dx if s.dh is None else dx + s.dh.to(f), "dgamma": torch.einsum("rc,rc,r->c", dy, h, r)}
    if s.op == "linear":
        z = torch.einsum("mk,nk->mn", s.x.to(f), s.w.to(f))
        if s.x_scale is not None:
            z *= s.x_scale.to(f)[:, None] * s.w_scale.to(f)[None, :]
        if s.bias is not None:
            z += s.bias.to(f)
        if s.act == "relu":
            y = torch.where(z > 0, z, torch.zeros_like(z))
        elif s.act == "silu":
            y = z * _exact_sigmoid(z)
        elif s.act == "gelu":       # (1 + tanh u) / 2 = sigmoid(2 u)
            y = z * _exact_sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        else:
            y = z.clone()
        if s.residual is not None:
            y += s.residual.to(f)
        return {"y": y, "z": z} if s.z is not None else {"y": y}
    dz = s.dz.to(f)
    dx = torch.einsum("mn,nk->mk", dz, s.w.to(f))
    if s.act == "relu":
        dx = torch.where(s.z_prev > 0, dx, torch.zeros_like(dx))
    elif s.act == "silu":
        z = s.z_prev.to(f)
        p = _exact_sigmoid(z)
        dx *= p + z * p * (1 - p)
    elif s.act == "gelu":
        z = s.z_prev.to(f)
        c = 2 * math.sqrt(2 / math.pi)
        p = _exact_sigmoid(c * (z + 0.044715 * z ** 3))
        dx *= p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z ** 2)
    dw = torch.einsum("mn,mk->nk", dz, s.x.to(f))
    out = {"dx": dx, "dw": dw + s.dw.to(f) if s.accumulate else dw}
    if s.dbias is not None:
        db = dz.sum(dim=0)
        out["dbias"] = db + s.dbias.to(f) if s.accumulate else db
    return out
