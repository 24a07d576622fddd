"""Cases and plain forms of the operators at the two ends of a language model
and between its blocks.

  embedding      y = table[token] * scale;  tokens outside the table give zeros
  embedding_grad dtable[v] += scale * sum of dy over the tokens that are v
  recurrence     h_t = h_{t-1} + c_t (x_t - h_{t-1}),  c = sigmoid(gate), along
                 the rows of each sequence of a packed batch, from h0 to hT
  recurrence_grad gradients of x, gate and h0 from those of y and hT
  checkpoint     an activation in e4m3 with a power of two for each 32 columns
  restore        the activation back from its checkpoint, through the
                 activation function, and the gradient passing it
  cross_entropy  loss and log-sum-exp of each row of logits, and the logits'
                 gradient

`own` selects between the plain form (elementary torch operations in 32 bits)
and the library's entry points.  A case is a dict of plain values; `prepare`
makes its tensors on the GPU from a seed, `run` is one pass, `work` what a
pass has to move and compute, `exact` the result in 64 bits.
"""

import math

import torch

own = False

BLOCK = 32                  # columns that share a checkpoint's scale
MIN_EXP = -116              # smallest exponent of a scale: restored values stay normal numbers
GELU_C = 0.7978845608028654

# The vocabulary and the widths of the repository's 16-layer workload are the
# upper ends of the drawn ones.
VOCAB = 128256
MAX_WIDTH = 14336
MAX_ROWS = 16384


def listed():
    return [
        # one token on its way into the model: a launch's latency
        dict(name="embedding 1 token", op="embedding", rows=1, cols=4096, vocab=VOCAB, dtype="bf16", out="bf16", index="int64",
             scaled=False, strided=False),
        # a batch of tokens into an fp32 residual stream
        dict(name="embedding 16384 tokens", op="embedding", rows=16384, cols=4096, vocab=VOCAB, dtype="bf16", out="fp32",
             index="int64", scaled=True, strided=False),
        # the way back: added to the main_grad of the whole table
        dict(name="embedding_grad 16384 tokens", op="embedding_grad", rows=16384, cols=4096, vocab=VOCAB, dtype="bf16",
             index="int64", scaled=True, strided=False),
        # a short ragged micro-batch of a small odd model
        dict(name="embedding_grad 777x1111", op="embedding_grad", rows=777, cols=1111, vocab=5003, dtype="fp32", index="int32",
             scaled=False, strided=True),
        # one new token for each of 64 sequences
        dict(name="recurrence 64 single tokens", op="recurrence", rows=64, cols=4096, sequences=64, ragged=False, dtype="bf16",
             keep=False, strided=False),
        # one long sequence in training
        dict(name="recurrence 16384 tokens", op="recurrence", rows=16384, cols=4096, sequences=1, ragged=False, dtype="bf16",
             keep=True, strided=False),
        # a packed batch of sequences on the way back
        dict(name="recurrence_grad 8192 packed", op="recurrence_grad", rows=8192, cols=4096, sequences=9, ragged=True,
             dtype="bf16", strided=False),
        # odd widths in fp32
        dict(name="recurrence_grad 1031x1023", op="recurrence_grad", rows=1031, cols=1023, sequences=7, ragged=True,
             dtype="fp32", strided=False),
        # an up projection's pre-activation put away until the backward pass
        dict(name="checkpoint 8192x14336", op="checkpoint", rows=8192, cols=14336, dtype="bf16", strided=False),
        # and taken out again, as the next product's operand and the gradient's argument
        dict(name="restore 8192x14336", op="restore", rows=8192, cols=14336, act="gelu", grad=True, strided=False),
        # the whole vocabulary of a batch of tokens
        dict(name="cross_entropy 8192 tokens", op="cross_entropy", rows=8192, cols=VOCAB, dtype="bf16", index="int64",
             grad=True, weighted=False, strided=False),
        # an odd vocabulary, few tokens, each with a weight of its own
        dict(name="cross_entropy 331x32003", op="cross_entropy", rows=331, cols=32003, dtype="bf16", index="int32", grad=True,
             weighted=True, strided=False),
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
    op = rng.choice(["embedding", "embedding_grad", "embedding_grad", "recurrence", "recurrence", "recurrence_grad",
                     "recurrence_grad", "checkpoint", "restore", "cross_entropy", "cross_entropy"])
    rows, strided = _log_int(rng, 1, MAX_ROWS), rng.random() < 0.2
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    index = rng.choice(["int32", "int64"])
    if op in ("embedding", "embedding_grad"):
        cols = _width(rng, 4096)
        c = dict(op=op, rows=rows, cols=cols, vocab=_log_int(rng, 100, VOCAB), dtype=dtype, index=index,
                 scaled=rng.random() < 0.5, strided=strided)
        if op == "embedding":
            c["out"] = rng.choice(["bf16", "fp32"])
        return c
    if op in ("recurrence", "recurrence_grad"):
        cols = _width(rng, 4096)
        rows = min(rows, 8192) if op == "recurrence_grad" else rows
        sequences = rng.choice([1, 1, min(rows, 2), min(rows, 16), max(1, rows // 100), rows])
        ragged = sequences > 1 and rng.random() < 0.6
        if not ragged:
            rows = rows // sequences * sequences
        c = dict(op=op, rows=rows, cols=cols, sequences=sequences, ragged=ragged, dtype=dtype, strided=strided)
        if op == "recurrence":
            c["keep"] = rng.random() < 0.7
        return c
    if op in ("checkpoint", "restore"):
        cols = _width(rng, MAX_WIDTH)
        rows = max(1, min(rows, 8192 * 14336 // cols))
        if op == "checkpoint":
            return dict(op=op, rows=rows, cols=cols, dtype=dtype, strided=strided)
        return dict(op=op, rows=rows, cols=cols, act=rng.choice(["none", "relu", "gelu", "silu"]), grad=rng.random() < 0.5,
                    strided=strided)
    cols = _width(rng, VOCAB)
    return dict(op=op, rows=min(rows, 8192) if dtype == "bf16" else min(rows, 4096), cols=cols, dtype=dtype, index=index,
                grad=rng.random() < 0.8, weighted=rng.random() < 0.5, strided=strided)


# ------------------------------------------------------------------ inputs --


class State:
    """The tensors of one case, by name."""


DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "int32": torch.int32, "int64": torch.int64}


def _normal(gen, shape, dtype=torch.bfloat16, std=1.0, mean=0.0, strided=False):
    """Normal values; `strided`: a slice of rows that are 24 elements wider."""
    wide = list(shape)
    wide[-1] += 24 if strided else 0
    t = torch.randn(wide, generator=gen, device="cuda", dtype=torch.float32).mul_(std).add_(mean).to(dtype)
    return t[..., 8:8 + shape[-1]] if strided else t


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _tokens(gen, rows, vocab, dtype):
    """Tokens as text has them, the k-th most frequent about 1 / k as often as
    the first (6 % of the batch for a large vocabulary), 2 % of them padding."""
    u = torch.rand(rows, generator=gen, device="cuda", dtype=torch.float64)
    t = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp_(0, vocab - 1)
    t = (t * 48271) % vocab if vocab % 48271 else t          # frequent tokens lie anywhere in the table
    pad = torch.rand(rows, generator=gen, device="cuda") < 0.02
    return torch.where(pad, torch.full_like(t, -1), t).to(dtype)


def _starts(gen, rows, sequences):
    """Ragged sequences, some of them empty, up to 3 % of the rows behind the last one."""
    end = rows - int(0.03 * rows)
    cuts = torch.rand(sequences - 1, generator=gen, device="cuda").mul_(end + 1).long().clamp_(0, end).sort().values
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    return torch.cat([zero, cuts, zero + end]).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = State()
    s.op = case["op"]
    strided = case["strided"]
    rows, cols = case["rows"], case["cols"]
    dt = DTYPES[case.get("dtype", "bf16")]
    if s.op in ("embedding", "embedding_grad"):
        s.tokens = _tokens(gen, rows, case["vocab"], DTYPES[case["index"]])
        s.scale = math.sqrt(cols) if case["scaled"] else 1.0
        if s.op == "embedding":
            s.table = _normal(gen, (case["vocab"], cols), dt, std=0.02)
            s.y = _empty((rows, cols + (24 if strided else 0)), DTYPES[case["out"]])[:, :cols]
            return s
        s.dy = _normal(gen, (rows, cols), dt, std=1e-2, strided=strided)
        s.dtable = _normal(gen, (case["vocab"], cols), torch.float32, std=1e-2)      # what main_grad holds already
        if own:      # a program keeps its workspace beside its buffers
            import mixed_precision_optimizer_gb300 as mp
            s.workspace = mp.embedding_workspace(rows, case["vocab"], cols)
        return s
    if s.op in ("recurrence", "recurrence_grad"):
        n = case["sequences"]
        s.sequences = n
        s.starts = _starts(gen, rows, n) if case["ragged"] else None
        s.x = _normal(gen, (rows, cols), dt, strided=strided)
        # channels remember from two to some hundred rows
        s.gate = _normal(gen, (rows, cols), torch.float32, strided=strided)
        s.gate += torch.rand(cols, generator=gen, device="cuda") * 6 - 6
        s.gate = s.gate.to(dt) if not strided else _wide_like(s.gate, dt)
        s.h0 = _normal(gen, (n, cols), torch.float32, std=0.5)
        if s.op == "recurrence":
            s.y = torch.zeros((rows, cols), dtype=dt, device="cuda")
            s.states = None
            s.hT = torch.empty_like(s.h0)
            if own and case["keep"]:
                import mixed_precision_optimizer_gb300 as mp
                s.states = mp.recurrence_states(rows, cols, dt)
            return s
        s.dy = _normal(gen, (rows, cols), dt, std=1e-2, strided=strided)
        s.dhT = _normal(gen, (n, cols), torch.float32, std=1e-2)
        s.dx, s.dgate = (torch.zeros((rows, cols), dtype=dt, device="cuda") for _ in range(2))
        s.dh0 = torch.empty_like(s.h0)
        # what the forward pass left behind: its states in fp32, all of them for the plain form
        if own:
            import mixed_precision_optimizer_gb300 as mp
            s.states = mp.recurrence_states(rows, cols, dt)
            mp.gated_recurrence(s.x, s.gate, torch.empty_like(s.dx), starts=s.starts, sequences=n, h0=s.h0, states=s.states)
        else:
            s.h = _recurrence_plain(s)[1]
        return s
    if s.op in ("checkpoint", "restore"):
        x = _normal(gen, (rows, cols), dt, std=1.5, strided=strided)
        x[:, :: max(1, cols // 8)] *= 12                 # a few channels far larger than the others
        if s.op == "checkpoint":
            s.x = x
            s.q, s.scale = _empty((rows, cols), torch.float8_e4m3fn), _empty((rows, -(-cols // BLOCK)), torch.uint8)
            return s
        s.q, s.scale = _checkpoint_plain(x.float())
        s.act = case["act"]
        s.dy = _normal(gen, (rows, cols), std=1e-2, strided=strided) if case["grad"] else None
        s.y, s.z = _empty((rows, cols), torch.bfloat16), _empty((rows, cols), torch.bfloat16)
        return s
    s.logits = _normal(gen, (rows, cols), dt, std=2.0, strided=strided)
    s.labels = torch.randint(0, cols, (rows,), generator=gen, device="cuda")
    s.logits[torch.arange(rows, device="cuda"), s.labels] += 6
    s.logits[:, cols - cols // 100:] = -math.inf                # columns that the grammar or the padding rules out
    s.labels = torch.where(s.labels < cols - cols // 100, s.labels, s.labels // 2)
    s.labels = torch.where(torch.rand(rows, generator=gen, device="cuda") < 0.05, torch.full_like(s.labels, -100), s.labels)
    s.labels = s.labels.to(DTYPES[case["index"]])
    s.scale = 1.0 / rows
    s.weight = torch.rand(rows, generator=gen, device="cuda") if case["weighted"] else None
    s.loss, s.lse = _empty((rows,), torch.float32), _empty((rows,), torch.float32)
    s.dlogits = _empty((rows, cols), dt) if case["grad"] else None
    return s


def _wide_like(t, dtype):
    """A slice of rows of the same distance in another type."""
    wide = torch.zeros((t.shape[0], t.stride(0)), dtype=dtype, device="cuda")
    part = wide[:, 8:8 + t.shape[1]]
    part.copy_(t)
    return part


# --------------------------------------------------------------- one pass --


def _act(z, act):
    if act == "relu":
        return torch.clamp_min(z, 0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(GELU_C * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        t = torch.tanh(GELU_C * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * GELU_C * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _checkpoint_plain(x):
    """Codes and exponent bytes: the smallest power of two that takes a block's
    largest magnitude to 448 or less."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    padded = torch.nn.functional.pad(x, (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    m, e = torch.frexp(padded.abs().amax(dim=2))               # amax = m 2^e with m in [0.5, 1);  448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, torch.full_like(e, MIN_EXP), e).clamp_min(MIN_EXP)
    q = torch.ldexp(padded, -e[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(rows, blocks * BLOCK)[:, :cols].contiguous(), (e + 127).to(torch.uint8)


def _sequence_of(s):
    """For each row its sequence, and whether it is its sequence's first and last
    row; for each sequence its first row and the one behind its last."""
    rows = s.x.shape[0]
    row = torch.arange(rows, device="cuda")
    starts = s.starts.long() if s.starts is not None else torch.arange(s.sequences + 1, device="cuda") * (rows // s.sequences)
    seq = torch.bucketize(row, starts, right=True) - 1
    inside = seq < s.sequences
    seq = seq.clamp_max(s.sequences - 1)
    return seq, inside & (row == starts[seq]), inside & (row + 1 == starts[seq + 1]), inside, starts


def _scan(s, a, b):
    """h_t = a_t h_{t-1} + b_t along the rows, by doubling up to the longest that
    a sequence can be."""
    step, longest = 1, a.shape[0] // s.sequences if s.starts is None else a.shape[0]
    while step < longest:
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _recurrence_plain(s):
    """The sequences' last states and every row's, in fp32."""
    seq, first, _, inside, starts = _sequence_of(s)
    g = s.gate.float()
    c, a = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))
    b = c * s.x.float()
    b = torch.where(first[:, None], b + a * s.h0[seq], b)
    h = _scan(s, torch.where(first[:, None], torch.zeros_like(a), a), b)
    h = torch.where(inside[:, None], h, torch.zeros_like(h))
    last, empty = (starts[1:] - 1).clamp_min(0), starts[1:] == starts[:-1]
    return torch.where(empty[:, None], s.h0, h[last]), h


def _recurrence_grad_plain(s):
    seq, first, last, inside, starts = _sequence_of(s)
    g = s.gate.float()
    c, a = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))
    before = torch.cat([torch.zeros_like(s.h[:1]), s.h[:-1]])
    before = torch.where(first[:, None], s.h0[seq], before)
    b = s.dy.float()
    b = torch.where(last[:, None], b + s.dhT[seq], b)
    keep = torch.cat([a[1:], torch.zeros_like(a[:1])])           # how much of the next row's gradient arrives here
    keep = torch.where(last[:, None], torch.zeros_like(keep), keep)
    lam = _scan(s, keep.flip(0), b.flip(0)).flip(0)
    lam = torch.where(inside[:, None], lam, torch.zeros_like(lam))
    empty = starts[1:] == starts[:-1]
    at = starts[:-1].clamp_max(a.shape[0] - 1)
    dh0 = torch.where(empty[:, None], s.dhT, a[at] * lam[at])
    return {"dx": (c * lam).to(s.x.dtype), "dgate": (c * a * lam * (s.x.float() - before)).to(s.x.dtype), "dh0": dh0}


def _plain(s):
    if s.op == "embedding":
        known = (s.tokens >= 0) & (s.tokens < s.table.shape[0])
        y = s.table[torch.where(known, s.tokens, 0).long()].float() * s.scale
        return {"y": torch.where(known[:, None], y, torch.zeros_like(y)).to(s.y.dtype)}
    if s.op == "embedding_grad":
        known = (s.tokens >= 0) & (s.tokens < s.dtable.shape[0])
        g = torch.where(known[:, None], s.dy.float() * s.scale, torch.zeros_like(s.dtable[:1]))
        s.dtable.index_add_(0, torch.where(known, s.tokens, 0).long(), g)
        return {"dtable": s.dtable}
    if s.op == "recurrence":
        hT, h = _recurrence_plain(s)
        return {"y": h.to(s.x.dtype), "hT": hT}
    if s.op == "recurrence_grad":
        return _recurrence_grad_plain(s)
    if s.op == "checkpoint":
        q, scale = _checkpoint_plain(s.x.float())
        return {"q": q, "scale": scale}
    if s.op == "restore":
        e = (s.scale.int() - 127).repeat_interleave(BLOCK, dim=1)[:, :s.q.shape[1]]
        z = torch.ldexp(s.q.float(), e)
        out = {"y": _act(z, s.act).to(torch.bfloat16)}
        if s.dy is not None:
            out["dz"] = (s.dy.float() * _act_grad(z, s.act)).to(torch.bfloat16)
        else:
            out["z"] = z.to(torch.bfloat16)
        return out
    x = s.logits.float()
    rows, cols = x.shape
    known = (s.labels >= 0) & (s.labels < cols)
    label = torch.where(known, s.labels, 0).long()
    top = x.amax(dim=1)
    lse = top + torch.log(torch.exp(x - top[:, None]).sum(dim=1))
    out = {"loss": torch.where(known, lse - x[torch.arange(rows, device="cuda"), label], torch.zeros_like(lse)), "lse": lse}
    if s.dlogits is not None:
        g = torch.exp(x - lse[:, None])
        g[torch.arange(rows, device="cuda"), label] -= 1
        w = known.float() * s.scale
        w = w if s.weight is None else w * s.weight
        out["dlogits"] = (g * w[:, None]).to(s.logits.dtype)
    return out


def _own(s):
    import mixed_precision_optimizer_gb300 as mp
    if s.op == "embedding":
        mp.embedding(s.tokens, s.table, s.y, scale=s.scale)
        return {"y": s.y}
    if s.op == "embedding_grad":
        mp.embedding_backward(s.tokens, s.dy, s.dtable, scale=s.scale, workspace=s.workspace)
        return {"dtable": s.dtable}
    if s.op == "recurrence":
        mp.gated_recurrence(s.x, s.gate, s.y, starts=s.starts, sequences=s.sequences, h0=s.h0, hT=s.hT, states=s.states)
        return {"y": s.y, "hT": s.hT}
    if s.op == "recurrence_grad":
        mp.gated_recurrence_backward(s.dy, s.x, s.gate, s.states, s.dx, s.dgate, starts=s.starts, sequences=s.sequences,
                                     h0=s.h0, dhT=s.dhT, dh0=s.dh0)
        return {"dx": s.dx, "dgate": s.dgate, "dh0": s.dh0}
    if s.op == "checkpoint":
        mp.checkpoint_save(s.x, s.q, s.scale)
        return {"q": s.q, "scale": s.scale}
    if s.op == "restore":
        if s.dy is None:
            mp.checkpoint_restore(s.q, s.scale, z=s.z, y=s.y, act=s.act)
            return {"y": s.y, "z": s.z}
        mp.checkpoint_restore(s.q, s.scale, y=s.y, act=s.act, dy=s.dy, dz=s.z)
        return {"y": s.y, "dz": s.z}
    mp.cross_entropy(s.logits, s.labels, s.loss, lse=s.lse, dlogits=s.dlogits, scale=s.scale, weight=s.weight)
    out = {"loss": s.loss, "lse": s.lse}
    if s.dlogits is not None:
        out["dlogits"] = s.dlogits
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------- bytes and flops --


def work(case):
    op, r, c = case["op"], case["rows"], case["cols"]
    e = 4 if case.get("dtype") == "fp32" else 2
    i = 4 if case.get("index") == "int32" else 8
    if op in ("embedding", "embedding_grad"):
        v = case["vocab"]          # distinct rows of the table that r such tokens are expected to meet
        distinct = sum(1 - (1 - 0.98 * math.log((k + 2) / (k + 1)) / math.log(v + 1)) ** r for k in range(v))
        if op == "embedding":
            return {"bytes": distinct * c * e + r * (c * (4 if case["out"] == "fp32" else 2) + i), "flops": r * c}
        return {"bytes": r * (c * e + i) + distinct * c * 8, "flops": r * c}
    if op == "recurrence":
        return {"bytes": 3 * r * c * e + 8 * case["sequences"] * c, "flops": 8 * r * c}
    if op == "recurrence_grad":
        return {"bytes": 5 * r * c * e + 12 * case["sequences"] * c, "flops": 16 * r * c}
    if op == "checkpoint":
        return {"bytes": r * (c * (e + 1) + -(-c // BLOCK)), "flops": 2 * r * c}
    if op == "restore":
        return {"bytes": r * (c * (7 if case["grad"] else 5) + -(-c // BLOCK)), "flops": 10 * r * c}
    b = r * (c * e + i + 8) + (r * c * e if case["grad"] else 0) + (4 * r if case["weighted"] else 0)
    return {"bytes": b, "flops": 4 * r * c}


# ------------------------------------------------------------- in 64 bits --


def _sigmoid64(t):
    e = torch.exp(-t.abs())
    return torch.where(t >= 0, 1 / (1 + e), e / (1 + e))


def _exact_recurrence(case, s):
    """One row after another."""
    f = torch.float64
    rows, n = case["rows"], case["sequences"]
    starts = s.starts.tolist() if s.starts is not None else [i * (rows // n) for i in range(n + 1)]
    x, c, a = s.x.to(f), _sigmoid64(s.gate.to(f)), _sigmoid64(-s.gate.to(f))
    before, h = torch.zeros_like(x), torch.zeros_like(x)
    hT = s.h0.to(f)
    for q in range(n):
        state = s.h0[q].to(f)
        for t in range(starts[q], starts[q + 1]):
            before[t] = state
            state = a[t] * state + c[t] * x[t]
            h[t] = state
        hT[q] = state
    if case["op"] == "recurrence":
        return {"y": h, "hT": hT}
    dy, lam, dh0 = s.dy.to(f), torch.zeros_like(x), s.dhT.to(f)
    for q in range(n):
        grad = s.dhT[q].to(f)
        for t in range(starts[q + 1] - 1, starts[q] - 1, -1):
            lam[t] = dy[t] + grad
            grad = a[t] * lam[t]
        dh0[q] = grad
    return {"dx": lam * c, "dgate": lam * (x - before) * c * a, "dh0": dh0}


def exact(case, seed):
    """The definitions in fp64, nothing rounded: an 8-bit value is the
    quotient that it stands in for."""
    s = prepare(case, seed)
    f = torch.float64
    op, rows, cols = case["op"], case["rows"], case["cols"]
    if op in ("recurrence", "recurrence_grad"):
        return _exact_recurrence(case, s)
    if op == "embedding":
        picked = [int(t) for t in s.tokens.tolist()]
        known = torch.tensor([0 <= t < case["vocab"] for t in picked], device="cuda")
        y = s.table.index_select(0, torch.tensor([max(0, t) for t in picked], device="cuda")).to(f)
        return {"y": y * known[:, None].to(f) * s.scale}
    if op == "embedding_grad":
        order = torch.argsort(s.tokens, stable=True)
        token, counts = torch.unique_consecutive(s.tokens[order], return_counts=True)
        run_of = torch.repeat_interleave(torch.arange(len(token), device="cuda"), counts)
        sums = torch.zeros((len(token), cols), dtype=f, device="cuda")
        sums.index_add_(0, run_of, s.dy[order].to(f))
        total = s.dtable.to(f)
        keep = token >= 0
        total[token[keep].long()] += sums[keep] * s.scale
        return {"dtable": total}
    if op in ("checkpoint", "restore"):
        blocks = -(-cols // BLOCK)
        if op == "checkpoint":
            x = s.x.to(f)
            wide = torch.zeros((rows, blocks * BLOCK), dtype=f, device="cuda")
            wide[:, :cols] = x.abs()
            amax = wide.view(rows, blocks, BLOCK).max(dim=2).values
            e = torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448)).clamp_min(MIN_EXP)
            e = torch.where(amax > 448 * 2.0 ** e, e + 1, e)
            return {"q": x * 2.0 ** -e[:, torch.arange(cols, device="cuda") // BLOCK], "scale": None}
        z = s.q.to(f) * 2.0 ** (s.scale.to(f) - 127)[:, torch.arange(cols, device="cuda") // BLOCK]
        c2 = 2 * math.sqrt(2 / math.pi)
        p = {"none": 1.0, "relu": (z > 0).to(f)}.get(case["act"])
        if p is not None:
            y, d = z * p, p
        elif case["act"] == "gelu":       # (1 + tanh u) / 2 = sigmoid(2 u)
            p = _sigmoid64(c2 * (z + 0.044715 * z ** 3))
            y, d = z * p, p + z * p * (1 - p) * c2 * (1 + 3 * 0.044715 * z ** 2)
        else:
            p = _sigmoid64(z)
            y, d = z * p, p + z * p * (1 - p)
        return {"y": y, "dz": s.dy.to(f) * d} if case["grad"] else {"y": y, "z": z}
    loss, lse = torch.zeros(rows, dtype=f, device="cuda"), torch.zeros(rows, dtype=f, device="cuda")
    dlogits = torch.zeros((rows, cols), dtype=f, device="cuda") if case["grad"] else None
    label = s.labels.long()
    known = (label >= 0) & (label < cols)
    for lo in range(0, rows, 512):
        part = slice(lo, min(lo + 512, rows))
        x = s.logits[part].to(f)
        lse[part] = torch.logsumexp(x, dim=1)
        hot = torch.zeros_like(x).scatter_(1, label[part].clamp(0, cols - 1)[:, None], 1.0)
        loss[part] = (lse[part] - x.gather(1, label[part].clamp(0, cols - 1)[:, None])[:, 0]) * known[part].to(f)
        if dlogits is not None:
            w = known[part].to(f) * s.scale * (1 if s.weight is None else s.weight[part].to(f))
            dlogits[part] = (torch.softmax(x, dim=1) - hot) * w[:, None]
    return {"loss": loss, "lse": lse, "dlogits": dlogits} if case["grad"] else {"loss": loss, "lse": lse}
