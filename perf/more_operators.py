"""Cases and plain forms of the operators at both ends of the sparse rows: the lookup of token rows in a table with its
gradient, and the gated feed-forward block over rows sorted by expert (or over all rows alike) with its gradient.

``run`` computes an operator from elementary torch operations in 32 bits, or, with ``own`` set, by this package's
entry points on the same inputs.  ``exact`` states each operator once more in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #

def listed():
    return [
        # the rows of a few tokens being decoded: latency is all
        {"name": "embed_decode", "kind": "lookup", "tokens": 8, "vocab": 32768, "d": 4096, "dtype": "bf16",
         "scale": 1.0, "idle": 0.0},
        # a batch of long prompts, rows scaled by the root of their length
        {"name": "embed_prompt", "kind": "lookup", "tokens": 32768, "vocab": 131072, "d": 4096, "dtype": "bf16",
         "scale": 64.0, "idle": 0.0},
        # a training batch: the whole table's gradient, most of whose rows are 0
        {"name": "embed_train", "kind": "embed_grad", "tokens": 16384, "vocab": 131072, "d": 2048, "dtype": "bf16",
         "out": "bf16", "scale": 1.0, "idle": 0.03, "micro": 1},
        # odd sizes, two micro-batches whose gradients add up in 32 bits
        {"name": "embed_odd", "kind": "embed_grad", "tokens": 5003, "vocab": 50021, "d": 1537, "dtype": "f32",
         "out": "f32", "scale": 1.5, "idle": 0.1, "micro": 2},
        # bytes as tokens: few rows, each the sum over many tokens
        {"name": "embed_bytes", "kind": "embed_grad", "tokens": 65536, "vocab": 300, "d": 1024, "dtype": "f16",
         "out": "f16", "scale": 1.0, "idle": 0.0, "micro": 1},
        # one token through two small experts: latency
        {"name": "ffn_one", "kind": "ffn", "tokens": 1, "k": 2, "experts": 8, "d": 1024, "f": 512, "dtype": "bf16",
         "act": "silu", "align": 1, "dropped": 0.0, "grad": False},
        # a decoding step of a batch: most experts are read for a token or two
        {"name": "ffn_decode", "kind": "ffn", "tokens": 16, "k": 8, "experts": 128, "d": 2048, "f": 768,
         "dtype": "bf16", "act": "silu", "align": 1, "dropped": 0.0, "grad": False},
        # a decoding step through a dense block: its weights have to be read
        {"name": "ffn_dense_decode", "kind": "ffn", "tokens": 4, "k": 1, "experts": 0, "d": 4096, "f": 12288,
         "dtype": "bf16", "act": "silu", "align": 1, "dropped": 0.0, "grad": False},
        # sparse experts over long prompts, segments padded to whole tiles
        {"name": "ffn_prefill", "kind": "ffn", "tokens": 16384, "k": 8, "experts": 128, "d": 2048, "f": 768,
         "dtype": "bf16", "act": "silu", "align": 128, "dropped": 0.0, "grad": False},
        # ragged segments of odd lengths, sizes that no tile divides, entries dropped by a capacity limit, a whole step
        {"name": "ffn_odd", "kind": "ffn", "tokens": 3001, "k": 3, "experts": 17, "d": 1544, "f": 1000,
         "dtype": "f16", "act": "gelu_tanh", "align": 1, "dropped": 0.1, "grad": True},
        # sparse experts, a training step forward and back
        {"name": "ffn_train", "kind": "ffn", "tokens": 16384, "k": 4, "experts": 64, "d": 2048, "f": 1024,
         "dtype": "bf16", "act": "silu", "align": 1, "dropped": 0.0, "grad": True},
        # a dense block, a training step forward and back
        {"name": "ffn_dense_train", "kind": "ffn", "tokens": 4096, "k": 1, "experts": 0, "d": 4096, "f": 12288,
         "dtype": "bf16", "act": "silu", "align": 1, "dropped": 0.0, "grad": True},
    ]


def _log(rng, lo, hi, step=1):
    """A size spread over the logarithm of [lo, hi], a multiple of `step`."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return max(lo, min(hi, v))


def draw(rng):
    kind = rng.choice(["lookup", "embed_grad", "ffn", "ffn"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if kind == "lookup":
        d = _log(rng, 16, 8192, rng.choice([1, 8]))
        return {"kind": kind, "tokens": _log(rng, 1, min(65536, int(2.5e8 / d))), "vocab": _log(rng, 250, int(min(262144, 1e9 / d))),
                "d": d, "dtype": dtype, "scale": rng.choice([1.0, 2.5, d ** 0.5]), "idle": rng.choice([0.0, 0.1])}
    if kind == "embed_grad":
        d = _log(rng, 16, 8192, rng.choice([1, 8]))
        return {"kind": kind, "tokens": _log(rng, 1, min(131072, int(1e8 / d))), "vocab": _log(rng, 250, int(min(262144, 2e8 / d))),
                "d": d, "dtype": dtype, "out": rng.choice([dtype, dtype, "f32"]), "scale": rng.choice([1.0, 2.5]),
                "idle": rng.choice([0.0, 0.1, 0.9]), "micro": rng.choice([1, 1, 2])}
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    step = 1 if dtype == "f32" else 8  # 16-bit rows as wide as a tensor core takes them, 32-bit ones of any width
    grad = rng.random() < 0.5
    most = 2.0e11 if dtype == "f32" else 2.5e12  # operations
    experts = rng.choice([0, _log(rng, 2, 128)])
    k = rng.randint(1, min(8, experts)) if experts else 1
    d, f = _log(rng, 64, 4096, step), _log(rng, 64, 4096 if experts else 12288, step)
    while max(1, experts) * d * f > 6e8:
        experts = max(k, experts // 2) if experts > k else experts
        d, f = max(64, d // 2 // step * step), f
    rows = int(min(65536, most / ((18 if grad else 6) * d * f)))
    return {"kind": kind, "tokens": _log(rng, 1, max(1, rows // k)), "k": k, "experts": experts, "d": d, "f": f, "dtype": dtype,
            "act": rng.choice(["silu", "silu", "gelu_tanh", "relu"]), "align": rng.choice([1, 1, 16, 128]) if experts else 1,
            "dropped": rng.choice([0.0, 0.0, 0.2]) if experts else 0.0, "grad": grad}


def _capacity(case):
    """Rows of the sorted matrix: every entry, and up to align - 1 rows of padding behind each used expert."""
    m, a = case["tokens"] * case["k"], case["align"]
    if not case["experts"]:
        return m
    return (m + min(m, case["experts"]) * (a - 1)) // a * a


def _distinct(tokens, vocab):
    """How many of a vocabulary's rows a batch of log-uniform tokens is expected to name."""
    i = torch.arange(vocab, dtype=torch.float64)
    p = torch.log((i + 2) / (i + 1)) / math.log(vocab + 1)
    return float(-torch.expm1(tokens * torch.log1p(-p)).sum())


def work(case):
    t, s, d = case["tokens"], SIZE[case["dtype"]], case["d"]
    if case["kind"] == "lookup":
        live = t * (1 - case["idle"])
        return {"bytes": t * 4 + t * d * s + _distinct(live, case["vocab"]) * d * s, "flops": live * d}
    if case["kind"] == "embed_grad":
        live, so = t * (1 - case["idle"]), SIZE[case["out"]]
        b = t * 4 + live * d * s + case["vocab"] * d * so
        if case["micro"] == 2:
            b += t * 4 + live * d * s + 2 * _distinct(live, case["vocab"]) * d * so
        return {"bytes": b, "flops": live * d * case["micro"]}
    m, f = t * case["k"] * (1 - case["dropped"]), case["f"]
    used = min(max(1, case["experts"]), m)  # experts whose weights are read
    weights = 3 * d * f * s
    b, ops = 2 * m * d * s + used * weights, 6 * m * d * f
    if case["grad"]:  # forward: gate and up out; back: those, xs, dy and the weights in, dxs and the weights' gradients out
        b += 2 * m * f * s + 2 * m * f * s + 3 * m * d * s + used * weights + max(1, case["experts"]) * weights
        ops *= 3
    return {"bytes": b, "flops": ops}


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, dev = DTYPES[case["dtype"]], "cuda"

    def randn(*shape, scale=1.0):
        if len(shape) == 3:  # a matrix at a time
            out = torch.empty(*shape, device=dev, dtype=dt)
            for part in out:
                part.copy_(torch.randn(*shape[1:], generator=g, device=dev, dtype=torch.float32).mul_(scale))
            return out
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(scale).to(dt)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=dev, dtype=torch.float32)

    t, d, st = case["tokens"], case["d"], {"case": case}
    if case["kind"] in ("lookup", "embed_grad"):
        v = case["vocab"]
        order = torch.randperm(v, generator=g, device=dev)  # frequent tokens lie anywhere in the table

        def tokens():  # their frequencies fall as 1 / rank; some positions are padding (-1)
            rank = torch.exp(rand(t).double() * math.log(v + 1)).to(torch.int64).sub_(1).clamp_(0, v - 1)
            return torch.where(rand(t) < case["idle"], torch.full_like(rank, -1), order[rank]).to(torch.int32)

        if case["kind"] == "lookup":
            st.update(ids=tokens(), table=randn(v, d))
        else:
            st["batches"] = [(tokens(), randn(t, d)) for _ in range(case["micro"])]
        return st
    f, e, k, rows = case["f"], case["experts"], case["k"], _capacity(case)
    lead = (e,) if e else ()
    st.update(w_gate=randn(*lead, f, d, scale=d ** -0.5), w_up=randn(*lead, f, d, scale=d ** -0.5),
              w_down=randn(*lead, d, f, scale=f ** -0.5), xs=randn(rows, d))
    if case["grad"]:
        st["dy"] = randn(rows, d)
    if not e:
        st["ends"], st["plan"] = [(0, rows)], None
        return st
    score = rand(t, e).log_().neg_().log_().neg_() + torch.randn(1, e, generator=g, device=dev) * 0.7  # some experts are liked
    ids = score.topk(k, dim=1).indices.to(torch.int32)
    if case["dropped"]:
        ids = torch.where(rand(t, k) < case["dropped"], torch.full_like(ids, -1), ids)
    counts = torch.bincount(ids.reshape(-1).to(torch.int64) + 1, minlength=e + 1)[1:].tolist()
    ends, at = [], 0
    filled = torch.zeros(rows, dtype=torch.bool, device=dev)
    for n in counts:
        n_padded = -(-n // case["align"]) * case["align"]
        filled[at:at + n] = True
        ends.append((at, at + n_padded))
        at += n_padded
    for name in ("xs", "dy"):  # as dispatch and the gradient of combine leave them: 0 in rows without a token
        if name in st:
            st[name].masked_fill_(~filled[:, None], 0.0)
    st.update(ids=ids, ends=ends, plan=None)
    if own:
        import sparse_matrix_vector_csr_gb300 as spmv

        st["plan"] = spmv.RoutePlan(ids, e, align=case["align"])
    return st


# --------------------------------------------------------------------------- #
# the operators
# --------------------------------------------------------------------------- #

def run(st):
    kind = st["case"]["kind"]
    if own:
        import sparse_matrix_vector_csr_gb300 as spmv

        return {"lookup": _own_lookup, "embed_grad": _own_embed_grad, "ffn": _own_ffn}[kind](spmv, st)
    return {"lookup": _plain_lookup, "embed_grad": _plain_embed_grad, "ffn": _plain_ffn}[kind](st)


def _own_lookup(spmv, st):
    return spmv.embed_rows(st["table"], st["ids"], scale=st["case"]["scale"])


def _own_embed_grad(spmv, st):
    c, grad = st["case"], None
    for ids, dx in st["batches"]:
        grad = spmv.embed_rows_grad(dx, ids, c["vocab"], scale=c["scale"], out=grad, accumulate=grad is not None,
                                    dtype=DTYPES[c["out"]])
    return grad


def _own_ffn(spmv, st):
    c, args = st["case"], (st["xs"], st["w_gate"], st["w_up"], st["w_down"])
    block = st["plan"].feed_forward if c["experts"] else spmv.feed_forward
    res = block(*args, activation=c["act"], keep=c["grad"])
    out = {"y": res.y}
    if c["grad"]:
        out.update(gate=res.gate, up=res.up)
        out["dxs"], out["dw_gate"], out["dw_up"], out["dw_down"] = res.grad(st["dy"])
    return out


def _plain_lookup(st):
    ids = st["ids"].to(torch.int64)
    rows = st["table"][ids.clamp(min=0)].float() * st["case"]["scale"]
    return torch.where(ids[:, None] >= 0, rows, 0.0).to(st["table"].dtype)


def _plain_embed_grad(st):
    c, grad = st["case"], None
    for ids, dx in st["batches"]:
        at = torch.where(ids >= 0, ids, c["vocab"]).to(torch.int64)
        part = torch.zeros(c["vocab"] + 1, c["d"], device=dx.device).index_add_(0, at, dx.float())[:-1] * c["scale"]
        grad = (part if grad is None else grad.float() + part).to(DTYPES[c["out"]])
    return grad


def _gelu_inner(x):
    return math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)


def _act(x, name):
    """The activation of x, and its derivative."""
    if name == "relu":
        return x.clamp(min=0), (x > 0).to(x.dtype)
    if name == "silu":
        s = 1.0 / (1.0 + (-x).exp())
        return x * s, s * (1.0 + x * (1.0 - s))
    s = 1.0 / (1.0 + (-2.0 * _gelu_inner(x)).exp())  # (1 + tanh) / 2
    slope = 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * x * x)
    return x * s, s + x * s * (1.0 - s) * slope


def _plain_ffn(st):
    c, dt = st["case"], st["xs"].dtype
    xs, rows = st["xs"].float(), st["xs"].shape[0]
    wg, wu, wd = (st[n].float() for n in ("w_gate", "w_up", "w_down"))
    if not c["experts"]:
        wg, wu, wd = wg[None], wu[None], wd[None]
    y = torch.zeros(rows, c["d"], device=xs.device)
    if c["grad"]:
        dy = st["dy"].float()
        gate, up = torch.zeros(rows, c["f"], device=xs.device, dtype=dt), torch.zeros(rows, c["f"], device=xs.device, dtype=dt)
        dxs = torch.zeros_like(y)
        dwg, dwu, dwd = torch.zeros_like(wg), torch.zeros_like(wu), torch.zeros_like(wd)
    for e, (a, b) in enumerate(st["ends"]):
        if a == b:
            continue
        x = xs[a:b]
        g, u = x @ wg[e].t(), x @ wu[e].t()
        y[a:b] = (_act(g, c["act"])[0] * u) @ wd[e].t()
        if c["grad"]:  # from the gate and up rows that the forward call returned
            gate[a:b], up[a:b] = g, u
            g, u = gate[a:b].float(), up[a:b].float()
            h, slope = _act(g, c["act"])
            dh = dy[a:b] @ wd[e]
            dg, du = dh * u * slope, dh * h
            dxs[a:b] = dg @ wg[e] + du @ wu[e]
            dwg[e], dwu[e], dwd[e] = dg.t() @ x, du.t() @ x, dy[a:b].t() @ (h * u)
    out = {"y": y.to(dt)}
    if c["grad"]:
        out.update(gate=gate, up=up, dxs=dxs.to(dt))
        for name, v in (("dw_gate", dwg), ("dw_up", dwu), ("dw_down", dwd)):
            out[name] = v.to(dt).view_as(st["w" + name[2:]])
    return out


# --------------------------------------------------------------------------- #
# the same from the definitions, in 64 bits
# --------------------------------------------------------------------------- #

def exact(case, seed):
    if case["kind"] == "ffn":
        if work(case)["flops"] > 8e12:
            return None
        return _exact_ffn(case, prepare(case, seed))
    st = prepare(case, seed)
    if case["kind"] == "lookup":
        one_more = torch.cat([st["table"], torch.zeros_like(st["table"][:1])])  # the row of "no token"
        return one_more[st["ids"].long()].double() * case["scale"]
    total = torch.zeros(case["vocab"], case["d"], dtype=torch.float64, device="cuda")
    for ids, dx in st["batches"]:
        there = ids >= 0
        total.index_put_((ids[there].long(),), dx[there].double() * case["scale"], accumulate=True)
    return total


def _exact_ffn(case, st):
    dt = torch.float64
    gates, ups, ys, back = [], [], [], []
    grads = {"w_gate": [], "w_up": [], "w_down": []}
    weights = {n: st[n] if case["experts"] else st[n][None] for n in grads}
    act = {"silu": torch.nn.functional.silu, "relu": torch.relu,
           "gelu_tanh": lambda v: 0.5 * v * (1.0 + torch.tanh(_gelu_inner(v)))}[case["act"]]
    end = 0
    for e, (a, end) in enumerate(st["ends"]):
        w = {n: v[e].to(dt).requires_grad_(case["grad"]) for n, v in weights.items()}
        x = st["xs"][a:end].to(dt).requires_grad_(case["grad"])
        with torch.set_grad_enabled(case["grad"]):
            g, u = torch.einsum("ti,oi->to", x, w["w_gate"]), torch.einsum("ti,oi->to", x, w["w_up"])
            y = torch.einsum("ti,oi->to", act(g) * u, w["w_down"])
        ys.append(y.detach())
        if case["grad"]:
            gates.append(g.detach()), ups.append(u.detach())
            dx, *dws = torch.autograd.grad(y, [x, *w.values()], st["dy"][a:end].to(dt))
            back.append(dx)
            for name, dw in zip(w, dws):
                grads[name].append(dw)
    rest = st["xs"].shape[0] - end  # rows behind the last segment

    def whole(parts):
        parts.append(torch.zeros(rest, parts[0].shape[1], dtype=dt, device="cuda"))
        return torch.cat(parts)

    out = {"y": whole(ys)}
    if case["grad"]:
        out.update(gate=whole(gates), up=whole(ups), dxs=whole(back))
        for name, v in grads.items():
            out["d" + name] = torch.stack(v).view_as(st[name])
    return out
