"""Cases and plain forms of the sparse-row operators: the largest entries of each row, rows sorted by expert and
back, and distillation from a teacher's top logits.

``run`` computes an operator from elementary torch operations in 32 bits, or, with ``own`` set, by this package's
entry points on the same inputs.  ``exact`` states each operator once more in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
LOWEST = float("-inf")


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #

def listed():
    return [
        # a router's choice for a few tokens being decoded: latency is all
        {"name": "gate_decode", "kind": "gate", "rows": 8, "n": 64, "k": 4, "dtype": "f32", "weights": "selected",
         "masked": 0.0, "grad": False},
        # a router's choice and its gradient over a training batch, a few experts masked out, some tokens padding
        {"name": "gate_train", "kind": "gate", "rows": 32768, "n": 256, "k": 8, "dtype": "bf16", "weights": "row",
         "masked": 0.05, "grad": True},
        # a teacher's top logits of a handful of rows (one row spread over many SMs)
        {"name": "top_few", "kind": "top", "rows": 4, "n": 131072, "k": 64, "dtype": "bf16", "temperature": 1.0},
        # a teacher's top logits over a batch, a vocabulary of odd size (rows start at any address)
        {"name": "top_odd", "kind": "top", "rows": 4096, "n": 50021, "k": 32, "dtype": "f16", "temperature": 2.0},
        # sparse experts serving a few tokens: sort, rows out, rows back
        {"name": "route_decode", "kind": "route", "rows": 4, "k": 8, "experts": 128, "d": 4096, "dtype": "bf16",
         "align": 1, "dropped": 0.0, "grad": False},
        # sparse experts over a long prompt, segments padded to whole tiles
        {"name": "route_prefill", "kind": "route", "rows": 16384, "k": 8, "experts": 128, "d": 4096, "dtype": "bf16",
         "align": 128, "dropped": 0.0, "grad": False},
        # odd sizes: few experts, rows of odd length in float32, entries dropped by a capacity limit
        {"name": "route_odd", "kind": "route", "rows": 3001, "k": 3, "experts": 17, "d": 1537, "dtype": "f32",
         "align": 16, "dropped": 0.1, "grad": True},
        # a training step's whole way: forward and both gradients
        {"name": "route_train", "kind": "route", "rows": 16384, "k": 4, "experts": 64, "d": 2048, "dtype": "bf16",
         "align": 1, "dropped": 0.0, "grad": True},
        # a small distillation step (loss and gradient at once)
        {"name": "distill_small", "kind": "distill", "rows": 8, "vocab": 32768, "k": 16, "dtype": "f32",
         "temperature": 2.0, "tail": False, "idle": 0.0, "mode": "fused"},
        # a full training batch, a large vocabulary, 64 teacher logits a token, padding tokens among them
        {"name": "distill_train", "kind": "distill", "rows": 8192, "vocab": 131072, "k": 64, "dtype": "bf16",
         "temperature": 1.0, "tail": False, "idle": 0.03, "mode": "fused"},
        # odd vocabulary, the rest of the teacher's mass as one more class, forward and gradient as two calls
        {"name": "distill_odd", "kind": "distill", "rows": 2047, "vocab": 50021, "k": 20, "dtype": "bf16",
         "temperature": 1.5, "tail": True, "idle": 0.03, "mode": "two"},
        # held-out loss only
        {"name": "distill_eval", "kind": "distill", "rows": 2048, "vocab": 65536, "k": 128, "dtype": "f16",
         "temperature": 1.0, "tail": True, "idle": 0.0, "mode": "loss"},
    ]


def _log(rng, lo, hi, odd=0.5):
    """A size spread over the logarithm of [lo, hi]; half of them multiples of 8 where that leaves room."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 64 and rng.random() >= odd:
        v -= v % 8
    v = max(lo, min(hi, v))
    return v + 1 if v == 3072 else v


def draw(rng):
    kind = rng.choice(["gate", "top", "route", "distill"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    most = 2.0e9  # bytes; the largest listed case has more than twice that
    if kind == "gate":
        rows, n = _log(rng, 1, 65536), _log(rng, 4, 512)
        return {"kind": kind, "rows": rows, "n": n, "k": rng.randint(1, min(16, n)), "dtype": dtype,
                "weights": rng.choice(["selected", "row"]), "masked": rng.choice([0.0, 0.1, 0.6]),
                "grad": rng.random() < 0.5}
    if kind == "top":
        n = _log(rng, 600, 200000)
        rows = _log(rng, 1, int(min(8192, most / 4 / (n * SIZE[dtype]))))
        return {"kind": kind, "rows": rows, "n": n, "k": _log(rng, 1, 128), "dtype": dtype,
                "temperature": rng.choice([0.7, 1.0, 2.0])}
    if kind == "route":
        k, d = rng.randint(1, 8), _log(rng, 64, 8192)
        rows = _log(rng, 1, int(min(32768, most / (k * d * SIZE[dtype] * 8))))
        return {"kind": kind, "rows": rows, "k": k, "experts": _log(rng, max(2, k), 512), "d": d, "dtype": dtype,
                "align": rng.choice([1, 16, 128]), "dropped": rng.choice([0.0, 0.0, 0.2]),
                "grad": rng.random() < 0.5}
    vocab = _log(rng, 500, 200000)
    rows = _log(rng, 1, int(min(16384, most / (vocab * SIZE[dtype] * 3))))
    return {"kind": kind, "rows": rows, "vocab": vocab, "k": _log(rng, 1, 128), "dtype": dtype,
            "temperature": rng.choice([0.7, 1.0, 2.0, 4.0]), "tail": rng.random() < 0.5,
            "idle": rng.choice([0.0, 0.1]), "mode": rng.choice(["fused", "two", "loss"])}


def _capacity(case):
    """Rows of the sorted matrix: every entry, and up to align - 1 rows of padding behind each used expert."""
    m, a = case["rows"] * case["k"], case["align"]
    return (m + min(m, case["experts"]) * (a - 1)) // a * a


def work(case):
    kind, t, k, s = case["kind"], case["rows"], case["k"], SIZE[case["dtype"]]
    if kind == "gate":
        b, f = t * case["n"] * s + t * k * 8, t * case["n"] * 4
        if case["grad"]:  # the weights' gradient in, the logits' gradient out
            b, f = b + t * k * 4 + t * case["n"] * s, f + t * case["n"] * 4
        return {"bytes": b, "flops": f}
    if kind == "top":
        return {"bytes": t * case["n"] * s + t * k * 8 + t * 4, "flops": t * case["n"] * 5}
    if kind == "route":
        d, rows, m = case["d"] * s, _capacity(case), t * k
        b = t * k * 4 * 3 + rows * 4 + (t + rows) * d + (m + t) * d  # ids, weights, slots, sources; out; back
        f = 2 * m * case["d"]
        if case["grad"]:
            b += (t + m + rows) * d + m * 4 + (m + t) * d  # of combine: dy, ys, dys, dw; of dispatch: dxs, dx
            f += 4 * m * case["d"]
        return {"bytes": b, "flops": f}
    passes = {"fused": 2, "two": 3, "loss": 1}[case["mode"]]
    return {"bytes": t * case["vocab"] * s * passes + t * k * 8 + t * 8,
            "flops": t * case["vocab"] * {"fused": 7, "two": 8, "loss": 4}[case["mode"]]}


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, dev = DTYPES[case["dtype"]], "cuda"

    def randn(*shape, scale=1.0, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(scale).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=dev, dtype=torch.float32)

    t, k, kind = case["rows"], case["k"], case["kind"]
    st = {"case": case}
    if kind == "gate":
        x = randn(t, case["n"], scale=2.0)
        if case["masked"]:
            x = torch.where(rand(t, case["n"]) < case["masked"], torch.full_like(x, LOWEST), x)
            x = torch.where(rand(t, 1) < 0.02, torch.full_like(x, LOWEST), x)  # tokens that are padding
        st["x"], st["dw"] = x, randn(t, k, dtype=torch.float32)
    elif kind == "top":
        st["x"] = randn(t, case["n"], scale=2.5)
    elif kind == "route":
        e, d = case["experts"], case["d"]
        score = rand(t, e).log_().neg_().log_().neg_() + randn(1, e, scale=0.7, dtype=torch.float32)  # some experts are liked
        ids = score.topk(k, dim=1).indices.to(torch.int32)
        if case["dropped"]:
            ids = torch.where(rand(t, k) < case["dropped"], torch.full_like(ids, -1), ids)
        w = rand(t, k) + 0.1
        st.update(ids=ids, w=w / w.sum(1, keepdim=True), x=randn(t, d), ys=randn(_capacity(case), d))
        if case["grad"]:
            st.update(dy=randn(t, d), dxs=randn(_capacity(case), d))
    else:
        v, tau = case["vocab"], case["temperature"]
        z = randn(t, v, scale=1.5)
        # k columns of each row, one from each of k equal parts of the vocabulary, in random order
        part = (torch.arange(k, device=dev, dtype=torch.float32) + rand(t, k)) * (v / k)
        ids = part.to(torch.int64).clamp_(max=v - 1)
        edge = (torch.arange(k + 1, device=dev, dtype=torch.float64) * v / k).ceil().to(torch.int64)
        ids = torch.minimum(torch.maximum(ids, edge[:-1]), edge[1:] - 1)
        ids = ids.gather(1, rand(t, k).argsort(1))
        teacher = (rand(t, k).log_().neg_() * 2.0 + 4.0).sort(1, descending=True).values
        z.scatter_add_(1, ids, (teacher * 0.7).to(dt))  # the student likes them too
        lse = torch.logsumexp(teacher / tau, 1) - torch.log1p(-(rand(t) * 0.3 + 0.01))
        ids = torch.where(rand(t, 1) < case["idle"], torch.full_like(ids, -1), ids)  # tokens without a target
        st.update(z=z, ids=ids.to(torch.int32), teacher=teacher, lse=lse if case["tail"] else None,
                  dloss=rand(t) + 0.5, scale=1.0 / t)
    return st


# --------------------------------------------------------------------------- #
# the operators
# --------------------------------------------------------------------------- #

def run(st):
    kind = st["case"]["kind"]
    if own:
        import sparse_matrix_vector_csr_gb300 as spmv

        return {"gate": _own_gate, "top": _own_top, "route": _own_route, "distill": _own_distill}[kind](spmv, st)
    return {"gate": _plain_gate, "top": _plain_top, "route": _plain_route, "distill": _plain_distill}[kind](st)


def _own_gate(spmv, st):
    c = st["case"]
    top = spmv.topk_rows(st["x"], c["k"], weights=c["weights"])
    out = {"ids": top.ids, "weights": top.weights}
    if c["grad"]:
        out["dx"] = top.grad(st["dw"])
    return out


def _own_top(spmv, st):
    c = st["case"]
    top = spmv.topk_rows(st["x"], c["k"], temperature=c["temperature"], lse=True)
    return {"ids": top.ids, "vals": top.vals, "lse": top.lse}


def _own_route(spmv, st):
    c = st["case"]
    plan = spmv.RoutePlan(st["ids"], c["experts"], align=c["align"])
    out = {"xs": plan.dispatch(st["x"]), "y": plan.combine(st["ys"], st["w"]), "offsets": plan.offsets,
           "slots": plan.slots, "sources": plan.sources}
    if c["grad"]:
        out["dys"], out["dw"] = plan.combine_grad(st["dy"], st["ys"], st["w"])
        out["dx"] = plan.dispatch_grad(st["dxs"])
    return out


def _own_distill(spmv, st):
    c = st["case"]
    args = (st["z"], st["ids"], st["teacher"])
    kw = {"teacher_lse": st["lse"], "temperature": c["temperature"]}
    if c["mode"] == "fused":
        loss, dz = spmv.distill_loss_grad(*args, **kw, scale=st["scale"])
        return {"loss": loss, "dz": dz}
    res = spmv.distill_loss(*args, **kw)
    return {"loss": res.loss, "dz": res.grad(st["dloss"])} if c["mode"] == "two" else {"loss": res.loss}


def _largest(f, k):
    """ids of the k largest of each row of f (32 bits), descending, ties to the lowest column; -1 for -inf."""
    n = f.shape[1]
    bits = (f + 0.0).view(torch.int32)
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64)  # ordered as the numbers are
    key = bits * (1 << 32) + (n - 1 - torch.arange(n, device=f.device))
    ids = key.topk(k, dim=1).indices
    vals = f.gather(1, ids)
    return torch.where(vals == LOWEST, torch.full_like(ids, -1), ids), vals


def _plain_lse(zt):
    """The log of the sum of exp over each row; -inf where nothing is finite."""
    m = zt.max(1, keepdim=True).values
    m0 = torch.where(m == LOWEST, torch.zeros_like(m), m)
    return m0 + (zt - m0).exp().sum(1, keepdim=True).log()


def _plain_gate(st):
    c, f = st["case"], st["x"].float()
    ids, vals = _largest(f, c["k"])
    none = ids < 0
    lse = _plain_lse(vals if c["weights"] == "selected" else f)
    w = torch.where(none, torch.zeros_like(vals), (vals - lse).exp())
    out = {"ids": ids.to(torch.int32), "weights": w}
    if c["grad"]:
        wd = w * st["dw"]
        dot = wd.sum(1, keepdim=True)
        if c["weights"] == "selected":
            dx, add = torch.zeros_like(f), wd - w * dot
        else:
            dx, add = torch.where(f == LOWEST, torch.zeros_like(f), (f - lse).exp()) * -dot, wd
        out["dx"] = dx.scatter_add(1, ids.clamp(min=0), add).to(st["x"].dtype)
    return out


def _plain_top(st):
    c, f = st["case"], st["x"].float()
    ids, vals = _largest(f, c["k"])
    return {"ids": ids.to(torch.int32), "vals": vals, "lse": _plain_lse(f / c["temperature"])[:, 0]}


def _plain_plan(ids, experts, align, rows):
    m, dev = ids.numel(), ids.device
    flat = ids.reshape(-1).to(torch.int64)
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    sorted_key, order = key.sort(stable=True)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=dev).scatter_add_(0, key, torch.ones_like(key))
    first = counts.cumsum(0) - counts
    padded = (counts[:experts] + align - 1) // align * align
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), padded.cumsum(0)])
    slot = offsets[sorted_key.clamp(max=experts - 1)] + torch.arange(m, device=dev) - first[sorted_key]
    used = sorted_key < experts
    slots = torch.empty_like(flat).scatter_(0, order, torch.where(used, slot, torch.full_like(slot, -1)))
    sources = torch.full((rows + 1,), -1, dtype=torch.int64, device=dev)
    sources.scatter_(0, torch.where(used, slot, torch.full_like(slot, rows)), torch.where(used, order, torch.full_like(order, -1)))
    return offsets, slots.view(ids.shape), sources[:rows]


def _plain_route(st):
    c = st["case"]
    k, rows, dt = c["k"], _capacity(c), st["x"].dtype
    offsets, slots, sources = _plain_plan(st["ids"], c["experts"], c["align"], rows)
    used, at = slots >= 0, slots.clamp(min=0)
    token, here = (sources.clamp(min=0) // k), sources >= 0

    def back(rows_of, weights):  # sum of each token's rows
        return (torch.where(used[..., None], rows_of.float()[at], 0.0) * weights[..., None]).sum(1).to(dt)

    out = {"xs": torch.where(here[:, None], st["x"][token], 0.0), "y": back(st["ys"], st["w"]),
           "offsets": offsets.to(torch.int32), "slots": slots.to(torch.int32), "sources": sources.to(torch.int32)}
    if c["grad"]:
        w_row = st["w"].reshape(-1)[sources.clamp(min=0)]
        out["dys"] = torch.where(here[:, None], st["dy"].float()[token] * w_row[:, None], 0.0).to(dt)
        out["dw"] = torch.where(used, (st["dy"].float()[:, None, :] * st["ys"].float()[at]).sum(2), 0.0)
        out["dx"] = back(st["dxs"], torch.ones_like(st["w"]))
    return out


def _plain_distill(st):
    c = st["case"]
    tau, zt = c["temperature"], st["z"].float() / c["temperature"]
    valid = st["ids"] >= 0
    at = st["ids"].clamp(min=0).to(torch.int64)
    live = valid.any(1, keepdim=True)
    tt = torch.where(valid, st["teacher"] / tau, LOWEST)
    lse = _plain_lse(zt)
    zk = zt.gather(1, at)
    zero = torch.zeros_like(tt)
    norm = _plain_lse(tt) if st["lse"] is None else st["lse"][:, None]
    p = torch.where(valid, (tt - norm).exp(), zero)
    loss = torch.where(p > 0, p * (tt - norm - zk + lse), zero).sum(1, keepdim=True)
    rest, lse_rest = None, None
    if st["lse"] is not None:
        rest = (1.0 - p.sum(1, keepdim=True)).clamp(min=0)
        top = torch.zeros_like(zt).scatter_add_(1, at, valid.float()) > 0
        lse_rest = _plain_lse(torch.where(top, LOWEST, zt))
        loss = loss + torch.where(rest > 0, rest * (rest.log() - lse_rest + lse), torch.zeros_like(rest))
    out = {"loss": torch.where(live, loss, torch.zeros_like(loss))[:, 0]}
    if c["mode"] != "loss":
        row = st["dloss"][:, None] if c["mode"] == "two" else st["scale"]
        dz = (zt - lse).exp()
        if rest is not None:
            dz = torch.where(top, dz, dz - rest * (zt - lse_rest).exp())
        dz = dz.scatter_add(1, at, -p)
        out["dz"] = torch.where(live, dz * (row / tau), torch.zeros_like(dz)).to(st["z"].dtype)
    return out


# --------------------------------------------------------------------------- #
# the same from the definitions, in 64 bits
# --------------------------------------------------------------------------- #

def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind in ("gate", "top"):
        return _exact_rows(case, st)
    return _exact_route(case, st) if kind == "route" else _exact_distill(case, st)


def _exact_rows(case, st):
    x, k, n = st["x"], case["k"], case["n"]
    tau = case.get("temperature", 1.0)
    parts = []
    step = max(1, int(2e8 // n))
    for a in range(0, x.shape[0], step):
        f = x[a:a + step].double()
        val, col = f.sort(dim=1, descending=True, stable=True)
        val, col = val[:, :k], col[:, :k].clone()
        none = val == LOWEST
        col[none] = -1
        if case["kind"] == "top":
            parts.append({"ids": col, "vals": val, "lse": torch.logsumexp(f / tau, 1)})
            continue
        every = torch.nan_to_num(torch.softmax(val if case["weights"] == "selected" else f, 1))
        w = every if case["weights"] == "selected" else every.gather(1, col.clamp(min=0))
        w = torch.where(none, 0.0, w)
        got = {"ids": col, "weights": w}
        if case["grad"]:
            dw = st["dw"][a:a + step].double()
            s = (w * dw).sum(1, keepdim=True)
            full = torch.zeros_like(f).scatter_add_(1, col.clamp(min=0), torch.where(none, 0.0, w * dw))
            like = every if case["weights"] == "row" else torch.zeros_like(f).scatter_add_(1, col.clamp(min=0), w)
            got["dx"] = full - like * s
        parts.append(got)
    return {name: torch.cat([p[name] for p in parts]) for name in parts[0]}


def _exact_route(case, st):
    ids, k, e, a = st["ids"].cpu().numpy(), case["k"], case["experts"], case["align"]
    rows, dev = _capacity(case), st["x"].device
    flat = ids.reshape(-1)
    lists = [np.flatnonzero(flat == j) for j in range(e)]
    offsets = np.zeros(e + 1, np.int64)
    slots, sources = np.full(flat.size, -1, np.int64), np.full(rows, -1, np.int64)
    for j, at in enumerate(lists):
        place = offsets[j] + np.arange(at.size)
        slots[at], sources[place] = place, at
        offsets[j + 1] = offsets[j] + -(-at.size // a) * a
    src = torch.from_numpy(sources).to(dev)
    filled = torch.from_numpy(np.flatnonzero(sources >= 0)).to(dev)
    token, w = src[filled] // k, st["w"].double().reshape(-1)[src[filled]]
    x, ys = st["x"], st["ys"]

    def spread(values):
        return torch.zeros(rows, x.shape[1], dtype=torch.float64, device=dev).index_copy_(0, filled, values)

    def gathered(values):  # in the order of the sorted rows, one column block at a time
        return torch.zeros(x.shape[0], x.shape[1], dtype=torch.float64, device=dev).index_add_(0, token, values)

    out = {"xs": spread(x.double()[token]), "y": gathered(ys.double()[filled] * w[:, None]),
           "offsets": torch.from_numpy(offsets), "slots": torch.from_numpy(slots.reshape(ids.shape)),
           "sources": src}
    if case["grad"]:
        dy = st["dy"].double()[token]
        out["dys"] = spread(dy * w[:, None])
        dw = torch.zeros(flat.size, dtype=torch.float64, device=dev)
        dw[src[filled]] = (dy * ys.double()[filled]).sum(1)
        out["dw"] = dw.view(*ids.shape)
        out["dx"] = gathered(st["dxs"].double()[filled])
    return out


def _exact_distill(case, st):
    t, v, tau = case["rows"], case["vocab"], float(case["temperature"])
    losses, grads = [], []
    step = max(1, int(1e8 // v))
    for a in range(0, t, step):
        z = st["z"][a:a + step].double() / tau
        ids, tt = st["ids"][a:a + step].long(), st["teacher"][a:a + step].double() / tau
        live = ids[:, 0] >= 0  # a row has all its entries, or none
        at = ids.clamp(min=0)
        logq = torch.log_softmax(z, 1)
        if st["lse"] is None:
            logp = torch.log_softmax(tt, 1)
        else:
            logp = tt - st["lse"][a:a + step].double()[:, None]
        p = logp.exp()
        kl = (p * (logp - logq.gather(1, at))).sum(1)
        q = logq.exp()
        target = torch.zeros_like(q).scatter_(1, at, p)
        if st["lse"] is not None:
            rest = 1.0 - p.sum(1)
            others = q.scatter(1, at, 0.0)
            mass = others.sum(1)
            kl = kl + rest * (rest.log() - mass.log())
            target += others * (rest / mass)[:, None]
        losses.append(torch.where(live, kl, 0.0))
        if case["mode"] != "loss":
            row = st["dloss"][a:a + step].double() if case["mode"] == "two" else torch.full_like(kl, st["scale"])
            grads.append(torch.where(live[:, None], (q - target) * (row / tau)[:, None], 0.0))
    out = {"loss": torch.cat(losses)}
    if case["mode"] != "loss":
        out["dz"] = torch.cat(grads)
    return out
