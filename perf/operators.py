"""Workloads of the training-step operators: counter-based dropout, and the
expert router with its per-expert counts and balance loss.

Each case is one call as a data-parallel training step makes it.  With
``own`` false ``run`` computes the operator from elementary torch operations
in fp32 (fp64 for sums over tokens); with ``own`` true it calls the library.
``exact`` evaluates the definitions in fp64, separately from the plain form.

Dropout of element i (row-major position in the tensor): the 16-bit dither d_i
is word (i & 7) >> 1 (low half for even i) of Philox4x32-10 with key = seed and
counter = (low 32 bits of i >> 3, the next 16 bits | worker << 16, round,
2^31 + site); with T = round(65536 p) the element is kept iff d_i >= T and
scaled by 65536 / (65536 - T).

Router: softmax over the experts, the k largest logits chosen (ties to the
lowest index, -inf never), gates = chosen probabilities, divided by their sum
if ``renorm``.  With c_e the choices and S_e the summed probabilities over the
N routed tokens of all workers, loss = E / (k N^2) * sum_e c_e S_e and
coef_e = E c_e / (k N^2) is its derivative by any token's probability of e.
"""
import math

import numpy as np
import torch

own = False


def _drop(name, rows, cols, dtype="bf16", p=0.1, residual=False, layout="flat", dir="fwd"):
    return {"name": name, "op": "dropout", "dir": dir, "rows": rows, "cols": cols, "dtype": dtype, "p": p,
            "residual": residual, "layout": layout}


def _route(name, tokens, experts, top_k, dtype="bf16", workers=1, renorm=True, mask=0.0, closed=0.0, dir="fwd"):
    return {"name": name, "op": "route", "dir": dir, "tokens": tokens, "experts": experts, "top_k": top_k,
            "dtype": dtype, "workers": workers, "renorm": renorm, "mask": mask, "closed": closed}


def listed():
    return [
        # a tiny batch's hidden state: launch latency
        _drop("dropout_small", 16, 256, residual=True),
        # the residual branch of a block: one worker's tokens by a hidden size
        _drop("dropout_block", 8192, 4096, residual=True),
        # its backward at an odd width: rows start at any alignment of the flat index
        _drop("dropout_backward_odd", 4097, 1337, p=0.25, dir="bwd"),
        # half of a wider fp32 projection (a strided view), rate as of attention outputs
        _drop("dropout_fp32_slice", 4096, 2048, dtype="f32", p=0.2, layout="slice"),
        # the largest: long sequences by a wide hidden size
        _drop("dropout_large", 16384, 8192, residual=True),
        # one token
        _route("route_one", 1, 64, 8),
        # one worker's tokens, fp32 logits as routers usually compute them
        _route("route_fp32", 8192, 64, 8, dtype="f32"),
        # odd token and expert counts, padding tokens masked off, some experts closed to some tokens
        _route("route_odd", 4099, 60, 4, renorm=False, mask=0.2, closed=0.1),
        # the largest: four workers' batches folded into one balance loss
        _route("route_workers", 131072, 256, 8, workers=4),
        # gradients by the logits, from the gates' and the loss's
        _route("route_backward_fp32", 8192, 64, 8, dtype="f32", dir="bwd"),
        _route("route_backward_workers", 131072, 256, 8, workers=4, dir="bwd"),
        # forward and backward through autograd, as a training step does
        _route("route_step", 16384, 128, 2, renorm=False, mask=0.1, dir="step"),
    ]


def _log(rng, lo, hi):
    """An integer in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.45:
        n = _log(rng, 16, 1 << 27)                       # elements, at most dropout_large's
        cols = max(1, min(n, _log(rng, 8, 8192)))
        if rng.random() < 0.6:
            cols = max(8, cols // 8 * 8)
        c = _drop("", max(1, n // cols), cols, rng.choice(["bf16", "bf16", "f32"]),
                  rng.choice([0.0, 0.05, 0.1, 0.25, 0.5, 0.9]), rng.random() < 0.5,
                  rng.choice(["flat", "flat", "slice"]), rng.choice(["fwd", "bwd"]))
        if c["dtype"] == "f32":                          # no more bytes than dropout_large moves
            c["rows"] = max(1, c["rows"] // 2)
        if c["dir"] == "bwd":
            c["residual"] = False
    else:
        experts = _log(rng, 4, 512)
        if rng.random() < 0.6:
            experts = max(4, experts // 4 * 4)
        workers = rng.choice([1, 1, 2, 4])
        dtype = rng.choice(["bf16", "f32"])
        cap = (1 << 26) // (experts * workers * (2 if dtype == "f32" else 1))
        c = _route("", _log(rng, 1, max(1, min(131072, cap))), experts, rng.randint(1, min(8, experts)), dtype, workers,
                   rng.random() < 0.6, rng.choice([0.0, 0.0, 0.2]), rng.choice([0.0, 0.0, 0.1]),
                   rng.choice(["fwd", "bwd", "step"]))
    del c["name"]
    return c


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


class _State:
    pass


def _prepare(case, seed):
    s = _State()
    s.case = case
    dt = _dtype(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    s.seed = (seed * 0x9E3779B97F4A7C15 + 5) % 2 ** 64    # the key of the run, the step, the worker, the call in the model
    s.round, s.worker, s.site = seed % 1000, seed % 5, 3

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    if case["op"] == "dropout":
        r, c = case["rows"], case["cols"]
        wide = 2 * c if case["layout"] == "slice" else c
        s.x = normal(r, wide).to(dt)[:, :c]              # activations, or their gradient
        s.residual = normal(r, wide).to(dt)[:, :c] if case["residual"] else None
        return s
    W, T, E, k = case["workers"], case["tokens"], case["experts"], case["top_k"]
    lean = normal(E)                                     # some experts are preferred
    s.logits, s.mask, s.dgates = [], [], []
    for _ in range(W):
        l = 2.0 * normal(T, E) + lean
        if case["closed"]:
            l = torch.where(torch.rand(T, E, generator=g, device="cuda") < case["closed"], -math.inf, l)
            l[torch.rand(T, generator=g, device="cuda") < 0.01] = -math.inf      # tokens with every expert closed
        s.logits.append(l.to(dt))
        s.mask.append(torch.rand(T, generator=g, device="cuda") >= case["mask"] if case["mask"] else None)
        s.dgates.append(normal(T, k) / max(1, W * T))    # of a mean over the tokens
    s.dloss = torch.full((1,), 0.01, device="cuda")      # the loss's weight
    return s


def prepare(case, seed):
    s = _prepare(case, seed)
    if case["op"] == "route" and case["dir"] == "bwd":   # what the forward left
        f = _route_plain(s)
        s.ids, s.coef = f["ids"], f["coef"]
    return s


# ---- plain forms ------------------------------------------------------------

def _words(seed, c0, c1, c2, c3):
    """Philox4x32-10 on int64 tensors of 32-bit values."""
    m32 = 0xFFFFFFFF
    k0, k1 = seed & m32, seed >> 32 & m32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32 & m32) ^ c1 ^ k0, b & m32, (a >> 32 & m32) ^ c3 ^ k1, a & m32
        k0, k1 = k0 + 0x9E3779B9 & m32, k1 + 0xBB67AE85 & m32
    return torch.stack((c0, c1, c2, c3), 1)


def _dropout_plain(s):
    x = s.x
    n = x.numel()
    block = torch.arange((n + 7) // 8, device=x.device)
    zero = torch.zeros_like(block)
    w = _words(s.seed, block & 0xFFFFFFFF, block >> 32 | s.worker << 16, zero + s.round, zero + (0x80000000 | s.site))
    d = torch.stack((w & 0xFFFF, w >> 16), 2).reshape(-1)[:n].reshape(x.shape)
    drop = round(s.case["p"] * 65536)
    y = torch.where(d >= drop, x.float() * (65536 / (65536 - drop)), 0.0)
    if s.residual is not None:
        y = s.residual.float() + y
    return y.to(x.dtype)


def _softmax(logits, mask):
    """(probabilities, routed tokens) in fp32; zero rows for tokens that are masked off or have no open expert."""
    l = logits.float()
    ok = torch.isfinite(l).any(1)
    if mask is not None:
        ok = ok & mask
    l = torch.where(ok[:, None], l, 0.0)
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True) * ok[:, None], ok


def _choose(logits, p, ok, k, renorm):
    v, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    ids = torch.where(ok[:, None] & (v[:, :k] > -math.inf), ids[:, :k], -1)
    g = torch.where(ids >= 0, p.gather(1, ids.clamp(min=0)), 0.0)
    if renorm:
        t = g.sum(1, keepdim=True)
        g = torch.where(t > 0, g / t, 0.0)
    return ids.int(), g


def _route_plain(s):
    c = s.case
    E, k = c["experts"], c["top_k"]
    dev = s.logits[0].device
    out = {"ids": [], "gates": []}
    counts = torch.zeros(E, dtype=torch.int64, device=dev)
    probs = torch.zeros(E, dtype=torch.float64, device=dev)
    tokens = torch.zeros((), dtype=torch.float64, device=dev)
    for logits, mask in zip(s.logits, s.mask):
        p, ok = _softmax(logits, mask)
        ids, g = _choose(logits, p, ok, k, c["renorm"])
        out["ids"].append(ids)
        out["gates"].append(g)
        counts += torch.bincount(ids.reshape(-1).long() + 1, minlength=E + 1)[1:]
        probs += p.sum(0, dtype=torch.float64)
        tokens += ok.sum()
    coef = counts * (E / k) / tokens.clamp(min=1) ** 2
    return {**out, "loss": (coef * probs).sum().float().reshape(1), "coef": coef.float(), "counts": counts}


def _route_backward_plain(s, ids_of, coef):
    c = s.case
    grads = []
    for logits, mask, ids, dg in zip(s.logits, s.mask, ids_of, s.dgates):
        p, _ = _softmax(logits, mask)
        a = s.dloss * coef
        open_ = ids >= 0
        at = ids.clamp(min=0).long()
        ps = torch.where(open_, p.gather(1, at), 0.0)
        dg = torch.where(open_, dg, 0.0)
        D = (p * a).sum(1, keepdim=True)
        if c["renorm"]:
            t = ps.sum(1, keepdim=True)
            g = torch.where(t > 0, ps / t, 0.0)
            top = g * (dg - (g * dg).sum(1, keepdim=True))
        else:
            D = D + (ps * dg).sum(1, keepdim=True)
            top = ps * dg
        grads.append((p * (a - D)).scatter_add(1, at, torch.where(open_, top, 0.0)).to(logits.dtype))
    return grads


# ---- one pass ---------------------------------------------------------------

def run(s):
    c = s.case
    if own:
        return _run_own(s)
    if c["op"] == "dropout":
        return _dropout_plain(s)
    if c["dir"] == "fwd":
        return _route_plain(s)
    if c["dir"] == "bwd":
        return _route_backward_plain(s, s.ids, s.coef)
    f = _route_plain(s)
    return {**f, "dlogits": _route_backward_plain(s, f["ids"], f["coef"])}


def _run_own(s):
    from compressed_hop_gradient_amd import dq, train
    c = s.case
    if c["op"] == "dropout":
        key = dict(seed=s.seed, rnd=s.round, worker=s.worker, site=s.site)
        if c["dir"] == "bwd":
            return dq.dropout_backward(s.x, c["p"], **key)
        return dq.dropout(s.x, c["p"], residual=s.residual, **key)
    k, renorm = c["top_k"], c["renorm"]
    if c["dir"] == "bwd":
        return [dq.route_backward(l, i, dgates=d, coef=s.coef, dloss=s.dloss, renorm=renorm, mask=m)
                for l, m, i, d in zip(s.logits, s.mask, s.ids, s.dgates)]
    if c["dir"] == "fwd":
        ids, gates, stats = [], [], None
        for l, m in zip(s.logits, s.mask):
            i, g, stats = dq.route(l, k, renorm=renorm, mask=m, stats=stats)
            ids.append(i)
            gates.append(g)
        loss, coef, counts = dq.balance(stats, k)
        return {"ids": ids, "gates": gates, "loss": loss, "coef": coef, "counts": counts}
    leaves = [l.detach().requires_grad_() for l in s.logits]
    r = train.route(leaves, k, renorm=renorm, masks=s.mask)
    grads = torch.autograd.grad([*r.gates, r.loss], leaves, [*s.dgates, s.dloss])
    return {"ids": r.ids, "gates": [g.detach() for g in r.gates], "loss": r.loss.detach(), "coef": r.coef,
            "counts": r.counts, "dlogits": list(grads)}


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"]
        # per 8 elements 10 rounds of two products and four xors; per element a comparison, a product, an addition
        return {"bytes": n * es * (3 if case["residual"] else 2), "flops": n * (60 / 8 + 3)}
    W, T, E, k = case["workers"], case["tokens"], case["experts"], case["top_k"]
    fwd = W * (T * E * es + 8 * T * k + (T if case["mask"] else 0)) + 12 * E
    bwd = W * (2 * T * E * es + 8 * T * k + (T if case["mask"] else 0)) + 4 * E
    step = W * (2 * T * E * es + 12 * T * k + (T if case["mask"] else 0)) + 12 * E
    n = W * T * E
    return {"bytes": {"fwd": fwd, "bwd": bwd, "step": step}[case["dir"]],
            "flops": {"fwd": 6 * n, "bwd": 9 * n, "step": 15 * n}[case["dir"]]}


# ---- the definitions in 64 bits ----------------------------------------------

def _dithers(seed, worker, rnd, site, n):
    """The 16-bit dithers of elements 0 .. n - 1, from numpy's unsigned integers."""
    u = np.uint64
    out = np.empty((n + 7) // 8 * 8, np.uint16)
    step = 1 << 18
    for b0 in range(0, (n + 7) // 8, step):
        b = np.arange(b0, min((n + 7) // 8, b0 + step), dtype=u)
        lo = u(0xFFFFFFFF)
        x = [b & lo, (b >> u(32)) | u(worker << 16), np.full_like(b, rnd), np.full_like(b, 0x80000000 + site)]
        key = [seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32]
        for _ in range(10):
            p, q = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)      # below 2^64: exact
            x = [(q >> u(32)) ^ x[1] ^ u(key[0]), q & lo, (p >> u(32)) ^ x[3] ^ u(key[1]), p & lo]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        o = out[8 * b0:8 * (b0 + len(b))]
        for j in range(4):
            o[2 * j::8] = x[j] & u(0xFFFF)
            o[2 * j + 1::8] = x[j] >> u(16)
    return out[:n]


def exact(case, seed):
    s = _prepare(case, seed)
    if case["op"] == "dropout":
        d = torch.from_numpy(_dithers(s.seed, s.worker, s.round, s.site, s.x.numel()).astype(np.int32))
        t = int(math.floor(case["p"] * 65536 + 0.5))
        y = s.x.double()
        y *= (d.to(s.x.device).reshape(s.x.shape) >= t)
        y *= 65536.0 / (65536 - t)
        return y if s.residual is None else y.add_(s.residual)
    E, k = case["experts"], case["top_k"]
    N, count, total, per = 0, torch.zeros(E, dtype=torch.int64), torch.zeros(E, dtype=torch.float64), []
    for logits, mask in zip(s.logits, s.mask):
        l = logits.double()
        if mask is not None:
            l[~mask] = -math.inf
        routed = (l > -math.inf).sum(1) > 0
        lse = torch.logsumexp(l, 1)
        lse[~routed] = 0.0
        p = torch.exp(l - lse[:, None])
        left = l.clone()
        ids, gates = [], []
        for _ in range(k):                               # the largest left, at its first place
            at = (left == left.amax(1, keepdim=True)).to(torch.uint8).argmax(1)
            v = left.gather(1, at[:, None])[:, 0]
            none = v == -math.inf
            gates.append(torch.where(none, 0.0, p.gather(1, at[:, None])[:, 0]))
            left.scatter_(1, at[:, None], -math.inf)
            ids.append(torch.where(none, -1, at))
        ids, gates = torch.stack(ids, 1), torch.stack(gates, 1)
        N += int(routed.sum())
        total += p.sum(0).cpu()
        count += torch.bincount(ids[ids >= 0], minlength=E).cpu()
        per.append((p, ids, gates))
    coef = E * count.double() / k / max(N, 1) ** 2
    if case["dir"] == "bwd":
        coef = coef.float().double()                     # as the backward is given it
    res = {"ids": [], "gates": [], "dlogits": []}
    for (p, ids, ps), dgates in zip(per, s.dgates):
        dg = torch.where(ids >= 0, dgates.double(), 0.0)
        norm = ps.sum(1, keepdim=True) if case["renorm"] else torch.ones_like(ps[:, :1])
        g = ps / norm.masked_fill(norm == 0, 1.0)
        res["ids"].append(ids)
        res["gates"].append(g)
        if case["dir"] != "fwd":
            # through the gates to the chosen probabilities, then through the softmax
            up = (s.dloss.double() * coef.to(p.device)).repeat(p.shape[0], 1)
            dps = (dg - (g * dg).sum(1, keepdim=True)) / norm.masked_fill(norm == 0, 1.0) if case["renorm"] else dg
            up.scatter_add_(1, ids.clamp(min=0), torch.where(ids >= 0, dps, 0.0))
            res["dlogits"].append(p * (up - (p * up).sum(1, keepdim=True)))
    if case["dir"] == "bwd":
        return res["dlogits"]
    res.update(loss=(coef * total).sum().reshape(1), coef=coef, counts=count)
    if case["dir"] == "fwd":
        del res["dlogits"]
    return res
