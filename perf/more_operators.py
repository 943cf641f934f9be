"""Workloads of the experts that follow the router: products grouped by expert
over ragged rows, their weights' gradient, the gated activation between them,
the rows' order and the way back, and activations kept in 8 bits for the
backward pass.

Each case is one call (or a call and its inverse) as a mixture-of-experts
training step or a serving program makes it.  With ``own`` false ``run``
computes the operator from elementary torch operations in fp32; with ``own``
true it calls the library.  ``exact`` evaluates the definitions in fp64,
separately from the plain form.

Rows: slot t k + j is token t's j-th choice ``ids[t, j]`` of E experts (-1:
none).  The slots sorted by expert, stably, are the rows; those without an expert
come last and belong to none.  ``offsets[e]`` is expert e's first row, ``source[r]``
the slot of row r, ``row[t, j]`` the row of a slot, -1 without an expert.

Products: y[r] = x[r] w[e(r)], or x[source[r] // k] w[e(r)] gathered; dw[e] = the
sum of x[r]^T dy[r] over e's rows.  Rows without an expert stay as they were.

Activation: from u = (g, v), a = gate silu(g) v; or a = gate max(u, 0); the gate is
the slot's.  Way back: y[t] = residual[t] + sum_j rows[row[t, j]].

8 bits: every 32 elements of a row share a power of two, 2^s the smallest (s >=
-110) with max|x| <= 127 2^s; |q| = floor((floor(|x| 2^(16 - s)) + d) / 2^16) with
the element's 16-bit dither d (32768: to the nearest), x kept as sign(x) |q| 2^s.
Dither of element i (row-major): word (i & 7) >> 1, low half for even i, of
Philox4x32-10 with key = seed and counter = (low 32 bits of i >> 3, the next 15
bits | 2^15 | worker << 16, round, 2^31 + site).
"""
import math

import numpy as np
import torch

own = False


def _rows(name, tokens, top_k, experts, mask=0.0, **more):
    return {"name": name, "tokens": tokens, "top_k": top_k, "experts": experts, "mask": mask, **more}


def _product(name, tokens, top_k, experts, inner, outer, dtype="bf16", gather=False, mask=0.0, turned=False):
    return _rows(name, tokens, top_k, experts, mask, op="product", inner=inner, outer=outer, dtype=dtype,
                 gather=gather, turned=turned)


def _weights(name, tokens, top_k, experts, inner, outer, dtype="bf16", gather="", mask=0.0, kept=False, out="bf16"):
    return _rows(name, tokens, top_k, experts, mask, op="weights", inner=inner, outer=outer, dtype=dtype, gather=gather,
                 kept=kept, out=out)


def _act(name, tokens, top_k, experts, width, act="swiglu", dtype="bf16", mask=0.0, kept=True):
    return _rows(name, tokens, top_k, experts, mask, op="act", width=width, act=act, dtype=dtype, kept=kept)


def _order(name, tokens, top_k, experts, width, dtype="bf16", mask=0.0, residual=False):
    return _rows(name, tokens, top_k, experts, mask, op="order", width=width, dtype=dtype, residual=residual)


def _keep(name, rows, cols, dtype="bf16", dither=True):
    return {"name": name, "op": "keep", "rows": rows, "cols": cols, "dtype": dtype, "dither": dither}


def listed():
    return [
        # one token of a serving program: eight experts' weights are read, latency counts
        _product("product_one_token", 1, 8, 64, 2048, 2816, gather=True),
        # one worker's batch into the gate and up projections, tokens gathered as they are read
        _product("product_forward", 8192, 8, 64, 2048, 2816, gather=True),
        # the gradient by the input of the same layer, padding tokens left out: weights read transposed
        _product("product_backward", 8191, 8, 64, 2816, 2048, mask=0.1, turned=True),
        # fp32 at odd widths, few experts
        _product("product_fp32_odd", 1001, 2, 16, 257, 515, dtype="f32", mask=0.05),
        # the weights' gradient of the up projection, from the tokens themselves
        _weights("weights_forward", 8192, 8, 64, 2048, 2816, gather="x"),
        # the same from activations kept in 8 bits, into fp32 as a gradient round takes it; ragged
        _weights("weights_kept", 4099, 4, 60, 1000, 1416, gather="x", mask=0.2, kept=True, out="f32"),
        # a serving batch's activation, forward and backward of a short step
        _act("act_small", 16, 2, 16, 256),
        # a training batch: forward with its input kept in 8 bits, and the backward from that
        _act("act_kept", 8192, 2, 64, 2048, mask=0.1),
        # a short batch's order and way back
        _order("order_small", 16, 2, 16, 256, residual=True),
        # a long batch over many experts
        _order("order_large", 32768, 8, 256, 2048, mask=0.1, residual=True),
        # a tiny batch's hidden state kept in 8 bits and restored
        _keep("keep_small", 16, 256),
        # a worker's tokens by a hidden size
        _keep("keep_block", 8192, 4096),
    ]


def _log(rng, lo, hi):
    """An integer in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    w = _log(rng, lo, hi)
    return w if rng.random() < 0.3 else max(8, w // 8 * 8)


def draw(rng):
    op = rng.choice(["product", "product", "weights", "weights", "act", "order", "keep"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "keep":
        n = _log(rng, 16, 1 << (25 if dtype == "bf16" else 24))
        cols = max(1, min(n, _width(rng, 8, 8192)))
        c = _keep("", max(1, n // cols), cols, dtype, rng.random() < 0.7)
    else:
        experts = _log(rng, 2, 256)
        k = rng.randint(1, min(8, experts))
        mask = rng.choice([0.0, 0.0, 0.2])
        if op == "order":
            width = _width(rng, 8, 4096)
            most = (1 << (28 if dtype == "bf16" else 27)) // (k * width)
            c = _order("", _log(rng, 1, max(1, min(32768, most))), k, experts, width, dtype, mask, rng.random() < 0.5)
        elif op == "act":
            width = _width(rng, 8, 4096)
            most = (1 << (24 if dtype == "bf16" else 23)) // (k * width)
            c = _act("", _log(rng, 1, max(1, min(8192, most))), k, experts, width, rng.choice(["swiglu", "swiglu", "relu"]),
                     dtype, mask, rng.random() < 0.6)
        else:
            inner, outer = _width(rng, 8, 4096), _width(rng, 8, 4096)
            # weights of 1.5 GB at most, and no more work than the largest listed product
            experts = max(2, min(experts, (3 << 28) // (inner * outer * (1 if dtype == "bf16" else 2))))
            k = min(k, experts)
            most = min(65536, (1 << 38) // (inner * outer)) // (1 if dtype == "bf16" else 16)
            tokens = _log(rng, 1, max(1, most // k))
            if op == "product":
                c = _product("", tokens, k, experts, inner, outer, dtype, rng.random() < 0.5, mask, rng.random() < 0.5)
            else:
                c = _weights("", tokens, k, experts, inner, outer, dtype, rng.choice(["", "x", "dout"]), mask,
                             rng.random() < 0.5, rng.choice([dtype, "f32"]))
    del c["name"]
    return c


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


class _State:
    pass


def prepare(case, seed):
    s = _State()
    s.case = c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    s.key = dict(seed=(seed * 0x9E3779B97F4A7C15 + 11) % 2 ** 64, rnd=seed % 1000, worker=seed % 5, site=2)

    def normal(*shape, scale=1.0, dtype=c["dtype"]):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(_dtype(dtype))

    if c["op"] == "keep":
        # activations with a few strong channels
        s.x = normal(c["rows"], c["cols"]) * (1 + 20 * (torch.rand(c["cols"], generator=g, device="cuda") < 0.01)).to(
            _dtype(c["dtype"]))
        return s
    T, k, E = c["tokens"], c["top_k"], c["experts"]
    # a router's choices: some experts are preferred, padding tokens have none
    logits = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    s.ids = logits.topk(k, dim=1).indices.int()
    if c["mask"]:
        s.ids[torch.rand(T, generator=g, device="cuda") < c["mask"]] = -1
    R = T * k
    if c["op"] == "order":
        s.y = normal(R, c["width"])
        s.residual = normal(T, c["width"]) if c["residual"] else None
        return s
    s.offsets, s.source, s.row = _order_plain(s.ids, E)      # the step's, made once for all its products
    if c["op"] == "act":
        F = c["width"]
        s.u = normal(R, F if c["act"] == "relu" else 2 * F)
        s.da = normal(R, F, scale=0.01)
        s.gates = torch.rand(T, k, generator=g, device="cuda")
        # rows without an expert are left as they were
        s.a, s.again = (torch.zeros(R, F, dtype=s.u.dtype, device="cuda") for _ in range(2))
        s.du = torch.zeros_like(s.u)
        return s
    K, N = c["inner"], c["outer"]
    if c["op"] == "product":
        s.x = normal(T if c["gather"] else R, K)
        w = normal(E, N, K, scale=K ** -0.5) if c["turned"] else normal(E, K, N, scale=K ** -0.5)
        s.w = w.transpose(1, 2) if c["turned"] else w
        s.out = torch.zeros(R, N, dtype=s.x.dtype, device="cuda")
        return s
    s.x = normal(T if c["gather"] == "x" else R, K)
    s.dout = normal(T if c["gather"] == "dout" else R, N, scale=0.01)
    if c["kept"]:                                            # what the forward pass left
        s.codes, s.exponents = _keep_plain(s.x, s.key)
        s.x = None
    return s


# ---- plain forms ------------------------------------------------------------

def _order_plain(ids, experts):
    flat = ids.reshape(-1).long()
    flat = torch.where(flat < 0, experts, flat)
    source = torch.sort(flat, stable=True).indices
    offsets = torch.bincount(flat, minlength=experts + 1).cumsum(0)
    row = torch.empty_like(source)
    row[source] = torch.arange(len(source), device=ids.device)
    row = torch.where(flat < experts, row, -1).reshape(ids.shape)
    first = torch.zeros(1, dtype=torch.int64, device=ids.device)
    return torch.cat((first, offsets[:experts])).int(), source.int(), row.int()


def _sum_plain(s, row):
    at = row.long()
    y = torch.where((at >= 0)[:, :, None], s.y.float()[at.clamp(min=0)], 0.0).sum(1)
    if s.residual is not None:
        y = s.residual.float() + y
    return y.to(s.y.dtype)


def _dithers_plain(key, n, device):
    """The 16-bit dithers of elements 0 .. n - 1: Philox4x32-10 on int64 tensors of 32-bit values."""
    m32 = 0xFFFFFFFF
    block = torch.arange((n + 7) // 8, device=device)
    c0, c1 = block & m32, block >> 32 | 1 << 15 | key["worker"] << 16
    c2, c3 = torch.full_like(block, key["rnd"]), torch.full_like(block, 0x80000000 | key["site"])
    k0, k1 = key["seed"] & m32, key["seed"] >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32 & m32) ^ c1 ^ k0, b & m32, (a >> 32 & m32) ^ c3 ^ k1, a & m32
        k0, k1 = k0 + 0x9E3779B9 & m32, k1 + 0xBB67AE85 & m32
    w = torch.stack((c0, c1, c2, c3), 1)
    return torch.stack((w & 0xFFFF, w >> 16), 2).reshape(-1)[:n]


def _power(e):
    """2^e in fp32, for -126 <= e <= 127."""
    return (e.int() + 127 << 23).view(torch.float32)


def _keep_plain(x, key):
    """(codes int8, s + 127 per 32 elements of a row) of finite values; without a key, to the nearest."""
    rows, cols = x.shape
    blocks = (cols + 31) // 32
    m = torch.nn.functional.pad(x.float().abs(), (0, 32 * blocks - cols)).view(rows, blocks, 32).amax(2)
    f, e = torch.frexp(m)                                    # m = f 2^e, f in [1/2, 1)
    e = (e - 7 + (f > 127 / 128).int()).clamp(min=-110)
    e = torch.where(m == 0, -110, e)
    d = 32768 if key is None else _dithers_plain(key, x.numel(), x.device).view(rows, cols)
    t = torch.floor(x.float().abs() * _power(16 - e).repeat_interleave(32, 1)[:, :cols]).long()
    q = (t + d) >> 16
    return torch.where(x < 0, -q, q).to(torch.int8), (e + 127).to(torch.uint8)


def _restore_plain(codes, exponents):
    return codes.float() * _power(exponents.int() - 127).repeat_interleave(32, 1)[:, :codes.shape[1]]


def _act_plain(u, gate, act):
    """(a, what backward needs) in fp32."""
    if act == "relu":
        h = u.clamp(min=0)
        return gate * h, h
    g, v = u.chunk(2, 1)
    h = g * torch.sigmoid(g) * v
    return gate * h, h


def _act_backward_plain(u, da, gate, act):
    """(du, gradient of the gates, a) in fp32."""
    a, h = _act_plain(u, gate, act)
    dgate = (da * h).sum(1)
    if act == "relu":
        return gate * da * (u > 0), dgate, a
    g, v = u.chunk(2, 1)
    sg = torch.sigmoid(g)
    d = gate * da
    return torch.cat((d * v * sg * (1 + g * (1 - sg)), d * g * sg), 1), dgate, a


# ---- one pass ---------------------------------------------------------------

def run(s):
    c = s.case
    if own:
        return _run_own(s)
    if c["op"] == "keep":
        return _restore_plain(*_keep_plain(s.x, s.key if c["dither"] else None)).to(s.x.dtype)
    if c["op"] == "order":
        offsets, source, row = _order_plain(s.ids, c["experts"])
        return {"offsets": offsets, "source": source, "row": row, "y": _sum_plain(s, row)}
    E, k = c["experts"], c["top_k"]
    at = s.offsets.tolist()
    n = at[E]
    if c["op"] == "act":
        gate = s.gates.reshape(-1)[s.source[:n].long()][:, None]
        u = s.u[:n].float()
        s.a[:n] = _act_plain(u, gate, c["act"])[0].to(s.u.dtype)
        if c["kept"]:
            u = _restore_plain(*_keep_plain(s.u[:n], s.key))
        du, dgate, a = _act_backward_plain(u, s.da[:n].float(), gate, c["act"])
        s.du[:n], s.again[:n] = du.to(s.u.dtype), a.to(s.u.dtype)
        dgates = torch.zeros(c["tokens"] * k, device=u.device)
        dgates[s.source[:n].long()] = dgate
        return {"a": s.a, "du": s.du, "dgates": dgates.view(-1, k), "again": s.again}
    token = s.source.long() // k
    if c["op"] == "product":
        for e in range(E):
            if at[e] < at[e + 1]:
                r = slice(at[e], at[e + 1])
                x = s.x[token[r]] if c["gather"] else s.x[r]
                s.out[r] = (x.float() @ s.w[e].float()).to(s.out.dtype)
        return s.out
    x = _restore_plain(s.codes, s.exponents) if c["kept"] else s.x
    dw = torch.zeros(E, x.shape[1], s.dout.shape[1], dtype=_dtype(c["out"]), device=x.device)
    for e in range(E):
        if at[e] < at[e + 1]:
            r = slice(at[e], at[e + 1])
            xe = x[token[r]] if c["gather"] == "x" else x[r]
            de = s.dout[token[r]] if c["gather"] == "dout" else s.dout[r]
            dw[e] = (xe.float().t() @ de.float()).to(dw.dtype)
    return dw


def _run_own(s):
    from compressed_hop_gradient_amd import dq
    c = s.case
    if c["op"] == "keep":
        return dq.restore8(dq.keep8(s.x, dither=c["dither"], **s.key))
    if c["op"] == "order":
        rows = dq.expert_rows(s.ids, c["experts"])
        return {"offsets": rows.offsets, "source": rows.source, "row": rows.row,
                "y": dq.expert_sum(s.y, rows, residual=s.residual)}
    rows = dq.ExpertRows(s.offsets, s.source, s.row)
    if c["op"] == "act":
        if c["kept"]:
            a, u = dq.expert_act(s.u, s.gates, rows, c["act"], out=s.a, keep=True, **s.key)
        else:
            a, u = dq.expert_act(s.u, s.gates, rows, c["act"], out=s.a), s.u
        du, dgates, again = dq.expert_act_backward(u, s.da, s.gates, rows, c["act"], du=s.du, a=s.again)
        return {"a": a, "du": du, "dgates": dgates, "again": again}
    if c["op"] == "product":
        return dq.expert_matmul(s.x, s.w, rows, gather=c["gather"], out=s.out)
    x = dq.Kept8(s.codes, s.exponents, _dtype(c["dtype"])) if c["kept"] else s.x
    return dq.expert_matmul_grad(x, s.dout, rows, gather=c["gather"] or None, dtype=_dtype(c["out"]))


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "keep":
        n = c["rows"] * c["cols"]
        # in, codes out; codes in, out; per 8 elements 10 rounds of two products and four xors; five more an element
        return {"bytes": n * (2 * es + 2) + 2 * c["rows"] * ((c["cols"] + 31) // 32),
                "flops": n * ((60 / 8 if c["dither"] else 0) + 5)}
    T, k, E = c["tokens"], c["top_k"], c["experts"]
    R = T * k
    n = int(R * (1 - c["mask"]))                             # rows of experts
    lists = 4 * (E + 1) + 4 * R
    if c["op"] == "order":
        return {"bytes": lists + 8 * R + es * c["width"] * (n + T * (2 if c["residual"] else 1)),
                "flops": n * c["width"]}
    if c["op"] == "act":
        F, U = c["width"], c["width"] * (1 if c["act"] == "relu" else 2)
        kept = 2 * (U + U // 32) if c["kept"] else es * U
        return {"bytes": n * (es * (2 * U + 3 * F) + kept + 8), "flops": n * (25 * F + (14 * U if c["kept"] else 0))}
    K, N = c["inner"], c["outer"]
    met = min(E, n) if n else 0                              # experts that have rows, at most
    ys = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "product":
        rows_in = min(T, n) if c["gather"] else n
        return {"bytes": lists + es * rows_in * K + es * met * K * N + ys * n * N, "flops": 2 * n * K * N}
    xs = 33 / 32 if c["kept"] else es
    rows_x, rows_d = (min(T, n) if c["gather"] == g else n for g in ("x", "dout"))
    out = 2 if c["out"] == "bf16" else 4
    return {"bytes": lists + xs * rows_x * K + es * rows_d * N + out * E * K * N, "flops": 2 * n * K * N}


# ---- the definitions in 64 bits ----------------------------------------------

def _philox16(key, first, n):
    """The dithers of elements first .. first + n - 1 (first a multiple of 8), from numpy's unsigned integers."""
    u = np.uint64
    lo = u(0xFFFFFFFF)
    b = np.arange(first // 8, (first + n + 7) // 8, dtype=u)
    x = [b & lo, (b >> u(32)) + u(32768 + 65536 * key["worker"]), np.full_like(b, key["rnd"]),
         np.full_like(b, 2 ** 31 + key["site"])]
    k = [key["seed"] % 2 ** 32, key["seed"] // 2 ** 32]
    for _ in range(10):
        p, q = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)          # below 2^64: exact
        x = [(q >> u(32)) ^ x[1] ^ u(k[0]), q & lo, (p >> u(32)) ^ x[3] ^ u(k[1]), p & lo]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    out = np.empty((len(b), 8), np.int32)
    for j in range(4):
        out[:, 2 * j], out[:, 2 * j + 1] = x[j] & u(0xFFFF), x[j] >> u(16)
    return out.reshape(-1)[:n]


def _two_to(e):
    """2^e in fp64."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _kept64(x, key):
    """What x is kept as, in fp64."""
    x = x.double()
    rows, cols = x.shape
    out = torch.empty_like(x)
    if key is None:
        d = torch.full_like(x, 32768.0)
    else:
        parts = [_philox16(key, i, min(1 << 21, x.numel() - i)) for i in range(0, x.numel(), 1 << 21)]
        d = torch.from_numpy(np.concatenate(parts) if parts else np.empty(0, np.int32)).to(x.device).double().view(rows, cols)
    for c0 in range(0, cols, 32):
        b = x[:, c0:c0 + 32]
        m = b.abs().amax(1, keepdim=True)
        step = _two_to(torch.log2(m.clamp(min=2.0 ** -120) / 127).ceil().clamp(min=-110.0))
        # the logarithm is rounded: one step further, or back, as the definition says
        step = torch.where(m > 127 * step, 2 * step, step)
        step = torch.where((m <= 127 * step / 2) & (step > 2.0 ** -110), step / 2, step)
        q = ((b.abs() / step * 65536).floor() + d[:, c0:c0 + 32]).div(65536).floor()
        out[:, c0:c0 + 32] = b.sign() * q * step
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "keep":
        return _kept64(s.x, s.key if c["dither"] else None)
    T, k, E = c["tokens"], c["top_k"], c["experts"]
    slots = s.ids.reshape(-1)
    # every expert's slots in order, then those of none
    lists = [(slots == e).nonzero()[:, 0] for e in range(E)]
    source = torch.cat([*lists, (slots < 0).nonzero()[:, 0]])
    sizes = [len(l) for l in lists]
    starts = [sum(sizes[:e]) for e in range(E + 1)]
    n = starts[E]
    if c["op"] == "order":
        row = torch.full((T * k,), -1, dtype=torch.int64, device=slots.device)
        row.scatter_(0, source[:n], torch.arange(n, device=slots.device))
        row = row.view(T, k)
        y = torch.zeros(T, c["width"], dtype=torch.float64, device=slots.device)
        for j in range(k):
            has = row[:, j] >= 0
            y[has] += s.y[row[has, j]].double()
        if s.residual is not None:
            y += s.residual.double()
        return {"offsets": torch.tensor(starts, device=slots.device), "source": source, "row": row, "y": y}
    if c["op"] == "act":
        gate = s.gates.double().view(-1, 1)[source[:n]]
        u, da = s.u[:n].double(), s.da[:n].double()
        kept = _kept64(s.u[:n], s.key) if c["kept"] else u
        res = {name: torch.zeros(T * k, t.shape[1], dtype=torch.float64, device=slots.device)
               for name, t in (("a", s.da), ("du", s.u), ("again", s.da))}
        dgates = torch.zeros(T * k, dtype=torch.float64, device=slots.device)
        F = c["width"]
        if c["act"] == "relu":
            res["a"][:n] = u.relu() * gate
            on = (kept > 0).double()
            h = kept * on
            res["du"][:n] = on * da * gate
        else:
            res["a"][:n] = u[:, :F] / (1 + torch.exp(-u[:, :F])) * u[:, F:] * gate
            g, v = kept[:, :F], kept[:, F:]
            sg = 1 / (1 + torch.exp(-g))
            h = g * sg * v
            res["du"][:n, :F] = da * gate * v * (sg + g * sg * (1 - sg))
            res["du"][:n, F:] = da * gate * g * sg
        res["again"][:n] = h * gate
        dgates.scatter_(0, source[:n], (h * da).sum(1))
        return {"a": res["a"], "du": res["du"], "dgates": dgates.view(T, k), "again": res["again"]}
    if c["op"] == "product":
        out = torch.zeros(T * k, c["outer"], dtype=torch.float64, device=slots.device)
        for e, l in enumerate(lists):
            if sizes[e]:
                x = s.x[torch.div(l, k, rounding_mode="floor")] if c["gather"] else s.x[starts[e]:starts[e + 1]]
                out[starts[e]:starts[e + 1]] = x.double().mm(s.w[e].double())
        return out
    x = _two_to(s.exponents.long() - 127).repeat_interleave(32, 1)[:, :c["inner"]] * s.codes if c["kept"] else s.x
    dw = torch.zeros(E, c["inner"], c["outer"], dtype=torch.float64, device=slots.device)
    for e, l in enumerate(lists):
        if sizes[e]:
            t = torch.div(l, k, rounding_mode="floor")
            mine = slice(starts[e], starts[e + 1])
            xe = (x[t] if c["gather"] == "x" else x[mine]).double()
            dw[e] = xe.t().mm((s.dout[t] if c["gather"] == "dout" else s.dout[mine]).double())
    return dw
