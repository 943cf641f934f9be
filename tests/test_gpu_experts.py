"""The experts' operators on the GPU against their plain fp64 forms
(experts_ref.py): lists and codes exactly, the rest within the roundings that
an fp32 evaluation makes."""
import numpy as np
import pytest
import torch

import experts_ref as ref
from compressed_hop_gradient_amd import dq, train

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]
U = ref.U
SENTINEL = 7.0


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def randn(shape, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


def choices(T, k, E, seed=0, none=0.2, skew=True):
    """ids of a router: some experts preferred, some tokens and choices without."""
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) + (torch.linspace(0, 2, E) if skew else 0)
    if E > 3:
        logits[:, E // 2] = -100                     # an expert that nobody takes
    ids = logits.topk(k, dim=1).indices.int()
    if none:
        ids[torch.rand(T, generator=g) < none] = -1
        ids[torch.rand(T, k, generator=g) < 0.05] = -1
    return ids


def wide(t, extra=3, at=1):
    """The same values as columns of a wider tensor."""
    w = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    w[:, at:at + t.shape[1]] = t
    return w[:, at:at + t.shape[1]]


def close(got, want, bound, dtype):
    """|got - want| <= bound and one rounding to dtype."""
    got, want = f64(got), np.asarray(want)
    err = np.abs(got - want)
    tol = bound * (1 + 2 * half_step(dtype)) + half_step(dtype) * np.abs(want) + 1e-37
    bad = ~(err <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(err / tol):.3g} of its bound"


def lists(rows):
    return rows.offsets.cpu().numpy(), rows.source.cpu().numpy(), rows.row.cpu().numpy()


# ---- order --------------------------------------------------------------------

@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (5, 2, 3), (64, 1, 2), (65, 2, 16), (511, 3, 60), (1024, 8, 64),
                                   (1025, 8, 64), (3000, 8, 1024), (9000, 1, 300), (700, 16, 512), (20000, 2, 7)])
def test_rows(T, k, E):
    ids = choices(T, min(k, E), E, seed=T)
    got = lists(dq.expert_rows(ids.cuda(), E))
    want = ref.Rows(ids.numpy(), E)
    for g, w in zip(got, (want.offsets, want.source, want.row)):
        assert np.array_equal(g, w)


def test_rows_odd_ids():
    """Ids out of range are no choice; an expert twice in a token's choices is two rows;
    nobody at all; no tokens."""
    ids = torch.tensor([[3, 3], [-7, 4], [2 ** 31 - 1, 0], [-2 ** 31, 2]], dtype=torch.int32)
    want = ref.Rows(ids.numpy(), 4)
    for g, w in zip(lists(dq.expert_rows(ids.cuda(), 4)), (want.offsets, want.source, want.row)):
        assert np.array_equal(g, w)
    none = dq.expert_rows(torch.full((33, 2), -1, dtype=torch.int32, device="cuda"), 5)
    assert (none.offsets == 0).all() and (none.row == -1).all()
    assert torch.equal(none.source.cpu(), torch.arange(66, dtype=torch.int32))
    empty = dq.expert_rows(torch.zeros((0, 2), dtype=torch.int32, device="cuda"), 5)
    assert (empty.offsets == 0).all() and empty.source.numel() == 0


def test_rows_of_very_many_slots():
    g = torch.Generator(device="cuda").manual_seed(0)
    for E in (4, 256, 1024):
        ids = torch.randint(-1, E, (150001, 7), generator=g, device="cuda", dtype=torch.int32)
        rows = dq.expert_rows(ids, E)
        key = torch.where(ids < 0, E, ids).reshape(-1).long()
        source = torch.sort(key, stable=True).indices
        assert torch.equal(rows.source.long(), source)
        assert torch.equal(rows.offsets.long()[1:], torch.bincount(key, minlength=E + 1).cumsum(0)[:E])
        row = torch.empty_like(source)
        row[source] = torch.arange(len(source), device="cuda")
        assert torch.equal(rows.row.long().view(-1), torch.where(key < E, row, -1))


# ---- products -------------------------------------------------------------------

SHAPES = [(1, 1, 1, 1, 1), (1, 2, 4, 64, 64), (1, 8, 16, 200, 72), (7, 2, 3, 33, 65), (40, 2, 4, 128, 128),
          (300, 2, 4, 72, 136), (300, 3, 5, 257, 131), (513, 1, 2, 64, 300), (129, 1, 1, 100, 128), (600, 4, 6, 520, 264)]


def product_bound(inner, mag):
    # every addition of the sum off by at most a step, 2 U of its magnitude
    return (inner + 2) * 2 * U * mag


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,K,N", SHAPES)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("turned", [False, True])
def test_matmul(T, k, E, K, N, gather, turned, dtype):
    ids = choices(T, k, E, seed=K, none=0.2 if T > 1 else 0)
    want = ref.Rows(ids.numpy(), E)
    rows = dq.expert_rows(ids.cuda(), E)
    x = randn((T if gather else T * k, K), dtype, 1)
    if not gather:
        x[want.n:] = float("nan")                    # nobody's rows
    w = randn((E, N, K) if turned else (E, K, N), dtype, 2)
    w = w.transpose(1, 2) if turned else w
    out = torch.full((T * k, N), SENTINEL, dtype=dtype, device="cuda")
    assert dq.expert_matmul(x, w, rows, gather=gather, out=out) is out
    y, mag = ref.matmul(f64(x), f64(w), want, gather)
    close(out[:want.n], y, product_bound(K, mag), dtype)
    assert (out[want.n:] == SENTINEL).all()
    # rows off their alignment, at other strides
    again = wide(torch.full((T * k, N), SENTINEL, dtype=dtype, device="cuda"))
    dq.expert_matmul(wide(x), w, rows, gather=gather, out=again)
    close(again[:want.n], y, product_bound(K, mag), dtype)
    assert (again[want.n:] == SENTINEL).all()
    base = again._base
    assert torch.isnan(base[:, 0]).all() and torch.isnan(base[:, -2:]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,K,N", SHAPES)
@pytest.mark.parametrize("gather", [None, "x", "dout"])
def test_matmul_grad(T, k, E, K, N, gather, dtype):
    ids = choices(T, k, E, seed=K + 1, none=0.2 if T > 1 else 0)
    want = ref.Rows(ids.numpy(), E)
    rows = dq.expert_rows(ids.cuda(), E)
    x, dy = randn((T if gather == "x" else T * k, K), dtype, 1), randn((T if gather == "dout" else T * k, N), dtype, 2)
    if gather != "x":
        x[want.n:] = float("nan")
    if gather != "dout":
        dy[want.n:] = float("nan")
    dw, mag = ref.matmul_grad(f64(x), f64(dy), want, gather)
    most = int(np.diff(want.offsets).max())
    for out in {dtype, torch.float32}:
        got = dq.expert_matmul_grad(x, dy, rows, gather=gather, dtype=out)
        assert got.dtype == out and got.shape == (E, K, N)
        close(got, dw, product_bound(most, mag), out)
    close(dq.expert_matmul_grad(wide(x), wide(dy), rows, gather=gather), dw, product_bound(most, mag), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,K,N", SHAPES)
@pytest.mark.parametrize("gather", [None, "x", "dout"])
def test_matmul_grad_from_kept(T, k, E, K, N, gather, dtype):
    """The same bits as from the restored tensor where both are read alike, and within
    the roundings always."""
    ids = choices(T, k, E, seed=K + 2, none=0.2 if T > 1 else 0)
    want = ref.Rows(ids.numpy(), E)
    rows = dq.expert_rows(ids.cuda(), E)
    x, dy = randn((T if gather == "x" else T * k, K), dtype, 1), randn((T if gather == "dout" else T * k, N), dtype, 2)
    if gather != "x":
        x[want.n:] = float("nan")
    kept = dq.keep8(x, site=4)
    dw, mag = ref.matmul_grad(f64(dq.restore8(kept)), f64(dy), want, gather)
    most = int(np.diff(want.offsets).max())
    close(dq.expert_matmul_grad(kept, dy, rows, gather=gather), dw, product_bound(most, mag), dtype)
    close(dq.expert_matmul_grad(kept, wide(dy), rows, gather=gather, dtype=torch.float32), dw,
          product_bound(most, mag), torch.float32)


# ---- way back -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,width", [(1, 1, 1), (1, 8, 2048), (5, 3, 9), (37, 2, 64), (33, 16, 1336), (300, 8, 72),
                                       (3, 5, 5000)])
@pytest.mark.parametrize("residual", [False, True])
def test_sum(T, k, width, residual, dtype):
    E = max(k, 8)
    ids = choices(T, k, E, seed=width)
    want = ref.Rows(ids.numpy(), E)
    rows = dq.expert_rows(ids.cuda(), E)
    y = randn((T * k, width), dtype, 1)
    y[want.n:] = float("nan")
    res = randn((T, width), dtype, 2) if residual else None
    out, mag = ref.back(f64(y), want, None if res is None else f64(res))
    bound = (k + 1) * U * mag
    close(dq.expert_sum(y, rows, residual=res), out, bound, dtype)
    close(dq.expert_sum(wide(y), rows, residual=res, out=wide(torch.zeros_like(y[:T]) if T <= y.shape[0] else y)), out,
          bound, dtype)
    if residual:
        same = res.clone()
        assert dq.expert_sum(y, rows, residual=same, out=same) is same
        close(same, out, bound, dtype)


# ---- 8 bits ---------------------------------------------------------------------

KEY = dict(seed=0x123456789ABCDEF1, rnd=77, worker=5, site=3)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 31), (2, 32), (5, 33), (4, 64), (3, 40), (7, 104), (2, 1337),
                                       (64, 256), (9, 7)])
@pytest.mark.parametrize("dither", [False, True])
def test_keep(rows, cols, dither, dtype):
    x = randn((rows, cols), dtype, cols) * torch.logspace(-3, 3, rows, device="cuda")[:, None].to(dtype)
    d = ref.dithers(rows * cols, **KEY) if dither else 32768
    codes, exps, values = ref.keep(f64(x), d)
    for view in (x, wide(x), wide(x, 8, 0)):
        kept = dq.keep8(view, dither=dither, **KEY)
        assert np.array_equal(kept.codes.cpu().numpy(), codes) and np.array_equal(kept.exponents.cpu().numpy(), exps)
        got = dq.restore8(kept)
        assert got.dtype == dtype and np.array_equal(f64(got), values)
    out = wide(torch.zeros_like(x))
    assert np.array_equal(f64(dq.restore8(kept, out=out)), values)


@pytest.mark.parametrize("dtype", DTYPES)
def test_keep_edges(dtype):
    """Blocks at the ends of a scale's range, zeros, subnormals, the largest finite
    values, and blocks that are not finite."""
    big = torch.finfo(dtype).max
    rows = [[127.0, 1.0], [127.5, -127.0], [128.0, -0.5], [0.0, -0.0], [1e-38, 1e-45], [big, -big], [-1.0, big / 2],
            [2.0 ** -103, -2.0 ** -109], [2.0 ** -110, 2.0 ** -120], [float("inf"), 1.0], [float("nan"), 1.0],
            [1.0, -float("inf")]]
    x = torch.zeros(len(rows), 40, dtype=dtype)
    x[:, :2] = torch.tensor(rows, dtype=torch.float64).to(dtype)
    x[:, 32:] = torch.linspace(-1, 1, 8).to(dtype)
    for dither in (False, True):
        d = ref.dithers(x.numel(), **KEY) if dither else 32768
        codes, exps, values = ref.keep(f64(x), d)
        kept = dq.keep8(x.cuda(), dither=dither, **KEY)
        assert np.array_equal(kept.codes.cpu().numpy(), codes) and np.array_equal(kept.exponents.cpu().numpy(), exps)
        assert np.array_equal(f64(dq.restore8(kept)), values, equal_nan=True)


def test_keep_is_unbiased():
    x = randn((1, 64), torch.float32, 3)
    n = 4096
    mean = sum(dq.restore8(dq.keep8(x, rnd=i)).double() for i in range(n)) / n
    step = torch.exp2(dq.keep8(x).exponents.double() - 127).repeat_interleave(32, 1)
    # a rounding up with probability p has variance p (1 - p) <= 1/4 of a step; truncation below 2^-16
    assert ((mean - x.double()).abs() <= (6 * 0.5 / n ** 0.5 + 2 ** -16) * step).all()


@pytest.mark.parametrize("shape", [(0,), (3, 0), (0, 5), (2, 3, 40), (70,)])
def test_keep_shapes(shape):
    x = randn(shape, torch.bfloat16)
    kept = dq.keep8(x, dither=False)
    assert kept.shape == x.shape and kept.exponents.shape == x.shape[:-1] + ((shape[-1] + 31) // 32,)
    got = dq.restore8(kept)
    assert got.shape == x.shape
    if x.numel():
        assert np.array_equal(f64(got).reshape(-1, shape[-1]), ref.keep(f64(x).reshape(-1, shape[-1]), 32768)[2])


# ---- activation -----------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,width", [(1, 1, 1, 1), (1, 8, 16, 256), (5, 2, 3, 9), (40, 2, 4, 32), (33, 3, 5, 72),
                                         (65, 2, 8, 1000), (20, 4, 8, 1337)])
@pytest.mark.parametrize("kind", ["swiglu", "relu"])
def test_act(T, k, E, width, kind, dtype):
    ids = choices(T, k, E, seed=width, none=0.2 if T > 1 else 0)
    want = ref.Rows(ids.numpy(), E)
    rows = dq.expert_rows(ids.cuda(), E)
    n, R, columns = want.n, T * k, width * (2 if kind == "swiglu" else 1)
    u = randn((R, columns), dtype, 1, scale=3.0)
    u[n:] = float("nan")
    da = randn((R, width), dtype, 2)
    da[n:] = float("nan")
    gates = torch.rand(T, k, generator=torch.Generator().manual_seed(3)).cuda()
    gate = f64(gates).reshape(-1)[want.source[:n]]
    (_, _, a), (_, _, e_a) = ref.act_backward(f64(u[:n]), f64(da[:n]), gate, kind)
    for view in (u, wide(u)):
        out = torch.full((R, width), SENTINEL, dtype=dtype, device="cuda")
        assert dq.expert_act(view, gates, rows, kind, out=out) is out
        close(out[:n], a, e_a, dtype)
        assert (out[n:] == SENTINEL).all()
        same, kept = dq.expert_act(view, gates, rows, kind, keep=True, **KEY)
        assert torch.equal(same[:n], out[:n])
        alone = dq.keep8(u, **KEY)
        assert torch.equal(kept.codes[:n], alone.codes[:n]) and torch.equal(kept.exponents[:n], alone.exponents[:n])
    for source, values in ((u, f64(u[:n])), (wide(u), f64(u[:n])), (kept, f64(dq.restore8(kept)[:n]))):
        (du, dgate, a), (e_du, e_gate, e_a) = ref.act_backward(values, f64(da[:n]), gate, kind)
        dgates = np.zeros(R)
        dgates[want.source[:n]] = dgate
        bound = np.zeros(R)
        bound[want.source[:n]] = e_gate
        for d in (da, wide(da)):
            got = [torch.full((R, c), SENTINEL, dtype=dtype, device="cuda") for c in (columns, width)]
            gdu, gdg, ga = dq.expert_act_backward(source, d, gates, rows, kind, du=got[0], a=got[1])
            close(gdu[:n], du, e_du, dtype)
            close(ga[:n], a, e_a, dtype)
            close(gdg, dgates.reshape(T, k), bound.reshape(T, k), torch.float32)
            assert (gdu[n:] == SENTINEL).all() and (ga[n:] == SENTINEL).all()
    assert dq.expert_act_backward(u, da, gates, rows, kind, again=False)[2] is None


@pytest.mark.parametrize("dtype", DTYPES)
def test_act_far_from_zero(dtype):
    """Gates' arguments where the sigmoid is 0 or 1 to the last bit, and not finite
    ones, which stay so."""
    g = torch.tensor([-1e30, -500.0, -100.0, -87.0, -30.0, 30.0, 89.0, 500.0, 1e30], dtype=torch.float64).to(dtype)
    n = len(g)
    u = torch.cat((g, torch.ones(n, dtype=dtype))).cuda()[None]
    rows = dq.expert_rows(torch.zeros((1, 1), dtype=torch.int32, device="cuda"), 1)
    gates = torch.ones(1, 1, device="cuda")
    a = dq.expert_act(u, gates, rows)
    g64 = f64(g)
    with np.errstate(over="ignore"):
        want = g64 / (1 + np.exp(-g64))
    # below -87 the sigmoid is held at that of -87, 1.7e-38
    close(a, want[None], (ref.SIGMOID + 4) * U * np.abs(want)[None] + 1.7e-38 * np.abs(g64)[None], dtype)
    du, dgates, _ = dq.expert_act_backward(u, torch.ones(1, n, dtype=dtype, device="cuda"), gates, rows)
    assert torch.isfinite(du).all() and torch.isfinite(dgates).all()
    for bad in (float("nan"), float("inf")):
        u[0, 0] = bad
        assert not torch.isfinite(dq.expert_act(u, gates, rows)[0, 0])
        assert torch.isfinite(dq.expert_act(u, gates, rows)[0, 1:]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_act_at_the_lowest_end(dtype):
    """Gates' arguments down to the type's lowest value, where silu is 0: as a mask
    leaves them."""
    lowest = torch.finfo(dtype).min
    g = torch.tensor([lowest, lowest / 2, -1e38, -1e36, -1e32, -88.0, -87.5, -86.0], dtype=torch.float64).to(dtype)
    n = len(g)
    u = torch.cat((g, torch.full((n,), 3.0, dtype=dtype))).cuda()[None]
    da = torch.full((1, n), 2.0, dtype=dtype, device="cuda")
    rows = dq.expert_rows(torch.zeros((1, 1), dtype=torch.int32, device="cuda"), 1)
    gates = torch.full((1, 1), 0.5, device="cuda")
    g64 = f64(g)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-g64))
    a = dq.expert_act(u, gates, rows)
    du, dgates, again = dq.expert_act_backward(u, da, gates, rows)
    # below -87 the sigmoid is 0 instead of e^g: off by at most 88 e^-87 < 2^-118 of the factors
    want = 0.5 * g64 * s * 3
    close(a, want[None], ((ref.SIGMOID + 4) * U * np.abs(want) + 1.5 * 2.0 ** -118)[None], dtype)
    assert torch.equal(again, a)
    slope = 3 * s * (1 + g64 * (1 - s))                  # gate da = 1
    back = np.concatenate((slope, g64 * s))
    bound = np.concatenate((3 * s * (2 * ref.SIGMOID + 8) * U * (1 + np.abs(g64)), (ref.SIGMOID + 4) * U * np.abs(g64 * s)))
    close(du, back[None], (bound + 3 * 2.0 ** -118)[None], dtype)
    close(dgates, np.array([[(2 * g64 * s * 3).sum()]]), n * 2.0 ** -115, torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [1, 8, 32])
def test_act_at_the_upper_end(width, dtype):
    """Gates' arguments up to the type's largest value, where the sigmoid is 1: a, both
    gradients, the gates' gradient and the activation again, from u and from codes."""
    most = torch.finfo(dtype).max
    g = torch.tensor([20.0, 88.0, 1e30, 1e38, 2.3e38, 2.36e38, 2.4e38, most / 2, most], dtype=torch.float64).to(dtype)
    n = len(g)
    u = torch.ones(n, 2 * width, dtype=dtype)
    u[:, 0], u[:, width:] = g, 0.75
    u, da = u.cuda(), torch.full((n, width), 0.5, dtype=dtype, device="cuda")
    rows = dq.expert_rows(torch.zeros((n, 1), dtype=torch.int32, device="cuda"), 1)
    gates = torch.full((n, 1), 0.5, device="cuda")
    a, kept = dq.expert_act(u, gates, rows, keep=True, dither=False)
    whole = kept.exponents[:, 0] != 255
    assert not whole[-1] and whole[:-1].all()            # beyond 127 2^121 alone a block is not kept
    for source, values, there in ((u, f64(u), torch.ones_like(whole)), (kept, f64(dq.restore8(kept)), whole)):
        du, dgates, again = dq.expert_act_backward(source, da, gates, rows)
        there = there.cpu().numpy()
        (wdu, wgate, wa), (e_du, e_gate, e_a) = ref.act_backward(values[there], f64(da)[there], np.full(there.sum(), 0.5), "swiglu")
        # from 20 on the sum 1 + e^-g is 1 in fp32 (e^-20 < 2^-28), and so are the sigmoid and the slope, but for
        # g e^-g < 2^-24: what is left of dg's roundings are its products'
        e_du[:, 0] = (ref.SIGMOID + 5) * U * np.abs(wdu[:, 0])
        if source is u:
            close(a, wa, e_a, dtype)
            assert torch.equal(again, a)
        close(again[whole if source is kept else slice(None)], wa, e_a, dtype)
        close(du[whole if source is kept else slice(None)], wdu, e_du, dtype)
        close(dgates[whole if source is kept else slice(None)], wgate[:, None], e_gate[:, None], torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
def test_act_of_infinities(dtype):
    """silu of +infinity is +infinity, of -infinity and NaN NaN, as g / (1 + exp(-g)) gives
    them; the neighbours keep their values."""
    inf = float("inf")
    u = torch.tensor([[inf, inf, -inf, float("nan"), 1.0, -1.0, 2.0, 0.0] + [0.5, -0.5] + [0.5] * 6], dtype=dtype).cuda()
    rows = dq.expert_rows(torch.zeros((1, 1), dtype=torch.int32, device="cuda"), 1)
    a = dq.expert_act(u, torch.ones(1, 1, device="cuda"), rows)[0]
    assert a[0] == inf and a[1] == -inf and torch.isnan(a[2:4]).all()
    u[0, :4] = 0
    assert torch.equal(a[4:], dq.expert_act(u, torch.ones(1, 1, device="cuda"), rows)[0, 4:])


@pytest.mark.parametrize("dtype", DTYPES)
def test_act_gradients_far_from_zero(dtype):
    """The far arguments of test_act_far_from_zero by value: below -87 the sigmoid is 0, from
    20 on it is 1."""
    g = torch.tensor([-1e30, -500.0, -100.0, -87.5, 30.0, 89.0, 500.0, 1e30], dtype=torch.float64).to(dtype)
    n = len(g)
    u = torch.cat((g, torch.ones(n, dtype=dtype))).cuda()[None]
    da = torch.full((1, n), 0.5, dtype=dtype, device="cuda")
    rows = dq.expert_rows(torch.zeros((1, 1), dtype=torch.int32, device="cuda"), 1)
    gates = torch.ones(1, 1, device="cuda")
    g64 = f64(g)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-g64))
    silu = g64 * s
    # below -87 off by at most 88 e^-87 < 2^-118 of the factors
    far = 2.0 ** -118
    close(dq.expert_act(u, gates, rows), silu[None], ((ref.SIGMOID + 4) * U * np.abs(silu) + far)[None], dtype)
    du, dgates, _ = dq.expert_act_backward(u, da, gates, rows)
    slope = np.where(g64 > 0, 1.0, s * (1 + g64 * (1 - s)))          # 30 e^-30 < 2^-38
    want = 0.5 * np.concatenate((slope, silu))
    close(du, want[None], ((ref.SIGMOID + 5) * U * np.abs(want) + far)[None], dtype)
    total = (0.5 * silu).sum()
    close(dgates, np.array([[total]]), (n + ref.SIGMOID + 5) * U * 0.5 * np.abs(silu).sum() + n * far, torch.float32)


# ---- larger shapes, against fp64 products on the GPU -------------------------------

def gpu_matmul(x, w, rows, gather):
    """(y, sum of |x| |w|) in fp64, expert by expert."""
    x = x[rows.source.long() // rows.top_k] if gather else x
    at = rows.offsets.tolist()
    y, mag = (torch.zeros(at[-1], w.shape[2], dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(rows.experts):
        r = slice(at[e], at[e + 1])
        y[r] = x[r].double() @ w[e].double()
        mag[r] = x[r].double().abs() @ w[e].double().abs()
    return y, mag


def gpu_grad(x, dy, rows, gather):
    token = rows.source.long() // rows.top_k
    x, dy = x[token] if gather == "x" else x, dy[token] if gather == "dout" else dy
    at = rows.offsets.tolist()
    dw, mag = (torch.zeros(rows.experts, x.shape[1], dy.shape[1], dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(rows.experts):
        r = slice(at[e], at[e + 1])
        dw[e] = x[r].double().t() @ dy[r].double()
        mag[e] = x[r].double().t().abs() @ dy[r].double().abs()
    return dw, mag, max(b - a for a, b in zip(at, at[1:]))


def near(got, want, bound, dtype):
    err = (got.double() - want).abs()
    tol = bound * (1 + 2 * half_step(dtype)) + half_step(dtype) * want.abs() + 1e-37
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.numel()} off, worst {(err / tol).max():.3g} of its bound"


# every tile: from few rows an expert to many, narrow and wide, whole steps and not
LARGE = [(3, 2, 4, 1024, 520), (200, 2, 8, 1032, 264), (400, 2, 8, 512, 1040), (2048, 2, 8, 264, 520), (4100, 2, 4, 320, 776),
         (1500, 1, 2, 96, 72), (9000, 2, 3, 40, 24), (700, 4, 5, 333, 1029), (60, 2, 33, 1024, 1000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,K,N", LARGE)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("turned", [False, True])
def test_matmul_large(T, k, E, K, N, gather, turned, dtype):
    rows = dq.expert_rows(choices(T, k, E, seed=N, none=0.1).cuda(), E)
    n = rows.offsets[-1].item()
    x = randn((T if gather else T * k, K), dtype, 1)
    w = randn((E, N, K) if turned else (E, K, N), dtype, 2)
    w = w.transpose(1, 2) if turned else w
    out = torch.full((T * k, N), SENTINEL, dtype=dtype, device="cuda")
    dq.expert_matmul(x, w, rows, gather=gather, out=out)
    y, mag = gpu_matmul(x, w, rows, gather)
    near(out[:n], y, product_bound(K, mag), dtype)
    assert (out[n:] == SENTINEL).all()
    again = torch.full_like(out, SENTINEL)
    dq.expert_matmul(x, w, rows, gather=gather, out=again)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,K,N", LARGE)
@pytest.mark.parametrize("gather", [None, "x", "dout"])
@pytest.mark.parametrize("kept", [False, True])
def test_matmul_grad_large(T, k, E, K, N, gather, kept, dtype):
    rows = dq.expert_rows(choices(T, k, E, seed=N, none=0.1).cuda(), E)
    x, dy = randn((T if gather == "x" else T * k, K), dtype, 1), randn((T if gather == "dout" else T * k, N), dtype, 2)
    given = x
    if kept:
        given = dq.keep8(x)
        x = dq.restore8(given)
    dw, mag, most = gpu_grad(x, dy, rows, gather)
    for out in {dtype, torch.float32}:
        got = dq.expert_matmul_grad(given, dy, rows, gather=gather, dtype=out)
        near(got, dw, product_bound(most, mag), out)
        assert torch.equal(got, dq.expert_matmul_grad(given, dy, rows, gather=gather, dtype=out))


# every tile of the products and of their gradients in many inner steps, so that its stages in
# LDS are gone round more than once; test_experts_cpu.py holds the lists of shapes to that
DEEP = [(4096, 2, 4, 264, 2056), (8192, 2, 4, 264, 2056), (2048, 2, 2, 1032, 4104), (1500, 2, 4, 2056, 2056),
        (1500, 2, 4, 1032, 1032), (65536, 2, 4, 64, 56), (16, 2, 4, 4104, 264)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,K,N", DEEP)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("turned", [False, True])
def test_matmul_deep(T, k, E, K, N, gather, turned, dtype):
    rows = dq.expert_rows(choices(T, k, E, seed=K, none=0.1).cuda(), E)
    n = rows.offsets[-1].item()
    x = randn((T if gather else T * k, K), dtype, 1)
    if not gather:
        x[n:] = float("nan")                         # nobody's rows
    w = randn((E, N, K) if turned else (E, K, N), dtype, 2)
    w = w.transpose(1, 2) if turned else w
    y, mag = gpu_matmul(x, w, rows, gather)
    bound = product_bound(K, mag)
    out = torch.full((T * k, N), SENTINEL, dtype=dtype, device="cuda")
    for _ in range(2):
        dq.expert_matmul(x, w, rows, gather=gather, out=out)
        near(out[:n], y, bound, dtype)
        assert (out[n:] == SENTINEL).all()
    again = wide(torch.full((T * k, N), SENTINEL, dtype=dtype, device="cuda"))
    dq.expert_matmul(wide(x), w, rows, gather=gather, out=again)
    near(again[:n], y, bound, dtype)
    assert (again[n:] == SENTINEL).all()
    base = again._base
    assert torch.isnan(base[:, 0]).all() and torch.isnan(base[:, -2:]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,K,N", DEEP)
@pytest.mark.parametrize("gather", [None, "x", "dout"])
@pytest.mark.parametrize("kept", [False, True])
def test_matmul_grad_deep(T, k, E, K, N, gather, kept, dtype):
    rows = dq.expert_rows(choices(T, k, E, seed=K, none=0.1).cuda(), E)
    n = rows.offsets[-1].item()
    x, dy = randn((T if gather == "x" else T * k, K), dtype, 1), randn((T if gather == "dout" else T * k, N), dtype, 2)
    if gather != "x":
        x[n:] = float("nan")
    if gather != "dout":
        dy[n:] = float("nan")
    given = x
    if kept:
        given = dq.keep8(x)
        x = dq.restore8(given)
    dw, mag, most = gpu_grad(x, dy, rows, gather)
    bound = product_bound(most, mag)
    for out in {dtype, torch.float32}:
        got = dq.expert_matmul_grad(given, dy, rows, gather=gather, dtype=out)
        near(got, dw, bound, out)
        assert torch.equal(got, dq.expert_matmul_grad(given, dy, rows, gather=gather, dtype=out))
    near(dq.expert_matmul_grad(given if kept else wide(x), wide(dy), rows, gather=gather), dw, bound, dtype)


def test_rows_far_apart():
    """Offsets of 2^31 bytes and more, which the kernels' 32-bit loads take, and beyond
    2^32, which they do not; outputs and experts as far apart."""
    E, K, N = 2, 72, 40
    ids = torch.tensor([[0, 1], [1, 0], [1, -1]], dtype=torch.int32, device="cuda")
    for apart in (1 << 30, 3 << 30):
        T = 2 if apart == 1 << 30 else 3
        rows = dq.expert_rows(ids[:T].contiguous(), E)
        n = rows.offsets[-1].item()
        mem = torch.empty((T - 1) * apart + 4096, dtype=torch.bfloat16, device="cuda")
        x = mem.as_strided((T, K), (apart, 1))
        x.copy_(randn((T, K), torch.bfloat16, 1))
        w = randn((E, K, N), torch.bfloat16, 2)
        y, mag = gpu_matmul(x, w, rows, True)
        near(dq.expert_matmul(x, w, rows, gather=True)[:n], y, product_bound(K, mag), torch.bfloat16)
        dy = randn((2 * T, N), torch.bfloat16, 3)
        dw, mag, most = gpu_grad(x, dy, rows, "x")
        near(dq.expert_matmul_grad(x, dy, rows, gather="x"), dw, product_bound(most, mag), torch.bfloat16)
        # the same memory as an output, and as weights
        far = mem.as_strided((T, N), (apart, 1), 256)
        z, mag = gpu_back(dy, rows)
        dq.expert_sum(dy, rows, out=far)
        near(far, z, 4 * U * mag, torch.bfloat16)
        wf = mem.as_strided((E, K, N), (apart, N, 1), 1024)
        wf.copy_(w)
        xs = x.contiguous()
        assert torch.equal(dq.expert_matmul(xs, wf, rows, gather=True)[:n], dq.expert_matmul(xs, w, rows, gather=True)[:n])
        kept = dq.keep8(x)
        assert torch.equal(kept.codes, dq.keep8(xs).codes)
        del mem, x, far, wf


def gpu_back(y, rows):
    at = rows.row.long()
    v = torch.where((at >= 0)[:, :, None], y.double()[at.clamp(min=0)], 0.0)
    return v.sum(1), v.abs().sum(1)


def test_keep_beyond_32_bits():
    """2^32 + 4096 elements of rows 1000 wide (dithers at any offset) and 1024 wide."""
    for cols in (1000, 1024):
        n = ((1 << 32) + 4096) // cols
        x = torch.empty((n, cols), dtype=torch.bfloat16, device="cuda").fill_(0.3)
        x[-1] = randn((cols,), torch.bfloat16, 1)
        kept = dq.keep8(x, **KEY)
        first = (n - 1) * cols
        b0 = first // 8
        key = dict(KEY)
        from oracle import pyoracle as po
        d = []
        for b in range(b0, b0 + cols // 8 + 1):
            w = po.philox4x32([b & 0xFFFFFFFF, (b >> 32) | 0x8000 | key["worker"] << 16, key["rnd"], (1 << 31) | key["site"]],
                              [key["seed"] & 0xFFFFFFFF, key["seed"] >> 32])
            d += [h for v in w for h in (int(v) & 0xFFFF, int(v) >> 16)]
        codes, exps, _ = ref.keep(f64(x[-1:]), np.array(d[first - 8 * b0:][:cols], np.int64))
        assert np.array_equal(kept.codes[-1:].cpu().numpy(), codes)
        assert np.array_equal(kept.exponents[-1:].cpu().numpy(), exps)
        assert torch.equal(dq.restore8(dq.Kept8(kept.codes[-1:].clone(), kept.exponents[-1:].clone(), kept.dtype))[0],
                           dq.restore8(kept)[-1])
        del x, kept


def test_entries_out_of_range_are_no_rows():
    """Lists that no call of expert_rows makes: slots out of range read as zeros, rows
    out of range add nothing, offsets are held to the rows there are."""
    dtype = torch.bfloat16
    ids = torch.tensor([[0], [1], [1], [0]], dtype=torch.int32, device="cuda")
    good = dq.expert_rows(ids, 2)
    x, w, dy = randn((4, 64), dtype, 1), randn((2, 64, 64), dtype, 2), randn((4, 64), dtype, 3)
    source = good.source.clone()
    source[1], source[2] = 1 << 30, -5
    bad = dq.ExpertRows(good.offsets, source, good.row)
    want = dq.expert_matmul(x, w, good, gather=True)
    got = dq.expert_matmul(x, w, bad, gather=True)
    assert torch.equal(got[[0, 3]], want[[0, 3]]) and (got[1:3] == 0).all()
    dy[1:3] = 0
    assert torch.equal(dq.expert_matmul_grad(x, dy, bad, gather="x"), dq.expert_matmul_grad(x, dy, good, gather="x"))
    row = good.row.clone()
    row[0], row[1] = 4, -(1 << 30)
    assert (dq.expert_sum(dy, dq.ExpertRows(good.offsets, good.source, row))[:2] == 0).all()
    gates = torch.ones(4, 1, device="cuda")
    a = dq.expert_act(x, gates, bad)
    assert (a[1:3] == 0).all() and torch.equal(a[[0, 3]], dq.expert_act(x, gates, good)[[0, 3]])
    high = dq.ExpertRows(torch.tensor([-3, 2, 1 << 30], dtype=torch.int32, device="cuda"), good.source, good.row)
    assert torch.equal(dq.expert_matmul(x, w, high, gather=True), want)
    none = dq.ExpertRows(torch.tensor([3, 2, 1], dtype=torch.int32, device="cuda"), good.source, good.row)
    out = torch.full((4, 64), SENTINEL, dtype=dtype, device="cuda")
    assert (dq.expert_matmul(x, w, none, gather=True, out=out) == SENTINEL).all()
    assert (dq.expert_matmul_grad(x, dy, none, gather="x") == 0).all()


def test_offsets_that_name_every_row_for_every_other_expert():
    """512 experts that claim all of 2^29 + 1 rows: 2^32 + 512 tiles of 64 rows.  What the blocks
    there are compute is right, and nothing beyond the rows is written."""
    slots, E = (1 << 29) + 1, 1024
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1::2] = slots
    source = torch.arange(slots, dtype=torch.int32, device="cuda")
    rows = dq.ExpertRows(offsets, source, torch.empty((slots, 1), dtype=torch.int32, device="cuda"))
    mem = torch.full((slots + 4096,), SENTINEL, device="cuda")
    x, w = torch.full((1, 1), 3.0, device="cuda"), torch.full((1, 1, 1), 2.0, device="cuda")
    for gather in (False, True):
        dq.expert_matmul(x.expand(slots, 1), w.expand(E, 1, 1), rows, gather=gather, out=mem[:slots].view(slots, 1))
        done = mem == 6.0
        assert (done | (mem == SENTINEL)).all() and not done[slots:].any()
        # a block for every tile of the rows at least, 64 or so of them at the same rows
        assert done.sum() > 1 << 25
        mem.fill_(SENTINEL)


def test_infinities_stay_in_their_rows():
    dtype = torch.bfloat16
    ids = choices(64, 2, 4, none=0).cuda()
    rows = dq.expert_rows(ids, 4)
    x, w = randn((64, 72), dtype, 1), randn((4, 72, 40), dtype, 2)
    clean = dq.expert_matmul(x, w, rows, gather=True)
    x[5, 3], x[9, 0] = float("inf"), float("nan")
    got = dq.expert_matmul(x, w, rows, gather=True)
    hit = torch.isin(rows.source // 2, torch.tensor([5, 9], device="cuda"))
    assert torch.equal(got[~hit], clean[~hit]) and not torch.isfinite(got[hit]).any()
    w[2] = float("nan")
    got = dq.expert_matmul(x, w, rows, gather=True)
    at = rows.offsets.tolist()
    other = torch.ones(128, dtype=torch.bool, device="cuda")
    other[at[2]:at[3]] = False
    assert torch.equal(got[other & ~hit], clean[other & ~hit])


def test_expanded_operands():
    ids = choices(40, 2, 4, none=0).cuda()
    rows = dq.expert_rows(ids, 4)
    row, w = randn((1, 64), torch.float32, 1), randn((1, 64, 24), torch.float32, 2)
    a = dq.expert_matmul(row.expand(40, 64), w.expand(4, 64, 24), rows, gather=True)
    assert torch.equal(a, dq.expert_matmul(row.repeat(40, 1), w.repeat(4, 1, 1), rows, gather=True))
    dy = randn((80, 24), torch.float32, 3)
    assert torch.equal(dq.expert_matmul_grad(row.expand(40, 64), dy, rows, gather="x"),
                       dq.expert_matmul_grad(row.repeat(40, 1), dy, rows, gather="x"))


# ---- through autograd, streams, graphs ----------------------------------------------

def layer(seed, T, k, E, H, F, kind, dtype, none=0.2):
    ids = choices(T, k, E, seed=seed, none=none).cuda()
    x, dy = randn((T, H), dtype, seed), randn((T, H), dtype, seed + 1)
    gates = torch.rand(T, k, generator=torch.Generator().manual_seed(seed)).cuda()
    w_in = randn((E, H, F * (2 if kind == "swiglu" else 1)), dtype, seed + 2, H ** -0.5)
    w_out = randn((E, F, H), dtype, seed + 3, F ** -0.5)
    return ids, x, dy, gates, w_in, w_out


def by_calls(ids, x, dy, gates, w_in, w_out, kind, keep, key):
    """The same layer by the calls it is made of."""
    rows = dq.expert_rows(ids, w_in.shape[0])
    u = dq.expert_matmul(x, w_in, rows, gather=True)
    a = dq.expert_act(u, gates, rows, kind)
    y = dq.expert_sum(dq.expert_matmul(a, w_out, rows), rows)
    kx, ku = x, u
    if keep:
        kx, ku = dq.keep8(x, **key), dq.keep8(u, **{**key, "site": key["site"] + 1})
    da = dq.expert_matmul(dy, w_out.transpose(1, 2), rows, gather=True)
    du, dgates, again = dq.expert_act_backward(ku, da, gates, rows, kind)
    return [y, dq.expert_sum(dq.expert_matmul(du, w_in.transpose(1, 2), rows), rows), dgates,
            dq.expert_matmul_grad(kx, du, rows, gather="x"), dq.expert_matmul_grad(again, dy, rows, gather="dout")]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["swiglu", "relu"])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("T,H,F", [(1, 64, 32), (50, 72, 40), (33, 65, 31), (300, 256, 128)])
def test_experts_autograd(T, H, F, keep, kind, dtype):
    ids, x, dy, gates, w_in, w_out = layer(T, T, 2, 4, H, F, kind, dtype, none=0.2 if T > 1 else 0)
    leaves = [t.clone().requires_grad_() for t in (x, gates, w_in, w_out)]
    y = train.experts(leaves[0], ids, *leaves[1:], act=kind, keep=keep, **KEY)
    got = [y.detach(), *torch.autograd.grad(y, leaves, dy)]
    for g, w in zip(got, by_calls(ids, x, dy, gates, w_in, w_out, kind, keep, KEY)):
        assert g.dtype == w.dtype and torch.equal(g, w)
    # only what is asked for
    y = train.experts(x, ids, gates, leaves[2], w_out, act=kind, keep=keep, **KEY)
    assert torch.equal(torch.autograd.grad(y, leaves[2], dy)[0], got[3])


@pytest.mark.parametrize("kind", ["swiglu", "relu"])
def test_experts_autograd_against_fp64(kind):
    """fp32 against autograd in fp64 of the plain loop.  Every step of the chain is off by
    less than (H + 2 F + 40) 2 U of its magnitude, and passes on at most 4 times what
    comes in (the slope of silu is below 1.1, gates below 1); magnitudes are the same
    loop's on absolute values, without the activation."""
    T, k, E, H, F = 60, 2, 4, 64, 48
    ids, x, dy, gates, w_in, w_out = layer(5, T, k, E, H, F, kind, torch.float32)
    leaves = [t.clone().requires_grad_() for t in (x, gates, w_in, w_out)]
    y = train.experts(leaves[0], ids, *leaves[1:], act=kind)
    got = [y.detach(), *torch.autograd.grad(y, leaves, dy)]

    def loop(x, gates, w_in, w_out, f):
        y = torch.zeros(T, H, dtype=torch.float64)
        for t in range(T):
            for j in range(k):
                e = int(ids[t, j])
                if e >= 0:
                    y[t] = y[t] + gates[t, j] * (f(x[t] @ w_in[e]) @ w_out[e])
        return y

    def swiglu(u):
        return torch.nn.functional.silu(u[:F]) * u[F:]

    args = [t.detach().cpu().double().requires_grad_() for t in leaves]
    want = loop(*args, swiglu if kind == "swiglu" else torch.relu)
    want = [want.detach(), *torch.autograd.grad(want, args, dy.cpu().double())]
    mags = [t.detach().cpu().double().abs().requires_grad_() for t in leaves]
    mag = loop(*mags, (lambda u: u[:F] * u[F:]) if kind == "swiglu" else (lambda u: u))
    mag = [mag.detach(), *torch.autograd.grad(mag, mags, dy.cpu().double().abs())]
    for g, w, m in zip(got, want, mag):
        err = (g.cpu().double() - w).abs()
        bound = 4 * 4 * (H + 2 * F + 40) * 2 * U * m
        assert (err <= bound).all(), (err / bound).max()


def test_kept_weight_gradient_is_right_in_the_mean():
    """x kept with dither: dw = sum of kept(x)^T du over draws comes near x^T du."""
    T, H, N = 64, 64, 8
    rows = dq.expert_rows(torch.zeros((T, 1), dtype=torch.int32, device="cuda"), 1)
    x, du = randn((T, H), torch.float32, 1), randn((T, N), torch.float32, 2)
    n = 400
    mean = sum(dq.expert_matmul_grad(dq.keep8(x, rnd=i), du, rows).double() for i in range(n)) / n
    want = x.double().t() @ du.double()
    step = torch.exp2(dq.keep8(x).exponents.double() - 127).repeat_interleave(32, 1)
    # an element's draw has a variance of at most step^2 / 4; sums of 64 of them
    sd = (0.25 * (step ** 2).t() @ du.double() ** 2).sqrt()[None] / n ** 0.5
    assert ((mean - want).abs() <= 6 * sd + 1e-4 * sd * n ** 0.5 + 2 ** -15 * sd * n ** 0.5).all()


def test_no_tokens():
    ids = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    for dtype in DTYPES:
        args = [torch.zeros(s, dtype=d, device="cuda", requires_grad=True) for s, d in
                (((0, 16), dtype), ((0, 2), torch.float32), ((3, 16, 8), dtype), ((3, 4, 16), dtype))]
        for keep in (False, True):
            y = train.experts(args[0], ids, *args[1:], keep=keep)
            assert y.shape == (0, 16)
            grads = torch.autograd.grad(y.sum(), args)
            assert all(g.shape == a.shape and (g == 0).all() for g, a in zip(grads, args))


def test_on_another_stream():
    ids, x, dy, gates, w_in, w_out = layer(3, 200, 2, 4, 64, 48, "swiglu", torch.bfloat16)
    want = by_calls(ids, x, dy, gates, w_in, w_out, "swiglu", True, KEY)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = by_calls(ids, x, dy, gates, w_in, w_out, "swiglu", True, KEY)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    rows = dq.expert_rows(ids, 4, stream=side)
    u = dq.expert_matmul(x, w_in, rows, gather=True, stream=side)
    a, kept = dq.expert_act(u, gates, rows, keep=True, stream=side, **KEY)
    y = dq.expert_sum(dq.expert_matmul(a, w_out, rows, stream=side), rows, stream=side)
    r = dq.restore8(dq.keep8(x, stream=side), stream=side)
    dw = dq.expert_matmul_grad(x, a, rows, gather="x", stream=side)
    side.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(r, dq.restore8(dq.keep8(x)))
    assert torch.equal(dw, dq.expert_matmul_grad(x, a, rows, gather="x"))


def test_layer_in_graph_replays():
    """Two captured layers over the same inputs, replayed in turn with other tokens,
    choices and rounds, and eager work between: every replay gives the eager bits."""
    T, k, E, H, F = 120, 2, 4, 64, 48
    ids, x, dy, gates, w_in, w_out = layer(7, T, k, E, H, F, "swiglu", torch.bfloat16)
    rnd = torch.zeros(1, dtype=torch.int32, device="cuda")
    key = dict(KEY, rnd=rnd)

    def step():
        return by_calls(ids, x, dy, gates, w_in, w_out, "swiglu", True, key)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for i in range(6):
        fresh = layer(100 + i, T, k, E, H, F, "swiglu", torch.bfloat16, none=0.2 if i % 2 else 0.9)
        for to, new in zip((ids, x, dy, gates), fresh):
            to.copy_(new)
        rnd.fill_(i)
        n = int((ids >= 0).sum())
        want = [t.clone() for t in step()]
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (i, n)


def test_route_experts_dropout_together():
    """A step of a mixture-of-experts block as a program runs it: route, experts with
    kept activations, dropout onto the residual, backward through all of them."""
    T, k, E, H, F = 200, 2, 8, 64, 48
    dtype = torch.bfloat16
    x = randn((T, H), dtype, 1)
    leaves = [randn(s, dtype, i, H ** -0.5).requires_grad_() for i, s in
              enumerate(((H, E), (E, H, 2 * F), (E, F, H)))]
    mask = torch.rand(T, generator=torch.Generator().manual_seed(0)) > 0.1
    xs = x.clone().requires_grad_()
    r = train.route((xs @ leaves[0]).float(), k, masks=mask.cuda())
    y = train.experts(xs, r.ids, r.gates, *leaves[1:], keep=True, rnd=3)
    z = train.dropout(y, 0.1, residual=xs, rnd=3)
    grads = torch.autograd.grad((z.float() ** 2).mean() + 0.01 * r.loss.sum(), [xs, *leaves])
    assert all(torch.isfinite(g).all() and g.abs().sum() > 0 for g in grads)
    # tokens left out: the experts add nothing, and their gradient is the residual's alone
    assert (y[~mask.cuda()] == 0).all() and torch.equal(z[~mask.cuda()], x[~mask.cuda()])
    dz = (2 * z.detach().float() / z.numel()).to(dtype)
    assert torch.equal(grads[0][~mask.cuda()], dz[~mask.cuda()])


def test_refusals():
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    rows = dq.expert_rows(ids, 3)
    x, w = torch.zeros(8, 16, device="cuda"), torch.zeros(3, 16, 24, device="cuda")
    gates = torch.ones(4, 2, device="cuda")
    for call in (lambda: dq.expert_matmul(x[:4], w, rows), lambda: dq.expert_matmul(x, w, rows, gather=True),
                 lambda: dq.expert_matmul(x, w[:2], rows), lambda: dq.expert_matmul(x, w.bfloat16(), rows),
                 lambda: dq.expert_matmul(x, w[:, :, ::2], rows), lambda: dq.expert_matmul(x.t(), w, rows),
                 lambda: dq.expert_matmul(x, w, rows, out=x), lambda: dq.expert_matmul(x, w, rows, out=torch.zeros(8, 24)),
                 lambda: dq.expert_matmul_grad(x, x, rows, gather="y"), lambda: dq.expert_matmul_grad(x, x[:4], rows),
                 lambda: dq.expert_matmul_grad(dq.keep8(x[:4]), x, rows),
                 lambda: dq.expert_matmul_grad(dq.keep8(x.bfloat16()), x, rows),
                 lambda: dq.expert_matmul_grad(x, x, rows, out=torch.zeros(3, 16, 15, device="cuda")),
                 lambda: dq.expert_sum(x[:4], rows), lambda: dq.expert_sum(x, rows, residual=x),
                 lambda: dq.expert_act(x, gates[:3], rows), lambda: dq.expert_act(x, gates, rows, "tanh"),
                 lambda: dq.expert_act(x[:, :15], gates, rows), lambda: dq.expert_act_backward(x, x, gates, rows),
                 lambda: dq.expert_act_backward(x, x[:, :8], gates, rows, du=x[:, :8]),
                 lambda: dq.expert_rows(ids, 0), lambda: dq.expert_rows(ids, 1025), lambda: dq.expert_rows(ids[0], 3),
                 lambda: dq.keep8(x, seed=-1), lambda: dq.keep8(x, worker=1 << 16), lambda: dq.keep8(x.t()),
                 lambda: dq.restore8(dq.keep8(x), out=x[:4]),
                 lambda: dq.Kept8(torch.zeros(4, 40, dtype=torch.int8, device="cuda"),
                                  torch.zeros(4, 1, dtype=torch.uint8, device="cuda"), torch.float32)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: dq.expert_matmul_grad(x, x, rows, dtype=torch.bfloat16), lambda: dq.expert_rows(ids.long(), 3),
                 lambda: dq.expert_act(x, gates.double(), rows), lambda: dq.keep8(x.half()),
                 lambda: dq.Kept8(torch.zeros(4, 40, dtype=torch.int8, device="cuda"),
                                  torch.zeros(4, 2, dtype=torch.uint8, device="cuda"), torch.float16)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(dq.DQError):
        dq.expert_sum(x, rows, out=x[:4])            # over its operand


def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_step.py")
    spec = importlib.util.spec_from_file_location("moe_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_moe_example_with_all_experts_at_once():
    """The example's gradients with grouped experts against its own loop, in fp32; with
    kept activations it runs and its gradients are finite."""
    moe = _example()
    grads = []
    for how in (dict(), dict(grouped=True), dict(grouped=True, keep=True)):
        leaves = {k: w.requires_grad_() for k, w in moe.init().items()}
        data = [moe.batch(0, 0, 128)]
        task, balance, _ = moe.losses([leaves], data, 0, **how)
        g = torch.autograd.grad(sum(task) + moe.BALANCE * balance.sum(), list(leaves.values()))
        grads.append(torch.cat([x.reshape(-1) for x in g]).double())
        assert torch.isfinite(grads[-1]).all()
    # a chain of 2 x 2 products forward and 2 x 4 back, each off by at most (FFN + 2) 2 U of its
    # magnitude, which for random terms is about FFN ** 0.5 times the value, by norm
    bound = 12 * (moe.FFN + 2) * 2 * U * moe.FFN ** 0.5
    assert (grads[1] - grads[0]).norm() <= bound * grads[0].norm()
    t = moe.Trainer(workers=2, tokens=64, keep=True)
    assert all(np.isfinite(v) for v in t.step(0)[:2])
