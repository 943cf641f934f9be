"""The experts' operators on the GPU against their plain fp64 forms
(experts_ref.py): lists and codes exactly, the rest within the roundings that
an fp32 evaluation makes."""
import numpy as np
import pytest
import torch

import experts_ref as ref
from compressed_hop_gradient_amd import dq

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
