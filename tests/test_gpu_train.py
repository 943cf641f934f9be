"""Training-step operators on the GPU against their plain fp64 forms
(train_ref.py): dropout bit for bit, the router's choices and counts exactly,
its gates, loss and gradients within the roundings that an fp32 evaluation
makes."""
import math

import numpy as np
import pytest
import torch

import train_ref as ref
from compressed_hop_gradient_amd import dq, train

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]
U = ref.U


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def half_step(dtype):
    """Relative error of one rounding to ``dtype`` (0 for fp32, whose rounding
    the magnitudes count)."""
    return torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def same(a, b):
    return torch.equal(bits(a.cpu()), bits(b.cpu()))


# ---- dropout ------------------------------------------------------------------

KEY = dict(seed=0x123456789ABCDEF1, rnd=77, worker=5, site=3)


def expected_dropout(x, p, residual=None, seed=1, rnd=0, worker=0, site=0):
    """On the CPU, from fp32 operations in the documented order (each correctly
    rounded, so the bits are determined)."""
    x = x.cpu().float()
    t = ref.threshold(p)
    d = torch.from_numpy(ref.dithers(x.numel(), seed, rnd, worker, site)).reshape(x.shape)
    scale = torch.tensor(0.0 if t == 65536 else 65536.0 / (65536 - t), dtype=torch.float32)
    y = torch.where(d >= t, x * scale, torch.zeros(()))
    return y if residual is None else residual.cpu().float() + y


def randn(shape, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (3, 5), (64, 8), (255,), (33, 72), (17, 1337), (2, 3, 4100),
                                   (), (0,), (4, 0)])
def test_dropout_bits(shape, with_residual, dtype):
    x = randn(shape, dtype)
    r = randn(shape, dtype, 1) if with_residual else None
    y = dq.dropout(x, 0.3, residual=r, **KEY)
    assert y.shape == x.shape and y.dtype == dtype
    assert same(y, expected_dropout(x, 0.3, r, **KEY).to(dtype))


@pytest.mark.parametrize("p", [0.0, 1e-9, 1 / 65536, 0.1, 0.5, 0.9, 65535 / 65536, 1.0])
@pytest.mark.parametrize("with_residual", [False, True])
def test_dropout_rates(p, with_residual):
    x, r = randn((5000,), torch.float32), randn((5000,), torch.float32, 1) if with_residual else None
    y = dq.dropout(x, p, residual=r, **KEY)
    assert same(y, expected_dropout(x, p, r, **KEY))
    if p == 1.0 and r is not None:
        assert torch.equal(y, r)
    if p < 1e-8 and r is None:
        assert torch.equal(y, x)


def test_dropout_keeps_the_mean_and_the_rate():
    n, p = 1 << 22, 0.1
    y = dq.dropout(torch.ones(n, device="cuda"), p, **KEY)
    t = ref.threshold(p)
    q = 1 - t / 65536
    kept = (y != 0).double().mean().item()
    assert abs(kept - q) < 6 * math.sqrt(q * (1 - q) / n)            # 6 standard deviations
    assert abs(y.double().mean().item() - 1) < 6 * math.sqrt((1 - q) / q / n)


@pytest.mark.parametrize("changed", [dict(seed=2), dict(rnd=78), dict(worker=6), dict(site=4)])
def test_dropout_key_parts_change_the_mask(changed):
    x = torch.ones(4096, device="cuda")
    key = {**KEY, **changed}
    y = dq.dropout(x, 0.5, **key)
    assert same(y, expected_dropout(x, 0.5, **key))
    assert not torch.equal(y, dq.dropout(x, 0.5, **KEY))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,wide,at", [(37, 64, 128, 0), (37, 64, 128, 64), (37, 61, 128, 0), (37, 64, 67, 1),
                                               (37, 8, 24, 8), (5, 1, 9, 2), (1024, 24, 1000, 16), (3, 2048, 4096, 0)])
def test_dropout_views_have_the_mask_of_their_copy(rows, cols, wide, at, dtype):
    """Row strides and alignments, of each operand on its own and of all."""
    big, other = randn((rows, wide), dtype), randn((rows, wide), dtype, 1)
    x, r = big[:, at:at + cols], other[:, at:at + cols]
    want = expected_dropout(x, 0.4, r, **KEY).to(dtype)
    for xv, rv in ((x, r), (x.contiguous(), r), (x, r.contiguous()), (x.contiguous(), r.contiguous())):
        assert same(dq.dropout(xv, 0.4, residual=rv, **KEY), want)
        out = torch.full((rows, wide), 7.0, dtype=dtype, device="cuda")
        dq.dropout(xv, 0.4, residual=rv, out=out[:, at:at + cols], **KEY)
        assert same(out[:, at:at + cols], want)
        out[:, at:at + cols] = 7.0
        assert bool((out == 7.0).all())                               # nothing beside the view
    assert same(dq.dropout(x, 0.4, **KEY), expected_dropout(x, 0.4, **KEY).to(dtype))


@pytest.mark.parametrize("off", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("dtype", DTYPES)
def test_dropout_unaligned_pieces(off, dtype):
    base = randn((4000,), dtype)
    x = base[off:off + 2777]
    out = torch.empty(4000, dtype=dtype, device="cuda")
    assert same(dq.dropout(x, 0.4, **KEY), expected_dropout(x, 0.4, **KEY).to(dtype))
    assert same(dq.dropout(x, 0.4, out=out[3:3 + 2777], **KEY), expected_dropout(x, 0.4, **KEY).to(dtype))


def test_dropout_three_dimensional_and_broadcast_views():
    x = randn((6, 4, 32), torch.bfloat16)
    v = x[:, :, 8:24]
    assert same(dq.dropout(v, 0.4, **KEY), expected_dropout(v, 0.4, **KEY).bfloat16())
    b = randn((32,), torch.bfloat16).expand(6, 32)                   # row stride 0
    assert same(dq.dropout(b, 0.4, **KEY), expected_dropout(b, 0.4, **KEY).bfloat16())
    with pytest.raises(ValueError):
        dq.dropout(x.transpose(1, 2), 0.4)


@pytest.mark.parametrize("dtype", DTYPES)
def test_dropout_in_place_and_halves_of_one_tensor(dtype):
    x, r = randn((19, 72), dtype), randn((19, 72), dtype, 1)
    want = expected_dropout(x, 0.4, r, **KEY).to(dtype)
    a = x.clone()
    assert same(dq.dropout(a, 0.4, residual=r, out=a, **KEY), want)
    a = r.clone()
    assert same(dq.dropout(x, 0.4, residual=a, out=a, **KEY), want)
    wide = torch.cat((x, r), 1)
    dq.dropout(wide[:, :72], 0.4, residual=r, out=wide[:, 72:], **KEY)
    assert same(wide[:, 72:], want) and same(wide[:, :72], x)
    with pytest.raises(dq.DQError):
        dq.dropout(wide[:, :72], 0.4, out=wide[:, 1:73])


@pytest.mark.parametrize("with_residual", [False, True])
def test_dropped_values_do_not_leak(with_residual):
    """Infinity and NaN at dropped places count as 0; at kept ones they pass."""
    n = 4096
    d = ref.dithers(n, **KEY)
    t = ref.threshold(0.5)
    drop = torch.from_numpy(d < t)
    for v in (math.nan, math.inf, -math.inf):
        x = torch.full((n,), v, device="cuda")
        r = torch.ones(n, device="cuda") if with_residual else None
        y = dq.dropout(x, 0.5, residual=r, **KEY).cpu()
        assert bool((y[drop] == (1.0 if with_residual else 0.0)).all())
        assert not bool(torch.isfinite(y[~drop]).any())


@pytest.mark.parametrize("dtype", DTYPES)
def test_dropout_gradient(dtype):
    """The gradient is the mask times the scale: the formula's, the operator's
    own differences (exact: it is linear, and powers of two pass it), and equal
    for a residual that is broadcast."""
    x = randn((33, 40), dtype).requires_grad_()
    r = randn((33, 40), dtype, 1).requires_grad_()
    dy = randn((33, 40), dtype, 2)
    y = train.dropout(x, 0.3, residual=r, **KEY)
    gx, gr = torch.autograd.grad(y, (x, r), dy)
    assert same(gx, expected_dropout(dy, 0.3, **KEY).to(dtype)) and same(gr, dy)
    zero = torch.zeros_like(x)
    step = dq.dropout(zero + 1, 0.3, **KEY)                            # f(0 + 1) - f(0)
    assert same(torch.autograd.grad(train.dropout(x, 0.3, **KEY).sum(), x)[0], step)
    row = randn((40,), dtype, 3).requires_grad_()
    y = train.dropout(x, 0.3, residual=row.expand(33, 40), **KEY)
    g, = torch.autograd.grad(y, row, torch.ones_like(dy))
    assert torch.equal(g.float(), torch.full((40,), 33.0, device="cuda"))
    y = train.dropout(row.expand(33, 40), 0.3, **KEY)                  # rows at stride 0
    g, = torch.autograd.grad(y.float().sum(), row)
    want = expected_dropout(torch.ones(33, 40), 0.3, **KEY).to(dtype).double().sum(0)
    assert torch.allclose(g.double().cpu(), want, rtol=2 * torch.finfo(dtype).eps, atol=0)


def test_dropout_needs_grad_only_where_asked():
    x, r = randn((64,), torch.float32), randn((64,), torch.float32, 1).requires_grad_()
    train.dropout(x, 0.5, residual=r).sum().backward()
    assert torch.equal(r.grad, torch.ones_like(r))
    x.requires_grad_()
    assert torch.equal(train.dropout(x, 0.5, residual=r.detach(), training=False), r.detach() + x)
    y = train.dropout(x, 0.5)
    g, = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), x)


def test_round_on_the_device_and_its_change_is_noticed():
    x = torch.ones(2048, device="cuda").requires_grad_()
    rnd = torch.tensor([78], dtype=torch.int32, device="cuda")
    key = dict(seed=1, worker=2, site=9)
    assert same(dq.dropout(x.detach(), 0.5, rnd=rnd, **key), expected_dropout(x.detach(), 0.5, rnd=78, **key))
    rnd.fill_(-1)                                                     # 2^32 - 1
    assert same(dq.dropout(x.detach(), 0.5, rnd=rnd, **key),
                expected_dropout(x.detach(), 0.5, rnd=2 ** 32 - 1, **key))
    y = train.dropout(x, 0.5, rnd=rnd, **key)
    rnd.add_(1)
    with pytest.raises(RuntimeError):
        y.sum().backward()


@pytest.mark.parametrize("bad", [dict(worker=65536), dict(worker=-1), dict(site=1 << 31), dict(rnd=1 << 32),
                                 dict(seed=-1), dict(seed=1 << 64)])
def test_dropout_key_is_checked(bad):
    with pytest.raises(ValueError):
        dq.dropout(torch.ones(8, device="cuda"), 0.5, **bad)


def test_dropout_refuses_mixed_operands():
    x = torch.ones(8, 8, device="cuda")
    for bad in (x[:4], x.bfloat16(), x.cpu()):
        with pytest.raises(ValueError):
            dq.dropout(x, 0.5, residual=bad)
        with pytest.raises(ValueError):
            dq.dropout(x, 0.5, out=bad)
    with pytest.raises(TypeError):
        dq.dropout(x, 0.5, rnd=torch.zeros(1, device="cuda"))
    with pytest.raises(dq.DQError):
        dq.dropout(x, 1.5)


@pytest.mark.slow
def test_dropout_beyond_32_bits():
    """2^35 + 44 bf16 elements, in place: element offsets pass 2^32, and the last
    blocks' index, its own second counter word (64 GiB of memory)."""
    n = (1 << 35) + 44
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    print("[dropout] 2^35 elements", flush=True)
    dq.dropout(x, 0.5, out=x, **KEY)
    for first, count in ((0, 4096), ((1 << 31) - 64, 4096), ((1 << 32) - 64, 4096), ((1 << 35) - 64, 108)):
        d = ref.dithers(count, first=first, **KEY)
        want = torch.from_numpy(np.where(d >= 32768, 2.0, 0.0)).bfloat16()
        assert same(x[first:first + count], want), first


def test_row_offsets_beyond_32_bits():
    """Rows 2^31 elements apart (13 GB a tensor, of which only the rows are
    touched): dropout at any alignment, the router and its gradient."""
    stride, E, k = (1 << 31) + 8, 64, 4
    x = torch.empty(3 * stride, dtype=torch.bfloat16, device="cuda").view(3, stride)
    y = torch.empty(3 * stride, dtype=torch.bfloat16, device="cuda").view(3, stride)
    for cols in (64, 61):
        rows, out = x[:, 3:3 + cols] if cols == 61 else x[:, :cols], y[:, :cols]
        rows.copy_(randn((3, cols), torch.bfloat16, cols))
        print(f"[offsets] {cols} columns", flush=True)
        dq.dropout(rows, 0.4, out=out, **KEY)
        assert same(out, expected_dropout(rows, 0.4, **KEY).bfloat16())
    l = x[:, :E]
    l.copy_(logits_of(3, E, torch.bfloat16))
    ids, gates, stats = dq.route(l, k)
    r = check_forward(l, k, True, None, ids, gates)
    dg, coef = randn((3, k), torch.float32), dq.balance(stats, k)[1]
    check_gradient(dq.route_backward(l, ids, dg, coef, out=y[:, :E]), r, dg, coef, 1.0, torch.bfloat16)


def test_dropout_on_another_stream():
    x = randn((1 << 20,), torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = dq.dropout(x, 0.3, stream=s, **KEY)
    with torch.cuda.stream(s):
        z = dq.dropout(y, 0.0)
    torch.cuda.current_stream().wait_stream(s)
    want = expected_dropout(x, 0.3, **KEY).bfloat16()
    assert same(y, want) and same(z, want)


# ---- router ---------------------------------------------------------------------

def logits_of(T, E, dtype, seed=0, closed=0.0, coarse=False):
    g = np.random.default_rng(seed * 1000 + E)
    l = g.normal(size=(T, E)) * 2 + g.normal(size=E)
    if coarse:
        l = np.round(l)                                               # many ties, -0 and +0 among them
    if closed:
        l[g.random((T, E)) < closed] = -np.inf
        l[::5] = -np.inf
    return torch.from_numpy(l).to(dtype).cuda()


def check_forward(logits, k, renorm, mask, ids, gates):
    r = ref.Routed(logits.double().cpu().numpy(), k, renorm, None if mask is None else mask.cpu().numpy())
    assert np.array_equal(ids.cpu().numpy(), r.ids)
    got = gates.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(r.gates))
    fine = ~np.isnan(got)
    assert np.all(np.abs(got - r.gates)[fine] <= r.roundings * U * r.gates[fine] + 1e-37)
    return r


def check_stats(stats, rs):
    """Counts and tokens exactly; sums of p within the roundings of a p and of
    the fp32 part of its sum (at most one addition per token)."""
    E = rs[0].l.shape[1]
    s = stats.fold().cpu().numpy()
    assert np.array_equal(s[:E], sum(r.counts for r in rs))
    assert s[2 * E] == sum(r.tokens for r in rs)
    want = sum(r.psum for r in rs)
    most = max(r.roundings + len(r.l) for r in rs)
    assert np.all(np.abs(s[E:2 * E] - want) <= most * U * want + 1e-37)
    return most


WIDTHS = [(1, 1), (2, 2), (3, 1), (7, 7), (8, 2), (9, 4), (16, 16), (31, 5), (32, 8), (60, 4), (64, 8), (65, 6),
          (96, 3), (128, 1), (160, 6), (192, 16), (250, 8), (256, 8), (257, 2), (384, 9), (512, 8), (513, 4),
          (1000, 16), (1024, 10)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,k", WIDTHS)
@pytest.mark.parametrize("coarse", [False, True])
def test_route_widths(E, k, coarse, dtype):
    for T, renorm in ((1, True), (67, False), (131, True)):
        l = logits_of(T, E, dtype, T, coarse=coarse)
        ids, gates, stats = dq.route(l, k, renorm)
        r = check_forward(l, k, renorm, None, ids, gates)
        check_stats(stats, [r])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,k", [(8, 2), (60, 4), (64, 8), (256, 8), (1024, 16), (7, 7)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_masks_and_closed_experts(E, k, renorm, dtype):
    """Tokens left out (their logits NaN), experts closed to some tokens, tokens
    with every expert closed, fewer open experts than choices."""
    T = 203
    l = logits_of(T, E, dtype, closed=0.5)
    l[7] = -math.inf
    l[7, E - 1] = 0.5                                                  # one open expert, the last
    mask = torch.arange(T, device="cuda") % 3 != 1
    l[1] = math.nan
    l[4] = math.inf
    for m in (mask, mask.to(torch.uint8) * 9):
        ids, gates, stats = dq.route(l, k, renorm, m)
        clean = l.clone()
        clean[1] = clean[4] = 0
        r = check_forward(clean, k, renorm, mask, ids, gates)
        check_stats(stats, [r])
        assert ids[1].eq(-1).all() and gates[4].eq(0).all() and ids[5].eq(-1).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_route_everything_left_out(dtype):
    l = torch.full((9, 12), -math.inf, dtype=dtype, device="cuda")
    for kw in (dict(), dict(mask=torch.zeros(9, dtype=torch.bool, device="cuda"))):
        x = l if not kw else torch.full_like(l, math.nan)
        ids, gates, stats = dq.route(x, 3, **kw)
        assert ids.eq(-1).all() and gates.eq(0).all()
        loss, coef, counts = dq.balance(stats, 3)
        assert loss.eq(0).all() and coef.eq(0).all() and counts.eq(0).all() and stats.fold().eq(0).all()
        d = dq.route_backward(x, ids, torch.full((9, 3), math.nan, device="cuda"), coef, **kw)
        assert d.eq(0).all()
    empty = torch.empty(0, 12, dtype=dtype, device="cuda")
    ids, gates, stats = dq.route(empty, 3)
    assert ids.shape == (0, 3) and stats.fold().eq(0).all()
    assert dq.route_backward(empty, ids).shape == (0, 12)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E", [5, 64, 300])
def test_route_nan_and_infinity(E, dtype):
    """NaN first (either sign), then +inf; the row's gates and its gradient are
    NaN, other rows are untouched, and the loss is NaN."""
    l = logits_of(6, E, dtype)
    l[1, 3] = math.nan
    l[2, E - 1] = -math.nan
    l[3, 2] = math.inf
    l[4, 4] = math.nan
    l[4, 1] = math.inf
    l[4, 0] = -math.inf
    ids, gates, stats = dq.route(l, 3)
    r = check_forward(l, 3, True, None, ids, gates)
    assert ids[4, 0] == 4 and ids[4, 1] == 1
    loss, coef, counts = dq.balance(stats, 3)
    assert np.array_equal(counts.cpu().numpy(), r.counts) and stats.fold()[2 * E] == 6
    assert loss.isnan().all()
    d = dq.route_backward(l, ids, torch.ones(6, 3, device="cuda"), torch.ones(E, device="cuda"))
    assert d[1:5].isnan().all() and not d[0].isnan().any() and not d[5].isnan().any()
    nan = torch.full((2, E), math.nan, dtype=dtype, device="cuda")
    ids, gates, _ = dq.route(nan, 2)
    assert ids.tolist() == [[0, 1], [0, 1]] and gates.isnan().all()


def test_route_extreme_logits():
    """Values near the ends of fp32, and rows that are all equal."""
    big = torch.finfo(torch.float32).max
    l = torch.tensor([[big, -big, 0.0, big], [-big, -big, -big, -big], [88.0, -88.0, 87.5, 0.0],
                      [-0.0, 0.0, -0.0, 0.0], [1e-40, -1e-40, 0.0, 1e-39]], device="cuda")
    ids, gates, stats = dq.route(l, 2)
    assert ids.tolist() == [[0, 3], [0, 1], [0, 2], [0, 1], [3, 0]]
    assert torch.equal(gates[0], torch.tensor([0.5, 0.5], device="cuda"))
    assert torch.equal(gates[1], torch.tensor([0.5, 0.5], device="cuda"))
    assert stats.fold()[8] == 5 and bool(torch.isfinite(stats.fold()).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E", [7, 64, 256])
def test_route_far_from_zero(E, dtype):
    """Rows of any size: the softmax depends on differences alone, which are
    exact for these logits (a few steps of the type around +-2^n).  Where the
    steps are large the probabilities are 0 and 1, ties share."""
    rng = np.random.default_rng(E)
    rows = []
    for n in (3, 10, 19, 20, 21, 24, 31, 33, 40, 60, 100, 120, 126):
        for sign in (1.0, -1.0):
            step = 2.0 ** n * torch.finfo(dtype).eps
            rows.append(sign * 2.0 ** n + step * rng.integers(0, 6, E))
    l = torch.from_numpy(np.array(rows)).to(dtype).cuda()
    assert bool((l.double().cpu() == torch.from_numpy(np.array(rows))).all())
    for renorm in (True, False):
        ids, gates, stats = dq.route(l, 3, renorm)
        x = l.double().cpu()
        assert torch.equal(ids.long().cpu(), torch.sort(x, dim=1, descending=True, stable=True)[1][:, :3])
        p = torch.softmax(x, 1)
        g = p.gather(1, ids.long().cpu())
        if renorm:
            g = g / g.sum(1, keepdim=True)
        # exponents: three roundings of differences that matter only below 104 (e^-104 is 0 in fp32)
        c = 2 * (3 * 104 + 48)
        assert bool(((gates.double().cpu() - g).abs() <= c * U * g + 1e-37).all())
        assert bool(((stats.fold()[E:2 * E].cpu() - p.sum(0)).abs() <= c * U * p.sum(0) + 1e-37).all())
        dg = randn((len(l), 3), torch.float32)
        d = dq.route_backward(l, ids, dg, renorm=renorm)
        assert bool(torch.isfinite(d).all())
        up = torch.zeros_like(x).scatter_(1, ids.long().cpu(), dg.double().cpu())
        if renorm:
            want = torch.zeros_like(x).scatter_(1, ids.long().cpu(), g * (dg.double().cpu() - (g * dg.double().cpu()).sum(1, keepdim=True)))
            mag = torch.zeros_like(x).scatter_(1, ids.long().cpu(), g * (dg.double().cpu().abs() + (g * dg.double().cpu().abs()).sum(1, keepdim=True)))
        else:
            want = p * (up - (p * up).sum(1, keepdim=True))
            mag = p * (up.abs() + (p * up.abs()).sum(1, keepdim=True))
        assert bool(((d.double().cpu() - want).abs() <= 2 * (c + 44) * U * mag + 1.01 * half_step(dtype) * want.abs() + 1e-37).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E", [1, 5, 64, 256])
def test_one_choice_has_gate_one_and_no_gradient(E, dtype):
    """A choice divided by itself is 1, and 1 has no gradient: exactly."""
    l = logits_of(300, E, dtype) * 7
    ids, gates, _ = dq.route(l, 1)
    assert bool((gates == 1).all())
    assert bool((dq.route_backward(l, ids, randn((300, 1), torch.float32)) == 0).all())
    if E > 1:
        l[:] = -math.inf
        l[:, E - 2] = 3.3
        ids, gates, _ = dq.route(l, 2 if E < 64 else 8)
        assert bool((gates[:, 0] == 1).all()) and bool((gates[:, 1:] == 0).all()) and bool((ids[:, 0] == E - 2).all())
        assert bool((dq.route_backward(l, ids, randn(gates.shape, torch.float32)) == 0).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,wide,at", [(64, 64, 0), (64, 128, 64), (64, 67, 1), (60, 64, 0), (256, 264, 8), (9, 10, 1)])
def test_route_strided_rows(E, wide, at, dtype):
    big = logits_of(150, wide, dtype)
    l = big[:, at:at + E]
    k = 4
    ids, gates, stats = dq.route(l, k)
    r = check_forward(l, k, True, None, ids, gates)
    i2, g2, s2 = dq.route(l.contiguous(), k)
    assert torch.equal(ids, i2)
    dg = randn((150, k), torch.float32)
    coef = dq.balance(stats, k)[1]
    d = dq.route_backward(l, ids, dg, coef)
    check_gradient(d, r, dg, coef, 1.0, dtype)
    out = torch.full((150, wide), 7.0, dtype=dtype, device="cuda")
    dq.route_backward(l, ids, dg, coef, out=out[:, at:at + E])
    assert same(out[:, at:at + E], d)
    out[:, at:at + E] = 7.0
    assert bool((out == 7.0).all())
    # in place, at this layout bit for bit; at another one sums run in another order
    again = big.clone()[:, at:at + E]
    assert same(dq.route_backward(again, ids, dg, coef, out=again), d)
    again = l.clone()
    check_gradient(dq.route_backward(again, ids, dg, coef, out=again), r, dg, coef, 1.0, dtype)
    row = l[:1].expand(70, E)                                          # all tokens alike
    i3 = dq.route(row, k)[0]
    assert torch.equal(i3, ids[:1].expand(70, k))


def check_gradient(d, r, dgates, coef, dloss, dtype):
    want, mag = ref.backward(r, None if dgates is None else dgates.double().cpu().numpy(),
                             None if coef is None else coef.double().cpu().numpy(), dloss)
    got = d.double().cpu().numpy()
    # beside the roundings of p and the gates: the sums of products (at most 40
    # deep) and four operations; bf16's own smallest step at 0
    tol = 2 * (r.roundings + 44) * U * mag + half_step(dtype) * np.abs(want) + 1e-37
    assert np.all(np.abs(got - want) <= tol * (1 + half_step(dtype)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,k", WIDTHS)
def test_route_backward_widths(E, k, dtype):
    for T, renorm in ((1, False), (67, True), (131, False)):
        l = logits_of(T, E, dtype, T, closed=0.2 if T > 1 else 0.0)
        mask = torch.arange(T, device="cuda") % 4 != 3
        ids, gates, stats = dq.route(l, k, renorm, mask)
        r = check_forward(l, k, renorm, mask, ids, gates)
        coef = dq.balance(stats, k)[1]
        dg = randn((T, k), torch.float32, E)
        dloss = torch.tensor([0.37], device="cuda")
        for kw in (dict(dgates=dg), dict(coef=coef), dict(dgates=dg, coef=coef, dloss=dloss), dict()):
            d = dq.route_backward(l, ids, renorm=renorm, mask=mask, **kw)
            check_gradient(d, r, kw.get("dgates"), kw.get("coef"), 0.37 if "dloss" in kw else 1.0, dtype)


def test_gradient_against_differences():
    """Directional derivatives of the GPU's own forward pass.  Central
    differences with h = 2^-7 are off by h^2/6 times the third derivative (at most
    a few times the scale of the direction, |v| <= 1: below 4e-4 of it) and by the
    outputs' roundings over 2 h (2^-24 x 64 x 400 gates / 2^-6: 2e-3 at most; they average)."""
    T, E, k = 40, 24, 3
    l = logits_of(T, E, torch.float32)
    w = randn((T, k), torch.float32, 5)
    x = l.clone().requires_grad_()
    r = train.route(x, k, renorm=True)
    g, = torch.autograd.grad((r.gates * w).sum() + 3 * r.loss, x)
    for seed in range(4):
        v = torch.rand(T, E, generator=torch.Generator().manual_seed(seed)).cuda() * 2 - 1
        h = 2.0 ** -7

        def value(sign):
            ids, gates, stats = dq.route(l + sign * h * v, k)
            # the same choices: the gates in the first call's order (ids may swap)
            full = torch.zeros(T, E, dtype=torch.float64)
            full.scatter_(1, ids.long().cpu(), gates.double().cpu())
            stay = torch.equal(ids.sort(1).values, r.ids.sort(1).values)
            s = stats.fold()
            s[:E] = r.counts.double()                                # counts have no derivative
            loss = (s[:E] * s[E:2 * E]).sum().item() * E / (k * s[2 * E].item() ** 2)
            return (full.gather(1, r.ids.long().cpu()) * w.double().cpu()).sum().item() + 3 * loss, stay

        (up, a), (down, b) = value(1), value(-1)
        if not (a and b):
            continue                                                 # a choice changed: no derivative there
        assert abs((up - down) / (2 * h) - (g * v).double().sum().item()) < 5e-3


@pytest.mark.parametrize("dtype", DTYPES)
def test_route_folds_workers_in_order(dtype):
    E, k = 48, 4
    ls = [logits_of(T, E, dtype, T) for T in (300, 1, 77, 0, 512)]
    stats, rs = None, []
    for l in ls:
        ids, gates, stats = dq.route(l, k, stats=stats)
        rs.append(check_forward(l, k, True, None, ids, gates) if len(l) else None)
    rs = [r for r in rs if r is not None]
    most = check_stats(stats, rs)
    loss, coef, counts = dq.balance(stats, k)
    wl, wc, wn, _ = ref.balance(rs)
    assert np.array_equal(counts.cpu().numpy(), wn)
    assert np.all(np.abs(coef.double().cpu().numpy() - wc) <= 2 * U * wc)
    assert abs(loss.item() - wl) <= (most + 4) * U * wl
    # the same in any grouping: folded in between, as a tensor, as the sum of
    # the statistics of several processes
    again = None
    for n, l in enumerate(ls):
        again = dq.route(l, k, stats=again)[2]
        if n % 2:
            again.fold()
    parts = [dq.route(l, k)[2].fold() for l in ls]
    total = sum(parts[1:], parts[0].clone())
    for s in (again, again.fold(), total):
        other = dq.balance(s, k)
        assert torch.equal(other[2], counts) and torch.equal(other[1], coef)
        assert abs(other[0].item() - wl) <= (most + 4) * U * wl
    # twice the same bits
    assert all(torch.equal(a, b) for a, b in zip(dq.balance(total, k), other))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,k", [(8, 2), (60, 4), (64, 8), (256, 8)])
def test_workers_in_one_launch_are_the_workers_one_by_one(E, k, dtype):
    """Bit for bit, with workers of different sizes, without tokens, with and
    without masks, and more of them than one launch takes."""
    sizes = [300, 0, 1, 77] + [40] * 15
    ls = [logits_of(T, E, dtype, T, closed=0.2 if T == 77 else 0.0) for T in sizes]
    masks = [torch.arange(T, device="cuda") % 4 != 1 if T == 300 else None for T in sizes]
    ids, gates, stats = dq.route(ls, k, mask=masks)
    one = None
    for l, m, i, g in zip(ls, masks, ids, gates):
        i1, g1, one = dq.route(l, k, mask=m, stats=one)
        assert torch.equal(i, i1) and torch.equal(g, g1)
    (loss, coef, counts), want = dq.balance(stats, k), dq.balance(one, k)
    assert torch.equal(counts, want[2]) and torch.equal(coef, want[1])
    assert abs(loss.item() - want[0].item()) <= 4 * U * want[0].item()     # (folded in other groups)
    dgs = [randn((T, k), torch.float32, T) if T != 77 else None for T in sizes]
    dloss = torch.tensor([0.4], device="cuda")
    ds = dq.route_backward(ls, ids, dgs, coef, dloss, mask=masks)
    for l, m, i, dg, d in zip(ls, masks, ids, dgs, ds):
        assert same(d, dq.route_backward(l, i, dg, coef, dloss, mask=m))
    outs = [torch.empty_like(l) for l in ls]
    again = dq.route_backward(ls, ids, dgs, coef, dloss, mask=masks, out=outs)
    assert all(a is o and same(a, d) for a, o, d in zip(again, outs, ds))
    held = [torch.empty_like(i) for i in ids], [torch.empty_like(g) for g in gates]
    got = dq.route(ls, k, mask=masks, ids=held[0], gates=held[1])
    assert all(a is b and torch.equal(a, c) for a, b, c in zip(got[0], held[0], ids))


def test_workers_of_different_alignment_in_one_launch():
    """One unaligned worker sends all of them element by element: choices stay,
    gates and gradients within the roundings."""
    E, k = 64, 8
    big = logits_of(90, E + 3, torch.bfloat16)
    ls = [logits_of(50, E, torch.bfloat16), big[:, 1:E + 1]]
    ids, gates, stats = dq.route(ls, k)
    rs = [check_forward(l, k, True, None, i, g) for l, i, g in zip(ls, ids, gates)]
    check_stats(stats, rs)
    coef = dq.balance(stats, k)[1]
    dgs = [randn(i.shape, torch.float32) for i in ids]
    for d, r, dg in zip(dq.route_backward(ls, ids, dgs, coef), rs, dgs):
        check_gradient(d, r, dg, coef, 1.0, torch.bfloat16)


@pytest.mark.parametrize("dtype", DTYPES)
def test_workers_in_columns_of_one_tensor(dtype):
    """Logits and gradients of the workers as interleaving windows, gradients in
    place and beside the logits: as from tensors of their own."""
    T, E, k = 75, 24, 3
    wide = logits_of(T, 4 * E, dtype)
    ls = [wide[:, :E], wide[:, E:2 * E]]
    ids, gates, stats = dq.route(ls, k)
    coef = dq.balance(stats, k)[1]
    dgs = [randn((T, k), torch.float32, w) for w in range(2)]
    want = dq.route_backward([l.clone() for l in ls], ids, dgs, coef)
    kept = wide.clone()
    outs = [wide[:, 3 * E:], wide[:, 2 * E:3 * E]]
    dq.route_backward(ls, ids, dgs, coef, out=outs)
    assert all(same(o, d) for o, d in zip(outs, want)) and same(wide[:, :2 * E], kept[:, :2 * E])
    dq.route_backward(ls, ids, dgs, coef, out=ls)
    assert all(same(o, d) for o, d in zip(ls, want)) and all(same(o, d) for o, d in zip(outs, want))
    x = kept[:, :E]
    y = dq.dropout(x, 0.4, residual=x, out=wide[:, E:2 * E], **KEY)
    assert same(y, expected_dropout(x, 0.4, x, **KEY).to(dtype)) and same(wide[:, :E], want[0])
    for bad in ([ls[1], outs[0]], [outs[0], outs[0]], [outs[0], wide[:, 2 * E + 1:3 * E + 1]]):
        with pytest.raises(dq.DQError):
            dq.route_backward(ls, ids, dgs, coef, out=bad)
    with pytest.raises(dq.DQError):
        dq.route(ls, k, ids=[ids[0], ids[0]])


def test_more_workers_than_one_fold_takes():
    E, k, n = 24, 2, 2 * dq.ROUTE_MAX_PARTS + 3
    ls = [logits_of(5 + w, E, torch.float32, w) for w in range(n)]
    stats = None
    for l in ls:
        stats = dq.route(l, k, stats=stats)[2]
    loss, coef, counts = dq.balance(stats, k)
    rs = [ref.Routed(l.double().cpu().numpy(), k) for l in ls]
    wl, wc, wn, N = ref.balance(rs)
    assert np.array_equal(counts.cpu().numpy(), wn)
    assert abs(loss.item() - wl) <= (max(r.roundings + len(r.l) for r in rs) + 4) * U * wl
    assert stats.fold()[2 * E] == N


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,k", [(4099, 60, 4), (20000, 8, 2), (33000, 64, 8), (9000, 256, 8)])
def test_route_many_tokens_and_the_same_bits_again(T, E, k, dtype):
    """Beyond one pass of the grid, against torch in fp64 on the CPU."""
    l = logits_of(T, E, dtype)
    ids, gates, stats = dq.route(l, k, False)
    x = l.double().cpu()
    order = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :k]
    p = torch.softmax(x, 1)
    assert torch.equal(ids.long().cpu(), order)
    span = (x.max() - x.min()).item()
    c = 2 * (3 * span + 48)
    want = p.gather(1, order)
    assert bool(((gates.double().cpu() - want).abs() <= c * U * want).all())
    s = stats.fold().cpu()
    assert torch.equal(s[:E], torch.bincount(order.reshape(-1), minlength=E).double()) and s[2 * E] == T
    assert bool(((s[E:2 * E] - p.sum(0)).abs() <= (c + T) * U * p.sum(0)).all())
    again = dq.route(l, k, False)
    assert torch.equal(ids, again[0]) and torch.equal(gates, again[1])
    assert torch.equal(stats.fold(), again[2].fold())
    coef = dq.balance(stats, k)[1]
    dg = randn((T, k), torch.float32)
    d = dq.route_backward(l, ids, dg, coef, renorm=False)
    assert same(d, dq.route_backward(l, ids, dg, coef, renorm=False))
    up = coef.double().cpu().expand(T, E).clone().scatter_add_(1, order, dg.double().cpu())
    want = p * (up - (p * up).sum(1, keepdim=True))
    mag = p * (up.abs() + (p * up.abs()).sum(1, keepdim=True))
    err = (d.double().cpu() - want).abs()
    assert bool((err <= 2 * (c + 44) * U * mag + half_step(dtype) * want.abs() * 1.01 + 1e-37).all())


def test_route_sums_of_very_many_tokens():
    """2^31 tokens that are all alike (one row, stride 0): every addition to an fp32
    sum rounds the same way, so only few may go into one."""
    T, E = 1 << 31, 7
    row = torch.zeros(1, E, dtype=torch.bfloat16, device="cuda")
    print("[route] 2^31 tokens", flush=True)
    ids, gates, stats = dq.route(row.expand(T, E), 1)
    assert bool((ids == 0).all()) and bool((gates == 1).all())
    s = stats.fold().cpu()
    assert s[0] == T and s[2 * E] == T and s[1:E].eq(0).all()
    # roundings of p as everywhere (no span), 64 additions in a lane, 40 between lanes
    assert bool(((s[E:2 * E] - T / E).abs() <= (2 * 48 + 64 + 40) * U * T / E).all())


def routed_in_fp64(l, k, renorm, mask):
    """(ids, gates, p) by torch in fp64: stable sorting keeps equal logits (-0 = +0)
    by index and has NaN first."""
    x = l.double()
    ok = ~(x == -math.inf).all(1)
    ok = ok if mask is None else ok & mask
    v, order = torch.sort(x, dim=1, descending=True, stable=True)
    ids = torch.where(ok[:, None] & (v[:, :k] != -math.inf), order[:, :k], -1)
    p = torch.where(ok[:, None], torch.softmax(x, 1), 0.0)
    g = torch.where(ids >= 0, p.gather(1, ids.clamp(min=0)), 0.0)
    return ids, torch.where(ids >= 0, g / g.sum(1, keepdim=True), 0.0) if renorm else g, p


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("E,sizes", [(136, [12000, 4500, 33]), (256, [40001]), (256, [12000, 0, 4500, 33]),
                                     (384, [16500]), (512, [12000, 4500, 33]), (513, [16400]), (1000, [16400]),
                                     (1024, [12000, 4500, 33])])
def test_route_many_tokens_of_many_experts(E, sizes, odd):
    """bf16 beyond 16384 tokens a call and 128 experts, where lists grow longer: every
    number of choices, masks, closed experts, ties, zeros of both signs; with odd,
    rows of NaN and +inf too (their probabilities, NaN, go into no sum here)."""
    ls, masks = [], []
    for n, T in enumerate(sizes):
        l = logits_of(T, E, torch.float32, n + 1)
        l[::3] = l[::3].round()                                       # ties, zeros of both signs among them
        l[1::7] = torch.where(l[1::7] > 0.5, -0.0, 0.0)               # only zeros
        l[2::5] = torch.where(torch.randn(l[2::5].shape, generator=torch.Generator("cuda").manual_seed(n), device="cuda")
                              < 0.3, -math.inf, l[2::5])
        l[4::11] = -math.inf
        if T > 20:
            l[15, E // 2 + 1:] = -math.inf
            l[15, :E // 2] = -math.inf                                # one open expert
        if odd:
            l[3::13, E // 3] = math.nan
            l[5::17, E - 1] = math.inf
        ls.append(l.bfloat16())
        masks.append(None if n == 1 else torch.arange(T, device="cuda") % 9 != 4)
    finite = [l[l.isfinite()].double() for l in ls if len(l)]
    c = 2 * (3 * max((f.max() - f.min()).item() for f in finite) + 48)
    for k in (1, 2, 3, 4, 8, 9, 16):
        renorm = k % 2 == 0
        ids, gates, stats = dq.route(ls, k, renorm, masks)
        count, psum, tokens = torch.zeros(E, device="cuda"), torch.zeros(E, dtype=torch.float64, device="cuda"), 0
        for l, m, i, g in zip(ls, masks, ids, gates):
            wi, wg, p = routed_in_fp64(l, k, renorm, m)
            assert torch.equal(i.long(), wi)
            assert torch.equal(g.isnan(), wg.isnan())
            assert bool(((g.double() - wg).abs() <= c * U * wg + 1e-37)[~wg.isnan()].all())
            count += torch.bincount(wi.reshape(-1) + 1, minlength=E + 1)[1:]
            psum += p.sum(0)
            tokens += int((wi[:, 0] >= 0).sum())
        s = stats.fold()
        assert torch.equal(s[:E], count.double()) and s[2 * E] == tokens
        if not odd:
            assert bool(((s[E:2 * E] - psum).abs() <= (c + max(sizes)) * U * psum + 1e-37).all())


@pytest.mark.parametrize("E", [250, 1000])
@pytest.mark.parametrize("sizes", [[9000, 3001], [9000, 3001, 0, 1], [2000, 1] * 8])
def test_balance_of_many_rows_of_several_parts(sizes, E):
    """Parts of unequal size, more rows than one block folds; alone, after earlier
    sums, and with the sums overwritten by the result (the C call allows it)."""
    k = 4
    ls = [logits_of(T, E, torch.bfloat16, n + 1) for n, T in enumerate(sizes)]
    outs = [dq.route(l, k)[2] for l in ls]
    parts = (dq.dq_route_part * len(ls))(*[(o.parts[0][1], T) for o, T in zip(outs, sizes)])
    want = torch.zeros(2 * E + 1, dtype=torch.float64, device="cuda")
    span = 0.0
    for l in ls:
        ids, _, p = routed_in_fp64(l, k, True, None)
        want[:E] += torch.bincount(ids.reshape(-1), minlength=E)
        want[E:2 * E] += p.sum(0)
        want[2 * E] += len(l)
        span = max(span, (l.double().max() - l.double().min()).item() if len(l) else 0.0)
    most = 2 * (3 * span + 48) + max(sizes)
    before = dq.route(logits_of(70, E, torch.bfloat16, 99), k)[2].fold()
    for sums in (None, before, before.clone()):
        stats = sums if sums is not None and sums is not before else torch.empty_like(want)
        total = want if sums is None else want + before
        n = total[2 * E].item()
        loss, coef = torch.empty(1, device="cuda"), torch.empty(E, device="cuda")
        counts = torch.empty(E, dtype=torch.int64, device="cuda")
        rc = dq.lib().dq_balance(parts, len(ls), None if sums is None else sums.data_ptr(), E, k, stats.data_ptr(),
                                 loss.data_ptr(), coef.data_ptr(), counts.data_ptr(),
                                 torch.cuda.current_stream().cuda_stream)
        assert rc == dq.DQ_OK
        assert torch.equal(stats[:E], total[:E]) and stats[2 * E] == n and torch.equal(counts, total[:E].long())
        assert bool(((stats[E:2 * E] - total[E:2 * E]).abs() <= most * U * total[E:2 * E]).all())
        wc = E * total[:E] / (k * n * n)
        assert bool(((coef.double() - wc).abs() <= 2 * U * wc).all())
        wl = (wc * total[E:2 * E]).sum().item()
        assert abs(loss.item() - wl) <= (most + 4) * U * wl


def test_route_loss_of_many_tokens():
    """fp32 sums stay short: 2^20 tokens, loss against fp64."""
    T, E, k = 1 << 20, 16, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    l = torch.randn(T, E, generator=g, device="cuda")
    _, _, stats = dq.route(l, k)
    p = torch.softmax(l.double(), 1).sum(0)
    assert bool(((stats.fold()[E:2 * E] - p).abs() <= 1e-6 * p).all())


def test_route_refuses():
    l = torch.zeros(8, 16, device="cuda")
    ids, gates, stats = dq.route(l, 2)
    for call in (lambda: dq.route(l[0], 2), lambda: dq.route(l.t(), 2), lambda: dq.route(l, 2, mask=torch.zeros(7, dtype=torch.bool, device="cuda")),
                 lambda: dq.route(l, 2, mask=torch.zeros(8, dtype=torch.bool)),
                 lambda: dq.route(l[:, :15], 2, stats=stats), lambda: dq.balance(stats.fold()[:-1], 2),
                 lambda: dq.route(l, 2, ids=ids[:, :1]), lambda: dq.route(l, 2, gates=gates.t()),
                 lambda: dq.route_backward(l, ids[:4]), lambda: dq.route_backward(l, ids, gates[:4]),
                 lambda: dq.route_backward(l, ids, coef=stats.fold()[:15].float()),
                 lambda: dq.route_backward(l, ids, out=l.bfloat16()),
                 lambda: dq.route_backward(l, ids, out=l[:4])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: dq.route(l, 2, mask=torch.zeros(8, device="cuda")), lambda: dq.route(l, 2, ids=ids.long()),
                 lambda: dq.route(l, 2, stats=stats.fold()), lambda: dq.balance(stats.fold().float(), 2), lambda: dq.route_backward(l, ids.long()),
                 lambda: dq.route_backward(l, ids, coef=torch.zeros(16, dtype=torch.float64, device="cuda"))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: dq.route(l, 0), lambda: dq.route([l, l[:, :8]], 2), lambda: dq.route([l, l.bfloat16()], 2),
                 lambda: dq.route([l, l], 2, mask=[None]), lambda: dq.route([l, l], 2, ids=[ids]),
                 lambda: dq.route_backward([l, l], [ids]), lambda: dq.route_backward([l, l], [ids, ids], [gates]),
                 lambda: dq.route_backward([l, l], [ids, ids], out=[l])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: dq.route(l, 17), lambda: dq.balance(stats, 17),
                 lambda: dq.route(torch.zeros(2, 1025, device="cuda"), 2),
                 lambda: dq.route(torch.zeros(2, 64, device="cuda"), 17),
                 lambda: dq.route_backward(l[1:], ids[1:], out=l[:-1])):
        with pytest.raises(dq.DQError):
            call()


def test_ids_out_of_range_are_no_choice():
    """The gradient does not index beyond the experts whatever ids hold."""
    E = 20
    l = logits_of(3, E, torch.float32)
    ids = torch.tensor([[1, E], [-7, 2 ** 31 - 1], [-2 ** 31, 4]], dtype=torch.int32, device="cuda")
    dg = torch.ones(3, 2, device="cuda")
    a = dq.route_backward(l, ids, dg, renorm=False)
    b = dq.route_backward(l, torch.where((ids >= 0) & (ids < E), ids, -1), dg, renorm=False)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,wide,k", [(12, 13, 3), (64, 64, 8), (256, 256, 8), (1000, 1000, 16)])
def test_left_out_tokens_get_zeros_whatever_the_loss_is(E, wide, k, dtype):
    """A loss scale that overflowed, or a bad coefficient, reaches routed tokens
    only."""
    T = 45
    l = logits_of(T, wide, dtype)[:, :E]
    l[::7] = -math.inf
    mask = torch.arange(T, device="cuda") % 3 != 1
    left = ~mask | (torch.arange(T, device="cuda") % 7 == 0)
    l[1] = math.nan
    for renorm in (True, False):
        ids, gates, stats = dq.route(l, k, renorm, mask)
        coef = dq.balance(stats, k)[1]
        dg = randn((T, k), torch.float32)
        for bad in (math.inf, -math.inf, math.nan):
            broken = coef.clone()
            broken[E // 2] = bad
            for kw in (dict(coef=coef, dloss=torch.full((1,), bad, device="cuda")), dict(coef=broken)):
                d = dq.route_backward(l, ids, dg, renorm=renorm, mask=mask, **kw)
                assert bool((d[left] == 0).all()) and bool(d[~left].isnan().any(1).all())

# ---- autograd, streams, graphs -----------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
def test_route_autograd(dtype):
    E, k = 40, 4
    ls = [logits_of(T, E, dtype, T).requires_grad_() for T in (50, 33)]
    masks = [None, torch.arange(33, device="cuda") % 5 != 0]
    dgs = [randn((50, k), torch.float32), randn((33, k), torch.float32, 1)]
    dloss = torch.tensor([0.21], device="cuda")
    r = train.route(ls, k, masks=masks)
    rs = [check_forward(l.detach(), k, True, m, i, g.detach()) for l, m, i, g in zip(ls, masks, r.ids, r.gates)]
    grads = torch.autograd.grad([*r.gates, r.loss], ls, [*dgs, dloss], retain_graph=True)
    for g, rr, dg in zip(grads, rs, dgs):
        check_gradient(g, rr, dg, r.coef, 0.21, dtype)
    # the loss alone, one worker's gates alone
    for g, rr in zip(torch.autograd.grad(r.loss, ls, retain_graph=True), rs):
        check_gradient(g, rr, None, r.coef, 1.0, dtype)
    g = torch.autograd.grad(r.gates[1].sum(), ls, retain_graph=True, allow_unused=True)
    assert g[0] is None
    check_gradient(g[1], rs[1], torch.ones(33, k), None, 1.0, dtype)
    assert not r.ids[0].requires_grad and not r.counts.requires_grad and not r.coef.requires_grad
    # one tensor, no list; a transposed one is copied
    one = train.route(ls[0].detach().t().contiguous().t().requires_grad_(), k)
    assert torch.equal(one.ids, r.ids[0])
    one.loss.backward()


def test_results_of_a_list_are_tensors_of_their_own():
    """Changing one worker's gates or gradient in place touches no other's."""
    ls = [logits_of(T, 24, torch.float32, T).requires_grad_() for T in (20, 30)]
    r = train.route(ls, 2)
    kept = r.gates[1].detach().clone()
    r.gates[0].mul_(2)
    assert torch.equal(r.gates[1], kept)
    (r.gates[0].sum() + r.gates[1].square().sum() + r.loss).backward()
    other = ls[1].grad.clone()
    ls[0].grad.zero_()
    assert torch.equal(ls[1].grad, other)


def test_balance_on_another_stream_than_the_parts():
    l = logits_of(3000, 64, torch.bfloat16)
    want = dq.balance(dq.route(l, 8)[2], 8)
    s = torch.cuda.Stream()
    for _ in range(20):
        stats = dq.route(l, 8)[2]
        s.wait_stream(torch.cuda.current_stream())
        got = dq.balance(stats, 8, stream=s)
        del stats                                  # its parts may be taken by what comes next here
        torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda")
        dq.route(l * 0, 8)
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_statistics_that_were_handed_out_keep_their_values():
    """A fold gives a tensor of its own: later tokens, the fold that a 17th part
    makes, and later folds leave it alone."""
    l = logits_of(500, 40, torch.float32)
    stats = dq.route(l, 4)[2]
    first = stats.fold()
    kept = first.clone()
    for _ in range(dq.ROUTE_MAX_PARTS + 1):
        dq.route(l, 4, stats=stats)
    second = stats.fold()
    assert torch.equal(first, kept) and second[80] == (dq.ROUTE_MAX_PARTS + 2) * 500
    assert stats.fold() is second                  # nothing new
    second.mul_(2)                                 # the latest one is the statistics
    assert torch.equal(dq.balance(stats, 4)[2], second[:40].long())


@pytest.mark.parametrize("form", ["stats", "tensor"])
@pytest.mark.parametrize("workers", [1, dq.ROUTE_MAX_PARTS + 2])
def test_balance_on_another_stream_than_the_fold(workers, form):
    """Folded statistics (the tensor, too) may be dropped right after another
    stream was given them."""
    E = 1000
    ls = [logits_of(300, E, torch.bfloat16, w) for w in range(workers)]
    want = dq.balance(dq.route(ls, 8)[2].fold(), 8)
    s = torch.cuda.Stream()
    for rep in range(20):
        stats = dq.route(ls, 8)[2]
        if rep % 2 or form == "tensor" or workers == 1:
            stats.fold()
        s.wait_stream(torch.cuda.current_stream())
        got = dq.balance(stats if form == "stats" else stats.fold(), 8, stream=s)
        del stats
        for _ in range(8):                             # the sums' memory, if it is free here
            torch.full((2 * E + 1,), 7.0, dtype=torch.float64, device="cuda")
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got[2], want[2]) and torch.equal(got[1], want[1])
        assert abs(got[0].item() - want[0].item()) <= 4 * U * want[0].item()


def test_two_forwards_before_their_backwards():
    """Nothing is shared between calls: gradients do not depend on what ran in
    between."""
    a, b = (logits_of(T, 24, torch.float32, T).requires_grad_() for T in (64, 96))
    want = [torch.autograd.grad(train.route(x, 2).loss, x)[0] for x in (a, b)]
    ra, rb = train.route(a, 2), train.route(b, 2)
    ga, gb = torch.autograd.grad(ra.loss, a)[0], torch.autograd.grad(rb.loss, b)[0]
    assert torch.equal(ga, want[0]) and torch.equal(gb, want[1])


def test_reduce_sees_the_statistics():
    l = logits_of(30, 12, torch.float32).requires_grad_()
    doubled = train.route(l, 2, reduce=lambda s: s.mul_(2))              # as if a second rank had the same
    alone = train.route(l, 2)
    assert torch.equal(doubled.counts, 2 * alone.counts)
    assert abs(doubled.loss.item() - alone.loss.item()) <= 4 * U * alone.loss.item()


def _routing_of_rank(rank, port, path):
    """One of two processes, each with its own worker's tokens."""
    import torch.distributed as dist
    dist.init_process_group("gloo", init_method=f"tcp://127.0.0.1:{port}", rank=rank, world_size=2)

    def reduce(stats):
        host = stats.cpu()                           # gloo works on host tensors
        dist.all_reduce(host)
        stats.copy_(host)

    l = logits_of((300, 77)[rank], 64, torch.bfloat16, rank).requires_grad_()
    r = train.route(l, 4, reduce=reduce)
    dl, = torch.autograd.grad(r.loss, l)
    torch.save([t.detach().cpu() for t in (r.ids, r.gates, r.loss, r.coef, r.counts, dl)], f"{path}{rank}")
    dist.destroy_process_group()


def test_reduce_over_two_processes(tmp_path):
    """The balance loss of two processes' workers is the one that a process with both
    computes, and so is each one's part of the gradient."""
    import socket
    import torch.multiprocessing as mp
    ls = [logits_of(T, 64, torch.bfloat16, n).requires_grad_() for n, T in enumerate((300, 77))]
    r = train.route(ls, 4)
    dls = torch.autograd.grad(r.loss, ls)
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    mp.spawn(_routing_of_rank, args=(port, str(tmp_path / "r")), nprocs=2, join=True)
    for rank in range(2):
        ids, gates, loss, coef, counts, dl = torch.load(tmp_path / f"r{rank}", weights_only=True)
        assert torch.equal(ids, r.ids[rank].cpu()) and torch.equal(gates, r.gates[rank].detach().cpu())
        assert torch.equal(counts, r.counts.cpu()) and torch.equal(coef, r.coef.cpu())
        assert abs(loss.item() - r.loss.item()) <= 4 * U * r.loss.item()
        assert same(dl, dls[rank])


def test_route_on_another_stream():
    l = logits_of(5000, 64, torch.bfloat16)
    want = dq.route(l, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dq.route(l, 8, stream=s)
    loss = dq.balance(got[2], 8, stream=s)
    d = dq.route_backward(l, got[0], coef=loss[1], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want[:2], got[:2]))
    want_loss = dq.balance(want[2], 8)
    assert all(torch.equal(a, b) for a, b in zip(want_loss, loss))
    assert same(d, dq.route_backward(l, want[0], coef=want_loss[1]))


def test_step_in_graph_replays():
    """Forward and backward of the router and of dropout with the round on the
    device, captured while an eager graph of the same leaf lives, replayed with
    new inputs and rounds between eager work."""
    T, E, k, H = 700, 64, 4, 96
    l, x = logits_of(T, E, torch.bfloat16), randn((T, H), torch.bfloat16)
    res, dg = randn((T, H), torch.bfloat16, 1), randn((T, k), torch.float32, 2)
    rnd = torch.zeros(1, dtype=torch.int32, device="cuda")
    dloss = torch.full((1,), 0.01, device="cuda")
    leaf = l.requires_grad_()
    alive = train.route(leaf, k)                                       # an eager graph of the leaf

    def step(out=None):
        ids, gates, stats = dq.route(l.detach(), k)
        loss, coef, counts = dq.balance(stats, k)
        y = dq.dropout(x, 0.1, residual=res, rnd=rnd, worker=1)
        d = dq.route_backward(l.detach(), ids, dg, coef, dloss)
        dx = dq.dropout_backward(y, 0.1, rnd=rnd, worker=1)
        return ids, gates, stats.fold(), loss, coef, counts, y, d, dx

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    torch.cuda.synchronize()
    for rep in range(4):
        with torch.no_grad():
            l.copy_(logits_of(T, E, torch.bfloat16, 10 + rep))
        rnd.fill_(rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b), rep
    assert alive.loss.item() > 0


# ---- together ------------------------------------------------------------------------

def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_step.py")
    spec = importlib.util.spec_from_file_location("moe_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_moe_example_learns_with_compressed_gradients():
    """Router, dropout and gradient round in one data-parallel step: the loss
    falls well below chance (ln 16 = 2.77) and tokens stay spread."""
    moe = _example()
    t = moe.Trainer(workers=4, tokens=256)
    first = t.step(0)
    for step in range(1, 60):
        last = t.step(step)
    assert first[0] > 2.0 and last[0] < 0.5 * first[0]
    assert all(c.sum().item() == 4 * 256 * moe.TOP_K for c in last[2])
    assert last[1] < 2.0


def test_moe_example_step_against_fp32_gradients():
    """The same step with its gradients summed in fp32: the forward pass is the
    same (up to the order of library sums), the compressed update differs by
    the round's quantisation only."""
    moe = _example()
    a, b = moe.Trainer(workers=2, tokens=64), moe.Trainer(workers=2, tokens=64, exact=True)
    ra, rb = a.step(0), b.step(0)
    assert abs(ra[0] - rb[0]) < 1e-5 and abs(ra[1] - rb[1]) < 1e-5
    start = moe.init()
    da = torch.cat([(w - start[k]).reshape(-1) for k, w in a.weights.items()]).double()
    db = torch.cat([(w - start[k]).reshape(-1) for k, w in b.weights.items()]).double()
    assert ((da - db).norm() / db.norm()).item() < 0.2
