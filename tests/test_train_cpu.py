"""Training-step operators without a GPU: the plain forms that the GPU tests
compare with (dithers against the oracle's Philox, gradients against
differences), and the argument checks of the C ABI and the binding."""
import ctypes as C
import re

import numpy as np
import pytest
import torch

import train_ref as ref
from compressed_hop_gradient_amd import dq, train


@pytest.fixture(scope="module")
def lib():
    return dq.lib()


# ---- the plain forms -----------------------------------------------------------

@pytest.mark.parametrize("block,seed,rnd,worker,site", [
    (0, 1, 0, 0, 0), (5, 0x123456789ABCDEF0, 7, 3, 2), ((1 << 32) + 9, 2 ** 64 - 1, 2 ** 32 - 1, 65535, 2 ** 31 - 1)])
def test_dithers_are_the_oracles_philox(block, seed, rnd, worker, site):
    got = ref.dithers(24, seed, rnd, worker, site, first=8 * block)
    for i in range(3):
        assert list(got[8 * i:8 * i + 8]) == ref.dithers_by_oracle(block + i, seed, rnd, worker, site)


def test_dithers_are_uniform_and_differ_by_worker_round_and_site():
    n = 1 << 16
    base = ref.dithers(n, 1, 0, 0, 0)
    # each of 16 ranges holds n / 16 of them, within 6 standard deviations
    h = np.bincount(base >> 12, minlength=16)
    assert np.all(np.abs(h - n / 16) < 6 * np.sqrt(n / 16))
    for other in (ref.dithers(n, 2, 0, 0, 0), ref.dithers(n, 1, 1, 0, 0), ref.dithers(n, 1, 0, 1, 0),
                  ref.dithers(n, 1, 0, 0, 1)):
        assert (other == base).mean() < 0.001
        assert abs(np.corrcoef(other, base)[0, 1]) < 6 / np.sqrt(n)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(5, 1), (9, 3), (16, 16)])
def test_reference_gradient_against_differences(E, k, renorm):
    """d/dl of sum_w (gates . dg) + dloss * loss, the choices held fixed (they
    change only where logits tie)."""
    rng = np.random.default_rng(E)
    ls = [rng.normal(size=(7, E)), rng.normal(size=(4, E))]
    if E > k + 1:
        ls[0][2, 1] = -np.inf
    ls[0][3] = -np.inf
    masks = [np.array([1, 1, 1, 1, 1, 0, 1]), None]
    dgs = [rng.normal(size=(len(l), k)) for l in ls]
    dloss = 0.7

    def value(x):
        rs = [ref.Routed(l, k, renorm, m) for l, m in zip(x, masks)]
        return sum((r.gates * np.where(r.ids >= 0, d, 0)).sum() for r, d in zip(rs, dgs)) + dloss * ref.balance(rs)[0]

    rs = [ref.Routed(l, k, renorm, m) for l, m in zip(ls, masks)]
    coef = ref.balance(rs)[1]
    h = 1e-5
    for w in range(2):
        g, _ = ref.backward(rs[w], dgs[w], coef, dloss)
        for t in range(len(ls[w])):
            for j in range(E):
                if not np.isfinite(ls[w][t, j]):
                    assert g[t, j] == 0
                    continue
                up, down = [l.copy() for l in ls], [l.copy() for l in ls]
                up[w][t, j] += h
                down[w][t, j] -= h
                # central differences: h^2 f''' / 6 and 2^-53 / h, both below 1e-9 here
                assert abs((value(up) - value(down)) / (2 * h) - g[t, j]) < 1e-8


def test_balance_is_one_when_balanced():
    l = np.full((8, 4), -20.0)
    l[np.arange(8), np.arange(8) % 4] = 20.0
    assert abs(ref.balance([ref.Routed(l, 1)])[0] - 1.0) < 1e-12
    l[:] = -20.0
    l[:, 0] = 20.0
    assert abs(ref.balance([ref.Routed(l, 1)])[0] - 4.0) < 1e-12      # all on one of four


# ---- the built kernels -----------------------------------------------------------

def test_no_kernel_uses_scratch_memory(lib):
    """By the kernels' metadata in the library (its values below 128 are one byte)."""
    with open(dq.LIB_PATH, "rb") as f:
        image = f.read()
    for key in (rb"private_segment_fixed_size", rb"vgpr_spill_count"):
        found = re.findall(rb"\." + key + rb"(.)", image, re.S)
        assert len(found) > 200 and set(found) == {b"\0"}


# ---- refusals of the C ABI -------------------------------------------------------

FAKE = 1 << 20      # never read: every call below fails its checks, or has nothing to do


def _dropout(lib, x=FAKE, res=None, y=4 * FAKE, kind=dq.BF16, rows=4, cols=64, xs=64, rs=64, ys=64, p=0.1, seed=1,
             rnd=0, d_round=None, worker=0, site=0):
    return lib.dq_dropout(x, res, y, kind, rows, cols, xs, rs, ys, p, seed, rnd, d_round, worker, site, None)


@pytest.mark.parametrize("bad", [
    dict(kind=dq.PACKED), dict(kind=-1), dict(rows=-1), dict(cols=-1), dict(p=-0.1), dict(p=1.1),
    dict(p=float("nan")), dict(worker=-1), dict(worker=65536), dict(site=1 << 31), dict(rows=1 << 40, cols=1 << 40),
    dict(rows=1 << 26, cols=1 << 25), dict(xs=-1), dict(rs=-1), dict(ys=63), dict(ys=0), dict(xs=1 << 51),
    dict(x=FAKE + 1), dict(y=4 * FAKE + 1), dict(res=FAKE + 1), dict(d_round=FAKE + 2),
    dict(kind=dq.F32, x=FAKE + 2),
    # outputs that meet an operand other than element on element
    dict(y=FAKE + 2), dict(y=FAKE + 128), dict(y=FAKE, xs=128), dict(y=FAKE + 2, rows=1), dict(res=4 * FAKE + 16),
    dict(y=FAKE + 126, xs=127, ys=127), dict(xs=0, x=4 * FAKE + 64)])
def test_dropout_refuses(lib, bad):
    assert _dropout(lib, **bad) == dq.DQ_EINVAL


def test_dropout_null_and_empty(lib):
    assert _dropout(lib, x=None) == dq.DQ_ENULL
    assert _dropout(lib, y=None) == dq.DQ_ENULL
    assert _dropout(lib, rows=0) == dq.DQ_OK
    assert _dropout(lib, cols=0, x=None, y=None, ys=0) == dq.DQ_OK


def _route(lib, l=FAKE, kind=dq.BF16, T=8, E=16, stride=16, mask=None, k=2, flags=1, ids=4 * FAKE, gates=5 * FAKE,
           part=7 * FAKE, nbytes=1 << 20, n=1):
    """One call; with n = 2 a worker of no tokens and nothing wrong comes first
    (the bad one must be found before anything is launched)."""
    io = (dq.dq_route_worker * 2)((None, 0, 0, None, None, None, 9 * FAKE, 1 << 20),
                                  (l, T, stride, mask, ids, gates, part, nbytes))
    at = C.byref(io, C.sizeof(dq.dq_route_worker)) if n == 1 else io
    return lib.dq_route(at, n, kind, E, k, flags, None)


@pytest.mark.parametrize("bad", [
    dict(kind=dq.PACKED), dict(T=-1), dict(T=(1 << 40) + 1), dict(E=0), dict(E=1025), dict(stride=-1), dict(k=0),
    dict(k=17, E=32), dict(k=3, E=2), dict(flags=4), dict(l=FAKE + 1), dict(kind=dq.F32, l=FAKE + 2),
    dict(ids=4 * FAKE + 2), dict(gates=5 * FAKE + 2)])
def test_route_refuses(lib, bad):
    assert _route(lib, **bad) == dq.DQ_EINVAL
    assert _route(lib, n=2, **bad) == dq.DQ_EINVAL


def test_route_worker_counts(lib):
    io = (dq.dq_route_worker * 17)()
    assert lib.dq_route(io, 17, dq.BF16, 16, 2, 1, None) == dq.DQ_EWORKSPACE                       # no part
    assert lib.dq_route(io, -1, dq.BF16, 16, 2, 1, None) == dq.DQ_EINVAL
    assert lib.dq_route(None, 1, dq.BF16, 16, 2, 1, None) == dq.DQ_ENULL
    assert lib.dq_route(None, 0, dq.BF16, 16, 2, 1, None) == dq.DQ_OK
    io = (dq.dq_route_grad * 17)()
    assert lib.dq_route_backward(io, 17, dq.BF16, 16, 2, 1, None, None, None) == dq.DQ_OK          # no tokens
    assert lib.dq_route_backward(io, -1, dq.BF16, 16, 2, 1, None, None, None) == dq.DQ_EINVAL
    assert lib.dq_route_backward(None, 1, dq.BF16, 16, 2, 1, None, None, None) == dq.DQ_ENULL
    assert lib.dq_route_backward(None, 0, dq.BF16, 16, 2, 1, None, None, None) == dq.DQ_OK


def test_route_null_and_part(lib):
    for name in ("l", "ids", "gates"):
        assert _route(lib, **{name: None}) == dq.DQ_ENULL
    need = lib.dq_route_part_bytes(8, 16)
    assert need > 0
    assert _route(lib, nbytes=need - 1) == dq.DQ_EWORKSPACE
    assert _route(lib, part=None) == dq.DQ_EWORKSPACE
    assert _route(lib, part=7 * FAKE + 128) == dq.DQ_EWORKSPACE
    for args in ((-1, 16), (8, 0), (8, 1025), ((1 << 40) + 1, 16)):
        assert lib.dq_route_part_bytes(*args) == 0
    # bounded however many tokens there are
    for E in (1, 8, 64, 256, 1024):
        assert lib.dq_route_part_bytes(0, E) > 0
        assert lib.dq_route_part_bytes(1 << 40, E) < 64 << 20


def _balance(lib, parts=((7 * FAKE, 8),), n=None, sums=None, E=16, k=2, stats=FAKE, loss=2 * FAKE, coef=3 * FAKE,
             counts=4 * FAKE):
    array = None if parts is None else (dq.dq_route_part * max(1, len(parts)))(*parts)
    return lib.dq_balance(array, len(parts or ()) if n is None else n, sums, E, k, stats, loss, coef, counts, None)


def test_balance_refuses(lib):
    for bad in (dict(E=0), dict(E=1025), dict(k=0), dict(k=17, E=32), dict(k=17), dict(n=-1), dict(n=17),
                dict(sums=FAKE + 4), dict(stats=FAKE + 4), dict(loss=FAKE + 2), dict(coef=FAKE + 2),
                dict(counts=FAKE + 4), dict(parts=((7 * FAKE, -1),)), dict(parts=((7 * FAKE + 128, 8),)),
                dict(parts=((7 * FAKE, (1 << 40) + 1),))):
        assert _balance(lib, **bad) == dq.DQ_EINVAL, bad
    for bad in (dict(parts=None, n=1), dict(parts=()), dict(parts=((None, 8),))):
        assert _balance(lib, **bad) == dq.DQ_ENULL, bad


def _backward(lib, l=FAKE, kind=dq.BF16, T=8, E=16, stride=16, mask=None, k=2, flags=1, ids=4 * FAKE, dg=5 * FAKE,
              coef=6 * FAKE, dloss=7 * FAKE, out=8 * FAKE, dstride=16):
    io = (dq.dq_route_grad * 2)((None, 0, 0, None, None, None, None, 0),
                                (l, T, stride, mask, ids, dg, out, dstride))
    return lib.dq_route_backward(io, 2, kind, E, k, flags, coef, dloss, None)


@pytest.mark.parametrize("bad", [
    dict(kind=7), dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=17, E=32), dict(flags=2), dict(dstride=15),
    dict(l=FAKE + 1), dict(out=8 * FAKE + 1), dict(ids=4 * FAKE + 1), dict(dg=5 * FAKE + 2), dict(coef=6 * FAKE + 2),
    dict(dloss=7 * FAKE + 2), dict(out=FAKE + 2), dict(out=FAKE, stride=32), dict(dstride=1 << 41)])
def test_route_backward_refuses(lib, bad):
    assert _backward(lib, **bad) == dq.DQ_EINVAL


def test_route_backward_null_and_empty(lib):
    for name in ("l", "ids", "out"):
        assert _backward(lib, **{name: None}) == dq.DQ_ENULL
    assert _backward(lib, T=0, l=None, ids=None, out=None) == dq.DQ_OK


# Outputs that meet an operand or each other.  T = 8, E = 16, k = 2 bf16: 256 bytes
# of logits, 64 of ids and of gates, 8 of the mask.

def _route_two(lib, **changed):
    """Two workers, 1 MB of addresses for every buffer; a change is to the second's
    or, with an _ in front, to the first's."""
    first = dict(l=1, mask=2, ids=3, gates=4, part=5)
    second = dict(l=6, mask=7, ids=8, gates=9, part=10)
    at = [{n: m * FAKE for n, m in w.items()} for w in (first, second)]
    for name, v in changed.items():
        at[0 if name[0] == "_" else 1][name.lstrip("_")] = v
    io = (dq.dq_route_worker * 2)(*[(w["l"], 8, 16, w["mask"], w["ids"], w["gates"], w["part"], FAKE) for w in at])
    return lib.dq_route(io, 2, dq.BF16, 16, 2, 1, None)


@pytest.mark.parametrize("bad", [
    dict(ids=6 * FAKE), dict(gates=6 * FAKE + 252), dict(part=6 * FAKE), dict(ids=7 * FAKE + 4), dict(gates=8 * FAKE),
    dict(gates=8 * FAKE + 60), dict(ids=10 * FAKE + 64), dict(part=9 * FAKE),
    # with the other worker's
    dict(ids=1 * FAKE + 128), dict(_ids=6 * FAKE), dict(gates=2 * FAKE), dict(ids=3 * FAKE), dict(ids=4 * FAKE + 32),
    dict(gates=4 * FAKE), dict(part=5 * FAKE), dict(part=5 * FAKE + 256), dict(_part=1 * FAKE), dict(_gates=10 * FAKE)])
def test_route_refuses_outputs_that_overlap(lib, bad):
    assert _route_two(lib, **bad) == dq.DQ_EINVAL


def _backward_two(lib, coef=11 * FAKE, dloss=12 * FAKE, stride=16, _stride=16, dstride=16, _dstride=16, **changed):
    first = dict(l=1, mask=2, ids=3, dg=4, out=5)
    second = dict(l=6, mask=7, ids=8, dg=9, out=10)
    at = [{n: m * FAKE for n, m in w.items()} for w in (first, second)]
    for name, v in changed.items():
        at[0 if name[0] == "_" else 1][name.lstrip("_")] = v
    io = (dq.dq_route_grad * 2)(*[(w["l"], 8, s, w["mask"], w["ids"], w["dg"], w["out"], d)
                                  for w, s, d in zip(at, (_stride, stride), (_dstride, dstride))])
    return lib.dq_route_backward(io, 2, dq.BF16, 16, 2, 1, coef, dloss, None)


@pytest.mark.parametrize("bad", [
    dict(out=6 * FAKE + 32), dict(out=7 * FAKE), dict(out=8 * FAKE), dict(out=9 * FAKE + 62), dict(out=11 * FAKE + 60),
    dict(out=12 * FAKE), dict(dloss=10 * FAKE + 252), dict(coef=5 * FAKE),
    # with the other worker's; in place where that is another worker's logits too
    dict(out=1 * FAKE), dict(_out=6 * FAKE), dict(out=2 * FAKE), dict(out=3 * FAKE), dict(out=4 * FAKE),
    dict(out=5 * FAKE), dict(out=5 * FAKE + 224), dict(l=1 * FAKE, out=1 * FAKE), dict(_out=FAKE, l=FAKE + 32),
    # windows of one tensor that interleave and meet: 3 elements, 1 element, at another stride
    dict(out=5 * FAKE + 26, dstride=64, _dstride=64), dict(out=5 * FAKE + 98, dstride=64, _dstride=64),
    dict(out=5 * FAKE + 32, dstride=64, _dstride=48)])
def test_route_backward_refuses_outputs_that_overlap(lib, bad):
    assert _backward_two(lib, **bad) == dq.DQ_EINVAL


@pytest.mark.parametrize("bad", [
    dict(sums=FAKE + 8), dict(sums=FAKE - 256), dict(loss=FAKE + 256), dict(coef=FAKE + 64), dict(counts=FAKE),
    dict(coef=4 * FAKE), dict(loss=3 * FAKE + 60), dict(sums=2 * FAKE), dict(stats=7 * FAKE + 512), dict(loss=7 * FAKE),
    dict(sums=7 * FAKE + 256), dict(parts=((7 * FAKE, 8), (7 * FAKE + 256, 8))), dict(parts=((7 * FAKE, 8), (7 * FAKE, 9)))])
def test_balance_refuses_outputs_that_overlap(lib, bad):
    assert _balance(lib, **bad) == dq.DQ_EINVAL


def test_dropout_refuses_an_output_over_its_round_index(lib):
    for at in (0, 4, 508):
        assert _dropout(lib, d_round=4 * FAKE + at) == dq.DQ_EINVAL

# ---- refusals of the binding -----------------------------------------------------

def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros(4, 8)
    for call in (lambda: dq.dropout(x, 0.1), lambda: dq.dropout_backward(x, 0.1), lambda: dq.route(x, 2),
                 lambda: dq.balance(torch.zeros(17, dtype=torch.float64), 2),
                 lambda: dq.route_backward(x, torch.zeros(4, 2, dtype=torch.int32)),
                 lambda: train.dropout(x, 0.1), lambda: train.route(x, 2), lambda: train.route([x, x], 2)):
        with pytest.raises(ValueError):
            call()
    for bad in (x.half(), x.double(), x.int(), None, 3.0):
        with pytest.raises(TypeError):
            dq.dropout(bad, 0.1)
        with pytest.raises(TypeError):
            dq.route(bad, 2)
    for bad in (torch.zeros(4, dtype=torch.float64), torch.zeros(1, dtype=torch.float64), torch.zeros(3, 3)):
        with pytest.raises(ValueError):
            dq.balance(bad, 2)
    for bad in (None, [1.0]):
        with pytest.raises(TypeError):
            dq.balance(bad, 2)


def test_rows_of_views():
    x = torch.zeros(6, 4, 32)
    assert dq._rows(x, "x") == (1, 768, 768)
    assert dq._rows(x[:, :, 3:9], "x") == (24, 6, 32)
    assert dq._rows(x[:, 1:2, 3:9], "x") == (6, 6, 128)
    assert dq._rows(x[2, :, :5], "x") == (4, 5, 32)
    assert dq._rows(x[:, :, :1], "x") == (24, 1, 32)
    assert dq._rows(torch.zeros(32).expand(6, 32), "x") == (6, 32, 0)
    assert dq._rows(x[:0, :, :5], "x")[1] == 0
    for bad in (x.transpose(1, 2), x[:, :2, :5], x[:, :, ::2], x[:, :3], torch.zeros(1).expand(5)):
        with pytest.raises(ValueError):
            dq._rows(bad, "x")


def test_folded_statistics_stay_until_other_streams_have_read_them(monkeypatch):
    """Sums that a fold made on one stream are recorded on the stream of a later
    balance or fold; a part and its sums on their own stream are not."""
    now, recorded = [1], []
    monkeypatch.setattr(dq, "_raw_stream", lambda dev: now[0])
    monkeypatch.setattr(dq, "_call", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: now[0])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    stats = dq.RouteStats(8, torch.device("cpu"))
    part = torch.empty(64, dtype=torch.uint8)
    stats._add(part, part.data_ptr(), 4)
    first = stats.fold()
    dq.balance(stats, 2)
    assert recorded == []
    now[0] = 2
    dq.balance(stats, 2)
    assert recorded == [(first.data_ptr(), 2)]
    stats._add(part, part.data_ptr(), 4)
    second = stats.fold()                      # reads the first on stream 2, makes another there
    dq.balance(stats, 2)
    assert recorded == 2 * [(first.data_ptr(), 2)]
    now[0] = 1
    dq.balance(stats, 2)
    assert recorded[2:] == [(second.data_ptr(), 1)]


def test_route_wrapper_checks_the_list():
    with pytest.raises(ValueError):
        train.route([], 2)
    with pytest.raises(ValueError):
        train.route([torch.zeros(4, 8)], 2, masks=[None, None])
    with pytest.raises(ValueError):
        train.route([torch.zeros(4, 8), torch.zeros(4, 9)], 2)
    for call in (lambda: dq.route([], 2), lambda: dq.route_backward([], []),
                 lambda: dq.route([torch.zeros(4, 8)], 2, mask=[None, None])):
        with pytest.raises(ValueError):
            call()


def test_eval_dropout_is_the_input():
    x = torch.zeros(4, 8)
    assert train.dropout(x, 0.5, training=False) is x
