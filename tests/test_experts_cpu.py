"""The experts' operators without a GPU: the plain forms that the GPU tests
compare with (gradients against differences, dithers against the kernels'
documented counter), and the argument checks of the C ABI and the binding."""
import ctypes as C
import os
import re
import struct
import subprocess

import numpy as np
import pytest
import torch

import experts_ref as ref
import test_gpu_experts as gpu
import train_ref
from compressed_hop_gradient_amd import build, dq, train

FAKE = 1 << 20      # never dereferenced: every call below fails its checks first, or has nothing to do


@pytest.fixture(scope="module")
def lib():
    return dq.lib()


# ---- the plain forms -------------------------------------------------------------

def test_rows_are_a_stable_sort():
    ids = np.array([[2, 0], [-1, 2], [1, 5], [0, 0]])
    r = ref.Rows(ids, 3)
    assert r.offsets.tolist() == [0, 3, 4, 6] and r.source.tolist() == [1, 6, 7, 4, 0, 3, 2, 5]
    assert r.row.tolist() == [[4, 0], [-1, 5], [3, -1], [1, 2]]


def test_dithers_are_apart_from_dropouts():
    """The counter is dropout's with bit 15 of its second word: element i + 2^50 of
    a dropout under the same numbers, which no memory holds."""
    key = dict(seed=0x123456789ABCDEF0, rnd=7, worker=3, site=2)
    assert ref.dithers(40, **key).tolist() == train_ref.dithers(40, first=1 << 50, **key).tolist()
    assert ref.dithers(40, **key).tolist() != train_ref.dithers(40, **key).tolist()


@pytest.mark.parametrize("dither", [False, True])
def test_kept_values_are_near(dither):
    rng = np.random.default_rng(0)
    x = rng.normal(size=(5, 70)) * np.exp(3 * rng.normal(size=(5, 70)))
    codes, exps, values = ref.keep(x, ref.dithers(350) if dither else 32768)
    step = np.repeat(2.0 ** (exps - 127), 32, 1)[:, :70]
    assert np.abs(codes).max() <= 127 and (np.abs(values - x) <= (1 if dither else 0.5) * step * (1 + 2 ** -15)).all()
    # the smallest power of two that fits
    for b in range(3):
        m = np.abs(x[:, 32 * b:32 * b + 32]).max(1)
        assert (m <= 127 * 2.0 ** (exps[:, b] - 127)).all() and (m > 127 * 2.0 ** (exps[:, b] - 128)).all()


@pytest.mark.parametrize("kind", ["swiglu", "relu"])
def test_reference_gradient_against_differences(kind):
    """Every input of an experts' layer, by central differences: h^2 f''' / 6 and 2^-53 /
    h, below 1e-8 here."""
    rng = np.random.default_rng(1)
    T, k, E, H, F = 5, 2, 3, 4, 3
    ids = np.array([[0, 2], [1, -1], [-1, -1], [2, 2], [1, 0]])
    rows = ref.Rows(ids, E)
    x, gates, dy = rng.normal(size=(T, H)), rng.uniform(size=(T, k)), rng.normal(size=(T, H))
    w_in, w_out = rng.normal(size=(E, H, F * (2 if kind == "swiglu" else 1))), rng.normal(size=(E, F, H))
    gate_of = lambda g: g.reshape(-1)[rows.source[:rows.n]]

    def value(x, gates, w_in, w_out):
        u = ref.matmul(x, w_in, rows, gather=True)[0]
        y = ref.matmul(ref.act(u, gate_of(gates), kind), w_out, rows)[0]
        return (ref.back(y, rows)[0] * dy).sum()

    args = [x, gates, w_in, w_out]
    u = ref.matmul(x, w_in, rows, gather=True)[0]
    da = ref.matmul(dy, w_out.transpose(0, 2, 1), rows, gather=True)[0]
    (du, dgate, a), _ = ref.act_backward(u, da, gate_of(gates), kind)
    dgates = np.zeros(T * k)
    dgates[rows.source[:rows.n]] = dgate
    grads = [ref.back(ref.matmul(du, w_in.transpose(0, 2, 1), rows)[0], rows)[0], dgates.reshape(T, k),
             ref.matmul_grad(x, du, rows, "x")[0], ref.matmul_grad(a, dy, rows, "dout")[0]]
    h = 1e-5
    for n, (arg, grad) in enumerate(zip(args, grads)):
        for i in np.ndindex(arg.shape):
            up, down = [a.copy() for a in args], [a.copy() for a in args]
            up[n][i] += h
            down[n][i] -= h
            assert abs((value(*up) - value(*down)) / (2 * h) - grad[i]) < 1e-7, (n, i)


# ---- refusals of the C ABI ---------------------------------------------------------

# Buffers of 1 MB of addresses each.  8 tokens, 2 choices, 4 experts: 16 slots.

def _lists(offsets=1 * FAKE, source=2 * FAKE, row=3 * FAKE, tokens=8, k=2, E=4):
    return C.byref(dq.dq_expert_lists(offsets, source, row, tokens, k, E))


def _lists_of(args):
    return _lists(**{n: args.pop(n) for n in ("offsets", "source", "row", "tokens", "k", "E") if n in args})


def _rows(lib, ids=1 * FAKE, tokens=8, k=2, E=4, offsets=2 * FAKE, source=3 * FAKE, row=4 * FAKE, work=5 * FAKE,
          size=FAKE):
    return lib.dq_expert_rows(ids, tokens, k, E, offsets, source, row, work, size, None)


def _matmul(lib, **a):
    l = _lists_of(a)
    d = dict(x=4 * FAKE, xs=32, flags=0, w=5 * FAKE, we=32 * 16, ws=16, y=6 * FAKE, ys=16, kind=dq.BF16, inner=32,
             outer=16)
    assert set(a) <= set(d), a
    return lib.dq_expert_matmul(l, *{**d, **a}.values(), None)


def _grad(lib, **a):
    l = _lists_of(a)
    d = dict(x=4 * FAKE, xs=32, codes=None, exponents=None, dy=5 * FAKE, dys=16, gather=0, dw=6 * FAKE, kind=dq.BF16,
             out=dq.BF16, inner=32, outer=16, work=7 * FAKE, size=FAKE)
    assert set(a) <= set(d), a
    return lib.dq_expert_matmul_grad(l, *{**d, **a}.values(), None)


def _sum(lib, **a):
    l = _lists_of(a)
    d = dict(y=4 * FAKE, ys=16, residual=5 * FAKE, rs=16, out=6 * FAKE, os=16, kind=dq.F32, width=16)
    assert set(a) <= set(d), a
    return lib.dq_expert_sum(l, *{**d, **a}.values(), None)


def _key(**a):
    d = dict(seed=1, d_round=None, round=0, worker=0, site=0, flags=1)
    return C.byref(dq.dq_keep_key(*{**d, **a}.values()))


KEYS = [dict(d_round=FAKE + 2), dict(worker=-1), dict(worker=65536), dict(site=1 << 31), dict(flags=2)]


def _keep(lib, x=1 * FAKE, kind=dq.BF16, rows=4, cols=40, xs=40, codes=2 * FAKE, exponents=3 * FAKE, key=None):
    return lib.dq_keep8(x, kind, rows, cols, xs, codes, exponents, key or _key(), None)


def _restore(lib, codes=1 * FAKE, exponents=2 * FAKE, kind=dq.BF16, rows=4, cols=40, y=3 * FAKE, ys=40):
    return lib.dq_restore8(codes, exponents, kind, rows, cols, y, ys, None)


def _act(lib, **a):
    l = _lists_of(a)
    d = dict(act=0, u=4 * FAKE, us=32, gates=5 * FAKE, a=6 * FAKE, as_=16, kind=dq.BF16, width=16, codes=7 * FAKE,
             exponents=8 * FAKE, key=_key())
    assert set(a) <= set(d), a
    return lib.dq_expert_act(l, *{**d, **a}.values(), None)


def _back(lib, **a):
    l = _lists_of(a)
    d = dict(act=0, u=4 * FAKE, us=32, codes=None, exponents=None, da=5 * FAKE, das=16, gates=6 * FAKE, du=7 * FAKE,
             dus=32, again=8 * FAKE, as_=16, dgates=9 * FAKE, kind=dq.BF16, width=16)
    assert set(a) <= set(d), a
    return lib.dq_expert_act_backward(l, *{**d, **a}.values(), None)


LISTS = [dict(tokens=-1), dict(tokens=1 << 30), dict(k=0), dict(k=17), dict(E=0), dict(E=1025), dict(offsets=FAKE + 2),
         dict(source=2 * FAKE + 1), dict(row=3 * FAKE + 2)]


@pytest.mark.parametrize("call", [_matmul, _grad, _sum, _act, _back])
def test_every_call_checks_its_lists(lib, call):
    for bad in LISTS:
        assert call(lib, **bad) == dq.DQ_EINVAL, bad
    for name in ("offsets", "source", "row"):
        assert call(lib, **{name: None}) == dq.DQ_ENULL, name


def test_rows_refuses(lib):
    for bad in (dict(tokens=-1), dict(tokens=1 << 30), dict(k=0), dict(k=17), dict(E=0), dict(E=1025), dict(ids=FAKE + 1),
                dict(offsets=2 * FAKE + 2), dict(source=3 * FAKE + 2), dict(row=4 * FAKE + 1), dict(offsets=FAKE + 60),
                dict(source=4 * FAKE), dict(row=2 * FAKE + 16), dict(row=5 * FAKE), dict(ids=3 * FAKE)):
        assert _rows(lib, **bad) == dq.DQ_EINVAL, bad
    for bad in (dict(ids=None), dict(offsets=None), dict(source=None), dict(row=None)):
        assert _rows(lib, **bad) == dq.DQ_ENULL, bad
    for bad in (dict(tokens=100000, work=None), dict(work=5 * FAKE + 128), dict(size=255), dict(tokens=100000, size=1024)):
        assert _rows(lib, **bad) == dq.DQ_EWORKSPACE, bad
    assert lib.dq_expert_rows_bytes(8, 2, 4) == 256 and lib.dq_expert_rows_bytes(1 << 30, 2, 4) == 0
    assert lib.dq_expert_rows_bytes(8, 0, 4) == 0 and lib.dq_expert_rows_bytes(8, 2, 1025) == 0


@pytest.mark.parametrize("bad", [
    dict(kind=2), dict(flags=4), dict(inner=0), dict(outer=0), dict(inner=(1 << 24) + 1), dict(xs=-1), dict(ws=-1),
    dict(we=-1), dict(ys=15), dict(xs=1 << 41), dict(x=4 * FAKE + 1), dict(w=5 * FAKE + 1), dict(y=6 * FAKE + 1),
    # y over x (whole, or the tokens alone), w, the lists
    dict(y=4 * FAKE + 1022), dict(y=4 * FAKE + 510, flags=1), dict(y=5 * FAKE + 4 * 512 * 2 - 2),
    dict(y=5 * FAKE + 4 * 512 * 2 - 2, flags=2, ws=32), dict(y=FAKE), dict(y=2 * FAKE + 62), dict(y=3 * FAKE)])
def test_matmul_refuses(lib, bad):
    assert _matmul(lib, **bad) == dq.DQ_EINVAL


def test_matmul_null_and_empty(lib):
    for name in ("x", "w", "y"):
        assert _matmul(lib, **{name: None}) == dq.DQ_ENULL
    assert _matmul(lib, tokens=0, source=None, row=None, x=None, y=None) == dq.DQ_OK


def test_products_refuse_more_tiles_than_a_launch_has(lib):
    """The checks pass, the tiles do not fit; before anything is launched."""
    far = dict(tokens=1 << 30, k=1, E=1, xs=0, inner=1)
    assert _matmul(lib, **far, kind=dq.F32, outer=1, ws=1, we=1, y=1 << 50, ys=1) == dq.DQ_EINVAL
    assert _matmul(lib, **far, outer=129, ws=129, we=129, y=1 << 50, ys=129) == dq.DQ_EINVAL
    assert _grad(lib, E=1024, inner=1 << 24, xs=1 << 24, outer=1, dys=1, x=1 << 44, dw=1 << 50) == dq.DQ_EINVAL


def test_extents_beyond_64_bits_are_seen(lib, tiles):
    """Weights whose last element lies 2^64 elements from the first, at the largest widths and
    strides there are: any result above them meets them.  Rows that far apart are not near
    enough for 32-bit offsets."""
    far = dict(E=1024, inner=1 << 24, we=1 << 40, ws=1 << 40, xs=0)
    assert _matmul(lib, **far, y=1 << 60) == dq.DQ_EINVAL
    assert _matmul(lib, **far, flags=dq.EXPERT_TURNED, outer=1 << 24, ys=1 << 24, y=1 << 60) == dq.DQ_EINVAL
    shape = (1, 2, 64, 64, 1, 0, 0)
    near, beyond, wrapped = tiles([("p", 0, 1 << 24, *shape, 64), ("p", 0, 1 << 24, *shape, 1 << 10),
                                   ("p", 0, (1 << 24) + 1, *shape, 1 << 40)])
    assert near[1] and not beyond[1] and not wrapped[1]


def test_too_many_tiles_are_refused_before_the_codes_are_restored(lib):
    """A product long enough that its codes are restored first: nothing is launched (without a GPU
    a launch fails with another error)."""
    assert _grad(lib, E=1024, inner=1 << 24, outer=1, dys=1, x=None, codes=1 << 44, exponents=1 << 46, dw=1 << 50,
                 work=1 << 54, size=1 << 50) == dq.DQ_EINVAL


@pytest.mark.parametrize("bad", [
    dict(kind=2), dict(out=2), dict(kind=dq.F32, out=dq.BF16), dict(gather=-1), dict(gather=3), dict(inner=0), dict(outer=0),
    dict(xs=-1), dict(dys=1 << 41), dict(x=4 * FAKE + 1), dict(dy=5 * FAKE + 1), dict(dw=6 * FAKE + 1),
    dict(out=dq.F32, dw=6 * FAKE + 2), dict(codes=8 * FAKE, exponents=9 * FAKE),
    dict(dw=4 * FAKE + 1022), dict(dw=5 * FAKE), dict(dw=5 * FAKE - 4094), dict(dw=FAKE), dict(dw=7 * FAKE),
    dict(work=4 * FAKE), dict(x=None, codes=8 * FAKE, exponents=9 * FAKE, dw=8 * FAKE),
    dict(x=None, codes=8 * FAKE, exponents=9 * FAKE, dw=9 * FAKE + 14)])
def test_matmul_grad_refuses(lib, bad):
    assert _grad(lib, **bad) == dq.DQ_EINVAL


def test_matmul_grad_null_and_workspace(lib):
    for bad in (dict(x=None), dict(dy=None), dict(dw=None), dict(codes=8 * FAKE), dict(x=None, exponents=8 * FAKE)):
        assert _grad(lib, **bad) == dq.DQ_ENULL, bad
    for bad in (dict(work=None), dict(work=7 * FAKE + 128), dict(size=255), dict(tokens=100000, size=4096)):
        assert _grad(lib, **bad) == dq.DQ_EWORKSPACE, bad
    size = lib.dq_expert_matmul_grad_bytes
    assert size(8, 2, 4, dq.BF16, 0, 32, 16, 0) == 256 and size(100000, 2, 4, dq.BF16, 0, 32, 16, 0) > 256
    # long products from codes hold x, of the tokens or of all rows
    for gather, rows in ((0, 2000), (1, 1000), (2, 2000)):
        assert size(1000, 2, 16, dq.BF16, gather, 2048, 1024, 1) == 256 + rows * 2048 * 2
    assert size(8, 2, 4, dq.BF16, 1, 32, 16, 1) == 256
    for bad in ((-1, 2, 4, 0, 0, 32, 16), (8, 17, 4, 0, 0, 32, 16), (8, 2, 0, 0, 0, 32, 16), (8, 2, 4, 2, 0, 32, 16),
                (8, 2, 4, 0, 3, 32, 16), (8, 2, 4, 0, -1, 32, 16), (8, 2, 4, 0, 0, 0, 16), (8, 2, 4, 0, 0, 32, 1 << 25)):
        assert size(*bad, 0) == 0


@pytest.mark.parametrize("bad", [
    dict(kind=2), dict(width=0), dict(width=(1 << 24) + 1), dict(ys=-1), dict(rs=-1), dict(os=15), dict(y=4 * FAKE + 2),
    dict(residual=5 * FAKE + 2), dict(out=6 * FAKE + 2), dict(out=4 * FAKE + 1020), dict(out=5 * FAKE + 64),
    dict(out=5 * FAKE, os=32), dict(out=FAKE), dict(out=3 * FAKE + 60)])
def test_sum_refuses(lib, bad):
    assert _sum(lib, **bad) == dq.DQ_EINVAL


def test_sum_null_and_empty(lib):
    assert _sum(lib, y=None) == dq.DQ_ENULL and _sum(lib, out=None) == dq.DQ_ENULL
    assert _sum(lib, tokens=0, y=None, out=None) == dq.DQ_OK


@pytest.mark.parametrize("bad", [
    dict(kind=2), dict(rows=-1), dict(cols=-1), dict(xs=-1), dict(rows=1 << 46), dict(cols=1 << 40), dict(x=FAKE + 1),
    dict(codes=FAKE + 319), dict(codes=3 * FAKE - 159), dict(exponents=FAKE), *[dict(key=_key(**k)) for k in KEYS],
    dict(key=_key(d_round=2 * FAKE + 156)), dict(key=_key(d_round=3 * FAKE))])
def test_keep_refuses(lib, bad):
    assert _keep(lib, **bad) == dq.DQ_EINVAL


@pytest.mark.parametrize("bad", [
    dict(kind=2), dict(rows=-1), dict(cols=-1), dict(ys=39), dict(y=3 * FAKE + 1), dict(y=FAKE + 158), dict(y=2 * FAKE),
    dict(y=2 * FAKE - 316)])
def test_restore_refuses(lib, bad):
    assert _restore(lib, **bad) == dq.DQ_EINVAL


def test_keep_and_restore_null_and_empty(lib):
    for name in ("x", "codes", "exponents"):
        assert _keep(lib, **{name: None}) == dq.DQ_ENULL
    for name in ("y", "codes", "exponents"):
        assert _restore(lib, **{name: None}) == dq.DQ_ENULL
    assert lib.dq_keep8(FAKE, 0, 4, 40, 40, 2 * FAKE, 3 * FAKE, None, None) == dq.DQ_ENULL
    for empty in (dict(rows=0), dict(cols=0)):
        assert _keep(lib, x=None, **empty) == dq.DQ_OK and _restore(lib, y=None, **empty) == dq.DQ_OK


@pytest.mark.parametrize("bad", [
    dict(act=2), dict(act=-1), dict(kind=2), dict(width=0), dict(us=-1), dict(as_=15), dict(u=4 * FAKE + 1),
    dict(gates=5 * FAKE + 2), dict(a=6 * FAKE + 1), *[dict(key=_key(**k)) for k in KEYS], dict(a=4 * FAKE + 1022),
    dict(a=5 * FAKE + 62), dict(a=7 * FAKE), dict(codes=8 * FAKE - 511), dict(exponents=4 * FAKE), dict(a=2 * FAKE),
    dict(key=_key(d_round=7 * FAKE + 508))])
def test_act_refuses(lib, bad):
    assert _act(lib, **bad) == dq.DQ_EINVAL


def test_act_null_and_empty(lib):
    for bad in (dict(u=None), dict(gates=None), dict(a=None), dict(codes=None), dict(exponents=None), dict(key=None)):
        assert _act(lib, **bad) == dq.DQ_ENULL, bad
    assert _act(lib, tokens=0, u=None, a=None) == dq.DQ_OK


@pytest.mark.parametrize("bad", [
    dict(act=2), dict(kind=2), dict(width=0), dict(us=-1), dict(das=-1), dict(dus=31), dict(as_=15), dict(u=4 * FAKE + 1),
    dict(da=5 * FAKE + 1), dict(gates=6 * FAKE + 2), dict(du=7 * FAKE + 1), dict(again=8 * FAKE + 1),
    dict(dgates=9 * FAKE + 2), dict(codes=10 * FAKE, exponents=11 * FAKE), dict(du=4 * FAKE), dict(du=5 * FAKE + 510),
    dict(again=5 * FAKE), dict(again=7 * FAKE), dict(dgates=6 * FAKE), dict(dgates=8 * FAKE + 508),
    dict(u=None, codes=10 * FAKE, exponents=11 * FAKE, du=10 * FAKE), dict(dgates=3 * FAKE)])
def test_act_backward_refuses(lib, bad):
    assert _back(lib, **bad) == dq.DQ_EINVAL


def test_act_backward_null_and_empty(lib):
    for bad in (dict(u=None), dict(da=None), dict(gates=None), dict(du=None), dict(codes=FAKE), dict(u=None, exponents=FAKE)):
        assert _back(lib, **bad) == dq.DQ_ENULL, bad
    assert _back(lib, tokens=0, u=None, da=None, du=None) == dq.DQ_OK


# ---- which kernel ------------------------------------------------------------------

@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    """Lines of tests/native/expert_tiles.cpp to its answers."""
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path_factory.mktemp("tiles") / "expert_tiles")
    subprocess.run([build.HIPCC, "-O1", "-I", os.path.join(build.ROOT, "include"), "-I", build.CSRC,
                    os.path.join(here, "native", "expert_tiles.cpp"), os.path.join(build.CSRC, "dq_expert_pick.cpp"),
                    "-o", exe], check=True, capture_output=True)

    def ask(lines):
        text = "\n".join(" ".join(str(int(v) if not isinstance(v, str) else v) for v in l) for l in lines) + "\n"
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")[:-1]
        assert len(out) == len(lines)
        return [(o.split()[0], *(int(v) for v in o.split()[1:])) for o in out]
    return ask


# bytes of a row of a step, and steps in LDS
RING = {"Any": (128, 2), "FewAny": (128, 2)}


def test_every_product_kernel_is_tested_in_many_steps(tiles):
    """By the rule that picks them, the shapes of the GPU tests reach every tile in both
    types, gathered or not, turned or not, in steps that go round its stages twice."""
    lines = [("p", f32, *shape, gather, turned, off) for shapes, offs in ((gpu.DEEP, (0, 1)), (gpu.LARGE, (0,)))
             for shape in shapes for f32 in (0, 1) for gather in (0, 1) for turned in (0, 1) for off in offs]
    met = set()
    for line, (tile, *_) in zip(lines, tiles(lines)):
        f32, K = line[1], line[5]
        row, stages = RING.get(tile, (64, 4))
        step = row // (4 if f32 else 2) * (4 if tile.startswith("Few") else 1)       # Few: a quarter for each wave
        if K > 2 * stages * step:
            met.add((tile, f32, *line[7:9]))
    want = {(tile, f32, gather, turned) for f32 in (0, 1) for gather in (0, 1) for turned in (0, 1)
            for tile in ("Big", "Mid", "Small", "Few", "Any", "FewAny") if not (f32 and tile == "Big")}
    assert met == want, want ^ met


def test_every_gradient_kernel_is_tested_in_many_steps(lib, tiles):
    lines = [("w", f32, *shape, gather, kept, off) for shapes, offs in ((gpu.DEEP, (0, 1)), (gpu.LARGE, (0,)))
             for shape in shapes for f32 in (0, 1) for gather in (0, 1, 2) for kept in (0, 1) for off in offs]
    asked = []
    for op, f32, T, k, E, K, N, gather, kept, off in lines:
        if kept:
            # codes of long products are restored first, and read as rows on 16 bytes
            size = [lib.dq_expert_matmul_grad_bytes(T, k, E, dq.F32 if f32 else dq.BF16, gather, K, N, c) for c in (0, 1)]
            if size[0] != size[1]:
                kept = 0
        asked.append((op, f32, T, k, E, K, N, gather, kept, off))
    met, split = set(), set()
    for line, (tile, x_lds, dy_lds, parts, _) in zip(asked, tiles(asked)):
        _, f32, T, k, E, K, N, gather, kept, off = line
        row, stages = RING.get(tile, (64, 4))
        loads = "kept" if kept else "lds" if tile != "Any" else "any"
        # of an average expert, a tenth of whose rows are left out
        if 0.85 * T * k / E / parts > 2 * stages * row // (4 if f32 else 2):
            met.add((tile, f32, gather, loads, dy_lds if kept else 1))
        split.add((tile, f32, parts > 1))
    want = {(tile, f32, gather, "lds", 1) for f32 in (0, 1) for gather in (0, 1, 2)
            for tile in (("Mid", "Small") if f32 else ("Big", "Mid", "Narrow"))}
    want |= {("Any", f32, gather, "any", 1) for f32 in (0, 1) for gather in (0, 1, 2)}
    want |= {("Any", f32, gather, "kept", dy) for f32 in (0, 1) for gather in (0, 1, 2) for dy in (0, 1)}
    assert met == want, want ^ met
    assert {("Any", 0, True), ("Any", 1, True), ("Narrow", 0, True), ("Mid", 0, True), ("Small", 1, True)} <= split


# ---- assembly -----------------------------------------------------------------------

def test_assembly_tells_the_compiler_of_m0():
    """Loads into LDS go where M0 says: it is an operand of the statement, never written
    behind the compiler's back."""
    loads = 0
    for name in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, name)) as f:
            statements = re.findall(r"asm volatile\((.*?)\);", f.read(), re.S)
        for s in statements:
            text = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', s.split(":")[0]))
            for line in text.split("\\n"):
                words = line.replace("\\t", " ").split()
                assert "m0" not in [w.strip(",") for w in words[1:2]], (name, line)
                if words and words[-1] == "lds":
                    loads += 1
                    assert '"{m0}"' in s, (name, line)
    assert loads


def _listings(tmp):
    """The library's gfx950 code, as the assembler's listing: [(address, instruction) ...] by
    address."""
    objdump = "/opt/rocm/llvm/bin/llvm-objdump"
    if not os.path.exists(objdump):
        pytest.skip("no llvm-objdump")
    with open(dq.LIB_PATH, "rb") as f:
        image = f.read()
    for m in re.finditer(b"__CLANG_OFFLOAD_BUNDLE__", image):
        at, entry = m.start(), m.start() + 32
        for _ in range(min(struct.unpack_from("<Q", image, at + 24)[0], 8)):
            off, size, n = struct.unpack_from("<QQQ", image, entry)
            name, entry = image[entry + 24:entry + 24 + n], entry + 24 + n
            if name.endswith(b"gfx950") and size:
                path = tmp / "code"
                path.write_bytes(image[at + off:at + off + size])
                text = subprocess.run([objdump, "-d", str(path)], capture_output=True, text=True, check=True).stdout
                found = re.findall(r"^\t(\S.*?)\s*// ([0-9A-F]+):", text, re.M)
                yield [(int(a, 16), i) for i, a in found]


def _scalars(operand):
    m = re.match(r"s\[(\d+):(\d+)\]$", operand)
    return {f"s{i}" for i in range(int(m[1]), int(m[2]) + 1)} if m else {operand}


def test_loads_into_lds_wait_for_their_scalars(tmp_path):
    """Nothing behind the compiler's back counts the waits in front of an instruction written
    out: five for a scalar that a vector instruction wrote (descriptor, M0), one for M0 from
    the scalar unit.  On every way to every such load of the built code."""
    loads = 0
    for code in _listings(tmp_path):
        jumps = {}
        for n, (a, i) in enumerate(code):
            if i.startswith(("s_branch", "s_cbranch")):
                to = int(i.split()[1])
                jumps.setdefault(a + 4 + 4 * (to - (to >> 15 << 16)), []).append(n)
        for at, (_, load) in enumerate(code):
            if not load.endswith(" lds"):
                continue
            loads += 1
            need = _scalars(load.split(None, 1)[1].split(", ")[1]) | {"m0"}
            ways, seen = [(at, 0)], set()
            while ways:
                n, waited = ways.pop()
                if (n, waited) in seen or waited >= 5:
                    continue
                seen.add((n, waited))
                # before instruction n: the one above it, and those that jump to it
                for b in ([n - 1] if n and not code[n - 1][1].startswith(("s_branch", "s_endpgm")) else []) + \
                        jumps.get(code[n][0], []):
                    words = code[b][1].replace(",", " ").split()
                    wrote = need & _scalars(words[1]) if len(words) > 1 else set()
                    assert not (wrote and words[0].startswith("v_")), (code[b], load, waited)
                    assert not ("m0" in wrote and words[0].startswith("s_") and waited < 1), (code[b], load)
                    ways.append((b, waited + (1 + int(words[1], 0) if words[0] == "s_nop" else 1)))
    assert loads > 500


# ---- refusals of the binding -----------------------------------------------------

def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros(4, 8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: dq.keep8(x), lambda: dq.expert_rows(i, 4), lambda: dq.expert_rows(x, 4),
                 lambda: dq.ExpertRows(i[0], i[0], i), lambda: dq.Kept8(x.to(torch.int8), x, torch.float32),
                 lambda: train.experts(x, i, x, x, x), lambda: train.experts(x, i, x, x, x, keep=True, site=(1 << 31) - 1)):
        with pytest.raises((ValueError, TypeError)):
            call()
    for call in (lambda: dq.expert_matmul(x, x, None), lambda: dq.expert_matmul_grad(x, x, i),
                 lambda: dq.expert_sum(x, None), lambda: dq.expert_act(x, x, None),
                 lambda: dq.expert_act_backward(x, x, x, None), lambda: dq.restore8(x), lambda: dq.keep8(x.half()),
                 lambda: dq.keep8(None)):
        with pytest.raises(TypeError):
            call()


def test_matrix_rows_of_views():
    x = torch.zeros(6, 4, 32)
    assert dq._matrix_rows(x, "x") == (24, 32, 32)
    assert dq._matrix_rows(x[:, :, 3:9], "x") == (24, 6, 32)
    assert dq._matrix_rows(x[0, 0], "x") == (1, 32, 32)
    assert dq._matrix_rows(x[:0], "x") == (0, 32, 32) and dq._matrix_rows(x[:, :, :0].contiguous(), "x")[0] == 0
    for bad in (x.transpose(1, 2), x[:, :, ::2], torch.zeros(())):
        with pytest.raises(ValueError):
            dq._matrix_rows(bad, "x")
