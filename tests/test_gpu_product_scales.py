"""Gradients of a gated pair whose matrices have very different global scales S, down to denormal ones."""
import pytest
import torch

from product_helpers import DEV, Weights, close, offsets, product, rows, sum_error

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
# of gate and up; quotients beyond binary32 in either direction, and denormal S
PAIRS = [(2.0 ** 30, 2.0 ** -100), (2.0 ** -100, 2.0 ** 30), (2.0 ** -10, 2.0 ** -140), (2.0 ** -140, 2.0 ** -10),
         (2.0 ** 20, 2.0 ** -70), (1.0, 1.0)]


def pair(E, out, inp, S):
    w, v = Weights(E, out, inp, 1, whole=True), Weights(E, out, inp, 2, whole=True)
    for k, one in enumerate((w, v)):
        one.values /= one.S.double()[:, None, None]
        one.S = torch.tensor([S[e % len(S)][k] for e in range(E)])
        one.values *= one.S.double()[:, None, None]
    return w, v


def inputs(T, out, dtype):
    """dH, G, U, of whole numbers; every third row has no gradient through the gate, every third none through up."""
    d, g, u = (rows((T, out), dtype, s, whole=True) for s in (3, 4, 5))
    g = g.abs() + 1
    u[1::3] = 0
    g[2::3] = -g[2::3]
    return d, g, u


def terms(d, g, u):
    return d.double() * u.double() * (g > 0), d.double() * g.double().clamp(min=0)


@DTYPES
@pytest.mark.parametrize("S", PAIRS, ids=range(len(PAIRS)))
@pytest.mark.parametrize("T, out, inp", [(1, 72, 320), (40, 203, 208), (140, 72, 320), (130, 1600, 144), (300, 513, 2064)])
def test_scales_far_apart(nv, T, out, inp, S, dtype):
    w, v = pair(1, out, inp, [S])
    d, g, u = inputs(T, out, dtype)
    got = nv.gated_backward(w.matrix(nv), v.matrix(nv), d.to(DEV), g.to(DEV), u.to(DEV), activation=nv.ACT_RELU)["dX"]
    dg, du = terms(d, g, u)
    (a, sa), (b, sb) = product(dg, w, [T], False), product(du, v, [T], False)
    close(got, a + b, sum_error(sa + sb, 2 * out, dtype), dtype, "dX")


@DTYPES
def test_experts_of_either_order(nv, dtype):
    counts = [130, 7, 0, 200, 33, 64]
    E, T, out, inp = len(counts), sum(counts), 136, 272
    w, v = pair(E, out, inp, PAIRS)
    d, g, u = inputs(T, out, dtype)
    got = nv.gated_backward(w.matrix(nv), v.matrix(nv), d.to(DEV), g.to(DEV), u.to(DEV), activation=nv.ACT_RELU,
                            seg_offsets=offsets(counts).to(DEV))["dX"]
    dg, du = terms(d, g, u)
    (a, sa), (b, sb) = product(dg, w, counts, False), product(du, v, counts, False)
    close(got, a + b, sum_error(sa + sb, 2 * out, dtype), dtype, "dX")


@pytest.mark.parametrize("S", PAIRS[:4], ids=range(4))
def test_large_tiles(nv, S):
    """Tiles of 256 x 256 (the reference in 64 bits on the GPU)."""
    T, out, inp = 300, 4104, 16416
    w, v = pair(1, out, inp, [S])
    d, g, u = inputs(T, out, BF16)
    got = nv.gated_backward(w.matrix(nv), v.matrix(nv), d.to(DEV), g.to(DEV), u.to(DEV), activation=nv.ACT_RELU)["dX"]
    want, size = 0, 0
    for t, one in zip(terms(d, g, u), (w, v)):
        t, values = t.to(DEV), one.values[0].to(DEV)
        want, size = want + (t @ values).cpu(), size + (t.abs() @ values.abs()).cpu()
    close(got, want, sum_error(size, 2 * out, BF16), BF16, "dX")
