"""Products of rows with as many matrices as each workgroup still searches by itself, and one more (a map of the tiles)."""
import pytest
import torch

from product_helpers import DEV, Weights, offsets, product, rows

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def same(got, want, what):
    assert torch.equal(got.cpu(), want.to(F32).to(got.dtype)), what


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("each", (1, 3, 40, 70))
@pytest.mark.parametrize("E", (127, 128, 129, 257))
def test_search_and_map(nv, E, each, dtype):
    out, inp = 24, 128
    counts = [each * (i % 3) for i in range(E - 1)] + [each + 1]
    w, v = Weights(E, out, inp, 1, whole=True), Weights(E, out, inp, 2, whole=True)
    m, n = w.matrix(nv), v.matrix(nv)
    T, seg = sum(counts), offsets(counts).to(DEV)
    x, d = rows((T, inp), dtype, 2, whole=True), rows((T, out), dtype, 3, whole=True)
    same(nv.linear(m, x.to(DEV), seg_offsets=seg), product(x, w, counts)[0], "Y")
    _, g, u = nv.gated(m, n, x.to(DEV), seg_offsets=seg, with_pre=True)
    same(g, product(x, w, counts)[0], "G")
    same(u, product(x, v, counts)[0], "U")
    r = nv.linear_backward(m, d.to(DEV), seg_offsets=seg, with_bias=True)
    same(r["dX"], product(d, w, counts, False)[0], "dX")
    same(r["dbias"], torch.stack([c.sum(0) for c in d.double().split(counts)]), "dbias")
    g, u = rows((T, out), dtype, 4, whole=True), rows((T, out), dtype, 5, whole=True)
    dx = nv.gated_backward(m, n, d.to(DEV), g.to(DEV), u.to(DEV), activation=nv.ACT_RELU, seg_offsets=seg)["dX"]
    dg, du = d.double() * u.double() * (g > 0), d.double() * g.double().clamp(min=0)
    same(dx, product(dg, w, counts, False)[0] + product(du, v, counts, False)[0], "dX of two")
