"""Products with NVFP4 matrices against the 64-bit model: sizes around every tile's edge with sums that are
exact in binary32 (the outputs then have to be the rounded exact values), activations, experts, gradients."""
import pytest
import torch

from product_helpers import (ACTS, DEV, HALF_STEP, Weights, act, act_error, act_model, by_row, close, offsets,
                             product, rows, sum_error)
from product_helpers import _E4M3 as E4M3, _LEVELS as LEVELS

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))

SIZES = [(1, 1, 16), (1, 16, 32), (2, 17, 48), (3, 128, 64), (1, 333, 2064), (5, 64, 1040), (15, 33, 80), (16, 129, 128),
         (17, 127, 144), (31, 250, 16), (33, 128, 272), (48, 48, 512), (63, 257, 256), (64, 256, 336), (65, 96, 128),
         (127, 130, 64), (128, 128, 1024), (129, 129, 528), (200, 1, 96), (255, 255, 256), (256, 512, 144),
         (257, 300, 1040), (512, 640, 192), (700, 260, 64)]


def same(got, want, dtype, what):
    """Equal to the exact value rounded once (whole numbers: the sums are exact)."""
    assert torch.equal(got.cpu(), want.to(F32).to(dtype)), what


@DTYPES
@pytest.mark.parametrize("T, out, inp", SIZES)
def test_linear_is_the_rounded_exact_sum(nv, T, out, inp, dtype):
    w = Weights(1, out, inp, 10 * T + out, whole=True)
    x, r = rows((T, inp), dtype, 1, whole=True), rows((T, out), dtype, 2, whole=True)
    b = rows((1, out), dtype, 3, whole=True)
    z = product(x, w, [T])[0]
    m = w.matrix(nv, squeeze=True)
    same(nv.linear(m, x.to(DEV)), z, dtype, "Y")
    y, pre = nv.linear(m, x.to(DEV), bias=b.to(DEV), activation=nv.ACT_RELU, residual=r.to(DEV), with_pre=True)
    z = z + b.double()
    same(pre, z, dtype, "Z")
    same(y, z.clamp(min=0) + r.double(), dtype, "Y of all")


@DTYPES
@pytest.mark.parametrize("T, out, inp", SIZES)
def test_gated_is_the_rounded_exact_sum(nv, T, out, inp, dtype):
    w, v = Weights(1, out, inp, 10 * T + out, whole=True), Weights(1, out, inp, 7 * T + out, whole=True)
    x = rows((T, inp), dtype, 1, whole=True)
    x[:, 3:] = torch.where(torch.rand((T, inp - 3), generator=torch.Generator().manual_seed(5)) < 0.9, 0, x[:, 3:])
    g, u = product(x, w, [T])[0], product(x, v, [T])[0]
    h, gg, uu = nv.gated(w.matrix(nv), v.matrix(nv), x.to(DEV), activation=nv.ACT_RELU, with_pre=True)
    same(gg, g, dtype, "G")
    same(uu, u, dtype, "U")
    # g and u are exact; their product is rounded to binary32, then to dtype
    close(h, g.clamp(min=0) * u, (g * u).abs() * 2.0 ** -24, dtype, "H")
    assert torch.equal(nv.gated(w.matrix(nv), v.matrix(nv), x.to(DEV), activation=nv.ACT_RELU), h)


@DTYPES
@pytest.mark.parametrize("T, out, inp", SIZES)
def test_gradient_is_the_rounded_exact_sum(nv, T, out, inp, dtype):
    w, v = Weights(1, out, inp, 10 * T + out, whole=True), Weights(1, out, inp, 7 * T + out, whole=True)
    d = rows((T, out), dtype, 1, whole=True)
    r = nv.linear_backward(w.matrix(nv), d.to(DEV), with_bias=True)
    same(r["dX"], product(d, w, [T], False)[0], dtype, "dX")
    same(r["dbias"], d.double().sum(0, keepdim=True), F32, "dbias")
    assert r["dZ"] is None
    # gate and up: relu and whole numbers; S of the two differ by powers of two
    g, u = rows((T, out), dtype, 2, whole=True), rows((T, out), dtype, 3, whole=True)
    r = nv.gated_backward(w.matrix(nv), v.matrix(nv), d.to(DEV), g.to(DEV), u.to(DEV), activation=nv.ACT_RELU)
    dg, du = d.double() * u.double() * (g > 0), d.double() * g.double().clamp(min=0)
    same(r["dG"], dg, dtype, "dG")
    same(r["dU"], du, dtype, "dU")
    same(r["dX"], product(dg, w, [T], False)[0] + product(du, v, [T], False)[0], dtype, "dX of two")


# sizes that have enough tiles of 256 x 256 for them, with edges inside; reductions of an odd number of steps
LARGE = [(1030, 8200, 4112), (300, 4104, 16416), (777, 20008, 1040)]


@DTYPES
@pytest.mark.parametrize("T, out, inp", LARGE)
def test_large_sums_are_rounded_once(nv, T, out, inp, dtype):
    """Forward, gated and backward by the largest tiles (the reference in 64 bits on the GPU: whole numbers)."""
    w, v = Weights(1, out, inp, 1, whole=True), Weights(1, out, inp, 2, whole=True)
    x, d = rows((T, inp), dtype, 3, whole=True).to(DEV), rows((T, out), dtype, 4, whole=True).to(DEV)
    g, u = rows((T, out), dtype, 5, whole=True).to(DEV), rows((T, out), dtype, 6, whole=True).to(DEV)
    wv, vv = w.values[0].to(DEV), v.values[0].to(DEV)
    m, n = w.matrix(nv), v.matrix(nv)
    same(nv.linear(m, x, residual=g), (x.double() @ wv.t() + g.double()).cpu(), dtype, "Y")
    h, gate, up = nv.gated(m, n, x, activation=nv.ACT_RELU, with_pre=True)
    same(gate, (x.double() @ wv.t()).cpu(), dtype, "G")
    same(up, (x.double() @ vv.t()).cpu(), dtype, "U")
    same(nv.linear_backward(m, d)["dX"], (d.double() @ wv).cpu(), dtype, "dX")
    r = nv.gated_backward(m, n, d, g, u, activation=nv.ACT_RELU)
    dg, du = d.double() * u.double() * (g > 0), d.double() * g.double().clamp(min=0)
    same(r["dX"], (dg @ wv + du @ vv).cpu(), dtype, "dX of two")


@DTYPES
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("T, out, inp", [(1, 130, 272), (19, 70, 528), (150, 200, 336)])
def test_linear_values(nv, T, out, inp, name, dtype):
    w = Weights(1, out, inp, T, whole=False)
    x, r, b = rows((T, inp), dtype, 1, 0.3), rows((T, out), dtype, 2), rows((1, out), dtype, 3)
    z, size = product(x, w, [T])
    z = z + b.double()
    error = sum_error(size + b.double().abs(), inp, dtype)
    y, pre = nv.linear(w.matrix(nv), x.to(DEV), bias=b.to(DEV), activation=act(nv, name), residual=r.to(DEV),
                       with_pre=True)
    close(pre, z, error, dtype, "Z")
    # the slopes are at most 1.13; the residual's addition is one more rounding
    a = act_model(z, name)[0]
    room = 1.13 * error + (act_error(z, dtype) if name not in ("none", "relu") else 0)
    close(y, a + r.double(), room + (a.abs() + r.double().abs()) * 2.0 ** -23, dtype, "Y")


@DTYPES
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("T, out, inp", [(1, 130, 272), (19, 70, 528), (150, 200, 336)])
def test_gated_values(nv, T, out, inp, name, dtype):
    w, v = Weights(1, out, inp, T), Weights(1, out, inp, T + 1)
    x = rows((T, inp), dtype, 1, 0.3)
    (g, gs), (u, us) = product(x, w, [T]), product(x, v, [T])
    h, gg, uu = nv.gated(w.matrix(nv), v.matrix(nv), x.to(DEV), activation=act(nv, name), with_pre=True)
    ge, ue = sum_error(gs, inp, dtype), sum_error(us, inp, dtype)
    close(gg, g, ge, dtype, "G")
    close(uu, u, ue, dtype, "U")
    a = act_model(g, name)[0]
    ae = 1.13 * ge + act_error(g, dtype)
    close(h, a * u, ae * (u.abs() + ue) + a.abs() * ue + (a * u).abs() * 2.0 ** -23, dtype, "H")


@DTYPES
@pytest.mark.parametrize("name", ACTS[1:])
@pytest.mark.parametrize("T, out, inp", [(1, 130, 272), (19, 72, 528), (150, 203, 336)])
def test_gradient_values(nv, T, out, inp, name, dtype):
    w, v = Weights(1, out, inp, T), Weights(1, out, inp, T + 1)
    d, z, u = rows((T, out), dtype, 1), rows((T, out), dtype, 2, 2.0), rows((T, out), dtype, 3)
    z[0, :6] = torch.tensor([0.0, 30.0, -30.0, 1e4, -1e4, -0.0]).to(dtype)       # flat ends
    a, slope = act_model(z.double(), name)
    error = act_error(z.double().clamp(-40, 40), dtype)
    r = nv.linear_backward(w.matrix(nv), d.to(DEV), Z=z.to(DEV), activation=act(nv, name), with_bias=True)
    dz = d.double() * slope
    dze = d.double().abs() * (error + slope.abs() * 2.0 ** -23)
    close(r["dZ"], dz, dze, dtype, "dZ")
    used = r["dZ"].cpu()                      # the product takes dZ as it is held
    dx, size = product(used, w, [T], False)
    close(r["dX"], dx, sum_error(size, out, dtype), dtype, "dX")
    close(r["dbias"], dz.sum(0, keepdim=True), dze.sum(0) + T * 2.0 ** -23 * dz.abs().sum(0), F32, "dbias")
    r = nv.gated_backward(w.matrix(nv), v.matrix(nv), d.to(DEV), z.to(DEV), u.to(DEV), activation=act(nv, name))
    du, dg = d.double() * a, d.double() * u.double() * slope
    big = (z.double().abs() + 1) * 2.0 ** -22
    close(r["dU"], du, d.double().abs() * (error + a.abs() * 2.0 ** -23 + big * (name != "relu")), dtype, "dU")
    close(r["dG"], dg, (d.double() * u.double()).abs() * (error + slope.abs() * 2.0 ** -22), dtype, "dG")
    (x1, s1), (x2, s2) = product(r["dG"].cpu(), w, [T], False), product(r["dU"].cpu(), v, [T], False)
    close(r["dX"], x1 + x2, sum_error(s1 + s2, 2 * out, dtype), dtype, "dX of two")


COUNTS = [[0, 0, 5], [3, 0, 1, 129, 0, 17, 64], [1] * 70, [0] * 130 + [40] + [0] * 20, [300, 1, 2], [16, 32, 48, 65],
          [2, 0, 1] * 30 + [200]]


@DTYPES
@pytest.mark.parametrize("behind", (0, 7))
@pytest.mark.parametrize("counts", COUNTS, ids=range(len(COUNTS)))
def test_experts(nv, counts, behind, dtype):
    """Rows of several matrices, some without any; rows behind the last are left as they were."""
    E, T, out, inp = len(counts), sum(counts), 72, 144
    w, v = Weights(E, out, inp, 1, whole=True), Weights(E, out, inp, 2, whole=True)
    pad = lambda t: torch.cat([t, torch.full((behind, t.shape[1]), float("nan"), dtype=dtype)]).to(DEV)  # noqa: E731
    x, b = rows((T, inp), dtype, 3, whole=True), rows((E, out), dtype, 4, whole=True)
    d, g, u = (rows((T, out), dtype, s, whole=True) for s in (5, 6, 7))
    seg, m, n = offsets(counts).to(DEV), w.matrix(nv), v.matrix(nv)

    def fresh(cols):
        return torch.full((T + behind, cols), 77.0, dtype=dtype, device=DEV)

    def check(got, want, what):
        same(got[:T], want, dtype, what)
        assert bool((got[T:] == 77).all()), f"{what}: rows behind the last matrix's"

    def space(n):
        return torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)

    n_rows = T + behind
    Y, Z = fresh(out), fresh(out)
    nv.nvfp4_linear(m, pad(x), n_rows, seg, b.to(DEV), nv.ACT_RELU, None, Z, Y,
                    space(nv.nvfp4_linear_workspace_size(dtype, n_rows, E, out, inp)))
    z = product(x, w, counts)[0] + by_row(b, counts)
    check(Z, z, "Z")
    check(Y, z.clamp(min=0), "Y")
    H, G, U = fresh(out), fresh(out), fresh(out)
    nv.nvfp4_gated(m, n, pad(x), n_rows, seg, nv.ACT_RELU, G, U, H,
                   space(nv.nvfp4_gated_workspace_size(dtype, n_rows, E, out, inp)))
    z_g, z_u = product(x, w, counts)[0], product(x, v, counts)[0]
    check(G, z_g, "G")
    check(U, z_u, "U")
    h = z_g.clamp(min=0) * z_u
    close(H[:T], h, h.abs() * 2.0 ** -24, dtype, "H")
    assert bool((H[T:] == 77).all())
    dX, dZ = fresh(inp), fresh(out)
    dbias = torch.full((E, out), 77.0, device=DEV)
    nv.nvfp4_linear_backward(m, pad(d), n_rows, seg, nv.ACT_RELU, pad(g), dZ, dbias, dX,
                             space(nv.nvfp4_linear_backward_workspace_size(dtype, n_rows, E, out, inp, True)))
    dz = d.double() * (g > 0)
    check(dZ, dz, "dZ")
    check(dX, product(dz, w, counts, False)[0], "dX")
    sums = torch.stack([c.sum(0) for c in dz.split(counts)])
    same(dbias, sums, F32, "dbias")
    dX, dG, dU = fresh(inp), fresh(out), fresh(out)
    nv.nvfp4_gated_backward(m, n, pad(d), n_rows, seg, nv.ACT_RELU, pad(g), pad(u), dG, dU, dX,
                            space(nv.nvfp4_gated_backward_workspace_size(dtype, n_rows, E, out, inp)))
    dg, du = d.double() * u.double() * (g > 0), d.double() * g.double().clamp(min=0)
    check(dG, dg, "dG")
    check(dU, du, "dU")
    check(dX, product(dg, w, counts, False)[0] + product(du, v, counts, False)[0], "dX of two")


@pytest.mark.parametrize("shift", (0, 1))
@pytest.mark.parametrize("T, out, inp", [(64, 129, 192), (65, 70, 64), (80, 201, 1088), (95, 128, 320), (96, 40, 2112),
                                         (97, 129, 192)])
def test_tens_of_rows(nv, T, out, inp, shift):
    """Tiles of 64 and 96 rows, whole and not; with rows laid out for 16-byte stores and not."""
    w, v = Weights(1, out, inp, T + out, whole=True), Weights(1, out, inp, T + inp, whole=True)
    x, r = rows((T, inp), BF16, 1, whole=True), rows((T, out), BF16, 2, whole=True)
    b = rows((1, out), BF16, 3, whole=True)
    wide = torch.zeros((T, out + 8 + shift), dtype=BF16, device=DEV)
    wide[:, shift:out + shift] = r.to(DEV)
    z = product(x, w, [T])[0] + b.double()
    y, pre = nv.linear(w.matrix(nv), x.to(DEV), bias=b.to(DEV), activation=nv.ACT_RELU,
                       residual=wide[:, shift:out + shift], with_pre=True)
    same(pre, z, BF16, "Z")
    same(y, z.clamp(min=0) + r.double(), BF16, "Y")
    _, g, u = nv.gated(w.matrix(nv), v.matrix(nv), x.to(DEV), with_pre=True)
    same(g, product(x, w, [T])[0], BF16, "G")
    same(u, product(x, v, [T])[0], BF16, "U")


@pytest.mark.parametrize("counts", ([65, 0, 130, 64], [300, 255, 1, 0, 200], [257, 256, 256], [200] * 3, [0, 0, 700, 1, 65],
                                    [70] + [0, 1, 200] * 50))
def test_experts_of_many_rows(nv, counts):
    E, T, out, inp = len(counts), sum(counts), 72, 192
    w, v = Weights(E, out, inp, 1, whole=True), Weights(E, out, inp, 2, whole=True)
    x, b, seg = rows((T, inp), BF16, 3, whole=True), rows((E, out), BF16, 4, whole=True), offsets(counts).to(DEV)
    z = product(x, w, counts)[0]
    same(nv.linear(w.matrix(nv), x.to(DEV), bias=b.to(DEV), seg_offsets=seg), z + by_row(b, counts), BF16, "Y")
    _, g, u = nv.gated(w.matrix(nv), v.matrix(nv), x.to(DEV), seg_offsets=seg, with_pre=True)
    same(g, z, BF16, "G")
    same(u, product(x, v, counts)[0], BF16, "U")


@DTYPES
@pytest.mark.parametrize("T", (1, 4, 40, 140))
def test_every_weight_is_exact(nv, T, dtype):
    """Every code under every scale byte, met by a one: the output is the weight."""
    out, inp = 127 * 16, 128
    w = Weights(1, out, inp, 1)
    o, i = torch.arange(out)[:, None], torch.arange(inp)[None]
    code = ((o // 127 + i) % 16).to(torch.uint8)[None]
    w.packed, w.scales = code[..., ::2] | code[..., 1::2] << 4, (o % 127 + 0 * i[:, ::16]).to(torch.uint8)[None].contiguous()
    w.S = torch.ones(1)
    w.values = LEVELS[code.long()] * E4M3[w.scales.long()].repeat_interleave(16, -1)
    x = torch.zeros((T, inp), dtype=dtype)
    at = torch.arange(T) * 37 % inp
    x[torch.arange(T), at] = 1
    same(nv.linear(w.matrix(nv), x.to(DEV)), w.values[0][:, at].t(), dtype, "Y")
    g, u = nv.gated(w.matrix(nv), w.matrix(nv), x.to(DEV), with_pre=True)[1:]
    same(g, w.values[0][:, at].t(), dtype, "G")
    assert torch.equal(g, u)


@pytest.mark.parametrize("inp", (64, 1040, 2064, 17408))
@pytest.mark.parametrize("power", (-90, -20, 0, 9, 90))
def test_few_rows_of_any_magnitude(nv, power, inp):
    """A row times a power of two; and small values beside one of 2^29 times theirs that meets weights of zero."""
    T, out = 4, 70
    w = Weights(1, out, inp, inp, whole=True)
    w.packed[..., 0] &= 0xF0                             # column 0: zeros
    w.values[..., 0] = 0
    x = rows((T, inp), BF16, 1, whole=True).double()
    if inp > 2064:                                       # whole numbers that bf16 holds
        x[torch.rand(x.shape, generator=torch.Generator().manual_seed(2)) < 0.9] = 0
    x[:2] *= 2.0 ** power
    x[2] *= 2.0 ** -power
    x[1:3, 0] = x[1:3].abs().amax(1) * 2.0 ** 29
    b = x.to(BF16)
    assert torch.equal(b.double(), x)
    z = product(x, w, [T])[0]
    same(nv.linear(w.matrix(nv), b.to(DEV)), z, BF16, "Y")
    g = nv.gated(w.matrix(nv), w.matrix(nv), b.to(DEV), with_pre=True)[1]
    same(g, z, BF16, "G")


@DTYPES
@pytest.mark.parametrize("name", ("none", "gelu"))
@pytest.mark.parametrize("counts, out", [([1], 16), ([33], 17), ([512], 40), ([513], 40), ([2000], 129), ([0, 3, 600, 1], 70),
                                         ([0, 3, 2700, 0, 1], 70), ([1, 0] * 90, 24), ([7000], 1)])
def test_bias_gradients(nv, counts, out, name, dtype):
    """One share of the rows and several, alone and beside the slopes."""
    E, T, inp = len(counts), sum(counts), 32
    w = Weights(E, out, inp, 1, whole=True)
    d, z = rows((T, out), dtype, 2, whole=True), rows((T, out), dtype, 3)
    seg = None if E == 1 else offsets(counts).to(DEV)
    got = nv.linear_backward(w.matrix(nv), d.to(DEV), Z=None if name == "none" else z.to(DEV), activation=act(nv, name),
                             seg_offsets=seg, with_bias=True)["dbias"].cpu()
    g = d.double() * act_model(z.double(), name)[1]
    want, size = torch.zeros((E, out), dtype=torch.float64), torch.zeros((E, out), dtype=torch.float64)
    at = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))
    want.index_add_(0, at, g)
    size.index_add_(0, at, d.double().abs())
    # whole numbers: exact; else slopes of at most 1.2, off by at most 16 steps, and sums of T of them
    off = 0 if name == "none" else (16 + T) * 2.0 ** -23 * 1.2 * size
    assert bool(((got.double() - want).abs() <= off).all())


@pytest.mark.parametrize("counts, out, inp", [([300, 260, 200, 400], 4096, 4096), ([70, 130], 264, 1040),
                                              ([129, 1, 200, 64], 136, 2064), ([140] * 40, 136, 272), ([140] * 70, 72, 272)])
def test_tiles_of_several_matrices(nv, counts, out, inp):
    """Few and many tiles of rows, large and small ones, in both directions."""
    E, T = len(counts), sum(counts)
    w, v = Weights(E, out, inp, 1, whole=True), Weights(E, out, inp, 2, whole=True)
    d, seg = rows((T, out), BF16, 3, whole=True), offsets(counts).to(DEV)
    want = product(d, w, counts, transposed=False)[0]
    same(nv.linear_backward(w.matrix(nv), d.to(DEV), seg_offsets=seg)["dX"], want, BF16, "dX")
    if out < 4096:
        x = rows((T, inp), F32, 4, whole=True)
        _, g, u = nv.gated(w.matrix(nv), v.matrix(nv), x.to(DEV), seg_offsets=seg, with_pre=True)
        same(g, product(x, w, counts)[0], F32, "G")
        same(u, product(x, v, counts)[0], F32, "U")
