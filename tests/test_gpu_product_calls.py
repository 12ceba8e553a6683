"""Calls of the products with NVFP4 matrices as programs make them: strided, offset and padded tensors, matrices that
lie apart, values that are no number, offsets that are no partition, workspaces, streams, graphs, memory beyond 32 bits;
and the calls together, as a layer's forward and backward pass and as a decode step."""
import pytest
import torch

from product_helpers import (DEV, Weights, act, act_error, act_model, close, offsets, product, rows, spans, sum_error)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
# rows for each kernel: few rows, some tens, tiles; the last two columns: whole pieces of 64 and odd ones
SHAPES = pytest.mark.parametrize("T, out, inp", [(3, 72, 320), (40, 72, 320), (140, 72, 320), (3, 37, 208), (40, 37, 208),
                                                 (140, 37, 208)])


def exact(x, w, counts=None):
    return product(x, w, counts or [x.shape[0]])[0]


def same(got, want, what=""):
    assert torch.equal(got.cpu(), want.to(F32).to(got.dtype)), what


def padded(t, ld, fill=float("nan"), shift=0):
    """t's rows in a larger buffer, `shift` elements from its start and ld apart; and the buffer."""
    buf = torch.full((shift + t.shape[0] * ld + 64,), fill, dtype=t.dtype, device=DEV)
    view = buf[shift:shift + t.shape[0] * ld].view(t.shape[0], ld)[:, :t.shape[1]]
    view.copy_(t)
    return view, buf


def untouched(buf, view, fill):
    """Nothing but the view was written."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool((buf[mask] == fill).all())


def space(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV) if n else None


@DTYPES
@SHAPES
@pytest.mark.parametrize("shift", (0, 1))
def test_strides(nv, T, out, inp, shift, dtype):
    """Rows with NaN between them, outputs in wider buffers whose rest stays, at odd offsets."""
    w, v = Weights(1, out, inp, 1, whole=True), Weights(1, out, inp, 2, whole=True)
    m, n = w.matrix(nv), v.matrix(nv)
    x, r = rows((T, inp), dtype, 3, whole=True), rows((T, out), dtype, 4, whole=True)
    d, g, u = (rows((T, out), dtype, s, whole=True) for s in (5, 6, 7))
    X = padded(x, inp + 24)[0]
    R = padded(r, out + 5 + shift, shift=shift)[0]

    def outputs(*cols, whole=False):
        made = [padded(torch.zeros((T, c), dtype=dtype), c + (16 + -c % 8 if whole else 3 + shift), 77.0,
                       0 if whole else shift) for c in cols]
        return [a for a, _ in made], made

    def check(made):
        for view, buf in made:
            assert untouched(buf, view, 77.0)

    (Y, Z), made = outputs(out, out)
    nv.nvfp4_linear(m, X, T, None, None, nv.ACT_NONE, R, Z, Y,
                    space(nv.nvfp4_linear_workspace_size(dtype, T, 1, out, inp)))
    same(Z, exact(x, w))
    same(Y, exact(x, w) + r.double())
    check(made)
    (H, G, U), made = outputs(out, out, out)
    nv.nvfp4_gated(m, n, X, T, None, nv.ACT_RELU, G, U, H,
                   space(nv.nvfp4_gated_workspace_size(dtype, T, 1, out, inp)))
    same(G, exact(x, w))
    same(U, exact(x, v))
    check(made)
    (dX,), made = outputs(inp)
    (dZ,), made2 = outputs(out, whole=dtype == BF16 and out % 8 == 0)
    D, Gi, Ui = (padded(t, out + 5 + shift, shift=shift)[0] for t in (d, g, u))
    nv.nvfp4_linear_backward(m, D, T, None, nv.ACT_RELU, Gi, dZ, None, dX,
                             space(nv.nvfp4_linear_backward_workspace_size(dtype, T, 1, out, inp, False)))
    dz = d.double() * (g > 0)
    same(dZ, dz)
    same(dX, product(dz, w, [T], False)[0])
    check(made + made2)
    (dX,), made = outputs(inp)
    (dG, dU), made2 = outputs(out, out, whole=dtype == BF16 and out % 8 == 0)
    nv.nvfp4_gated_backward(m, n, D, T, None, nv.ACT_RELU, Gi, Ui, dG, dU, dX,
                            space(nv.nvfp4_gated_backward_workspace_size(dtype, T, 1, out, inp)))
    dg, du = d.double() * u.double() * (g > 0), d.double() * g.double().clamp(min=0)
    same(dX, product(dg, w, [T], False)[0] + product(du, v, [T], False)[0])
    check(made + made2)


@DTYPES
@SHAPES
def test_residual_in_place(nv, T, out, inp, dtype):
    w = Weights(1, out, inp, 1, whole=True)
    x, r = rows((T, inp), dtype, 3, whole=True), rows((T, out), dtype, 4, whole=True)
    Y = r.to(DEV)
    nv.nvfp4_linear(w.matrix(nv), x.to(DEV), T, None, None, nv.ACT_NONE, Y, None, Y,
                    space(nv.nvfp4_linear_workspace_size(dtype, T, 1, out, inp)))
    same(Y, exact(x, w) + r.double())


@DTYPES
@SHAPES
@pytest.mark.parametrize("shift", (1, 2, 4, 8))
def test_matrices_at_any_offset(nv, T, out, inp, shift, dtype):
    """Codes at a multiple of 8 bytes, scale bytes anywhere."""
    w = Weights(1, out, inp, 1, whole=True)
    x, d = rows((T, inp), dtype, 3, whole=True), rows((T, out), dtype, 4, whole=True)
    codes = torch.zeros(w.packed.numel() + 64, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(w.scales.numel() + 64, dtype=torch.uint8, device=DEV)
    p, s = codes[8 * shift:8 * shift + w.packed.numel()], scales[shift:shift + w.scales.numel()]
    p.copy_(w.packed.flatten())
    s.copy_(w.scales.flatten())
    m = nv.Matrix(p.view(out, inp // 2), s.view(out, inp // 16), w.S.to(DEV))
    same(nv.linear(m, x.to(DEV)), exact(x, w))
    same(nv.linear_backward(m, d.to(DEV))["dX"], product(d, w, [T], False)[0])


@DTYPES
@pytest.mark.parametrize("counts", ([2, 3], [50, 0, 33], [130, 7, 200]))
def test_matrices_that_lie_apart(nv, counts, dtype):
    """Gate and up as halves of the rows of one stacked batch."""
    E, out, inp, T = len(counts), 40, 192, sum(counts)
    both = Weights(E, 2 * out, inp, 3, whole=True)
    p, s, S = both.packed.to(DEV), both.scales.to(DEV), both.S.to(DEV)
    m, n = nv.Matrix(p[:, :out], s[:, :out], S), nv.Matrix(p[:, out:], s[:, out:], S)
    x, d = rows((T, inp), dtype, 1, whole=True), rows((T, out), dtype, 2, whole=True)
    seg = offsets(counts).to(DEV)
    _, g, u = nv.gated(m, n, x.to(DEV), activation=nv.ACT_RELU, seg_offsets=seg, with_pre=True)
    want = exact(x, both, counts)
    same(g, want[:, :out])
    same(u, want[:, out:])
    dx = torch.zeros((T, inp), dtype=torch.float64)
    for e, r in spans(counts):
        dx[r] = d[r].double() @ both.values[e, out:]
    same(nv.linear_backward(n, d.to(DEV), seg_offsets=seg)["dX"], dx)


@DTYPES
@SHAPES
def test_what_is_no_number_stays_in_its_row(nv, T, out, inp, dtype):
    w, v = Weights(1, out, inp, 1, whole=True), Weights(1, out, inp, 2, whole=True)
    m, n = w.matrix(nv), v.matrix(nv)
    x, d, z = rows((T, inp), dtype, 3, whole=True), rows((T, out), dtype, 4, whole=True), rows((T, out), dtype, 5, whole=True)
    bad = {0: float("nan"), T - 1: float("inf")}
    xb, db = x.clone(), d.clone()
    for t, value in bad.items():
        xb[t, inp // 2], db[t, out // 2] = value, value
    keep = torch.tensor([t not in bad for t in range(T)])
    for a, b in ((nv.linear(m, xb.to(DEV)), nv.linear(m, x.to(DEV))),
                 (nv.gated(m, n, xb.to(DEV)), nv.gated(m, n, x.to(DEV))),
                 (nv.linear_backward(m, db.to(DEV))["dX"], nv.linear_backward(m, d.to(DEV))["dX"]),
                 (nv.gated_backward(m, n, db.to(DEV), z.to(DEV), z.to(DEV))["dX"],
                  nv.gated_backward(m, n, d.to(DEV), z.to(DEV), z.to(DEV))["dX"])):
        assert torch.equal(a[keep], b[keep])
        assert not torch.isfinite(a[0]).any()
    # an S that is no number: its matrix's rows alone
    two = Weights(2, out, inp, 6, whole=True)
    two.S[0] = float("nan")
    y = nv.linear(two.matrix(nv), x.to(DEV), seg_offsets=torch.tensor([0, 1, T], device=DEV))
    assert torch.isnan(y[:1]).all() and torch.isfinite(y[1:]).all()


@DTYPES
@SHAPES
@pytest.mark.parametrize("value", (float("nan"), float("inf"), -float("inf")))
def test_no_sum_of_a_row_hides_what_is_no_number(nv, T, out, inp, value, dtype):
    w, v = Weights(1, out, inp, 1, whole=True), Weights(1, out, inp, 2, whole=True)
    m, n = w.matrix(nv), v.matrix(nv)
    x, d, z = rows((T, inp), dtype, 3, whole=True), rows((T, out), dtype, 4, whole=True), rows((T, out), dtype, 5, whole=True)
    x[0, 0] = x[1, inp - 1] = d[0, 0] = d[1, out - 1] = value
    g, u = nv.gated(m, n, x.to(DEV), with_pre=True)[1:]
    for y in (nv.linear(m, x.to(DEV)), g, u, nv.linear_backward(m, d.to(DEV))["dX"],
              nv.gated_backward(m, n, d.to(DEV), z.to(DEV), z.to(DEV))["dX"]):
        assert not torch.isfinite(y[:2]).any() and torch.isfinite(y[2:]).all()


@DTYPES
@pytest.mark.parametrize("seg", ([0, 40, 10, 90], [0, -5, 30, 1 << 40], [50, 20, 10, 0], [0, 0, 0, 0], [0, 1 << 62, -1, 90]))
def test_offsets_that_are_no_partition(nv, seg, dtype):
    """Unspecified values in the rows, nothing outside them; every call ends."""
    T, out, inp, E = 90, 40, 96, len(seg) - 1
    w = Weights(E, out, inp, 1, whole=True)
    m, s = w.matrix(nv), torch.tensor(seg, dtype=torch.int64, device=DEV)
    x, d = rows((T, inp), dtype, 2, whole=True).to(DEV), rows((T, out), dtype, 3, whole=True).to(DEV)
    Y, buf = padded(torch.zeros((T, out), dtype=dtype), out + 8, 77.0, 64)
    nv.nvfp4_linear(m, x, T, s, None, nv.ACT_NONE, None, None, Y,
                    space(nv.nvfp4_linear_workspace_size(dtype, T, E, out, inp)))
    assert untouched(buf, Y, 77.0)
    dX, buf = padded(torch.zeros((T, inp), dtype=dtype), inp + 8, 77.0, 64)
    nv.nvfp4_linear_backward(m, d, T, s, nv.ACT_NONE, None, None, torch.empty((E, out), device=DEV), dX,
                             space(nv.nvfp4_linear_backward_workspace_size(dtype, T, E, out, inp, True)))
    assert untouched(buf, dX, 77.0)
    nv.gated(m, m, x, seg_offsets=s)
    nv.gated_backward(m, m, d, d, d, seg_offsets=s)
    torch.cuda.synchronize()


@DTYPES
@pytest.mark.parametrize("each", (1, 3, 40, 70))
@pytest.mark.parametrize("E", (129, 700))
def test_many_matrices(nv, E, each, dtype):
    """More matrices than each workgroup searches by itself."""
    out, inp = 24, 80
    counts = [each * (i % 3) for i in range(E)]
    w, x = Weights(E, out, inp, 1, whole=True), rows((sum(counts), inp), dtype, 2, whole=True)
    seg = offsets(counts).to(DEV)
    same(nv.linear(w.matrix(nv), x.to(DEV), seg_offsets=seg), exact(x, w, counts))
    d = rows((sum(counts), out), dtype, 3, whole=True)
    r = nv.linear_backward(w.matrix(nv), d.to(DEV), seg_offsets=seg, with_bias=True)
    same(r["dX"], product(d, w, counts, False)[0])
    same(r["dbias"], torch.stack([c.sum(0) for c in d.double().split(counts)]))


def test_one_matrix_with_offsets(nv):
    """A batch of one whose rows end before the tensor does."""
    w = Weights(1, 40, 96, 1, whole=True)
    for T, n in ((4, 3), (50, 33), (300, 150), (300, 0)):
        x = rows((T, 96), BF16, 2, whole=True)
        Y = torch.full((T, 40), 77.0, dtype=BF16, device=DEV)
        nv.nvfp4_linear(w.matrix(nv), x.to(DEV), T, torch.tensor([0, n], device=DEV), None, nv.ACT_NONE, None, None, Y,
                        space(nv.nvfp4_linear_workspace_size(BF16, T, 1, 40, 96)))
        same(Y[:n], exact(x[:n], w))
        assert bool((Y[n:] == 77).all())


@DTYPES
@pytest.mark.parametrize("T, out, inp, E", [(2, 70, 1040, 1), (33, 200, 2048, 1), (130, 129, 2064, 1), (150, 72, 320, 5),
                                            (300, 41, 128, 150)])
def test_workspaces_are_large_enough(nv, T, out, inp, E, dtype):
    """The size asked for and no byte more, between guards."""
    w, v = Weights(E, out, inp, 1, whole=True), Weights(E, out, inp, 2, whole=True)
    m, n = w.matrix(nv), v.matrix(nv)
    counts = [T // E] * E
    counts[-1] += T - sum(counts)
    seg = offsets(counts).to(DEV) if E > 1 else None
    x, d, g = rows((T, inp), dtype, 3, whole=True), rows((T, out), dtype, 4, whole=True), rows((T, out), dtype, 5, whole=True)

    def guarded(size):
        buf = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device=DEV)
        return buf, buf[256:256 + size] if size else None

    def empty(cols):
        return torch.empty((T, cols), dtype=dtype, device=DEV)

    def intact(buf, size):
        assert bool((buf[:256] == 0xA5).all()) and bool((buf[256 + size:] == 0xA5).all())

    size = nv.nvfp4_linear_workspace_size(dtype, T, E, out, inp)
    buf, ws = guarded(size)
    Y = empty(out)
    nv.nvfp4_linear(m, x.to(DEV), T, seg, None, nv.ACT_NONE, None, None, Y, ws)
    same(Y, exact(x, w, counts))
    intact(buf, size)
    size = nv.nvfp4_gated_workspace_size(dtype, T, E, out, inp)
    buf, ws = guarded(size)
    H, G, U = empty(out), empty(out), empty(out)
    nv.nvfp4_gated(m, n, x.to(DEV), T, seg, nv.ACT_RELU, G, U, H, ws)
    same(U, exact(x, v, counts))
    intact(buf, size)
    size = nv.nvfp4_linear_backward_workspace_size(dtype, T, E, out, inp, True)
    buf, ws = guarded(size)
    dX, dZ, db = empty(inp), empty(out), torch.empty((E, out), device=DEV)
    nv.nvfp4_linear_backward(m, d.to(DEV), T, seg, nv.ACT_RELU, g.to(DEV), dZ, db, dX, ws)
    dz = d.double() * (g > 0)
    same(dX, product(dz, w, counts, False)[0])
    same(db, torch.stack([c.sum(0) for c in dz.split(counts)]))
    intact(buf, size)
    size = nv.nvfp4_gated_backward_workspace_size(dtype, T, E, out, inp)
    buf, ws = guarded(size)
    dX, dG, dU = empty(inp), empty(out), empty(out)
    nv.nvfp4_gated_backward(m, n, d.to(DEV), T, seg, nv.ACT_RELU, g.to(DEV), g.to(DEV), dG, dU, dX, ws)
    same(dX, product(d.double() * g.double() * (g > 0), w, counts, False)[0]
         + product(d.double() * g.double().clamp(min=0), v, counts, False)[0])
    intact(buf, size)


def test_memory_beyond_32_bits(nv):
    """Experts behind 4 GiB of codes, and outputs and rows behind 2^32 elements."""
    E, out, inp = 40, 14336, 16384
    w = Weights(1, 8, inp, 1, whole=True)
    p = torch.zeros((E, out, inp // 2), dtype=torch.uint8, device=DEV)
    s = torch.zeros((E, out, inp // 16), dtype=torch.uint8, device=DEV)
    p[-1, -8:], s[-1, -8:] = w.packed[0].to(DEV), w.scales[0].to(DEV)
    S = torch.ones(E, device=DEV) * w.S.to(DEV)
    m = nv.Matrix(p, s, S)
    for T in (2, 40, 200):
        x = rows((T, inp), BF16, T, whole=True)
        seg = torch.tensor([0] * E + [T], device=DEV)
        same(nv.linear(m, x.to(DEV), seg_offsets=seg)[:, -8:], exact(x, w))
        d = torch.zeros((T, out), dtype=BF16)
        d[:, -8:] = rows((T, 8), BF16, T + 1, whole=True)
        same(nv.linear_backward(m, d.to(DEV), seg_offsets=seg)["dX"], product(d[:, -8:], w, [T], False)[0])
    del p, s, m
    T, w = 140000, Weights(1, 32768, 16, 2, whole=True)
    x = torch.zeros((T, 16), dtype=BF16, device=DEV)
    last = rows((5, 16), BF16, 3, whole=True)
    x[-5:] = last.to(DEV)
    y = nv.linear(w.matrix(nv), x)
    same(y[-5:], exact(last, w))
    d = rows((5, 8), BF16, 4, whole=True)
    y.zero_()
    y[-5:, -8:] = d.to(DEV)
    same(nv.linear_backward(w.matrix(nv), y)["dX"][-5:], d.double() @ w.values[0, -8:])


def _block(nv, gate, up, down, x, name):
    """A gated feed-forward block with a residual, and its gradient for a given one of its output."""
    h, g, u = nv.gated(gate, up, x, activation=act(nv, name), with_pre=True)
    y = nv.linear(down, h, residual=x)
    return y, h, g, u


def _block_backward(nv, gate, up, down, dy, g, u, name):
    dh = nv.linear_backward(down, dy)["dX"]
    r = nv.gated_backward(gate, up, dh, g, u, activation=act(nv, name))
    return r["dX"] + dy, dh, r


@DTYPES
@pytest.mark.parametrize("name", ("silu", "gelu"))
@pytest.mark.parametrize("T", (1, 30, 200))
def test_feed_forward_block(nv, T, name, dtype):
    """Forward and backward pass of a block of the four calls, each step against the model on what it was given."""
    hidden, inner = 192, 144
    gate, up, down = (Weights(1, o, i, s) for o, i, s in ((inner, hidden, 1), (inner, hidden, 2), (hidden, inner, 3)))
    M = [w.matrix(nv) for w in (gate, up, down)]
    x, dy = rows((T, hidden), dtype, 4, 0.3), rows((T, hidden), dtype, 5, 0.1)
    y, h, g, u = _block(nv, *M, x.to(DEV), name)
    (gw, gs), (uw, us) = product(x, gate, [T]), product(x, up, [T])
    ge, ue = sum_error(gs, hidden, dtype), sum_error(us, hidden, dtype)
    close(g, gw, ge, dtype, "g")
    close(u, uw, ue, dtype, "u")
    a = act_model(gw, name)[0]
    close(h, a * uw, (1.13 * ge + act_error(gw, dtype)) * (uw.abs() + ue) + a.abs() * ue + (a * uw).abs() * 2.0 ** -23,
          dtype, "h")
    yw, ys = product(h.cpu(), down, [T])
    close(y, yw + x.double(), sum_error(ys, inner, dtype) + (yw.abs() + x.double().abs()) * 2.0 ** -23, dtype, "y")
    dx, dh, r = _block_backward(nv, *M, dy.to(DEV), g, u, name)
    dw, ds = product(dy, down, [T], False)
    close(dh, dw, sum_error(ds, hidden, dtype), dtype, "dh")
    (x1, s1), (x2, s2) = product(r["dG"].cpu(), gate, [T], False), product(r["dU"].cpu(), up, [T], False)
    close(r["dX"], x1 + x2, sum_error(s1 + s2, 2 * inner, dtype), dtype, "dx")
    # the block's gradient against differences of the block in 64 bits, along one direction
    def loss(v):
        gv, uv = product(v, gate, [T])[0], product(v, up, [T])[0]
        return ((product(act_model(gv, name)[0] * uv, down, [T])[0] + v) * dy.double()).sum()
    way = rows((T, hidden), F32, 6).double()
    diff = (loss(x.double() + 1e-6 * way) - loss(x.double() - 1e-6 * way)) / 2e-6
    got = (dx.cpu().double() * way).sum()
    # four roundings to dtype on the way (g, u, dh, and dG or dU) and two of the sums and dx: of the sum of magnitudes
    room = 8 * (2.0 ** -8 if dtype == BF16 else 2.0 ** -20) * (dx.cpu().double() * way).abs().sum() + 1e-5 * diff.abs()
    assert abs(got - diff) <= room


def test_same_bits_every_time(nv):
    for T, out, inp, dtype in ((1, 300, 4096, BF16), (40, 300, 4096, BF16), (333, 1003, 2064, F32), (300, 513, 1024, BF16)):
        w = Weights(1, out, inp, 1)
        m, x, d = w.matrix(nv), rows((T, inp), dtype, 2).to(DEV), rows((T, out), dtype, 3).to(DEV)
        first = nv.linear(m, x), nv.linear_backward(m, d, with_bias=True)
        for _ in range(3):
            again = nv.linear(m, x), nv.linear_backward(m, d, with_bias=True)
            assert torch.equal(first[0], again[0])
            assert torch.equal(first[1]["dX"], again[1]["dX"]) and torch.equal(first[1]["dbias"], again[1]["dbias"])


def test_two_streams_at_once(nv):
    """Blocks on two streams, with tensors made on a third; each equals the one run alone."""
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    work = []
    for k, T in enumerate((60, 300)):
        M = [Weights(1, o, i, 10 * k + s).matrix(nv) for o, i, s in ((528, 256, 1), (528, 256, 2), (256, 528, 3))]
        x, dy = rows((T, 256), BF16, k, 0.3).to(DEV), rows((T, 256), BF16, k + 5, 0.1).to(DEV)
        y, h, g, u = _block(nv, *M, x, "silu")
        work.append((M, x, dy, (y, _block_backward(nv, *M, dy, g, u, "silu")[0])))
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for side, (M, x, dy, _) in zip(sides, work):
            side.wait_stream(torch.cuda.current_stream())
            h, g, u = nv.gated(M[0], M[1], x, with_pre=True, stream=side)
            y = nv.linear(M[2], h, residual=x, stream=side)
            dh = nv.linear_backward(M[2], dy, stream=side)["dX"]
            r = nv.gated_backward(M[0], M[1], dh, g, u, stream=side)
            got.append((y, r["dX"]))
        for side in sides:
            torch.cuda.current_stream().wait_stream(side)
        for (y, dx), (M, x, dy, (yw, dxw)) in zip(got, work):
            assert torch.equal(y, yw) and torch.equal(dx + dy, dxw)
        torch.cuda.synchronize()


@pytest.mark.parametrize("T", (1, 40, 200))
def test_graph(nv, T):
    """A block of experts, forward and backward, captured; replays with new inputs and the program's own work between
    them equal the eager calls."""
    E, hidden, inner = 4, 128, 200
    counts = [T // 2, 0, T - T // 2, 0]
    seg = offsets(counts).to(DEV)
    M = [Weights(E, o, i, s).matrix(nv) for o, i, s in ((inner, hidden, 1), (inner, hidden, 2), (hidden, 208, 3))]
    x, dy = torch.zeros((T, hidden), dtype=BF16, device=DEV), torch.zeros((T, hidden), dtype=BF16, device=DEV)

    def call():
        h, g, u = nv.gated(M[0], M[1], x, seg_offsets=seg, with_pre=True)
        wide = torch.zeros((T, 208), dtype=BF16, device=DEV)
        wide[:, :inner] = h
        y = nv.linear(M[2], wide, activation=nv.ACT_GELU, residual=x, seg_offsets=seg, with_pre=True)
        r = nv.linear_backward(M[2], dy, Z=y[1], activation=nv.ACT_GELU, seg_offsets=seg, with_bias=True)
        b = nv.gated_backward(M[0], M[1], r["dX"][:, :inner].contiguous(), g, u, seg_offsets=seg)
        return y[0], r["dX"], r["dbias"], b["dX"]

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in range(4):
        x.copy_(rows((T, hidden), BF16, seed, 0.3).to(DEV))
        dy.copy_(rows((T, hidden), BF16, seed + 50, 0.1).to(DEV))
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, call()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_decode_step_with_the_cache(nv):
    """A layer's decode step: projections of the new tokens, the cache's append and attention over it, the output
    projection onto the residual and the feed-forward block; captured, and equal to the eager step."""
    heads, group, dim, hidden, inner, n = 2, 2, 64, 256, 192, 3
    q, k, v, o = (Weights(1, a, b, s).matrix(nv) for a, b, s in
                  ((heads * group * dim, hidden, 1), (heads * dim, hidden, 2), (heads * dim, hidden, 3),
                   (hidden, heads * group * dim, 4)))
    ffn = [Weights(1, a, b, s).matrix(nv) for a, b, s in ((inner, hidden, 5), (inner, hidden, 6), (hidden, inner, 7))]
    S = torch.full((1, heads), 0.02, device=DEV)
    cache = nv.KVCache.empty(1, 12, heads, dim, 16, 4, 3, S, S)
    cache.pages.zero_()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    cu, slots, one = i32([0, 1, 2, 3]), i32([2, 0, 1]), i32([1, 1, 1])
    x = rows((n, hidden), BF16, 9, 0.3).to(DEV)

    def layer():
        nv.kv_append(cache, 0, nv.linear(k, x).view(n, heads, dim), nv.linear(v, x).view(n, heads, dim), cu, slots)
        a, _ = nv.kv_attention(cache, 0, nv.linear(q, x).view(n, heads * group, dim), cu, slots, max_q=1)
        y = nv.linear(o, a.view(n, -1), residual=x)
        return nv.linear(ffn[2], nv.gated(ffn[0], ffn[1], y), residual=y)

    assert nv.kv_reserve(cache, slots, one).item() == nv.KV_DONE
    eager = layer().clone()
    assert torch.isfinite(eager).all() and not torch.equal(eager, x)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = layer()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_matrix_of_a_search(nv):
    """What the search returns goes into a product as it is: the layer's output is off by what output_error says."""
    g = torch.Generator(device=DEV).manual_seed(1)
    W = (torch.randn((96, 256), generator=g, device=DEV) * 0.02).to(BF16)
    X = torch.randn((64, 256), generator=g, device=DEV).to(BF16)
    S = nv.global_scale(W)
    q = nv.scale_search(W, None, S, nv.MSE, -3, 7)
    m = nv.Matrix(q["packed"], q["scales"], S)
    err = nv.output_error(X, W, q["packed"], q["scales"], S)
    off = (nv.linear(m, X.float()).double() - X.double() @ W.double().t()).square().sum(0)
    assert torch.allclose(off, err, rtol=1e-3)               # output_error itself holds 16 bits of each weight's error


def test_binding_refusals(nv):
    w = Weights(1, 32, 64, 1)
    m, x = w.matrix(nv, squeeze=True), rows((4, 64), BF16, 1).to(DEV)
    d = rows((4, 32), BF16, 2).to(DEV)
    for bad in (x.half(), x.double()):
        with pytest.raises(TypeError):
            nv.linear(m, bad)
    with pytest.raises(ValueError):
        nv.linear(m, x[:, :48])
    with pytest.raises(ValueError):
        nv.linear(m, x.t())
    with pytest.raises(ValueError):
        nv.linear(m, x, residual=d[:3])
    with pytest.raises(TypeError):
        nv.linear(m, x, residual=d.float())
    with pytest.raises(TypeError):
        nv.linear(m, x, seg_offsets=torch.tensor([0, 4], dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        nv.linear(m, x, seg_offsets=torch.tensor([0, 2, 4], device=DEV))
    with pytest.raises(ValueError):
        nv.linear(m, x, bias=d[0, :31])
    with pytest.raises(nv.Nvfp4Error):
        nv.linear(m, x, activation=9)
    with pytest.raises(nv.Nvfp4Error):
        nv.linear_backward(m, d, activation=nv.ACT_SILU)           # no Z
    with pytest.raises(nv.Nvfp4Error):
        nv.gated(m, Weights(1, 48, 64, 1).matrix(nv), x)
    with pytest.raises(nv.Nvfp4Error):
        nv.linear(Weights(2, 32, 64, 1).matrix(nv), x)             # a batch needs seg_offsets
    with pytest.raises(TypeError):
        nv.linear(m, x.cpu())
    with pytest.raises(ValueError):
        nv.Matrix(m.packed, m.scales[:16], m.S)
    with pytest.raises(ValueError):
        nv.Matrix(m.packed[:, :16], m.scales[:, :2], m.S)
    with pytest.raises(TypeError):
        nv.Matrix(m.packed, m.scales, m.S.double())
    # no rows: nothing is done
    assert nv.linear(m, x[:0]).shape == (0, 32) and nv.gated(m, m, x[:0]).shape == (0, 32)
    r = nv.linear_backward(m, d[:0], with_bias=True)
    assert r["dX"].shape == (0, 64) and bool((r["dbias"] == 0).all())
    assert nv.gated_backward(m, m, d[:0], d[:0], d[:0])["dX"].shape == (0, 64)
