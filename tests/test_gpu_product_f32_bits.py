"""binary32 rows with all 24 bits in use: one value a row meets weights that are powers of two, so every output is that
value times a power of two, exact in binary32. A product that drops any of a value's bits shows."""
import pytest
import torch

from product_helpers import DEV, Weights, offsets
from product_helpers import _LEVELS as LEVELS

pytestmark = pytest.mark.gpu
F32 = torch.float32


def powers(batch, out, inp, seed):
    """Matrices of zeros and powers of two."""
    w = Weights(batch, out, inp, seed, whole=True)
    w.values = None
    pick = torch.tensor([0, 1, 2, 4, 6, 9, 10, 12, 14], dtype=torch.uint8)           # 0, 0.5, 1, 2, 4, negative ones
    g = torch.Generator().manual_seed(seed)
    code = pick[torch.randint(0, len(pick), (batch, out, inp), generator=g)]
    return set_codes(w, code)


def set_codes(w, code):
    w.code, w.packed = code, code[..., ::2] | code[..., 1::2] << 4
    scale = torch.exp2((w.scales.double() - 56) / 8)                                 # 48, 56, 64: 0.5, 1, 2
    w.values = LEVELS[code.long()] * scale.repeat_interleave(16, -1) * w.S.double()[:, None, None]
    return w


def one_a_row(T, cols, seed):
    """Rows of zeros but for one value, whose mantissa's last bit is set; the column and the value of each."""
    g = torch.Generator().manual_seed(seed)
    bits = torch.randint(0, 1 << 23, (T,), generator=g) | 1
    value = (1 + bits.double() * 2.0 ** -23) * 2.0 ** torch.randint(-30, 30, (T,), generator=g).double()
    value[1::2] *= -1
    at = torch.randint(0, cols, (T,), generator=g)
    at[::3] = cols - 1 - at[::3] % min(cols, 20)                                     # the last ones too
    x = torch.zeros((T, cols), dtype=F32)
    x[torch.arange(T), at] = value.to(F32)
    assert torch.equal(x[torch.arange(T), at].double(), value)
    return x, at, value


def same(got, want, what):
    got, bits = got.cpu(), want.to(F32)
    assert torch.equal(bits.double(), want) and torch.equal(got, bits), what


SIZES = [(T, out, inp) for T in (1, 4, 40, 140, 300) for out, inp in ((70, 1040), (72, 320), (37, 208), (203, 4112))]


@pytest.mark.parametrize("T, out, inp", SIZES + [(300, 4104, 16416)])
def test_forward(nv, T, out, inp):
    w = powers(1, out, inp, 1)
    x, at, value = one_a_row(T, inp, T)
    same(nv.linear(w.matrix(nv), x.to(DEV)), w.values[0].t()[at] * value[:, None], "Y")


@pytest.mark.parametrize("T, out, inp", SIZES)
def test_gated_forward(nv, T, out, inp):
    w, v = powers(1, out, inp, 1), powers(1, out, inp, 2)
    x, at, value = one_a_row(T, inp, T)
    _, g, u = nv.gated(w.matrix(nv), v.matrix(nv), x.to(DEV), with_pre=True)
    same(g, w.values[0].t()[at] * value[:, None], "G")
    same(u, v.values[0].t()[at] * value[:, None], "U")


@pytest.mark.parametrize("T, out, inp", SIZES + [(300, 4104, 16416)])
def test_gradient(nv, T, out, inp):
    w = powers(1, out, inp, 1)
    d, at, value = one_a_row(T, out, T)
    r = nv.linear_backward(w.matrix(nv), d.to(DEV))
    same(r["dX"], w.values[0][at] * value[:, None], "dX")
    z = torch.ones_like(d)
    r = nv.linear_backward(w.matrix(nv), d.to(DEV), Z=z.to(DEV), activation=nv.ACT_RELU)
    same(r["dZ"], d.double(), "dZ")
    same(r["dX"], w.values[0][at] * value[:, None], "dX")


@pytest.mark.parametrize("T, out, inp", SIZES)
def test_gated_gradient(nv, T, out, inp):
    """Each column of dX is of one of the two matrices: the other is zero there."""
    w, v = powers(1, out, inp, 1), powers(1, out, inp, 2)
    w.code[..., 1::2] = 0
    v.code[..., ::2] = 0
    set_codes(w, w.code), set_codes(v, v.code)
    d, at, value = one_a_row(T, out, T)
    g, u = torch.full_like(d, 2.0), torch.full_like(d, -0.5)
    r = nv.gated_backward(w.matrix(nv), v.matrix(nv), d.to(DEV), g.to(DEV), u.to(DEV), activation=nv.ACT_RELU)
    same(r["dG"], -0.5 * d.double(), "dG")
    same(r["dU"], 2 * d.double(), "dU")
    same(r["dX"], (-0.5 * w.values[0][at] + 2 * v.values[0][at]) * value[:, None], "dX")


@pytest.mark.parametrize("counts", ([2, 0, 1, 3], [40, 0, 17, 129], [1, 2] * 80))
def test_experts(nv, counts):
    E, T, out, inp = len(counts), sum(counts), 72, 1040
    w, e = powers(E, out, inp, 3), torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    seg, m = offsets(counts).to(DEV), w.matrix(nv)
    x, at, value = one_a_row(T, inp, 5)
    same(nv.linear(m, x.to(DEV), seg_offsets=seg), w.values[e, :, at] * value[:, None], "Y")
    d, at, value = one_a_row(T, out, 6)
    same(nv.linear_backward(m, d.to(DEV), seg_offsets=seg)["dX"], w.values[e, at] * value[:, None], "dX")
