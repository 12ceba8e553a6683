"""A 64-bit model of the products with NVFP4 matrices, on the CPU, and the tensors that the tests give to it and
to the library."""
import math

import torch

import oracle

DEV = "cuda"
ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu")
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}

_LEVELS = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
_E4M3 = torch.tensor([oracle.e4m3_value(c) if c else 0.0 for c in range(127)], dtype=torch.float64)


def act(nv, name):
    return {"none": nv.ACT_NONE, "silu": nv.ACT_SILU, "gelu": nv.ACT_GELU, "gelu_tanh": nv.ACT_GELU_TANH,
            "relu": nv.ACT_RELU}[name]


class Weights:
    """`batch` matrices: codes, scale bytes and S on the CPU, and their values in 64 bits. whole: scales
    and S are powers of two near 1, so that products with small whole numbers sum without rounding."""

    def __init__(self, batch, out, inp, seed, whole=False):
        g = torch.Generator().manual_seed(seed)
        self.shape = (batch, out, inp)
        self.packed = torch.randint(0, 256, (batch, out, inp // 2), generator=g, dtype=torch.uint8)
        if whole:
            pick = torch.tensor([48, 56, 64], dtype=torch.uint8)             # 0.5, 1, 2
            self.scales = pick[torch.randint(0, 3, (batch, out, inp // 16), generator=g)]
            self.S = 2.0 ** torch.randint(-2, 2, (batch,), generator=g).float()
        else:
            self.scales = torch.randint(0, 127, (batch, out, inp // 16), generator=g, dtype=torch.uint8)
            self.scales[torch.rand(self.scales.shape, generator=g) < 0.9] //= 2
            self.S = (0.5 + torch.rand(batch, generator=g)) * 2.0 ** -5
        code = torch.stack([self.packed & 15, self.packed >> 4], -1).flatten(-2).long()
        scale = _E4M3[self.scales.long()].repeat_interleave(16, -1)
        self.values = _LEVELS[code] * scale * self.S.double()[:, None, None]

    def matrix(self, nv, squeeze=False):
        p, s = self.packed.to(DEV), self.scales.to(DEV)
        return nv.Matrix(p[0], s[0], self.S.to(DEV)) if squeeze else nv.Matrix(p, s, self.S.to(DEV))


def offsets(counts):
    return torch.tensor([0] + list(counts)).cumsum(0)


def spans(counts):
    at = offsets(counts).tolist()
    return [(e, slice(at[e], at[e + 1])) for e in range(len(counts)) if counts[e]]


def product(x, w, counts, transposed=True):
    """x times each row's matrix (transposed: x [T, in], else x [T, out]), and the sums of magnitudes."""
    x = x.double()
    y = torch.zeros((x.shape[0], w.shape[1 if transposed else 2]), dtype=torch.float64)
    size = torch.zeros_like(y)
    for e, r in spans(counts):
        v = w.values[e].t() if transposed else w.values[e]
        y[r] = x[r] @ v
        size[r] = x[r].abs() @ v.abs()
    return y, size


def by_row(t, counts):
    return torch.repeat_interleave(t.double(), torch.tensor(list(counts)), 0)


def act_model(z, name):
    """act(z), act'(z)."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)


def sum_error(size, terms, dtype):
    """Binary32 sums of exact products: each addition is off by at most a step (2^-23, the matrix unit may
    truncate) of a partial sum, which is at most `size`; binary32 rows enter as three parts of a value. The
    scaling by S, a bias and a change of matrix add three more roundings."""
    parts = 3 if dtype == torch.float32 else 1
    return (parts * terms + 4) * 2.0 ** -23 * size


def act_error(z, dtype):
    """How far act(z) may be off for exact z. bf16: the exponential's argument is rounded (|z| 2^-23 of its
    value) and exponential, reciprocal and the products are a few steps off; erfc, exp and tanh's form in
    binary32 are off by less than 8 steps of values up to 1 (or |z|) and of the cubic's argument."""
    return (z.abs() + 1) * (z.abs() + 8) * 2.0 ** -22


def close(got, want, error, dtype, what):
    got = got.cpu().double()
    room = error + (want.abs() + error) * HALF_STEP[dtype] + 1e-37
    bad = ~((got - want).abs() <= room)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0].item()} for {want[bad][0].item()} +- {room[bad][0].item()}")


def rows(shape, dtype, seed, scale=1.0, whole=False):
    g = torch.Generator().manual_seed(seed)
    if whole:
        return torch.randint(-4, 5, shape, generator=g).to(dtype)
    return (torch.randn(shape, generator=g) * scale).to(dtype)
