"""Bias gradients of nvfp4_linear_backward where there are many of them: more than 2^24, with fewer rows than matrices."""
import pytest
import torch

from product_helpers import DEV, act, act_model, close, offsets, rows, sum_error
from product_helpers import _E4M3 as E4M3, _LEVELS as LEVELS

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def matrices(nv, E, out, inp):
    """Random matrices, made on the GPU."""
    g = torch.Generator(device=DEV).manual_seed(E + out)
    p = torch.randint(0, 256, (E, out, inp // 2), generator=g, dtype=torch.uint8, device=DEV)
    s = torch.randint(40, 70, (E, out, inp // 16), generator=g, dtype=torch.uint8, device=DEV)
    return nv.Matrix(p, s, torch.ones(E, device=DEV))


def values(m, e):
    """Matrix e's weights [out, in] in 64 bits, on the CPU."""
    p, s = m.packed[e].cpu(), m.scales[e].cpu()
    code = torch.stack([p & 15, p >> 4], -1).flatten(-2).long()
    return LEVELS[code] * E4M3[s.long()].repeat_interleave(16, -1) * m.S[e].double().cpu()


def backward(nv, m, d, name, z, seg, dbias):
    """nvfp4_linear_backward into a dbias that is there before."""
    T = d.shape[0]
    dX = torch.empty((T, m.inp), dtype=d.dtype, device=DEV)
    dZ = torch.empty_like(d) if name != "none" else None
    need = nv.nvfp4_linear_backward_workspace_size(d.dtype, T, m.batch, m.out, m.inp, True)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    nv.nvfp4_linear_backward(m, d, T, seg, act(nv, name), z if name != "none" else None, dZ, dbias, dX, ws)
    return dX


# rows of the matrices that have any; out a multiple of 8 and not
CASES = [(1024, 16416, {3: 1, 500: 30, 501: 4, 1023: 5}), (1024, 16416, {0: 40}), (1024, 16416, {}),
         (128, 131080, {0: 70, 64: 20, 127: 10}), (128, 131083, {5: 3}), (8, 2100000, {})]


@pytest.mark.parametrize("dtype", (BF16, F32), ids=("bf16", "f32"))
@pytest.mark.parametrize("name", ("none", "relu"))
@pytest.mark.parametrize("E, out, having", CASES, ids=range(len(CASES)))
def test_many_biases_of_few_rows(nv, E, out, having, name, dtype):
    """Every bias is written, with the exact sum (whole numbers) or zero."""
    counts = [having.get(e, 0) for e in range(E)]
    T, m = sum(counts), matrices(nv, E, out, 16)
    d, z = rows((T, out), dtype, 1, whole=True), rows((T, out), dtype, 2, whole=True)
    dbias = torch.full((E, out), float("nan"), device=DEV)
    backward(nv, m, d.to(DEV), name, z.to(DEV), offsets(counts).to(DEV), dbias)
    at = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))
    dz = d.double() * act_model(z.double(), name)[1]
    want = torch.zeros((E, out), dtype=torch.float64).index_add_(0, at, dz)
    assert torch.equal(dbias.cpu(), want.float())


def test_slopes_and_many_biases_beyond_one_launch(nv):
    """Values by the slopes' pass and bias workgroups that have more than 2^32 threads between them: the call is one of
    those that the sizes allow (the rows that belong to no matrix are never written: what they hold does not matter)."""
    E, out, inp = 65528, 8193, 16
    T = (2 ** 31 - 1) // ((out + 7) // 8)
    assert E * out <= 2 ** 29 and T * ((out + 7) // 8) < 2 ** 31
    assert E * ((out + 63) // 64) * 256 + T * ((out + 7) // 8) > 2 ** 32
    m = matrices(nv, E, out, inp)
    having = {0: 3, 40000: 50, E - 1: 4}
    counts = [having.get(e, 0) for e in range(E)]
    n = sum(counts)
    d = torch.empty((T, out), dtype=BF16, device=DEV)
    head = rows((n, out), BF16, 1, whole=True)
    d[:n] = head.to(DEV)
    dbias = torch.full((E, out), float("nan"), device=DEV)
    dX = backward(nv, m, d, "none", None, offsets(counts).to(DEV), dbias)
    at = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))
    for e in having:
        assert torch.equal(dbias[e].cpu(), head[at == e].double().sum(0).float())
        dbias[e] = 0
    assert int(torch.count_nonzero(dbias)) == 0
    for e in having:
        w = values(m, e)
        want, size = head[at == e].double() @ w, head[at == e].double().abs() @ w.abs()
        close(dX[:n].cpu()[at == e], want, sum_error(size, out, BF16), BF16, f"dX of matrix {e}")
    del d, dX, dbias, m
    torch.cuda.empty_cache()
