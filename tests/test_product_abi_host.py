"""Argument errors of the products with NVFP4 matrices: found on the host, before anything is enqueued (no call
here reaches a kernel); workspace sizes; and the 64-bit model of the GPU tests against differences."""
import ctypes
import os

import pytest
import torch

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "block_scale_search_amd", "libnvfp4.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libnvfp4.so not built")

FAKE, ODD = 1 << 20, (1 << 20) + 1           # never dereferenced
BIG = 1 << 60


@pytest.fixture(scope="module")
def n():
    from block_scale_search_amd import nvfp4
    return nvfp4


def _matrix(n, **kw):
    a = dict(packed=FAKE, scales=FAKE, S=FAKE, batch=1, out=40, in_=64, stride=0)
    a.update(kw)
    return ctypes.byref(n.MatrixStruct(**a))


def _linear(n, W=None, **kw):
    a = dict(X=FAKE, dt=1, tokens=4, ldx=64, seg=None, bias=None, act=1, res=FAKE, ldr=40, Z=FAKE, ldz=40, Y=FAKE,
             ldy=40, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return n._lib.nvfp4_linear(_matrix(n) if W is None else W, *a.values(), None)


def _gated(n, W=None, V=None, **kw):
    a = dict(X=FAKE, dt=1, tokens=4, ldx=64, seg=None, act=1, G=FAKE, ldg=40, U=FAKE, ldu=40, H=FAKE, ldh=40,
             ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    W = _matrix(n) if W is None else W
    return n._lib.nvfp4_gated(W, W if V is None else V, *a.values(), None)


def _linear_backward(n, W=None, **kw):
    a = dict(dY=FAKE, dt=1, tokens=4, lddy=40, seg=None, act=1, Z=FAKE, ldz=40, dZ=FAKE, lddz=40, dbias=FAKE,
             dX=FAKE, lddx=64, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return n._lib.nvfp4_linear_backward(_matrix(n) if W is None else W, *a.values(), None)


def _gated_backward(n, W=None, V=None, **kw):
    a = dict(dH=FAKE, dt=1, tokens=4, lddh=40, seg=None, act=1, G=FAKE, ldg=40, U=FAKE, ldu=40, dG=FAKE, lddg=40,
             dU=FAKE, lddu=40, dX=FAKE, lddx=64, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    W = _matrix(n) if W is None else W
    return n._lib.nvfp4_gated_backward(W, W if V is None else V, *a.values(), None)


CALLS = [_linear, _gated, _linear_backward, _gated_backward]

BAD_MATRICES = [
    (dict(out=0), "SHAPE"), (dict(out=-1), "SHAPE"), (dict(in_=0), "SHAPE"), (dict(in_=40), "SHAPE"),
    (dict(in_=-16), "SHAPE"), (dict(batch=-1), "SHAPE"), (dict(batch=65536), "SHAPE"),
    (dict(out=1 << 31), "SHAPE"), (dict(in_=1 << 22, out=1), "SHAPE"), (dict(in_=16, out=1 << 22), "SHAPE"), (dict(out=1 << 27, in_=256), "SHAPE"),
    (dict(batch=2, stride=40 * 64 - 16), "SHAPE"), (dict(batch=2, stride=BIG), "SHAPE"),
    (dict(packed=None), "NULL"), (dict(scales=None), "NULL"), (dict(S=None), "NULL"),
    (dict(packed=FAKE + 4), "ALIGN"), (dict(S=FAKE + 2), "ALIGN"), (dict(batch=2, stride=40 * 64 + 8), "ALIGN")]


@pytest.mark.parametrize("call", CALLS)
def test_matrices(n, call):
    for bad, want in BAD_MATRICES:
        assert call(n, _matrix(n, **bad), seg=FAKE) == getattr(n, "ERR_" + want), bad
    assert call(n, ctypes.POINTER(n.MatrixStruct)()) == n.ERR_NULL
    assert call(n, dt=2) == n.ERR_DTYPE
    assert call(n, act=5) == n.ERR_ARG
    assert call(n, act=-1) == n.ERR_ARG
    assert call(n, tokens=-1) == n.ERR_SHAPE
    assert call(n, tokens=1 << 31) == n.ERR_SHAPE
    assert call(n, _matrix(n, batch=2, stride=4096)) == n.ERR_NULL               # a batch needs seg_offsets
    assert call(n, seg=FAKE + 4) == n.ERR_ALIGN
    # a grid beyond 2^31 workgroups
    assert call(n, _matrix(n, out=1 << 21, in_=8192), tokens=(1 << 31) - 1) == n.ERR_SHAPE
    # nothing to do
    assert call(n, _matrix(n, batch=0)) == n.ERR_NULL
    assert call(n, _matrix(n, batch=0), seg=FAKE) == n.OK


@pytest.mark.parametrize("call", [_gated, _gated_backward])
def test_two_matrices(n, call):
    for other in (dict(out=41), dict(in_=80), dict(batch=2, stride=4096)):
        assert call(n, None, _matrix(n, **other)) == n.ERR_SHAPE
    assert call(n, None, ctypes.POINTER(n.MatrixStruct)()) == n.ERR_NULL
    assert call(n, None, _matrix(n, packed=ODD)) == n.ERR_ALIGN


@pytest.mark.parametrize("call, names", [
    (_linear, {"X": "ldx", "Y": "ldy"}), (_gated, {"X": "ldx", "H": "ldh"}),
    (_linear_backward, {"dY": "lddy", "Z": "ldz", "dZ": "lddz", "dX": "lddx"}),
    (_gated_backward, {"dH": "lddh", "G": "ldg", "U": "ldu", "dG": "lddg", "dU": "lddu", "dX": "lddx"})])
def test_row_tensors(n, call, names):
    for name, ld in names.items():
        assert call(n, **{name: None}) == n.ERR_NULL, name
        assert call(n, **{name: ODD}) == n.ERR_ALIGN, name
        assert call(n, **{ld: 39}) == n.ERR_SHAPE, name
        assert call(n, **{ld: BIG}) == n.ERR_SHAPE, name


def test_optional_row_tensors(n):
    for name, ld in (("res", "ldr"), ("Z", "ldz")):
        assert _linear(n, **{name: ODD}) == n.ERR_ALIGN
        assert _linear(n, **{ld: 39}) == n.ERR_SHAPE
    assert _linear(n, bias=ODD) == n.ERR_ALIGN
    assert _gated(n, G=None) == n.ERR_NULL and _gated(n, U=None) == n.ERR_NULL       # both or neither
    assert _linear_backward(n, dbias=FAKE + 2) == n.ERR_ALIGN
    # rows that the products read 16 bytes at a time
    assert _linear(n, ldx=68) == n.ERR_ALIGN and _linear(n, X=FAKE + 8) == n.ERR_ALIGN
    assert _linear(n, dt=0, ldx=66) == n.ERR_ALIGN
    assert _linear_backward(n, act=0, lddy=44) == n.ERR_ALIGN
    assert _linear_backward(n, lddz=44) == n.ERR_ALIGN
    assert _gated_backward(n, lddg=48) == n.ERR_SHAPE                            # dG and dU unlike
    assert _linear(n, ldx=1 << 22) == n.ERR_SHAPE
    assert _gated_backward(n, lddg=44) == n.ERR_ALIGN and _gated_backward(n, dU=FAKE + 2) == n.ERR_ALIGN


def test_workspaces(n):
    bf16, f32 = torch.bfloat16, torch.float32
    assert n.nvfp4_linear_workspace_size(bf16, 100, 1, 40, 64) == 0
    assert n.nvfp4_gated_workspace_size(bf16, 100, 1, 40, 64) == 0
    for size in (n.nvfp4_linear_workspace_size, n.nvfp4_gated_workspace_size):
        assert size(f32, 100, 1, 40, 64) >= 3 * 2 * 100 * 64
        assert size(f32, 0, 1, 40, 64) == 0 and size(f32, 100, 1, 40, 65) == 0 and size(f32, -1, 1, 40, 64) == 0
    back = n.nvfp4_linear_backward_workspace_size
    assert back(bf16, 100, 1, 40, 64, False) == 0
    assert back(bf16, 100, 1, 41, 64, False) >= 2 * 100 * 48
    assert back(bf16, 100, 3, 40, 64, True) >= 4 * 3 * 40
    assert n.nvfp4_gated_backward_workspace_size(f32, 100, 1, 40, 64) >= 2 * 3 * 2 * 100 * 40
    assert back(bf16, 100, 0, 40, 64, True) >= 0 and back(f32, 0, 0, 40, 64, True) >= 0      # no matrix
    with pytest.raises(TypeError):
        n.nvfp4_linear_workspace_size(torch.float16, 100, 1, 40, 64)
    # short, missing, misaligned
    need = n.nvfp4_linear_workspace_size(f32, 4, 1, 40, 64)
    assert _linear(n, dt=0, ws=None) == n.ERR_WORKSPACE and _linear(n, dt=0, ws_bytes=need - 1) == n.ERR_WORKSPACE
    assert _linear(n, dt=0, ws=FAKE + 8) == n.ERR_ALIGN
    assert _gated(n, dt=0, ws_bytes=need - 1) == n.ERR_WORKSPACE
    need = back(bf16, 4, 1, 40, 64, True)
    assert _linear_backward(n, ws_bytes=need - 1) == n.ERR_WORKSPACE
    need = n.nvfp4_gated_backward_workspace_size(f32, 4, 1, 40, 64)
    assert _gated_backward(n, dt=0, ws_bytes=need - 1) == n.ERR_WORKSPACE


def test_empty_calls(n):
    assert _linear(n, tokens=0, X=None, Y=None, res=None, Z=None) == n.OK
    assert _gated(n, tokens=0, X=None, H=None) == n.OK
    assert _linear_backward(n, tokens=0, dY=None, dX=None, dbias=None) == n.OK
    assert _gated_backward(n, tokens=0, dH=None, dX=None) == n.OK


def test_binding_refuses_host_tensors(n):
    with pytest.raises(TypeError):
        n.Matrix(torch.zeros((4, 8), dtype=torch.uint8), torch.zeros((4, 1), dtype=torch.uint8), torch.ones(1))


def test_model_gradients_by_differences():
    """The 64-bit slopes and input gradients that the GPU tests use, against central differences."""
    from product_helpers import ACTS, Weights, act_model, product, spans
    g = torch.Generator().manual_seed(1)
    z = torch.randn(200, generator=g, dtype=torch.float64) * 3
    h = 1e-6
    for name in ACTS:
        slope = act_model(z, name)[1]
        diff = (act_model(z + h, name)[0] - act_model(z - h, name)[0]) / (2 * h)
        assert torch.allclose(slope, diff, rtol=0, atol=1e-7), name
    counts, w, v = [2, 0, 3], Weights(3, 7, 32, 1), Weights(3, 7, 32, 2)
    x, d = torch.randn((5, 32), generator=g, dtype=torch.float64), torch.randn((5, 7), generator=g, dtype=torch.float64)

    def loss(x):
        gate, up = product(x, w, counts)[0], product(x, v, counts)[0]
        return (act_model(gate, "silu")[0] * up * d).sum()

    gate, up = product(x, w, counts)[0], product(x, v, counts)[0]
    a, slope = act_model(gate, "silu")
    dx = product(d * up * slope, w, counts, False)[0] + product(d * a, v, counts, False)[0]
    for t, i in ((0, 0), (1, 31), (2, 5), (4, 17)):
        e = torch.zeros_like(x)
        e[t, i] = h
        assert abs((loss(x + e) - loss(x - e)) / (2 * h) - dx[t, i]) <= 1e-5 * (1 + dx[t, i].abs())
    assert [e for e, _ in spans(counts)] == [0, 2]


@pytest.mark.parametrize("call, rows", [(_linear, "X"), (_gated, "X"), (_linear_backward, "dY"), (_gated_backward, "dH")])
def test_launches_beyond_32_bits(n, call, rows):
    most = ((1 << 32) - 256) // 8                        # 8 pieces of 8 columns a row
    assert call(n, tokens=most, **{rows: None}) == n.ERR_NULL
    assert call(n, tokens=most + 1, **{rows: None}) == n.ERR_SHAPE
    many = dict(batch=65535, in_=16)
    assert call(n, _matrix(n, out=1 << 17, stride=1 << 21, **many), seg=FAKE) == n.ERR_SHAPE          # biases
    if call in (_linear, _gated):                        # tiles of 4 rows by 16
        assert call(n, _matrix(n, out=1 << 15, stride=1 << 19, **many), tokens=65536, seg=FAKE) == n.ERR_SHAPE
