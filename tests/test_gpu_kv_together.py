"""The cache's calls together, as a serving loop makes them: prompts, decode steps, a fork, a slot freed
and a compaction, over two layers; and a decode step captured in a graph and replayed."""
import pytest
import torch

from kv_helpers import DEV, attention, check_attention, i32

pytestmark = pytest.mark.gpu

L, H, G, D, P = 2, 2, 4, 128, 16


def _rows(n, heads, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn((n, heads, D), generator=g, device=DEV).to(torch.bfloat16)


def _cache(nv, pages=64, slots=6, width=12):
    S = [torch.full((L, H), s, device=DEV) for s in (0.004, 0.006)]
    return nv.KVCache.empty(L, pages, H, D, P, slots, width, *S)


def _step(nv, c, slots, new, seed):
    """Room, then every layer's append and attention; checked against the 64-bit model."""
    cu = [0] + torch.tensor(new).cumsum(0).tolist()
    assert nv.kv_reserve(c, i32(slots), i32(new)).item() == nv.KV_DONE
    for layer in range(L):
        k, v = _rows(cu[-1], H, seed + layer), _rows(cu[-1], H, seed + layer + 100)
        q = _rows(cu[-1], H * G, seed + layer + 200)
        nv.kv_append(c, layer, k, v, i32(cu), i32(slots))
        out, lse = nv.kv_attention(c, layer, q, i32(cu), i32(slots), max_q=max(new))
        torch.cuda.synchronize()
        check_attention(out, lse, attention(c, layer, q, cu, slots, D ** -0.5, True, 0), f"{new}")


def test_serving_loop(nv):
    c = _cache(nv)
    _step(nv, c, [0, 1, 2], [37, 16, 5], 1)              # prompts
    _step(nv, c, [2, 0, 1], [1, 1, 1], 2)
    assert nv.kv_fork(c, i32([0, 0, 1]), i32([3, 4, 5])).item() == nv.KV_DONE
    _step(nv, c, [0, 1, 2, 3, 4, 5], [1] * 6, 3)         # the copies go their own ways
    assert nv.kv_free(c, i32([0, 2])).item() == nv.KV_DONE
    used = nv.kv_compact(c).item()
    assert used == int((c.refs > 0).sum()) and bool((c.refs[:used] > 0).all())
    _step(nv, c, [1, 3, 4, 5], [1, 4, 2, 1], 4)          # drafts of several tokens
    _step(nv, c, [0, 3], [20, 1], 5)                     # a new prompt beside a running slot
    assert nv.kv_free(c, i32(range(6))).item() == nv.KV_DONE
    assert bool((c.refs == 0).all()) and bool((c.table == -1).all())


def test_graph_of_a_decode_step(nv):
    """Reserve, append and attention of a step in one graph, with the program's eager work between the
    replays; each replay equals the eager calls on a copy of the cache."""
    slots, new = [1, 0, 3], [1, 1, 1]
    cu, sl, one = i32([0, 1, 2, 3]), i32(slots), i32(new)
    c, e = _cache(nv), _cache(nv)
    for x in (c, e):
        x.pages.zero_()
        assert nv.kv_reserve(x, i32([0, 1, 3]), i32([30, 100, 15])).item() == nv.KV_DONE
        first = i32([0, 30, 130, 145])
        for layer in range(L):
            nv.kv_append(x, layer, _rows(145, H, 7), _rows(145, H, 8), first, i32([0, 1, 3]))
    K, V, Q = (torch.zeros((3, h, D), dtype=torch.bfloat16, device=DEV) for h in (H, H, H * G))

    def step(x):
        outs = [nv.kv_reserve(x, sl, one)]
        for layer in range(L):
            nv.kv_append(x, layer, K, V, cu, sl)
            outs += nv.kv_attention(x, layer, Q, cu, sl, max_q=1)
        return outs

    side = torch.cuda.Stream()
    keep = [t.clone() for t in (c.table, c.lens, c.refs)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c)                                           # warm-up, then taken back
    torch.cuda.synchronize()
    for t, k in zip((c.table, c.lens, c.refs), keep):
        t.copy_(k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        outs = step(c)
    torch.cuda.synchronize()
    for rep in range(20):                                 # past page borders
        for t, h in ((K, H), (V, H), (Q, H * G)):
            t.copy_(_rows(3, h, 50 + rep + h))
        for t in outs:
            t.fill_(3)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = step(e)
        torch.cuda.synchronize()
        assert outs[0].item() == 0
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), f"replay {rep}"
        for a, b in ((c.table, e.table), (c.lens, e.lens), (c.refs, e.refs)):
            assert torch.equal(a, b), f"replay {rep}"


def test_two_streams_two_workspaces(nv):
    """Two attention calls over one cache at once, on streams and workspaces of their own."""
    c = _cache(nv, pages=400, slots=2, width=200)
    assert nv.kv_reserve(c, i32([0, 1]), i32([3000, 2500])).item() == 0
    for layer in range(L):
        nv.kv_append(c, layer, _rows(5500, H, 3), _rows(5500, H, 4), i32([0, 3000, 5500]))
    cu = i32([0, 1, 2])
    q = [_rows(2, H * G, 9), _rows(2, H * G, 10)]
    want = [nv.kv_attention(c, i, q[i], cu) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(nv.kv_attention(c, i, q[i], cu))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
