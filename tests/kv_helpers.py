"""Plain 64-bit models of the paged NVFP4 key/value cache for its tests: the cached values read through
the documented record layout, attention over them, and the page bookkeeping on host lists."""
import math

import torch

DEV = "cuda"
LEVELS = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
E4M3 = torch.tensor([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                     for e in range(16) for m in range(8)] * 2, dtype=torch.float64)


def regions(cache, layer):
    """Host views (K codes [N,H,P,D/2], V codes [N,H,P/4,16,4,E], K scales, V scales)."""
    H, P, D = cache.heads, cache.page_size, cache.head_dim
    rec = cache.pages[layer].cpu()[:, :H * P * D * 9 // 8]
    a, b = H * P * D // 2, H * P * D // 16
    n = rec.shape[0]
    return (rec[:, :a].reshape(n, H, P, D // 2),
            rec[:, a:2 * a].reshape(n, H, P // 4, 16, 4, D // 32),
            rec[:, 2 * a:2 * a + b].reshape(n, H, P, D // 16),
            rec[:, 2 * a + b:].reshape(n, H, P // 4, D // 16, 4))


def plain_codes(cache, layer):
    """Codes [N,H,P,D/2] and scale bytes [N,H,P,D/16] of K and of V in token order."""
    kc, vc, ks, vs = regions(cache, layer)
    vc = vc.permute(0, 1, 2, 4, 3, 5).reshape(kc.shape)
    vs = vs.permute(0, 1, 2, 4, 3).reshape(ks.shape)
    return kc, ks, vc, vs


def values(codes, scales, S):
    """float64 level * E4M3 * S, S [H]."""
    c = codes.long()
    v = torch.stack([LEVELS[c & 15], LEVELS[c >> 4]], -1).flatten(-2)
    e = E4M3[scales.long() & 127] * S.double().cpu()[None, :, None, None]
    return (v.unflatten(-1, (-1, 16)) * e[..., None]).flatten(-2)


def cached(cache, layer, slot, n):
    """float64 K, V [n, H, D] of positions 0..n-1 of a slot, and which of them are in the cache."""
    P = cache.page_size
    kc, ks, vc, vs = plain_codes(cache, layer)
    t = torch.arange(n)
    page = cache.table.cpu()[slot, t // P].long()
    ok = (page >= 0) & (page < cache.num_pages)
    page = page.clamp(0, max(cache.num_pages - 1, 0))
    at = (page, slice(None), t % P)
    out = []
    for c, s, S in ((kc, ks, cache.S_k[layer]), (vc, vs, cache.S_v[layer])):
        out.append(values(c[at][:, :, None], s[at][:, :, None], S)[:, :, 0])
    return out[0], out[1], ok


def attention(cache, layer, Q, cu, slots, scale, causal, window):
    """float64 (out, lse) and, for tolerances, sum p |v| per value, the largest scale * sum |q k| of a
    visible position per row, and the visible positions' sum |v| per value."""
    T, HQ, D = Q.shape
    G = HQ // cache.heads
    q = Q.double().cpu()
    out = torch.zeros((T, HQ, D), dtype=torch.float64)
    mag = torch.zeros_like(out)
    every = torch.zeros_like(out)
    lse = torch.full((T, HQ), -math.inf, dtype=torch.float64)
    big = torch.zeros((T, HQ), dtype=torch.float64)
    for i, s in enumerate(slots):
        a, b = int(cu[i]), int(cu[i + 1])
        if not 0 <= s < cache.table.shape[0] or a == b:
            continue
        n = min(max(int(cache.lens[s]), 0), cache.table.shape[1] * cache.page_size)
        k, v, ok = cached(cache, layer, s, n)
        pos = torch.arange(n - (b - a), n)[:, None]
        p = torch.arange(n)[None]
        see = ok[None].expand(b - a, n)
        if causal:
            see = see & (p <= pos)
        if window:
            see = see & (p > pos - window)
        for j in range(HQ):
            kh, vh = k[:, j // G], v[:, j // G]
            x = (q[a:b, j] @ kh.T * scale).masked_fill(~see, -math.inf)
            m = x.amax(1, keepdim=True) if n else torch.full((b - a, 1), -math.inf)
            w = (x - torch.where(m == -math.inf, 0.0, m)).exp()
            l = w.sum(1, keepdim=True)
            w = w / torch.where(l == 0, 1.0, l)
            out[a:b, j] = w @ vh
            mag[a:b, j] = w @ vh.abs()
            every[a:b, j] = see.double() @ vh.abs()
            lse[a:b, j] = (m + l.log())[:, 0]
            if n:
                big[a:b, j] = (q[a:b, j].abs() @ kh.abs().T * scale).masked_fill(~see, 0).amax(1)
    return out, lse, mag, big, every


def check_attention(got, lse, want, what=""):
    """The kernel against the 64-bit model, with the error of its arithmetic:
      logits    binary32 sums of D products (and of the f16 halves): at most (D + 16) 2^-24 of the
                row's largest sum |q k|, plus 2^-22 of the f32 query's split; a relative error of
                twice that in every probability, and 2^-22 of it from the exponential
      weights   rounded to f16 for bf16 outputs (2^-11), split into two halves for f32 (2^-21)
                and, scaled so that the row's largest is 2^15 or, while the maximum rises, at least
                2^7, off by half of f16's least step, 2^-25: 2^-32 of the largest weight (which is
                at most the sum of weights) for every visible position
      sums      binary32 over N positions, at most N/8 + 64 roundings of 2^-24 one after another
      output    rounded once: 2^-8 (bf16) or 2^-24 (f32) of the value."""
    out, ref_lse, mag, big, every = want
    D, bf16 = out.shape[-1], got.dtype == torch.bfloat16
    g, e = got.double().cpu(), lse.double().cpu()
    dl = big * ((D + 16) * 2.0 ** -24 + (0 if bf16 else 2.0 ** -22))
    n_terms = 2.0 ** -24 * (check_attention.positions / 8 + 64)
    rel = torch.expm1(2 * dl) + 2.0 ** -22 + 2 * n_terms + (2.0 ** -11 if bf16 else 2.0 ** -21)
    tol = (2.0 ** -8 if bf16 else 2.0 ** -24) * out.abs() * 1.01 + rel[..., None] * mag + 2.0 ** -32 * every
    bad = ((g - out).abs() > tol) | ~torch.isfinite(g)
    assert not bad.any(), f"{what}: {int(bad.sum())} outputs off, worst " \
        f"{float(((g - out).abs() / tol.clamp(min=1e-300)).max()):.2f} of the tolerance"
    empty = torch.isinf(ref_lse)
    assert torch.equal(empty, e == -math.inf), f"{what}: rows without a position"
    err = (e - ref_lse)[~empty].abs()
    lim = (dl + n_terms + 2.0 ** -21 + 2.0 ** -22 * ref_lse.abs())[~empty]
    assert bool((err <= lim).all()), f"{what}: lse off by {float((err / lim).max()):.2f} of the tolerance"


check_attention.positions = 1 << 13


class Pool:
    """The page calls on host lists."""

    def __init__(self, num_pages, page, max_slots, max_pages):
        self.page, self.max_pages = page, max_pages
        self.refs = [0] * num_pages
        self.rows = [[] for _ in range(max_slots)]
        self.lens = [0] * max_slots

    def _free(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def _known(self, slots):
        return all(0 <= s < len(self.rows) for s in slots) and len(set(slots)) == len(slots)

    def reserve(self, slots, counts):
        if not self._known(slots):
            return 1
        if any(c < 0 or self.lens[s] + c > self.max_pages * self.page for s, c in zip(slots, counts)):
            return 2
        need = [-(-(self.lens[s] + c) // self.page) - len(self.rows[s]) for s, c in zip(slots, counts)]
        free = self._free()
        if sum(need) > len(free):
            return 3
        for s, c, k in zip(slots, counts, need):
            for p in free[:k]:
                self.refs[p] = 1
            self.rows[s] += free[:k]
            del free[:k]
            self.lens[s] += c
        return 0

    def fork(self, parents, children):
        """Status and the copied (from, to) pages."""
        if not self._known(children) or any(not 0 <= p < len(self.rows) or p in children for p in parents) \
                or any(self.lens[c] for c in children):
            return 1, []
        free = self._free()
        if sum(self.lens[p] % self.page > 0 for p in parents) > len(free):
            return 3, []
        copies = []
        for p, c in zip(parents, children):
            row = list(self.rows[p])
            if self.lens[p] % self.page:
                copies.append((row[-1], free[0]))
                row[-1] = free.pop(0)
            for q in row:
                self.refs[q] += 1
            self.rows[c], self.lens[c] = row, self.lens[p]
        return 0, copies

    def free(self, slots):
        if not self._known(slots):
            return 1
        for s in slots:
            for p in self.rows[s]:
                self.refs[p] -= 1
            self.rows[s], self.lens[s] = [], 0
        return 0

    def compact(self):
        """Used pages and the moves (from, to)."""
        used = [i for i, r in enumerate(self.refs) if r > 0]
        U = len(used)
        holes = [i for i in range(U) if self.refs[i] == 0]
        moves = list(zip([i for i in used if i >= U], holes))
        to = dict(moves)
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        return U, moves

    def check(self, cache, what=""):
        t = torch.full(cache.table.shape, -1, dtype=torch.int32)
        for s, r in enumerate(self.rows):
            t[s, :len(r)] = torch.tensor(r, dtype=torch.int32)
        assert cache.lens.tolist() == self.lens, f"{what}: lens"
        assert cache.refs.tolist() == self.refs, f"{what}: refs"
        assert torch.equal(cache.table.cpu(), t), f"{what}: table"


def i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


def make_cache(nv, lens, heads, dim, page, layers=1, extra_pages=3, extra_slots=0, seed=0, width=None):
    """A cache whose slots have these lengths, pages scattered, with random S. Its records are filled with
    255, which is no scale byte and no state that a call may leave in a result."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-n // page) for n in lens]
    num_pages = sum(held) + extra_pages
    width = max(held + [1]) if width is None else width
    S = [(0.003 + 0.01 * torch.rand((layers, heads), generator=g)).to(DEV) for _ in range(2)]
    c = nv.KVCache.empty(layers, num_pages, heads, dim, page, len(lens) + extra_slots, width, *S)
    c.pages.fill_(255)
    order = torch.randperm(num_pages, generator=g).to(torch.int32)
    at = 0
    for s, k in enumerate(held):
        c.table[s, :k] = order[at:at + k].to(DEV)
        c.refs[order[at:at + k].long().to(DEV)] = 1
        at += k
    c.lens[:len(lens)] = i32(lens)
    return c


def fill_cache(nv, cache, lens, seed=0, layer=0, dtype=torch.bfloat16):
    """Appends normal rows for every position of the slots 0..len(lens)-1."""
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    T = sum(lens)
    k = torch.randn((T, cache.heads, cache.head_dim), generator=g, device=DEV)
    v = torch.randn((T, cache.heads, cache.head_dim), generator=g, device=DEV)
    cu = i32([0] + torch.tensor(lens).cumsum(0).tolist())
    nv.kv_append(cache, layer, k.to(dtype), v.to(dtype), cu)
