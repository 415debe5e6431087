"""Tree attention over compressed caches against a plain implementation in 64 bits.

Tolerance, per output row and in the 2-norm (the rotation of the codec keeps it).  With unit
roundoff u of the operands (fp32: 2^-24; bf16 caches compute with fp16 operands: 2^-11) and n
roundings between a stored number and a product,
  a logit is off by at most   E_t = n u ||q|| (||gamma K_a|| + ||r~||) / sqrt(D)
                                    (+ the fp32 sum of D terms: D 2^-24 of the same),
  a probability by the factor exp(2 E) with E the largest E_t (numerator and sum), and
  a value row by               n u (||gamma V_a|| + ||r~||) + u of its weight,
so ||do|| <= sum_t p_t [ (exp(2 E) - 1) ||V_t - o|| + (n + 1) u Vn_t ] + h ||o||, h the half step of
the output's type (bf16: 2^-8, fp32: 2^-24).  n = 3 for the rounded operands (a query or anchor, the
rebuilt row, its scale); for fp32 the sums' 128 terms stand in for it.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from kv_cache_compression_anchorkv_b200 import api, capi
from kv_cache_compression_anchorkv_b200.synthetic import CacheSpec, make_decode_queries, make_layer
from oracle import anchorkv_oracle as O

gpu = pytest.mark.gpu
D = 128


def ancestors(g, batch, T, width=4):
    out = torch.zeros(batch, T, dtype=torch.int64)
    for b in range(batch):
        for t in range(T):
            p = int(torch.randint(max(-1, t - width), t, (1,), generator=g)) if t else -1
            w = (int(out[b, p]) if p >= 0 else 0) & ((1 << 64) - 1) | 1 << t
            out[b, t] = w - (1 << 64) if w >= 1 << 63 else w
    return out


class Problem:
    """Layouts, pages and drafts of one call, with the dense rows in 64 bits."""

    def __init__(self, dtype="bf16", H=2, G=4, N=1500, theta=0.2, B=2, T=5, lens=None, page=16, layouts=None, mode=0,
                 n_new=None, mask="tree", seed=1, q_scale=3.0, prefix=True, spare=2, room=0):
        g = torch.Generator().manual_seed(seed)
        self.p = api.AnchorKVParams(n_tokens=N, n_kv_heads=H, n_q_heads=H * G, theta=theta, dtype=dtype, mode=mode)
        po = O.Params(n_tokens=N, n_kv_heads=H, n_q_heads=H * G, theta=theta, dtype=dtype, mode=mode)
        dt = self.p.torch_dtype
        self.B, self.T, self.H, self.G = B, T, H, G
        L = layouts or B
        self.layout_of = torch.tensor([b % L for b in range(B)], dtype=torch.int32)
        self.comp, self.dense = None, [None] * L
        if prefix:
            images = []
            for i in range(L):
                spec = CacheSpec(1, H, H * G, N, n_dirs=32, dtype=dtype, seed=seed * 100 + i)
                K, V, Q = make_layer(spec, 0)
                out, ws = api.compress(self.p, K.cuda(), V.cuda(), Q.cuda())
                assert api.read_status(ws)[0] == 0
                images.append(out)
                parts = O.unpack_layout(out.cpu().numpy(), po)
                none = dict(parts, codes=np.zeros((0, D), np.uint8))
                full, bare = O.reconstruct(parts, po), O.reconstruct(none, po)
                # dense rows and the norms the rounding bound needs, K then V
                self.dense[i] = [(torch.tensor(f), torch.tensor(np.linalg.norm(a, axis=-1) + np.linalg.norm(f - a, axis=-1)))
                                 for f, a in zip(full, bare)]
            stride = (len(images[0]) + 15) // 16 * 16
            self.comp = torch.zeros(L, stride, dtype=torch.uint8, device="cuda")
            for i, x in enumerate(images):
                self.comp[i, :len(x)] = x
            q = make_decode_queries(CacheSpec(1, H, H * G, N, n_dirs=32, dtype=dtype, seed=seed * 100), 0, 0, B * T)
            self.q = (q.float() * q_scale).to(dt).reshape(B, T, H * G, D)
        else:
            self.q = (q_scale * torch.randn(B, T, H * G, D, generator=g)).to(dt)
        self.Kn, self.Vn = (torch.randn(B, T, H, D, generator=g).to(dt) for _ in range(2))
        self.n_new = None if n_new is None else torch.tensor(n_new, dtype=torch.int32)
        self.mask = ancestors(g, B, T) if isinstance(mask, str) and mask == "tree" else mask
        self.pages = None
        self.lens = lens or [0] * B
        if lens is not None:
            need = [-(-n // page) for n in lens]
            n_pages, maxp = sum(need) + spare, max(max(need), 1) + room
            self.pages = api.PageSpec(n_pages=n_pages, page_size=page, n_slots=B, max_pages=maxp, n_kv_heads=H, dtype=dtype)
            ids = torch.randperm(n_pages, generator=g).tolist()
            state = torch.zeros(self.pages.state_numel, dtype=torch.int32)
            v = api.pages_view(self.pages, state)
            v["table"].fill_(-1)
            for b, k in enumerate(need):
                v["len"][b] = lens[b]
                for j in range(k):
                    v["table"][b, j] = ids.pop()
            self.state = state
            self.Kp, self.Vp = (torch.randn(n_pages, H, page, D, generator=g).to(dt) for _ in range(2))

    def call(self, out=None, **over):
        cu = lambda x: None if x is None else x.cuda()                       # noqa: E731
        kw = dict(n_new=cu(self.n_new), mask=cu(self.mask), layout_of=cu(self.layout_of) if self.comp is not None else None)
        if self.pages is not None:
            kw.update(pages=self.pages, state=self.state.cuda(), K_pages=self.Kp.cuda(), V_pages=self.Vp.cuda())
        args = dict(q=self.q.cuda(), K_new=self.Kn.cuda(), V_new=self.Vn.cuda())
        args.update({k: over.pop(k) for k in list(over) if k in args})
        kw.update(over)
        return api.tree_attn(self.p, self.comp, *args.values(), out=out, **kw)

    def expect(self):
        """(outputs, tolerance of every row's 2-norm) in 64 bits."""
        B, T, H, G = self.B, self.T, self.H, self.G
        want, tol = torch.zeros(B, T, H * G, D, dtype=torch.float64), torch.zeros(B, T, H * G, dtype=torch.float64)
        fp32 = self.p.dtype == "fp32"
        u, n, half = (2.0 ** -24, 128, 2.0 ** -24) if fp32 else (2.0 ** -11, 3, 2.0 ** -8)
        for b in range(B):
            m = T if self.n_new is None else int(self.n_new[b])
            for h in range(H):
                rows = []
                for side in range(2):
                    x, xn = [], []
                    if self.comp is not None:
                        d, dn = self.dense[int(self.layout_of[b])][side]
                        x.append(d[h])
                        xn.append(dn[h])
                    if self.pages is not None and self.lens[b]:
                        pool, P = (self.Kp, self.Vp)[side], self.pages.page_size
                        row = api.pages_view(self.pages, self.state)["table"][b]
                        tail = torch.cat([pool[int(i), h] for i in row[:-(-self.lens[b] // P)]])[:self.lens[b]].double()
                        x.append(tail)
                        xn.append(tail.norm(dim=1))
                    new = (self.Kn, self.Vn)[side][b, :m, h].double()
                    x.append(new)
                    xn.append(new.norm(dim=1))
                    rows.append((torch.cat(x), torch.cat(xn)))
                (K, Kn), (V, Vn) = rows
                before = K.shape[0] - m
                for t in range(m):
                    word = (2 << t) - 1 if self.mask is None else int(self.mask[b, t])
                    seen = torch.tensor([True] * before + [bool(word >> i & 1) for i in range(m)])
                    if not seen.any():
                        continue
                    q = self.q[b, t, h * G:(h + 1) * G].double()
                    s = q @ K[seen].T / math.sqrt(D)
                    pr = torch.softmax(s, 1)
                    o = pr @ V[seen]
                    E = (n * u + D * 2.0 ** -24) * (q.norm(dim=1)[:, None] * Kn[seen]).amax(1) / math.sqrt(D)
                    far = torch.cdist(o, V[seen])
                    want[b, t, h * G:(h + 1) * G] = o
                    tol[b, t, h * G:(h + 1) * G] = (pr * (torch.expm1(2 * E)[:, None] * far + (n + 1) * u * Vn[seen])).sum(1) \
                        + half * o.norm(dim=1)
        return want, tol

    def check(self, out=None):
        got = (self.call() if out is None else out).cpu().double()
        want, tol = self.expect()
        off = (got - want).norm(dim=3)
        assert torch.isfinite(got).all()
        assert (off <= tol).all(), (off / tol.clamp(min=1e-30)).max()
        if want.norm() > 0:                       # and far inside it on the whole
            rel = float((got - want).norm() / want.norm())
            assert rel < (2e-6 if self.p.dtype == "fp32" else 4e-3), rel
        return got


CASES = {
    "one-token": dict(T=1, lens=[37, 0]),
    "one-token-no-tail": dict(T=1, B=1),
    "mha": dict(G=1, H=3, T=7, lens=[5, 130]),
    "gqa3": dict(G=3, H=2, T=6, lens=[64, 31], page=32),
    "gqa16-64-drafts": dict(G=16, H=1, T=64, B=1, lens=[200], page=64, N=700),
    "64-drafts": dict(G=4, H=2, T=64, lens=[129, 1], page=128),
    "33-drafts": dict(G=5, H=1, T=33, B=3, lens=[16, 15, 17], N=900),
    "unequal": dict(T=9, B=4, lens=[0, 1, 50, 16], n_new=[9, 0, 1, 5]),
    "chain": dict(T=12, mask=None, lens=[20, 3]),
    "no-residuals": dict(theta=0.001, lens=[10, 10]),
    "every-residual": dict(theta=1.5, lens=[10, 10]),
    "all-anchors": dict(N=33, theta=0.5, lens=[3, 90], T=3),
    "tile-edge": dict(N=1024, lens=[1, 128], page=128, T=2),
    "tile-edge-1": dict(N=1025, lens=[127, 129], page=64, T=2),
    "naive-codec": dict(mode=api.mode_bits(naive_codec=True), lens=[10, 10]),
    "shared-layout": dict(B=5, layouts=2, T=3, lens=[3, 40, 0, 18, 70]),
    "pages-only": dict(prefix=False, T=4, lens=[1, 77]),
    "drafts-only": dict(prefix=False, T=10, B=2),
    "flat-queries": dict(q_scale=0.01, lens=[9, 300]),
    "sharp-queries": dict(q_scale=20.0, lens=[9, 300]),
    "room-in-the-tables": dict(T=3, B=3, lens=[3, 700, 0], page=64, room=500),
    "room-and-a-short-prefix": dict(N=150, T=2, B=2, lens=[900, 1], page=16, room=3000),
    "long": dict(N=9000, B=1, T=8, lens=[1000], page=64, theta=0.1),
}


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("name", list(CASES))
def test_against_64_bits(name, dtype):
    Problem(dtype=dtype, **CASES[name]).check()


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_rows_without_anything_to_see_are_zero(dtype):
    """No prefix, no tail and an empty mask word; a neighbour that sees something is unaffected."""
    pr = Problem(dtype=dtype, prefix=False, T=6, B=2)
    pr.mask[0, 2] = 0
    pr.mask[1, 5] = 1 << 40                     # only bits behind the drafts
    got = pr.check()
    assert (got[0, 2] == 0).all() and (got[1, 5] == 0).all()


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_rows_behind_the_drafts_stay(dtype):
    pr = Problem(dtype=dtype, T=7, B=3, lens=[3, 3, 3], n_new=[7, 0, 2])
    out = torch.full(pr.q.shape, 5.0, dtype=pr.p.torch_dtype, device="cuda")
    pr.call(out=out)
    assert (out[1] == 5).all() and (out[2, 2:] == 5).all()
    assert not (out[0] == 5).all(dim=-1).any() and not (out[2, :2] == 5).all(dim=-1).any()


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), "lowest"])
def test_masked_drafts_may_hold_anything(dtype, bad):
    """Row 3 is seen by row 3 alone: whatever it holds, the others are what they were."""
    pr = Problem(dtype=dtype, T=6, B=1, lens=[5])
    pr.mask[0] = torch.tensor([1, 3, 5, 15, 19, 33])
    clean = pr.call()
    value = torch.finfo(pr.p.torch_dtype).min if bad == "lowest" else bad
    pr.Kn[0, 3, :, ::3] = value
    pr.Vn[0, 3, :, 1::5] = value
    got = pr.call()
    keep = [0, 1, 2, 4, 5]
    assert torch.equal(got[0, keep], clean[0, keep])
    if bad != "lowest":
        assert not torch.isfinite(got[0, 3]).all()
    # drafts behind n_new and rows of the pool behind the tail are never seen
    pr = Problem(dtype=dtype, T=6, B=1, lens=[5], n_new=[3])
    clean = pr.call()
    pr.Kn[0, 3:], pr.Vn[0, 3:] = value, value
    first = int(api.pages_view(pr.pages, pr.state)["table"][0, 0])
    pr.Kp[first, :, 5:], pr.Vp[first, :, 5:] = value, value
    others = [i for i in range(pr.pages.n_pages) if i != first]
    pr.Kp[others], pr.Vp[others] = value, value
    assert torch.equal(pr.call()[0, :3], clean[0, :3])


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_infinite_values_that_are_seen(dtype):
    """An infinity in a seen value makes its coordinate infinite for the rows that see it, and no other."""
    pr = Problem(dtype=dtype, T=4, B=1, lens=[5])
    pr.mask[0] = torch.tensor([1, 3, 4, 8])
    clean = pr.call()
    pr.Vn[0, 1, 0, 7] = float("inf")
    got = pr.call()
    assert (got[0, 1, :pr.G, 7] == float("inf")).all()
    got[0, 1, :pr.G, 7] = clean[0, 1, :pr.G, 7]
    assert torch.equal(got, clean)


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e6, 1e18])
def test_magnitudes(dtype, scale):
    """Values far from one, and tails that differ from the prefix by as much."""
    pr = Problem(dtype=dtype, T=3, lens=[40, 7])
    pr.Vp = (pr.Vp.float() * scale).to(pr.p.torch_dtype)
    pr.Vn = (pr.Vn.float() * scale).to(pr.p.torch_dtype)
    got = pr.call().cpu().double()
    want, tol = pr.expect()
    assert ((got - want).norm(dim=3) <= tol).all()
    pr = Problem(dtype=dtype, T=3, lens=[40, 7])
    pr.Vp[0, :, 3] = (pr.Vp[0, :, 3].float() * scale).to(pr.p.torch_dtype)
    got = pr.call().cpu().double()
    want, tol = pr.expect()
    assert ((got - want).norm(dim=3) <= tol).all()


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [1, 8, 40])
@pytest.mark.parametrize("up", [True, False])
def test_logits_and_values_that_keep_growing(dtype, T, up):
    """Every tile's logits and values are larger than all before (or smaller), by far more than a reference holds."""
    pr = Problem(dtype=dtype, T=T, B=1, lens=[1500], page=64, N=300, q_scale=1.0)
    table = api.pages_view(pr.pages, pr.state)["table"][0]
    g = torch.Generator().manual_seed(3)
    u = torch.randn(D, generator=g)
    q = pr.q.float()
    pr.q = (0.3 * q + u).to(pr.p.torch_dtype)
    for j, page in enumerate(table.tolist()):
        step = j if up else len(table) - j
        pr.Kp[page] = (0.05 * pr.Kp[page].float() + step * u).to(pr.p.torch_dtype)
        pr.Vp[page] = (pr.Vp[page].float() * 2.0 ** (3 * step)).to(pr.p.torch_dtype)
    got = pr.call().cpu().double()
    want, tol = pr.expect()
    assert ((got - want).norm(dim=3) <= tol).all()


@gpu
@pytest.mark.parametrize("T", [1, 3, 24])
@pytest.mark.parametrize("scale", [2.0 ** -122, 2.0 ** -110, 2.0 ** 110, 2.0 ** 120, 2.0 ** 123, 3.3e38])
def test_finite_values_near_the_ends_of_their_type(scale, T):
    """bf16 values of drafts and tail close to the largest and to the smallest normal number: the outputs are averages
    of them, so they are finite too; below the normal range a step of the output is 2^-133."""
    g = torch.Generator().manual_seed(11)
    pr = Problem(T=T, lens=[900, 7], page=64, prefix=False)
    sign = lambda x: torch.where(torch.rand(x.shape, generator=g) < 0.5, -1.0, 1.0)                # noqa: E731
    span = lambda x: (0.5 + 0.5 * torch.rand(x.shape, generator=g)) * scale                        # noqa: E731
    for signs in (sign, lambda x: 1.0):
        pr.Vp, pr.Vn = ((signs(x) * span(x)).to(torch.bfloat16) for x in (pr.Vp, pr.Vn))
        assert torch.isfinite(pr.Vp).all() and torch.isfinite(pr.Vn).all()
        got = pr.call().cpu().double()
        want, tol = pr.expect()
        assert torch.isfinite(got).all()
        off = (got - want).norm(dim=3)
        assert (off <= tol + 2.0 ** -134 * math.sqrt(D)).all(), (off / tol).max()


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("size", [1.0, 64.0, 2048.0, 32768.0])
@pytest.mark.parametrize("T", [1, 20])
def test_equal_logits_of_any_size(dtype, size, T):
    """Tokens with one and the same key weigh alike, in parts of unequal length and however large the logit is (up to
    1e10, where fp32 counts in steps of 1024): the output is the mean of the values.  Errors: a value's row, 2^-11 of
    it (fp32: the sums' 128 terms), and the output's half step."""
    n = 1000
    pr = Problem(dtype=dtype, T=T, B=1, lens=[n], page=64, prefix=False, mask=torch.zeros(1, T, dtype=torch.int64))
    pr.q = torch.full_like(pr.q, size)
    pr.Kp = torch.full_like(pr.Kp, size)
    got = pr.call()[0].cpu().double()
    table = api.pages_view(pr.pages, pr.state)["table"][0].long()
    V = pr.Vp[table].double().permute(1, 0, 2, 3).reshape(pr.H, -1, D)[:, :n].repeat_interleave(pr.G, 0)
    u, half = (129 * 2.0 ** -24, 2.0 ** -24) if dtype == "fp32" else (2.0 ** -11, 2.0 ** -8)
    want, tol = V.mean(1), u * V.norm(dim=2).mean(1) + half * V.mean(1).norm(dim=1)
    assert ((got - want).norm(dim=2) <= tol).all(), ((got - want).norm(dim=2) / tol).max()


def sink_tolerance(q, K, V, Kn, Vn, u, n, half):
    """(outputs, tolerance) of rows q over tokens K, V, with a logit's error counted token by token.

    With |delta_t| <= E_t = (n u + D 2^-24) |q| Kn_t / sqrt(D) the error of the probabilities moves the output by at
    most e^max(E) sum_t p_t (e^E_t - 1) |V_t - o|, and rounding p_t w_t and a value's row by (n + 1) u p_t Vn_t each;
    the output's own step is half of ||o||.  No term leaves room for tokens that are dropped."""
    s = q @ K.T / math.sqrt(D)
    pr = torch.softmax(s, 1)
    o = pr @ V
    E = (n * u + D * 2.0 ** -24) * q.norm(dim=1)[:, None] * Kn / math.sqrt(D)
    far = torch.cdist(o, V)
    tol = E.amax(1).exp() * (pr * torch.expm1(E) * far).sum(1) + (n + 1) * u * (pr @ Vn) + half * o.norm(dim=1)
    return o, tol


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("tokens,gap,spread,size", [
    (32768, 14.0, 0.3, 1.0), (32768, 16.0, 0.3, 0.1), (32768, 14.0, 1.0, 1.0), (131072, 14.0, 0.3, 1.0),
    (131072, 16.0, 1.0, 0.1), (131072, 17.0, 0.1, 0.3)])
def test_sink_before_many_small_tokens(dtype, tokens, gap, spread, size):
    """The first token takes nearly all, tens of thousands of small ones behind it together a few percent, all in one
    part (as many sequences as fill the SMs): none of what the small ones add is lost.  Exact tokens of bf16 caches
    are fp16 operands without a rounding (n = 0)."""
    H, B, page, g = 4, 37, 128, torch.Generator().manual_seed(5)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    u = torch.randn(H, D, generator=g)
    u /= u.norm(dim=1, keepdim=True)
    q = (8 * (u + 0.02 * torch.randn(B, H, D, generator=g))).to(dt)
    along = spread * math.sqrt(D) / 8 * torch.randn(H, tokens, 1, generator=g)
    K = along * u[:, None] + 0.01 * torch.randn(H, tokens, D, generator=g)
    K[:, 0] = gap * math.sqrt(D) / 8 * u
    V = 1 + 0.3 * torch.randn(H, tokens, D, generator=g)
    V[:, 0] = size * torch.randn(H, D, generator=g)
    K, V = K.to(dt), V.to(dt)
    spec = api.PageSpec(n_pages=tokens // page, page_size=page, n_slots=B, max_pages=tokens // page, n_kv_heads=H, dtype=dtype)
    state = torch.zeros(spec.state_numel, dtype=torch.int32)
    v = api.pages_view(spec, state)
    v["len"][:] = tokens
    v["table"][:] = torch.arange(spec.n_pages)
    p = api.AnchorKVParams(n_tokens=1024, n_kv_heads=H, n_q_heads=H, dtype=dtype)
    pools = [x.reshape(H, -1, page, D).transpose(0, 1).contiguous().cuda() for x in (K, V)]
    Kn, Vn = (torch.randn(B, 1, H, D, generator=g).to(dt) for _ in range(2))
    mask = torch.zeros(B, 1, dtype=torch.int64)                              # the draft sees the tail alone
    got = api.tree_attn(p, None, q[:, None].cuda(), Kn.cuda(), Vn.cuda(), mask=mask.cuda(), pages=spec, state=state.cuda(),
                        K_pages=pools[0], V_pages=pools[1])[:, 0].cpu().double()
    unit, n, half = (2.0 ** -24, 128, 2.0 ** -24) if dtype == "fp32" else (2.0 ** -11, 0, 2.0 ** -8)
    for h in range(H):
        k, x = K[h].double(), V[h].double()
        want, tol = sink_tolerance(q[:, h].double(), k, x, k.norm(dim=1), x.norm(dim=1), unit, n, half)
        off = (got[:, h] - want).norm(dim=1)
        assert (off <= tol).all(), (off / tol).max()


@gpu
def test_sink_before_a_million_tokens():
    """2^20 exact tokens, as many as page tables may reach, for as many sequences as there are SMs: what the sums of a
    part round away stays below an operand's rounding.  The reference is on the GPU, in 64 bits."""
    B, n, page, g = 148, 1 << 20, 128, torch.Generator(device="cuda").manual_seed(7)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")                                  # noqa: E731
    u = rand(D)
    u /= u.norm()
    q = (8 * (u + 0.02 * rand(B, D))).bfloat16()
    K = 0.3 * math.sqrt(D) / 8 * rand(n, 1) * u + 0.01 * rand(n, D)
    K[0] = 18 * math.sqrt(D) / 8 * u
    V = 1 + 0.3 * rand(n, D)
    V[0] = rand(D)
    K, V = K.bfloat16(), V.bfloat16()
    spec = api.PageSpec(n_pages=n // page, page_size=page, n_slots=B, max_pages=n // page, n_kv_heads=1)
    state = torch.zeros(spec.state_numel, dtype=torch.int32)
    v = api.pages_view(spec, state)
    v["len"][:] = n
    v["table"][:] = torch.arange(spec.n_pages)
    p = api.AnchorKVParams(n_tokens=1024, n_kv_heads=1, n_q_heads=1)
    new = rand(B, 1, 1, D).bfloat16()
    got = api.tree_attn(p, None, q[:, None, None], new, new, mask=torch.zeros(B, 1, dtype=torch.int64).cuda(), pages=spec,
                        state=state.cuda(), K_pages=K.reshape(-1, 1, page, D), V_pages=V.reshape(-1, 1, page, D))[:, 0, 0].double()
    k, x = K.double(), V.double()
    for i in range(0, B, 37):
        want, tol = sink_tolerance(q[i:i + 37].double(), k, x, k.norm(dim=1), x.norm(dim=1), 2.0 ** -11, 0, 2.0 ** -8)
        off = (got[i:i + 37] - want).norm(dim=1)
        assert (off <= tol).all(), (off / tol).max()


@gpu
def test_sink_of_a_compressed_prompt():
    """The same behind a compressed prompt, whose rows are rounded like all others."""
    H, B, N, g = 4, 37, 32768, torch.Generator().manual_seed(6)
    u = torch.randn(H, D, generator=g)
    u /= u.norm(dim=1, keepdim=True)
    q = (8 * (u + 0.02 * torch.randn(B, H, D, generator=g))).bfloat16()
    K = 0.4 * torch.randn(H, N, 1, generator=g) * u[:, None] + 0.1 * torch.randn(H, N, D, generator=g)
    K[:, 0] = 14 * math.sqrt(D) / 8 * u
    V = 1 + 0.3 * torch.randn(H, N, D, generator=g)
    V[:, 0] = torch.randn(H, D, generator=g)
    p = api.AnchorKVParams(n_tokens=N, n_kv_heads=H, n_q_heads=H, theta=0.05)
    po = O.Params(n_tokens=N, n_kv_heads=H, n_q_heads=H, theta=0.05, dtype="bf16")
    comp, ws = api.compress(p, K.bfloat16().cuda(), V.bfloat16().cuda(), q[:32].transpose(0, 1).contiguous().cuda())
    assert api.read_status(ws)[0] == 0
    parts = O.unpack_layout(comp.cpu().numpy(), po)
    full, bare = O.reconstruct(parts, po), O.reconstruct(dict(parts, codes=np.zeros((0, D), np.uint8)), po)
    dense = [(torch.tensor(f), torch.tensor(np.linalg.norm(a, axis=-1) + np.linalg.norm(f - a, axis=-1)))
             for f, a in zip(full, bare)]
    Kn, Vn = (torch.randn(B, 1, H, D, generator=g).bfloat16() for _ in range(2))
    got = api.tree_attn(p, comp, q[:, None].cuda(), Kn.cuda(), Vn.cuda(), mask=torch.zeros(B, 1, dtype=torch.int64).cuda(),
                        layout_of=torch.zeros(B, dtype=torch.int32).cuda())[:, 0].cpu().double()
    for h in range(H):
        (k, kn), (x, xn) = ((d[h].double(), m[h].double()) for d, m in dense)
        want, tol = sink_tolerance(q[:, h].double(), k, x, kn, xn, 2.0 ** -11, 3, 2.0 ** -8)
        off = (got[:, h] - want).norm(dim=1)
        assert (off <= tol).all(), (off / tol).max()


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("gamma", [0.0, 6e-8, 1e-5, 1e-3, -1.0, "by token"])
@pytest.mark.parametrize("sigma", [0.0, 1.0, 6e4])
def test_scales_of_tokens_and_residuals(dtype, gamma, sigma):
    """Layouts whose anchors or residuals weigh next to nothing, or all there is, or count backwards."""
    pr = Problem(dtype=dtype, T=3, B=1, N=700, theta=0.4, lens=[9], q_scale=1.0)
    po = O.Params(n_tokens=700, n_kv_heads=pr.H, n_q_heads=pr.H * pr.G, theta=0.4, dtype=dtype)
    off, N, R = O.layout(po)["off"], po.n_tokens, O.layout(po)["R"]
    image = pr.comp[0].cpu().numpy()
    tok = image[off["tok"]:off["tok"] + 8 * pr.H * N].view(np.uint32)
    g16 = np.float16([0.0, 6e-8, 1e-5, 1e-3, -1.0, 1.0, 30.0])[np.arange(len(tok)) % 7] if gamma == "by token" \
        else np.full(len(tok), gamma, np.float16)
    tok[:] = tok & 0xFFFF | g16.view(np.uint16).astype(np.uint32) << 16
    sig = image[off["res_sigma"]:off["res_sigma"] + 2 * R].view(np.float16)
    sig[:] = (sig.astype(np.float64) * sigma).clip(0, 6e4).astype(np.float16)
    pr.comp[0] = torch.tensor(image)
    parts = O.unpack_layout(image, po)
    full, bare = O.reconstruct(parts, po), O.reconstruct(dict(parts, codes=np.zeros((0, D), np.uint8)), po)
    pr.dense[0] = [(torch.tensor(f), torch.tensor(np.linalg.norm(a, axis=-1) + np.linalg.norm(f - a, axis=-1)))
                   for f, a in zip(full, bare)]
    got = pr.call().cpu().double()
    want, tol = pr.expect()
    assert torch.isfinite(got).all() and ((got - want).norm(dim=3) <= tol).all()


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("lens,T", [([0], 1), ([0], 4), ([130], 1), ([300], 6)])
def test_seen_keys_whose_logits_are_minus_infinity(dtype, lens, T):
    """A logit of -inf weighs nothing, also where it is all that a part of the tokens has for a row."""
    pr = Problem(dtype=dtype, T=T, B=1, lens=lens, page=64)
    pr.q[..., 0] = 1
    word = [int(x) for x in pr.mask[0]]
    last = T - 1
    pr.mask[0] = torch.tensor([w & ~(1 << last) for w in word])
    clean = pr.call()
    masked, pr.mask = pr.mask, torch.tensor([word])
    pr.Kn[0, last, :, 0] = -float("inf")
    assert torch.equal(pr.call(), clean)                       # a draft: as if nobody saw it
    table = api.pages_view(pr.pages, pr.state)["table"][0]
    pages = table.tolist()
    for j in pages[0:4:2] if lens[0] == 300 else pages[2:]:    # whole pages, or the last one's rows
        pr.Kp[j, :, :, 0] = -float("inf")
    got = pr.call().cpu().double()
    rest = [1, 3, 4] if lens[0] == 300 else [0, 1]             # the pages that weigh anything
    if lens[0]:
        table[:len(rest)] = torch.tensor([pages[j] for j in rest])
        pr.lens = [172 if lens[0] == 300 else 128]
    pr.mask = masked
    want, tol = pr.expect()
    assert torch.isfinite(got).all() and ((got - want).norm(dim=3) <= tol).all()


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_infinity_in_a_committed_value(dtype):
    """All rows see it: its coordinate is not finite, the others are what they were."""
    pr = Problem(dtype=dtype, T=4, B=2, lens=[20, 9])
    clean = pr.call()
    page = int(api.pages_view(pr.pages, pr.state)["table"][0, 1])
    pr.Vp[page, 1, 2, 100] = float("inf")
    got = pr.call()
    heads = slice(pr.G, 2 * pr.G)
    assert not torch.isfinite(got[0, :, heads, 100]).any()
    got[0, :, heads, 100] = clean[0, :, heads, 100]
    assert torch.equal(got, clean)


@gpu
@pytest.mark.parametrize("T", [1, 8, 16, 32])
@pytest.mark.parametrize("tail", [0, 6000])
def test_long_parts_of_every_block_size(T, tail):
    """As many sequences as give every SM one block of 16, 32, 64 or 128 rows with a whole prompt in one part, so that
    each place of the pipeline is used over and over; 16 replays give the same bits."""
    H, G, B, N = 4, 4, 37, 8192
    pr = Problem(H=H, G=G, N=N, B=B, layouts=1, T=T, theta=0.1, lens=[tail] + [0] * (B - 1) if tail else None, page=64)
    first = pr.call()
    for _ in range(16):
        assert torch.equal(pr.call(), first)
    one = Problem.__new__(Problem)                                        # sequences 0 and 36, by themselves
    for b in (0, B - 1):
        one.__dict__.update(pr.__dict__)
        one.B, one.layout_of, one.lens = 1, pr.layout_of[b:b + 1], pr.lens[b:b + 1]
        one.q, one.Kn, one.Vn, one.mask = (x[b:b + 1] for x in (pr.q, pr.Kn, pr.Vn, pr.mask))
        if b:
            one.pages = None
        one.check(out=first[b:b + 1])


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_many_beams_of_one_prompt(dtype):
    """More sequences than a warp has lanes, on one layout, with tails of every length."""
    Problem(dtype=dtype, H=1, G=2, N=400, B=37, layouts=1, T=2, lens=[3 * b for b in range(37)]).check()


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_strided_inputs(dtype):
    """Slices of one fused projection, as a model produces them, and padded batches."""
    pr = Problem(dtype=dtype, T=5, B=3, lens=[3, 20, 0])
    H, Hq = pr.H, pr.H * pr.G
    plain = pr.call()
    fused = torch.full((3, 9, Hq + 2 * H + 1, D), 9.0, dtype=pr.p.torch_dtype, device="cuda")
    fused[:, :5, :Hq], fused[:, :5, Hq:Hq + H], fused[:, :5, Hq + H:Hq + 2 * H] = pr.q.cuda(), pr.Kn.cuda(), pr.Vn.cuda()
    got = pr.call(q=fused[:, :5, :Hq], K_new=fused[:, :5, Hq:Hq + H], V_new=fused[:, :5, Hq + H:Hq + 2 * H])
    assert torch.equal(got, plain)


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_entries_out_of_range_are_latched(dtype):
    """A page or layout that does not exist: NaN for that sequence, code 3, the others as they were."""
    for what in ("page", "page_below", "layout", "len"):
        pr = Problem(dtype=dtype, T=3, B=3, lens=[40, 40, 40])
        clean = pr.call()
        v = api.pages_view(pr.pages, pr.state)
        if what == "page":
            v["table"][1, 1] = pr.pages.n_pages
        elif what == "page_below":
            v["table"][1, 2] = -1
        elif what == "layout":
            pr.layout_of[1] = 3
        else:
            v["len"][1] = pr.pages.max_pages * pr.pages.page_size + 1
        ws = torch.empty(api.tree_workspace_bytes(pr.p, 3, 3, pr.pages), dtype=torch.uint8, device="cuda")
        got = pr.call(workspace=ws)
        assert torch.isnan(got[1]).all(), what
        assert torch.equal(got[[0, 2]], clean[[0, 2]]), what
        with pytest.raises(capi.AnchorKVError):
            api.read_status(ws)
        pr2 = Problem(dtype=dtype, T=3, B=3, lens=[40, 40, 40])
        assert torch.equal(pr2.call(workspace=ws), clean)          # the next call clears the word
        assert api.read_status(ws)[0] == 0


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [1, 8, 16, 40])
def test_bad_page_at_the_end_of_a_long_tail(dtype, T):
    """What is found wrong in a part's last tile makes all rows of the sequence NaN, in blocks of every size."""
    pr = Problem(dtype=dtype, T=T, B=2, lens=[5000, 5000], page=64)
    clean = pr.call()
    api.pages_view(pr.pages, pr.state)["table"][1, 78] = pr.pages.n_pages
    ws = torch.empty(api.tree_workspace_bytes(pr.p, 2, T, pr.pages), dtype=torch.uint8, device="cuda")
    got = pr.call(workspace=ws)
    assert torch.isnan(got[1]).all() and torch.equal(got[0], clean[0])
    with pytest.raises(capi.AnchorKVError):
        api.read_status(ws)


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_deterministic_on_streams_and_in_graphs(dtype):
    """Two calls at once on two streams, and a captured call on new inputs, give the eager bits."""
    pr = Problem(dtype=dtype, T=6, lens=[100, 30], N=3000)
    eager = pr.call()
    other = Problem(dtype=dtype, T=6, lens=[100, 30], N=3000, seed=2)
    eager2 = other.call()
    q, Kn, Vn = pr.q.cuda(), pr.Kn.cuda(), pr.Vn.cuda()
    kw = dict(pages=pr.pages, state=pr.state.cuda(), K_pages=pr.Kp.cuda(), V_pages=pr.Vp.cuda(), mask=pr.mask.cuda())
    size = api.tree_workspace_bytes(pr.p, 2, 6, pr.pages)
    outs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, ws in zip(streams, spaces):
            with torch.cuda.stream(s):
                outs.append(api.tree_attn(pr.p, pr.comp, q, Kn, Vn, workspace=ws, **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(o, eager) for o in outs)
    # captured, then replayed with other drafts and lengths in the same buffers
    out, graph = torch.zeros_like(eager), torch.cuda.CUDAGraph()
    comp = pr.comp.clone()
    with torch.cuda.graph(graph):
        api.tree_attn(pr.p, comp, q, Kn, Vn, workspace=spaces[0], out=out, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    for dst, src in ((comp, other.comp), (q, other.q), (Kn, other.Kn), (Vn, other.Vn), (kw["state"], other.state),
                     (kw["K_pages"], other.Kp), (kw["V_pages"], other.Vp), (kw["mask"], other.mask)):
        dst.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager2)


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_one_draft_is_the_dense_tail_decode(dtype):
    """One draft over pages answers what decode_attn answers over the same rows as a dense tail."""
    pr = Problem(dtype=dtype, T=1, B=2, lens=[33, 33], page=16)
    got = pr.call().float()
    table = api.pages_view(pr.pages, pr.state)["table"].long()
    tails = []
    for pool, new in ((pr.Kp, pr.Kn), (pr.Vp, pr.Vn)):
        rows = pool[table].permute(0, 2, 1, 3, 4).reshape(2, pr.H, -1, D)[:, :, :33]
        tails.append(torch.cat([rows, new.permute(0, 2, 1, 3)], 2).contiguous().cuda())
    want = api.decode_attn(pr.p, pr.comp, pr.q[:, 0].contiguous().cuda(), *tails, tail_len=34)
    _, tol = pr.expect()
    assert ((got[:, 0] - want).norm(dim=2).cpu().double() <= 2 * tol[:, 0]).all()


@gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_decode_loop_with_beams(dtype):
    """Drafts, verification, beams: attention, commit, fork and compaction in turn, against dense rows kept apart."""
    H, G, P, slots, T, steps = 2, 4, 16, 4, 5, 7
    g = torch.Generator().manual_seed(8)
    pr = Problem(dtype=dtype, H=H, G=G, N=600, B=slots, layouts=1, T=T, lens=[0] * slots)
    dt = pr.p.torch_dtype
    spec = api.PageSpec(n_pages=14, page_size=P, n_slots=slots, max_pages=5, n_kv_heads=H, dtype=dtype)
    Kp, Vp = (torch.zeros(spec.pool_shape, dtype=dt, device="cuda") for _ in range(2))
    state = api.pages_init(spec)
    dense = [[torch.zeros(0, H, D, dtype=dt) for _ in range(2)] for _ in range(slots)]
    pr.pages, pr.lens = spec, None
    for step in range(steps):
        pr.q = (2 * torch.randn(slots, T, H * G, D, generator=g)).to(dt)
        pr.Kn, pr.Vn = (torch.randn(slots, T, H, D, generator=g).to(dt) for _ in range(2))
        pr.mask = ancestors(g, slots, T)
        got = api.tree_attn(pr.p, pr.comp, pr.q.cuda(), pr.Kn.cuda(), pr.Vn.cuda(), mask=pr.mask.cuda(),
                            layout_of=pr.layout_of.cuda(), pages=spec, state=state, K_pages=Kp[0], V_pages=Vp[0])
        # the oracle reads one page per sequence that holds its dense rows
        most = max(max(len(d[0]) for d in dense), 1)
        ref = Problem.__new__(Problem)
        ref.__dict__.update(pr.__dict__)
        ref.lens = [len(d[0]) for d in dense]
        ref.pages = api.PageSpec(n_pages=slots, page_size=most, n_slots=slots, max_pages=1, n_kv_heads=H, dtype=dtype)
        ref.state = torch.zeros(ref.pages.state_numel, dtype=torch.int32)
        api.pages_view(ref.pages, ref.state)["table"][:, 0] = torch.arange(slots)
        ref.Kp, ref.Vp = (torch.zeros(slots, H, most, D, dtype=dt) for _ in range(2))
        for b, d in enumerate(dense):
            ref.Kp[b, :, :len(d[0])], ref.Vp[b, :, :len(d[1])] = d[0].transpose(0, 1), d[1].transpose(0, 1)
        ref.check(out=got)
        # each sequence accepts the path to a random draft
        paths, n = torch.zeros(slots, T, dtype=torch.int32), []
        for b in range(slots):
            word = int(pr.mask[b, int(torch.randint(0, T, (1,), generator=g))])
            path = [i for i in range(T) if word >> i & 1]
            paths[b, :len(path)] = torch.tensor(path)
            n.append(len(path))
            dense[b] = [torch.cat([d, x[b, path]]) for d, x in zip(dense[b], (pr.Kn, pr.Vn))]
        api.pages_commit(spec, state, Kp, Vp, pr.Kn[None].cuda(), pr.Vn[None].cuda(),
                         torch.tensor(n, dtype=torch.int32).cuda(), path=paths.cuda())
        if step % 2:
            parents = torch.randint(0, slots, (slots,), generator=g)
            dense = [list(dense[int(i)]) for i in parents]
            api.pages_fork(spec, state, Kp, Vp, parents.int().cuda())
        if step % 3 == 1:
            api.pages_compact(spec, state, Kp, Vp)
        assert api.read_status(state)[0] == 0


@gpu
def test_last_layout_and_page_far_into_memory():
    """Offsets past 2^31 bytes: the last page of a pool and the last layout of a batch."""
    pr = Problem(T=2, B=1, lens=[20], N=700)
    want = pr.call()
    pages = (1 << 31) // (pr.H * 16 * D * 2) + 3
    spec = api.PageSpec(n_pages=pages, page_size=16, n_slots=1, max_pages=2, n_kv_heads=pr.H)
    Kp, Vp = (torch.zeros(spec.pool_shape[1:], dtype=torch.bfloat16, device="cuda") for _ in range(2))
    state = torch.zeros(spec.state_numel, dtype=torch.int32)
    v, old = api.pages_view(spec, state), api.pages_view(pr.pages, pr.state)
    v["len"][0] = 20
    for j in range(2):
        v["table"][0, j] = pages - 1 - j
        Kp[pages - 1 - j], Vp[pages - 1 - j] = pr.Kp[int(old["table"][0, j])].cuda(), pr.Vp[int(old["table"][0, j])].cuda()
    n = (1 << 31) // pr.comp.shape[1] + 2
    comp = torch.zeros(n, pr.comp.shape[1], dtype=torch.uint8, device="cuda")
    comp[-1] = pr.comp[0]
    got = api.tree_attn(pr.p, comp, pr.q.cuda(), pr.Kn.cuda(), pr.Vn.cuda(), mask=pr.mask.cuda(),
                        layout_of=torch.tensor([n - 1], dtype=torch.int32).cuda(), pages=spec, state=state.cuda(),
                        K_pages=Kp, V_pages=Vp)
    assert torch.equal(got, want)


@gpu
def test_tensor_checks():
    pr = Problem(T=2, B=2, lens=[3, 3])
    q, Kn, Vn = pr.q.cuda(), pr.Kn.cuda(), pr.Vn.cuda()
    for bad in (dict(q=pr.q), dict(q=q.float()), dict(q=q[:, :, ::2]), dict(K_new=Kn.transpose(1, 2)),
                dict(K_new=Kn[:, :1]), dict(mask=pr.mask.int().cuda()), dict(n_new=torch.ones(3, dtype=torch.int32).cuda()),
                dict(state=pr.state[:-1].cuda()), dict(K_pages=pr.Kp[:-1].cuda()), dict(out=q[:, :1]),
                dict(layout_of=pr.layout_of.long().cuda()), dict(state=None)):
        with pytest.raises(ValueError):
            pr.call(**{**dict(q=q, K_new=Kn, V_new=Vn), **bad})
    with pytest.raises(capi.AnchorKVError) as e:
        pr.call(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == capi.ENOSPC


# --- host side ---------------------------------------------------------------

FAKE = 0x10000


def host_call(p=None, ws=FAKE, ws_bytes=1 << 40, **over):
    p = p or api.AnchorKVParams(n_tokens=1000, n_kv_heads=2, n_q_heads=8)
    t = capi.Tree(batch=2, n_draft=3, compressed=FAKE, seq_stride_bytes=1 << 20, n_layouts=2, q=FAKE, q_seq_stride=4096,
                  q_tok_stride=1024, K_new=FAKE, V_new=FAKE, new_seq_stride=4096, new_tok_stride=256, out=FAKE)
    pages = over.pop("spec", None)
    if pages is not None:
        t.pages, t.state, t.K_pages, t.V_pages = ctypes.pointer(pages.c()), FAKE, FAKE, FAKE
    for k, v in over.items():
        setattr(t, k, v)
    return capi.lib().anchorkv_tree_attn(ctypes.byref(p.c()), ctypes.byref(t), ws, ws_bytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), capi.EINVAL), (dict(n_draft=0), capi.EINVAL), (dict(n_draft=65), capi.EINVAL),
    (dict(batch=40000), capi.EUNSUPPORTED), (dict(batch=1, p=api.AnchorKVParams(n_tokens=100, n_kv_heads=32768, n_q_heads=32768)), capi.EUNSUPPORTED), (dict(q=None), capi.EINVAL), (dict(K_new=None), capi.EINVAL),
    (dict(V_new=None), capi.EINVAL), (dict(out=None), capi.EINVAL), (dict(ws=None), capi.EINVAL),
    (dict(n_layouts=1), capi.EINVAL), (dict(n_layouts=0, layout_of=FAKE), capi.EINVAL),
    (dict(seq_stride_bytes=1 << 10), capi.EINVAL), (dict(seq_stride_bytes=(1 << 20) + 8), capi.EINVAL),
    (dict(q_tok_stride=1016), capi.EINVAL), (dict(q_tok_stride=1028), capi.EINVAL), (dict(q_seq_stride=-8), capi.EINVAL),
    (dict(new_tok_stride=128), capi.EINVAL), (dict(new_seq_stride=4097), capi.EINVAL), (dict(q=FAKE + 8), capi.EINVAL),
    (dict(K_new=FAKE + 2), capi.EINVAL), (dict(out=FAKE + 4), capi.EINVAL), (dict(compressed=FAKE + 8), capi.EINVAL),
    (dict(mask=FAKE + 4), capi.EINVAL), (dict(n_new=FAKE + 2), capi.EINVAL), (dict(ws_bytes=1000), capi.ENOSPC),
    (dict(batch=0), capi.OK)])
def test_bad_arguments_refused(over, status):
    assert host_call(**over) == status


@pytest.mark.parametrize("spec,status", [
    (api.PageSpec(n_pages=4, n_slots=1, n_kv_heads=2), capi.EINVAL),                     # fewer slots than sequences
    (api.PageSpec(n_pages=4, n_slots=2, n_kv_heads=1), capi.EINVAL),
    (api.PageSpec(n_pages=4, n_slots=2, n_kv_heads=2, dtype="fp32"), capi.EINVAL),
    (api.PageSpec(n_pages=4, n_slots=2, n_kv_heads=2, page_size=20), capi.EINVAL),
    (api.PageSpec(n_pages=4, n_slots=2, n_kv_heads=2, page_size=128, max_pages=8193), capi.EUNSUPPORTED)])
def test_bad_pages_refused(spec, status):
    assert host_call(spec=spec) == status
    good = api.PageSpec(n_pages=4, n_slots=2, n_kv_heads=2)
    for field in ("state", "K_pages", "V_pages"):
        assert host_call(spec=good, **{field: None}) == capi.EINVAL
        assert host_call(spec=good, **{field: FAKE + 8}) == capi.EINVAL


def test_null_arguments_refused():
    p, n = api.AnchorKVParams(n_tokens=1000), ctypes.c_size_t()
    assert capi.lib().anchorkv_tree_attn(ctypes.byref(p.c()), None, FAKE, 1 << 30, None) == capi.EINVAL
    assert capi.lib().anchorkv_tree_workspace_bytes(ctypes.byref(p.c()), 1, 1, None, None) == capi.EINVAL
    assert capi.lib().anchorkv_tree_workspace_bytes(None, 1, 1, None, ctypes.byref(n)) == capi.EINVAL


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("prefix", [True, False])
def test_a_workspace_serves_smaller_calls(dtype, prefix):
    """What a program takes for its largest tree and batch is enough for all others."""
    p = api.AnchorKVParams(n_tokens=32768, n_kv_heads=8, n_q_heads=32, dtype=dtype)
    spec = api.PageSpec(n_pages=64, page_size=64, n_slots=40, max_pages=32, n_kv_heads=8, dtype=dtype)
    kw = dict(p=p, spec=spec, q_tok_stride=4096, q_seq_stride=4096 * 64, new_tok_stride=1024, new_seq_stride=1024 * 64,
              n_layouts=40, seq_stride_bytes=1 << 30, **({} if prefix else dict(compressed=None)))
    for batch, drafts in ((8, 64), (4, 48), (40, 64), (40, 3), (19, 40), (37, 17)):
        size = api.tree_workspace_bytes(p, batch, drafts, spec)
        assert host_call(batch=batch, n_draft=drafts, ws_bytes=size, **kw) != capi.ENOSPC
        for b in range(1, batch + 1):
            for t in range(1, drafts + 1):
                assert host_call(batch=b, n_draft=t, ws_bytes=size, **kw) != capi.ENOSPC, (batch, drafts, b, t)


@gpu
@pytest.mark.parametrize("dtype,N,B,T", [("fp32", 3000, 5, 48), ("bf16", 5000, 3, 32)])
def test_small_calls_in_the_workspace_of_a_large_one(dtype, N, B, T):
    """Fewer parts than the call would have by itself: the same answer, inside the same bytes."""
    small = Problem(dtype=dtype, H=8, G=4, N=N, B=B, layouts=1, T=T, lens=[300, 20, 7, 0, 64][:B], page=64)
    own, size = (api.tree_workspace_bytes(small.p, B, t, small.pages) for t in (T, T + 1))
    assert size < own
    ws = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
    small.check(out=small.call(workspace=ws[:size]))
    assert (ws[size:] == 77).all()
