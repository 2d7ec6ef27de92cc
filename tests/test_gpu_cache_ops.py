"""GPU parity of the shared-prefix decode attention and of the eviction by
accumulated weight, through the public calls, against float64 oracles.

Tolerances of the attention, derived per element (no fitted constants):
* a logit is a sum of d products of bf16 values accumulated in fp32 (tensor
  cores may truncate: one whole unit per term), scaled and exponentiated in
  fp32: |ds| <= delta = (d + 8) 2^-23 reach + 2^-20, reach the largest
  sum |q k| / sqrt(d) of a seen key;
* hence |d lse| <= delta + (n + 8) 2^-23 (n keys summed in fp32) + |lse| 2^-23;
* a softmax weight p has relative error <= delta + |d lse| + 2^-22;
* in o = sum p v every p is also rounded to bf16 (2^-8 relative) before the
  product and o once after it: |do| <= (2^-8 + error of p + (n + 8) 2^-23)
  sum p |v| + 2^-8 (|o| + that);
* a score adds T r of them to the old one: |dw| <= (error of p) sum p + T r 2^-23 |w|.
"""
import numpy as np
import pytest
import torch

import block_sparse_gqa_05_b200 as M
from oracle import cache_oracle as CO

pytestmark = pytest.mark.gpu
NAN = float("nan")


def mshape(B, T, H, G, d, C):
    return M.Shape(B, T, C, 0, H, G, d, 64, 128, 4)


class Case:
    """Inputs on the CPU; rows past a length hold NaN and Inf in K and V."""

    def __init__(self, B, T, H, G, d, Np, C, lens, seed=0, slack=0, scale=2.0):
        g = torch.Generator().manual_seed(1000 + seed)
        bf = torch.bfloat16
        self.B, self.T, self.H, self.G, self.d, self.Np, self.C, self.lens = B, T, H, G, d, Np, C, lens
        self.q = (torch.randn(B, T, H, d, generator=g) * scale).to(bf)
        self.k, self.v = (torch.randn(B, G, C, d, generator=g).to(bf) for _ in range(2))
        self.kp, self.vp = (torch.randn(G, Np + slack, d, generator=g).to(bf) for _ in range(2))
        for b, n in enumerate(lens):
            self.k[b, :, max(n, 0):] = NAN
            self.v[b, :, max(n, 0):] = NAN
            self.v[b, :, max(n, 0) + 1:] = float("inf")
        self.kp[:, Np:], self.vp[:, Np:] = NAN, NAN
        self.w = torch.rand(B, G, C, generator=g)
        self.shape = mshape(B, T, H, G, d, C)
        self.seed = seed

    def oracle(self):
        lens = [min(max(n, 0), self.C) for n in self.lens]
        return CO.prefix_attention(self.q, self.kp[:, :self.Np], self.vp[:, :self.Np], self.k, self.v, lens,
                                   self.w)

    def dev(self, x):
        return x.contiguous().cuda()

    def run(self, scored=True, **kw):
        kw = dict(kw)
        if scored:
            kw.setdefault("weights", self.dev(self.w))
            kw.setdefault("weights_out", torch.full_like(kw["weights"], -7.0))
        lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        pre = {}
        if self.kp.shape[1]:
            pre = dict(k_prefix=self.dev(self.kp), v_prefix=self.dev(self.vp), prefix_len=self.Np)
        return M.prefix_attn_decode(self.shape, self.dev(self.q), self.dev(self.k), self.dev(self.v), lens,
                                    **pre, **kw)

    def paged(self):
        """Pools with shuffled pages, unused pages NaN, table entries past each length -1."""
        B, G, d, C, Np = self.B, self.G, self.d, self.C, self.Np
        nb, npb = -(-C // 128), -(-Np // 128)
        P = B * nb + npb + 3
        perm = np.random.default_rng(self.seed).permutation(P)
        kp, vp = (torch.full((P, G, 128, d), NAN, dtype=torch.bfloat16) for _ in range(2))
        table = np.full((B, nb), -1, dtype=np.int32)
        for b, n in enumerate(self.lens):
            for j in range(-(-n // 128)):
                pg = table[b, j] = perm[b * nb + j]
                r1 = min((j + 1) * 128, C)
                kp[pg, :, :r1 - j * 128], vp[pg, :, :r1 - j * 128] = \
                    self.k[b, :, j * 128:r1], self.v[b, :, j * 128:r1]
        pages = perm[B * nb:B * nb + npb].astype(np.int32)
        for j, pg in enumerate(pages):
            r1 = min((j + 1) * 128, Np)
            kp[pg, :, :r1 - j * 128], vp[pg, :, :r1 - j * 128] = \
                self.kp[:, j * 128:r1], self.vp[:, j * 128:r1]
        return kp, vp, table, pages

    def run_paged(self, tables=None, **kw):
        kp, vp, table, pages = tables or self.paged()
        kw["weights"] = self.dev(self.w)
        kw["weights_out"] = torch.full_like(kw["weights"], -7.0)
        lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        return M.prefix_attn_decode_paged(self.shape, self.dev(self.q), self.dev(kp), self.dev(vp), lens,
                                          torch.from_numpy(table).cuda(), torch.from_numpy(pages).cuda(),
                                          self.Np, **kw)

    def check(self, o, lse, w, ref=None, skip=()):
        ro, rl, rw, absum, reach = ref or self.oracle()
        n = self.Np + max([1] + [min(max(x, 0), self.C) for x in self.lens])
        r = self.H // self.G
        delta = (self.d + 8) * 2.0**-23 * reach + 2.0**-20
        dl = delta + (n + 8) * 2.0**-23 + np.where(np.isfinite(rl), np.abs(rl), 0) * 2.0**-23
        dp = delta + dl + 2.0**-22
        do = (2.0**-8 + dp[..., None] + (n + 8) * 2.0**-23) * absum
        do = do + 2.0**-8 * (np.abs(ro) + do)
        rows = [b for b in range(self.B) if b not in skip]
        go, gl = o.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()
        for b in rows:
            err = np.abs(go[b] - ro[b])
            assert np.all(err <= do[b]), f"o of {b}: {err.max():.3g}, {np.nanmax(err - do[b]):.3g} over"
            if gl is not None:
                assert np.array_equal(np.isneginf(gl[b]), np.isneginf(rl[b]))
                fin = np.isfinite(rl[b])
                err = np.abs(gl[b][fin] - rl[b][fin])
                assert np.all(err <= dl[b][fin]), f"lse of {b}: {err.max():.3g}"
        if w is None:
            return
        gw = w.double().cpu().numpy()
        for b in rows:
            ln = min(max(self.lens[b], 0), self.C)
            for g in range(self.G):
                e = dp[b, :, g * r:(g + 1) * r].max()
                add = rw[b, g, :ln] - self.w[b, g, :ln].double().numpy()
                tol = e * add + (self.T * r + 2) * 2.0**-23 * rw[b, g, :ln] + 1e-12
                err = np.abs(gw[b, g, :ln] - rw[b, g, :ln])
                assert np.all(err <= tol), f"weights of {b}, {g}: {err.max():.3g}, {(err - tol).max():.3g} over"
                assert np.all(gw[b, g, ln:] == -7.0), "a score past the length was written"


CASES = [
    # one block, one sequence, the smallest sizes
    dict(B=1, T=1, H=1, G=1, d=64, Np=0, C=1, lens=[1]),
    dict(B=1, T=1, H=2, G=1, d=128, Np=1, C=1, lens=[0]),
    dict(B=2, T=1, H=8, G=2, d=64, Np=200, C=96, lens=[90, 1]),
    # ragged own caches with empty and full ones, lengths around the block size
    dict(B=9, T=1, H=16, G=2, d=128, Np=300, C=300, lens=[0, 1, 2, 127, 128, 129, 255, 256, 300], slack=5),
    # every ratio of heads to groups
    dict(B=3, T=1, H=4, G=4, d=64, Np=129, C=140, lens=[1, 130, 140]),
    dict(B=3, T=2, H=8, G=4, d=128, Np=128, C=140, lens=[2, 130, 140]),
    dict(B=2, T=3, H=16, G=4, d=64, Np=127, C=131, lens=[3, 131]),
    dict(B=2, T=1, H=32, G=2, d=128, Np=515, C=257, lens=[17, 257]),
    # drafted tokens: fewer own rows than new tokens, causal among the new ones
    dict(B=5, T=5, H=8, G=1, d=128, Np=0, C=200, lens=[0, 2, 5, 133, 200]),
    dict(B=4, T=16, H=8, G=1, d=64, Np=260, C=270, lens=[16, 3, 128, 270]),     # 128 rows a sequence
    dict(B=2, T=128, H=1, G=1, d=128, Np=70, C=400, lens=[400, 131]),
    dict(B=2, T=8, H=16, G=1, d=128, Np=1000, C=130, lens=[130, 129]),
    # one row tile and one row over, several tiles, an odd number of tiles
    dict(B=16, T=1, H=8, G=1, d=64, Np=1000, C=40, lens=list(range(16))),
    dict(B=17, T=1, H=8, G=1, d=128, Np=700, C=40, lens=list(range(17))),
    dict(B=33, T=1, H=16, G=2, d=64, Np=390, C=40, lens=list(range(33))),
    dict(B=50, T=1, H=8, G=1, d=128, Np=256, C=17, lens=[i % 18 for i in range(50)]),
    # more work than one block per SM, long own caches, no prefix
    dict(B=6, T=1, H=16, G=4, d=128, Np=0, C=3000, lens=[3000, 5, 0, 1234, 2999, 128]),
    dict(B=3, T=2, H=8, G=2, d=64, Np=9000, C=2100, lens=[2100, 2, 1]),
    dict(B=200, T=1, H=4, G=2, d=64, Np=64, C=9, lens=[i % 10 for i in range(200)]),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_prefix_attention(i):
    c = Case(seed=i, **CASES[i])
    o, lse, w = c.run()
    torch.cuda.synchronize()
    assert M.device_status() == 0
    c.check(o, lse, w)
    # without the scores, the same outputs; without lse too
    o2, lse2, none = c.run(scored=False)
    assert none is None and torch.equal(o, o2) and torch.equal(lse, lse2)
    o3, none, _ = c.run(scored=False, want_lse=False)
    assert none is None and torch.equal(o, o3)


@pytest.mark.parametrize("i", [2, 3, 6, 8, 9, 13, 16, 17])
def test_paged_caches_give_the_contiguous_result(i):
    c = Case(seed=50 + i, **CASES[i])
    o, lse, w = c.run()
    op, lp, wp = c.run_paged()
    torch.cuda.synchronize()
    assert M.device_status() == 0                     # no entry past a length was read
    assert torch.equal(o, op) and torch.equal(lse, lp) and torch.equal(w, wp)
    c.check(op, lp, wp)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", [
    dict(B=4, T=1, H=8, G=1, Np=200001, C=300, lens=[300, 0, 1, 177]),      # one tile, few rows
    dict(B=20, T=1, H=8, G=1, Np=100000, C=300, lens=[15 * i for i in range(20)]),   # a pair
    dict(B=11, T=1, H=8, G=1, Np=150000, C=130, lens=[13 * i for i in range(11)]),   # one full tile
    dict(B=2, T=1, H=8, G=1, Np=0, C=90000, lens=[90000, 61111]),           # long own caches
    dict(B=2, T=5, H=8, G=1, Np=300, C=50000, lens=[49999, 3]),
])
def test_many_blocks_per_cta(kw, d):
    c = Case(d=d, seed=60, **kw)
    got = c.run()
    torch.cuda.synchronize()
    assert M.device_status() == 0
    c.check(*got)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(got, c.run()))
    assert M.device_status() == 0


@pytest.mark.parametrize("C, lens", [(9000, [9000, 8190]), (9001, [9001, 8193]), (8192, [8192, 6145])])
def test_scores_of_long_caches(C, lens):
    c = Case(B=2, T=2, H=8, G=2, d=64, Np=100, C=C, lens=lens, seed=77)
    c.check(*c.run())


def test_scores_in_place_and_from_zero():
    c = Case(seed=70, **CASES[3])
    _, _, w = c.run()
    mine = c.dev(c.w)
    _, _, same = c.run(weights=mine, weights_out=mine)
    live = torch.arange(c.C)[None, None] < torch.tensor(c.lens)[:, None, None]
    live = live.expand(c.B, c.G, c.C).cuda()
    assert same is mine and torch.equal(mine[live], w[live])
    assert torch.equal(mine[~live].cpu(), c.w[~live.cpu()])       # untouched past each length
    zero = torch.full_like(mine, NAN)
    sh, lens = c.shape, torch.tensor(c.lens, dtype=torch.int32).cuda()
    _, _, z = M.prefix_attn_decode(sh, c.dev(c.q), c.dev(c.k), c.dev(c.v), lens, c.dev(c.kp), c.dev(c.vp),
                                   prefix_len=c.Np, weights_out=zero)
    got = z[live].double() + c.w[live.cpu()].cuda().double()
    assert torch.allclose(got, w[live].double(), rtol=2e-7, atol=1e-7) and torch.isnan(z[~live]).all()


def test_large_logits_and_equal_logits():
    # logits of several hundred: the running maximum moves by far more than fp32's range of exp
    c = Case(B=3, T=1, H=8, G=2, d=64, Np=700, C=300, lens=[300, 1, 129], seed=71, scale=60.0)
    c.check(*c.run())
    # all keys equal: every weight is 1 / n
    c = Case(B=2, T=2, H=8, G=1, d=128, Np=333, C=260, lens=[260, 7], seed=72)
    c.k[:, :, :], c.kp[:, :c.Np] = c.k[0, 0, 0], c.k[0, 0, 0]
    c.check(*c.run())
    # keys that rise along the cache: the maximum grows in every block
    c = Case(B=1, T=1, H=4, G=1, d=64, Np=2000, C=900, lens=[900], seed=73)
    c.kp[:] = (torch.arange(c.Np)[None, :, None] / c.Np * 3).to(torch.bfloat16)
    c.k[:] = (3 + torch.arange(c.C)[None, None, :, None] / c.C * 3).to(torch.bfloat16)
    c.q[:] = 2.0
    c.check(*c.run())


def test_repeated_calls_are_bit_identical():
    c = Case(B=20, T=1, H=32, G=4, d=128, Np=5000, C=700, lens=[37 * i % 701 for i in range(20)], seed=74)
    first = c.run()
    for _ in range(3):
        again = c.run()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_bad_lengths_are_clamped_and_flagged():
    c = Case(B=3, T=1, H=8, G=2, d=64, Np=50, C=200, lens=[-4, 200, 60], seed=75)
    given = c.lens
    c.lens = [-4, 777, 60]
    o, lse, w = c.run()
    assert M.device_status() == 2
    c.lens = given
    c.check(o, lse, w)


def test_bad_pages_are_flagged():
    c = Case(B=3, T=1, H=8, G=2, d=64, Np=300, C=300, lens=[300, 200, 60], seed=76)
    kp, vp, table, pages = c.paged()
    table[0, 1] = kp.shape[0] + 5
    o, lse, w = c.run_paged(tables=(kp, vp, table, pages))
    assert M.device_status() == 4
    c.check(o, lse, w, skip=(0,))
    table[0, 1] = -3
    c.run_paged(tables=(kp, vp, table, pages))
    assert M.device_status() == 4


# ------------------------------------------------------------------ eviction

def scores(kind, B, G, C, g):
    if kind == "ties":
        return torch.randint(0, 4, (B, G, C), generator=g).float()
    if kind == "equal":
        return torch.full((B, G, C), 0.25)
    if kind == "odd":                      # NaN, infinities, signed zeros, denormals, negatives
        pool = torch.tensor([NAN, -NAN, float("inf"), -float("inf"), 0.0, -0.0, 1e-42, -1e-42, 1.0, -1.0,
                             3.4e38, -3.4e38])
        return pool[torch.randint(0, len(pool), (B, G, C), generator=g)]
    if kind == "close":                    # neighbouring floats
        return (torch.randint(0, 40, (B, G, C), generator=g) + 0x3f800000).to(torch.int32).view(torch.float32)
    return torch.exp(2 * torch.randn(B, G, C, generator=g))


class Cache:
    def __init__(self, B, G, d, C, lens, kind="tail", shuffled=False, seed=0):
        g = torch.Generator().manual_seed(2000 + seed)
        self.B, self.G, self.d, self.C, self.lens = B, G, d, C, lens
        self.k, self.v = (torch.randn(B, G, C, d, generator=g).to(torch.bfloat16) for _ in range(2))
        self.w = scores(kind, B, G, C, g)
        pos = torch.cumsum(torch.randint(1, 3, (B, G, C), generator=g), -1).to(torch.int32) - 1
        if shuffled:
            for b, n in enumerate(lens):
                for x in range(G):
                    p = torch.randperm(n, generator=g)
                    pos[b, x, :n] = pos[b, x, :n][p]
        self.pos = pos
        self.shape = M.Shape(B, 1, C, C - 1, G, G, d, 64, 128, 4)
        self.seed = seed

    def dev(self, x):
        return x.contiguous().cuda()

    def run(self, budget, first=0, recent=0, in_place=False, **kw):
        k, v, w, pos = (self.dev(x) for x in (self.k, self.v, self.w, self.pos))
        if not in_place:
            kw.update(weights_out=torch.full_like(w, -7.0), positions_out=torch.full_like(pos, -7))
        lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        wo, po, new = M.cache_evict(self.shape, k, v, lens, w, pos, budget, first=first, recent=recent, **kw)
        torch.cuda.synchronize()
        if not in_place:
            assert torch.equal(w.view(torch.int32).cpu(), self.w.view(torch.int32))
            assert torch.equal(pos.cpu(), self.pos)
        return k, v, wo, po, new

    def check(self, got, budget, first, recent, in_place=False):
        k, v, wo, po, new = (x.cpu() for x in got)
        lens = [min(max(n, 0), self.C) for n in self.lens]
        rk, rv, rw, rp, rn = CO.evict(self.k, self.v, self.w.numpy(), self.pos.numpy(), lens, budget, first,
                                      recent)
        assert np.array_equal(new.numpy(), rn)
        if not in_place:
            for b, n in enumerate(lens):
                rw[b, :, n:], rp[b, :, n:] = -7.0, -7
        assert np.array_equal(po.numpy(), rp)
        assert np.array_equal(wo.numpy().view(np.int32), np.ascontiguousarray(rw).view(np.int32))
        assert torch.equal(k.view(torch.int16), rk.view(torch.int16))
        assert torch.equal(v.view(torch.int16), rv.view(torch.int16))


EVICT = [
    (dict(B=1, G=1, d=64, C=1, lens=[1]), 1, 0, 0),
    (dict(B=3, G=1, d=64, C=2, lens=[0, 1, 2]), 1, 0, 0),
    (dict(B=2, G=2, d=128, C=300, lens=[300, 299]), 256, 4, 32),
    (dict(B=4, G=2, d=64, C=130, lens=[130, 0, 64, 65], kind="ties", shuffled=True), 64, 2, 10),
    (dict(B=2, G=1, d=128, C=1000, lens=[1000, 999], kind="equal", shuffled=True), 400, 0, 0),
    (dict(B=2, G=4, d=64, C=777, lens=[777, 500], kind="odd"), 333, 3, 3),
    (dict(B=2, G=2, d=64, C=2050, lens=[2050, 2049], kind="close", shuffled=True), 2048, 16, 100),
    (dict(B=2, G=2, d=64, C=600, lens=[600, 555]), 100, 50, 80),       # more rows stay than the budget
    (dict(B=2, G=2, d=64, C=600, lens=[600, 555], kind="ties"), 100, 1 << 20, 0),
    (dict(B=2, G=2, d=64, C=600, lens=[600, 555], kind="ties"), 100, 0, 1 << 30),
    (dict(B=2, G=2, d=64, C=600, lens=[600, 555]), 600, 0, 0),         # nothing to drop
    (dict(B=1, G=2, d=128, C=9000, lens=[8999], shuffled=True), 1, 0, 0),
    (dict(B=3, G=2, d=64, C=5000, lens=[5000, 4097, 100], shuffled=True), 4096, 4, 256),
    (dict(B=1, G=1, d=64, C=40001, lens=[40000], kind="ties"), 10000, 4, 999),
    (dict(B=1, G=2, d=64, C=70000, lens=[69999], shuffled=True), 35001, 64, 4096),
    (dict(B=40, G=8, d=64, C=150, lens=[(7 * i) % 151 for i in range(40)], kind="ties"), 70, 1, 5),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("i", range(len(EVICT)))
def test_evict(i, in_place):
    c, budget, first, recent = EVICT[i]
    c = Cache(seed=i, **c)
    got = c.run(budget, first, recent, in_place)
    assert M.device_status() == 0
    c.check(got, budget, first, recent, in_place)


# rows too many for a cluster's shared memory: chosen by chunks of 8192
LONG = [
    (dict(B=1, G=1, d=64, C=330000, lens=[330000]), 30000, 4, 5000),
    (dict(B=1, G=1, d=64, C=330001, lens=[330001], kind="ties", shuffled=True), 300000, 2, 10),
    (dict(B=2, G=1, d=64, C=330003, lens=[329999, 8193], kind="odd"), 8000, 0, 0),
    (dict(B=1, G=1, d=128, C=330000, lens=[327680], kind="equal", shuffled=True), 9000, 0, 77),
    (dict(B=1, G=2, d=64, C=330004, lens=[330002], kind="close", shuffled=True), 5000, 16, 100),
    (dict(B=1, G=1, d=64, C=330000, lens=[329990]), 1000, 50, 80000),       # more rows stay than the budget
    (dict(B=1, G=1, d=64, C=330000, lens=[330000], kind="odd", shuffled=True), 10000, 1 << 20, 0),
    (dict(B=3, G=1, d=64, C=330000, lens=[330000, 5000, 0]), 6000, 0, 1),   # nothing to drop for two
    (dict(B=2, G=1, d=64, C=330000, lens=[1, 330000]), 330000, 9, 9),       # for nobody
    (dict(B=1, G=1, d=64, C=330000, lens=[330000], kind="equal"), 1, 0, 0),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("i", range(len(LONG)))
def test_evict_long_rows(i, in_place):
    c, budget, first, recent = LONG[i]
    c = Cache(seed=60 + i, **c)
    got = c.run(budget, first, recent, in_place)
    assert M.device_status() == 0
    c.check(got, budget, first, recent, in_place)


def test_evict_long_rows_that_just_fit():
    c = Cache(B=1, G=1, d=64, C=330000, lens=[330000], seed=75)
    pos = c.pos[0, 0].long()
    budget = int(((pos < 100) | (pos > pos.max() - 9000)).sum())           # exactly the rows that stay
    c.check(c.run(budget, 100, 9000), budget, 100, 9000)


def test_evict_long_rows_captured_and_replayed():
    c = Cache(B=1, G=1, d=64, C=330000, lens=[329000], shuffled=True, seed=76)
    k, v, w, pos = (c.dev(x) for x in (c.k, c.v, c.w, c.pos))
    k0, v0 = k.clone(), v.clone()
    lens, new = (torch.tensor(c.lens, dtype=torch.int32).cuda() for _ in range(2))
    wo, po = torch.full_like(w, -7.0), torch.full_like(pos, -7)
    ws = M.alloc_workspace(c.shape, M.OP_CACHE_EVICT)
    call = lambda: M.cache_evict(c.shape, k, v, lens, w, pos, 2000, 4, 20, weights_out=wo, positions_out=po,
                                 new_lens=new, ws=ws)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        k.copy_(k0), v.copy_(v0), wo.fill_(-7.0), po.fill_(-7), new.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        c.check((k, v, wo, po, new), 2000, 4, 20)


@pytest.mark.parametrize("budget", [300, 430, 495])
def test_evict_nan_ties_with_minus_infinity(budget):
    c = Cache(B=2, G=2, d=64, C=500, lens=[500, 499], kind="odd", seed=31)      # the cut reaches the lowest
    c.check(c.run(budget, 0, 0), budget, 0, 0)


def test_evict_again_moves_the_same_rows():
    c = Cache(B=2, G=2, d=64, C=900, lens=[900, 700], seed=30)
    k, v, w, pos = (c.dev(x) for x in (c.k, c.v, c.w, c.pos))
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    for _ in range(2):
        wo, po, new = M.cache_evict(c.shape, k, v, lens, w, pos, 300, 4, 20,
                                    weights_out=torch.full_like(w, -7.0),
                                    positions_out=torch.full_like(pos, -7))
        torch.cuda.synchronize()
        c.check((k, v, wo, po, new), 300, 4, 20)


@pytest.mark.parametrize("i", [2, 3, 6, 12, 15])
def test_evict_paged(i):
    c, budget, first, recent = EVICT[i]
    c = Cache(seed=40 + i, **c)
    nb = -(-c.C // 128)
    P = c.B * nb + 2
    perm = np.random.default_rng(i).permutation(P)
    table = perm[:c.B * nb].reshape(c.B, nb).astype(np.int32)
    pools = [torch.full((P, c.G, 128, c.d), 3.0, dtype=torch.bfloat16) for _ in range(2)]
    for pool, x in zip(pools, (c.k, c.v)):
        for b in range(c.B):
            for j in range(nb):
                r1 = min((j + 1) * 128, c.C)
                pool[table[b, j], :, :r1 - j * 128] = x[b, :, j * 128:r1]
    for b, n in enumerate(c.lens):
        table[b, -(-n // 128):] = -1                  # never read
    kp, vp, w, pos = (c.dev(x) for x in (*pools, c.w, c.pos))
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    wo, po, new = M.cache_evict_paged(c.shape, kp, vp, lens, torch.from_numpy(table).cuda(), w, pos, budget,
                                      first, recent, weights_out=torch.full_like(w, -7.0),
                                      positions_out=torch.full_like(pos, -7))
    torch.cuda.synchronize()
    assert M.device_status() == 0
    back = []
    for pool, x in ((kp, c.k), (vp, c.v)):
        y = x.clone()
        for b, n in enumerate(c.lens):
            for j in range(-(-n // 128)):
                r1 = min((j + 1) * 128, c.C)
                y[b, :, j * 128:r1] = pool[table[b, j], :, :r1 - j * 128].cpu()
        back.append(y)
    c.check((*back, wo, po, new), budget, first, recent)
    free = torch.tensor(sorted(set(range(P)) - set(table[table >= 0].tolist())))
    for pool, old in ((kp, pools[0]), (vp, pools[1])):
        assert torch.equal(pool.cpu()[free], old[free])            # pages of nobody keep their bits


def test_evict_bad_lengths_and_pages_are_flagged():
    c = Cache(B=3, G=2, d=64, C=300, lens=[300, 0, 200], seed=45)
    c.lens = [301, -1, 200]
    got = c.run(100, 2, 9)
    assert M.device_status() == 2
    c.lens = [300, 0, 200]
    c.check(got, 100, 2, 9)
    # a page that does not exist: its rows stay where they are, everything else moves
    nb, P = 3, 9
    table = np.arange(P, dtype=np.int32).reshape(3, nb)
    pool = torch.zeros(P, 2, 128, 64, dtype=torch.bfloat16)
    for b in range(3):
        for j in range(nb):
            r1 = min((j + 1) * 128, 300)
            pool[b * nb + j, :, :r1 - j * 128] = c.k[b, :, j * 128:r1]
    bad = table.copy()
    bad[0, 2] = P + 1
    kp, vp = c.dev(pool), c.dev(pool)
    w, pos = c.dev(c.w), c.dev(c.pos)
    _, po, new = M.cache_evict_paged(c.shape, kp, vp, torch.tensor(c.lens, dtype=torch.int32).cuda(),
                                     torch.from_numpy(bad).cuda(), w, pos, 100, 2, 9)
    torch.cuda.synchronize()
    assert M.device_status() == 4 and new.tolist() == [100, 0, 100]
    got, old = kp.cpu(), c.k
    for b in (0, 2):
        for g in range(2):
            frm, to = CO.evict_plan(c.w[b, g].numpy(), c.pos[b, g].numpy(), c.lens[b], 100, 2, 9)
            for f, t in zip(frm, to):
                ref = old[b, g, t] if b == 0 and f >= 256 else old[b, g, f]
                assert torch.equal(got[b * nb + t // 128, g, t % 128], ref)


# ------------------------------------------------- both together, as a loop runs them

def _loop_inputs(seed=90):
    return Case(B=5, T=1, H=16, G=4, d=64, Np=260, C=200, lens=[1, 190, 128, 77, 200], seed=seed)


def test_a_bounded_decode_loop():
    """attend (scored) -> evict -> append, for many steps: every step against
    the oracle on the caches as they are, the eviction by the scores as they are."""
    c = _loop_inputs()
    budget, first, recent, steps = 60, 2, 8, 12
    gen = torch.Generator().manual_seed(5)
    k, v = c.dev(torch.nan_to_num(c.k, 0, 0, 0)), c.dev(torch.nan_to_num(c.v, 0, 0, 0))
    w = c.dev(c.w)
    pos = torch.arange(c.C, dtype=torch.int32).expand(c.B, c.G, c.C).contiguous().cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    now = torch.tensor(c.lens)
    rows = torch.arange(c.B).cuda()
    kp, vp = c.dev(c.kp), c.dev(c.vp)
    for step in range(steps):
        q = (torch.randn(c.B, 1, c.H, c.d, generator=gen) * 2).to(torch.bfloat16)
        c.q, c.k, c.v, c.w, c.lens = q, k.cpu(), v.cpu(), w.cpu(), lens.tolist()
        before = w.clone()
        o, lse, _ = M.prefix_attn_decode(c.shape, q.cuda(), k, v, lens, kp, vp, weights=w)
        torch.cuda.synchronize()
        shown = w.clone()
        for b, n in enumerate(c.lens):
            assert torch.equal(shown[b, :, n:], before[b, :, n:])
            shown[b, :, n:] = -7.0
        c.check(o, lse, shown)
        old = Cache.__new__(Cache)
        old.__dict__.update(B=c.B, G=c.G, C=c.C, lens=c.lens, k=c.k, v=c.v, w=w.cpu(), pos=pos.cpu())
        _, _, lens = M.cache_evict(c.shape, k, v, lens, w, pos, budget, first, recent)
        torch.cuda.synchronize()
        old.check((k, v, w, pos, lens), budget, first, recent, in_place=True)
        new = (torch.randn(2, c.B, c.G, c.d, generator=gen)).to(torch.bfloat16).cuda()
        at = lens.long()
        k[rows, :, at], v[rows, :, at] = new[0], new[1]
        w[rows, :, at] = 0.0
        pos[rows, :, at] = now.to(torch.int32).cuda()[:, None]
        now += 1
        lens = lens + 1
    assert M.device_status() == 0 and int(lens.max()) == budget + 1


def test_calls_back_to_back_see_the_lengths_just_written():
    """attend and evict in turn with nothing in between, the lengths in two halves
    of one small array, against the same calls with a synchronisation after each."""
    c = _loop_inputs(seed=93)
    c.k, c.v = torch.nan_to_num(c.k, 0, 0, 0), torch.nan_to_num(c.v, 0, 0, 0)
    q = (torch.randn(12, c.B, 1, c.H, c.d, generator=torch.Generator().manual_seed(6)) * 2).bfloat16().cuda()
    kp, vp = c.dev(c.kp), c.dev(c.vp)

    def chain(packed):
        k, v, w = c.dev(c.k), c.dev(c.v), c.dev(c.w)
        pos = torch.arange(c.C, dtype=torch.int32).expand(c.B, c.G, c.C).contiguous().cuda()
        both = torch.zeros(2, c.B, dtype=torch.int32).cuda()
        lens = [both[0], both[1]] if packed else [both[0].clone(), both[1].clone()]
        lens[0].copy_(torch.tensor(c.lens, dtype=torch.int32))
        out = []
        for step in range(12):
            a, z = lens[step % 2], lens[1 - step % 2]
            o, lse, _ = M.prefix_attn_decode(c.shape, q[step], k, v, a, kp, vp, weights=w)
            if not packed:
                torch.cuda.synchronize()
            M.cache_evict(c.shape, k, v, a, w, pos, 190 - 15 * step, 2, 8, new_lens=z)
            if not packed:
                torch.cuda.synchronize()
            out += [o, lse]
        torch.cuda.synchronize()
        return out + [k, v, w, pos, lens[0].clone()]

    ref = chain(False)
    assert ref[-1].tolist() == [min(n, 190 - 15 * 11) for n in c.lens]
    for _ in range(3):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(ref, chain(True)))
    assert M.device_status() == 0


def test_captured_and_replayed():
    """One step (scored attention, then eviction) captured once and replayed
    gives the eager calls' bits, on inputs changed between replays."""
    c = _loop_inputs(91)
    d = {n: c.dev(getattr(c, n)) for n in ("q", "k", "v", "kp", "vp", "w")}
    pos = torch.arange(c.C, dtype=torch.int32).expand(c.B, c.G, c.C).contiguous().cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    out = dict(o=torch.empty_like(d["q"]), lse=torch.empty(c.B, 1, c.H, device="cuda"),
               ws=M.alloc_workspace(c.shape, M.OP_PREFIX_DECODE_WEIGHTS))
    ev = dict(positions_out=torch.zeros_like(pos), new_lens=torch.zeros_like(lens),
              ws=M.alloc_workspace(c.shape, M.OP_CACHE_EVICT))
    wo = torch.zeros_like(d["w"])
    kv = [d["k"].clone(), d["v"].clone()]

    def step():
        kv[0].copy_(d["k"])
        kv[1].copy_(d["v"])
        M.prefix_attn_decode(c.shape, d["q"], *kv, lens, d["kp"], d["vp"], weights=d["w"], weights_out=wo, **out)
        M.cache_evict(c.shape, *kv, lens, wo, pos, 60, 2, 8, **ev)
        return [x.clone() for x in (out["o"], out["lse"], wo, *kv, ev["positions_out"], ev["new_lens"])]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for r in range(3):
        d["q"].mul_(0.75)
        lens.copy_(torch.tensor([(n + 31 * r) % (c.C + 1) for n in c.lens], dtype=torch.int32))
        d["k"].nan_to_num_(0, 0, 0), d["v"].nan_to_num_(0, 0, 0)
        wo.zero_(), ev["positions_out"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in held]
        wo.zero_(), ev["positions_out"].zero_()
        eager = step()
        torch.cuda.synchronize()
        for a, b in zip(replayed, eager):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert M.device_status() == 0


def test_on_streams_of_their_own():
    """Two calls at once on two streams, workspaces and outputs allocated by the
    calls, give what the calls alone give."""
    cs = [Case(B=8, T=1, H=32, G=4, d=128, Np=3000, C=500, lens=[60 * i + 7 for i in range(8)], seed=92 + i)
          for i in range(2)]
    alone = [c.run() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    dev = []
    for c in cs:
        dev.append([c.dev(x) for x in (c.q, c.k, c.v)] + [torch.tensor(c.lens, dtype=torch.int32).cuda()]
                   + [c.dev(x) for x in (c.kp, c.vp, c.w)])
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for c, s, x in zip(cs, streams, dev):
            wo = torch.full_like(x[6], -7.0)
            s.wait_stream(torch.cuda.current_stream())
            got.append(M.prefix_attn_decode(c.shape, *x[:6], weights=x[6], weights_out=wo, stream=s))
            junk = [torch.full((1 << 22,), NAN, device="cuda") for _ in range(3)]   # reuse of freed memory
            del junk
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_expired_waits_are_reported_and_the_context_recovers():
    """With a wait limit of 0 every wait that is not complete at once gives up:
    the call returns, the error word says so, the next call is right again."""
    c = Case(B=20, T=1, H=32, G=4, d=128, Np=5000, C=700, lens=[37 * i % 701 for i in range(20)], seed=95)
    good = c.run()
    torch.cuda.synchronize()
    assert M.device_status() == 0
    try:
        M.set_wait_limit_ns(0)
        c.run()
        torch.cuda.synchronize()
        flags = M.device_status()
    finally:
        M.set_wait_limit_ns(2_000_000_000)
    assert flags & 1, flags
    again = c.run()
    torch.cuda.synchronize()
    assert M.device_status() == 0 and all(torch.equal(a, b) for a, b in zip(good, again))


def test_nan_and_infinite_queries_stay_in_their_rows():
    c = Case(B=3, T=2, H=8, G=2, d=64, Np=300, C=200, lens=[200, 2, 90], seed=96)
    c.check(*c.run())
    ref = c.run()
    c.q[1, 0, 3, 5] = NAN
    c.q[2, 1, 0] = float("inf")
    o, lse, w = c.run()
    torch.cuda.synchronize()
    assert torch.isnan(o[1, 0, 3]).all() and torch.isnan(lse[1, 0, 3])
    assert torch.isnan(o[2, 1, 0]).all() and torch.isnan(lse[2, 1, 0])
    hit = torch.zeros(3, 2, 8, dtype=torch.bool)
    hit[1, 0, 3] = hit[2, 1, 0] = True
    assert torch.equal(o.cpu()[~hit], ref[0].cpu()[~hit]) and torch.equal(lse.cpu()[~hit], ref[1].cpu()[~hit])
    assert M.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("op", [M.OP_PREFIX_DECODE, M.OP_PREFIX_DECODE_WEIGHTS])
def test_workspace_at_any_multiple_of_16_bytes(op, d):
    """A slice of a caller's arena that starts 16 bytes past a multiple of 32 and
    is no longer than asked for: the same bits, nothing written beside it."""
    c = Case(B=5, T=2, H=8, G=2, d=d, Np=700, C=600, lens=[600, 2, 0, 131, 555], seed=97)
    scored = op == M.OP_PREFIX_DECODE_WEIGHTS
    ref = c.run(scored)
    n = M.workspace_size(c.shape, op)
    arena = torch.full((n + 96,), 0x5A, dtype=torch.uint8, device="cuda")
    at = 32 - arena.data_ptr() % 32 + 16
    got = c.run(scored, ws=arena[at:at + n])
    torch.cuda.synchronize()
    assert all(x is y is None or torch.equal(x, y) for x, y in zip(ref, got))
    assert (arena[:at] == 0x5A).all() and (arena[at + n:] == 0x5A).all()
    assert M.device_status() == 0


@pytest.mark.parametrize("fill", [0, 0x7F, 0xFF])
def test_expired_waits_leave_no_index_to_chance(fill):
    """Some fourteen segments a CTA, of which a walk that gives up announces eight
    at most: whatever the workspace held for the others, the second kernel ends,
    reads no index from it and the error word says why."""
    c = Case(B=256, T=1, H=8, G=8, d=64, Np=300, C=40, lens=[1 + 7 * i % 40 for i in range(256)], seed=98)
    good = c.run()
    torch.cuda.synchronize()
    assert M.device_status() == 0
    ws = M.alloc_workspace(c.shape, M.OP_PREFIX_DECODE_WEIGHTS)
    ws.fill_(fill)
    try:
        M.set_wait_limit_ns(0)
        c.run(ws=ws)
        torch.cuda.synchronize()
        flags = M.device_status()
    finally:
        M.set_wait_limit_ns(2_000_000_000)
    assert flags == 1, flags
    again = c.run(ws=ws)
    torch.cuda.synchronize()
    assert M.device_status() == 0 and all(torch.equal(a, b) for a, b in zip(good, again))


def _calls_that_allocate():
    """name -> (call with ``stream`` still to give, workspace given)."""
    c = Case(B=4, T=1, H=16, G=4, d=64, Np=300, C=260, lens=[260, 9, 128, 77], seed=99)
    sh = M.Shape(4, 1, 260, 259, 16, 4, 64, 64, 128, 2)
    g = torch.Generator().manual_seed(99)
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    q, k, v, kp, vp, w = (c.dev(torch.nan_to_num(x, 0.0, 0.0, 0.0)) for x in (c.q, c.k, c.v, c.kp, c.vp, c.w))
    pos = torch.arange(260, dtype=torch.int32).expand(4, 4, 260).contiguous().cuda()
    qi, ki = (torch.randn(*x, generator=g).to(torch.bfloat16).cuda() for x in ((4, 1, 4, 64), (4, 260, 64)))
    sel = M.block_topk(sh, M.index_scores(sh, qi, ki))
    ws = {op: M.alloc_workspace(sh, op) for op in (M.OP_PREFIX_DECODE, M.OP_CACHE_EVICT, M.OP_DENSE_DECODE,
                                                   M.OP_SPARSE_DECODE)}
    kept = (k.clone(), v.clone(), w.clone(), pos.clone())
    return {
        "prefix": lambda **kw: M.prefix_attn_decode(sh, q, k, v, lens, kp, vp, ws=ws[M.OP_PREFIX_DECODE], **kw)[:2],
        "evict": lambda **kw: M.cache_evict(sh, *kept[:2], lens, *kept[2:], 100, ws=ws[M.OP_CACHE_EVICT], **kw)[2:],
        "dense": lambda **kw: M.dense_attn_decode(sh, q, k, v, ws=ws[M.OP_DENSE_DECODE], **kw),
        "sparse": lambda **kw: M.sparse_attn_decode(sh, q, k, v, sel, ws=ws[M.OP_SPARSE_DECODE], **kw),
        "scores": lambda **kw: (M.index_scores(sh, qi, ki, **kw),),
    }


@pytest.mark.parametrize("name", ["prefix", "evict", "dense", "sparse", "scores"])
def test_outputs_of_a_call_on_another_stream_are_not_written_late(name):
    """Memory that was freed while kernels of the current stream still write to it
    is not what a call on another stream returns its outputs in, nor is an output
    reused while the current stream still reads it."""
    call = _calls_that_allocate()[name]
    ref = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    host = torch.empty(1 << 30, dtype=torch.uint8).pin_memory()
    big = torch.empty_like(host, device="cuda")
    for held in (False, True):                   # the first time to load what there is to load
        late = [[torch.empty_like(x) for _ in range(64)] for x in ref]
        if held:                                 # a copy of some 20 ms holds the stream, and no SM
            big.copy_(host, non_blocking=True)
        for xs in late:
            torch._foreach_zero_(xs)
        del xs, late
    got = call(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, got))
    # handed to the current stream: freed while it still has to read them
    torch.cuda.current_stream().wait_stream(s)
    big.copy_(host, non_blocking=True)
    read = [x.clone() for x in got]
    del got
    with torch.cuda.stream(s):
        over = [torch.full_like(x, 7) for x in ref for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, read)) and over
    assert M.device_status() == 0


NOT_FINITE = [
    dict(B=3, T=3, H=8, G=2, d=128, Np=300, C=300, lens=[300, 3, 130]),        # spread and whole tiles, two blocks
    dict(B=3, T=5, H=16, G=2, d=64, Np=0, C=700, lens=[700, 2, 643]),          # a length below T; 40 rows
    dict(B=2, T=2, H=4, G=4, d=64, Np=5000, C=1200, lens=[1200, 1025]),        # spread tiles of 2 rows
    dict(B=2, T=16, H=16, G=2, d=128, Np=40, C=2000, lens=[2000, 1930]),       # a tile of 128 rows
    dict(B=2, T=128, H=2, G=2, d=128, Np=129, C=260, lens=[255, 100]),         # most rows are unseen by some
]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("i", range(len(NOT_FINITE)))
def test_values_of_later_tokens_stay_out_of_earlier_queries(i, paged):
    """Infinities and NaNs in V of the new tokens reach the queries that see them
    and no other: those give the bits they give with finite values there.  (Which of
    them a query gets is not told: a weight times an infinity is one, but a weight
    that was rounded to 0, or a tile's zero for another warp's key, makes it NaN.)"""
    c = Case(**NOT_FINITE[i], seed=120 + i)
    run = (lambda: c.run_paged()) if paged else (lambda: c.run())
    ref = run()
    rng = np.random.default_rng(i)
    r, hit = c.H // c.G, torch.zeros(c.q.shape, dtype=torch.bool)
    for b, n in enumerate(c.lens):
        for g in range(c.G):
            for x in rng.choice(range(max(n - c.T, 0), n), size=min(3, n, c.T), replace=False):
                for col, val in zip(rng.choice(c.d, 3, replace=False), rng.permutation([NAN, np.inf, -np.inf])):
                    c.v[b, g, int(x), int(col)] = float(val)
                    hit[b, max(int(x) - n + c.T, 0):, g * r:(g + 1) * r, int(col)] = True
    o, lse, w = run()
    torch.cuda.synchronize()
    assert hit.any() and not hit.all()
    assert torch.equal(torch.isfinite(o.cpu()), ~hit)
    assert torch.equal(o.cpu()[~hit], ref[0].cpu()[~hit])
    assert torch.equal(lse, ref[1]) and torch.equal(w, ref[2])
    assert M.device_status() == 0


@pytest.mark.parametrize("B, H", [(1, 8), (40, 32)])       # spread tiles; pairs of tiles
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("d", [64, 128])
def test_an_infinite_value_shows_at_any_weight(d, sign, B, H):
    """A seen key's weight is positive, if smaller than fp32 tells from 0: an
    infinity in its V is one in the output (or NaN, as 0 times it), not nothing."""
    c = Case(B=B, T=1, H=H, G=4, d=d, Np=700, C=200, lens=[200 - i for i in range(B)], seed=140)
    c.q[:], c.k[:], c.kp[:] = 4.0, 4.0 * sign, -4.0 * sign     # logits of +-16 d^0.5: weights of 2^-369 and less
    c.vp[:, 650, 3], c.vp[:, 2, 5] = float("inf"), NAN
    c.v[:, :, 130, 7], c.v[:, :, 40, 9] = float("-inf"), NAN
    o, lse, w = c.run()
    torch.cuda.synchronize()
    bad = torch.zeros(d, dtype=torch.bool)
    bad[[3, 5, 7, 9]] = True
    assert not torch.isfinite(o[..., bad]).any()
    assert torch.isfinite(o[..., ~bad]).all() and torch.isfinite(lse).all()
    assert M.device_status() == 0


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("Np", [0, 300])
def test_runs_of_idle_slots(Np, T):
    """A batch of fixed width with few sequences in it: runs of length 0 before,
    between and behind them, longer than the CTAs of the grid."""
    lens = [0] * 400
    lens[160], lens[161], lens[399 if T == 1 else 290] = 130, T, 64
    c = Case(B=400, T=T, H=4, G=2, d=64, Np=Np, C=140, lens=lens, seed=150)
    got = c.run()
    torch.cuda.synchronize()
    assert M.device_status() == 0
    c.check(*got)


def test_a_batch_without_any_key():
    c = Case(B=300, T=1, H=4, G=2, d=64, Np=0, C=140, lens=[0] * 300, seed=151)
    got = c.run()
    torch.cuda.synchronize()
    assert M.device_status() == 0
    c.check(*got)


def test_capacity_far_above_the_lengths():
    """Caches allocated for 100,000 rows that hold a few hundred."""
    c = Case(B=2, T=2, H=8, G=2, d=64, Np=129, C=100_000, lens=[300, 2], seed=152)
    got = c.run()
    torch.cuda.synchronize()
    assert M.device_status() == 0
    c.check(*got)
    for C in (100_001, 330_000):                           # clusters, chunks
        c = Cache(B=2, G=2, d=64, C=C, lens=[700, 65], kind="ties", shuffled=True, seed=153)
        for in_place in (False, True):
            got = c.run(100, 4, 20, in_place)
            assert M.device_status() == 0
            c.check(got, 100, 4, 20, in_place)


def test_idle_slots_between_two_sequences_take_no_wait_limit():
    """The warp that looks for the next sequence passes 600,000 idle slots well within
    30 ms, while the others wait for it (one at a time took ten times that)."""
    B, C, d = 600_000, 4, 64
    sh = mshape(B, 1, 1, 1, d, C)
    g = torch.Generator(device="cuda").manual_seed(154)
    q = torch.randn(B, 1, 1, d, generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.full((B, 1, C, d), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    busy = [0, 299_999, B - 1]
    for b, n in zip(busy, (3, 4, 1)):
        lens[b] = n
        k[b, 0, :n], v[b, 0, :n] = (torch.randn(n, d, generator=g, device="cuda").to(torch.bfloat16)
                                    for _ in range(2))
    ws = M.alloc_workspace(sh, M.OP_PREFIX_DECODE)
    M.prefix_attn_decode(sh, q, k, v, lens, ws=ws)
    torch.cuda.synchronize()
    M.device_status()
    try:
        M.set_wait_limit_ns(30_000_000)
        o, lse, _ = M.prefix_attn_decode(sh, q, k, v, lens, ws=ws)
        torch.cuda.synchronize()
        assert M.device_status() == 0
    finally:
        M.set_wait_limit_ns(2_000_000_000)
    for b in busy:
        n = int(lens[b])
        ro, rl, _, absum, _ = CO.prefix_attention(q[b:b + 1], torch.zeros(1, 0, d), torch.zeros(1, 0, d),
                                                  k[b:b + 1], v[b:b + 1], [n])
        # as Case.check, with delta far below 2^-9
        tol = (2.0**-8 + 2.0**-9) * absum + 2.0**-8 * np.abs(ro) + 2.0**-15 * absum
        assert np.all(np.abs(o[b:b + 1].double().cpu().numpy() - ro) <= tol)
        assert abs(float(lse[b]) - float(rl[0, 0, 0])) < 2.0**-12
        o[b], lse[b] = 0, -float("inf")
    assert not o.any() and torch.isneginf(lse).all()
