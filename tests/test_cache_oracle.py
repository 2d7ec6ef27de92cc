"""Pins of the shared-prefix attention and eviction oracles: against torch's
dense attention over concatenated caches, closed forms and hand-built cases."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as CO


def _rand(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("T", [1, 3])
def test_prefix_attention_is_dense_attention_over_both_parts(T):
    B, H, G, d, Np, C = 3, 4, 2, 8, 11, 9
    lens = [9, 4, 6]
    q, kp, vp = _rand(B, T, H, d), _rand(G, Np, d, seed=1), _rand(G, Np, d, seed=2)
    k, v = _rand(B, G, C, d, seed=3), _rand(B, G, C, d, seed=4)
    o, lse, w, absum, reach = CO.prefix_attention(q, kp, vp, k, v, lens)
    for b in range(B):
        kk = torch.cat([kp, k[b, :, :lens[b]]], 1).repeat_interleave(H // G, 0)
        vv = torch.cat([vp, v[b, :, :lens[b]]], 1).repeat_interleave(H // G, 0)
        n = Np + lens[b]
        mask = torch.arange(n)[None] <= (n - T + torch.arange(T))[:, None]
        ref = torch.nn.functional.scaled_dot_product_attention(
            q[b].transpose(0, 1), kk, vv, attn_mask=mask[None])
        assert np.allclose(o[b], ref.transpose(0, 1).numpy(), atol=1e-12)
        s = (q[b].transpose(0, 1) @ kk.transpose(1, 2)) / math.sqrt(d)
        s = s.masked_fill(~mask[None], -math.inf)
        assert np.allclose(lse[b], torch.logsumexp(s, -1).T.numpy(), atol=1e-12)
        p = torch.softmax(s, -1).sum(1).reshape(G, H // G, n).sum(1)
        assert np.allclose(w[b, :, :lens[b]], p[:, Np:].numpy(), atol=1e-12)
        assert np.all(w[b, :, lens[b]:] == 0)


def test_prefix_attention_empty_rows_and_sums():
    B, T, H, G, d, C = 2, 2, 2, 1, 4, 5
    q, k, v = _rand(B, T, H, d), _rand(B, G, C, d, seed=1), _rand(B, G, C, d, seed=2)
    none = torch.zeros(G, 0, d, dtype=torch.float64)
    o, lse, w, _, _ = CO.prefix_attention(q, none, none, k, v, [1, 0])
    # one row and two new tokens: the first sees nothing, the second the row
    assert np.all(o[0, 0] == 0) and np.all(np.isneginf(lse[0, 0]))
    assert np.allclose(o[0, 1], v[0, 0, 0].numpy()) and np.allclose(w[0, 0], [2, 0, 0, 0, 0])
    assert np.all(o[1] == 0) and np.all(np.isneginf(lse[1])) and np.all(w[1] == 0)
    w0 = torch.arange(10.).reshape(B, G, C)
    _, _, w1, _, _ = CO.prefix_attention(q, none, none, k, v, [5, 5], w0)
    # every query hands out exactly 1
    assert np.allclose((w1 - w0.numpy()).sum((1, 2)), T * H)


def test_evict_plan_by_hand():
    pos = list(range(8))
    w = [5., 1., 7., 1., 9., 2., 8., 0.]
    frm, to = CO.evict_plan(w, pos, 8, 4, 0, 0)          # kept 4, 6, 2, 0
    assert frm.tolist() == [4, 6] and to.tolist() == [1, 3]
    frm, to = CO.evict_plan(w, pos, 8, 4, 2, 1)          # 0, 1, 7 stay, then 4
    assert frm.tolist() == [4, 7] and to.tolist() == [2, 3]
    frm, to = CO.evict_plan([1.] * 8, pos, 8, 5, 0, 0)   # ties: the lowest rows
    assert frm.size == 0 and to.size == 0
    frm, to = CO.evict_plan([math.nan, 0., -0., 3.], pos, 4, 3, 0, 0)
    assert frm.tolist() == [3] and to.tolist() == [0]    # NaN goes first
    frm, to = CO.evict_plan(w, [7, 0, 1, 2, 3, 4, 5, 6], 8, 2, 0, 2)   # newest rows by position
    assert frm.tolist() == [7] and to.tolist() == [1]
    frm, to = CO.evict_plan(w, pos, 8, 3, 8, 0)          # more rows stay than fit: the best of them
    assert frm.tolist() == [4, 6] and to.tolist() == [0, 1]


def test_evict_keeps_the_attention_of_the_kept_rows():
    B, G, C, d, n = 2, 2, 12, 4, 7
    k, v = _rand(B, G, C, d, seed=5), _rand(B, G, C, d, seed=6)
    w = np.random.default_rng(0).random((B, G, C))
    pos = np.tile(np.arange(C), (B, G, 1))
    k2, v2, w2, p2, new = CO.evict(k, v, w, pos, [12, 10], n, 1, 2)
    assert new.tolist() == [7, 7]
    for b, ln in enumerate((12, 10)):
        for g in range(G):
            rows = p2[b, g, :n]
            assert len(set(rows.tolist())) == n and 0 in rows and ln - 1 in rows and ln - 2 in rows
            assert torch.equal(k2[b, g, :n], k[b, g, rows]) and torch.equal(v2[b, g, :n], v[b, g, rows])
            assert np.array_equal(w2[b, g, :n], w[b, g, rows])
            assert np.all(w2[b, g, n:ln] == 0) and np.all(p2[b, g, n:ln] == -1)
            assert np.array_equal(w2[b, g, ln:], w[b, g, ln:])
            assert torch.equal(k2[b, g, n:], k[b, g, n:])
