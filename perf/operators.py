"""The decode-side cache operators as a serving loop calls them, in plain torch and through the library.

attend: one decode step of a batch whose sequences share a prefix.  T new tokens per sequence attend the shared
prefix K/V [G, Cp, d] and their own ragged caches [B, G, C, d]; with ``weights`` the softmax weight that each own
key received is added to a running score per key.

evict: every (sequence, group) of an own cache keeps its ``budget`` best rows by that score; rows of low positions
(``first``) and of the newest positions (``recent``) come before all others.  Kept rows past the new length move into
the rows that were dropped.
"""
import math
import random

import numpy as np
import torch

own = False
BLOCK = 128


def _spread(lo, hi, n):
    """n lengths in [lo, hi], ragged, the ends among them; they go by the case alone."""
    x = [lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]
    x[-1] = hi
    return x


def _attend(name, B, T, H, G, d, prefix, own_lo, own_hi, cap, weights, paged):
    return {"name": name, "op": "attend", "B": B, "T": T, "H": H, "G": G, "d": d, "prefix": prefix, "own_lo": own_lo,
            "own_hi": own_hi, "cap": cap, "weights": weights, "paged": paged}


def _evict(name, B, G, d, cap, len_lo, len_hi, budget, first, recent, settled, paged):
    return {"name": name, "op": "evict", "B": B, "G": G, "d": d, "cap": cap, "len_lo": len_lo, "len_hi": len_hi,
            "budget": budget, "first": first, "recent": recent, "settled": settled, "paged": paged}


def listed():
    return [
        # a small model answering two users after a short system prompt: latency only
        _attend("attend_two_users", 2, 1, 8, 2, 64, 200, 0, 90, 96, False, False),
        # a chat service: 32 sequences behind one 8K prompt, scored for later eviction
        _attend("attend_chat_8k", 32, 1, 64, 8, 128, 8192, 1, 1024, 1024, True, False),
        # five drafted tokens per sequence checked at once, paged caches, an odd prefix
        _attend("attend_drafts_paged", 24, 5, 64, 8, 128, 20011, 5, 700, 700, True, True),
        # a wide batch on a long document: the prefix product is bound by the tensor cores
        _attend("attend_wide_32k", 256, 1, 64, 8, 128, 32768, 1, 256, 256, False, False),
        # a few questions on a context of a million tokens: bound by reading the prefix
        _attend("attend_few_1m", 4, 1, 64, 8, 128, 1048576, 1, 300, 384, False, False),
        # no prefix: long own caches of different lengths, scored every step
        _attend("attend_own_16k", 16, 1, 64, 8, 128, 0, 0, 16384, 16384, True, False),
        # one key/value head per query head, heads of 64, odd lengths, three tokens, paged
        _attend("attend_odd_heads", 7, 3, 16, 16, 64, 4999, 2, 333, 333, True, True),
        # the settled loop: each step appends a row and drops one, some sequences not full yet
        _evict("evict_one_of_4k", 32, 8, 128, 4224, 3900, 4097, 4096, 4, 256, True, False),
        # after a long prompt: 128K caches cut to a quarter
        _evict("evict_128k_to_32k", 4, 8, 128, 131072, 100000, 131072, 32768, 4, 1024, False, False),
        # paged caches cut so that whole pages come free
        _evict("evict_paged_8k_to_2k", 16, 8, 128, 8192, 1000, 8192, 2048, 16, 128, False, True),
        # a small cache: latency only
        _evict("evict_small", 1, 2, 64, 320, 300, 300, 256, 4, 32, True, False),
        # one context of a million tokens cut to 64K
        _evict("evict_one_1m", 1, 8, 128, 1048576, 1048570, 1048570, 65536, 64, 4096, False, False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    d = rng.choice((64, 128, 128))
    G = rng.choice((2, 4, 8, 8, 16))
    paged = rng.random() < 0.4
    if rng.random() < 0.55:
        r = rng.choice((1, 2, 4, 8, 8, 16))
        T = rng.choice((1, 1, 1, 2, 3, 5, 8))
        B = _log_int(rng, 1, 256)
        cap = max(T, _log_int(rng, 16, max(64, min(16384, 4_000_000_000 // (B * G * d * 4) // 4))))
        lo = rng.choice((0, 1, T, cap // 2))
        most = 150e9 / (4 * B * T * G * r * d)
        prefix = 0 if rng.random() < 0.1 else _log_int(rng, 1, int(max(2, min(400000, most, 2e9 / (B * T * G * r)))))
        c = _attend("", B, T, G * r, G, d, prefix, lo, cap - rng.randrange(0, min(cap, 9)) if cap > T + 9 else cap, cap,
                    rng.random() < 0.6, paged)
        c["own_lo"] = min(c["own_lo"], c["own_hi"])
    else:
        B = _log_int(rng, 1, 64)
        cap = _log_int(rng, 100, max(200, min(400000, 4_000_000_000 // (B * G * d * 4))))
        hi = cap - rng.randrange(0, 20)
        budget = max(1, min(hi, int(hi * rng.choice((0.1, 0.25, 0.5, 0.9, 1.0))) - rng.randrange(0, 3)))
        c = _evict("", B, G, d, cap, max(1, int(hi * rng.choice((0.2, 0.7, 1.0)))), hi, budget,
                   rng.choice((0, 4, 16)), rng.randrange(0, max(1, budget // 2)), rng.random() < 0.5, paged)
    del c["name"]
    return c


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _lens(case):
    lo, hi = (case["own_lo"], case["own_hi"]) if case["op"] == "attend" else (case["len_lo"], case["len_hi"])
    return _spread(lo, hi, case["B"])


def _bf16(g, *shape, scale=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    x.normal_(0.0, scale, generator=g)
    return x


def prepare(case, seed):
    g = _gen(seed)
    B, G, d, cap = case["B"], case["G"], case["d"], case["cap"]
    lens = _lens(case)
    s = {"case": case, "seq_lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    nb = -(-cap // BLOCK)
    if case["paged"]:
        npp = -(-case.get("prefix", 0) // BLOCK)
        P = B * nb + npp
        perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
        s["page_table"] = perm[: B * nb].reshape(B, nb).contiguous()
        s["prefix_pages"] = perm[B * nb:].contiguous()
        s["k"], s["v"] = _bf16(g, P, G, BLOCK, d), _bf16(g, P, G, BLOCK, d)
    else:
        s["k"], s["v"] = _bf16(g, B, G, cap, d), _bf16(g, B, G, cap, d)
    live = torch.arange(cap, device="cuda")[None, None, :] < s["seq_lens"][:, None, None]
    if case["op"] == "attend":
        # queries larger than keys: logits spread over several units, as trained heads' are
        s["q"] = _bf16(g, B, case["T"], case["H"], d, scale=2.0)
        if case["prefix"] and not case["paged"]:
            s["k_prefix"], s["v_prefix"] = _bf16(g, G, case["prefix"], d), _bf16(g, G, case["prefix"], d)
        if case["weights"]:
            w = torch.rand((B, G, cap), generator=g, device="cuda")
            s["weights"] = torch.where(live, w, 0.0)
    else:
        # scores with the long tail of accumulated attention, and rows that never got any
        w = torch.exp(2.0 * torch.randn((B, G, cap), generator=g, device="cuda"))
        w = torch.where(torch.rand((B, G, cap), generator=g, device="cuda") < 0.05, 0.0, w)
        s["weights"] = torch.where(live, w, 0.0)
        pos = torch.cumsum(torch.randint(1, 4, (B, G, cap), generator=g, device="cuda"), -1)
        if case["settled"]:
            # earlier evictions have left the rows in no order
            key = torch.where(live, torch.rand((B, G, cap), generator=g, device="cuda"), 2.0)
            pos = torch.gather(pos, -1, torch.argsort(key, dim=-1))
        s["positions"] = torch.where(live, pos, -1).to(torch.int32)
    if own:
        import block_sparse_gqa_05_b200 as M

        T, H = case.get("T", 1), case.get("H", G)
        s["shape"] = M.Shape(B, T, cap, cap - T, H, G, d, 64, BLOCK, 1)
        if case["op"] == "attend":
            op = M.OP_PREFIX_DECODE_WEIGHTS if case["weights"] else M.OP_PREFIX_DECODE
            s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty((B, T, H), device="cuda")
        else:
            op = M.OP_CACHE_EVICT
            s["new_lens"] = torch.empty_like(s["seq_lens"])
            s["positions_out"] = torch.full_like(s["positions"], -1)
        if "weights" in s:
            s["weights_out"] = torch.zeros_like(s["weights"])
        s["ws"] = M.alloc_workspace(s["shape"], op)
    return s


def _rows(pages, table, rows):
    """Rows 0 .. rows-1 that a table [..., nb] lists of pages [P, G, 128, d]: [..., G, rows, d]."""
    x = pages[table.long()].transpose(-4, -3)
    return x.reshape(*x.shape[:-3], -1, x.shape[-1])[..., :rows, :]


def _plain_attend(s):
    c = s["case"]
    B, T, H, G, d, cap, N = c["B"], c["T"], c["H"], c["G"], c["d"], c["cap"], c["prefix"]
    r = H // G
    k, v = s["k"], s["v"]
    if c["paged"]:
        kp, vp = _rows(k, s["prefix_pages"], N), _rows(v, s["prefix_pages"], N)
        k, v = _rows(k, s["page_table"], cap), _rows(v, s["page_table"], cap)
    elif N:
        kp, vp = s["k_prefix"], s["v_prefix"]
    else:
        kp, vp = k[0, :, :0], v[0, :, :0]
    q = s["q"].float().reshape(B, T, G, r, d) / math.sqrt(d)
    # the prefix: the rows of every sequence against one copy of it
    sp = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(G, B * T * r, d), kp.float().transpose(1, 2))
    # the own caches: token t of T sees the rows up to len - T + t
    so = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(B, G, T * r, d), k.float().transpose(2, 3))
    last = s["seq_lens"][:, None] - T + torch.arange(T, device="cuda")[None, :]
    seen = torch.arange(cap, device="cuda")[None, None, :] <= last[:, :, None]
    seen = seen[:, None, :, None, :].expand(B, G, T, r, cap).reshape(B, G, T * r, cap)
    so = torch.where(seen, so, -math.inf)
    neg = torch.full((), -math.inf, device="cuda")
    mp = sp.amax(-1) if N else neg.expand(G, B * T * r)
    m = torch.maximum(mp.reshape(G, B, T * r).transpose(0, 1), so.amax(-1))
    m = torch.where(m == -math.inf, 0.0, m)
    sp = torch.exp_(sp - m.transpose(0, 1).reshape(G, B * T * r, 1))
    so = torch.exp_(so - m[..., None])
    total = sp.sum(-1).reshape(G, B, T * r).transpose(0, 1) + so.sum(-1)
    acc = torch.matmul(sp, vp.float()).reshape(G, B, T * r, d).transpose(0, 1) + torch.matmul(so, v.float())
    some = torch.where(total > 0, total, 1.0)
    o = (acc / some[..., None]).reshape(B, G, T, r, d).permute(0, 2, 1, 3, 4).reshape(B, T, H, d)
    lse = torch.where(total > 0, m + torch.log(some), -math.inf)
    out = {"o": o.to(torch.bfloat16), "lse": lse.reshape(B, G, T, r).transpose(1, 2).reshape(B, T, H)}
    if c["weights"]:
        out["weights"] = s["weights"] + (so / some[..., None]).sum(2)
    return out


def _plain_evict(s):
    c = s["case"]
    cap = c["cap"]
    w, pos, lens = s["weights"], s["positions"], s["seq_lens"]
    x = torch.arange(cap, device="cuda").expand_as(w)
    ln = lens[:, None, None]
    n = torch.clamp(ln, max=c["budget"])
    live = x < ln
    end = torch.where(live, pos, -1).amax(-1, keepdim=True) + 1
    fixed = live & ((pos < c["first"]) | (pos >= end - c["recent"]))
    # best first: live rows, those that stay in any case, larger scores, lower rows
    order = torch.sort(torch.where(torch.isnan(w), -math.inf, w), dim=-1, descending=True, stable=True).indices
    kind = torch.gather(live.to(torch.int32) + fixed.to(torch.int32), -1, order)
    order = torch.gather(order, -1, torch.sort(kind, dim=-1, descending=True, stable=True).indices)
    keep = torch.empty_like(live).scatter_(-1, order, x < n)
    hole, mover = ~keep & (x < n), keep & (x >= n)
    movers = torch.sort((~mover).to(torch.int32), dim=-1, stable=True).indices
    rank = (torch.cumsum(hole.to(torch.int32), -1) - 1).clamp(min=0)
    src = torch.where(hole, torch.gather(movers, -1, rank), x)
    gone = live & (x >= n)
    k, v = s["k"], s["v"]
    b = torch.arange(c["B"], device="cuda")[:, None, None]
    g = torch.arange(c["G"], device="cuda")[None, :, None]
    if c["paged"]:
        at = torch.gather(s["page_table"].long()[:, None, :].expand(-1, c["G"], -1), -1, src // BLOCK)
        to = s["page_table"].long()[b, x // BLOCK]
        kk, vv = k.clone(), v.clone()
        kk[to, g.expand_as(x), x % BLOCK] = k[at, g, src % BLOCK]
        vv[to, g.expand_as(x), x % BLOCK] = v[at, g, src % BLOCK]
    else:
        kk, vv = k[b, g, src], v[b, g, src]
    return {"k": kk, "v": vv, "weights": torch.where(gone, 0.0, torch.gather(w, -1, src)),
            "positions": torch.where(gone, -1, torch.gather(pos, -1, src)), "lens": n.reshape(-1)}


def _own_attend(s):
    import block_sparse_gqa_05_b200 as M

    c = s["case"]
    more = {"o": s["o"], "lse": s["lse"], "weights": s.get("weights"), "weights_out": s.get("weights_out"), "ws": s["ws"]}
    if c["paged"]:
        o, lse, w = M.prefix_attn_decode_paged(s["shape"], s["q"], s["k"], s["v"], s["seq_lens"], s["page_table"],
                                               prefix_pages=s["prefix_pages"], prefix_len=c["prefix"], **more)
    else:
        o, lse, w = M.prefix_attn_decode(s["shape"], s["q"], s["k"], s["v"], s["seq_lens"],
                                         k_prefix=s.get("k_prefix"), v_prefix=s.get("v_prefix"), **more)
    return {"o": o, "lse": lse, "weights": w} if c["weights"] else {"o": o, "lse": lse}


def _own_evict(s):
    import block_sparse_gqa_05_b200 as M

    c = s["case"]
    call = M.cache_evict_paged if c["paged"] else M.cache_evict
    at = (s["page_table"],) if c["paged"] else ()
    w, pos, lens = call(s["shape"], s["k"], s["v"], s["seq_lens"], *at, s["weights"], s["positions"], c["budget"],
                        first=c["first"], recent=c["recent"], weights_out=s["weights_out"],
                        positions_out=s["positions_out"], new_lens=s["new_lens"], ws=s["ws"])
    return {"k": s["k"], "v": s["v"], "weights": w, "positions": pos, "lens": lens}


def run(state):
    attend = state["case"]["op"] == "attend"
    if own:
        return _own_attend(state) if attend else _own_evict(state)
    return _plain_attend(state) if attend else _plain_evict(state)


def work(case):
    lens, G, d = _lens(case), case["G"], case["d"]
    if case["op"] == "attend":
        B, T, H, N = case["B"], case["T"], case["H"], case["prefix"]
        seen = sum(max(0, n - T + t + 1) for n in lens for t in range(T))
        size = 4 * G * d * (N + sum(lens)) + 4 * B * T * H * d + 4 * B * T * H
        return {"bytes": size + (8 * G * sum(lens) if case["weights"] else 0), "flops": 4 * H * d * (B * T * N + seen)}
    kept = [min(n, case["budget"]) for n in lens]
    # rows past the new length that are kept, as many as a random choice keeps there
    moved = sum((n - m) * m / n for n, m in zip(lens, kept) if n)
    return {"bytes": G * (16 * sum(lens) + 8 * d * moved), "flops": 0}


def _exact_attend(s):
    c = s["case"]
    B, T, H, G, d, N = c["B"], c["T"], c["H"], c["G"], c["d"], c["prefix"]
    r, lens = H // G, _lens(c)
    o = torch.zeros((B, T, H, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device="cuda")
    w = s["weights"].double() if c["weights"] else None

    def cache(x, g, b):
        if not c["paged"]:
            return x[b, g, : lens[b]].double()
        return x[s["page_table"][b].long(), g].reshape(-1, d)[: lens[b]].double()

    for g in range(G):
        heads = slice(g * r, (g + 1) * r)
        if c["paged"]:
            kp, vp = (x[s["prefix_pages"].long(), g].reshape(-1, d)[:N].double() for x in (s["k"], s["v"]))
        elif N:
            kp, vp = s["k_prefix"][g].double(), s["v_prefix"][g].double()
        else:
            kp = vp = torch.zeros((0, d), dtype=torch.float64, device="cuda")
        for b in range(B):
            ko, vo = cache(s["k"], g, b), cache(s["v"], g, b)
            for t in range(T):
                n = max(0, lens[b] - T + t + 1)
                if N + n == 0:
                    continue
                q = s["q"][b, t, heads].double()
                z = torch.cat([q @ kp.T, q @ ko[:n].T], 1) * d ** -0.5
                top = z.amax(1, keepdim=True)
                e = torch.exp(z - top)
                z = e.sum(1, keepdim=True)
                o[b, t, heads] = (e[:, :N] @ vp + e[:, N:] @ vo[:n]) / z
                lse[b, t, heads] = (top + torch.log(z))[:, 0]
                if w is not None:
                    w[b, g, :n] += (e[:, N:] / z).sum(0)
    out = {"o": o, "lse": lse}
    if w is not None:
        out["weights"] = w
    return out


def _exact_evict(s):
    c = s["case"]
    B, G = c["B"], c["G"]
    w, pos = s["weights"].double().cpu().numpy(), s["positions"].cpu().numpy()
    k, v, lens, new = s["k"].clone(), s["v"].clone(), _lens(c), []
    for b, ln in enumerate(lens):
        n = min(ln, c["budget"])
        new.append(n)
        for g in range(G):
            if n == ln:
                continue
            p, x = pos[b, g, :ln].copy(), w[b, g, :ln].copy()
            fixed = (p < c["first"]) | (p > p.max() - c["recent"])
            score = np.where(np.isnan(x), -np.inf, x)
            best = np.lexsort((np.arange(ln), -score, ~fixed))[:n]
            mask = np.zeros(ln, dtype=bool)
            mask[best] = True
            to, at = np.flatnonzero(~mask[:n]), n + np.flatnonzero(mask[n:])
            w[b, g, to], pos[b, g, to] = x[at], p[at]
            w[b, g, n:ln], pos[b, g, n:ln] = 0.0, -1
            ti, ai = torch.from_numpy(to).cuda(), torch.from_numpy(at).cuda()
            if c["paged"]:
                table = s["page_table"][b].long()
                for z in (k, v):
                    z[table[ti // BLOCK], g, ti % BLOCK] = z[table[ai // BLOCK], g, ai % BLOCK]
            else:
                for z in (k, v):
                    z[b, g, ti] = z[b, g, ai]
    return {"k": k, "v": v, "weights": torch.from_numpy(w), "positions": torch.from_numpy(pos),
            "lens": torch.tensor(new, dtype=torch.int32)}


def exact(case, seed):
    state = prepare(case, seed)
    return _exact_attend(state) if case["op"] == "attend" else _exact_evict(state)


if __name__ == "__main__":
    rng = random.Random(0)
    for one in listed() + [draw(rng) for _ in range(6)]:
        print(one, work(one))
