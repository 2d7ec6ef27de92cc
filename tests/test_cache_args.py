"""Host checks of the shared-prefix decode and eviction calls: what the C ABI
refuses before it touches a device, and what the binding refuses before that."""
import ctypes

import pytest
import torch

import block_sparse_gqa_05_b200 as M
from block_sparse_gqa_05_b200 import msa as B
from tests.test_binding_args import calls  # noqa: F401  (the library as a stub)

BIG = 1 << 40
OK = ctypes.c_void_p(1 << 20)             # never dereferenced: validation fails first
MIS = ctypes.c_void_p((1 << 20) + 8)
ODD = ctypes.c_void_p((1 << 20) + 2)


def shape(**kw):
    d = dict(batch=3, seq_q=1, seq_kv=1000, q_offset=0, n_q_heads=16, n_kv_heads=4, head_dim=64,
             index_dim=32, block=128, topk=4)
    d.update(kw)
    return M.Shape(**d)


def size(s, op):
    n = ctypes.c_size_t(7)
    return B.lib().msa_workspace_size(ctypes.byref(s), op, ctypes.byref(n)), n.value


def attend(s, np_=100, cap=100, lens=OK, q=OK, kp=OK, vp=OK, k=OK, v=OK, o=OK, lse=None, w=None,
           wo=None, ws=OK, n=BIG):
    return B.lib().msa_prefix_attn_decode(ctypes.byref(s), np_, cap, lens, q, kp, vp, k, v, o, lse,
                                          w, wo, ws, n, None)


def attend_paged(s, pages=8, np_=100, pp=OK, lens=OK, table=OK, q=OK, k=OK, v=OK, o=OK, ws=OK, n=BIG):
    return B.lib().msa_prefix_attn_decode_paged(ctypes.byref(s), pages, np_, pp, lens, table, q, k,
                                                v, o, None, None, None, ws, n, None)


def arrays(s):
    """Disjoint made-up addresses of the eviction's arrays."""
    step = 1 << 30
    names = ("lens", "w", "pos", "k", "v", "wo", "po", "new")
    return {n: (i + 1) * step for i, n in enumerate(names)}


def evict(s, budget=10, first=0, recent=0, ws=OK, n=BIG, pages=None, table=OK, **at):
    a = dict(arrays(s), **at)
    p = [None if a[x] is None else ctypes.c_void_p(a[x]) for x in a]
    L = B.lib()
    if pages is None:
        return L.msa_cache_evict(ctypes.byref(s), budget, first, recent, *p, ws, n, None)
    return L.msa_cache_evict_paged(ctypes.byref(s), pages, budget, first, recent, p[0], table,
                                   *p[1:], ws, n, None)


def test_workspace_sizes():
    s = shape()
    st, plain = size(s, M.OP_PREFIX_DECODE)
    st2, scored = size(s, M.OP_PREFIX_DECODE_WEIGHTS)
    st3, ev = size(s, M.OP_CACHE_EVICT)
    assert st == st2 == st3 == 0 and scored >= plain >= 0 and ev > 0
    # a shape only the decode takes: 128 rows of a sequence and group at most
    assert size(shape(seq_q=32), M.OP_PREFIX_DECODE)[0] == 0
    assert size(shape(seq_q=33), M.OP_PREFIX_DECODE)[0] == 5
    assert size(shape(seq_q=8, seq_kv=7), M.OP_PREFIX_DECODE)[0] == 1


@pytest.mark.parametrize("bad,code", [
    (dict(block=64), 5), (dict(head_dim=96), 5), (dict(n_q_heads=18), 1), (dict(n_q_heads=24), 5),
    (dict(n_kv_heads=3, n_q_heads=12), 5), (dict(seq_q=0), 1), (dict(batch=0), 1),
    (dict(seq_kv=0), 1), (dict(batch=1 << 20, seq_kv=1 << 20), 5),
])
def test_shapes(bad, code):
    s = shape(**bad)
    assert size(s, M.OP_PREFIX_DECODE)[0] == code and attend(s) == code and attend_paged(s) == code
    if "seq_q" not in bad:
        assert size(s, M.OP_CACHE_EVICT)[0] == code and evict(s) == code
        assert evict(s, pages=8) == code


def test_attend_arguments():
    s = shape()
    assert attend(s, np_=-1) == 1 and attend(s, np_=101, cap=100) == 1
    assert attend(s, np_=0, cap=1 << 30) == 5
    for name in ("lens", "q", "kp", "vp", "k", "v", "o", "ws"):
        assert attend(s, **{name: None}) == 2, name
    for name in ("q", "kp", "vp", "k", "v", "o", "ws"):
        assert attend(s, **{name: MIS}) == 3, name
    for name in ("lens", "lse", "wo"):
        assert attend(s, **{name: ODD}) == 3, name
    assert attend(s, w=OK) == 2                             # weights without weights_out
    assert attend(s, w=OK, wo=ctypes.c_void_p((1 << 20) + 400)) == 5     # overlapping
    assert attend(s, n=8) == 4
    assert B.lib().msa_prefix_attn_decode(None, 0, 0, OK, OK, OK, OK, OK, OK, OK, None, None, None,
                                          OK, BIG, None) == 2
    # no prefix: its pointers are not looked at; the workspace check is reached
    assert attend(s, np_=0, cap=0, kp=None, vp=None, n=8) == 4


def test_attend_paged_arguments():
    s = shape()
    assert attend_paged(s, pages=0) == 1 and attend_paged(s, pages=1 << 29) == 5
    assert attend_paged(s, np_=-1) == 1 and attend_paged(s, np_=1 << 29) == 5
    for name in ("pp", "lens", "table", "q", "k", "v", "o", "ws"):
        assert attend_paged(s, **{name: None}) == 2, name
    for name in ("pp", "lens", "table"):
        assert attend_paged(s, **{name: ODD}) == 3, name
    assert attend_paged(s, n=8) == 4 and attend_paged(s, np_=0, pp=None, n=8) == 4


@pytest.mark.parametrize("pages", [None, 8])
def test_evict_arguments(pages):
    s = shape()
    a = arrays(s)
    assert evict(s, budget=0, pages=pages) == 1 and evict(s, first=-1, pages=pages) == 1
    assert evict(s, recent=-1, pages=pages) == 1
    for name in a:
        assert evict(s, pages=pages, **{name: None}) == 2, name
        assert evict(s, pages=pages, **{name: a[name] + 2}) == 3, name
    assert evict(s, pages=pages, n=8) == 4 and evict(s, pages=pages, ws=None) == 2
    # in place is fine (the workspace check is reached), partly overlapping is not
    assert evict(s, pages=pages, n=8, wo=a["w"], po=a["pos"]) == 4
    for x, y in (("wo", "w"), ("po", "pos"), ("po", "wo"), ("po", "w"), ("wo", "pos"),
                 ("new", "wo"), ("new", "lens"), ("new", "pos"), ("lens", "wo"), ("lens", "po")):
        assert evict(s, pages=pages, **{x: a[y] + 4}) == 5, (x, y)
    assert evict(s, pages=pages, new=a["lens"]) == 5
    if pages:
        assert evict(s, pages=0) == 1 and evict(s, pages=1 << 29) == 5
        assert evict(s, pages=8, table=None) == 2 and evict(s, pages=8, table=ODD) == 3


def _tensors(s, pages=0):
    bf, G, d, C = torch.bfloat16, s.n_kv_heads, s.head_dim, s.seq_kv
    x = dict(q=torch.zeros(s.batch, s.seq_q, s.n_q_heads, d, dtype=bf),
             lens=torch.ones(s.batch, dtype=torch.int32),
             w=torch.zeros(s.batch, G, C), pos=torch.zeros(s.batch, G, C, dtype=torch.int32),
             kp=torch.zeros(G, 200, d, dtype=bf), vp=torch.zeros(G, 200, d, dtype=bf),
             k=torch.zeros(s.batch, G, C, d, dtype=bf), v=torch.zeros(s.batch, G, C, d, dtype=bf),
             pages=torch.zeros(40, G, 128, d, dtype=bf),
             table=torch.zeros(s.batch, s.nb, dtype=torch.int32),
             pp=torch.zeros(2, dtype=torch.int32))
    return x


def test_binding_accepts_the_layouts(calls):  # noqa: F811
    s = shape()
    x = _tensors(s)
    o, lse, w = M.prefix_attn_decode(s, x["q"], x["k"], x["v"], x["lens"], x["kp"], x["vp"])
    assert o.shape == x["q"].shape and lse.shape == (3, 1, 16) and w is None
    o, lse, w = M.prefix_attn_decode(s, x["q"], x["k"], x["v"], x["lens"], weights=x["w"], want_lse=False)
    assert lse is None and w is x["w"]                      # in place
    o, lse, w = M.prefix_attn_decode(s, x["q"], x["k"], x["v"], x["lens"], x["kp"], x["vp"], prefix_len=7,
                                     weights_out=x["w"])
    assert w is x["w"]
    M.prefix_attn_decode_paged(s, x["q"], x["pages"], x["pages"], x["lens"], x["table"], x["pp"], 130,
                               weights=x["w"])
    w, pos, new = M.cache_evict(s, x["k"], x["v"], x["lens"], x["w"], x["pos"], 10)
    assert w is x["w"] and pos is x["pos"] and new.shape == (3,) and new.dtype == torch.int32
    M.cache_evict_paged(s, x["pages"], x["pages"], x["lens"], x["table"], x["w"], x["pos"], 10, first=1,
                        recent=2)
    assert [c for c in calls if c != "msa_workspace_size"] == \
        ["msa_prefix_attn_decode"] * 3 + ["msa_prefix_attn_decode_paged", "msa_cache_evict",
                                          "msa_cache_evict_paged"]


def test_binding_refuses(calls):  # noqa: F811
    s = shape()
    x = _tensors(s)
    with pytest.raises(ValueError, match="k_prefix: .* elements"):
        M.prefix_attn_decode(s, x["q"], x["k"], x["v"], x["lens"], x["kp"][:2], x["vp"])
    with pytest.raises(ValueError, match="v_prefix: expected torch.bfloat16"):
        M.prefix_attn_decode(s, x["q"], x["k"], x["v"], x["lens"], x["kp"], x["vp"].float())
    with pytest.raises(ValueError, match="weights: .* elements"):
        M.prefix_attn_decode(s, x["q"], x["k"], x["v"], x["lens"], weights=x["w"][:2])
    with pytest.raises(ValueError, match="seq_lens: expected torch.int32"):
        M.prefix_attn_decode(s, x["q"], x["k"], x["v"], x["lens"].long())
    with pytest.raises(ValueError, match="prefix_pages: .* elements"):
        M.prefix_attn_decode_paged(s, x["q"], x["pages"], x["pages"], x["lens"], x["table"], x["pp"], 300)
    with pytest.raises(ValueError, match="positions: expected torch.int32"):
        M.cache_evict(s, x["k"], x["v"], x["lens"], x["w"], x["pos"].long(), 10)
    with pytest.raises(ValueError, match="page_table: .* elements"):
        M.cache_evict_paged(s, x["pages"], x["pages"], x["lens"], x["table"][:1], x["w"], x["pos"], 10)
    with pytest.raises(ValueError, match="one device"):
        M.cache_evict(s, x["k"], x["v"], x["lens"], x["w"], x["pos"].to("meta"), 10)
    assert set(calls) <= {"msa_workspace_size"}             # no compute call was made


def test_attend_workspace_has_room_for_its_alignment():
    """The workspace may start at any multiple of 16 bytes, the attention stores
    32 at a time: the size holds the arrays from the next multiple of 32 on."""
    s = shape()                    # 3 sequences x 4 groups, r = 4, d = 64; 12 prefix rows, 4 own ones
    up = lambda n: -(-n // 256) * 256
    pre, own = 2 * (4 + 256) * 12 * 4, 2 * (12 + 256) * 4 * 4
    plain = up(16 * 8) + up(pre * 8) + up(pre * 256) + up(own * 8) + up(own * 256)
    assert size(s, M.OP_PREFIX_DECODE) == (0, plain + 16)
    assert size(s, M.OP_PREFIX_DECODE_WEIGHTS) == (0, plain + 12 * 4 * 1024 * 4 + 16)
    exact = plain + 16
    assert attend(s, ws=ctypes.c_void_p((1 << 20) + 16), n=exact - 1) == 4


@pytest.mark.parametrize("past", [1 << 31, (1 << 32) + 5, -(1 << 32) + 5])
def test_binding_refuses_integers_past_32_bits(calls, past):  # noqa: F811
    """ctypes cuts an int to its low 32 bits: a budget of 2^32 + 5 would keep 5 rows."""
    s = shape()
    x = _tensors(s)
    with pytest.raises(ValueError, match="32 bits"):
        M.prefix_attn_decode(s, x["q"], x["k"], x["v"], x["lens"], x["kp"], x["vp"], prefix_len=past)
    for kw in (dict(budget=past), dict(budget=5, first=past), dict(budget=5, recent=past)):
        with pytest.raises(ValueError, match="32 bits"):
            M.cache_evict(s, x["k"], x["v"], x["lens"], x["w"], x["pos"], **kw)
        with pytest.raises(ValueError, match="32 bits"):
            M.cache_evict_paged(s, x["pages"], x["pages"], x["lens"], x["table"], x["w"], x["pos"], **kw)
    if past < 0:
        with pytest.raises(ValueError, match="32 bits"):
            M.prefix_attn_decode_paged(s, x["q"], x["pages"], x["pages"], x["lens"], x["table"], x["pp"], past)
    assert set(calls) <= {"msa_workspace_size"}


def test_binding_takes_the_largest_integers(calls):  # noqa: F811
    s = shape()
    x = _tensors(s)
    M.cache_evict(s, x["k"], x["v"], x["lens"], x["w"], x["pos"], (1 << 31) - 1, first=(1 << 31) - 1,
                  recent=(1 << 31) - 1)
    assert "msa_cache_evict" in calls


def test_binding_refuses_prefixes_of_two_capacities(calls):  # noqa: F811
    """The capacity is a stride: the groups of a longer v_prefix would be read at
    the wrong rows.  Half a prefix would be taken for none."""
    s = shape()
    x = _tensors(s)
    longer = torch.zeros(4, 201, 64, dtype=torch.bfloat16)
    for kp, vp in ((x["kp"], longer), (longer, x["vp"]), (None, x["vp"]), (x["kp"], None)):
        with pytest.raises(ValueError, match="one capacity"):
            M.prefix_attn_decode(s, x["q"], x["k"], x["v"], x["lens"], kp, vp)
    assert not calls
    empty = longer[:, :0]                     # no prefix, as tensors without rows
    M.prefix_attn_decode(s, x["q"], x["k"], x["v"], x["lens"], empty, empty)
    assert "msa_prefix_attn_decode" in calls


def test_evict_ignores_the_query_fields():
    for kw in (dict(seq_q=0), dict(seq_q=77), dict(q_offset=-3), dict(q_offset=1 << 30), dict(index_dim=7)):
        assert size(shape(**kw), M.OP_CACHE_EVICT) == size(shape(), M.OP_CACHE_EVICT)
        assert evict(shape(**kw), n=8) == 4 and evict(shape(**kw), pages=8, n=8) == 4
    for kw, code in ((dict(topk=65), 5), (dict(topk=0), 1), (dict(n_q_heads=18), 1)):
        assert size(shape(**kw), M.OP_CACHE_EVICT)[0] == code
