"""The boundary of the window, prefix and paging calls, on the CPU: every rejection with its status,
workspace sizes, the binding's own refusals, the kernels' register budgets, and the oracle against
closed forms.  Every call runs under the validate-only hook: no placeholder address reaches a
kernel."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from rope_attention_gb300 import build, native
from test_attention_boundary import A16, V1, cache, packed, paged
from test_kernel_resources import ptxas_report


@pytest.fixture(scope="module")
def L():
    build.build()
    lib = native.load()
    lib.ra_test_validate_only(1)
    yield lib
    lib.ra_test_validate_only(0)


ref = lambda x: None if x is None else ctypes.byref(x)
GIVEN = object()


def call_packed(L, w=GIVEN, p=None, **over):
    a = dict(q=A16, k=A16, v=A16, out=A16, lse=None, cq=None, ck=None, ws=A16, n=64 << 20)
    a.update(over)
    w = native.AttentionWindow(window=10, sinks=2) if w is GIVEN else w
    st = L.packed_window_attention(ref(p or packed()), ref(w), *(a[x] for x in ("q", "k", "v", "out", "lse", "cq", "ck", "ws", "n")), None)
    return st, L.ra_last_error().decode()


PAGED = dict(q=A16, kc=A16, vc=A16, lens=A16, table=A16, cq=None, ks=None, vs=None, ko=None, vo=None, out=A16, lse=None, err=None,
             ws=A16, n=1 << 30)


def call_window(L, w=GIVEN, c=None, p=None, **over):
    a = {**PAGED, **over}
    w = native.AttentionWindow(window=10, sinks=2) if w is GIVEN else w
    st = L.paged_window_attention(ref(c or cache()), ref(p or paged()), ref(w), *a.values(), None)
    return st, L.ra_last_error().decode()


def call_prefix(L, x=GIVEN, c=None, p=None, **over):
    a = {**PAGED, "plen": A16, "ptable": A16, **over}
    x = native.AttentionPrefix(max_prefix_len=100, table_entries=4) if x is GIVEN else x
    order = ["q", "kc", "vc", "plen", "ptable", "lens", "table", "cq", "ks", "vs", "ko", "vo", "out", "lse", "err", "ws", "n"]
    st = L.paged_prefix_attention(ref(c or cache()), ref(p or paged()), ref(x), *(a[k] for k in order), None)
    return st, L.ra_last_error().decode()


NORM = dict(cache_mode=native.RA_CACHE_NORM, block_num=0, block_size=0, cache_seq_len=64)
W = lambda window, sinks=0: native.AttentionWindow(window=window, sinks=sinks)
X = lambda n, entries=4: native.AttentionPrefix(max_prefix_len=n, table_entries=entries)


def test_accepts(L):
    assert call_packed(L) == (0, "")
    assert call_packed(L, W(1 << 62, 1 << 62)) == (0, "")
    assert call_window(L) == (0, "")
    assert call_window(L, c=cache(**V1)) == (0, "")
    assert call_window(L, c=cache(**NORM), p=paged(block_table_stride=0), table=None) == (0, "")
    assert call_prefix(L) == (0, "")
    assert call_prefix(L, X(0)) == (0, "")
    assert call_prefix(L, c=cache(**V1), p=paged(causal=0)) == (0, "")


@pytest.mark.parametrize("w,code", [(None, -1), (W(0), -1), (W(-3), -1), (W(5, -1), -1), (W(-(1 << 62)), -1)])
def test_windows_rejected(L, w, code):
    for call in (call_packed, call_window):
        st, msg = call(L, w)
        assert st == code and "window" in msg or "sinks" in msg


def test_a_window_needs_the_causal_mask(L):
    st, msg = call_packed(L, p=packed(causal=0))
    assert st == -1 and "causal" in msg
    st, msg = call_window(L, p=paged(causal=0))
    assert st == -1 and "causal" in msg


@pytest.mark.parametrize("x,c,over,code", [
    (None, {}, {}, -1), (X(-1), {}, {}, -1), (X(1 << 31), {}, {}, -1), (X(5, 0), {}, {}, -1), (X(5, 1 << 32), {}, {}, -1),
    (GIVEN, {}, dict(plen=None), -1), (GIVEN, {}, dict(ptable=None), -1), (GIVEN, {}, dict(plen=A16 + 2), -3),
    (GIVEN, {}, dict(ptable=A16 + 1), -3), (GIVEN, {}, dict(n=4096), -4), (GIVEN, {}, dict(ws=A16 + 8), -3),
    (GIVEN, {}, dict(table=None), -1), (GIVEN, {}, dict(q=None), -1), (GIVEN, dict(Dkv=272), {}, -2),
])
def test_prefixes_rejected(L, x, c, over, code):
    st, msg = call_prefix(L, x, cache(**c), **over)
    assert st == code and msg


def test_a_prefix_and_what_follows_stay_within_31_bits(L):
    for n, code in ((1000, 0), (1001, -1), ((1 << 31) - 256, -1)):
        st, msg = call_prefix(L, X(n), p=paged(max_seq_len=(1 << 31) - 1256))
        assert st == code and (st == 0) == (msg == "")


def test_a_prefix_needs_pages(L):
    st, msg = call_prefix(L, c=cache(**NORM), p=paged(block_table_stride=0), table=None)
    assert st == -2 and "NORM" in msg


@pytest.mark.parametrize("over,code", [(dict(q=None), -1), (dict(out=A16 + 8), -3), (dict(lse=A16 + 1), -3), (dict(n=100), -4), (dict(ws=None), -1)])
def test_the_calls_behind_keep_their_checks(L, over, code):
    for call in (call_packed, call_window):
        st, msg = call(L, **over)
        assert st == code and msg


def test_prefix_workspace(L):
    n = ctypes.c_size_t()
    size = lambda c, p, x: (L.paged_prefix_attention_workspace_bytes(ref(c), ref(p), ref(x), ctypes.byref(n)), n.value)
    for c in (cache(), cache(**V1), cache(Dkv=256, Dv=256), cache(**V1, ckv_cache_dtype=native.RA_INT8)):
        p = paged(total_q=50, num_heads=64, max_seq_len=1 << 20, block_table_stride=1 << 15)
        st, big = size(c, p, X(1 << 20, 1 << 15))
        rows = 50 * 64 * c.Dv * 4
        assert st == 0 and rows < big <= rows + (129 << 20)
        for len_own, len_prefix in ((10, 1 << 20), (1 << 20, 10), (0, 0)):
            p.max_seq_len = len_own
            st, small = size(c, p, X(len_prefix))
            assert st == 0 and rows < small <= big
    assert L.paged_prefix_attention_workspace_bytes(ref(cache()), ref(paged()), ref(X(5)), None) == -1
    assert size(cache(), paged(), None)[0] == -1 and size(None, paged(), X(5))[0] == -1 and size(cache(), None, X(5))[0] == -1
    assert size(cache(**NORM), paged(block_table_stride=0), X(5))[0] == -2


# ---------------------------------------------------------------- paging
def paging(**kw):
    base = dict(B=3, block_num=20, block_size=16, block_table_stride=5, max_tokens=40)
    base.update(kw)
    return native.KvCachePagingParams(**base)


EXTEND = ["new", "lens", "table", "free", "count", "index", "cu", "new_lens", "new_count", "err"]
SLOTS = ["starts", "counts", "table", "index", "cu", "err"]
TRUNCATE = ["keep", "lens", "table", "free", "count", "new_lens", "new_count", "err"]
OPTIONAL = {"err", "starts", "keep"}


def call_paging(L, name, p, **over):
    names = {"kv_cache_extend": EXTEND, "kv_cache_slots": SLOTS, "kv_cache_truncate": TRUNCATE}[name]
    st = getattr(L, name)(ref(p), *(over.get(x, A16) for x in names), None)
    return st, L.ra_last_error().decode()


@pytest.mark.parametrize("name,names", [("kv_cache_extend", EXTEND), ("kv_cache_slots", SLOTS), ("kv_cache_truncate", TRUNCATE)])
def test_paging_checks(L, name, names):
    assert call_paging(L, name, paging()) == (0, "")
    for x in names:
        st, msg = call_paging(L, name, paging(), **{x: None})
        assert (st, bool(msg)) == ((0, False) if x in OPTIONAL else (-1, True)), x
        st, msg = call_paging(L, name, paging(), **{x: A16 + 2})
        assert st == -3 and msg, x
    if "index" in names:
        assert call_paging(L, name, paging(), index=A16 + 4)[0] == -3
    assert call_paging(L, name, None)[0] == -1
    for kw, code in ((dict(B=0), -1), (dict(max_tokens=0), -1), (dict(block_num=0), -1), (dict(block_num=1 << 31), -1),
                     (dict(block_size=0), -1), (dict(block_size=1 << 31), -1), (dict(block_table_stride=0), -1),
                     (dict(block_table_stride=1 << 31), -1), (dict(B=16385), -2), (dict(max_tokens=(1 << 30) + 1), -2),
                     (dict(B=16384, block_table_stride=1 << 17), -2)):
        st, msg = call_paging(L, name, paging(**kw))
        assert st == code and msg, kw
    assert call_paging(L, name, paging(B=16384, block_table_stride=(1 << 17) - 1, max_tokens=1 << 30)) == (0, "")


# ---------------------------------------------------------------- the binding
def ints(n):
    return torch.zeros(n, dtype=torch.int32)


def test_binding_refuses_short_and_wrong_tensors():
    p = paging()
    good = dict(new_tokens=ints(3), seq_lens=ints(3), block_table=ints(15).view(3, 5), free_pages=ints(20), free_count=ints(1),
                index=torch.zeros(40, dtype=torch.int64), cu_seqlens=ints(4), new_seq_lens=ints(3), new_free_count=ints(1))
    for name, t in good.items():
        with pytest.raises(ValueError, match=f"^{name}: the call needs"):
            native.kv_cache_extend(p, **{**good, name: t.flatten()[:-1].clone()})
        with pytest.raises(ValueError, match=f"^{name}: expected torch.int"):
            native.kv_cache_extend(p, **{**good, name: torch.zeros(t.shape, dtype=torch.float64)})
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        native.kv_cache_extend(p, **good)
    with pytest.raises(TypeError, match="KvCachePagingParams"):
        native.kv_cache_extend(paged(), **good)
    with pytest.raises(ValueError, match="^block_table: expected a contiguous"):
        native.kv_cache_extend(p, **{**good, "block_table": ints(30).view(3, 10)[:, :5]})
    with pytest.raises(ValueError, match="^starts: the call needs 12"):
        native.kv_cache_slots(p, ints(3), good["block_table"], good["index"], ints(4), starts=ints(2))
    with pytest.raises(ValueError, match="^keep: expected torch.int32"):
        native.kv_cache_truncate(p, ints(3), good["block_table"], ints(20), ints(1), ints(3), ints(1), keep=torch.zeros(3, dtype=torch.int64))


def test_binding_refuses_bad_forms():
    c, p = cache(), paged()
    rows = torch.zeros(8 * 2 * 32 * 192, dtype=torch.bfloat16)
    args = dict(q=torch.zeros(6, 4, 192, dtype=torch.bfloat16), k_cache=rows, ckv_cache=rows, seq_lens=ints(2),
                out=torch.zeros(6, 4, 128, dtype=torch.bfloat16), workspace=torch.zeros(1 << 20, dtype=torch.uint8),
                block_table=ints(8).view(2, 4))
    with pytest.raises(TypeError, match="AttentionWindow"):
        native.paged_window_attention(c, p, X(5), **args)
    with pytest.raises(ValueError, match="^q: the call needs"):
        native.paged_window_attention(c, p, W(5), **{**args, "q": args["q"][:5].contiguous()})
    more = dict(prefix_len=ints(1), prefix_table=ints(4))
    with pytest.raises(TypeError, match="AttentionPrefix"):
        native.paged_prefix_attention(c, p, W(5), **args, **more)
    with pytest.raises(ValueError, match="^prefix_table: the call needs 20"):
        native.paged_prefix_attention(c, p, X(5, 5), **args, **more)
    with pytest.raises(ValueError, match="^prefix_len: expected torch.int32"):
        native.paged_prefix_attention(c, p, X(5), **args, **{**more, "prefix_len": torch.zeros(1, dtype=torch.int64)})
    with pytest.raises(ValueError, match="^block_table: expected .2, pages"):
        native.paged_prefix_attention(c, p, X(5), **{**args, "block_table": ints(8)}, **more)
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        native.paged_prefix_attention(c, p, X(5, 0), **args, **more)
    q = torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    pp = native.packed_attention_params(q, q, q, q, causal=True)
    with pytest.raises(TypeError, match="AttentionWindow"):
        native.packed_window_attention(pp, pp, q, q, q, q, args["workspace"])
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        native.packed_window_attention(pp, W(5), q, q, q, q, args["workspace"])


# ---------------------------------------------------------------- kernels
@pytest.mark.parametrize("file,kernel,budget", [
    ("packed_window.cu", "tile_attention_kernel", {168: 4}),
    ("paged_tile_extended.cu", "tile_attention_kernel", {168: 4, 128: 4}),
    ("paged_extended.cu", "paged_attention_kernel", {128: 4}),
    ("paged_tokens.cu", "paged_tokens_kernel", {168: 16}),   # 2 x 208 + 88 = 3 x 168
])
def test_register_budgets(file, kernel, budget, tmp_path):
    """As for the calls without a window or prefix: what the warpgroups give out is what they were
    launched with."""
    try:
        build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    rep = ptxas_report(file, str(tmp_path))
    hits = [v for n, v in rep.items() if kernel in n]
    assert {r: sum(h[0] == r for h in hits) for r in {h[0] for h in hits}} == budget, hits
    assert all(spill <= (384 if 128 in budget and 168 in budget else 192) for _, spill in hits), hits
    assert all((regs <= 64 and spill <= 128) if "Li4" in n else (regs <= 128 and spill == 0)
               for n, (regs, spill) in rep.items() if "attention_join_kernel" in n)


def test_paging_kernels_fit_1024_threads(tmp_path):
    try:
        build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    rep = ptxas_report("cache_paging.cu", str(tmp_path))
    assert len(rep) == 7 and all(regs <= 64 and spill == 0 for regs, spill in rep.values()), rep


# ---------------------------------------------------------------- the oracle
def test_oracle_windows():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((9, 4)), rng.standard_normal((9, 3))
    # equal scores: the mean of what is seen
    o, lse, _ = oracle.attention.attend(np.zeros((9, 4)), k, v, 1.0, True, window=3, sinks=2)
    for i in range(9):
        seen = [j for j in range(i + 1) if j > i - 3 or j < 2]
        assert np.allclose(o[i], v[seen].mean(0)) and np.isclose(lse[i], np.log(len(seen)))
    # a window over everything, or sinks over everything, is no window
    want = oracle.attention.attend(k, k, v, 0.5, True)
    for kw in (dict(window=9), dict(window=1, sinks=9)):
        assert all(np.array_equal(a, b) for a, b in zip(want, oracle.attention.attend(k, k, v, 0.5, True, **kw)))
    # a window of one key without sinks: the query's own
    assert np.allclose(oracle.attention.attend(k, k, v, 0.5, True, window=1)[0], v)
    # more queries than keys: the first rows see nothing
    o, lse, _ = oracle.attention.attend(rng.standard_normal((11, 4)), k, v, 1.0, True, window=4, sinks=1)
    assert (o[:2] == 0).all() and (lse[:2] == -np.inf).all() and np.allclose(o[2], v[0])


def test_oracle_prefix_is_attention_over_both():
    rng = np.random.default_rng(1)
    bs, P, own = 16, 21, 19
    kc, vc = (rng.integers(0, 1 << 14, (6, 2, bs, 8)).astype(np.uint16) for _ in range(2))
    q = rng.standard_normal((3, 4, 8))
    kw = dict(variant=2, starts_q=[0, 3], scale=0.3, causal=True, block_size=bs)
    got = oracle.attention.paged_attention(q, kc, vc, seq_lens=[own], table=[[3, 1]], prefix_len=P, prefix_table=[5, 0], **kw)
    # the same rows laid out as one sequence
    one = lambda c: np.concatenate([c[5], c[0][:, :P - bs], c[3], c[1][:, :own - bs]], axis=1)
    flat = lambda c: np.moveaxis(np.pad(one(c), ((0, 0), (0, 48 - P - own), (0, 0))).reshape(2, 3, bs, 8), 1, 0)
    want = oracle.attention.paged_attention(q, flat(kc), flat(vc), seq_lens=[P + own], table=[[0, 1, 2]], **kw)
    for x in ("out", "lse", "spread"):
        assert np.allclose(got[x], want[x])


def test_oracle_paging_by_hand():
    table = np.array([[7, -1, -1], [3, 4, -1]])
    r = oracle.paging.extend([3, 20], [15, 30], table, [9, 8, 6, 0], 3, block_num=10, block_size=16, max_tokens=25)
    # the first takes page 6 (the top); 30 + 20 passes the second's row of 48
    assert r["table"].tolist() == [[7, 6, -1], [3, 4, -1]] and r["new_free_count"] == 2
    assert r["new_seq_lens"].tolist() == [18, 30] and r["errors"] == 1
    assert r["index"].tolist() == [7 * 16 + 15, 96, 97] + [-1] * 22 and r["cu_seqlens"].tolist() == [0, 3, 23]
    r = oracle.paging.extend([3, 18], [15, 30], table, [9, 8, 6, 0], 3, block_num=10, block_size=16, max_tokens=21)
    assert r["table"].tolist() == [[7, 6, -1], [3, 4, 8]] and r["new_free_count"] == 1 and r["errors"] == 0
    assert r["index"][3:6].tolist() == [4 * 16 + 14, 4 * 16 + 15, 8 * 16]
    back = oracle.paging.truncate([15, 30], r["new_seq_lens"], r["table"], [9, -1, -1, -1], 1, block_num=10, block_size=16)
    assert back["free_pages"][:3].tolist() == [9, 8, 6] and back["new_free_count"] == 3
    s = oracle.paging.slots([14], [4], np.array([[2, 11]]), block_num=10, block_size=16, max_tokens=5)
    assert s["index"].tolist() == [46, 47, -1, -1, -1] and s["errors"] == 2 and s["cu_seqlens"].tolist() == [0, 4]


def test_block_tables_stay_within_31_bits(L):
    for stride, code in (((1 << 31) - 256, 0), ((1 << 31) - 255, -2), ((1 << 31) - 1, -2)):
        for name in ("kv_cache_extend", "kv_cache_slots", "kv_cache_truncate"):
            st, msg = call_paging(L, name, paging(B=1, block_table_stride=stride))
            assert st == code and (st == 0) == (msg == "")
