"""The calls with windows and shared prefixes and those of the pages as a server uses them: with stalled
pipelines, replayed from CUDA graphs beside one another, on streams of their own, between guard bands and
on workspaces of any 16 bytes, with non-finite queries, and together: pages for new tokens, their keys
and values, the attention over them, pages given back."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from attention_util import check_attention, half_values
from paged_forms_util import Case, check_rows
from rope_attention_gb300 import native, runner, synth
from test_attention_use import DEFAULT_WAIT_NS, Packed

pytestmark = pytest.mark.gpu


class PackedWindow(Packed):
    def __init__(self, seed, lens, nq, nkv, d, window, sinks):
        super().__init__(seed, lens, nq, nkv, d, True)
        self.window, self.sinks = window, sinks

    def run(self, stream=None, out=None, lse="own"):
        native.packed_window_attention(self.params, native.AttentionWindow(window=self.window, sinks=self.sinks), self.q, self.k,
                                       self.v, self.out if out is None else out, self.ws, self.lse if lse == "own" else lse,
                                       self.cu, self.cu, stream)

    def check(self, what):
        ref = oracle.attention.packed_attention(self.qv, self.kv, self.vv, starts_q=self.starts, starts_k=self.starts,
                                                scale=self.params.softmax_scale, causal=True, window=self.window, sinks=self.sinks)
        check_attention(self.out, self.lse, ref, what, dtype=self.dtype, Dk=self.d)


V1 = dict(variant=1, heads=16, Dkv=576, Dv=512)
FEW = dict(variant=2, heads=8, N=2)
SHARED = dict(variant=2, lens=[(7 * i) % 40 for i in range(96)], news=[1] * 96, heads=16, N=8, prefix=1100)
# one case and more for each kernel and form
CASES = {
    "packed": lambda s: PackedWindow(s, [200, 90], 4, 2, 128, 70, 3),
    "packed_cut": lambda s: PackedWindow(s, [3, 2000], 1, 1, 64, 900, 5),
    "window_few_rows": lambda s: Case(s, lens=[900, 77], news=[1, 2], window=600, sinks=4, **FEW),
    "window_few_rows_int8": lambda s: Case(s, lens=[900, 77], news=[1, 1], window=600, sinks=4, kt="int8", vt="int8", **FEW),
    "window_rows": lambda s: Case(s, lens=[900, 77], news=[9, 9], window=600, sinks=4, kt="int8", vt="int8", **FEW),
    "window_v1_int8": lambda s: Case(s, lens=[900, 77], news=[1, 2], window=600, sinks=4, kt="int8", vt="int8", **V1),
    "window_chunk": lambda s: Case(s, lens=[900, 150], news=[120, 120], window=300, sinks=4, **FEW),
    "prefix_few_rows": lambda s: Case(s, lens=[90, 77], news=[1, 2], prefix=300, kt="int8", vt="int8", **FEW),
    "prefix_v1": lambda s: Case(s, lens=[90, 77], news=[1, 2], prefix=300, **V1),
    "prefix_chunk_int8": lambda s: Case(s, lens=[200, 150], news=[120, 120], prefix=300, kt="int8", vt="int8", **FEW),
    "prefix_shared": lambda s: Case(s, kt="int8", vt="int8", **SHARED),
    "prefix_shared_v1": lambda s: Case(s, lens=[(5 * i) % 30 for i in range(150)], news=[1] * 150, prefix=4000, **V1),
}


def done(x):
    torch.cuda.synchronize()
    assert x.status() == 0


@pytest.mark.parametrize("name", CASES)
def test_stalled_pipeline_reports_timeout_and_context_survives(name):
    x = CASES[name](1)
    torch.cuda.synchronize()
    native.ra_set_wait_timeout_ns(2_000_000)  # 2 ms per wait
    try:
        native.ra_test_stall_next_attention()
        x.run()
        v = ctypes.c_int32()
        st = native.load().attention_status(ctypes.c_void_p(x.ws.data_ptr()), None, ctypes.byref(v))
        assert st == -6 and v.value == 1, (st, v.value)
        x.run()                        # cleared by the read; the hook applied to one call only
        done(x)
    finally:
        native.ra_set_wait_timeout_ns(DEFAULT_WAIT_NS)
    x.check("call after a timed-out launch")


@pytest.mark.parametrize("name", CASES)
def test_replays_from_cuda_graphs_beside_one_another(name):
    x, y = CASES[name](2), CASES[name](3)  # two graphs, each with its own workspace
    graphs = []
    for c in (x, y):
        c.run()
        done(c)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    first = [c.out.clone() for c in (x, y)]
    for c in (x, y):
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, f in zip((x, y), first):
        assert c.status() == 0
        c.check("graph replay")
        assert torch.equal(c.out.view(torch.int16), f.view(torch.int16))


@pytest.mark.parametrize("name", CASES)
def test_calls_behind_one_another_on_a_stream_of_their_own(name):
    # the next call's first launch writes the workspace that the last one's second launch reads
    x = CASES[name](4)
    s = torch.cuda.Stream()
    outs = [torch.full_like(x.out, 7.0) for _ in range(6)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        x.run(s.cuda_stream if i % 2 else s, out=o)
    x.run(s)
    s.synchronize()
    done(x)
    x.check("on its own stream")
    for o in outs:
        assert torch.equal(o.view(torch.int16), x.out.view(torch.int16))


@pytest.mark.parametrize("at", [0, 16])
@pytest.mark.parametrize("name", CASES)
def test_outputs_and_workspace_stay_between_their_bands(name, at):
    x = CASES[name](5)
    out = torch.full((x.out.shape[0] + 2, *x.out.shape[1:]), 7.0, dtype=x.out.dtype, device="cuda")
    lse = torch.full((x.lse.shape[0] + 2, x.lse.shape[1]), 7.0, device="cuda")
    n = x.ws.numel()
    ws = torch.full((at + n + 4096,), 77, dtype=torch.uint8, device="cuda")
    ws[at:at + n] = 0
    x.out, x.lse, x.ws = out[1:-1], lse[1:-1], ws[at:at + n]
    x.run()
    done(x)
    x.check("bands")
    for t in (out, lse):
        assert (t[0] == 7).all() and (t[-1] == 7).all()
    assert (ws[:at] == 77).all() and (ws[at + n:] == 77).all()


@pytest.mark.parametrize("name", CASES)
def test_a_nan_query_is_its_own_rows_alone(name):
    x, y = CASES[name](6), CASES[name](6)
    x.q[1, -1, 3] = float("nan")
    for c in (x, y):
        c.run()
        done(c)
    assert torch.isnan(x.out[1, -1]).all() and torch.isnan(x.lse[1, -1])
    x.out[1, -1], x.lse[1, -1] = y.out[1, -1], y.lse[1, -1]
    x.check("the other rows")


def test_runners_over_the_projection_and_the_cache():
    case = synth.make_qkv("use_q", 5, B=2, S=150, H=256, num_heads=4, num_kv_heads=2, head_dim=64)
    q = runner.QkvRun(case)
    q.run()
    a = runner.PackedAttentionRun(q, window=native.AttentionWindow(window=40, sinks=3))
    a.run()
    torch.cuda.synchronize()
    assert q.status() == 0 and a.status() == 0
    ref = oracle.attention.packed_attention(*(t.double().cpu().numpy() for t in (a.q, a.k, a.v)), starts_q=[0, 150, 300],
                                            starts_k=[0, 150, 300], scale=0.125, causal=True, window=40, sinks=3)
    check_attention(a.out, a.lse, ref, "behind the projection", dtype="bf16", Dk=64)


# ---------------------------------------------------------------- together
class Server:
    """Requests over one cache whose row 0 is their shared beginning.  The host holds nothing but what
    the oracle says: lengths, pages and starts stay on the device from call to call."""

    STRIDE, T = 12, 160                          # table entries a row, tokens a step at most

    def __init__(self, seed, kind, variant, heads, bs, B=5):
        self.B, self.bs, self.heads, self.variant, self.seed = B, bs, heads, variant, seed
        self.N = 1 if variant == 1 else 2
        dims = dict(Dkv=576, Dv=512) if variant == 1 else dict(Dkv=192, Dv=128)
        self.block_num = 40
        quant = kind != "bf16"
        self.case = lambda s: synth.make_kv("server", seed * 100 + s, variant=variant, B=1, N=self.N, S=self.T, block_size=bs,
                                            block_num=self.block_num, quant_k=quant, quant_v=quant, **dims)
        self.kv = runner.KvRun(self.case(0))
        self.c, self.kind, self.quant = self.kv.case, kind, quant
        dev = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")
        self.host = dict(lens=np.zeros(B, np.int32), table=np.full((B, self.STRIDE), -1, np.int32),
                         free=synth.stream(seed, 70).permutation(self.block_num).astype(np.int32), count=self.block_num)
        self.lens, self.table, self.free = (dev(self.host[k]) for k in ("lens", "table", "free"))
        self.count, self.err = dev([self.block_num]), dev([0])
        self.index = torch.empty(self.T, dtype=torch.int64, device="cuda")
        self.cu = torch.empty(B + 1, dtype=torch.int32, device="cuda")
        self.rows, self.step = [[] for _ in range(B)], 0
        self.scale = self.c.Dkv ** -0.5

    def paging(self, tokens=None):
        return native.KvCachePagingParams(B=self.B, block_num=self.block_num, block_size=self.bs, block_table_stride=self.STRIDE,
                                          max_tokens=self.T if tokens is None else tokens)

    def extend(self, new):
        """Pages for the new tokens, then their keys and values."""
        self.step += 1
        fresh = runner.KvRun(self.case(self.step))
        d = torch.tensor(new, dtype=torch.int32, device="cuda")
        native.kv_cache_extend(self.paging(), d, self.lens, self.table, self.free, self.count, self.index, self.cu, self.lens,
                               self.count, self.err)
        fresh.index, fresh.k_cache, fresh.ckv_cache = self.index, self.kv.k_cache, self.kv.ckv_cache
        fresh.k_scale, fresh.k_offset, fresh.v_scale, fresh.v_offset = (self.kv.k_scale, self.kv.k_offset, self.kv.v_scale,
                                                                        self.kv.v_offset)
        fresh.run()
        h = self.host
        want = oracle.paging.extend(new, h["lens"], h["table"], h["free"], h["count"], block_num=self.block_num, block_size=self.bs,
                                    max_tokens=self.T)
        assert want["errors"] == 0 and int(self.err) == 0 and int(fresh.err) == 0
        assert np.array_equal(self.index.cpu().numpy(), want["index"])
        h.update(lens=want["new_seq_lens"], table=want["table"], count=want["new_free_count"])
        at = 0
        for b, n in enumerate(new):              # the rows that the writer gave out beside the cache's
            self.rows[b] += [(fresh.k_rope[0, :, at + i], fresh.c_kv[0, :, at + i]) for i in range(n)]
            at += n
        self.fits()

    def truncate(self, keep):
        h = self.host
        native.kv_cache_truncate(self.paging(), self.lens, self.table, self.free, self.count, self.lens, self.count,
                                 keep=torch.tensor(keep, dtype=torch.int32, device="cuda"), dev_error_count=self.err)
        want = oracle.paging.truncate(keep, h["lens"], h["table"], h["free"], h["count"], block_num=self.block_num, block_size=self.bs)
        h.update(lens=want["new_seq_lens"], free=want["free_pages"], count=want["new_free_count"])
        self.rows = [r[:n] for r, n in zip(self.rows, h["lens"])]
        self.fits()

    def fits(self):
        h = self.host
        assert np.array_equal(self.lens.cpu().numpy(), h["lens"]) and int(self.count) == h["count"]
        held = [self.table[b, i].item() for b in range(self.B) for i in range(-(-int(h["lens"][b]) // self.bs))]
        free = self.free[:h["count"]].tolist()
        assert sorted(held + free) == list(range(self.block_num))       # every page once

    def attend(self, new, window=None, prefix=False):
        """The last new[b] tokens of rows 1.. over their positions, in a window or behind row 0's."""
        h, B = self.host, self.B - 1
        starts = [0] + list(np.cumsum(new))
        qb, qv = half_values(self.seed * 100 + self.step, 80, (starts[-1], self.heads, self.c.Dkv), "bf16", 0.5)
        q = torch.from_numpy(qb.view(np.int16)).cuda().view(torch.bfloat16)
        form = None if window is None else native.AttentionWindow(window=window[0], sinks=window[1])
        first = (int(h["lens"][0]), h["table"][0]) if prefix else None
        run = runner.PagedAttentionRun(self.kv, q, h["lens"][1:].tolist(), h["table"][1:], starts, window=form, prefix=first)
        run.lens, run.table, run.starts = self.lens[1:], self.table[1:], self.cu[1:]      # where the calls left them
        if prefix:
            run.prefix_len, run.prefix_table = self.lens[:1], self.table[0]
        run.run()
        torch.cuda.synchronize()
        assert run.status() == 0 and int(run.err) == 0
        host = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy()
        c, quant = self.c, self.quant
        kt, vt = (c.k_qtype, c.v_qtype) if quant else ("bf16", "bf16")
        ref = oracle.attention.paged_attention(
            qv, host(self.kv.k_cache), host(self.kv.ckv_cache), variant=self.variant, seq_lens=h["lens"][1:], starts_q=starts,
            scale=self.scale, causal=True, cache_mode=c.cache_mode, block_size=self.bs, table=h["table"][1:], k_type=kt, v_type=vt,
            k_scale=c.k_scale, k_offset=c.k_offset, v_scale=c.v_scale, v_offset=c.v_offset, window=window[0] if window else None,
            sinks=window[1] if window else 0, prefix_len=int(h["lens"][0]) if prefix else 0,
            prefix_table=h["table"][0] if prefix else None)
        per_head = lambda x: None if x is None else np.repeat(x, self.heads // self.N, axis=0) if x.ndim == 2 else x
        check_rows(run.out, run.lse, ref, f"step {self.step} {new} {window} {prefix}", dtype="bf16", Dk=c.Dkv,
                   p_type="fp16" if quant else "bf16", q_step=2.0 ** -11 if quant else 0.0, v_scale=per_head(c.v_scale),
                   v_offset=per_head(c.v_offset), keys=int(max(h["lens"][1:]) + h["lens"][0]), joined=prefix)
        assert B == len(new)

    def read(self):
        """Whole contexts, request after request: the rows that the writer gave out."""
        h, total = self.host, int(self.host["lens"].sum())
        index, cu = torch.empty(total, dtype=torch.int64, device="cuda"), torch.empty(self.B + 1, dtype=torch.int32, device="cuda")
        native.kv_cache_slots(self.paging(total), self.lens, self.table, index, cu, dev_error_count=self.err)
        assert cu.tolist() == [0] + np.cumsum(h["lens"]).tolist() and int(self.err) == 0
        p = runner.kv_params(self.c)
        p.B, p.S = 1, total
        k = torch.empty(1, self.N, total, self.c.k_width, dtype=torch.bfloat16, device="cuda")
        v = torch.empty(1, self.N, total, self.c.ckv_width, dtype=torch.bfloat16, device="cuda")
        r = self.kv
        native.kv_cache_read(p, index, r.k_cache, r.ckv_cache, k, v, r.k_scale, r.v_scale, r.k_offset, r.v_offset)
        rows = [x for b in range(self.B) for x in self.rows[b]]
        assert len(rows) == total
        for got, want, scale in ((k[0], torch.stack([x[0] for x in rows], 1), r.k_scale), (v[0], torch.stack([x[1] for x in rows], 1), r.v_scale)):
            if not self.quant:
                assert torch.equal(got, want)
                continue
            # a code is off by half a step of 1 / scale where it is not clipped (a row's values that leave
            # [-128, 127] after scale and offset are), a tie or the fp32 arithmetic before it by 2^-10 of a step
            # more, and both sides are rounded to bf16
            s = scale[:, None] if scale.dim() == 2 else scale
            o = r.k_offset if scale is r.k_scale else r.v_offset
            o = o[:, None] if o.dim() == 2 else o
            code = want.double() * s + o
            inside = (code > -127) & (code < 126)
            tol = (0.5 + 2.0 ** -10) / s + 2.0 ** -8 * (want.double().abs() + got.double().abs())
            assert inside.double().mean() > 0.8
            assert ((got.double() - want.double()).abs() <= tol)[inside].all()


@pytest.mark.parametrize("kind,variant,heads,bs", [("bf16", 2, 8, 32), ("bf16", 2, 16, 16), ("bf16", 1, 16, 32),
                                                   ("int8", 2, 8, 32), ("int8", 2, 16, 32), ("int8", 1, 16, 32)])
def test_requests_come_grow_and_go(kind, variant, heads, bs):     # (codes: pages of 32 slots at least)
    s = Server(1 + variant, kind, variant, heads, bs)
    s.extend([70, 0, 0, 0, 0])                        # what all begin with
    s.extend([0, 90, 33, 1, 5])                       # prompts
    s.attend([90, 33, 1, 5], prefix=True)
    s.attend([90, 33, 1, 5], window=(20, 3))
    for _ in range(3):
        s.extend([0, 1, 1, 1, 1])
        s.attend([1, 1, 1, 1], window=(40, 4))
        s.attend([1, 1, 1, 1], prefix=True)
    s.read()
    s.truncate([70, 1000, 30, 0, 2])                  # one goes on, one steps back, one ends
    s.extend([0, 2, 1, 60, 4])                        # another takes its row and its pages
    s.attend([2, 1, 60, 4], prefix=True)
    s.attend([2, 1, 60, 4], window=(7, 0))
    s.truncate([70, 0, 31, 60, 6])
    s.extend([0, 11, 0, 1, 1])
    s.attend([11, 0, 1, 1], prefix=True)
    s.attend([11, 0, 1, 1], window=(64, 1))
    s.read()
    s.truncate([0] * 5)
    assert s.host["count"] == s.block_num


def test_a_captured_decode_step():
    """Pages, keys and values, both attentions and one query set, replayed while the requests grow over
    page ends: lengths, table and list stay on the device."""
    s = Server(9, "int8", 2, 8, 32)
    s.extend([70, 0, 0, 0, 0])
    s.extend([0, 40, 15, 16, 1])
    T, heads = s.T, s.heads
    most = s.STRIDE * s.bs
    fresh = runner.KvRun(s.case(50))
    fresh.index, fresh.k_cache, fresh.ckv_cache = s.index, s.kv.k_cache, s.kv.ckv_cache
    fresh.k_scale, fresh.k_offset, fresh.v_scale, fresh.v_offset = s.kv.k_scale, s.kv.k_offset, s.kv.v_scale, s.kv.v_offset
    qb, qv = half_values(10, 0, (4, heads, s.c.Dkv), "bf16", 0.5)
    q = torch.from_numpy(qb.view(np.int16)).cuda().view(torch.bfloat16)
    new = torch.tensor([0, 1, 1, 1, 1], dtype=torch.int32, device="cuda")
    runs = [runner.PagedAttentionRun(s.kv, q, [most] * 4, s.host["table"][1:], window=native.AttentionWindow(window=20, sinks=2)),
            runner.PagedAttentionRun(s.kv, q, [most] * 4, s.host["table"][1:], prefix=(most, s.host["table"][0]))]
    for r in runs:
        r.lens, r.table = s.lens[1:], s.table[1:]
    runs[1].prefix_len, runs[1].prefix_table = s.lens[:1], s.table[0]

    def step():
        native.kv_cache_extend(s.paging(), new, s.lens, s.table, s.free, s.count, s.index, s.cu, s.lens, s.count, s.err)
        fresh.run()
        for r in runs:
            r.run()

    for r in runs:
        r.run()
    fresh.index = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    fresh.run()                                       # one eager call each; the writer's touches no row
    fresh.index = s.index
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    h, c = s.host, s.c
    for i in range(20):
        g.replay()
        torch.cuda.synchronize()
        want = oracle.paging.extend([0, 1, 1, 1, 1], h["lens"], h["table"], h["free"], h["count"], block_num=s.block_num,
                                    block_size=s.bs, max_tokens=T)
        h.update(lens=want["new_seq_lens"], table=want["table"], count=want["new_free_count"])
        s.fits()
        if i % 5:
            continue
        for r, form in zip(runs, (dict(window=20, sinks=2), dict(prefix_len=70, prefix_table=h["table"][0]))):
            assert r.status() == 0 and int(r.err) == 0
            ref = oracle.attention.paged_attention(
                qv, s.kv.k_cache.cpu().numpy(), s.kv.ckv_cache.cpu().numpy(), variant=2, seq_lens=h["lens"][1:], starts_q=[0, 1, 2, 3, 4],
                scale=s.scale, causal=True, cache_mode=c.cache_mode, block_size=s.bs, table=h["table"][1:], k_type=c.k_qtype,
                v_type=c.v_qtype, k_scale=c.k_scale, k_offset=c.k_offset, v_scale=c.v_scale, v_offset=c.v_offset, **form)
            per_head = lambda x: None if x is None else np.repeat(x, heads // s.N, axis=0)
            check_rows(r.out, r.lse, ref, f"replay {i} {form}", dtype="bf16", Dk=c.Dkv, p_type="fp16", q_step=2.0 ** -11,
                       v_scale=per_head(c.v_scale), v_offset=per_head(c.v_offset), keys=most, joined=True)
    assert int(s.err) == 0
