"""The attention operators as a serving loop uses them: behind the projection and the cache
writer, replayed from CUDA graphs, on streams of their own, with stalled pipelines, between
guard bands, over many items per block, and with non-finite rows."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from attention_util import HALF_STEP, TORCH, check_attention, half_values
from rope_attention_gb300 import native, runner, synth

pytestmark = pytest.mark.gpu

DEFAULT_WAIT_NS = 2_000_000_000


class Packed:
    """Sequences of lens tokens, bf16, with their oracle."""

    def __init__(self, seed, lens, nq, nkv, d, causal, dtype="bf16"):
        self.starts = [0] + list(np.cumsum(lens))
        self.d, self.causal, self.dtype = d, causal, dtype
        (qb, self.qv), (kb, self.kv), (vb, self.vv) = (half_values(seed, i, (self.starts[-1], n, d), dtype)
                                                       for i, n in enumerate((nq, nkv, nkv)))
        self.q, self.k, self.v = (torch.from_numpy(b.view(np.int16)).cuda().view(TORCH[dtype]) for b in (qb, kb, vb))
        self.out = torch.full_like(self.q, 7.0)
        self.lse = torch.full((self.starts[-1], nq), 7.0, device="cuda")
        self.cu = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.params = native.packed_attention_params(self.q, self.k, self.v, self.out, B=len(lens), causal=causal)
        self.ws = torch.zeros(native.packed_attention_workspace_bytes(self.params), dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        native.packed_attention(self.params, self.q, self.k, self.v, self.out, self.ws, self.lse, self.cu, self.cu, stream)

    def status(self):
        return native.attention_status(self.ws)

    def check(self, what):
        ref = oracle.attention.packed_attention(self.qv, self.kv, self.vv, starts_q=self.starts, starts_k=self.starts,
                                                scale=self.params.softmax_scale, causal=self.causal)
        check_attention(self.out, self.lse, ref, what, dtype=self.dtype, Dk=self.d)


class Paged:
    """New tokens over a cache that kv_rms_norm_rope_cache wrote; V2, or V1 with 16-bit or int8 rows."""

    def __init__(self, seed, lens, news, heads, N=1, variant=2, quant=False, block_size=32):
        B, S = len(lens), max(lens)
        pages = -(-S // block_size)
        dims = dict(Dkv=576, Dv=512) if variant == 1 else dict(Dkv=192, Dv=128)
        case = synth.make_kv("use", seed, variant=variant, B=B, N=N, S=S, block_size=block_size, block_num=B * pages + 1,
                             quant_k=quant, quant_v=quant, **dims)
        table = synth.stream(seed, 50).permutation(B * pages + 1)[:B * pages].reshape(B, pages).astype(np.int32)
        pos = np.arange(S)
        case.index = (table[:, pos // block_size].astype(np.int64) * block_size + pos % block_size).reshape(case.index.shape)
        self.kv = runner.KvRun(case)
        self.starts = [0] + list(np.cumsum(news))
        qb, self.qv = half_values(seed, 60, (self.starts[-1], heads, dims["Dkv"]), "bf16", std=0.5)
        q = torch.from_numpy(qb.view(np.int16)).cuda().view(torch.bfloat16)
        self.lens, self.table, self.variant, self.quant = lens, table, variant, quant
        self.run_ = runner.PagedAttentionRun(self.kv, q, lens, table, self.starts)
        self.run_.out.fill_(7.0)
        self.out, self.lse = self.run_.out, self.run_.lse

    def run(self, stream=None):
        self.run_.run(stream)

    def status(self):
        return self.run_.status()

    def check(self, what, qv=None, lens=None, starts=None, out=None, lse=None):
        """Against the oracle's attention over the bytes that are in the cache."""
        c = self.kv.case
        if qv is None:
            qv, lens, starts, out, lse = self.qv, self.lens, self.starts, self.out, self.lse
        host = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy()
        kt = c.k_qtype if self.quant else "bf16"
        q = self.quant
        ref = oracle.attention.paged_attention(
            qv, host(self.kv.k_cache), host(self.kv.ckv_cache), variant=self.variant, seq_lens=lens,
            starts_q=starts, scale=c.Dkv ** -0.5, causal=True, cache_mode=c.cache_mode, block_size=c.block_size,
            table=self.table, k_type=kt, v_type=c.v_qtype if q else "bf16", k_scale=c.k_scale, k_offset=c.k_offset,
            v_scale=c.v_scale, v_offset=c.v_offset)
        g = qv.shape[1] // c.N
        per_head = lambda x: None if x is None else np.repeat(x, g, axis=0) if x.ndim == 2 else x
        check_attention(out, lse, ref, what, dtype="bf16", Dk=c.Dkv, p_type="fp16" if q else "bf16",
                        q_step=2.0 ** -11 if q else 0.0, v_scale=per_head(c.v_scale), v_offset=per_head(c.v_offset),
                        keys=max(lens))
        assert int(self.run_.err) == 0


# one case for each kernel
CASES = {
    "packed": lambda s: Packed(s, [200, 90], 4, 2, 128, True),
    "packed_small_heads": lambda s: Packed(s, [500], 2, 2, 64, False),
    "decode": lambda s: Paged(s, [300, 77], [1, 1], 8, N=2),
    "decode_int8": lambda s: Paged(s, [300, 77], [1, 1], 8, N=2, quant=True),
    "decode_v1": lambda s: Paged(s, [300, 77], [1, 2], 16, variant=1),
    "decode_v1_int8": lambda s: Paged(s, [300, 77], [1, 2], 16, variant=1, quant=True),
    "chunk": lambda s: Paged(s, [300, 120], [120, 120], 4, N=2),
    "chunk_int8": lambda s: Paged(s, [300, 120], [120, 120], 4, N=2, quant=True),
}


def write_cache(x):
    if isinstance(x, Paged):
        x.kv.run()


@pytest.mark.parametrize("name", CASES)
def test_stalled_pipeline_reports_timeout_and_context_survives(name):
    x = CASES[name](1)
    write_cache(x)
    torch.cuda.synchronize()
    native.ra_set_wait_timeout_ns(2_000_000)  # 2 ms per wait
    try:
        native.ra_test_stall_next_attention()
        x.run()
        ws = x.ws if isinstance(x, Packed) else x.run_.workspace
        v = ctypes.c_int32()
        st = native.load().attention_status(ctypes.c_void_p(ws.data_ptr()), None, ctypes.byref(v))
        assert st == -6 and v.value == 1, (st, v.value)
        assert "ran out of time" in native.load().ra_last_error().decode()
        # cleared by the read; the hook applied to one launch only
        x.run()
        torch.cuda.synchronize()
        assert x.status() == 0
    finally:
        native.ra_set_wait_timeout_ns(DEFAULT_WAIT_NS)
    x.check("call after a timed-out launch")


@pytest.mark.parametrize("name", CASES)
def test_replays_from_a_cuda_graph(name):
    x, y = CASES[name](2), CASES[name](3)  # two graphs, each with its own workspace
    graphs = []
    for c in (x, y):
        write_cache(c)
        c.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    first = x.out.clone()
    for c in (x, y):
        c.out.fill_(7.0)
    # both at once, on streams of their own
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert x.status() == 0 and y.status() == 0
    x.check("graph replay")
    y.check("graph replay beside another")
    assert torch.equal(x.out.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("name", ["packed", "decode_int8", "chunk"])
def test_on_a_stream_behind_the_writer(name):
    """Writer and reader on one stream that is not the current one: nothing else orders them."""
    x = CASES[name](4)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    if isinstance(x, Paged):
        x.kv.run(s.cuda_stream)
    for stream in (s.cuda_stream, s):  # the second call reuses the workspace that the first one's join reads
        x.run(stream)
    s.synchronize()
    assert x.status() == 0
    x.check("on its own stream")


def test_prompt_from_the_projection():
    """row_quantize -> qkv_cte_mx -> packed_attention, in both layouts of the projection."""
    outs = []
    for layout in (native.RA_LAYOUT_BSD, native.RA_LAYOUT_NBSD):
        case = synth.make_qkv("use_q", 5, B=2, S=150, H=256, num_heads=4, num_kv_heads=2, head_dim=64)
        q = runner.QkvRun(case, layout=layout)
        q.run()
        a = runner.PackedAttentionRun(q, causal=True)
        a.run()
        torch.cuda.synchronize()
        assert q.status() == 0 and a.status() == 0
        vals = [t.double().cpu().numpy() for t in (a.q, a.k, a.v)]
        ref = oracle.attention.packed_attention(*vals, starts_q=[0, 150, 300], starts_k=[0, 150, 300], scale=0.125, causal=True)
        check_attention(a.out, a.lse, ref, "behind the projection", dtype="bf16", Dk=64)
        outs.append(a.out)
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("variant,quant", [(2, False), (2, True), (1, False), (1, True)])
def test_prompt_then_decode_over_the_cache(variant, quant):
    """kv_rms_norm_rope_cache writes a prompt; the chunk kernel, the decode kernel and
    kv_cache_read read it."""
    lens, heads = [130, 130], 4
    x = Paged(6, lens, [100, 100], heads, variant=variant, quant=quant)
    x.kv.run()
    x.run()
    torch.cuda.synchronize()
    x.check("chunk")
    c = x.kv.case
    for i in (0, 37, 99):               # token i of the chunk, as a step of its own
        seen = [n - 100 + i + 1 for n in lens]
        q = torch.stack([x.run_.q[i], x.run_.q[100 + i]]).contiguous()
        one = runner.PagedAttentionRun(x.kv, q, seen, x.table)
        one.run()
        torch.cuda.synchronize()
        assert one.status() == 0
        x.check("one token", np.stack([x.qv[i], x.qv[100 + i]]), seen, [0, 1, 2], one.out, one.lse)
    dt = torch.bfloat16
    ko = torch.empty(c.B, c.N, c.S, c.k_width, dtype=dt, device="cuda")
    vo = torch.empty(c.B, c.N, c.S, c.ckv_width, dtype=dt, device="cuda")
    native.kv_cache_read(x.kv.params, x.kv.index, x.kv.k_cache, x.kv.ckv_cache, ko, vo, x.kv.k_scale, x.kv.v_scale,
                         x.kv.k_offset, x.kv.v_offset)
    if not quant:
        assert torch.equal(ko, x.kv.k_rope) and torch.equal(vo, x.kv.c_kv)
    # the rows read back, attended as packed prompts: the same keys and values in 16 bits
    if variant == 2 and not quant:
        return
    keys = torch.cat([vo, ko], -1) if variant == 1 else ko
    k, v = keys[:, 0].reshape(-1, c.Dkv).double().cpu(), vo[:, 0].reshape(-1, c.ckv_width).double().cpu()
    q = torch.from_numpy(x.qv[99])
    p = torch.softmax(q @ k[:130].T * c.Dkv ** -0.5, -1)
    # The read rows are rounded to bf16: a score moves by 2^-8 of its reach, which moves the
    # result by twice that of the values' size (and by the square of it: 2^-8 reach < 1 / 8 here),
    # and the values move by 2^-8.  The kernel's own: 2^-8 for out and for P, 2^-11 of the reach.
    # A quantised value's size is that of its code over the scale.
    reach = float((q.abs() @ k[:130].abs().T).max()) * c.Dkv ** -0.5
    assert reach < 32
    size = float(v[:130].abs().max())
    if c.v_offset is not None:
        size += float(np.abs(c.v_offset / c.v_scale).max())
    tol = (3 * reach + 3) * 2.0 ** -8 * size
    assert (x.out[99].double().cpu() - p @ v[:130]).abs().max() <= tol


@pytest.mark.parametrize("lens,nq,causal", [
    ([40] * 20, 128, True),                # strided whole items: 16 or more for each block
    ([40] * 37 + [0] * 5 + [300], 64, True),  # the same over more sequences than a warp holds
    ([9, 300, 0, 33] * 30, 32, True),      # whole items in consecutive runs, over many sequences
    ([9, 300, 0, 33] * 30, 32, False),
    ([1] * 300, 16, False),
], ids=["strided", "strided_more", "runs_causal", "runs_full", "single_tokens"])
def test_many_items_per_block(lens, nq, causal):
    x = Packed(7, lens, nq, max(1, nq // 4), 64, causal)
    x.run()
    torch.cuda.synchronize()
    assert x.status() == 0
    x.check("many items")


def test_long_prompt_is_cut_and_joined():
    # few row blocks against many keys: every item is cut, over eight pieces and more
    for lq, lk in ((3, 40000), (300, 9000)):
        (qb, qv), (kb, kv), (vb, vv) = (half_values(8, i, (n, 1, 128), "bf16") for i, n in enumerate((lq, lk, lk)))
        q, k, v = (torch.from_numpy(b.view(np.int16)).cuda().view(torch.bfloat16) for b in (qb, kb, vb))
        out, lse = torch.full_like(q, 7.0), torch.full((lq, 1), 7.0, device="cuda")
        p = native.packed_attention_params(q, k, v, out, causal=True)
        ws = torch.zeros(native.packed_attention_workspace_bytes(p), dtype=torch.uint8, device="cuda")
        native.packed_attention(p, q, k, v, out, ws, lse)
        torch.cuda.synchronize()
        ref = oracle.attention.packed_attention(qv, kv, vv, starts_q=[0, lq], starts_k=[0, lk], scale=p.softmax_scale, causal=True)
        check_attention(out, lse, ref, "cut", dtype="bf16", Dk=128)


def test_outputs_stay_between_their_bands():
    """Rows of out apart from one another (strides wider than the rows), and bands around out
    and lse: what lies between is left as it was."""
    T, n, d = 300, 3, 48
    x = Packed(9, [130, 170], n, 1, d, True)
    for layout in ("tokens", "heads"):
        wide = torch.full((T + 2, n, d + 16) if layout == "tokens" else (n, T + 2, d + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        out = wide[1:-1, :, :d] if layout == "tokens" else wide[:, 1:-1, :d].transpose(0, 1)
        lse = torch.full((T + 2, n), 7.0, device="cuda")
        p = native.packed_attention_params(x.q, x.k, x.v, out, B=2, causal=True)
        ws = torch.full((native.packed_attention_workspace_bytes(p) + 256,), 0, dtype=torch.uint8, device="cuda")
        ws[-256:] = 77
        native.packed_attention(p, x.q, x.k, x.v, out, ws[:-256], lse[1:-1], x.cu, x.cu)
        torch.cuda.synchronize()
        x.out, x.lse = out.contiguous(), lse[1:-1]
        x.check(layout)
        keep = wide.clone()
        (keep[1:-1, :, :d] if layout == "tokens" else keep[:, 1:-1, :d]).fill_(7.0)
        assert (keep == 7).all() and (lse[0] == 7).all() and (lse[-1] == 7).all() and (ws[-256:] == 77).all()


@pytest.mark.parametrize("name", ["decode", "decode_v1_int8", "chunk", "chunk_int8"])
def test_paged_outputs_stay_between_their_bands(name):
    x = CASES[name](10)
    write_cache(x)
    shape, r = x.out.shape, x.run_
    out = torch.full((shape[0] + 2, *shape[1:]), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((shape[0] + 2, shape[1]), 7.0, device="cuda")
    n = r.workspace.numel()
    ws = torch.zeros(n + 256, dtype=torch.uint8, device="cuda")
    ws[-256:] = 77
    r.out, r.lse, r.workspace = out[1:-1], lse[1:-1], ws[:n]
    x.out, x.lse = r.out, r.lse
    x.run()
    torch.cuda.synchronize()
    x.check("bands")
    assert (out[0] == 7).all() and (out[-1] == 7).all() and (lse[0] == 7).all() and (lse[-1] == 7).all() and (ws[-256:] == 77).all()


@pytest.mark.parametrize("name", CASES)
def test_a_nan_query_is_its_own_rows_alone(name):
    x, y = CASES[name](11), CASES[name](11)
    q = x.q if isinstance(x, Packed) else x.run_.q
    q[0, 1, 3] = float("nan")
    for c in (x, y):
        write_cache(c)
        c.run()
    torch.cuda.synchronize()
    assert torch.isnan(x.out[0, 1]).all() and torch.isnan(x.lse[0, 1])
    x.out[0, 1], x.lse[0, 1] = y.out[0, 1], y.lse[0, 1]
    x.check("the other rows")


@pytest.mark.parametrize("name", CASES)
def test_a_second_call_gives_the_same_bits(name):
    x = CASES[name](12)
    write_cache(x)
    x.run()
    first, lse = x.out.clone(), x.lse.clone()
    for _ in range(5):
        x.out.fill_(7.0)
        x.run()
        assert torch.equal(x.out.view(torch.int16), first.view(torch.int16)) and torch.equal(x.lse, lse)


@pytest.mark.parametrize("name", ["decode", "chunk_int8"])
def test_blockwise_written_caches_have_the_bnsd_layout(name):
    x = CASES[name](13)
    write_cache(x)
    x.run()
    first = x.out.clone()
    x.out.fill_(7.0)
    x.kv.params.cache_mode = native.RA_CACHE_PA_BLK_BNSD
    x.run()
    assert torch.equal(x.out.view(torch.int16), first.view(torch.int16))


def test_two_threads_call_at_once():
    """Two host threads, each with its own stream, workspace and case."""
    import threading

    cases, errors = [CASES["decode"](14), CASES["chunk_int8"](15)], []
    for c in cases:
        write_cache(c)
    torch.cuda.synchronize()

    def work(c):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                c.run(s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001 -- reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for c in cases:
        assert c.status() == 0
        c.check("beside another thread")


def test_rows_and_strides_past_32_bits():
    """Pages and heads more than 2^32 bytes into their tensors."""
    Dk, Dv, bs, pages = 192, 128, 128, 90000        # 4.4 GB of keys, 2.9 GB of values
    kc = torch.empty(pages, 1, bs, Dk, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty(pages, 1, bs, Dv, dtype=torch.bfloat16, device="cuda")
    table = np.array([[pages - 1, 3, pages - 2]], np.int32)
    (kb, kv), (vb, vv) = (half_values(16, i, (3, 1, bs, w), "bf16") for i, w in enumerate((Dk, Dv)))
    at = torch.from_numpy(table[0].astype(np.int64)).cuda()
    kc[at] = torch.from_numpy(kb.view(np.int16)).cuda().view(torch.bfloat16)
    vc[at] = torch.from_numpy(vb.view(np.int16)).cuda().view(torch.bfloat16)
    cache = native.KvRmsNormRopeCacheParams(B=1, N=1, S=300, Dkv=Dk, Dv=Dv, rope_size=64, variant=2,
                                            cache_mode=native.RA_CACHE_PA_BNSD, block_num=pages, block_size=bs,
                                            kv_dtype=native.RA_BF16, k_cache_dtype=native.RA_BF16,
                                            ckv_cache_dtype=native.RA_BF16, epsilon=1e-5)
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    keys, values = kv.transpose(0, 2, 1, 3).reshape(-1, 1, Dk)[:300], vv.transpose(0, 2, 1, 3).reshape(-1, 1, Dv)[:300]
    for new in (1, 90):
        qb, qv = half_values(16, 5, (new, 2, Dk), "bf16")
        q = torch.from_numpy(qb.view(np.int16)).cuda().view(torch.bfloat16)
        out, lse = torch.empty(new, 2, Dv, dtype=torch.bfloat16, device="cuda"), torch.empty(new, 2, device="cuda")
        p = native.PagedAttentionParams(B=1, total_q=new, num_heads=2, causal=1, softmax_scale=Dk ** -0.5, max_seq_len=300,
                                        block_table_stride=3)
        ws = torch.zeros(native.paged_attention_workspace_bytes(cache, p), dtype=torch.uint8, device="cuda")
        native.paged_attention(cache, p, q, kc, vc, lens, out, ws, torch.from_numpy(table).cuda(), lse=lse)
        ref = oracle.attention.packed_attention(qv, keys, values, starts_q=[0, new], starts_k=[0, 300], scale=p.softmax_scale,
                                                causal=True)
        check_attention(out, lse, ref, "far pages", dtype="bf16", Dk=Dk)
    index = torch.from_numpy((table[0][:, None].astype(np.int64) * bs + np.arange(bs)).reshape(-1)[:300].copy()).cuda()
    ko = torch.empty(1, 1, 300, Dk, dtype=torch.bfloat16, device="cuda")
    native.kv_cache_read(cache, index, kc, vc, ko, None)
    assert np.array_equal(ko[0, 0].double().cpu().numpy(), keys[:, 0])
    del kc, vc

    # two heads 2^31 + 64 elements apart, inputs and output
    far = 2 ** 31 + 64
    buf = torch.empty(far + 4 * 200 * 64, dtype=torch.bfloat16, device="cuda")
    x = Packed(17, [200], 2, 2, 64, True)
    views = []
    for i, t in enumerate((x.q, x.k, x.v, x.out)):
        v = buf[i * 200 * 64:].as_strided((200, 2, 64), (64, far, 1))
        v.copy_(t)
        views.append(v)
    p = native.packed_attention_params(*views, causal=True)
    ws = torch.zeros(native.packed_attention_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    native.packed_attention(p, *views, ws, x.lse)
    torch.cuda.synchronize()
    x.out = views[3].contiguous()
    x.check("heads far apart")
