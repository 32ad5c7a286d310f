"""Calls from host threads.  Two threads at a time call one kernel with sizes that need different amounts
of shared memory, each on a stream and on tensors of its own: every call is accepted, whatever the other
thread launches between its checks and its launch.  And a call is the first CUDA call that its thread makes.
The results are the oracle's."""
import threading

import numpy as np
import pytest
import torch

import oracle
from parity_util import as_f64, check_kv, check_qkv, qkv_reference
from rope_attention_gb300 import native, runner, synth
from test_cache_paging import Pages, dev

pytestmark = pytest.mark.gpu


def beside_one_another(calls, times):
    """Each of `calls` (of a stream) `times` times, in a thread of its own."""
    start, errors = threading.Barrier(len(calls)), []

    def work(call):
        stream = torch.cuda.Stream()
        start.wait()
        try:
            for i in range(times):
                call(stream)
                if i % 100 == 99:
                    stream.synchronize()
        except Exception as e:  # noqa: BLE001 (reported below)
            errors.append(e)
        finally:
            stream.synchronize()

    for c in calls:                      # what a first call sets up
        c(torch.cuda.current_stream())
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors


class Paging:
    """extend, slots and truncate of B requests, none of them in place."""

    def __init__(self, seed, B):
        rng = np.random.default_rng(seed)
        p = self.p = Pages(seed, rng.integers(0, 60, B), 8, 16, 2 * B)
        self.new, self.keep = rng.integers(0, 3, B), rng.integers(0, 60, B)
        self.T = int(self.new.sum()) + 5
        self.params = p.params(self.T)
        self.lens, self.count, self.free = dev(p.lens), dev([p.count]), dev(p.free)
        self.table, self.full, self.back = dev(p.table), dev(p.table), dev(p.free)
        self.new_d, self.keep_d = dev(self.new), dev(self.keep)
        out = lambda n: torch.full((n,), 77, dtype=torch.int32, device="cuda")
        index = lambda: torch.full((self.T,), 77, dtype=torch.int64, device="cuda")
        self.extended = index(), out(B + 1), out(B), out(1)
        self.slots = index(), out(B + 1)
        self.cut = out(B), out(1)

    def __call__(self, stream):
        native.kv_cache_extend(self.params, self.new_d, self.lens, self.full, self.free, self.count, *self.extended, stream=stream)
        native.kv_cache_slots(self.params, self.new_d, self.table, *self.slots, stream=stream)
        native.kv_cache_truncate(self.params, self.lens, self.table, self.back, self.count, *self.cut, keep=self.keep_d, stream=stream)

    def check(self):
        p = self.p
        size = dict(block_num=p.block_num, block_size=p.bs)
        e = oracle.paging.extend(self.new, p.lens, p.table, p.free, p.count, max_tokens=self.T, **size)
        s = oracle.paging.slots(None, self.new, p.table, max_tokens=self.T, **size)
        t = oracle.paging.truncate(self.keep, p.lens, p.table, p.free, p.count, **size)
        got = (*self.extended, self.full, *self.slots, *self.cut, self.back)
        want = (e["index"], e["cu_seqlens"], e["new_seq_lens"], [e["new_free_count"]], e["table"], s["index"], s["cu_seqlens"],
                t["new_seq_lens"], [t["new_free_count"]], t["free_pages"])
        for i, (g, w) in enumerate(zip(got, want)):
            assert np.array_equal(g.cpu().numpy(), np.asarray(w)), i


def test_paging_calls_of_many_and_of_fewer_requests():
    calls = [Paging(1, 16384), Paging(2, 4000)]
    beside_one_another(calls, 2000)
    for c in calls:
        c.check()


@pytest.mark.parametrize("layout", [native.RA_LAYOUT_BSD, native.RA_LAYOUT_NBSD], ids=["bsd", "nbsd"])
@pytest.mark.parametrize("first", ["project", "norm_rope"])
def test_a_projection_call_is_its_threads_first(first, layout):
    c = synth.make_qkv("threads_first", 60, S=64, H=256, num_heads=2, num_kv_heads=2, head_dim=64)
    r = runner.QkvRun(c, layout=layout)
    stream, errors = torch.cuda.Stream(), []
    if first == "norm_rope":
        r.project(stream)

    def work():
        try:
            if first == "project":
                r.project(stream)
            r.norm_rope(stream)
        except Exception as e:  # noqa: BLE001 (reported below)
            errors.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert r.status() == 0
    out = r.out if layout == native.RA_LAYOUT_BSD else r.out.permute(1, 0, 2).reshape(c.T, c.I)
    check_qkv(c, as_f64(out), qkv_reference(c), "a thread's first call")


KV = dict(variant=2, B=2, block_size=32, skip_frac=0.1)
KV_PAIRS = {
    "pipelined": (dict(N=8, S=21, Dkv=192, Dv=128, quant_k=True, quant_v=True), dict(N=8, S=21, Dkv=192, Dv=128)),
    "register": (dict(N=8, S=9, Dkv=512, Dv=512, quant_k=True, quant_v=True), dict(N=8, S=9, Dkv=512, Dv=256, quant_k=True, quant_v=True)),
}


@pytest.mark.parametrize("name", KV_PAIRS)
def test_cache_writers_of_wide_and_of_narrow_tables(name):
    cases = [synth.make_kv(f"threads_{name}_{i}", 40 + i, **KV, **kw) for i, kw in enumerate(KV_PAIRS[name])]
    runs = [runner.KvRun(c) for c in cases]
    beside_one_another([r.run for r in runs], 4000)
    assert native.kv_rms_norm_rope_cache_status() == 0
    for c, r in zip(cases, runs):
        r.err.zero_()
        r.run()
        torch.cuda.synchronize()
        check_kv(c, r, name)


@pytest.mark.parametrize("layout", [native.RA_LAYOUT_BSD, native.RA_LAYOUT_NBSD], ids=["bsd", "nbsd"])
def test_norm_passes_of_many_and_of_few_heads(layout):
    cases = [synth.make_qkv(f"threads_{n}", 50 + n, S=64, H=256, num_heads=n, num_kv_heads=n, head_dim=64) for n in (12, 2)]
    runs = [runner.QkvRun(c, layout=layout) for c in cases]
    beside_one_another([r.run for r in runs], 4000)
    for c, r in zip(cases, runs):
        assert r.status() == 0
        out = r.out if layout == native.RA_LAYOUT_BSD else r.out.permute(1, 0, 2).reshape(c.T, c.I)
        check_qkv(c, as_f64(out), qkv_reference(c), "threads")
