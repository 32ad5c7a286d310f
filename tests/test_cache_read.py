"""kv_cache_read on the GPU: rows written by kv_rms_norm_rope_cache read back, bit for bit for
16-bit caches, and within the rounding of one fp32 quotient and one 16-bit rounding for
quantised ones; skipped and illegal slots give zeros and are counted."""
import numpy as np
import pytest
import torch

import oracle
from attention_util import HALF_STEP, TORCH
from rope_attention_gb300 import native, runner, synth

pytestmark = pytest.mark.gpu

CASES = {
    "v1_int8": dict(variant=1, B=3, N=1, S=37, Dkv=576, Dv=512, block_size=32, block_num=6, quant_k=True, quant_v=True),
    "v1_scalar": dict(variant=1, B=2, N=1, S=20, Dkv=576, Dv=512, block_size=32, block_num=2, quant_k=True, quant_v=True,
                      k_scalar=True, v_scalar=True),
    "v1_bf16_norm": dict(variant=1, B=2, N=1, S=21, Dkv=136, Dv=128, rope_size=8, cache_mode="Norm", cache_seq=40),
    "v1_mixed": dict(variant=1, B=2, N=1, S=33, Dkv=576, Dv=512, block_size=32, block_num=3, quant_v=True),
    "v2_int8": dict(variant=2, B=2, N=8, S=21, Dkv=192, Dv=128, block_size=32, block_num=2, quant_k=True, quant_v=True),
    "v2_fp8_pa": dict(variant=2, B=2, N=4, S=50, Dkv=72, Dv=40, rope_size=8, block_size=32, block_num=4, cache_mode="PA",
                      quant_k=True, quant_v=True, k_qtype="e4m3", v_qtype="e5m2"),
    "v2_blk": dict(variant=2, B=3, N=2, S=50, Dkv=192, Dv=128, block_size=32, cache_mode="PA_BLK_BNSD", quant_k=True,
                   k_qtype="e5m2", offsets=False),
    "v2_fp16_norm": dict(variant=2, B=2, N=2, S=19, Dkv=192, Dv=128, cache_mode="Norm", cache_seq=24, dtype="fp16",
                         quant_k=True, quant_v=True),
    "v2_one_token": dict(variant=2, B=1, N=1, S=1, Dkv=64, Dv=8, rope_size=8, block_size=16, block_num=1),
}


def read(run, index=None, k=True, v=True):
    c = run.case
    dt = TORCH[c.dtype]
    ko = torch.full((c.B, c.N, c.S, c.k_width), 7.0, dtype=dt, device="cuda") if k else None
    vo = torch.full((c.B, c.N, c.S, c.ckv_width), 7.0, dtype=dt, device="cuda") if v else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.kv_cache_read(run.params, run.index if index is None else index, run.k_cache, run.ckv_cache, ko, vo,
                         run.k_scale, run.v_scale, run.k_offset, run.v_offset, err)
    torch.cuda.synchronize()
    return ko, vo, int(err)


def check(run, index, ko, vo, err):
    c = run.case
    for got, cache, scale, offset, q in ((ko, run.k_cache, c.k_scale, c.k_offset, c.k_qtype),
                                         (vo, run.ckv_cache, c.v_scale, c.v_offset, c.v_qtype)):
        if got is None:
            continue
        host = cache.view(torch.int16).cpu().numpy().view(np.uint16) if cache.dtype in TORCH.values() else cache.cpu().numpy()
        want, bad = oracle.attention.kv_cache_read(index, host, B=c.B, N=c.N, S=c.S, cache_mode=c.cache_mode,
                                                   block_size=c.block_size, stored=c.dtype if scale is None else q,
                                                   scale=scale, offset=offset)
        got = got.double().cpu().numpy()
        assert bad == err
        if scale is None:
            assert np.array_equal(got, want)
            continue
        # (code - o) in fp32: half a step of the difference, which |code| + |o| bounds; the
        # reciprocal and the product: a half step each; then the 16-bit rounding
        s = np.asarray(scale, np.float64)
        o = np.zeros_like(s) if offset is None else np.abs(offset)
        per = (lambda x: x[None, :, None, :]) if s.ndim == 2 else (lambda x: x)
        slack = 3 * 2.0 ** -24 * (np.abs(want) + per(o / np.abs(s))) + 2.0 ** -25
        assert np.all(np.abs(got - want) <= HALF_STEP[c.dtype] * (np.abs(want) + slack) + slack)


@pytest.mark.parametrize("name", CASES)
def test_reads_back_what_was_written(name):
    run = runner.KvRun(synth.make_kv("read_" + name, 11, **{"skip_frac": 0.1, **CASES[name]}))
    run.run()
    ko, vo, err = read(run)
    check(run, run.case.index, ko, vo, err)


def test_unquantised_rows_come_back_as_the_writer_output_them():
    run = runner.KvRun(synth.make_kv("read_same", 12, variant=2, B=2, N=4, S=40, Dkv=192, Dv=128, block_size=16, block_num=6))
    run.run()
    ko, vo, _ = read(run)
    assert torch.equal(ko, run.k_rope) and torch.equal(vo, run.c_kv)


@pytest.mark.parametrize("mode", ["PA", "PA_BNSD", "PA_BLK_BNSD", "Norm"])
def test_illegal_and_repeated_slots(mode):
    kw = dict(cache_seq=64) if mode == "Norm" else dict(block_size=32, block_num=6)
    run = runner.KvRun(synth.make_kv("read_bad", 13, variant=2, B=2, N=2, S=64, Dkv=64, Dv=64, rope_size=8, cache_mode=mode,
                                     quant_k=True, **kw))
    run.run()
    index = run.case.index.copy()
    flat = index.reshape(-1)
    last = 64 if mode == "Norm" else 6 * 32
    flat[0], flat[1], flat[2] = -1, last - 1, -5
    flat[3] = {"PA_BLK_BNSD": last - 7, "Norm": last}.get(mode, last)
    if flat.size > 8:
        flat[4], flat[5], flat[6] = flat[7], flat[7], 1 << 40
    ko, vo, err = read(run, torch.from_numpy(index).cuda())
    assert err > 0
    check(run, index, ko, vo, err)


def test_one_cache_alone():
    run = runner.KvRun(synth.make_kv("read_one", 14, variant=1, B=2, N=1, S=40, Dkv=576, Dv=512, block_size=32, block_num=3,
                                     quant_k=True, quant_v=True))
    run.run()
    ko, vo, err = read(run, k=False)
    assert ko is None
    check(run, run.case.index, ko, vo, err)
    ko, vo, err = read(run, v=False)
    assert vo is None
    check(run, run.case.index, ko, vo, err)
