"""Paged cases with a window or a shared prefix against the oracle, and their rounding bound.

The bound is attention_util's, and for a shared prefix the joining of a row's two results: log2 of
each sum of exponentials L is off by at most (|L| + 1) 2^-23 (two roundings), which moves the
shares that the results are weighed with, so the row by at most
2 ln 2 (|L| + 1) 2^-23 * spread < 2^-21 (1 + |lse|) * spread; the division and the two products add
less than 2^-21 * spread."""
import numpy as np
import torch

import oracle
from attention_util import HALF_STEP, TORCH, half_values
from rope_attention_gb300 import native, synth
from test_attention_paged import CODE, device, stored


def check_rows(got, lse, ref, what, *, dtype, Dk, p_type=None, q_step=0.0, v_scale=None, v_offset=None, keys=1, joined=False):
    """attention_util.check_attention's comparison, with the term for joined rows."""
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    real = ~np.isnan(ref["out"][:, :, 0])
    y, spread, want = ref["out"][real], ref["spread"][real], ref["lse"][real]
    if v_scale is not None:
        o = 0.0 if v_offset is None else np.abs(v_offset)
        spread = spread + np.broadcast_to(o / np.abs(v_scale), ref["out"].shape)[real]
    e = (Dk * 2.0 ** -24 + q_step) * ref["reach"][real][:, None]
    rel = HALF_STEP[p_type or dtype] + 2 * e + 2.0 ** -17
    if joined:
        rel = rel + 2.0 ** -21 * (2 + np.where(np.isfinite(want), np.abs(want), 0.0))[:, None]
    under = keys * 2.0 ** -25 * spread if (p_type or dtype) == "fp16" else 0.0
    tol = HALF_STEP[dtype] * np.abs(y) + rel * spread + under + 2.0 ** -24
    err = np.abs(got[real] - y)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside; worst {np.nanmax(err / tol)} at "
                           f"{np.argwhere(bad)[0]}, got {got[real][bad][:4]} want {y[bad][:4]}")
    seen = np.isfinite(want)
    l_tol = e[seen][:, 0] + 2.0 ** -17 * (1 + np.abs(want[seen]))
    assert np.all(np.abs(lse[real][seen] - want[seen]) <= l_tol), (what, "lse", np.max(np.abs(lse[real][seen] - want[seen]) / l_tol))
    assert np.all(lse[real][~seen] == -np.inf), (what, "lse of rows that see nothing")


def visible(lq, n, window, sinks):
    """Positions that some of the last lq of n positions sees in a window."""
    lo = max(0, n - lq - window + 1)
    seen = np.zeros(n, bool)
    seen[:min(n, sinks)] = True
    seen[lo:] = True
    return seen


class Case:
    """Sequences of lens own positions, the last news of them attending; every slot that no query
    may look at holds NaN (an odd code), and pages of a window that none sees have no entry."""

    def __init__(self, seed, *, variant, lens, news, heads, N=1, Dkv=192, Dv=128, R=64, mode="PA_BNSD", bs=32, kt="bf16",
                 vt="bf16", dtype="bf16", causal=True, scalar=False, offsets=True, tail=0, bad_pages=(), bad_prefix=(), std=1.0,
                 given_starts=True, window=None, sinks=0, prefix=None, spare=0):
        B = len(lens)
        self.kw, self.vw = kw, vw = (R, Dv) if variant == 1 else (Dkv, Dv)
        pages = [-(-n // bs) for n in lens]
        ahead = -(-(prefix or 0) // bs)
        n_pages = sum(pages) + ahead + 2
        if mode == "Norm":
            cap = max(max(lens), 1) + 5
            shape = (B, N, cap)
        else:
            shape = (n_pages, bs, N) if mode == "PA" else (n_pages, N, bs)
        ps = lambda w: ((1,) if scalar else (w,)) if variant == 1 else (N, w)
        kc, ks, ko = stored(seed, 10, shape + (kw,), kt, ps(kw), offsets)
        vc, vs, vo = stored(seed, 20, shape + (vw,), vt, ps(vw), offsets)
        used = np.zeros(shape[:2] if mode == "PA" else (shape[0], shape[2]), bool)
        table = first = None
        if mode == "Norm":
            for b, n in enumerate(lens):
                used[b, :n] = True
        else:
            ids = synth.stream(seed, 1).permutation(n_pages)
            table = np.full((B, max(max(pages), 1) + 1), 1 << 30, np.int32)
            at = 0
            for b, n in enumerate(lens):
                table[b, :pages[b]] = ids[at:at + pages[b]]
                at += pages[b]
                seen = np.ones(n, bool) if window is None else visible(news[b], n, window, sinks)
                for i in range(pages[b]):
                    if seen[i * bs:(i + 1) * bs].any():
                        used[table[b, i], :min(bs, n - i * bs)] = True
                    else:
                        table[b, i] = -5          # the page went to another sequence
            if prefix is not None:
                first = np.full(max(ahead, 1) + spare, 1 << 30, np.int32)
                first[:ahead] = ids[at:at + ahead]
                for j in range(prefix):
                    used[first[j // bs], j % bs] = True
                for i, value in bad_prefix:
                    first[i] = value
            for b, i, value in bad_pages:
                table[b, i] = value
        for c, kind in ((kc, kt), (vc, vt)):
            fill = {"int8": -77, "e4m3": 0x7F, "e5m2": 0x7F}.get(kind, 0x7FBF)
            if mode == "PA":
                c[~used] = fill
            else:
                np.moveaxis(c, 1, 2)[~used] = fill
        self.starts = starts = [0] + list(np.cumsum(news))
        qb, self.qv = half_values(seed, 0, (starts[-1] + tail, heads, Dkv), dtype, std)
        self.q = torch.from_numpy(qb.view(np.int16)).cuda().view(TORCH[dtype])
        self.out = torch.full((starts[-1] + tail, heads, vw), 7.0, dtype=TORCH[dtype], device="cuda")
        self.lse = torch.full((starts[-1] + tail, heads), 7.0, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cache = native.KvRmsNormRopeCacheParams(
            B=B, N=N, S=1, Dkv=Dkv, Dv=Dv, rope_size=R, variant=variant, cache_mode=synth.CACHE_MODES[mode],
            block_num=0 if mode == "Norm" else n_pages, block_size=0 if mode == "Norm" else bs, kv_dtype=CODE[dtype],
            k_cache_dtype=CODE[kt], ckv_cache_dtype=CODE[vt], epsilon=1e-5, cache_seq_len=cap if mode == "Norm" else 0,
            k_quant_scalar=1 if scalar and ks is not None else 0, c_kv_quant_scalar=1 if scalar and vs is not None else 0)
        self.scale = Dkv ** -0.5
        self.params = native.PagedAttentionParams(B=B, total_q=starts[-1] + tail, num_heads=heads, causal=1 if causal else 0,
                                                  softmax_scale=self.scale, max_seq_len=max(lens),
                                                  block_table_stride=0 if table is None else table.shape[1])
        dev = lambda x: None if x is None else torch.from_numpy(np.asarray(x)).cuda()
        self.args = dict(block_table=dev(table), k_rope_scale=dev(ks), c_kv_scale=dev(vs), k_rope_offset=dev(ko), c_kv_offset=dev(vo),
                         cu_seqlens_q=torch.tensor(starts, dtype=torch.int32, device="cuda") if given_starts else None)
        self.lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.kd, self.vd = device(kc, kt), device(vc, vt)
        if prefix is None:
            self.form = native.AttentionWindow(window=window, sinks=sinks)
            self.ws = torch.zeros(native.paged_attention_workspace_bytes(self.cache, self.params), dtype=torch.uint8, device="cuda")
        else:
            self.form = native.AttentionPrefix(max_prefix_len=prefix + spare, table_entries=len(first))
            self.prefix_len = torch.tensor([prefix], dtype=torch.int32, device="cuda")
            self.first = dev(first)
            self.ws = torch.zeros(native.paged_prefix_attention_workspace_bytes(self.cache, self.params, self.form),
                                  dtype=torch.uint8, device="cuda")
        self.lens, self.news, self.prefix, self.window, self.sinks = lens, news, prefix, window, sinks
        self.dtype, self.kt, self.vt, self.Dkv, self.heads, self.N, self.tail = dtype, kt, vt, Dkv, heads, N, tail
        self.bad = bool(bad_pages) or bool(bad_prefix)
        self.ref_args = dict(variant=variant, seq_lens=lens, starts_q=starts, scale=self.scale, causal=causal, cache_mode=mode,
                             block_size=bs, table=table, k_type=kt if ks is not None else dtype,
                             v_type=vt if vs is not None else dtype, k_scale=ks, k_offset=ko, v_scale=vs, v_offset=vo,
                             window=window, sinks=sinks, prefix_len=prefix or 0, prefix_table=first)
        self.quant_k = ks is not None or (variant == 1 and vs is not None)
        self.host = (kc, vc, vs, vo)

    def run(self, stream=None, out=None, lse="own"):
        out, lse = self.out if out is None else out, self.lse if lse == "own" else lse
        if self.prefix is None:
            native.paged_window_attention(self.cache, self.params, self.form, self.q, self.kd, self.vd, self.lens_d, out, self.ws,
                                          lse=lse, dev_error_count=self.err, stream=stream, **self.args)
        else:
            args = dict(self.args)
            native.paged_prefix_attention(self.cache, self.params, self.form, self.q, self.kd, self.vd, self.prefix_len, self.first,
                                          self.lens_d, args.pop("block_table"), out, self.ws, lse=lse, dev_error_count=self.err,
                                          stream=stream, **args)

    def status(self):
        return native.attention_status(self.ws)

    def check(self, what=""):
        kc, vc, vs, vo = self.host
        ref = oracle.attention.paged_attention(self.qv, kc, vc, **self.ref_args)
        g = self.heads // self.N
        per_head = lambda x: None if x is None else np.repeat(x, g, axis=0) if x.ndim == 2 else x
        check_rows(self.out, self.lse, ref, f"{what} {self.kt} {self.vt} {self.lens} {self.news} {self.window} {self.sinks} {self.prefix}",
                   dtype=self.dtype, Dk=self.Dkv, p_type="fp16" if vs is not None else self.dtype,
                   q_step=2.0 ** -11 if self.quant_k else 0.0, v_scale=per_head(vs), v_offset=per_head(vo),
                   keys=max(self.lens + [1]) + (self.prefix or 0), joined=self.prefix is not None)

    def run_and_check(self):
        self.run()
        torch.cuda.synchronize()
        assert self.status() == 0
        self.check()
        assert (int(self.err) > 0) == self.bad
        if self.tail and self.args["cu_seqlens_q"] is not None:
            assert (self.out[self.starts[-1]:] == 7).all() and (self.lse[self.starts[-1]:] == 7).all()
        # the same call again, on a workspace that holds the first one's partial results
        again = torch.full_like(self.out, 7.0)
        self.run(out=again, lse=None)
        assert torch.equal(again.view(torch.int16), self.out.view(torch.int16))
