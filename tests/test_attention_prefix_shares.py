"""paged_prefix_attention where a row's two results have large log-sum-exps a little apart: the shares that
they are joined with.

Scores are exact, A B + d with powers of two A and B and a small whole d, so that only what happens after the
products can be off.  All keys of a side have one score and one value (1 of the own positions, -1 of the
prefix's): a row is (a - b) / (a + b) with a = n e^4 for n own positions and b = p for p of the prefix.

Tolerance.  Within a side nothing depends on the score's size: every weight is one number w in [2^-1/64, 2^1/64]
times a power of two (the rounding of score * log2(e), half a step of 2^-6 at 2^18), the weighted sum has it
rounded to half a step u of the type, and the sum of weights goes with the maximum to the join.  So each
side's row is off by u, the output's rounding adds u, the exponentials and fp32 sums less than 2^-17 as
in attention_util: |got - y| <= u |y| + u + 2^-17.  For u = 2^-11 (fp16) that is 1e-3, where log2 of a side's
sum of weights, held as one fp32 number of size 2^17.5, would be off by up to 2^-7 on each side and
the row by up to 2^-7 ln 2 = 5e-3."""
import numpy as np
import pytest
import torch

from rope_attention_gb300 import native

pytestmark = pytest.mark.gpu

A, B = 256.0, 512.0
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("kw", [
    dict(variant=2, lens=[1 + (7 * i) % 40 for i in range(96)], heads=16, N=8, prefix=1100),            # few rows, then tiles
    dict(variant=2, lens=[1 + i for i in range(2)], heads=8, N=8, prefix=40000),                        # few rows, cut into many parts
    dict(variant=2, lens=[1 + (7 * i) % 40 for i in range(96)], heads=16, N=8, prefix=1100, Dkv=256, Dv=208),
    dict(variant=1, lens=[1 + (5 * i) % 30 for i in range(150)], heads=16, N=1, prefix=4000, Dkv=576, Dv=512),
], ids=["v2", "v2_long", "v2_wide", "v1"])
def test_shares_of_large_scores(kw, dtype):
    kw = {"Dkv": 192, "Dv": 128, **kw}
    variant, lens, heads, N, prefix, Dkv, Dv = (kw[x] for x in ("variant", "lens", "heads", "N", "prefix", "Dkv", "Dv"))
    n, bs, R = len(lens), 32, 64
    ahead, pages = -(-prefix // bs), -(-max(lens) // bs)
    blocks = ahead + n * pages
    k_width = R if variant == 1 else Dkv
    k = torch.zeros(blocks, N, bs, k_width, dtype=dtype, device="cuda")
    v = torch.empty(blocks, N, bs, Dv, dtype=dtype, device="cuda")
    k[..., 0], v[:ahead], v[ahead:] = B, -1.0, 1.0
    k[ahead:, ..., 1] = 4.0
    q = torch.zeros(n, heads, Dkv, dtype=dtype, device="cuda")
    at = Dv if variant == 1 else 0              # V1: the key is the value's channels, then the k cache's
    q[..., at], q[..., at + 1] = A, 1.0
    half = native.RA_FP16 if dtype == torch.float16 else native.RA_BF16
    cache = native.KvRmsNormRopeCacheParams(B=n, N=N, S=1, Dkv=Dkv, Dv=Dv, rope_size=R, variant=variant,
                                            cache_mode=native.RA_CACHE_PA_BNSD, block_num=blocks, block_size=bs, kv_dtype=half,
                                            k_cache_dtype=half, ckv_cache_dtype=half, epsilon=1e-5)
    params = native.PagedAttentionParams(B=n, total_q=n, num_heads=heads, causal=1, softmax_scale=1.0, max_seq_len=max(lens),
                                         block_table_stride=pages)
    form = native.AttentionPrefix(max_prefix_len=prefix, table_entries=ahead)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out, lse = torch.full((n, heads, Dv), 7.0, dtype=dtype, device="cuda"), torch.full((n, heads), 7.0, device="cuda")
    ws = torch.zeros(native.paged_prefix_attention_workspace_bytes(cache, params, form), dtype=torch.uint8, device="cuda")
    native.paged_prefix_attention(cache, params, form, q, k, v, i32([prefix]), i32(range(ahead)), i32(lens),
                                  i32(range(ahead, blocks)).view(n, pages), out, ws, lse=lse)
    torch.cuda.synchronize()
    assert native.attention_status(ws) == 0
    a, b = np.array(lens) * np.exp(4.0), float(prefix)
    y = ((a - b) / (a + b))[:, None, None]
    err = np.abs(out.double().cpu().numpy() - y)
    tol = U[dtype] * np.abs(y) + U[dtype] + 2.0 ** -17
    assert (err <= tol).all(), (np.max(err / tol), np.max(err))
    want = A * B + np.log(a + b)[:, None]
    assert (np.abs(lse.double().cpu().numpy() - want) <= 2.0 ** -17 * want).all()
