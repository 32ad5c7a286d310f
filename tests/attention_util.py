"""Cases and rounding bounds shared by the attention tests.

Bounds, per output element, for a value y = sum_j w_j v_j computed from rounded weights:
  |got - y| <= u_out |y| + (u_p + 2 e + 2^-17) * spread + under,
  u       half a step of the type, eps / 2 (bf16 2^-8, fp16 2^-11);
  spread  sum_j w_j |v_j| (times the value's quantisation, see below);
  u_p     the rounding of the probabilities to the tensor core's type;
  e       the error of a score: the accumulation of Dk products in fp32, at most
          Dk * 2^-24 * reach (reach = scale * sum_c |q_c k_c|), and for quantised keys the
          rounding of q / scale to fp16, 2^-11 * reach (a mixed key's 16-bit part keeps its
          own type, half a step of which the power-of-two row scale leaves exact).
          An error e of every score changes a weight by a factor within exp(+-2 e);
  2^-17   exp2's error (2 ulp), the fp32 products before it (|t| 2^-24, |t| < 2^6 where a
          weight counts) and the sums over up to 2^6 tiles;
  under   fp16 probabilities below the normal range: at most 2^-25 each against a sum >= 1.
For a quantised V the weighted sum is of codes and the offset comes off afterwards, so
spread is that of the codes, over the scale.
The lse is off by at most e + 2^-17 (1 + |lse|).
"""
from __future__ import annotations

import numpy as np
import torch

import oracle
from rope_attention_gb300 import synth

HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_values(seed, k, shape, dtype, std=1.0):
    """(bit patterns, float64 values) of N(0, std) rounded to bf16 or fp16."""
    x = synth.stream(seed, k).standard_normal(shape, dtype=np.float32) * np.float32(std)
    bits = {"bf16": synth.encode_bf16, "fp16": synth.encode_fp16}[dtype](x)
    return bits, {"bf16": oracle.decode_bf16, "fp16": oracle.codes.decode_fp16}[dtype](bits)


def check_attention(got, lse, ref, what, *, dtype, Dk, p_type=None, q_step=0.0, v_scale=None, v_offset=None, keys=1):
    """got [T, heads, Dv] and lse [T, heads] against an oracle result; rows that the oracle
    leaves NaN (outside every sequence) are not looked at.  Returns the largest error over
    its bound."""
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    real = ~np.isnan(ref["out"][:, :, 0])
    y, spread = ref["out"][real], ref["spread"][real]
    if v_scale is not None:          # |code| <= |x s| + |o|: the spread of the codes over s
        o = 0.0 if v_offset is None else np.abs(v_offset)
        spread = spread + np.broadcast_to(o / np.abs(v_scale), ref["out"].shape)[real]
    u_p = HALF_STEP[p_type or dtype]
    e = (Dk * 2.0 ** -24 + q_step) * ref["reach"][real][:, None]
    under = keys * 2.0 ** -25 * spread if (p_type or dtype) == "fp16" else 0.0
    tol = HALF_STEP[dtype] * np.abs(y) + (u_p + 2 * e + 2.0 ** -17) * spread + under + 2.0 ** -24
    err = np.abs(got[real] - y)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside; worst "
                           f"{np.nanmax(err / tol)} at {np.argwhere(bad)[0]}, got {got[real][bad][:4]} want {y[bad][:4]}")
    seen = np.isfinite(ref["lse"]) & real
    l_tol = e[np.isfinite(ref["lse"][real])][:, 0] + 2.0 ** -17 * (1 + np.abs(ref["lse"][seen]))
    assert np.all(np.abs(lse[seen] - ref["lse"][seen]) <= l_tol), \
        (what, "lse", np.max(np.abs(lse[seen] - ref["lse"][seen]) / l_tol))
    assert np.all(lse[real & ~seen] == -np.inf), (what, "lse of rows that see nothing")
    return float((err / tol).max()) if err.size else 0.0
