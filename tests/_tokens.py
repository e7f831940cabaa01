"""Error bounds of the rotary-position and cache-row tests, from the kernels' arithmetic.

A rounding is off by at most half a step of its type.  cos and sin come from the angle's
exact fraction of a turn, rounded once to 32 bits at most pi / 4 from a quarter turn (2^-24
of that) and a function good to two units in the last place (2^-23 of at most 1), times the
amplitude (2^-24); the two products and their sum are rounded three times at most.  In
all, less than 8 * 2^-24 amplitude (|a| + |b|), and then once to the output's type.
"""
import numpy as np
import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def rounded(want, error, dtype):
    """Bound of a value `want`, off by `error` before it was rounded to dtype."""
    return error + HALF_STEP[dtype] * (np.abs(want) + error) + TINY[dtype]


def pair_sums(x, rot_offset, pairs, interleaved):
    """|a| + |b| of the pair that each column belongs to (0 for copied columns)."""
    s = np.zeros_like(x)
    for i in range(pairs):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        v = np.abs(x[..., rot_offset + ia]) + np.abs(x[..., rot_offset + ib])
        s[..., rot_offset + ia] = s[..., rot_offset + ib] = v
    return s


def rope_bound(want, x, dtype, pairs, *, rot_offset=0, interleaved=False, amplitude=1.0):
    sums = pair_sums(x, rot_offset, pairs, interleaved)
    err = 8 * 2.0 ** -24 * abs(amplitude) * sums
    return np.where(sums == 0, 0.0, rounded(want, err, dtype))


def row_bound(want, kv, pairs, *, norm, interleaved=False, amplitude=1.0):
    """Rows of the cache (bf16).  A latent value is divided by the root of a mean: the sum
    of 512 squares has at most 22 roundings in a row (16 terms, 5 levels over the warp, the
    square itself), of which the root leaves half; the scaling of the mean, eps, the root (two
    units) and two products add 8 half-steps at most: 20 * 2^-24 of the value."""
    bound = rope_bound(want, kv, torch.bfloat16, pairs, rot_offset=512, interleaved=interleaved,
                       amplitude=amplitude)
    err = 20 * 2.0 ** -24 * np.abs(want[:, :512]) if norm else 0.0 * want[:, :512]
    bound[:, :512] = rounded(want[:, :512], err, torch.bfloat16)
    return bound
