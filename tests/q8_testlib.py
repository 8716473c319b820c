"""Shared pieces of the tests of the paged 8-bit cache."""

import numpy as np
import torch

from oracle import paged_q8 as ref

TORCH_CODE = {ref.INT8: torch.int8, ref.E4M3: torch.float8_e4m3fn}


def np_codes(t, code):
    """Codes of a store tensor as the oracle takes them."""
    t = t.detach().cpu()
    return t.numpy().copy() if code == ref.INT8 else t.view(torch.uint8).numpy().copy()


def to_store(codes, code, device="cuda"):
    t = torch.from_numpy(codes.copy())
    return (t if code == ref.INT8 else t.view(torch.float8_e4m3fn)).to(device)


def random_store(rng, pages, heads, code, spread=1.0):
    """Codes of every value and scales over a few powers of two."""
    shape = (pages, heads, ref.PAGE, 128)
    if code == ref.INT8:
        c = rng.integers(-127, 128, shape).astype(np.int8)
    else:
        c = rng.integers(0, 127, shape).astype(np.uint8) | (rng.integers(0, 2, shape).astype(np.uint8) << 7)
        c = np.where((c & 127) > 0x70, c & 0xef, c)      # most values below 128
        c = c.astype(np.uint8)
    s = 2.0 ** rng.integers(-3, 2, (pages, heads)) / (64.0 if code == ref.INT8 else 64.0) * spread
    if code == ref.INT8:
        s = s * rng.uniform(0.6, 1.0, s.shape)
    return c, s.astype(np.float32)


def scattered_table(rng, lens, width, pages):
    """A page table over distinct, scattered pages; unused entries -1."""
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // ref.PAGE)
        table[b, :k] = order[at:at + k]
        at += k
    return table


def rows_of(codes, scale, table_row, length, code):
    """[length, heads, 128] float64 values of one request."""
    k = -(-length // ref.PAGE)
    pg = table_row[:k]
    x = ref.decode(codes[pg], code) * scale[pg].astype(np.float64)[..., None, None]
    return x.transpose(0, 2, 1, 3).reshape(k * ref.PAGE, codes.shape[1], 128)[:length]


def step_floor(codes, scale, table_row, length, code, heads, dtype):
    """What fp16's smallest steps may cost a row's output, [heads, 128].

    A weight w_j is taken relative to M, the largest of score + log2 s_v so far
    (or at most 2^15 times it): the largest one is at least 1 for the prompt
    kernel, 2^14 for the other.  fp16 holds it to 2^-25 at worst, so the
    numerator sum w_j c_j is off by at most 2^-25 sum |c_j|, and the denominator
    sum w_j / s_j is at least 1 / max s (the largest weight's own term): an
    error of at most 2^-25 sum |c_j| max s, 2^-39 of it where weights start at
    2^14 (fp32 queries run on that kernel alone)."""
    k = -(-length // ref.PAGE)
    pg = table_row[:k]
    c = np.abs(ref.decode(codes[pg], code)).transpose(1, 0, 2, 3).reshape(codes.shape[1], -1, 128)[:, :length].sum(1)
    f = c * scale[pg].max(0).astype(np.float64)[:, None] * 2.0 ** (-25 if dtype == torch.bfloat16 else -39)
    return np.repeat(f, heads // codes.shape[1], 0)


def bound(out, mass, size, dtype, cap=0.0, bias=0.0):
    """Elementwise bound on the error of the kernels' attention.

    The output's own rounding is half a step: 2^-8 of it in bf16, 2^-24 in
    fp32.  Weights: fp16, 2^-11 each for bf16 queries, two fp16 parts (2^-22)
    for fp32, on the mass sum p |v|.  A score of 128 products summed in fp32 is
    off by at most 128 * 2^-24 * size = 2^-17 size (fp32 queries' two parts add
    2^-22 size), scaling and the steps behind it a few 2^-24 of |x| <= size
    each; log2 of the value scale and the exponentials 2^-20 together; the cap
    has a derivative of at most 1 and adds 2^-20 cap.  A score error d moves
    every weight by a factor e^(+-2d) at most, numerator and denominator."""
    bf16 = dtype == torch.bfloat16
    d = 2.0 ** -16 * size + 2.0 ** -20 * (1.0 + cap) + 2.0 ** -22 * bias
    rel = (2.0 ** -11 if bf16 else 2.0 ** -21) * 2 + 3.0 * d
    return (2.0 ** -8 if bf16 else 2.0 ** -23) * np.abs(out) + rel * mass + 1e-30
