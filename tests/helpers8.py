"""Plain forms of the 8-bit linear layers' operators, on the host: quantised
blocks as fp32 arithmetic defines them (bit for bit), everything else in 64 bits."""
from __future__ import annotations

import torch

BLOCK = 128
LARGEST = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24,
             torch.float8_e4m3fn: 2.0 ** -4, torch.float8_e5m2: 2.0 ** -3}
# half the distance of the values below the smallest normal number
SMALL_STEP = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0,
              torch.float8_e4m3fn: 2.0 ** -10, torch.float8_e5m2: 2.0 ** -17}
U = 2.0 ** -24  # half a step of fp32


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def expand(scale, n: int, d: int, squares: bool):
    """Scales as one value per element of [n][d]."""
    s = scale.repeat_interleave(BLOCK, 1)[:, :d]
    return s.repeat_interleave(BLOCK, 0)[:n] if squares else s


def block_amax(x, squares: bool):
    """Largest magnitudes of the blocks of x [n][d] (not finite: NaN)."""
    n, d = x.shape
    rows = BLOCK if squares else 1
    x = torch.nn.functional.pad(x, (0, blocks(d) * BLOCK - d, 0, -(-n // rows) * rows - n))
    a = x.view(-1, rows, blocks(d), BLOCK).abs().amax((1, 3))  # amax hands NaN on
    return torch.where(torch.isfinite(a), a, torch.full_like(a, float("nan")))


def quantise(x, squares: bool, dtype):
    """(q, scale) of x [n][d] on the host: every operation in fp32."""
    x = x.float()
    n, d = x.shape
    scale = torch.maximum(block_amax(x, squares) / LARGEST[dtype], torch.tensor(2.0 ** -126))
    inv = 1.0 / scale
    return (x * expand(inv, n, d, squares)).to(dtype), scale


def dequantise(q, scale, squares: bool):
    """What a quantised matrix stands for, in 64 bits."""
    q = q.cpu()
    return q.double() * expand(scale.cpu().double(), *q.shape, squares)


def same_bytes(a, b) -> bool:
    """Equal 8-bit values, any NaN equal to any NaN, the zeros' signs apart."""
    a, b = a.cpu().float(), b.cpu().float()
    return bool(torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)))


def strided(t, pad: int):
    """The same values on the GPU in rows of the width + pad elements, NaN between them."""
    n, d = t.shape
    base = torch.full((n, d + pad), float("nan"), device="cuda").to(t.dtype)
    out = base[:, :d]
    out.copy_(t)
    return out


def normal(shape, seed: int, dtype=torch.float32, std: float = 1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)
