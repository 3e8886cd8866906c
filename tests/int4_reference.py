"""Rotary positions and the 4-bit cache format from their definitions, on the CPU in
binary64 (angles in whole fractions of a turn), apart from the library's own code."""
import math
from fractions import Fraction

import torch

GROUP, TOP_SCALE = 32, 9344.0
# dim j of eight stands in nibble ORDER[j] of their 32-bit word
ORDER = [0, 4, 1, 5, 2, 6, 3, 7]
TWO_PI = Fraction("6.283185307179586476925286766559005768394338798750211641949889184615632812572417997256069650684234136")


def frequencies(r, base=10000.0, scaling=None, factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """(radians per position of every pair, amplitude)."""
    if scaling == "ntk" and r > 2:
        base = base * factor ** (r / (r - 2))
    f = [base ** (-2 * i / r) for i in range(r // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "yarn":
        keep = [min(max((original_len * x / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow), 0.0), 1.0) for x in f]
        f = [x * k + x / factor * (1 - k) for x, k in zip(f, keep)]
        return f, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def angles(positions, freq):
    """binary64 [N, pairs] in (-pi, pi], from exact products."""
    turns = [Fraction(f) / TWO_PI for f in freq]
    rows = []
    for p in positions.tolist():
        row = []
        for t in turns:
            x = p * t
            row.append(float((x - round(x)) * TWO_PI))
        rows.append(row)
    return torch.tensor(rows, dtype=torch.float64).reshape(len(rows), len(turns))


def rotate(x, positions, freq, amplitude, interleaved):
    """(rotated x [N, H, d] in binary64, |x_a| + |x_b| of every element's pair (0: not rotated))."""
    x = x.cpu().double()
    half = len(freq)
    r = 2 * half
    t = angles(positions.cpu(), freq)[:, None]
    cos, sin = amplitude * torch.cos(t), amplitude * torch.sin(t)
    first = torch.arange(0, r, 2) if interleaved else torch.arange(half)
    second = first + 1 if interleaved else first + half
    a, b = x[..., first], x[..., second]
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    mag[..., first] = mag[..., second] = (a.abs() + b.abs()) * abs(amplitude)
    return y, mag


def scales(x):
    """float16 scales of binary64 x [..., d]."""
    g = x.unflatten(-1, (-1, GROUP)).abs()
    top = torch.where(torch.isnan(g), 0.0, g).amax(-1) / 7
    m, e = torch.frexp(torch.where(torch.isinf(top), 0.0, top))
    s = torch.ldexp(torch.round(m * 256), e - 8)  # 8 significant bits: bf16
    s = torch.where(torch.isinf(top), TOP_SCALE, s).clamp(max=TOP_SCALE)
    # to float16: multiples of 2^-24 below its normal range, ties to even
    return torch.where(s < 2.0 ** -14, torch.round(s * 2 ** 24) / 2 ** 24, s).to(torch.float16)


def codes(x, s):
    """Integers in +-7 of binary64 x [..., d] under float16 scales [..., d / 32]."""
    s = s.double()[..., None].expand(*s.shape, GROUP).flatten(-2)
    c = torch.round(x / torch.where(s > 0, s, 1.0)).clamp(-7, 7)
    return torch.where((s > 0) & ~torch.isnan(x), c, 0.0)


def pack(c):
    """Codes [..., d] -> bytes [..., d / 2]."""
    u = (c + 8).to(torch.int64).unflatten(-1, (-1, 8))
    word = sum(u[..., j] << (4 * ORDER[j]) for j in range(8))
    return torch.stack([word >> (8 * k) & 255 for k in range(4)], -1).flatten(-2).to(torch.uint8)


def values(cache, scale):
    """binary64 [..., d] of bytes [..., d / 2] and scales [..., d / 32]."""
    b = cache.cpu().long().unflatten(-1, (-1, 4))
    word = b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16 | b[..., 3] << 24
    u = torch.stack([word >> (4 * ORDER[j]) & 15 for j in range(8)], -1).flatten(-2)
    return (u - 8).double() * scale.cpu().double().repeat_interleave(GROUP, -1)


def token_major(cache, scale):
    """The values as [num_blocks, block_size, Hkv, d]."""
    return values(cache, scale).transpose(1, 2)


def empty_cache(nb, H, bs, d, seed=0, device="cpu"):
    """Caches with arbitrary content: (k_cache, v_cache, k_scale, v_scale)."""
    g = torch.Generator().manual_seed(seed)
    cs = [torch.randint(0, 256, (nb, H, bs, d // 2), generator=g, dtype=torch.uint8) for _ in range(2)]
    ss = [(torch.randint(1, 256, (nb, H, bs, d // 32), generator=g) / 64).to(torch.float16) for _ in range(2)]
    return tuple(t.to(device) for t in cs + ss)


def stored(caches, key, value, slots):
    """The caches after key / value (binary64 [N, H, d]) went to `slots`."""
    out = [c.cpu().clone() for c in caches]
    bs = out[0].shape[2]
    n = out[0].shape[0] * bs
    for x, c, s in ((key, out[0], out[2]), (value, out[1], out[3])):
        for i, slot in enumerate(slots.tolist()):
            if 0 <= slot < n:
                sc = scales(x[i])
                c[slot // bs, :, slot % bs] = pack(codes(x[i], sc))
                s[slot // bs, :, slot % bs] = sc
    return out
