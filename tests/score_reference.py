"""Attention with score rules in binary64, written from its definition, with the
largest error that the kernels' roundings can cause in each output element.

Tolerance.  Let w be a row's exact softmax weights and o = sum w v its output.
  * Scores: the kernels' f32 dot products over 128 terms err by at most
    128 x 2^-24 x sum |q k| scale, which stays below SCORE = 2^-11 for the inputs
    used (|q| up to about 4 x 3, |k| up to about 5: the sum is below 60); the scale,
    cap and bias add a few 2^-23 of values below 2^6, the exponential 2^-22.
    A score error e changes o by at most 2 e sum w |v|.
  * P is rounded to 16 bits, at most half a step u = eps / 2 of its type relative to
    itself, in the product and in the row sum: at most 2 u sum w |v|.
  * Below f16's normal range P is rounded to multiples of 2^-24, at most 2^-25 off.
    The row's largest P (with the V scale of an 8-bit cache in it) is at least 1: the
    reference is the maximum of the block that set it.  So 1 / sum p <= vs* for that
    key's scale vs* (1 in a 16-bit cache), and the error is at most 2^-25 vs* sum
    |code| <= 2^-25 x visible keys x V's largest magnitude.
  * The output is rounded once: u |o|.  f32 sums add 2^-24 x keys relative, below
    2^-12 for up to 4096 terms in a chain.
"""
import torch

SCORE = 2.0 ** -11


def cdiv(a, b):
    return -(-a // b)


def dequantize(cache, scale):
    """[num_blocks, bs, Hkv, d] in binary64."""
    if cache.dtype == torch.uint8:
        x = cache.cpu().view(torch.float8_e4m3fn).double()
    else:
        x = cache.cpu().double()
    return x if scale is None else x * scale.cpu().double()[:, None, :, None]


def attention(q, k, v, pos, lo, hi, scale, softcap=0.0, slopes=None):
    """One sequence.  q [n, Hq, d], k / v [T, Hkv, d] binary64, pos / lo / hi [n]
    -> (out [n, Hq, d], sum of w |v|, visible keys [n, 1, 1])."""
    n, Hq, _ = q.shape
    T, Hkv, _ = k.shape
    G = Hq // Hkv
    t = torch.arange(T)
    seen = (t >= lo[:, None]) & (t < hi[:, None])
    out, mag = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        live = seen.any(0)  # rows of keys nobody sees may hold anything
        kh = torch.where(live[:, None], kh, 0.0)
        vh = torch.where(live[:, None], vh, 0.0)
        s = scale * (q[:, h].double() @ kh.T)
        if softcap:
            s = softcap * torch.tanh(s / softcap)
        if slopes is not None:
            s = s - slopes[h].double() * (pos[:, None] - t).abs()
        s = s.masked_fill(~seen, float("-inf"))
        w = torch.softmax(s, -1).masked_fill(~seen.any(1, keepdim=True), 0.0)
        out[:, h] = w @ vh
        mag[:, h] = w @ vh.abs()
    return out, mag, seen.sum(1).double()[:, None, None]


def tolerance(ref, dtype, p_dtype, vmax):
    out, mag, keys = ref
    u, up = torch.finfo(dtype).eps / 2, torch.finfo(p_dtype).eps / 2
    small = 2.0 ** -25 * keys * vmax if p_dtype == torch.float16 else 0.0
    return (2 * SCORE + 2 * up + 2.0 ** -12) * mag + u * out.abs() + small + 1e-30


def rows_of(cache, table, total):
    bs = cache.shape[1]
    ids = table[:cdiv(total, bs)].long().cpu()
    return cache[ids].flatten(0, 1)[:total]


def prefill(q, kc, vc, tables, starts, ns, scale, softcap=0.0, slopes=None, key_starts=None, prefix=None):
    """kc / vc binary64 caches on the CPU; returns attention()'s of all rows."""
    parts, at = [], 0
    for b, (s, n) in enumerate(zip(starts, ns)):
        total = s + n
        pos = torch.arange(s, total)
        lo = torch.zeros(n, dtype=torch.long) if key_starts is None else key_starts[at:at + n].cpu().long()
        hi = pos + 1 if prefix is None else torch.clamp(torch.clamp(pos + 1, min=int(prefix[b])), max=total)
        parts.append(attention(q[at:at + n].cpu(), rows_of(kc, tables[b], total), rows_of(vc, tables[b], total), pos,
                               lo, hi, scale, softcap, None if slopes is None else slopes.cpu()))
        at += n
    return tuple(torch.cat(x) for x in zip(*parts))


def assert_within(got, ref, v_cache, v_scale=None):
    """got against attention()'s result over the cache v_cache (codes when v_scale is given)."""
    v = dequantize(v_cache, v_scale)
    p_dtype = got.dtype if v_scale is None else torch.float16
    tol = tolerance(ref, got.dtype, p_dtype, v[torch.isfinite(v)].abs().max())
    err = (got.cpu().double() - ref[0]).abs()
    assert torch.isfinite(got).all()
    assert bool((err <= tol).all()), f"worst error / tolerance {(err / tol).max().item():.3g}, max abs {err.max().item():.3g}"
