"""Plain 64-bit implementations of the calls around a step (torch, CPU), for the tests: straight from
the definitions in include/jf.h, one sequence and one row at a time.  They share no code with the
kernels."""
import math

import torch

PAGE = 16
PROMPT = 1 << 30


def half_step(dtype):
    """The most a rounding to dtype is off, relative to the value."""
    return torch.finfo(dtype).eps / 2


def rotate(x, pos, freq, interleaved, scale, weight, eps):
    """Heads x [n, H, D] of n tokens at positions pos [n].  Returns (y, tol), both float64; tol bounds
    the kernel's distance.  u = 2^-24 is one fp32 rounding.
      Norm: D squares and sums (a thread's 16 in a row, then log2(D / 16) <= 3 levels), / D, + eps,
      sqrt, 1 /, * w, * x: under 26 u relative.
      Turn: the fraction of a turn is rounded to fp32 once (at most half a turn: pi u radians) and
      carries 2^-51 of the whole angle (freq / 2 pi rounded twice in 53 bits; the reference's own
      pos * freq once); sine and cosine 2 u each, * scale u, two products and a sum 3 u: under 10 u of
      |a| + |b|.
    The stored value is rounded to bf16 once more."""
    u = 2.0 ** -24
    x = x.double()
    off = torch.zeros_like(x)
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
        off = 26 * u * x.abs()
    if freq is not None:
        n = freq.numel()
        at = torch.arange(n)
        lo, hi = (2 * at, 2 * at + 1) if interleaved else (at, at + n)
        angle = pos.double()[:, None, None] * freq.double()
        cos, sin = scale * torch.cos(angle), scale * torch.sin(angle)
        a, b = x[..., lo], x[..., hi]
        size = abs(scale) * (a.abs() + b.abs())
        err = size * (10 * u + 2.0 ** -51 * angle.abs()) + abs(scale) * (off[..., lo] + off[..., hi])
        x, off = x.clone(), off.clone()
        x[..., lo], x[..., hi] = a * cos - b * sin, b * cos + a * sin
        off[..., lo], off[..., hi] = err, err
    h = half_step(torch.bfloat16)
    return x, off * (1 + h) + h * x.abs() + 2.0 ** -133     # the last: bf16's subnormal step


def adjust(x, had, prompt, rep, pres, freq, bias, ok, masked, dtype):
    """One row: logits x [V], had [V] times generated, prompt [V] bool, ok [V] bool or None.  Returns
    (y, tol): a quotient or product, frequency * c + presence, their sum and the bias round five
    times, each by u of a partial result no larger than the sizes' sum, then once to dtype."""
    u = 2.0 ** -24
    x = x.double()
    seen = (had > 0) | prompt
    y = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    pen = torch.where(had > 0, pres + freq * had.double(), 0.0)
    add = torch.zeros_like(y) if bias is None else bias.double()
    size = y.abs() + pen.abs() + add.abs()
    y = y - pen + add
    tol = torch.where(torch.isfinite(size), 5 * u * size, 0.0)
    tol = tol + half_step(dtype) * torch.where(torch.isfinite(y), y.abs() + tol, 0.0)
    if ok is not None:
        y = torch.where(ok, y, masked)
        tol = torch.where(ok, tol, half_step(dtype) * abs(masked) if math.isfinite(masked) else 0.0)
    return y, tol


def within(got, want, tol):
    """|got - want| <= tol, with equal infinities and NaN for NaN."""
    got = got.double()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    return bool((same | ((got - want).abs() <= tol)).all())


def unpack(bits, V):
    """Grammar row [words] int32 -> bool [V]."""
    v = torch.arange(V)
    return ((bits.long()[v // 32] >> (v % 32)) & 1).bool()


def random_trees(B, N, g, back=6):
    """(parent [B, N], ancestor-or-self bool [B, N, N])."""
    parent = torch.full((B, N), -1, dtype=torch.int64)
    sees = torch.eye(N, dtype=torch.bool).repeat(B, 1, 1)
    for b in range(B):
        for i in range(1, N):
            parent[b, i] = max(0, i - int(torch.randint(1, back + 1, (1,), generator=g)))
            sees[b, i] |= sees[b, parent[b, i]]
    return parent.to(torch.int32), sees


def pack_bits(sees):
    """Bool [..., N, N] -> int64 [..., N, ceil(N / 64)]."""
    N = sees.shape[-1]
    words = torch.nn.functional.pad(sees, (0, -N % 64)).unflatten(-1, (-1, 64))
    return (words.long() << torch.arange(64)).sum(-1)
