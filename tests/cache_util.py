"""Plain 64-bit forms of the 4-bit cache and eviction operators for the tests,
written from their definitions on the CPU, and the error bounds the kernels
are held to."""
import math

import numpy as np
import torch

DC, DR, D, PAGE, ROW = 512, 64, 576, 64, 416


def bf16(x):
    """fp32 numpy values rounded to bf16, as a torch tensor."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def four_bit_scale(a):
    """Smallest number with four significant bits that is >= a / 7, by integers:
    a is m * 2^e with m an integer below 256."""
    m, e = math.frexp(a)
    m, e = int(m * 256), e - 8
    # s = k * 2^f, k in 8 .. 15, 7 k 2^f >= m 2^e; try exponents from below
    f = e
    while 7 * 15 * 2 ** (f - e + 20) < m * 2 ** 20:
        f += 1
    while 7 * 8 * 2 ** (f - e + 20) >= m * 2 ** 20:
        f -= 1
    for f in (f, f + 1):
        for k in range(8, 16):
            if 7 * k * 2 ** (f - e + 20) >= m * 2 ** 20:
                return k * 2.0 ** f
    raise AssertionError


def quantise(rows):
    """bf16 rows [N, 576] -> uint8 [N, 416] by the definition."""
    out = np.zeros((rows.shape[0], ROW), np.uint8)
    x = f64(rows)
    rope = rows[:, DC:].contiguous().view(torch.uint8).cpu().numpy().copy()
    for r in range(rows.shape[0]):
        poison = False
        scales = np.zeros(16, np.float32)
        for g in range(16):
            v = x[r, 32 * g:32 * g + 32]
            codes = [8] * 32
            top = np.abs(v).max()
            if not top < 2.0 ** 120:
                poison = True
            elif top >= 2.0 ** -118:
                s = four_bit_scale(float(top))
                scales[g] = s
                codes = []
                for y in v:
                    low = math.floor(y / s)
                    rest = y - low * s
                    codes.append(8 + low + int(2 * rest > s or (2 * rest == s and low % 2 != 0)))
            for w in range(4):
                c = codes[8 * w:8 * w + 8]
                word = sum(c[2 * k] << (4 * k) | c[2 * k + 1] << (4 * k + 16) for k in range(4))
                out[r, 16 * g + 4 * w:16 * g + 4 * w + 4] = np.frombuffer(np.uint32(word).tobytes(), np.uint8)
        out[r, 256:288] = bf16(scales).view(torch.uint8).numpy()
        out[r, 288:] = np.frombuffer(b"\xff\x7f" * 64, np.uint8) if poison else rope[r]
    return out


def values(raw):
    """uint8 rows [..., 416] -> fp64 values [..., 576]."""
    raw = np.ascontiguousarray(raw)
    lead = raw.shape[:-1]
    word = raw[..., :256].copy().view(np.uint32).reshape(*lead, 64)
    scale = f64(torch.from_numpy(raw[..., 256:288].copy()).view(torch.bfloat16)).reshape(*lead, 16)
    rope = f64(torch.from_numpy(raw[..., 288:].copy()).view(torch.bfloat16)).reshape(*lead, 64)
    v = np.zeros((*lead, 64, 8))
    for j in range(8):
        v[..., j] = ((word >> np.uint32(4 * (j // 2 + 4 * (j % 2)))) & 15).astype(np.float64) - 8
    return np.concatenate([v.reshape(*lead, DC) * np.repeat(scale, 32, -1), rope], -1)


class Paged:
    """A shuffled page table over a pool with spare pages."""

    def __init__(self, lens, seed=0, spare=3, extra=0):
        rng = np.random.default_rng(seed)
        need = [-(-max(n, 1) // PAGE) + extra for n in lens]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), max(need)), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n

    def row(self, b, i):
        if i < 0 or i >= self.table.shape[1] * PAGE:
            return -1
        pg = self.table[b, i // PAGE]
        return int(pg) * PAGE + i % PAGE if 0 <= pg < self.pages else -1

    def rows(self, b, pos):
        return np.array([self.row(b, int(i)) for i in pos], np.int64)

    @property
    def cuda(self):
        return torch.from_numpy(self.table).cuda()


def latents(n, seed, std=0.7):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, D, generator=g) * std).to(torch.bfloat16)


def queries(B, T, H, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, T, H, D, generator=g) * std).to(torch.bfloat16)


def attend(q, kv, scale):
    """One query token in 64 bits: q [H, 576], kv [n, 576] -> o, lse, and bounds
    of what a kernel may be off in each.

    A score is an fp32 sum of 576 exact products in some order (each partial
    sum rounded or cut, at most 2^-23 of it): off by ds <= 580 * 2^-23 * scale
    * sum|q k|, and by its own scaling, 2^-23 |s|.  A weight then is off by 2 ds
    (relative, in numerator and denominator), by ex2's 2^-21, and by the one
    rounding of P to bf16, 2^-8; the output is rounded to bf16 once, 2^-8."""
    H = q.shape[0]
    if kv.shape[0] == 0:
        return np.zeros((H, DC)), np.full(H, -np.inf), np.zeros((H, DC)), np.zeros(H)
    s = q @ kv.T * scale
    ds = (580 * 2.0 ** -23 * abs(scale) * (np.abs(q) @ np.abs(kv).T) + 2.0 ** -23 * np.abs(s)).max(-1)
    m = s.max(-1, keepdims=True)
    e = np.exp(s - m)
    tot = e.sum(-1, keepdims=True)
    lse = (m + np.log(tot))[:, 0]
    p = e / tot
    o, mass = p @ kv[:, :DC], p @ np.abs(kv[:, :DC])
    tol_o = (2.0 ** -8 + 4 * ds[:, None] + 2.0 ** -19) * mass * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(o) + 1e-30
    tol_lse = ds + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)
    return o, lse, tol_o, tol_lse


def check(got, want, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    off = np.abs(np.where(same, 0.0, got - np.where(same, 0.0, want)))
    off = np.where(same, 0.0, off)
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(off / np.maximum(tol, 1e-300)):.3g} x the bound"


def check_attention(o, lse, q, kv_of, scale, what):
    """o, lse of a kernel against attend() for every (b, t); kv_of(b, t) gives the
    values attended to."""
    B, T, H, _ = q.shape
    qd = f64(q)
    o, lse = f64(o), f64(lse)
    for b in range(B):
        for t in range(T):
            ro, rl, to, tl = attend(qd[b, t], kv_of(b, t), scale)
            check(lse[b, t], rl, tl, f"{what}: lse of ({b}, {t})")
            check(o[b, t], ro, to, f"{what}: o of ({b}, {t})")


def plan(acc, pos, n, K, n_sink, n_recent):
    """One sequence's eviction plan by sorting: src list of min(n, K) slots."""
    m = min(n, K)
    if n <= K:
        return list(range(m))
    end = max(pos[:n]) + 1
    safe = [pos[i] < n_sink or pos[i] >= end - n_recent for i in range(n)]
    weight = [-math.inf if math.isnan(a) else a for a in acc[:n]]
    order = sorted(range(n), key=lambda i: (not safe[i], 0.0 if safe[i] else -weight[i], i))
    stays = set(order[:K])
    movers = iter(sorted(i for i in stays if i >= m))
    return [i if i in stays else next(movers) for i in range(m)]
