"""The operators around the attention in 64 bits, from their definitions (CPU, small sizes)."""
import math

import torch

TINY = 2.0 ** -126
F64 = torch.float64


def rope_parts(x, positions, inv_freq, offset, interleaved, inverse=False, amplitude=1.0):
    """x (tokens, heads, dim) rotated, and per value the sum of the magnitudes of its pair (0 where not rotated)."""
    x = x.to(F64)
    y, mag = x.clone(), torch.zeros_like(x)
    n = inv_freq.numel()
    for i in range(n):
        a, b = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + i + n)
        # whole turns are dropped exactly: position and frequency as integers over 2^80
        turns = [(int(p) * int(float(inv_freq[i]) * 2 ** 80)) for p in positions]
        two_pi = int(math.pi * 2 ** 52) * 2 ** 29 + _PI_REST
        angle = torch.tensor([(t % two_pi) / 2 ** 80 for t in turns], dtype=F64)[:, None]
        c, s = angle.cos() * amplitude, angle.sin() * amplitude * (-1 if inverse else 1)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, mag


def _two_pi_rest():
    """2 pi 2^80 - int(pi 2^52) 2^29, from Machin's formula in integers."""
    one = 1 << 120

    def arctan_inv(q):
        total, term, k, sign = 0, one // q, 1, 1
        while term:
            total += sign * (term // k)
            term //= q * q
            k += 2
            sign = -sign
        return total
    pi = 4 * (4 * arctan_inv(5) - arctan_inv(239))
    return (2 * pi >> 40) - int(math.pi * 2 ** 52) * 2 ** 29


_PI_REST = _two_pi_rest()


def store_values(x, weight, eps, positions, inv_freq, offset, interleaved, amplitude=1.0):
    """(tokens, heads, dim) values before they are rounded to a cache format, and the pair magnitudes."""
    x = x.to(F64).clone()
    n = min(x.shape[-1], 512)
    if eps is not None:
        ms = x[..., :n].square().mean(-1, keepdim=True)
        x[..., :n] = x[..., :n] / torch.sqrt(ms + eps) * (weight.to(F64) if weight is not None else 1.0)
    if inv_freq is None:
        return x, torch.zeros_like(x)
    return rope_parts(x, positions, inv_freq, offset, interleaved, False, amplitude)


def visible(q_len, length, ratio, residual, causal):
    """Keys each of the q_len queries of a sequence may see."""
    out = []
    for i in range(q_len):
        p = length * ratio + residual - q_len + i
        out.append(sum((j + 1) * ratio <= p + 1 for j in range(length)) if causal else length)
    return out


def scores(q, k, w, ks=None):
    """(queries, keys) index scores and the sums of magnitudes behind them; q (t, h, d), k (n, d), w (t, h), ks (n)."""
    q, k, w = q.to(F64), k.to(F64), w.to(F64)
    s = torch.einsum("thd,nd->thn", q, k)
    m = torch.einsum("thd,nd->thn", q.abs(), k.abs())
    scale = ks.to(F64) if ks is not None else torch.ones(k.shape[0], dtype=F64)
    return (torch.einsum("thn,th->tn", s.clamp(min=0), w) * scale,
            torch.einsum("thn,th->tn", m, w.abs()) * scale)


def topk(row, k, length, block=1, first=0, last=0):
    """Selected indices of one row (a list of Python floats), ascending and padded with -1."""
    have = -(-length // block)
    best = []
    for j in range(have):
        v = [x for x in row[j * block:min((j + 1) * block, length)] if x == x and x > -math.inf]
        if j < first or j >= have - last:
            best.append((-math.inf, -1.0, j))
        elif v:
            best.append((-max(v), 0.0, j))
    best.sort(key=lambda t: (t[1], t[0] if t[1] == 0.0 else 0.0, t[2]))
    got = sorted(j for _, _, j in best[:k])
    return got + [-1] * (k - len(got))
