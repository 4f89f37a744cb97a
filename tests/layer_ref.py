"""Plain 64-bit implementations of rotation by position, prompt attention and attention behind a shared prefix."""
import numpy as np

import mx_ref


def rotate(x, positions, freqs, interleaved):
    """x [tokens, heads, dim]; freqs fp32 [rotary / 2] -> (rotated, |a| + |b| of each value's pair)."""
    n = 2 * len(freqs)
    angle = positions.astype(np.float64)[:, None, None] * freqs.astype(np.float64)
    c, s = np.cos(angle), np.sin(angle)
    y, size = x.astype(np.float64).copy(), np.abs(x)
    at = (slice(0, n, 2), slice(1, n, 2)) if interleaved else (slice(0, n // 2), slice(n // 2, n))
    a, b = x[..., at[0]], x[..., at[1]]
    y[..., at[0]], y[..., at[1]] = a * c - b * s, b * c + a * s
    size[..., at[0]] = size[..., at[1]] = np.abs(a) + np.abs(b)
    return y, size


def softmax_rows(q, k, v, seen, scale):
    """q [rows, dim], k and v [positions, dim], seen [rows, positions] -> (out, sum of p|v|, largest |q||k|)."""
    x = q @ k.T * scale
    size = (np.abs(q) @ np.abs(k).T * abs(scale) * seen).max(1, initial=0)
    x = np.where(seen, x, -np.inf)
    top = x.max(1, initial=-np.inf, keepdims=True)
    p = np.where(seen, np.exp(x - np.where(np.isfinite(top), top, 0)), 0)
    total = p.sum(1, keepdims=True)
    p = p / np.where(total == 0, 1, total)
    return p @ v, p @ np.abs(v), size


def prompt(q, k, v, starts, scale, window=0):
    """q [tokens, heads, dim], k and v [tokens, kv, dim] -> as softmax_rows, for every token of a sequence."""
    out, weight, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2] + (1,))
    group = q.shape[1] // k.shape[1]
    for b, e in zip(starts[:-1], starts[1:]):
        i = np.arange(e - b)
        seen = i <= i[:, None]
        if window:
            seen &= i > i[:, None] - window
        for h in range(q.shape[1]):
            out[b:e, h], weight[b:e, h], size[b:e, h, 0] = softmax_rows(q[b:e, h], k[b:e, h // group], v[b:e, h // group], seen, scale)
    return out, weight, size


def shared(q, cache, prefix, prefix_len, table, lens, scale):
    """q [seqs, q_len, heads, dim] -> as softmax_rows, and the largest |v|."""
    seqs, q_len, heads, dim = q.shape
    out, weight, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3] + (1,))
    kp, vp = cache.rows(prefix[None], 0, prefix_len)
    group = heads // kp.shape[0]
    v_top = np.abs(vp).max(initial=0)
    for s in range(seqs):
        ko, vo = cache.rows(table, s, lens[s])
        k, v = np.concatenate([kp, ko], 1), np.concatenate([vp, vo], 1)
        v_top = np.fmax(v_top, np.abs(vo).max(initial=0))
        n = prefix_len + lens[s]
        seen = np.arange(n) <= (n - q_len + np.arange(q_len))[:, None]
        for h in range(heads):
            out[s, :, h], weight[s, :, h], size[s, :, h, 0] = softmax_rows(q[s, :, h], k[h // group], v[h // group], seen, scale)
    return out, weight, size, v_top


def codes_of(x, slack, exponent):
    """The e4m3 codes that x may become under a scale, x being known to within `slack`."""
    scale = np.ldexp(1.0, exponent - 127)
    return [mx_ref.encode_e4m3(np.clip((x + d) / scale, -448, 448)) for d in (-slack, 0, slack)]
