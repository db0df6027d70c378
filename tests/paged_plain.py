"""Plain 64-bit forms of the paged-cache operators, from their definitions, on
CPU tensors: one row, one head, one position at a time where that is the
definition.  The tests compare the kernels with these."""
import math

import torch


def norm_rope(x, weight, eps, offset, positions, inv_freq, interleaved):
    """Rows [T, heads, D] of any float type to float64."""
    x = x.double()
    T, _, D = x.shape
    if weight is not None:
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * (weight.double() + offset)
    if inv_freq is None:
        return x
    out = x.clone()
    half = len(inv_freq)
    for p in range(half):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        a = positions.double() * float(inv_freq[p])
        c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
        out[..., i] = x[..., i] * c - x[..., j] * s
        out[..., j] = x[..., i] * s + x[..., j] * c
    return out


def visible(n_k, p, window, sinks):
    """Positions of 0..n_k-1 that a row at position p sees."""
    return [j for j in range(n_k) if j <= p and (window == 0 or j > p - window or j < sinks)]


def attend_row(q, K, V, idx, scale):
    """One row's softmax over the positions idx, float64; zeros if there are none."""
    if not idx:
        return torch.zeros(V.shape[-1], dtype=torch.float64)
    x = (K[idx].double() @ q.double()) * scale
    w = torch.exp(x - x.max())
    return (w / w.sum()) @ V[idx].double()


def attend(q, K, V, first, scale, window, sinks):
    """q [n, Hq, D] at positions first.., K and V [N, Hkv, D]: float64 [n, Hq, D]."""
    n, Hq, _ = q.shape
    G = Hq // K.shape[1]
    out = torch.zeros(n, Hq, V.shape[-1], dtype=torch.float64)
    for i in range(n):
        idx = visible(K.shape[0], first + i, window, sinks)
        for h in range(Hq):
            out[i, h] = attend_row(q[i, h], K[:, h // G], V[:, h // G], idx, scale)
    return out


def gather(cache, table, length, page_size, layout, scale=None):
    """Positions 0..length-1 of one sequence as float64 [length, Hkv, D] (pages of -1: zeros)."""
    view = cache if layout == "NHD" else cache.transpose(1, 2)
    rows = []
    for j in range(length):
        page = int(table[j // page_size])
        row = view[page, j % page_size].double() if page >= 0 else torch.zeros(view.shape[2:], dtype=torch.float64)
        rows.append(row)
    x = torch.stack(rows) if rows else torch.zeros((0,) + tuple(view.shape[2:]), dtype=torch.float64)
    return x if scale is None else x * scale.double()[None, :, None]


def inv_freq(rot, theta=10000.0):
    return [theta ** (-2.0 * p / rot) for p in range(rot // 2)]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def attention_tolerance(v_abs_max, roundings=1):
    """What an attention output in bf16 may be off by: its own rounding (half a
    step of a value at most v_abs_max), the rounding of each probability
    (2^-8 relative at bf16, so at most that share of v_abs_max once for the
    numerator), and fp32 arithmetic over the slots, far below both."""
    return v_abs_max * (half_step(torch.bfloat16) * (1 + roundings) + 2.0 ** -14)


def e4m3_values():
    """All finite non-negative e4m3 values, ascending."""
    vals = []
    for bits in range(127):
        e, m = bits >> 3, bits & 7
        vals.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return vals


