"""Plain CPU oracle for the paged dense cache: bookkeeping, norm and rotation, attention.

TEST INFRASTRUCTURE.  Only ``tests/`` may import this module.  It shares no code with the HIP
library.  Whole numbers are Python integers, row by row; everything else is float64 from the
stored values, by the formulas of ``include/fadkv.h``.
"""
from __future__ import annotations

import math

import numpy as np


def pages_advance(page, new_lens, lens, table, ring, ring_state, max_tokens):
    """One step; returns a dict of the arrays after it (inputs are not changed)."""
    table, ring = np.array(table), np.array(ring)
    R, width = table.shape
    head, count = int(ring_state[0]), int(ring_state[1])
    num = len(ring)
    entering = ring.copy()
    asked = taken = put = total = 0
    cu, status, lens_out = [0], [], []
    slots, positions = np.full(max_tokens, -1, np.int64), np.full(max_tokens, -1, np.int64)
    for r in range(R):
        n, add = min(max(int(lens[r]), 0), width * page), int(new_lens[r])
        held = -(-n // page)
        if add < 0:
            for i in range(held):
                ring[(head + count + put) % num] = table[r, i]
                put += 1
            cu.append(cu[-1])
            status.append(2)
            lens_out.append(0)
            continue
        fits = n + add <= width * page
        need = -(-(n + add) // page) - held if fits else 0
        asked += need
        total += add
        ok = add == 0 or (fits and total <= max_tokens and (need == 0 or asked <= count))
        if ok:
            for i in range(need):
                table[r, held + i] = entering[(head + taken) % num]
                taken += 1
        begin, end = cu[-1], min(total, max_tokens)
        for i in range(end - begin):
            positions[begin + i] = n + i
            if ok:
                pid = int(table[r, (n + i) // page])
                slots[begin + i] = pid * page + (n + i) % page if 0 <= pid < num else -1
        cu.append(end)
        status.append(0 if ok else 1)
        lens_out.append(n + add if ok else n)
    return {"table": table, "ring": ring, "lens": np.array(lens_out, np.int64),
            "ring_state": np.array([(head + taken) % num, count - taken + put]),
            "cu": np.array(cu), "status": np.array(status, np.int64), "slots": slots,
            "positions": positions}


def rope_freqs(rot_dim, base, kind="plain", factor=1.0, low=1.0, high=4.0, original_len=8192.0):
    """(frequencies, mscale), pair by pair."""
    out = []
    for i in range(rot_dim // 2):
        f = base ** (-2.0 * i / rot_dim)
        if kind == "linear":
            f /= factor
        elif kind == "bands":
            wavelength = 2 * math.pi / f
            if wavelength > original_len / low:
                f /= factor
            elif wavelength >= original_len / high:
                mix = (original_len / wavelength - low) / (high - low)
                f = (1 - mix) * f / factor + mix * f
        elif kind == "yarn":
            def pair(turns):
                return rot_dim * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))
            first, last = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot_dim - 1)
            if last <= first:
                last = first + 0.001
            ramp = min(max((i - first) / (last - first), 0.0), 1.0)
            f = f * (1 - ramp) + f / factor * ramp
        out.append(f)
    m = 0.1 * math.log(factor) + 1 if kind == "yarn" and factor > 1 else 1.0
    return np.array(out), m


def norm_rope(x, weight, positions, freqs, eps, interleaved, mscale):
    """x [n][heads][d] -> (y, size): y normed and rotated, size the |.| that rounding acts on."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    z, size = y.copy(), np.abs(y)
    half = 0 if freqs is None else len(freqs)
    for t in range(x.shape[0]):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            angle = float(positions[t]) * float(freqs[i])
            c, s = mscale * math.cos(angle), mscale * math.sin(angle)
            z[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            z[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
            size[t, :, a] = size[t, :, b] = abs(mscale) * (np.abs(y[t, :, a]) + np.abs(y[t, :, b]))
    return z, size


def visible(pos, t, window, sinks):
    return t <= pos and (window == 0 or t > pos - window or t < sinks)


def attend_query(q, pos, K, V, there, scale, window, sinks):
    """One query q [d] at position pos over K, V [tokens][d] (there[t]: the token has a valid page).
    Returns (out [d], weight [d] = sum p |v|, largest |score|, largest sum |q k| * |scale|)."""
    seen = [t for t in range(min(pos + 1, K.shape[0])) if there[t] and visible(pos, t, window, sinks)]
    if not seen:
        z = np.zeros_like(q)
        return z, z, 0.0, 0.0
    k, v = K[seen], V[seen]
    s = scale * (k @ q)
    p = np.exp(s - s.max())
    p = p / p.sum()
    return p @ v, p @ np.abs(v), float(np.abs(s).max()), float(abs(scale) * (np.abs(k) @ np.abs(q)).max())
