"""Plain 64-bit forms of the verify pass over a 4-bit cache, for the tests."""
import math

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    """The 127 non-negative finite e4m3 values by code."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append((m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))
    return np.array(out)


E4M3 = e4m3_values()


def nearest_even(v, grid):
    """Index of the nearest grid value (ties to the even index), v >= 0, clamped to the last."""
    hi = np.minimum(np.searchsorted(grid, v), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - v, v - grid[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quantize(x, unit):
    """[..., hd] float64 -> (codes [..., hd/2] uint8, scales [..., hd/16] uint8)."""
    big = 3.3895313892515355e38  # the largest finite bf16
    x = np.clip(np.where(np.isnan(x), 0.0, x), -big, big)
    g = x.reshape(*x.shape[:-1], -1, 16)
    e = nearest_even(np.minimum(np.abs(g).max(-1) / (6.0 * unit), 448.0), E4M3)
    step = (E4M3[e] * unit)[..., None]
    y = np.where(step > 0, np.abs(g) / np.where(step > 0, step, 1.0), 0.0)
    c = (nearest_even(np.minimum(y, 6.0), GRID) | (np.signbit(g).astype(np.int64) << 3)).reshape(x.shape)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8), e.astype(np.uint8)


def dequantize(codes, scales, unit):
    full = np.concatenate([GRID, -GRID])
    v = np.stack([full[codes & 15], full[codes >> 4]], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    s = np.where(scales == 127, np.nan, E4M3[np.minimum(scales & 127, 126)])
    return v * np.repeat(s, 16, -1) * unit


def rope_freqs(rot, base, scaling="plain", factor=1.0, low=1.0, high=4.0, orig_len=8192.0):
    i = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "wavelen":
        w = np.clip((orig_len * f / (2 * math.pi) - low) / (high - low), 0, 1)
        return f * ((1 - w) / factor + w), 1.0
    if scaling == "yarn":
        d = lambda n: rot * math.log(orig_len / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
        a, e = max(math.floor(d(high)), 0), min(math.ceil(d(low)), rot - 1)
        w = np.clip((i - a) / max(e - a, 0.001), 0, 1)
        return f * (w / factor + 1 - w), 0.1 * math.log(factor) + 1
    return f, 1.0


def qkv_heads(x, H, KVH, hd, q_norm, k_norm, eps, rope, pos):
    """x [rows][(H + 2 KVH) hd] -> (q, k, v) [rows][heads][hd] and the normed magnitude
    bound per head; rope: (freqs, amp, rot, interleaved) or None."""
    y = x.reshape(len(x), -1, hd).astype(np.float64)
    parts = [y[:, :H], y[:, H:H + KVH], y[:, H + KVH:]]
    for i, n in enumerate((q_norm, k_norm)):
        z = parts[i]
        if n is not None:
            z = z / np.sqrt((z ** 2).mean(-1, keepdims=True) + eps) * n
        if rope is not None:
            f, amp, rot, inter = rope
            a = (pos.astype(np.float64)[:, None] * f)[:, None]
            c, s = amp * np.cos(a), amp * np.sin(a)
            out = z.copy()
            p, r = (z[..., 0:rot:2], z[..., 1:rot:2]) if inter else (z[..., :rot // 2], z[..., rot // 2:rot])
            lo, hi = p * c - r * s, r * c + p * s
            if inter:
                out[..., 0:rot:2], out[..., 1:rot:2] = lo, hi
            else:
                out[..., :rot // 2], out[..., rot // 2:rot] = lo, hi
            z = out
        parts[i] = z
    return parts


def attend(Q, k, v, tk, tv, see, scale):
    """One request: Q [R][H][hd]; k, v [P][KVH][hd]; tk, tv [R][KVH][hd]; see [R][R] bool.
    -> o, lse, sum p|v| (per output), the largest sum |q||k| * scale per row."""
    R, H, hd = Q.shape
    KVH = tk.shape[1]
    K, V = np.concatenate([k, tk]), np.concatenate([v, tv])
    vis = np.concatenate([np.ones((R, len(k)), bool), see], 1)
    o, lse = np.zeros((R, H, hd)), np.full((R, H), -np.inf)
    mag, big = np.zeros((R, H, hd)), np.zeros((R, H))
    for h in range(H):
        kh = h // (H // KVH)
        for i in range(R):
            on = vis[i]
            if not on.any():
                continue
            s = K[on, kh] @ Q[i, h] * scale
            m = s.max()
            p = np.exp(s - m)
            lse[i, h] = m + np.log(p.sum())
            o[i, h] = p @ V[on, kh] / p.sum()
            mag[i, h] = p @ np.abs(V[on, kh]) / p.sum()
            big[i, h] = (np.abs(K[on, kh]) @ np.abs(Q[i, h])).max() * scale
    return o, lse, mag, big


def process(logits, counts, paths, pen, bias_tok, bias_val, allowed):
    """One row in fp32, each operation rounded: the definition of tree_logits_process."""
    f = np.float32
    V = len(logits)
    z = logits.astype(f).copy()
    c = (counts & 32767).astype(np.int64) if counts is not None else np.zeros(V, np.int64)
    for t in paths:
        if 0 <= t < V:
            c[t] += 1
    seen = c > 0
    if counts is not None:
        seen |= (counts & 32768) != 0
    rep, freq, pres = (f(p) for p in pen) if pen is not None else (f(1), f(0), f(0))
    with np.errstate(invalid="ignore", over="ignore"):
        z = np.where(seen, np.where(z > 0, z / rep, z * rep), z).astype(f)
        z = np.where(c > 0, ((z - (freq * c.astype(f)).astype(f)).astype(f) - pres).astype(f), z)
        add = {}
        for t, x in zip(bias_tok, bias_val):
            if 0 <= t < V:
                add[t] = f(add[t] + f(x)) if t in add else f(x)
        for t, x in add.items():
            z[t] = f(z[t] + x)
    if allowed is not None:
        z = np.where(allowed, z, f(-np.inf))
    return z
