"""Plain float64 restatement of the calls around the verification step:
rotary positions with several axes, the 8-bit cache formats and attention of
one new token (TEST INFRASTRUCTURE ONLY)."""

import numpy as np

TINY = 2.0 ** -100


def axis_of_pair_ref(sections, section_order):
    """The axis whose position pair i takes."""
    left, out, a = list(sections), [], 0
    while any(left):
        if left[a]:
            out.append(a)
            left[a] -= 1
            if section_order:
                a = (a + 1) % len(left)
        else:
            a = (a + 1) % len(left)
    return out


def rope_axes_ref(x, positions, inv_freq, sections, style, section_order):
    """x [rows][heads][D], positions [axes][rows], inv_freq [pairs] (float32
    values) -> float64 rotated rows."""
    x = np.asarray(x, np.float64)
    axis = axis_of_pair_ref(sections, section_order)
    n = len(axis)
    ang = np.asarray(positions, np.float64)[axis].T * np.asarray(inv_freq, np.float64)   # [rows][n]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    out = x.copy()
    ia, ib = (np.arange(n), np.arange(n) + n) if style else (2 * np.arange(n), 2 * np.arange(n) + 1)
    a, b = x[..., ia], x[..., ib]
    out[..., ia] = a * c - b * s
    out[..., ib] = b * c + a * s
    return out


def round_e4m3_ref(y):
    """Nearest e4m3 value (ties to even), |y| <= 464."""
    y = np.asarray(y, np.float64)
    _, e = np.frexp(y)                                   # |y| in [2^(e-1), 2^e)
    step = np.ldexp(1.0, np.maximum(e, -5) - 4)          # 4 significant bits, spacing >= 2^-9
    return np.clip(np.rint(y / step) * step, -448.0, 448.0)


def kv_quant_ref(x, fmt):
    """Rows x [..., D] -> (code values float64 [..., D], scale float32 [...]).
    fmt: "e4m3" or "int8"."""
    x = np.asarray(x, np.float64)
    finite = np.isfinite(x).all(-1)
    x = np.where(finite[..., None], x, 0.0)
    top = np.abs(x).max(-1)
    if fmt == "e4m3":
        scale = np.full(top.shape, TINY)
        for n in range(-100, 121):
            scale = np.where(top > 448.0 * scale, 2.0 ** (n + 1), scale)
        code = round_e4m3_ref(x / scale[..., None])
    else:
        top = np.maximum(top, TINY)
        scale = top / 127.0
        code = np.rint(127.0 * x / top[..., None])
    code = np.where(finite[..., None], code, 0.0)
    return code, np.where(finite, scale, np.nan).astype(np.float32)


def decode_attention_ref(q, k, v, scale):
    """One token: q [Hq][D], k and v [n][Hkv][D] -> (out [Hq][D], lse [Hq],
    weight-averaged |v| [Hq][D], largest sum of |q||k| [Hq])."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    hq, d = q.shape
    n, hkv = k.shape[:2]
    if n == 0:
        return np.zeros((hq, d)), np.full(hq, -np.inf), np.zeros((hq, d)), np.zeros(hq)
    out, lse, absv, big = np.empty((hq, d)), np.empty(hq), np.empty((hq, d)), np.empty(hq)
    for h in range(hq):
        g = h // (hq // hkv)
        s = scale * (k[:, g] @ q[h])
        m = s.max()
        p = np.exp(s - m)
        out[h] = p @ v[:, g] / p.sum()
        absv[h] = p @ np.abs(v[:, g]) / p.sum()
        lse[h] = m + np.log(p.sum())
        big[h] = (np.abs(k[:, g]) @ np.abs(q[h])).max() * scale
    return out, lse, absv, big
