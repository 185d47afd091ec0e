"""The paged 8-bit cache in 64 bits, from its definition: one sequence, page and head at a time.

Shares no code with the CUDA path.  Tolerances are derived here from the storage types.
"""
import numpy as np
import torch

E4M3 = np.array([(-1.0 if c & 128 else 1.0) * (
    (c & 7) * 2.0 ** -9 if (c >> 3) & 15 == 0 else (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10))
    if c & 127 != 127 else np.nan for c in range(256)])


def values(pages, scales):
    """float64 values of e4m3 codes [P][U][T][d] with scales [P][U]."""
    return E4M3[pages.view(torch.uint8).cpu().numpy()] * \
        scales.cpu().double().numpy()[:, :, None, None]


def rotate(x, pos, base):
    """Rotate-half rotation of x [..., d] (float64) at scalar position pos; base 0: none."""
    if base == 0:
        return x
    h = x.shape[-1] // 2
    z = (x[..., :h] + 1j * x[..., h:]) * np.exp(1j * pos * base ** (-np.arange(h) / h))
    return np.concatenate([z.real, z.imag], -1)


def scale_for(a):
    """The least power of two s with a <= 448 s, at least 2^-100."""
    e = -100
    while a > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(step, K, V, k_pages, v_pages, k_scales, v_scales):
    """Returns [(values, tolerance, scales)] for keys and values: the exact values [P][U][T][d]
    that the codes stand for before rounding, how far a code's value may be off (0 where the bytes
    must not change) and the exact scales."""
    out = []
    for x, pages, scales, rot in ((K, k_pages, k_scales, step["base"] != 0),
                                  (V, v_pages, v_scales, False)):
        x = x.detach().cpu().double().numpy()
        vals = values(pages, scales)
        sc = scales.cpu().double().numpy().copy()
        tol = np.zeros_like(vals)
        T, d = vals.shape[2], vals.shape[3]
        for b, n in enumerate(step["lens"]):
            m_all = step["offs"][b + 1] - step["offs"][b]
            m = min(m_all, n)
            for j in range((n - m) // T, (n - 1) // T + 1) if m else ():
                pg = step["table"][b][j]
                lo, hi = max(n - m, j * T), min(n, (j + 1) * T)
                rows = x[step["offs"][b] + m_all - n + lo:step["offs"][b] + m_all - n + hi]
                size = np.abs(rows)
                size = np.where(np.isfinite(size), size, 0.0)
                if rot:
                    size = size[..., :d // 2] + size[..., d // 2:]
                for u in range(vals.shape[1]):
                    s = scale_for(size[:, u].max())
                    if lo > j * T:
                        s = max(s, sc[pg, u])
                        if s != sc[pg, u]:  # earlier codes are rounded again
                            tol[pg, u, :lo - j * T] = half_step(vals[pg, u, :lo - j * T], s)
                    sc[pg, u] = s
                    for t in range(lo, hi):
                        y = rows[t - lo, u]
                        with np.errstate(invalid="ignore"):
                            # an fp32 rotation: products and the sum round, and an angle of up to
                            # half a turn is held to 2^-24 of a turn: under 2^-21 of |a|+|b|
                            r = rotate(y, t, step["base"]) if rot else y
                            err = 2.0 ** -21 * (np.tile(size[t - lo, u], 2) if rot else 0.0)
                        r = np.clip(r, -448.0 * s, 448.0 * s)
                        vals[pg, u, t - j * T] = r
                        tol[pg, u, t - j * T] = half_step(np.abs(r) + err, s) + err
        out.append((vals, tol, sc))
    return out


def half_step(v, s):
    """Half a step of e4m3 at v with scale s: 2^-4 relative, 2^-10 in the subnormal range."""
    return np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10 * s)


def attend(step, q, k_pages, v_pages, k_scales, v_scales, hq, dtype):
    """(out, tolerance) [n][hq][d] in float64; NaN in `out` where a row belongs to no sequence."""
    q = q.detach().cpu().double().numpy()
    K, V = values(k_pages, k_scales), values(v_pages, v_scales)
    P, U, T, d = K.shape
    G = hq // U
    scale = step.get("scale") or 1.0 / np.sqrt(d)
    out = np.full((q.shape[0], hq, d), np.nan)
    tol = np.zeros_like(out)
    # relative error of a query element and of a probability: 2^-11 where the storage type has
    # fewer bits than that, 2^-23 (two roundings) in 32 bits; a dot product of d terms in 32 bits
    # adds d 2^-24 of the sum of its terms' sizes, a sum over tokens (in tiles) 2^-24 for each of a
    # tile's 128 terms and of the tiles; the output's own rounding is 2^-8 and 2^-24
    fine = dtype == torch.float32
    rel, own = (2.0 ** -23, 2.0 ** -24) if fine else (2.0 ** -11, 2.0 ** -8)
    for b, n in enumerate(step["lens"]):
        m = step["offs"][b + 1] - step["offs"][b]
        for i in range(m):
            pos = n - m + i
            row = step["offs"][b] + i
            lo = max(0, pos + 1 - step["window"]) if step["window"] else 0
            t = np.array([x for x in range(lo, pos + 1) if 0 <= step["table"][b][x // T] < P], int)
            if not len(t):
                out[row] = 0.0
                continue
            pg = np.array([step["table"][b][x // T] for x in t])
            for u in range(U):
                kk, vv = K[pg, u, t % T], V[pg, u, t % T]
                for h in range(u * G, (u + 1) * G):
                    r = rotate(q[row, h], pos, step["base"])
                    s = kk @ r * scale
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    o = p @ vv
                    off = (np.abs(kk) @ np.abs(r)) * scale * (rel + (d + 8) * 2.0 ** -24)
                    # each weight is off by a factor within exp(+-off) (1 +- rel), the
                    # normaliser by as much
                    sums = (128 + len(t) / 128) * 2.0 ** -24
                    w = np.expm1(2 * off.max()) + 2 * rel + 2 * sums
                    out[row, h] = o
                    tol[row, h] = w * (p @ np.abs(vv)) + own * np.abs(o) * (1 + w) + 1e-30
    return out, tol
