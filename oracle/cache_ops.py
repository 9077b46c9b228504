"""Float64 CPU oracle of the operators around the attention: per-head RMS norm
with position rotation and its gradients, the paged 8-bit cache (write and
read-back) and attention over what it holds.

TEST INFRASTRUCTURE, like attention.py; it shares no code with the CUDA path.

  norm + rotation (a row x of d values):  r = 1/sqrt(mean(x^2) + eps), z = x r w,
      y_a = z_a cos - z_b sin, y_b = z_b cos + z_a sin for each pair (a, b);
      columns >= rot pass. Gradients by the chain rule, the norm's Jacobian
      written out: dz/dx = r (I - x x^T r^2 / d) diag-scaled by w.
  cache: a page's scale is the smallest power of two 2^e, -100 <= e <= 120, with
      amax <= 448 * 2^e; a value is stored as the nearest e4m3 number of
      value / scale (ties to even), a non-finite one as NaN.

Pins (tests/test_oracle_ops.py): norms of rotated rows, angles of shifted
positions, finite differences of every gradient, the 256 e4m3 values against
torch's conversion, idempotent quantisation, attention against attention.py.
"""

from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -100, 120


def _pair_index(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, cos, sin, interleaved=False):
    """Turn the first 2 * cos.shape[-1] columns of x [..., d]; cos, sin [..., rot / 2] broadcast."""
    rot = 2 * cos.shape[-1]
    a, b = _pair_index(rot, interleaved)
    y = np.array(x, dtype=np.float64)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def norm_rope(x, w, cos, sin, interleaved=False, eps=1e-6):
    """x [..., d] -> y; w [d] or None."""
    x = np.asarray(x, dtype=np.float64)
    z = x
    if w is not None:
        z = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)
    return rotate(z, cos, sin, interleaved)


def norm_rope_backward(dy, x, w, cos, sin, interleaved=False, eps=1e-6):
    """(dx, dw) of sum(y * dy); dw is None without weights."""
    g = rotate(np.asarray(dy, dtype=np.float64), cos, -sin, interleaved)
    if w is None:
        return g, None
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    h = g * np.asarray(w, dtype=np.float64)
    dx = r * h - x * (r ** 3 / d) * np.sum(h * x, axis=-1, keepdims=True)
    dw = np.sum((g * x * r).reshape(-1, d), axis=0)
    return dx, dw


def e4m3_values():
    """The value of each of the 256 codes (bias 7, no infinities, 0x7f and 0xff NaN)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = np.nan
        out[c] = -v if c & 128 else v
    return out


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:127]  # codes 0 .. 126 in increasing order


def to_e4m3(x):
    """Nearest e4m3 code of each value (ties to the even code, saturating); NaN -> 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=E4M3_MAX, neginf=-E4M3_MAX)), E4M3_MAX)
    hi = np.clip(np.searchsorted(_POSITIVE, mag), 0, 126)
    lo = np.maximum(hi - 1, 0)
    d_hi, d_lo = _POSITIVE[hi] - mag, mag - _POSITIVE[lo]
    code = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code = np.where(np.signbit(x), code | 128, code).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(0x7F), code)


def from_e4m3(code):
    return _VALUES[np.asarray(code, dtype=np.uint8)]


def page_scale(amax):
    """The smallest 2^e with amax <= 448 * 2^e, e held to [MIN_EXP, MAX_EXP]."""
    e = MIN_EXP
    while e < MAX_EXP and amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def cache_append(x, code, scale, table, lens, counts):
    """Write the last counts[b] of lens[b] tokens, x [B, Hkv, n, d], into copies of the
    pool: code uint8 [pages, Hkv, page, d], scale [pages, Hkv]. Returns (code, scale)."""
    code, scale = np.array(code), np.array(scale, dtype=np.float64)
    page = code.shape[2]
    for b in range(x.shape[0]):
        start = int(lens[b]) - int(counts[b])
        for p in range(start // page, -(-int(lens[b]) // page)):
            lo, hi = max(start, p * page), min(int(lens[b]), (p + 1) * page)
            if lo >= hi:
                continue
            pid = int(table[b, p])
            held = lo - p * page  # tokens the page already has
            for h in range(code.shape[1]):
                rows = np.asarray(x[b, h, lo - start:hi - start], dtype=np.float64)
                finite = np.abs(rows[np.isfinite(rows)])
                s = page_scale(finite.max() if finite.size else 0.0)
                if held:
                    s = max(s, scale[pid, h])
                    if s > scale[pid, h]:
                        code[pid, h, :held] = to_e4m3(from_e4m3(code[pid, h, :held]) * (scale[pid, h] / s))
                scale[pid, h] = s
                code[pid, h, held:held + hi - lo] = to_e4m3(np.where(np.isfinite(rows), rows / s, np.nan))
    return code, scale


def cache_rows(code, scale, table, n):
    """The n rows one sequence's page list holds: float64 [Hkv, n, d]."""
    page, Hkv, d = code.shape[2], code.shape[1], code.shape[3]
    out = np.empty((Hkv, n, d))
    for p in range(-(-n // page)):
        m = min(page, n - p * page)
        pid = int(table[p])
        out[:, p * page:p * page + m] = from_e4m3(code[pid, :, :m]) * np.asarray(scale[pid], np.float64)[:, None, None]
    return out


def cache_attention(q, kc, ks, vc, vs, table, lens, counts, causal, scale):
    """Attention of q [B, Hq, Nq, d] over the cache; query i < counts[b] stands at position
    lens[b] - counts[b] + i. Returns (O, L); rows >= counts[b] are NaN, a row
    that sees no key has O = 0 and L = -inf."""
    B, Hq, Nq, d = q.shape
    g = Hq // kc.shape[1]
    o = np.full((B, Hq, Nq, d), np.nan)
    lse = np.full((B, Hq, Nq), np.nan)
    for b in range(B):
        n, c = int(lens[b]), int(counts[b])
        k, v = (cache_rows(x, s, table[b], n) for x, s in ((kc, ks), (vc, vs)))
        for h in range(Hq):
            for i in range(c):
                m = max(0, min(n, n - c + i + 1)) if causal else n
                if m == 0:
                    o[b, h, i], lse[b, h, i] = 0.0, -np.inf
                    continue
                t = scale * (k[h // g, :m] @ np.asarray(q[b, h, i], dtype=np.float64))
                top = t.max()
                e = np.exp(t - top)
                o[b, h, i] = (e / e.sum()) @ v[h // g, :m]
                lse[b, h, i] = top + np.log(e.sum())
    return o, lse
