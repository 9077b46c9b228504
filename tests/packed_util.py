"""Packed batches for the tests, and their attention in 64 bits with what the kernels' roundings may add.

The bounds are per element and count half steps of bf16 (2^-8 of a value):
 - O = P V / l: the weights are rounded to bf16 for the product while l sums the
   unrounded ones, so an element is off by at most 2^-8 sum_j P_ij |v_jc|, and
   rounded once itself. Scores are fp32 sums of d exact products: d 2^-23 of the
   sum of absolute terms, which moves a weight by as much relative to itself
   (and the sum of the row likewise); exponentials and the fp32 sums are within 2^-18.
 - dV = P^T dO: the same rounding of P, P = exp(S - L) with the stored L (half a
   step of fp32 of |L|, 2^-24 |L|, moves a weight by as much).
 - dS = P o (dP - D), with P in fp32 and rounded to bf16: 2^-8 of |dS|, and P times
   what the fp32 sums dP and D (d terms each) are off. dQ = scale dS K, dK = scale dS^T Q.
 - The exponential returns 0 where its result is below the smallest normal fp32
   number: every weight may be off by 2^-126 more, which counts where a key has
   no larger one (its dV is then 0 instead of, say, 1e-40, as are the terms of dQ and dK).
"""

from __future__ import annotations

import numpy as np

from attn_inputs import bf16_bits_to_f64, f32_to_bf16_bits
from gpu_util import to_device

H16 = 2.0 ** -8
TINY = 2.0 ** -126


def starts(lens, lead=0):
    return np.concatenate([[lead], lead + np.cumsum(lens)]).astype(np.int32)


def randn(rng, *shape, spread=1.0):
    bits = f32_to_bf16_bits((rng.standard_normal(shape) * spread).astype(np.float32))
    return bits, bf16_bits_to_f64(bits)


class Batch:
    """q, k, v as views of one packed projection [rows, Hq + 2 Hkv, d], do, and their 64-bit values. Rows of no
    sequence hold NaN and infinities."""

    def __init__(self, lens, Hq, Hkv, d, seed, lead=0, tail=0, spread=1.5):
        import torch
        rng = np.random.default_rng(seed)
        self.lens, self.Hq, self.Hkv, self.d = list(lens), Hq, Hkv, d
        self.cu = starts(lens, lead)
        self.rows = int(self.cu[-1]) + tail
        bits, self.x = randn(rng, self.rows, Hq + 2 * Hkv, d, spread=spread)
        do_bits, self.do = randn(rng, self.rows, Hq, d)
        self.qkv, self.d_do = to_device(bits), to_device(do_bits)
        for t in (self.qkv, self.d_do):
            for part in (t[:lead], t[self.rows - tail:]):
                part[..., ::2] = float("nan")
                part[..., 1::2] = float("inf")
        self.d_cu = torch.tensor(self.cu, device="cuda")
        self.q, self.k, self.v = self.x[:, :Hq], self.x[:, Hq:Hq + Hkv], self.x[:, Hq + Hkv:]
        self.d_q, self.d_k, self.d_v = self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hkv], self.qkv[:, Hq + Hkv:]

    def sequences(self):
        return [slice(int(a), int(b)) for a, b in zip(self.cu, self.cu[1:]) if b > a]

    def held(self):
        m = np.zeros(self.rows, bool)
        m[self.cu[0]:self.cu[-1]] = True
        return m


def _weights(q, k, causal, scale):
    """Scores and the sums of their absolute terms, masked."""
    s, mag = scale * (q @ k.T), scale * (np.abs(q) @ np.abs(k).T)
    if causal:
        hide = np.triu(np.ones(s.shape, bool), 1)
        s, mag = np.where(hide, -np.inf, s), np.where(hide, 0.0, mag)
    return s, mag


def forward_ref(b, causal, scale):
    """O, L and the bounds of their errors; NaN in rows of no sequence."""
    o = np.full((b.rows, b.Hq, b.d), np.nan)
    lse = np.full((b.Hq, b.rows), np.nan)
    bo, bl = np.zeros_like(o), np.zeros_like(lse)
    g = b.Hq // b.Hkv
    for r in b.sequences():
        for h in range(b.Hq):
            s, mag = _weights(b.q[r, h], b.k[r, h // g], causal, scale)
            m = s.max(-1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(-1, keepdims=True)
            p /= l
            v = b.v[r, h // g]
            o[r, h] = p @ v
            lse[h, r] = (m + np.log(l))[:, 0]
            off = b.d * 2.0 ** -23 * mag.max(-1, keepdims=True)
            bo[r, h] = H16 * np.abs(o[r, h]) + (H16 + 2 * off + 2.0 ** -18) * (p @ np.abs(v))
            bl[h, r] = off[:, 0] + 2.0 ** -18 * (1 + np.abs(lse[h, r]))
    return o, lse, bo, bl


def backward_ref(b, o, lse, causal, scale):
    """dQ, dK, dV for the outputs o, lse that the backward pass is given, and the bounds of their errors."""
    g, d = b.Hq // b.Hkv, b.d
    dq = np.full((b.rows, b.Hq, d), np.nan)
    dk, dv = np.full((b.rows, b.Hkv, d), np.nan), np.full((b.rows, b.Hkv, d), np.nan)
    bq, bk, bv = np.zeros_like(dq), np.zeros_like(dk), np.zeros_like(dv)
    for r in b.sequences():
        dk[r] = dv[r] = 0.0
        for h in range(b.Hq):
            q, k, v, do = b.q[r, h], b.k[r, h // g], b.v[r, h // g], b.do[r, h]
            s, mag = _weights(q, k, causal, scale)
            L = lse[h, r][:, None]
            p = np.exp(s - L)
            dp, D = do @ v.T, (do * o[r, h]).sum(-1, keepdims=True)
            ds = p * (dp - D)
            rel = d * 2.0 ** -23 * mag.max(-1, keepdims=True) + 2.0 ** -23 * np.abs(L) + 2.0 ** -18  # of a weight
            off = d * 2.0 ** -23 * (np.abs(do) @ np.abs(v).T + (np.abs(do) * np.abs(o[r, h])).sum(-1, keepdims=True))
            ds_off = (H16 + rel) * np.abs(ds) + 1.01 * p * off + TINY * (1 + np.abs(dp - D))
            dq[r, h] = scale * (ds @ k)
            bq[r, h] = H16 * np.abs(dq[r, h]) + 1.01 * scale * (ds_off @ np.abs(k))
            dk[r, h // g] += scale * (ds.T @ q)
            bk[r, h // g] += 1.01 * scale * (ds_off.T @ np.abs(q))
            dv[r, h // g] += p.T @ do
            bv[r, h // g] += 1.01 * (((H16 + rel) * p + TINY).T @ np.abs(do))
        bk[r] += H16 * np.abs(dk[r])
        bv[r] += H16 * np.abs(dv[r])
    return (dq, dk, dv), (bq, bk, bv)


def within(got, ref, bound, held):
    """Largest error in units of its bound, over the rows (first dimension) of a sequence."""
    e = np.abs(got - ref)[held] / np.maximum(bound[held], TINY)
    return float(e.max()) if e.size else 0.0
