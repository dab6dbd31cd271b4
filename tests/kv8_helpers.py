"""Caches, oracle results and tolerances for the tests of the 8-bit cache operators.

Tolerances of the attention outputs (per head and dimension, from the arithmetic alone):

* a score x = (q . k) a / sqrt(d): products of 8-bit values with the fp16 parts of q are
  exact; an fp32 query loses at most 2^-22 of each element in its two fp16 parts; 8 chained
  fp32 sums of 16 products each may drop up to 2 units of 2^-23 of the largest partial sum,
  which sum_i |q_i k_i| bounds; factor and scale round 3 times at 2^-24.  So
  |dx| <= 20 * 2^-23 * S with S = max_j a_j sum_i |q_i k_ij| / sqrt(d);
* p = 2^.. / l and the value sum: a score error changes p by a factor e^(2 dx) against its
  normalisation; the exponential has 2 units of 2^-22, the two fp16 parts of a term 2^-22,
  and sums over n keys chain at most n / 128 + 8 terms per warp (2 units each) and a few
  for the merges.  So |dout| <= (40 * 2^-23 * S + (64 + n / 32) * 2^-23) * sum_j p_j |v_j|;
* a position's weight: the same factor on p, the stored score's own rounding (2^-24 of |x| <= S
  log2(e), twice), and one rounding of the sum.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import kv8_ref as ref

D = 128
U = 2.0 ** -23
QT = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def to_bytes(stored, fmt):
    """Format values (float64) as a torch tensor of the format (exact)."""
    return torch.from_numpy(np.ascontiguousarray(stored, dtype=np.float32)).to(QT[fmt])


def as_values(t):
    """An 8-bit tensor's format values as float64."""
    return t.cpu().to(torch.float32).double().numpy()


def quantise(x, block, fmt, pow2=True):
    """x [..., L, d] float64 -> (stored values, scales [..., L / block])."""
    y = x.reshape(*x.shape[:-2], -1, block * D)
    s = ref.block_scale(np.abs(y).max(-1), fmt)
    if not pow2:                                     # scales as another quantiser writes them
        s = np.maximum(np.abs(y).max(-1) / ref.FMAX[fmt], 1e-30).astype(np.float32).astype(np.float64)
    return ref.round8(y / s[..., None], fmt).reshape(x.shape), s


class Case:
    """A cache on CPU (float64 format values and scales) and its upload, contiguous or paged."""

    def __init__(self, B, Hkv, L, fmt="e4m3", block=16, page=0, seed=0, spread=2, pow2=True, amp=1.0,
                 codes=False, empty=False, spare=3):
        self.rng = rng = np.random.default_rng(seed)
        self.B, self.Hkv, self.fmt, self.block, self.page = B, Hkv, fmt, block, page
        unit = max(block, page)
        self.L = L
        self.cap = cap = -(-L // unit) * unit
        parts = []
        for _ in "kv":
            x = rng.standard_normal((B, Hkv, cap, D)) * amp
            x[..., rng.choice(D, 4, replace=False)] *= 10
            x *= np.exp2(rng.integers(-spread, spread + 1, (B, Hkv, cap // block, 1))).repeat(block, 2)
            if empty:
                x[:] = 0
            parts.append(quantise(x, block, fmt, pow2))
        (self.k, self.ks), (self.v, self.vs) = parts
        self.codes = np.zeros((B, Hkv, cap, 32), np.uint8) if codes else None
        self.table = None
        if page:
            nb = cap // page
            self.num_pages = B * nb + spare
            self.table = rng.permutation(self.num_pages)[:B * nb].reshape(B, nb).astype(np.int32)

    def values(self):
        f = lambda x, s: (x.reshape(self.B, self.Hkv, -1, self.block, D)  # noqa: E731
                          * s[..., None, None]).reshape(x.shape)
        return f(self.k, self.ks), f(self.v, self.vs)

    def _pages(self, x, per, fill):
        """[B, Hkv, n, ...] -> pages [P, Hkv, per, ...]."""
        B, H = x.shape[:2]
        out = np.full((self.num_pages, H, per, *x.shape[3:]), fill, x.dtype)
        y = x.reshape(B, H, -1, per, *x.shape[3:])
        for b in range(B):
            for j, p in enumerate(self.table[b]):
                out[p] = y[b, :, j]
        return out

    def _seq(self, pages):
        B, nb = self.table.shape
        y = pages[self.table]                        # [B, nb, H, per, ...]
        y = np.moveaxis(y, 2, 1)
        return y.reshape(B, y.shape[1], nb * y.shape[3], *y.shape[4:])

    def upload(self, ad, device="cuda", max_seq_len=None):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
        ts = []
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            s = s.astype(np.float32)
            if self.page:
                x, s = self._pages(x, self.page, 0.0), self._pages(s, self.page // self.block, 1.0)
            ts.append((to_bytes(x, self.fmt).to(device), dev(s)))
        codes = None
        if self.codes is not None:
            codes = dev(self._pages(self.codes, self.page, 0) if self.page else self.codes)
        table = dev(self.table) if self.page else None
        (k, ks), (v, vs) = ts
        return ad.KV8Cache(k, v, ks, vs, self.block, codes=codes, block_table=table,
                           max_seq_len=max_seq_len if self.page else None)

    def download(self, cache):
        """(k, k_scale, v, v_scale, codes) of an uploaded cache, by position."""
        seq = self._seq if self.page else (lambda x: x)
        c = None if cache.codes is None else seq(cache.codes.cpu().numpy())
        return (seq(as_values(cache.k)), seq(cache.k_scale.cpu().double().numpy()),
                seq(as_values(cache.v)), seq(cache.v_scale.cpu().double().numpy()), c)


def attention_oracle(q, c, lists):
    """q [B, Hq, d] float64, c: the Case (or (K, V, V scale per position)), lists(b, h):
    positions.  Returns out, its tolerance [B, Hq, d], weights per position [B, Hkv, L]
    and their tolerance."""
    K, V, C = (*c.values(), c.vs.repeat(c.block, 2)) if isinstance(c, Case) else c
    B, Hq, _ = q.shape
    Hkv, L = K.shape[1:3]
    out, tol = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    w, wtol = np.zeros((B, Hkv, L)), np.zeros((B, Hkv, L))
    for b in range(B):
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            pos = np.asarray(lists(b, h), dtype=np.int64)
            o, p = ref.attention(q[b, h], K[b, kv], V[b, kv], pos)
            out[b, h] = o
            if len(pos) == 0:
                continue
            S = float((np.abs(K[b, kv, pos]) @ np.abs(q[b, h])).max() / np.sqrt(D))
            rel = 40 * U * S + (64 + len(pos) / 32) * U
            pc = p * C[b, kv, pos]
            tol[b, h] = rel * (p @ np.abs(V[b, kv, pos])) + 2.0 ** -37 * pc.max() * np.sum(
                np.abs(V[b, kv, pos]) / np.maximum(C[b, kv, pos], 1e-300)[:, None], 0)
            np.add.at(w[b, kv], pos, p)
            np.add.at(wtol[b, kv], pos, p * (rel + 2 * S * U))
    return out, tol, w, wtol


def check(got, want, tol, what):
    got = got.detach().cpu().double().numpy()
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - want) / np.maximum(tol, 1e-300)
    over[np.abs(got - want) == 0] = 0
    worst = float(over.max()) if over.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} times the tolerance"
    return worst
