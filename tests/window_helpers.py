"""Cases of windowed attention over a bf16 or e4m3 paged cache, the float64 answers and the
error bounds they are held to.

Every cache row that no query of a sequence sees is poisoned (bf16 NaN; the NaN code with
scale byte 255), and every block-table entry of a block without a visible key is an
impossible block id, so that reading either shows.

Bounds.  Let u(t) = finfo(t).eps / 2 and `mass` = sum_j p_j |v_jd|, n the visible keys.
  scores: a float32 product of D terms, each operation (in the tensor cores, truncating) off
    by at most 2^-23 relative, the fp16 query of the e4m3 path off by 2^-25 of its largest
    element per element (|q|max * sum|k| <= D * that row's share, bounded by
    2^-25 * qmax * kabs), multiplied by the scale: ds = (D + 8) * 2^-23 * spread + that;
    the exponent's argument and ex2.approx add less than 2^-20 + 2^-22 * |s - max| with
    weights below 2^-30 of no weight: + 2^-17;
  weights: rounded to `weight_bits` significant bits: 2^-weight_bits relative;
  sums over n keys in float32: n * 2^-23 relative to the mass;
  output: bf16, u = 2^-8 relative.
An output is off by at most 2^-8 |o| + (2 ds + 2^-weight_bits + n 2^-23) * mass, the lse by
ds + n 2^-23 + 2^-22 * (1 + |lse|).
"""

from __future__ import annotations

import math

import numpy as np
import torch

from oracle.paged_attention import bf16_to_f64
from oracle.window_attention import attend, dequantise_rows, gather, quantise_rows, seen
from synth.device import bf16_tensor, i32
from synth.workloads import POISON_BF16, bf16_bits_from_f32

BAD_IDS = (-1, 1 << 30, -(1 << 31))
ROW_BITS = {False: 16, True: 11}     # weight bits of the few-row kernel: bf16 / e4m3 cache
TILE_BITS = 8                        # weights rounded to bf16 by the 128-row kernel


class Case:
    def __init__(self, seed, lens, news, hq=4, hkv=2, d=64, bs=16, fp8=True, window=0, sinks=0,
                 q_mult=1.0, scale=None, spread_scales=False, extra_rows=0):
        rng = np.random.default_rng(seed)
        self.lens, self.news = list(lens), list(news)
        self.hq, self.hkv, self.d, self.bs, self.fp8 = hq, hkv, d, bs, fp8
        self.window, self.sinks = window, sinks
        self.scale = 1.0 / math.sqrt(d) if scale is None else scale
        need = [max(1, -(-n // bs)) for n in lens]
        self.num_blocks = sum(need) + 3
        order = rng.permutation(self.num_blocks)
        self.tables = np.full((len(lens), max(need)), -1, np.int64)
        at = 0
        for b, k in enumerate(need):
            self.tables[b, :k] = order[at:at + k]
            at += k
        rows = (self.num_blocks, bs, hkv, d)
        kv = rng.standard_normal((2,) + rows).astype(np.float32)
        if spread_scales:     # rows of very different size
            kv *= np.exp2(rng.integers(-30, 30, size=(2,) + rows[:3])).astype(np.float32)[..., None]
            kv[0] = np.clip(kv[0], -8, 8)
        self.kv_bits = bf16_bits_from_f32(kv).reshape((2,) + rows)
        if fp8:
            self.codes, self.scales = quantise_rows(self.kv_bits)
            self.values = dequantise_rows(self.codes, self.scales)
        else:
            self.values = bf16_to_f64(self.kv_bits)
        self.total = sum(news)
        q = rng.standard_normal((self.total + extra_rows, hq, d)).astype(np.float32) * np.float32(q_mult)
        self.q = bf16_bits_from_f32(q).reshape(q.shape)
        self.cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        # what must not be read
        live = np.zeros((self.num_blocks, bs), bool)
        self.device_tables = self.tables.copy()
        for b, (n, m) in enumerate(zip(lens, news)):
            vis = np.zeros(n, bool)
            for p in range(n - m, n):
                vis |= seen(n, p, window, sinks)
            for j in np.nonzero(vis)[0]:
                live[self.tables[b, j // bs], j % bs] = True
            for j in range(self.tables.shape[1]):
                if not vis[j * bs:(j + 1) * bs].any():
                    self.device_tables[b, j] = BAD_IDS[(b + j) % 3]
        self.live = live

    def device(self, dev):
        t = dict(q=bf16_tensor(self.q, dev), tables=i32(self.device_tables, dev), cu=i32(self.cu, dev),
                 lens=i32(np.asarray(self.lens), dev))
        dead = ~self.live
        for i, x in enumerate("kv"):
            if self.fp8:
                codes, scales = self.codes[i].copy(), self.scales[i].copy()
                codes[dead] = 0x7F
                scales[dead] = 255
                t[x + "_cache"] = torch.from_numpy(codes).to(dev).view(torch.float8_e4m3fn)
                t[x + "_scales"] = torch.from_numpy(np.ascontiguousarray(scales.transpose(0, 2, 1))).to(dev)
            else:
                bits = self.kv_bits[i].copy()
                bits[dead] = POISON_BF16
                t[x + "_cache"] = bf16_tensor(bits, dev)
                t[x + "_scales"] = None
        return t

    def answers(self):
        """(out, lse, out bound without the weights' rounding, mass, lse bound) of all rows."""
        parts = []
        q = bf16_to_f64(self.q)
        for b, (n, m) in enumerate(zip(self.lens, self.news)):
            k = gather(self.values[0], self.tables[b], n, self.bs)
            v = gather(self.values[1], self.tables[b], n, self.bs)
            qb = q[self.cu[b]:self.cu[b + 1]]
            out, lse, mass, spread = attend(qb, k, v, np.arange(n - m, n), self.window, self.sinks, self.scale)
            nvis = n if self.window == 0 else min(n, self.window + self.sinks + m)
            ds = (self.d + 8) * 2.0 ** -23 * spread + 2.0 ** -17
            if self.fp8 and n:
                kabs = np.abs(k).sum(-1).max(0)                                # [Hkv]
                ds = ds + 2.0 ** -25 * abs(self.scale) * np.abs(qb).max(-1) * \
                    np.repeat(kabs, self.hq // self.hkv)[None, :]
            fin = np.where(np.isfinite(lse), lse, 0.0)
            parts.append((out, lse, 2.0 ** -8 * np.abs(out) + (2 * ds + nvis * 2.0 ** -23)[..., None] * mass,
                          mass, ds + nvis * 2.0 ** -23 + 2.0 ** -22 * (1 + np.abs(fin))))
        return [np.concatenate(x) for x in zip(*parts)]


def check_answers(case, out, lse, weight_bits, what, rows=None):
    o, l, ob, mass, lb = case.answers()
    got = out.detach().double().cpu().numpy()[:case.total]
    gl = lse.detach().double().cpu().numpy()[:case.total]
    bound = ob + 2.0 ** -weight_bits * mass + 1e-30
    bad = ~(np.abs(got - o) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outputs off, first at {i}: "
                             f"{got[i]} for {o[i]}, bound {bound[i]}")
    both = np.isneginf(gl) & np.isneginf(l)
    with np.errstate(invalid="ignore"):
        badl = ~(both | (np.abs(gl - l) <= lb))
    if badl.any():
        i = tuple(np.argwhere(badl)[0])
        raise AssertionError(f"{what}: lse off at {i}: {gl[i]} for {l[i]}, bound {lb[i]}")
