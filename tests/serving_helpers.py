"""Batches over a 4-bit cache for the tests: built on the CPU by the oracle's quantiser."""
import numpy as np
import torch

from oracle import serving_ref as ref
from rope_attention_fwd_b200 import binding as rb

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def pack_pages(x, d):
    """x [pages, H, blocks, 16, d] float32 -> uint8 [pages, H, blocks, half a block's bytes]."""
    codes, step, lo = ref.quantise(x)
    c = (codes[..., 0::2] | (codes[..., 1::2] << 4))
    p = np.ascontiguousarray(np.stack([step, lo], -1)).view(np.uint8)
    return np.concatenate([c.reshape(x.shape[:3] + (-1,)), p.reshape(x.shape[:3] + (-1,))], -1)


class Batch:
    """lens: (new tokens, cached tokens in all) of every sequence.  What no sequence caches holds
    0xFF bytes: the pairs there are NaN."""

    def __init__(self, lens, Hq, Hkv, d, page, dtype, seed=0, causal=True, window=0, extra=0,
                 q_scale=1.0, v_scale=1.0, max_q=0, scale=0.0, spare=2):
        g = np.random.default_rng(seed)
        self.lens, self.Hq, self.Hkv, self.d, self.page = lens, Hq, Hkv, d, page
        self.dtype, self.causal, self.window = DT[dtype], causal, window
        need = [-(-L // page) for _, L in lens]
        pages = sum(need) + spare
        ids = g.permutation(pages)
        self.table = np.full((len(lens), max(max(need), 1)), 0, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        blocks = page // 16
        shape = (pages, Hkv, blocks, 16, d)
        gain = np.exp(0.3 * g.standard_normal((Hkv, 1, 1, d)))
        k = (g.standard_normal(shape) * gain).astype(np.float32)
        v = (v_scale * g.standard_normal(shape)).astype(np.float32)
        self.cache = np.concatenate([pack_pages(k, d), pack_pages(v, d)], -1)
        half = self.cache.shape[-1] // 2
        used = np.zeros((pages, page), bool)
        for b, (_, L) in enumerate(lens):
            for p in range(L):
                used[self.table[b, p // page], p % page] = True
        for p, t in zip(*np.nonzero(~used)):
            blk, row = t // 16, t % 16
            for h0 in (0, half):
                part = self.cache[p, :, blk, h0:h0 + half]
                part[:, row * d // 2:(row + 1) * d // 2] = 0xFF
                w = 4 * d // 64
                part[:, 8 * d + row * w:8 * d + (row + 1) * w] = 0xFF
        self.indptr = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        self.kv_len = np.array([L for _, L in lens], np.int32)
        self.T = int(self.indptr[-1]) + extra
        q = q_scale * torch.from_numpy(g.standard_normal((self.T, Hq, d))).float()
        self.q = q.to(self.dtype)
        self.scale = scale
        self.plan = rb.cache_plan(len(lens), self.T, Hq, Hkv, d, self.dtype, pages, page,
                                  self.table.shape[1], causal=causal, window=window, max_q=max_q,
                                  scale=scale)

    def device(self):
        self.c = {k: torch.from_numpy(getattr(self, k)).cuda()
                  for k in ("cache", "table", "indptr", "kv_len")}
        self.c["q"] = self.q.cuda()
        self.c["ws"] = rb.cache_workspace(self.plan, "cuda")
        return self

    @property
    def head(self):
        c = self.c
        return self.plan, c["cache"], c["table"], c["indptr"], c["kv_len"]

    def attn(self, **kw):
        return rb.rope_attn_cache_attn(*self.head, self.c["q"], ws=self.c["ws"], **kw)

    def status(self):
        return rb.rope_attn_device_status(self.c["ws"])

    def rows(self):
        """k, v [Hkv, L, d] float64 of every sequence."""
        kk, vv = ref.unpack_cache(self.cache, self.d)
        return [tuple(ref.sequence_rows(x, self.table[b], L, self.page) for x in (kk, vv))
                for b, (_, L) in enumerate(self.lens)]

    def check(self, o, lse, q=None, rows=None, skip=(), label=""):
        """Every row against the float64 oracle.  Tolerance of an element, U = 2^-24:
          stored type: half a step of |o|;
          a score: fp32 products and sums over d channels and the two affine terms of each
            group, at most (d + 16) U scale sum |q| (|k| + the 8 steps that the codes may be moved
            by) =: ds, which moves p by 2 ds relative (numerator and sum).  (Where the codes
            enter as 0..15, the terms are 15 steps + |lo|, at most 3 |k|, with some 16
            roundings: (d + 16) 2.07 is more than 16 x 3.);
          exp2 and the sums of p: 2^-20 relative (2 ulp of ex2.approx, rescales, sums of at
            most 2^11 terms per lane and step in fp32);
          bf16, more than 64 rows per kv head: p and v are rounded to fp16 (2^-11 each; below 2^-14
            by at most 2^-25 absolute);
          bf16, up to 64 rows: p step is rounded to fp16 (2^-11 relative, 2^-25 below 2^-14) and
            multiplies codes of -8..7 (0..15, and -8 by the same operand): 8 step (2^-11 +
            L 2^-25 / step) at most, with step <= 2 vmax / 15; the fp32 sums of the products may
            lose 2^-23 of themselves with each 16 keys of a warp.  A warp has every fourth 32
            keys; its sums hold 8 step of all its keys, and 15 step and -8 step of the last 128:
            (L / 64 + 2) 2^-23 (8 + 15 + 8) step, below L / 16 2^-23 8 step + 2^-17 step.
        All of it relative to sum_j p_j |v_j|; lse moves by ds + 2^-20 and its own rounding."""
        U, bf = 2.0 ** -24, self.dtype == torch.bfloat16
        q = self.q.double().numpy() if q is None else q
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        scale = self.scale or self.d ** -0.5
        worst = 0.0
        for b, (n, L) in enumerate(self.lens):
            if b in skip:
                continue
            k, v = (rows or self._rows())[b]
            at = slice(int(self.indptr[b]), int(self.indptr[b]) + n)
            wo, wl, mag = ref.attention(q[at], k, v, scale, self.causal, self.window)
            kmax = np.nanmax(abs(k)) if k.size and not np.isnan(k).all() else 0.0
            q1 = abs(q[at]).sum(-1)
            ds = ((self.d + 16) * U * scale * q1 * kmax * (1 + 16 / 15))[..., None]
            vmax = np.nanmax(abs(v)) if v.size and not np.isnan(v).all() else 0.0
            tol = torch.finfo(self.dtype).eps / 2 * abs(wo) + (2 * ds + 2.0 ** -20) * mag + 1e-30
            if bf and n * (self.Hq // self.Hkv) > 64:
                tol = tol + 2 * 2.0 ** -11 * mag * 1.01 + L * 2.0 ** -25 * vmax + 2.0 ** -25
            elif bf:
                step = 2 * vmax / 15 * 1.01
                tol = tol + 8 * step * (2.0 ** -11 + L / 16 * 2.0 ** -23 + 2.0 ** -20)
                tol = tol + 8 * L * 2.0 ** -25
            err = abs(o[at] - wo)
            assert np.isfinite(o[at]).all(), (label, b)
            assert (err <= tol).all(), (label, b, float((err / tol).max()))
            worst = max(worst, float((err / tol).max()) if err.size else 0.0)
            empty = np.isinf(wl)
            assert (np.isneginf(lse[at]) == empty).all() and (o[at][empty] == 0).all(), (label, b)
            el = abs(lse[at][~empty] - wl[~empty])
            tl = (ds[..., 0] + 2.0 ** -19 + 2 * U * abs(np.where(empty, 0, wl)))[~empty]
            if bf:
                tl = tl + L * 2.0 ** -25
            assert (el <= tl).all(), (label, b, float((el / tl).max()))
        return worst

    def _rows(self):
        if not hasattr(self, "_cached_rows"):
            self._cached_rows = self.rows()
        return self._cached_rows
