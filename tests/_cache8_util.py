"""Cases and error bounds of the 8-bit cache's tests.

Bounds (u = 2^-24, half a step of fp32).  The cache's numbers are exact.  A
score sums d_h + r products: each addition is off by 2 u of the running sum of
magnitudes at most (the tensor cores cut), the sums of the parts add 16/15 of
that and a few roundings, p = q B^K is a sum of d_h products in fp32:
  2 u (d_h + 3 r + 24) (sum |q k| + sum |p| |z|).
A number x enters as e4m3 parts, each leaving a 16th of what was left, or 2^-10
in its own units where that is more.  q (8 bits, four parts, its largest
magnitude in [128, 256)) is exact but for 2^-22 / 128 of the largest; p (six
parts) leaves 2^-24 of itself, or 2^-30 / 128 of the largest:
  2^-29 max|q| sum |k| + 2^-24 sum |p| |z| + 2^-37 max|p| sum |z|.
A probability enters the value products, times its block's scale over a power
of two within a factor of two of the tile's largest, as six parts: off by 2^-24
of itself and by 2^-37 of the largest scale of its tile at most.
"""
import numpy as np
import torch

import _budget_util as T
from compressed_cache_decode_gb300 import inputs, lrkv
from oracle import lrkv_oracle as O

U = T.U
NAMES = lrkv.Cache8.NAMES


def pack(x):
    """(e4m3 numbers, scales) of rows x [B, L, heads, width] (fp64), blocks filled from row 0 on."""
    B, L, H, W = x.shape
    pad = -L % O.BLOCK8
    blocks = np.concatenate([x, np.zeros((B, pad, H, W))], axis=1).reshape(B, (L + pad) // O.BLOCK8, O.BLOCK8, H, W)
    top = np.abs(blocks).max(axis=(2, 4)) if W else np.zeros(blocks.shape[:2] + (H,))
    m, e = np.frexp(top)
    scale = np.where(top > 0, np.exp2(np.maximum(np.where(m <= 0.875, e - 9, e - 8), -126).astype(float)), 2.0 ** -126)
    v = O.e4m3_round(blocks / scale[:, :, None, :, None]).reshape(B, L + pad, H, W)[:, :L]
    return v, scale


def to8(v):
    return torch.from_numpy(np.asarray(v)).to(torch.float32).to(torch.float8_e4m3fn)


class Case:
    """A decode case whose cache is in 8 bits: numbers and scales [B, L, heads,
    width], [B, blocks, heads] (shared rows: one head) and what they stand for."""

    def __init__(self, B, H, dh, r, L, lens, seed=0, q_scale=1.0, scales=None):
        self.B, self.H, self.dh, self.r, self.L, self.lens = B, H, dh, r, L, list(lens)
        c = inputs.random_decode_case(seed=seed, batch=B, heads=H, head_dim=dh, rank=max(r, 1), max_len=L,
                                      dtype="bf16", lens=self.lens, q_scale=q_scale)
        if r == 0:
            for n in ("z_k", "z_v", "b_k", "b_v"):
                c[n] = c[n][..., :0].contiguous()
        self.c, self.values, self.scales = c, {}, {}
        for n in ("k_s", "v_s", "z_k", "z_v"):
            x = T.f64(c[n])
            x = x[:, :, None] if n.endswith("s") else x
            self.values[n], self.scales[n] = pack(x)
            if scales is not None:   # other scales: the cache then stands for other numbers
                self.scales[n] = scales(self.scales[n], n)

    def rows(self, n):
        """fp64 rows [B, L, heads, width] that the cache stands for."""
        s = np.repeat(self.scales[n], O.BLOCK8, axis=1)[:, :self.L]
        return self.values[n] * s[..., None]

    def reference(self, b, h, scale=None, keep=None):
        """(out, lse, bounds of both) of one sequence and head; keep: rows whose block has a page (others read zero)."""
        L, c = self.lens[b], self.c
        scale = self.dh ** -0.5 if scale is None else scale
        q, Bk, Bv = T.f64(c["q"][b, h]), T.f64(c["b_k"])[h], T.f64(c["b_v"])[h]
        ks, vs = self.rows("k_s")[b, :L, 0], self.rows("v_s")[b, :L, 0]
        zk, zv = (self.rows(n)[b, :L, h] if self.r else np.zeros((L, 0)) for n in ("z_k", "z_v"))
        if keep is not None:
            ks, vs, zk, zv = (np.where(keep[:L, None], x, 0) for x in (ks, vs, zk, zv))
        s = scale * ((ks + zk @ Bk.T) @ q)
        p = np.abs(q) @ np.abs(Bk)
        qk, pz, z = np.abs(ks) @ np.abs(q), np.abs(zk) @ p, np.abs(zk).sum(1)
        err = (2 * U * (self.dh + 3 * self.r + 24) * (qk + pz) + 2.0 ** -29 * np.abs(q).max() * np.abs(ks).sum(1)
               + 2.0 ** -24 * pz + 2.0 ** -37 * (p.max() if self.r else 0.0) * z) * scale
        lse = s.max() + np.log(np.exp(s - s.max()).sum())
        w, a = T.weight_bound(s[None], np.array([lse]), err[None])
        V = vs + zv @ Bv.T
        mag = np.abs(vs) + np.abs(zv) @ np.abs(Bv).T
        # 2^-37 of the largest scale of a row's tile, times the largest e4m3 number
        floor = np.zeros(self.dh)
        for t in range(0, L, 128):
            blocks = slice(t // 16, -(-min(L, t + 128) // 16))
            top = [self.scales["v_s"][b, blocks].max(), self.scales["z_v"][b, blocks, h].max() if self.r else 0.0]
            n = min(L, t + 128) - t
            floor += 2.0 ** -37 * n * 448 * (top[0] + top[1] * np.abs(Bv).sum(1))
        out_err = (w + a[0] * (2.0 ** -24 + 2 * U * (L + 128))) @ mag + floor
        return a[0] @ V, lse, out_err, err.max() + (abs(lse) + 4 + L) * 2 * U

    def cuda(self, page=0, seed=0, garbage=True):
        """(q, Cache8, b_k, b_v, lens, block_table) on the device; what no call may read holds NaN."""
        B, L, lens = self.B, self.L, self.lens
        table, lead, where = None, (B, L), None
        if page:
            used = [(b, j) for b in range(B) for j in range(L // page) if j * page < lens[b]]
            pages = len(used) + 3
            perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
            table = torch.full((B, L // page), 2 ** 30, dtype=torch.int32)
            for k, (b, j) in enumerate(used):
                table[b, j] = perm[k]
            lead, where = (pages, page), (used, perm)
        held = {}
        for n in ("k_s", "v_s", "z_k", "z_v"):
            v, s = to8(self.values[n]), torch.from_numpy(self.scales[n]).float()
            if garbage:
                for b in range(B):
                    v.view(torch.uint8)[b, lens[b]:] = 0x7f
                    s[b, -(-lens[b] // 16):] = float("nan")
            if where:
                used, perm = where
                pv = torch.full((lead[0], page) + tuple(v.shape[2:]), 0xff, dtype=torch.uint8).view(torch.float8_e4m3fn)
                ps = torch.full((lead[0], page // 16, v.shape[2]), float("inf"))
                for k, (b, j) in enumerate(used):
                    pv.view(torch.uint8)[perm[k]] = v.view(torch.uint8)[b, j * page:(j + 1) * page]
                    ps[perm[k]] = s[b, j * page // 16:(j + 1) * page // 16]
                v, s = pv, ps
            if n.endswith("s"):
                v, s = v[:, :, 0], s[:, :, 0]
            held[n], held[n + "_scale"] = v.contiguous().cuda(), s.contiguous().cuda()
        if self.r == 0:
            held.update({n: None for n in ("z_k", "z_v", "z_k_scale", "z_v_scale")})
        c = self.c
        return (c["q"].cuda(), lrkv.Cache8(**held), c["b_k"].cuda(), c["b_v"].cuda(), c["seq_lens"].cuda(),
                None if table is None else table.cuda())

    def check(self, out, lse, scale=None, pairs=None, keep=None):
        out, lse = T.f64(out), T.f64(lse)
        worst = 0.0
        for b in range(self.B):
            if self.lens[b] == 0:
                assert np.all(out[b] == 0) and np.all(lse[b] == -np.inf)
                continue
            for h in range(self.H):
                if pairs is not None and (b, h) not in pairs:
                    continue
                o, l, oe, le = self.reference(b, h, scale, None if keep is None else keep[b])
                assert abs(lse[b, h] - l) <= le, (b, h, lse[b, h], l, le)
                off = np.abs(out[b, h] - o)
                assert np.all(off <= oe), (b, h, int(np.argmax(off - oe)), off.max(), oe.max())
                worst = max(worst, float((off / oe).max()))
        return worst
