"""Inputs, calls and error bounds shared by the tests of prompts, windows with sinks and four-bit caches."""

import numpy as np
import torch

from oracle import streams as O

from long_context_helpers import TORCH, f64, make_tables

BAD = 1 << 28  # a block id outside every pool


def pools_16(nb, H, bs, D, dtype, rng):
    """(device tensor, 64-bit pool) of K and of V."""
    res = []
    for _ in range(2):
        t = torch.from_numpy(rng.standard_normal((nb, H, bs, D))).to(TORCH[dtype])
        res.append([t.cuda(), f64(t)])
    return res


def pools_4(nb, H, bs, D, rng):
    """((codes, scales), 64-bit pool) of K and of V, of random codes and scales between 2^-4 and 2."""
    res = []
    for _ in range(2):
        c = rng.integers(0, 256, (nb, H, bs, D // 2)).astype(np.uint8)
        s = rng.integers(24, 64, (nb, H, bs, D // 16)).astype(np.uint8)
        res.append([(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()), O.values_fp4(c, s)])
    return res


def hide_unseen(pools, tables, lens, new, bs, window, sinks):
    """Rows that no new token sees get NaN and infinities, and table entries of blocks nobody sees a bad id."""
    tables = tables.copy()
    for i, (n, m) in enumerate(zip(lens, new)):
        if n < 1 or n < m or m < 1:
            continue
        seen = O.visible(np.arange(n - m, n), -(-n // bs) * bs, window, sinks).any(0).reshape(-1, bs)
        for b, rows in enumerate(seen):
            where = torch.from_numpy(np.nonzero(~rows)[0])
            for t, host in pools:
                t[int(tables[i, b]), :, where.cuda()] = float("nan") if b % 2 else float("inf")
                host[int(tables[i, b]), :, where.numpy()] = np.nan if b % 2 else np.inf
            if not rows.any():
                tables[i, b] = BAD
    return tables


def tolerance(ref, mass, size, D, n, scale, weight_dtype, out_dtype, vmax=0.0):
    """Bound of |out - ref| for every output, with M = sum p |v| (`mass`) and S = the query's largest sum |q k|:
    a score is a sum of D products in fp32, each addition off by at most 2^-23 of what is summed (tensor cores cut), so
    off by (D + 4) 2^-23 |scale| S, and a weight and the denominator by twice that; the hardware's exp2 and the scaling to
    log2 units add 2^-20; the weight's own rounding for the second product half a step of its type (where it is kept in
    two f16 parts, the second scaled by 2^11: 2^-21, and for weights below 2^-25 of the largest one 2^-47 of that, for each
    of n values of at most vmax); sums over n rows add 2^-23 for each 8 of them, and 64 for joins; the result's rounding half a
    step of its type."""
    dx = (D + 4) * 2.0 ** -23 * abs(scale) * size[..., None]
    part = 2.0 ** -21 if weight_dtype is None else torch.finfo(weight_dtype).eps / 2
    tol = (4 * dx + 2.0 ** -20 + part + (n / 8 + 64) * 2.0 ** -23) * mass + n * 2.0 ** -47 * vmax
    if out_dtype != torch.float32:
        tol = tol + torch.finfo(out_dtype).eps / 2 * np.abs(ref) * (1 + 2 ** -7) + float(torch.finfo(out_dtype).tiny)
    return tol + 1e-30


def close(out, ref, tol, what=""):
    """Equal where ref is not finite, within tol elsewhere."""
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(out), np.isnan(ref)), what + " NaN differ"
    inf = np.isinf(ref)
    assert np.array_equal(out[inf], ref[inf]), what + " infinities differ"
    err = np.abs(out - np.where(fine, ref, 0))[fine] / tol[fine]
    assert err.size == 0 or err.max() <= 1, f"{what} error {err.max():.3g} times the bound"


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Prompt:
    """A ragged batch: `new` tokens of sequences with `rows` rows each."""

    def __init__(self, new, rows, Hq, H, D, bs, dtype, window=None, sinks=0, seed=0, garbage=True, pad=3):
        rng = np.random.default_rng(seed)
        self.new, self.rows, self.H, self.D, self.bs = new, rows, H, D, bs
        self.window, self.sinks, self.dtype = window, sinks, TORCH[dtype]
        self.tables, nb, _ = make_tables(rows, bs, 2, rng)
        self.pools = pools_16(nb, H, bs, D, dtype, rng)
        if garbage:
            self.tables = hide_unseen(self.pools, self.tables, rows, new, bs, window, sinks)
        self.starts = [0]
        for m in new:
            self.starts.append(self.starts[-1] + m)
        T = self.starts[-1] + pad  # rows behind the last sequence
        self.q = torch.from_numpy(1.5 * rng.standard_normal((T, Hq, D))).to(self.dtype).cuda()
        self.out = torch.full((T, Hq, D), 7.0, dtype=self.dtype, device="cuda")
        self.scale = D ** -0.5

    def device(self):
        return torch.from_numpy(self.tables).cuda(), int32(self.starts), int32(self.rows)

    def workspace(self, kvc):
        return kvc.new_prompt_workspace(len(self.new), len(self.q), self.q.shape[1], self.H, self.D, self.bs,
                                        self.tables.shape[1])

    def run(self, kvc, workspace=None, stream=None):
        tables, starts, rows = self.device()
        ws = self.workspace(kvc) if workspace is None else workspace
        kvc.prompt_attention(self.q, self.pools[0][0], self.pools[1][0], tables, starts, rows, self.scale, self.out,
                             ws, window=self.window, sinks=self.sinks, stream=stream)
        torch.cuda.synchronize()
        return self.out

    def check(self, skip=()):
        out = f64(self.out)
        for i, (m, n) in enumerate(zip(self.new, self.rows)):
            if m == 0 or i in skip:
                continue
            at = slice(self.starts[i], self.starts[i] + m)
            ref, mass, size = O.attend(f64(self.q[at]), self.pools[0][1], self.pools[1][1], self.tables[i], n,
                                       self.scale, self.window, self.sinks)
            close(out[at], ref, tolerance(ref, mass, size, self.D, n, self.scale, self.dtype, self.dtype),
                  f"sequence {i}")
        assert (out[self.starts[-1]:] == 7.0).all()  # left as they were


class Decode:
    """The newest T tokens of every sequence over a 16-bit ("bf16", "f16") or four-bit ("fp4") cache."""

    def __init__(self, lens, T, Hq, H, D, bs, kind, window=None, sinks=0, seed=0, garbage=True, q_dtype="bf16",
                 out_dtype=torch.float32):
        rng = np.random.default_rng(seed)
        self.lens, self.T, self.H, self.D, self.bs, self.kind = lens, T, H, D, bs, kind
        self.window, self.sinks = window, sinks
        self.tables, nb, _ = make_tables(lens, bs, 2, rng)
        if kind == "fp4":
            self.pools = pools_4(nb, H, bs, D, rng)
            if garbage:  # any code of rows and any scale of rows that nobody sees, the scales' NaN among them
                fake = [[s.float(), np.zeros(s.shape)] for (_, s), _ in self.pools]
                for f, ((_, s), _) in zip(fake, self.pools):
                    tables = hide_unseen([f], self.tables, lens, [T] * len(lens), bs, window, sinks)
                    s[~torch.isfinite(f[0])] = 0x7f
                self.tables = tables
                for (_, s), host in self.pools:
                    host[np.repeat(s.cpu().numpy() == 0x7f, 16, -1)] = np.nan
        else:
            q_dtype = kind
            self.pools = pools_16(nb, H, bs, D, kind, rng)
            if garbage:
                self.tables = hide_unseen(self.pools, self.tables, lens, [T] * len(lens), bs, window, sinks)
        self.q = torch.from_numpy(1.5 * rng.standard_normal((len(lens), T, Hq, D))).to(TORCH[q_dtype]).cuda()
        self.out = torch.full(self.q.shape, 7.0, dtype=out_dtype, device="cuda")
        self.scale = D ** -0.5

    def workspace(self, kvc):
        return kvc.new_scored_workspace(len(self.lens), self.T, self.q.shape[2], self.H, self.D, self.bs,
                                        self.tables.shape[1], scored=False)

    def call(self, kvc, tables, lens, ws, stream=None):
        (k, _), (v, _) = self.pools
        if self.kind == "fp4":
            kvc.decode_attention_fp4(self.q, k[0], v[0], k[1], v[1], tables, lens, self.scale, self.out, ws,
                                     window=self.window, sinks=self.sinks, stream=stream)
        else:
            kvc.decode_attention_sinks(self.q, k, v, tables, lens, self.scale, self.window, self.sinks, self.out, ws,
                                       stream=stream)

    def run(self, kvc, workspace=None, stream=None):
        ws = self.workspace(kvc) if workspace is None else workspace
        self.call(kvc, torch.from_numpy(self.tables).cuda(), int32(self.lens), ws, stream)
        torch.cuda.synchronize()
        return self.out

    def check(self, skip=()):
        out = f64(self.out)
        for i, n in enumerate(self.lens):
            if i in skip:
                continue
            ref, mass, size = O.attend(f64(self.q[i]), self.pools[0][1], self.pools[1][1], self.tables[i], n,
                                       self.scale, self.window, self.sinks)
            V = self.pools[1][1]
            close(out[i], ref, tolerance(ref, mass, size, self.D, n, self.scale, None, self.out.dtype,
                                         float(np.abs(V[np.isfinite(V)]).max())), f"sequence {i}")
