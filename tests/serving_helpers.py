"""Shared by the tests of the serving operators: paged caches with poisoned unused
rows, 64-bit references written from the formulas, and the tolerances.

Tolerances, half a rounding step being finfo.eps / 2 (bf16 2^-8, fp32 2^-24, e4m3 2^-4):

  rotation    two fp32 products and a sum of values of at most |a| + |b|, a cosine and
              a sine off by at most 2^-22 (argument, function and amplitude in fp32):
              2^-21 * A (|a| + |b|), and half a step of the result's type
  attention   z = scale q.k sums d fp32 products: |dz| <= e = (d + 4) 2^-24 scale |q|.|k|
              (the tensor core may truncate: twice that); weights and their sum move by a
              factor within 1 +- 2 (2 e) + 2^-20 (the exponential, the sums); each weight is
              rounded to bf16 (2^-8), so with W = sum_s w_s |v_s| / sum_s w_s:
              |do| <= (2^-8 + 4 e + 2^-18) W + 2^-8 |o| (the result's own rounding)
              |dlse| <= 2 e + 2^-20 + 2^-23 |lse|
"""
import math

import numpy as np
import torch

BF16 = 2.0 ** -8


class Cache:
    """Key and value pools [n_pages, page, Hkv, d] (bf16) holding the sequences' rows in a
    random page order; every other row holds NaN, every other table entry -1."""

    def __init__(self, lens, Hkv, d, page, seed, device="cuda", spare=3, width=0):
        rng = np.random.Generator(np.random.PCG64(seed))
        nb = [-(-n // page) for n in lens]
        self.n_pages, self.page = sum(nb) + spare, page
        width = max(max(nb + [1]), width)
        perm = rng.permutation(self.n_pages).astype(np.int32)
        table = np.full((len(lens), width), -1, dtype=np.int32)
        g = torch.Generator().manual_seed(seed)
        kp = torch.full((self.n_pages, page, Hkv, d), float("nan"), dtype=torch.bfloat16)
        vp = kp.clone()
        self.K, self.V = [], []
        o = 0
        for b, n in enumerate(lens):
            ids = perm[o:o + nb[b]]
            table[b, :nb[b]] = ids
            o += nb[b]
            k = torch.randn((n, Hkv, d), generator=g).to(torch.bfloat16)
            v = torch.randn((n, Hkv, d), generator=g).to(torch.bfloat16)
            self.K.append(k)
            self.V.append(v)
            for i, pg in enumerate(ids):
                m = min(page, n - i * page)
                kp[pg, :m] = k[i * page:i * page + m]
                vp[pg, :m] = v[i * page:i * page + m]
        self.table = torch.from_numpy(table).to(device)
        self.k_pages, self.v_pages = kp.to(device), vp.to(device)


def attention_row(q, K, V, scale):
    """One query head q [d] over its visible keys K, V [n, d] (64 bits): the result, its
    log-sum, and the tolerances of both."""
    d = q.numel()
    if K.shape[0] == 0:
        return torch.zeros(d, dtype=torch.float64), -math.inf, torch.zeros(d, dtype=torch.float64), 0.0
    z = (K @ q) * scale
    e = 2 * (d + 4) * 2.0 ** -24 * scale * float((K.abs() @ q.abs()).max())
    lse = torch.logsumexp(z, 0)
    w = torch.exp(z - lse)
    o = w @ V
    W = w @ V.abs()
    tol = (BF16 + 4 * e + 2.0 ** -18) * W + BF16 * o.abs()
    return o, float(lse), tol, 2 * e + 2.0 ** -20 + 2.0 ** -23 * abs(float(lse))


def check_rows(out, lse, rows, Q, cache, seqs, sees, G, scale):
    """Every (row t, head h) of `rows` against attention_row over the keys sees(t)."""
    out, Qd = out.double().cpu(), Q.double().cpu()
    lse = None if lse is None else lse.double().cpu()
    for t in rows:
        keys = sees(t)
        b = seqs[t]
        for h in range(Q.shape[1]):
            K = cache.K[b][keys, h // G].double()
            V = cache.V[b][keys, h // G].double()
            o, l, tol, tl = attention_row(Qd[t, h], K, V, scale)
            bad = (out[t, h] - o).abs() > tol
            assert not bad.any() and not torch.isnan(out[t, h]).any(), (
                f"row {t} head {h}: {int(bad.sum())} of {bad.numel()} off, worst "
                f"{float(((out[t, h] - o).abs() - tol).max())}")
            if lse is not None:
                got = float(lse[t, h])
                assert got == l or abs(got - l) <= tl, f"row {t} head {h}: lse {got} against {l}"


def rotated(x, positions, inv_freq, offset, interleaved, amplitude, transpose=False):
    """The rotation of x [n, H, d] in 64 bits (numpy), and |a| + |b| of each element's pair."""
    x = np.asarray(x, dtype=np.float64)
    y, mag = x.copy(), np.abs(x)
    half = len(inv_freq)
    sign = -1.0 if transpose else 1.0
    for i in range(half):
        ia, ib = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + half + i)
        phi = np.asarray(positions, dtype=np.float64) * float(inv_freq[i])
        c, s = amplitude * np.cos(phi)[:, None], sign * amplitude * np.sin(phi)[:, None]
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
        mag[..., ia] = mag[..., ib] = abs(amplitude) * (np.abs(a) + np.abs(b))
    return y, mag
