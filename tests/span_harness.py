"""Shared by the tests of the 4-bit caches and the windowed attention: paged
caches whose unused slots hold NaN patterns, the oracle's answers, and the
tolerances.

Tolerances, from the roundings (half a step is 2^-8 of a bf16 value, 2^-11 of an
f16 one), with A = sum p |z| / sum p of the row and column:
* the output's rounding to bf16:                  2^-8 |ref|
* the weights' rounding before the product with the latents: 2^-11 A over E4M3
  and 4-bit caches (f16), 2^-8 A for bf16 prompts, 2^-16 A for bf16 tokens
  (roundings and remainders), taken as w A below
* fp32 arithmetic: a weight is 2^x with x = score * log2(e) / sqrt(d) - reference
  known to some 4 * 2^-24 * (|x| + |reference|), and sums over up to a few
  thousand terms: (2^-20 (1 + X) + 2^-18) A with X the row's largest
  |score * log2(e)|
* weights below 2^-14 of the reference's are f16 subnormals, whose half step is
  2^-25 whatever their size.  The reference never exceeds the row's maximum (it
  starts as the maximum of the row's first step and only follows larger ones), so
  the row's largest weight is at least 1 and the weights' sum l at least 1: the
  terms' errors add up to at most sum 2^-25 |z| / l <= 2^-25 S, S = sum |z| over
  the row's tokens (over E4M3 and 4-bit caches)
"""
from __future__ import annotations

import numpy as np
import torch

import sparse_decode_attention_basiskv_b200 as bkv
from oracle import span_oracle as SO

FMT_WEIGHT = {"bf16_token": 2.0 ** -16, "bf16_prompt": 2.0 ** -8, "e4m3": 2.0 ** -11,
              "4bit": 2.0 ** -11}


def dims_of(B, Hq, Hkv, d, r_v, r_k, page, max_pages, phys, **kw):
    return bkv.Dims(B=B, Hq=Hq, Hkv=Hkv, d=d, hidden=128, r_v=r_v, r_k=r_k, page_size=page,
                    max_pages_per_seq=max_pages, num_phys_pages=phys, **kw)


class Paged:
    """Rows of one kind (width w) of every sequence in a paged cache of a format;
    slots without a row hold NaN patterns (4 bits: bytes 0xff)."""

    def __init__(self, rows, fmt, page, table, phys, lead=None):
        # rows: list over sequences of float64 [T][Hkv][w]
        self.fmt, self.page = fmt, page
        Hkv, w = rows[0].shape[1:]
        lead = w if lead is None else lead
        if fmt == "4bit":
            buf = np.full((phys, Hkv, page * w // 16 * 9), 0xFF, dtype=np.uint8)
        else:
            buf = np.full((phys, Hkv, page, w), np.nan)
        self.values = []
        for b, x in enumerate(rows):
            vals = np.zeros_like(x)
            for p in range(-(-x.shape[0] // page)):
                blk = x[p * page:(p + 1) * page]
                n = blk.shape[0]
                for g in range(Hkv):
                    if fmt == "4bit":
                        full = np.zeros((page, w))
                        full[:n] = blk[:, g]
                        t = SO.pack_tile(full)
                        codes, sc = t[:page * w // 2].reshape(page, -1), t[page * w // 2:].reshape(page, -1)
                        dst = buf[table[b, p], g]
                        dst[:page * w // 2].reshape(page, -1)[:n] = codes[:n]
                        dst[page * w // 2:].reshape(page, -1)[:n] = sc[:n]
                        vals[p * page:p * page + n, g] = SO.unpack_tile(t, page, w)[:n]
                    else:
                        buf[table[b, p], g, :n] = blk[:, g]
            self.values.append(vals)
        if fmt == "4bit":
            self.tensor = torch.from_numpy(buf)
        else:
            t = torch.from_numpy(buf)
            if fmt == "e4m3":
                q = t.clamp(-448, 448).to(torch.float8_e4m3fn)
            else:
                q = t.to(torch.bfloat16)
            back = q.to(torch.float64)
            for b, x in enumerate(rows):
                tok = np.arange(x.shape[0])
                self.values[b] = back[torch.from_numpy(table[b, tok // page].astype(np.int64)), :,
                                      torch.from_numpy(tok % page)].numpy().reshape(x.shape)
            if lead < w:  # a narrow router's tiles: [S][lead], then [S][w - lead]
                q = torch.cat([q[..., :lead].reshape(phys, Hkv, -1),
                               q[..., lead:].reshape(phys, Hkv, -1)], -1).reshape(q.shape)
            self.tensor = q.view(torch.uint8) if fmt == "e4m3" else q
        self.tensor = self.tensor.contiguous().cuda()


def table_of(rng, B, max_pages, phys):
    assert phys >= B * max_pages
    return rng.permutation(phys)[:B * max_pages].reshape(B, max_pages).astype(np.int32)


def bf16(x):
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16)


def reference(q, K, Z, see):
    """(a, A, (X, S)) of one KV head's rows: q [n][d] float64, see [n][T]."""
    a, A, S = (np.zeros((q.shape[0], Z.shape[1])) for _ in range(3))
    X = np.zeros(q.shape[0])
    for i in range(q.shape[0]):
        t = np.flatnonzero(see[i])
        if len(t) == 0:
            continue
        s = K[t] @ q[i] / np.sqrt(q.shape[1])
        p = np.exp(s - s.max())
        p /= p.sum()
        a[i], A[i] = p @ Z[t], p @ np.abs(Z[t])
        X[i] = np.abs(s).max() * 1.4427
        S[i] = np.abs(Z[t]).sum(0)
    return a, A, (X, S)


def assert_rows(got, a, A, X, w, what=""):
    X, S = X
    bound = 2.0 ** -8 * np.abs(a) + (w + 2.0 ** -20 * (1 + X[:, None]) + 2.0 ** -18) * A
    if w == FMT_WEIGHT["4bit"]:
        bound = bound + 2.0 ** -25 * S
    err = np.abs(got - a)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} values off, worst "
                           f"{np.nanmax(err - bound):.3e} above its bound; row "
                           f"{np.argwhere(bad)[0].tolist()}")


def random_rows(rng, lens, Hkv, w, scale=1.0):
    return [rng.standard_normal((L, Hkv, w)) * scale for L in lens]
