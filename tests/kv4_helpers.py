"""Shared helpers for the tests of the rotary positions and the 4-bit cache."""
import numpy as np

import oracle.kv4 as o
from helpers import to_dev, to_host

HALF = 2.0 ** -24     # half a step of fp32, relative


def random_pages(rng, n, P, n_kv, hd):
    """Pages of uniform codes and scales of 8 bits of either sign."""
    pages = np.empty((n, n_kv, 2, P * (hd // 2 + hd // 16)), np.uint8)
    code = P * hd // 2
    pages[..., :code] = rng.integers(0, 256, (n, n_kv, 2, code), dtype=np.uint8)
    d = rng.integers(128, 256, (n, n_kv, 2, P * hd // 32)) * 2.0 ** rng.integers(-11, -8, (n, n_kv, 2, P * hd // 32))
    d *= rng.choice([-1.0, 1.0], d.shape)
    pages[..., code:] = np.ascontiguousarray(d.astype(np.float16)).view(np.uint8)
    return pages.reshape(n, -1)


class Batch:
    """A ragged batch over a filled cache: lens[b] tokens of which n[b] are
    rows; pages in random order, spare ones among them."""

    def __init__(self, seed, n, lens, P, n_kv, hd, uniform=False):
        rng = self.rng = np.random.default_rng([4004, seed])
        self.n, self.P, self.n_kv, self.hd = list(n), P, n_kv, hd
        self.lens = np.array(lens, np.int32)
        per = max(1, -(-max(max(lens), 1) // P))
        n_pages = per * len(lens) + 2
        self.table = rng.permutation(n_pages)[: per * len(lens)].reshape(len(lens), per).astype(np.int32)
        self.pages = random_pages(rng, n_pages, P, n_kv, hd)
        self.q_start = None if uniform else np.concatenate(([0], np.cumsum(n))).astype(np.int32)
        self.n_tok = int(sum(n))

    def cache(self, gq):
        return gq.KV4Cache(to_dev(self.pages), to_dev(self.table), self.P, self.n_kv, self.hd)

    def dev(self):
        return to_dev(self.lens), None if self.q_start is None else to_dev(self.q_start)

    def sequence(self, b, pages=None):
        return o.sequence(self.pages if pages is None else pages, self.table, b, int(self.lens[b]), self.P, self.n_kv,
                          self.hd)


def attention_bound(mag, big, vmax, keys, hd):
    """How far fp32-accurate attention may be from the formula, per channel.

    A score is a sum of hd products: q in two fp16 parts is off by 2^-22 of
    each, the fp32 sum by at most (hd + 16) half steps of their sum's
    magnitude `big` (16: the row's scale, the two parts' order, the exponent's
    argument); a weight's relative error is the score's, twice (itself and
    against the maximum), 2^-20 for the exponential, 2^-22 for its two fp16
    parts. The weighted sum adds a half step per key and the total another;
    weights too small for fp16's steps add 2^-25 each against a total of at
    least 1. Numerator and total both carry the weights' error.
    """
    score = big * (2.0 ** -22 + (hd + 16) * HALF)
    weight = 2 * score + 2.0 ** -20 + 2.0 ** -22
    return mag * (2 * weight + 2 * (keys + 16) * HALF) + keys * 2.0 ** -24 * vmax


def check_attention(batch, out, q, scale, causal, window, pages=None, rows=None):
    """out [n_tok, heads, hd] against the oracle, row by row (all, or `rows`)."""
    where = o.rows(batch.q_start, batch.lens, batch.n_tok)
    kv = {}
    worst = 0.0
    for t in range(batch.n_tok) if rows is None else rows:
        b, pos = where[t]
        if b not in kv:
            kv[b] = batch.sequence(b, pages)
        K, V = kv[b]
        want, mag, big = o.attention(q[t], pos, int(batch.lens[b]), K, V, scale, causal, window)
        got = out[t].astype(np.float64)
        bad = np.isnan(want)
        assert np.array_equal(np.isnan(got), bad), f"row {t}: NaN in other places"
        tol = attention_bound(mag, big[:, None], np.nanmax(np.abs(V)) if V.size else 0.0, len(K), batch.hd)
        err = np.abs(got - want)
        assert (err <= tol)[~bad].all(), f"row {t}: {np.nanmax(err / np.maximum(tol, 1e-300))} of the bound"
        if (~bad).any() and tol.any():
            worst = max(worst, float((err / np.maximum(tol, 1e-300))[~bad].max()))
    return worst


__all__ = ["HALF", "Batch", "attention_bound", "check_attention", "random_pages", "to_dev", "to_host", "o"]
