"""Plain float64 forms of the packed prefill attention and of the paged cache
operators, written from their definitions, and the tolerances of the GPU tests.

bf16 values are passed as float64 arrays that hold them exactly.  The paged
cache is a ``Pool``: numpy arrays in the layout of kvc_paged_cache.

Tolerances.  A bf16 rounding is off by at most 2^-8 of the value, an fp32 one
by 2^-24.  The logit scale * sum_c q_c k_c is accumulated in fp32 over d
products (exact from bf16); an accumulation step may truncate (2^-23), so its
error is at most
    E = (d + 4) 2^-23 scale sum_c |q_c| |k_c|  +  2^-22 |s|
(the last term: the products with scale * log2(e)), and a probability, formed
with ex2.approx (2^-22) against a log-sum-exp with the same error, is off by at
most 2 E + 2^-20 of itself.  The sums over keys add at most 2^-20 (pairwise and
tiled sums of positive terms).  With A = sum_j p_j |v_j| (the size of the
terms of an output):
    prefill:  |out - ref| <= (2^-8 + 2 E + 2^-19) A + 2^-8 |out|   (P and out rounded to bf16; |out| <= 1.01 A)
    decode:   |out - ref| <= (2^-23 + 2 E + 2^-19) A               (P as three bf16 terms: 24 bits)
    lse:      |lse - ref| <= E + 2^-20 + 2^-23 |lse|
    weights:  |w - ref|   <= (2 E + 2^-19) sum_h p + 2^-24 G |w|
E is taken as its largest value over the keys of a row.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np


@dataclass
class Rows:
    """Attention of one query row over its visible keys, with error sizes."""
    out: np.ndarray
    lse: float
    p: np.ndarray
    size: np.ndarray  # A per output element
    E: float


def attend(q, k, v, scale) -> Rows:
    """q [d], k and v [n][d], float64; n may be 0."""
    if k.shape[0] == 0:
        return Rows(np.zeros(v.shape[1]), -math.inf, np.zeros(0), np.zeros(v.shape[1]), 0.0)
    s = scale * (k @ q)
    m = s.max()
    z = m + math.log(np.exp(s - m).sum())
    p = np.exp(s - z)
    absn = scale * (np.abs(k) @ np.abs(q))
    E = float((q.shape[0] + 4) * 2.0 ** -23 * absn.max() + 2.0 ** -22 * np.abs(s).max())
    return Rows(p @ v, z, p, p @ np.abs(v), E)


def prefill_varlen(q, k, v, cu_q, cu_k, scale):
    """out, lse, and the tolerances of both, [total_q][H](...)."""
    Tq, H, d = q.shape
    G = H // k.shape[1]
    out = np.zeros((Tq, H, d))
    lse = np.zeros((Tq, H))
    tol, tol_lse = np.zeros_like(out), np.zeros_like(lse)
    for b in range(len(cu_q) - 1):
        lq, lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(lq):
            n = max(0, min(lk, i + lk - lq + 1))
            for h in range(H):
                ks = slice(cu_k[b], cu_k[b] + n)
                r = attend(q[cu_q[b] + i, h], k[ks, h // G], v[ks, h // G], scale)
                out[cu_q[b] + i, h], lse[cu_q[b] + i, h] = r.out, r.lse
                tol[cu_q[b] + i, h] = (2.0 ** -8 + 2 * r.E + 2.0 ** -19) * r.size + 2.0 ** -8 * 1.01 * r.size
                tol_lse[cu_q[b] + i, h] = r.E + 2.0 ** -20 + (2.0 ** -23 * abs(r.lse) if n else 0.0)
    return out, lse, tol, tol_lse


@dataclass
class Pool:
    k: np.ndarray        # [P][Hkv][page][d], any dtype (bits or float64)
    v: np.ndarray
    weights: np.ndarray  # [P][Hkv][page] float32
    pos: np.ndarray      # int32
    table: np.ndarray    # [B][max_pages]
    seq_lens: np.ndarray
    next_pos: np.ndarray

    @property
    def page(self):
        return self.k.shape[2]

    def at(self, b, g, slots):
        """Index of slots of sequence b, head g in k, v, weights and pos."""
        slots = np.asarray(slots, dtype=np.int64)
        return self.table[b, slots // self.page], g, slots % self.page


def paged_decode(pool: Pool, q, scale):
    """q [B][H][d] -> out, lse, weight additions [B][Hkv] lists, tolerances."""
    B, H, d = q.shape
    Hkv = pool.k.shape[1]
    G = H // Hkv
    out, lse = np.zeros((B, H, d)), np.zeros((B, H))
    tol, tol_lse = np.zeros((B, H, d)), np.zeros((B, H))
    add, tol_add = {}, {}
    for b in range(B):
        n = int(pool.seq_lens[b])
        for g in range(Hkv):
            at = pool.at(b, g, np.arange(n))
            k, v = pool.k[at], pool.v[at]
            w, tw = np.zeros(n), np.zeros(n)
            for h in range(g * G, (g + 1) * G):
                r = attend(q[b, h], k, v, scale)
                out[b, h], lse[b, h] = r.out, r.lse
                tol[b, h] = (2.0 ** -23 + 2 * r.E + 2.0 ** -19) * r.size
                tol_lse[b, h] = r.E + 2.0 ** -20 + (2.0 ** -23 * abs(r.lse) if n else 0.0)
                w += r.p
                tw += (2 * r.E + 2.0 ** -19) * r.p
            add[b, g], tol_add[b, g] = w, tw
    return out, lse, add, tol, tol_lse, tol_add


def append(pool: Pool, k, v, cu, idx=None, scores=None) -> None:
    """k, v [T][Hkv][d] in the pool's own representation."""
    Hkv = k.shape[1]
    for b in range(len(cu) - 1):
        n = int(cu[b + 1] - cu[b])
        kept = n if idx is None else min(n, idx.shape[2])
        for g in range(Hkv):
            t = np.arange(kept) if idx is None else idx[b, g, :kept].astype(np.int64)
            at = pool.at(b, g, pool.seq_lens[b] + np.arange(kept))
            pool.k[at], pool.v[at] = k[cu[b] + t, g], v[cu[b] + t, g]
            pool.pos[at] = pool.next_pos[b] + t
            pool.weights[at] = 0.0 if scores is None else scores[g, cu[b] + t]
        pool.seq_lens[b] += kept
        pool.next_pos[b] += n


def evict(pool: Pool, budget: int, recent: int) -> None:
    Hkv = pool.k.shape[1]
    for b in range(len(pool.seq_lens)):
        n = int(pool.seq_lens[b])
        if n <= budget:
            continue
        for g in range(Hkv):
            at = pool.at(b, g, np.arange(n))
            w, pos = pool.weights[at].astype(np.float64), pool.pos[at]

            def rank(s):
                new = recent > 0 and pos[s] >= pool.next_pos[b] - recent
                low = math.isnan(w[s])
                return (0 if new else 2 if low else 1, 0.0 if new or low else -w[s], s)

            kept = set(sorted(range(n), key=rank)[:budget])
            give = [s for s in range(budget) if s not in kept]
            take = [s for s in range(budget, n) if s in kept]
            assert len(give) == len(take)
            to, of = pool.at(b, g, give), pool.at(b, g, take)
            for x in (pool.k, pool.v, pool.weights, pool.pos):
                x[to] = x[of]
        pool.seq_lens[b] = budget
