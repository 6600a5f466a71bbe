"""CPU pins of the float64 forms the serving operators are tested against:
the oracle's own attention routines, torch's, and hand-made evictions."""
import math

import numpy as np
import pytest
import torch

import workloads
from tests import paged_reference as ref


def _bits(rng, *shape):
    return workloads.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32))


def _f64(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def test_prefill_form_matches_the_oracle_and_sdpa(orc):
    rng = np.random.default_rng(3)
    n, H, Hkv, d = 37, 4, 2, 128
    q, k, v = _bits(rng, n, H, d), _bits(rng, n, Hkv, d), _bits(rng, n, Hkv, d)
    scale = 1 / math.sqrt(d)
    out, lse, tol, _ = ref.prefill_varlen(_f64(q), _f64(k), _f64(v), [0, n], [0, n], scale)
    o_out, o_lse = orc.prefill_attention(q, k, v, H, Hkv, scale)
    np.testing.assert_allclose(out, np.asarray(o_out).reshape(out.shape), atol=1e-12)
    np.testing.assert_allclose(lse, np.asarray(o_lse).reshape(lse.shape), atol=1e-12)
    assert (tol > 0).all()
    # a chunk: the last 5 positions give the same rows
    c_out, c_lse, _, _ = ref.prefill_varlen(_f64(q)[n - 5:], _f64(k), _f64(v), [0, 5], [0, n], scale)
    np.testing.assert_array_equal(c_out, out[n - 5:])
    np.testing.assert_array_equal(c_lse, lse[n - 5:])
    t = [torch.from_numpy(_f64(x)).transpose(0, 1) for x in (q, k, v)]
    sd = torch.nn.functional.scaled_dot_product_attention(t[0], t[1].repeat_interleave(2, 0), t[2].repeat_interleave(2, 0),
                                                          is_causal=True, scale=scale)
    np.testing.assert_allclose(out, sd.transpose(0, 1).numpy(), atol=1e-12)


def test_prefill_form_of_rows_without_keys():
    q, k = np.ones((3, 1, 64)), np.ones((1, 1, 64))
    out, lse, _, _ = ref.prefill_varlen(q, k, 2.0 * k, [0, 3], [0, 1], 1.0)
    assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all()
    assert (out[2] == 2).all() and lse[2, 0] == 64


def _pool(page, lens, Hkv=1, d=64, seed=0):
    rng = np.random.default_rng(seed)
    need = [-(-n // page) + 1 for n in lens]
    P = sum(need) + 1
    order = rng.permutation(P)
    table = np.zeros((len(lens), max(need)), np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (P, Hkv, page)
    return ref.Pool(rng.standard_normal(shape + (d,)), rng.standard_normal(shape + (d,)),
                    rng.random(shape).astype(np.float32), np.zeros(shape, np.int32), table,
                    np.array(lens, np.int32), np.array(lens, np.int32))


def test_decode_form_matches_the_oracle(orc):
    rng = np.random.default_rng(5)
    H, Hkv, d, n = 4, 2, 64, 45
    kb, vb, qb = _bits(rng, Hkv, n, d), _bits(rng, Hkv, n, d), _bits(rng, H, d)
    pool = _pool(16, [n], Hkv, d)
    for g in range(Hkv):
        at = pool.at(0, g, np.arange(n))
        pool.k[at], pool.v[at] = _f64(kb[g]), _f64(vb[g])
    out, lse, add, _, _, _ = ref.paged_decode(pool, _f64(qb)[None], 0.125)
    want = np.asarray(orc.decode_attention(qb, kb, vb, H, Hkv, 0.125)).reshape(H, d)
    np.testing.assert_allclose(out[0], want, atol=1e-12)
    for g in range(Hkv):  # every head of the group pays one unit of attention
        assert add[0, g].sum() == pytest.approx(2.0, abs=1e-12)


def test_evict_form_by_hand():
    pool = _pool(16, [6])
    at = pool.at(0, 0, np.arange(6))
    pool.weights[at] = [0.5, 0.1, 0.5, np.nan, 0.7, 0.0]
    pool.pos[at] = np.arange(6)
    k = pool.k[at].copy()
    ref.evict(pool, 4, 1)  # kept: 5 (recent), 4, 0, 2; given up: 1, 3
    assert pool.seq_lens[0] == 4
    np.testing.assert_array_equal(pool.pos[at][:4], [0, 4, 2, 5])
    np.testing.assert_array_equal(pool.k[at][:4], k[[0, 4, 2, 5]])


def test_evict_form_ties_keep_the_lower_slots():
    pool = _pool(16, [5])
    at = pool.at(0, 0, np.arange(5))
    pool.weights[at], pool.pos[at] = 1.0, np.arange(5)
    ref.evict(pool, 3, 0)
    np.testing.assert_array_equal(pool.pos[at][:3], [0, 1, 2])


def test_append_form_with_selected_rows():
    pool = _pool(16, [2, 0])
    k = np.arange(5, dtype=np.float64)[:, None, None] * np.ones((5, 1, 64))
    idx = np.array([[[0, 2]], [[0, 1]]], np.int32)
    ref.append(pool, k, -k, [0, 3, 5], idx, np.arange(5, dtype=np.float32)[None])
    assert list(pool.seq_lens) == [4, 2] and list(pool.next_pos) == [5, 2]
    at = pool.at(0, 0, [2, 3])
    np.testing.assert_array_equal(pool.k[at][:, 0], [0, 2])
    np.testing.assert_array_equal(pool.pos[at], [2, 4])
    np.testing.assert_array_equal(pool.weights[at], [0, 2])
