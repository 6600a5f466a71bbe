"""GPU tests of the serving operators -- packed causal prefill attention and
the paged cache (append, decode attention, eviction) -- against their float64
forms, with the tolerances derived there, at the sizes and masks where they
can go wrong, and of the errors only the device can see."""
import math

import numpy as np
import pytest
import torch

import long_context_kv_window_b200 as kvc
import workloads
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvc.lib()
    torch.cuda.set_device(0)


def _bf16(rng, *shape, scale=1.0):
    """bf16 draws: (float64 values, CUDA bfloat16 tensor)."""
    bits = workloads.f32_to_bf16_bits((scale * rng.standard_normal(shape)).astype(np.float32))
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64), workloads.torch_bf16(bits, "cuda")


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def _dev_i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _close(got, want, tol, what):
    """|got - want| <= tol; equal where the reference is not finite."""
    fine = np.isfinite(want)
    np.testing.assert_array_equal(got[~fine], want[~fine], err_msg=what)
    excess = np.abs(got[fine] - want[fine]) - tol[fine]
    assert excess.size == 0 or excess.max() <= 0, f"{what}: {excess.max()} past its tolerance"


# --------------------------------------------------------------------------- #
# packed prefill attention
# --------------------------------------------------------------------------- #
def _run_prefill(q, k, v, lq, lk, pad=0, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((q.shape[0] + pad, q.shape[1], q.shape[2]), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0] + pad, q.shape[1]), 7.0, device="cuda")
    if pad:
        q = torch.cat([q, torch.full_like(q[:1], float("nan")).expand(pad, -1, -1)])
    kvc.kvc_prefill_attention_varlen(q, k, v, _dev_i32(_cu(lq)), _dev_i32(_cu(lk)), max(lq), max(lk), out=out, lse=lse,
                                     dev_err=err, **kw)
    torch.cuda.synchronize()
    assert err.item() == 0
    return out, lse


@pytest.mark.parametrize("lq,lk,H,Hkv,d", [
    ([1], [1], 1, 1, 64),
    ([1], [1], 8, 2, 128),
    ([128], [128], 4, 1, 128),
    ([129], [129], 2, 2, 64),
    ([1, 127, 0, 128, 300, 2], [1, 127, 0, 128, 300, 2], 8, 2, 128),
    ([64, 63, 65, 1, 33], [64, 63, 65, 1, 33], 8, 2, 64),
    ([1, 5, 64, 3], [300, 5, 777, 128], 8, 2, 128),     # chunks: the last positions of longer prompts
    ([1, 5, 64, 3], [255, 129, 385, 256], 4, 2, 64),
    ([10, 140, 3, 130], [4, 0, 3, 129], 4, 2, 128),     # more queries than keys: rows without any key
    ([100, 37], [100, 401], 3, 1, 128),                 # groups that do not divide 128
    ([70, 200], [70, 200], 10, 2, 64),
    ([90, 31], [190, 31], 7, 1, 128),
    ([5, 9], [140, 9], 16, 1, 128),
    ([3, 2], [130, 2], 128, 1, 64),                     # one token per tile
    ([4], [200], 100, 1, 128),
    ([32], [3000], 8, 2, 128),                          # few rows over many keys: their keys are split over CTAs
    ([7, 40, 0, 3], [2500, 900, 10, 1], 4, 1, 64),
    ([1], [5001], 8, 2, 128),
    ([130], [2100], 5, 1, 128),
    ([600], [600], 2, 1, 64),
    ([20, 700], [5, 690], 2, 1, 128),
])
def test_prefill_varlen_matches_the_form(lq, lk, H, Hkv, d):
    rng = np.random.default_rng(sum(lq) * 131 + sum(lk) + H + d)
    q, qd = _bf16(rng, sum(lq), H, d)
    k, kd = _bf16(rng, max(1, sum(lk)), Hkv, d)
    v, vd = _bf16(rng, max(1, sum(lk)), Hkv, d)
    out, lse = _run_prefill(qd, kd, vd, lq, lk)
    w_out, w_lse, tol, tol_lse = ref.prefill_varlen(q, k, v, _cu(lq), _cu(lk), 1 / math.sqrt(d))
    _close(_np(lse), w_lse, tol_lse, "lse")
    _close(_np(out), w_out, tol, "out")


@pytest.mark.parametrize("G,d", [(1, 128), (4, 128), (4, 64), (5, 128)])
def test_prefill_varlen_reference_moves(G, d):
    """Keys whose logits climb far past the running reference, in later tiles
    and late in a tile, and rows of very different maxima."""
    rng = np.random.default_rng(G + d)
    n = 420
    q, qd = _bf16(rng, n, G, d)
    k, _ = _bf16(rng, n, 1, d)
    for j, f in ((3, 4.0), (127, 8.0), (128, 12.0), (300, 20.0), (383, 26.0), (384, 30.0), (419, 40.0)):
        k[j, 0] = f * q[(j * 7) % n, 0] / math.sqrt(d)
    k = (workloads.f32_to_bf16_bits(k.astype(np.float32)).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    kd = torch.from_numpy(k).to(torch.bfloat16).cuda()
    v, vd = _bf16(rng, n, 1, d)
    out, lse = _run_prefill(qd, kd, vd, [n], [n])
    w_out, w_lse, tol, tol_lse = ref.prefill_varlen(q, k, v, [0, n], [0, n], 1 / math.sqrt(d))
    _close(_np(lse), w_lse, tol_lse, "lse")
    _close(_np(out), w_out, tol, "out")


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_prefill_varlen_split_keys_with_non_finite_values(bad):
    rng = np.random.default_rng(19)
    lq, lk, H, d = [40], [2000], 4, 128
    q, qd = _bf16(rng, 40, H, d)
    _, kd = _bf16(rng, 2000, 1, d)
    _, vd = _bf16(rng, 2000, 1, d)
    assert kvc.prefill_varlen_workspace_size(H, 1, d, 1, 40, 40, 2000) > 0  # split
    clean, clean_lse = _run_prefill(qd, kd, vd, lq, lk)
    vd[1980, 0, 7] = bad  # position of query 20
    out, lse = _run_prefill(qd, kd, vd, lq, lk)
    assert torch.equal(lse, clean_lse) and torch.equal(out[:20], clean[:20])
    assert not torch.isfinite(out[20:, :, 7]).any()
    rest = [c for c in range(d) if c != 7]
    assert torch.equal(out[:, :, rest], clean[:, :, rest])


@pytest.mark.parametrize("n,at,G", [(700, 650, 4), (700, 130, 1), (1200, 1199, 2), (300, 299, 5)])
def test_prefill_varlen_logits_far_above_the_first_tile(n, at, G):
    """Logits hundreds above everything in the first 128 keys (the block is
    computed again with the rows' maxima); later rows see them, earlier do not."""
    rng = np.random.default_rng(n + at)
    d = 128
    q, _ = _bf16(rng, n, G, d)
    q = np.abs(q)
    k, _ = _bf16(rng, n, 1, d, scale=0.1)
    k[at, 0] = 32.0  # scale * q . k of about 32 * 0.8 * sqrt(128) = 290
    k[at // 2, 0] = -16.0
    v, vd = _bf16(rng, n, 1, d)
    qd, kd = (torch.from_numpy(x).to(torch.bfloat16).cuda() for x in (q, k))
    out, lse = _run_prefill(qd, kd, vd, [n], [n])
    w_out, w_lse, tol, tol_lse = ref.prefill_varlen(q, k, v, [0, n], [0, n], 1 / math.sqrt(d))
    assert w_lse.max() > 200
    _close(_np(lse), w_lse, tol_lse, "lse")
    _close(_np(out), w_out, tol, "out")


def test_prefill_varlen_first_keys_at_minus_infinity():
    """The first 128 logits of every row are -inf, the others far below 0: the
    later rows are those of a sequence without the first keys."""
    rng = np.random.default_rng(5)
    n, H, d = 400, 2, 128
    q, _ = _bf16(rng, n, H, d)
    q[:, :, :2] = 2.0
    k, _ = _bf16(rng, n, 1, d)
    k[:, :, :2] = 0.0
    k[128:, :, 1] = -2000.0  # logits near -4000 / sqrt(128)
    v, vd = _bf16(rng, n, 1, d)
    qd = torch.from_numpy(q).to(torch.bfloat16).cuda()
    k[:128, :, 0] = -np.inf
    kd = torch.from_numpy(k).to(torch.bfloat16).cuda()
    k = _np(kd)
    out, lse = _run_prefill(qd, kd, vd, [n], [n])
    w_out, w_lse, tol, tol_lse = ref.prefill_varlen(q[128:], k[128:], v[128:], [0, n - 128], [0, n - 128], 1 / math.sqrt(d))
    assert w_lse.max() < -300
    _close(_np(lse)[128:], w_lse, tol_lse, "lse")
    _close(_np(out)[128:], w_out, tol, "out")


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_varlen_fused_projection_views_and_rows_behind(d):
    """q, k, v as views of one [n][(H + 2 Hkv) d] projection; rows behind the
    last sequence keep what they held."""
    rng = np.random.default_rng(d)
    H, Hkv, lens = 6, 2, [40, 129, 7]
    n = sum(lens)
    x, xd = _bf16(rng, n, H + 2 * Hkv, d)
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = _dev_i32(_cu(lens))
    out = torch.full((n, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, H), 7.0, device="cuda")
    cu_short = _dev_i32(_cu(lens[:2]))  # the last sequence is left out: its rows are behind the last one
    kvc.kvc_prefill_attention_varlen(xd[:, :H], xd[:, H:H + Hkv], xd[:, H + Hkv:], cu_short, cu_short, 129, 129,
                                     out=out, lse=lse, dev_err=err)
    w_out, w_lse, tol, tol_lse = ref.prefill_varlen(q, k, v, _cu(lens), _cu(lens), 1 / math.sqrt(d))
    m = sum(lens[:2])
    assert (out[m:] == 7).all() and (lse[m:] == 7).all()
    _close(_np(lse)[:m], w_lse[:m], tol_lse[:m], "lse")
    _close(_np(out)[:m], w_out[:m], tol[:m], "out")
    kvc.kvc_prefill_attention_varlen(xd[:, :H], xd[:, H:H + Hkv], xd[:, H + Hkv:], cu, cu, 129, 129, out=out, lse=lse,
                                     dev_err=err)
    _close(_np(out), w_out, tol, "out")
    assert err.item() == 0


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("what", ["k", "v"])
def test_prefill_varlen_masked_places_may_hold_anything(what, bad):
    """A non-finite key or value changes the rows that see it and no other:
    not earlier rows of its sequence, not the neighbouring sequences."""
    rng = np.random.default_rng(17)
    lens, H, d = [70, 150, 40], 4, 128
    n, at = sum(lens), 70 + 100  # position 100 of the second sequence
    q, qd = _bf16(rng, n, H, d)
    k, kd = _bf16(rng, n, 1, d)
    v, vd = _bf16(rng, n, 1, d)
    clean, clean_lse = _run_prefill(qd, kd, vd, lens, lens)
    (kd if what == "k" else vd)[at, 0, 5] = bad
    out, lse = _run_prefill(qd, kd, vd, lens, lens)
    sees = np.zeros(n, bool)
    sees[at:70 + 150] = True
    rest = torch.from_numpy(~sees).cuda()
    assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])
    hit = out[torch.from_numpy(sees).cuda()].float()
    if what == "v":
        one = hit[:, :, 5]
        assert torch.isnan(one).all() if math.isnan(bad) else (one == bad).all()
        rest_cols = [c for c in range(d) if c != 5]
        assert torch.equal(out[:, :, rest_cols], clean[:, :, rest_cols])
        assert torch.equal(lse, clean_lse)
    elif math.isnan(bad):
        assert torch.isnan(hit).all()


def test_prefill_varlen_rows_beside_one_that_outgrows_its_reference():
    """Keys past the first tile that lift the rows behind them by far, to +inf
    among them, leave the rows before them as they were, bit for bit."""
    rng = np.random.default_rng(31)
    lens, H, d = [300], 4, 128
    q, qd = _bf16(rng, 300, H, d)
    k, kd = _bf16(rng, 300, 1, d)
    v, vd = _bf16(rng, 300, 1, d)
    clean, clean_lse = _run_prefill(qd, kd, vd, lens, lens)
    for bad in (float("inf"), 300.0):
        kd[270, 0] = bad
        out, lse = _run_prefill(qd, kd, vd, lens, lens)
        assert torch.equal(out[:270], clean[:270]) and torch.equal(lse[:270], clean_lse[:270])
        assert not torch.equal(out[270:], clean[270:])


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_varlen_more_blocks_than_sms(d):
    """A CTA computes one block after another: blocks without keys, of one key
    tile and of several, some of them computed again with the rows' maxima,
    some with infinities among their masked values.  Every sequence comes out
    as it does alone, and as defined."""
    rng = np.random.default_rng(33)
    B, H, Hkv = 90, 8, 4
    lens_k = [int(x) for x in rng.integers(0, 420, B)]
    lens_q = [int(rng.integers(0, n + 1)) if b % 3 else n for b, n in enumerate(lens_k)]
    lens_q[7], lens_k[8], lens_q[8] = lens_k[7] + 40, 0, 3  # rows that see no key
    cu_q, cu_k = np.cumsum([0] + lens_q), np.cumsum([0] + lens_k)
    q, qd = _bf16(rng, sum(lens_q), H, d)
    k, kd = _bf16(rng, sum(lens_k), Hkv, d)
    v, vd = _bf16(rng, sum(lens_k), Hkv, d)
    clean = _run_prefill(qd, kd, vd, lens_q, lens_k)
    w_out, w_lse, tol, tol_lse = ref.prefill_varlen(q, k, v, cu_q, cu_k, 1 / math.sqrt(d))
    _close(_np(clean[0]), w_out, tol, "out")
    _close(_np(clean[1]), w_lse, tol_lse, "lse")
    again = [b for b in range(B) if lens_k[b] > 200 and lens_q[b] > 150]
    assert len(again) > 10
    for b in again:
        at = cu_k[b + 1] - 20
        if b % 2:
            kd[at] = 90.0  # lifts the rows behind it by far, where q sums to more than 0
        else:
            vd[at] = float("inf")
    graph, out, lse = torch.cuda.CUDAGraph(), torch.zeros_like(clean[0]), torch.zeros_like(clean[1])
    cq, ck = _dev_i32(cu_q), _dev_i32(cu_k)
    with torch.cuda.graph(graph):
        kvc.kvc_prefill_attention_varlen(qd, kd, vd, cq, ck, max(lens_q), max(lens_k), out=out, lse=lse)
    for _ in range(3):
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            rows = slice(int(cu_q[b]), int(cu_q[b + 1]))
            if b not in again:
                assert torch.equal(out[rows], clean[0][rows]) and torch.equal(lse[rows], clean[1][rows]), b
                continue
            before = slice(int(cu_q[b]), int(cu_q[b + 1]) - 20)  # the rows that do not see the key
            assert torch.equal(out[before], clean[0][before]) and torch.equal(lse[before], clean[1][before]), b
            behind = slice(int(cu_q[b + 1]) - 20, int(cu_q[b + 1]))
            if b % 2 == 0:
                assert torch.isposinf(out[behind].float()).all() and torch.equal(lse[behind], clean[1][behind])
    hit = [b for b in again if b % 2]
    sel_q = np.concatenate([np.arange(cu_q[b], cu_q[b + 1]) for b in hit])
    sel_k = np.concatenate([np.arange(cu_k[b], cu_k[b + 1]) for b in hit])
    w_out, w_lse, tol, tol_lse = ref.prefill_varlen(
        q[sel_q], _np(kd)[sel_k], v[sel_k], np.cumsum([0] + [lens_q[b] for b in hit]),
        np.cumsum([0] + [lens_k[b] for b in hit]), 1 / math.sqrt(d))
    _close(_np(out)[sel_q], w_out, tol, "out")
    _close(_np(lse)[sel_q], w_lse, tol_lse, "lse")


def test_prefill_varlen_head_major_layout():
    """q, k, v stored [heads][n][d], seen as [n][heads][d]."""
    rng = np.random.default_rng(27)
    lens, H, Hkv, d = [150, 60], 6, 2, 64
    n = sum(lens)
    q, qd = _bf16(rng, H, n, d)
    k, kd = _bf16(rng, Hkv, n, d)
    v, vd = _bf16(rng, Hkv, n, d)
    out, lse = _run_prefill(*(x.transpose(0, 1) for x in (qd, kd, vd)), lens, lens)
    q, k, v = (x.transpose(1, 0, 2) for x in (q, k, v))
    w_out, w_lse, tol, tol_lse = ref.prefill_varlen(q, k, v, _cu(lens), _cu(lens), 1 / math.sqrt(d))
    _close(_np(lse), w_lse, tol_lse, "lse")
    _close(_np(out), w_out, tol, "out")


def test_prefill_varlen_agrees_with_the_single_sequence_call():
    rng = np.random.default_rng(23)
    n, H, Hkv, d = 1300, 8, 2, 128
    _, q = _bf16(rng, n, H, d)
    _, k = _bf16(rng, n, Hkv, d)
    v, vd = _bf16(rng, n, Hkv, d)
    one, one_lse = kvc.kvc_prefill_attention(q, k, vd)
    out, lse = _run_prefill(q, k, vd, [n], [n])
    assert (lse - one_lse).abs().max().item() < 1e-5
    # both round P and out to bf16: twice 2 * 2^-8 of the values' size
    assert (out.float() - one.float()).abs().max().item() <= 4 * 2.0 ** -8 * np.abs(v).max()
    again, lse2 = _run_prefill(q, k, vd, [n], [n])
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_varlen_long_rows_after_non_finite_memory(d):
    """Long prompts (the K/V ring goes round many times), and shared memory
    full of NaN from the call before: every row against the plain fp64 form."""
    rng = np.random.default_rng(d + 1)
    n, H = 5000, 2
    q, qd = _bf16(rng, n, H, d)
    k, kd = _bf16(rng, n, 1, d)
    v, vd = _bf16(rng, n, 1, d)
    nan = torch.full_like(vd, float("nan"))
    _run_prefill(torch.full_like(qd, float("nan")), nan, nan, [n], [n])
    out, lse = _run_prefill(qd, kd, vd, [n], [n])
    t = [torch.from_numpy(x).cuda().transpose(0, 1) for x in (q, k, v)]
    s = t[0] @ t[1].transpose(1, 2) / math.sqrt(d)
    s.masked_fill_(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -math.inf)
    z = torch.logsumexp(s, 2)
    p = (s - z[..., None]).exp()
    size = (p @ t[2].abs()).transpose(0, 1).cpu().numpy()
    # E of the module's tolerances with |q|, |k| at their largest norms
    E = (d + 4) * 2.0 ** -23 / math.sqrt(d) * np.linalg.norm(q, axis=2).max() * np.linalg.norm(k, axis=2).max() + 2e-5
    _close(_np(lse), z.t().cpu().numpy(), np.full((n, H), E + 1e-5), "lse")
    _close(_np(out), (p @ t[2]).transpose(0, 1).cpu().numpy(), (2.02 * 2.0 ** -8 + 2 * E) * size, "out")


def test_prefill_varlen_many_sequences():
    """More sequences than a warp holds, some empty, in one call."""
    rng = np.random.default_rng(29)
    lens = [int(x) for x in rng.integers(0, 40, 70)]
    q, qd = _bf16(rng, sum(lens), 4, 64)
    k, kd = _bf16(rng, sum(lens), 2, 64)
    v, vd = _bf16(rng, sum(lens), 2, 64)
    out, lse = _run_prefill(qd, kd, vd, lens, lens)
    w_out, w_lse, tol, tol_lse = ref.prefill_varlen(q, k, v, _cu(lens), _cu(lens), 0.125)
    _close(_np(lse), w_lse, tol_lse, "lse")
    _close(_np(out), w_out, tol, "out")


def test_prefill_varlen_lse_only_and_bad_seqlens():
    rng = np.random.default_rng(31)
    _, q = _bf16(rng, 60, 4, 128)
    _, k = _bf16(rng, 60, 2, 128)
    _, v = _bf16(rng, 60, 2, 128)
    full, full_lse = _run_prefill(q, k, v, [20, 40], [20, 40])
    out, lse = kvc.kvc_prefill_attention_varlen(q, k, v, _dev_i32([0, 20, 60]), _dev_i32([0, 20, 60]), 40, 40,
                                                want_out=False)
    assert out is None and torch.equal(lse, full_lse)
    # (cu, max_seqlen, rows of the sequence that is malformed or too long)
    for cu, most, bad in (([0, 30, 20], 60, slice(30, 60)), ([0, 20, 61], 60, slice(20, 60)),
                          ([-4, 20, 60], 60, slice(0, 20)), ([0, 20, 60], 39, slice(20, 60))):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((60, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        kvc.kvc_prefill_attention_varlen(q, k, v, _dev_i32(cu), _dev_i32(cu), most, most, out=out, dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == kvc.KVC_DEV_ERR_SEQLENS, cu
        assert (out[bad] == 7).all(), cu
        good = slice(0, bad.start) if bad.start else slice(bad.stop, 60)
        assert cu[1] == 30 or torch.equal(out[good], full[good]), cu


def test_prefill_varlen_without_keys_or_queries():
    q = torch.randn(5, 4, 128, device="cuda").bfloat16()
    none = torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    out, lse = _run_prefill(q, none, none, [2, 3], [0, 0])
    assert (out == 0).all() and (lse == -math.inf).all()
    k = torch.randn(4, 2, 128, device="cuda").bfloat16()
    out, lse = kvc.kvc_prefill_attention_varlen(q[:0], k, k, _dev_i32([0, 0]), _dev_i32([0, 4]), 0, 4)
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)


def test_one_index_dimensions_may_have_any_stride():
    """A size-1 token or head dimension whose stride no dense tensor has."""
    rng = np.random.default_rng(37)
    q, qd = _bf16(rng, 1, 1, 64)
    k, kd = _bf16(rng, 9, 1, 64)
    odd = torch.as_strided(qd, (1, 1, 64), (3, 5, 1))
    kodd = torch.as_strided(kd, (9, 1, 64), (64, 1, 1))
    out, lse = _run_prefill(odd, kodd, kodd, [1], [9])
    w_out, w_lse, tol, tol_lse = ref.prefill_varlen(q, k, k, [0, 1], [0, 9], 0.125)
    _close(_np(out), w_out, tol, "out")
    _close(_np(lse), w_lse, tol_lse, "lse")
    t = Paged(rng, [30], 1, 64, 16, room=4)
    out, _ = kvc.kvc_paged_decode_attention(odd, t.cache)
    _close(_np(out), ref.paged_decode(t.pool, q, 0.125)[0], ref.paged_decode(t.pool, q, 0.125)[3], "out")
    kvc.kvc_paged_append(t.cache, odd, odd, dev_err=t.err)
    ref.append(t.pool, q, q, [0, 1])
    t.check_state()


# --------------------------------------------------------------------------- #
# paged cache
# --------------------------------------------------------------------------- #
class Paged:
    """A cache on the device and its reference pool, with random entries."""

    def __init__(self, rng, lens, Hkv, d, page, room=0, fused=False, tail=0.0):
        B = len(lens)
        need = [max(1, -(-(n + room) // page)) for n in lens]
        P = sum(need) + 2
        order = rng.permutation(P)
        table = np.zeros((B, max(need)), np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        table_dev = np.where(np.arange(max(need))[None] < np.array(need)[:, None], table, -9)  # unused: no page
        shape = (P, Hkv, page)
        k, kd = _bf16(rng, *shape, d)
        v, vd = _bf16(rng, *shape, d)
        w = rng.random(shape).astype(np.float32)
        self.pool = ref.Pool(k, v, w, np.zeros(shape, np.int32), table, np.array(lens, np.int32),
                             np.array(lens, np.int32) + 3)
        for b in range(B):
            n = need[b] * page
            for g in range(Hkv):
                self.pool.pos[self.pool.at(b, g, np.arange(n))] = rng.permutation(n)
                if tail != 0.0:  # what lies behind the entries
                    behind = self.pool.at(b, g, np.arange(lens[b], n))
                    kd[behind], vd[behind] = tail, tail
        if fused:  # k and v side by side in one pool: page stride of two pages
            both = torch.empty((P, 2, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
            both[:, 0], both[:, 1] = kd, vd
            kd, vd = both[:, 0], both[:, 1]
        self.cache = kvc.PagedCache(kd, vd, _dev_i32(table_dev), _dev_i32(self.pool.seq_lens),
                                    weights=torch.from_numpy(w.copy()).cuda(), pos=_dev_i32(self.pool.pos),
                                    next_pos=_dev_i32(self.pool.next_pos))
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def check_state(self, what=""):
        """Entries, weights and positions of every held slot are the reference's, bit for bit."""
        c, p = self.cache, self.pool
        torch.cuda.synchronize()
        assert self.err.item() == 0
        np.testing.assert_array_equal(c.seq_lens.cpu().numpy(), p.seq_lens, err_msg=what)
        np.testing.assert_array_equal(c.next_pos.cpu().numpy(), p.next_pos, err_msg=what)
        k, v = _np(c.k), _np(c.v)
        w, pos = c.weights.cpu().numpy(), c.pos.cpu().numpy()
        for b, n in enumerate(p.seq_lens):
            for g in range(k.shape[1]):
                at = p.at(b, g, np.arange(n))
                np.testing.assert_array_equal(pos[at], p.pos[at], err_msg=f"{what} pos {b} {g}")
                np.testing.assert_array_equal(w[at], p.weights[at], err_msg=f"{what} weights {b} {g}")
                np.testing.assert_array_equal(k[at], p.k[at], err_msg=f"{what} k {b} {g}")
                np.testing.assert_array_equal(v[at], p.v[at], err_msg=f"{what} v {b} {g}")

    def decode(self, rng, H, accumulate, **kw):
        """One decode call against the form; returns (out, lse)."""
        c, p = self.cache, self.pool
        q, qd = _bf16(rng, len(p.seq_lens), H, c.head_dim)
        before = c.weights.clone()
        out, lse = kvc.kvc_paged_decode_attention(qd, c, accumulate=accumulate, dev_err=self.err, **kw)
        torch.cuda.synchronize()
        assert self.err.item() == 0
        w_out, w_lse, add, tol, tol_lse, tol_add = ref.paged_decode(p, q, 1 / math.sqrt(c.head_dim))
        _close(_np(lse), w_lse, tol_lse, "lse")
        _close(_np(out), w_out, tol, "out")
        if not accumulate:
            assert torch.equal(before, c.weights)
            return out, lse
        want, tol_w = before.cpu().numpy().astype(np.float64), np.zeros(before.shape)
        for (b, g), w in add.items():
            at = p.at(b, g, np.arange(len(w)))
            want[at] += w
            tol_w[at] = tol_add[b, g] + 2.0 ** -24 * (H // c.num_kv_heads + 1) * np.abs(want[at])
        _close(_np(c.weights), want, tol_w, "weights")  # entries behind the held ones: unchanged
        p.weights = c.weights.cpu().numpy().copy()
        return out, lse


DECODE = [
    ([1], 1, 1, 64, 16), ([1, 0, 15, 16, 17], 4, 2, 64, 16), ([127, 128, 129, 0, 33], 8, 2, 128, 16),
    ([63, 64, 65, 500], 6, 2, 128, 32), ([255, 256, 257], 5, 1, 128, 64), ([300, 31, 1000], 16, 2, 128, 128),
    ([513, 1], 32, 2, 128, 256), ([700, 90], 7, 1, 64, 64), ([40, 41], 8, 8, 128, 16), ([2500], 3, 3, 128, 32),
    ([1200, 77, 3], 16, 1, 64, 128), ([90] * 40, 4, 1, 64, 16),
]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("lens,H,Hkv,d,page", DECODE)
def test_paged_decode_matches_the_form(lens, H, Hkv, d, page, accumulate):
    rng = np.random.default_rng(sum(lens) + H * d + page)
    t = Paged(rng, lens, Hkv, d, page, tail=float("nan"))
    t.decode(rng, H, accumulate)
    t.decode(rng, H, accumulate)  # the workspace's counters are back at zero


@pytest.mark.parametrize("tail", [float("nan"), float("inf"), float("-inf"), 3e38])
def test_paged_decode_ignores_what_lies_behind_the_entries(tail):
    rng = np.random.default_rng(7)
    for lens, page in (([5, 130, 47], 64), ([257, 16, 1], 128)):
        Paged(rng, lens, 2, 128, page, tail=tail).decode(rng, 8, True)


@pytest.mark.parametrize("lens", [[40], [3000], [70, 900]])
def test_paged_decode_non_finite_entries(lens):
    """Values: an infinity or NaN among the entries is what the output's column
    becomes, and the other columns stay.  A NaN key makes the row NaN."""
    rng = np.random.default_rng(sum(lens))
    t = Paged(rng, lens, 2, 128, 16)
    _, q = _bf16(rng, len(lens), 8, 128)
    clean, lse = (x.clone() for x in kvc.kvc_paged_decode_attention(q, t.cache))
    for e, at, x in ((3, 7, math.inf), (9, 39, -math.inf), (12, 0, math.nan), (30, 5, math.inf), (30, 6, -math.inf)):
        page, g, slot = t.pool.at(0, 1, at)
        t.cache.v[int(page), g, int(slot), e] = x
    out, lse2 = kvc.kvc_paged_decode_attention(q, t.cache)
    assert torch.equal(lse, lse2)
    hit = out[0, 4:]
    assert (hit[:, 3] == math.inf).all() and (hit[:, 9] == -math.inf).all() and hit[:, [12, 30]].isnan().all()
    keep = [e for e in range(128) if e not in (3, 9, 12, 30)]
    assert torch.equal(hit[:, keep], clean[0, 4:][:, keep]) and torch.equal(out[0, :4], clean[0, :4])
    assert torch.equal(out[1:], clean[1:])
    page, g, slot = t.pool.at(0, 0, 11)
    t.cache.k[int(page), g, int(slot), 2] = math.nan
    out, lse2 = kvc.kvc_paged_decode_attention(q, t.cache)
    assert out[0, :4].isnan().all() and lse2[0, :4].isnan().all() and torch.equal(lse2[0, 4:], lse[0, 4:])


def test_paged_decode_views_and_bounds():
    """A fused pool (page stride of two pages), strided queries, a tight max_len."""
    rng = np.random.default_rng(9)
    t = Paged(rng, [100, 33], 2, 128, 16, fused=True)
    t.decode(rng, 8, True, max_len=100)
    q, qd = _bf16(rng, 2, 16, 128)
    out, lse = kvc.kvc_paged_decode_attention(qd[:, ::2], t.cache)
    w_out, w_lse, _, tol, tol_lse, _ = ref.paged_decode(t.pool, q[:, ::2], 1 / math.sqrt(128))
    _close(_np(out), w_out, tol, "out")
    _close(_np(lse), w_lse, tol_lse, "lse")


def test_paged_decode_large_logits():
    """Entries whose logits pass the running reference by far, late in the cache."""
    rng = np.random.default_rng(13)
    t = Paged(rng, [900, 310], 1, 128, 64)
    for b, at, f in ((0, 3, 3.0), (0, 450, 9.0), (0, 899, 30.0), (1, 0, 20.0), (1, 309, 5.0)):
        i = t.pool.at(b, 0, at)
        t.pool.k[i] = np.round(f * t.pool.k[i])  # whole numbers up to 256: exact in bf16
        t.pool.k[i] = np.clip(t.pool.k[i], -256, 256)
        t.cache.k[int(i[0]), 0, int(i[2])] = torch.from_numpy(t.pool.k[i]).to(torch.bfloat16).cuda()
    t.decode(rng, 4, True)


def test_paged_decode_shared_pages_and_one_long_sequence():
    rng = np.random.default_rng(15)
    t = Paged(rng, [64, 80], 2, 64, 16)
    t.pool.table[1, :4] = t.pool.table[0, :4]  # a shared prefix
    t.cache.block_table[1, :4] = t.cache.block_table[0, :4]
    t.decode(rng, 4, False)
    t = Paged(rng, [9001], 1, 64, 32)
    t.decode(rng, 2, True)


def test_paged_decode_is_deterministic():
    rng = np.random.default_rng(19)
    t = Paged(rng, [3000, 5, 1700], 2, 128, 16)
    _, q = _bf16(rng, 3, 8, 128)
    first = [x.clone() for x in kvc.kvc_paged_decode_attention(q, t.cache)]
    for _ in range(5):
        again = kvc.kvc_paged_decode_attention(q, t.cache)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_pages_past_the_reach_of_32_bits():
    """A pool of more than 2^32 elements: its last pages are written, read and moved within."""
    rng = np.random.default_rng(25)
    P, Hkv, page, d = 16450, 8, 128, 128
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough device memory")
    both = torch.empty((P, 2, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    assert (P - 3) * both.stride(0) > 2 ** 32
    small = Paged(rng, [0, 0], Hkv, d, page, room=250)  # the same entries in a small pool
    table = _dev_i32([[P - 1, P - 3], [P - 2, 0]])
    shape = (P, Hkv, page)
    big = kvc.PagedCache(both[:, 0], both[:, 1], table, _dev_i32([0, 0]),
                         weights=torch.zeros(shape, device="cuda"), pos=torch.zeros(shape, dtype=torch.int32, device="cuda"),
                         next_pos=_dev_i32([3, 3]))
    lens = [240, 100]
    _, k = _bf16(rng, sum(lens), Hkv, d)
    _, v = _bf16(rng, sum(lens), Hkv, d)
    sc = torch.rand((Hkv, sum(lens)), device="cuda")
    _, q = _bf16(rng, 2, 2 * Hkv, d)
    got = []
    for c in (small.cache, big):
        kvc.kvc_paged_append(c, k, v, _dev_i32(_cu(lens)), 240, scores=sc, dev_err=small.err)
        a = kvc.kvc_paged_decode_attention(q, c, max_len=256, accumulate=True, dev_err=small.err)
        kvc.kvc_paged_evict(c, 90, 10, max_len=256, dev_err=small.err)
        b = kvc.kvc_paged_decode_attention(q, c, max_len=256, dev_err=small.err)
        at = c.block_table[0, 0].long()
        got.append([*a, *b, c.k[at, :, :90], c.v[at, :, :90], c.weights[at, :, :90], c.pos[at, :, :90]])
    torch.cuda.synchronize()
    assert small.err.item() == 0
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_paged_decode_flags_bad_pages_and_lengths():
    rng = np.random.default_rng(21)
    for kind in ("page", "long", "negative"):
        t = Paged(rng, [200, 90], 2, 128, 16)
        q, qd = _bf16(rng, 2, 4, 128)
        if kind == "page":
            t.cache.block_table[0, 7] = 1 << 20
        elif kind == "long":
            t.cache.seq_lens[0] = t.cache.capacity + 1
        else:
            t.cache.seq_lens[0] = -3
        before = t.cache.weights.clone()
        out, lse = kvc.kvc_paged_decode_attention(qd, t.cache, accumulate=True, dev_err=t.err)
        torch.cuda.synchronize()
        assert t.err.item() == kvc.KVC_DEV_ERR_PAGES, kind
        assert (out[0] == 0).all() and (lse[0] == -math.inf).all(), kind
        w_out, w_lse, add, tol, tol_lse, _ = ref.paged_decode(t.pool, q, 1 / math.sqrt(128))
        _close(_np(out)[1], w_out[1], tol[1], "the other sequence")
        untouched = [int(p) for p in t.pool.table[0, :13]]
        assert torch.equal(t.cache.weights[untouched], before[untouched]), kind


@pytest.mark.parametrize("lens,held,Hkv,d,page", [
    ([1, 0, 3, 40], [0, 5, 16, 15], 2, 64, 16), ([70, 1, 200], [1, 64, 63], 8, 128, 64), ([300], [0], 1, 128, 256),
    ([33] * 40, [7] * 40, 3, 64, 32)])
def test_append_whole_prompts(lens, held, Hkv, d, page):
    rng = np.random.default_rng(sum(lens) + d)
    t = Paged(rng, held, Hkv, d, page, room=2 * max(lens))
    for scored in (False, True):
        k, kd = _bf16(rng, sum(lens), Hkv, d)
        v, vd = _bf16(rng, sum(lens), Hkv, d)
        sc = rng.random((Hkv, sum(lens))).astype(np.float32) if scored else None
        kvc.kvc_paged_append(t.cache, kd, vd, _dev_i32(_cu(lens)), max(lens), dev_err=t.err,
                             scores=None if sc is None else torch.from_numpy(sc).cuda())
        ref.append(t.pool, k, v, _cu(lens), scores=sc)
        t.check_state(f"scored {scored}")


@pytest.mark.parametrize("kk", [1, 8, 50])
def test_append_selected(kk):
    rng = np.random.default_rng(kk)
    lens, Hkv, d = [20, 100, 0, 7], 2, 128
    t = Paged(rng, [0, 3, 9, 16], Hkv, d, 16, room=kk)
    k, kd = _bf16(rng, sum(lens), Hkv + 1, d)  # strided: the pool has one head fewer
    v, vd = _bf16(rng, sum(lens), Hkv + 1, d)
    sc = rng.random((Hkv, sum(lens))).astype(np.float32)
    idx = np.full((4, Hkv, kk), -1, np.int32)
    for b, n in enumerate(lens):
        for g in range(Hkv):
            idx[b, g, :min(n, kk)] = np.sort(rng.permutation(n)[:kk])
    kvc.kvc_paged_append(t.cache, kd[:, 1:], vd[:, 1:], _dev_i32(_cu(lens)), 100, idx=_dev_i32(idx),
                         scores=torch.from_numpy(sc).cuda(), dev_err=t.err)
    ref.append(t.pool, k[:, 1:], v[:, 1:], _cu(lens), idx, sc)
    t.check_state()


def test_append_one_token_each_step():
    rng = np.random.default_rng(41)
    t = Paged(rng, [0, 15, 16, 31], 3, 64, 16, room=20)
    for step in range(20):
        k, kd = _bf16(rng, 4, 3, 64)
        v, vd = _bf16(rng, 4, 3, 64)
        kvc.kvc_paged_append(t.cache, kd, vd, dev_err=t.err)
        ref.append(t.pool, k, v, np.arange(5))
    t.check_state()


def test_append_flags_what_does_not_fit():
    rng = np.random.default_rng(43)
    _, k = _bf16(rng, 30, 1, 64)
    cases = [([0, 10, 30], kvc.KVC_DEV_ERR_PAGES, [14, 3], 20),      # the second is past its table
             ([0, 10, 5], kvc.KVC_DEV_ERR_SEQLENS, [14, 3], 20),
             ([0, 10, 30], kvc.KVC_DEV_ERR_SEQLENS, [14, 3], 19)]    # longer than max_seqlen says
    for cu, bit, lens, most in cases:
        t = Paged(rng, [4, 3], 1, 64, 16)
        t.cache.block_table[:, 0] = torch.tensor([0, 1], dtype=torch.int32)
        before = t.cache.k.clone()
        kvc.kvc_paged_append(t.cache, k, k, _dev_i32(cu), most, dev_err=t.err)
        torch.cuda.synchronize()
        assert t.err.item() == bit and t.cache.seq_lens.tolist() == lens
        assert torch.equal(t.cache.k[1], before[1]) and torch.equal(t.cache.k[0, 0, 4:14], k[:10, 0])
    t = Paged(rng, [4, 3], 1, 64, 16, room=16)
    t.cache.block_table[1, 0] = -1
    before = t.cache.k.clone()
    kvc.kvc_paged_append(t.cache, k[:2], k[:2], dev_err=t.err)
    torch.cuda.synchronize()
    assert t.err.item() == kvc.KVC_DEV_ERR_PAGES
    assert (t.cache.k != before).flatten(1).any(1).sum() == 1  # sequence 0's page alone
    t = Paged(rng, [0], 1, 64, 16, room=16)
    idx = _dev_i32([[[0, 10, -1]]])
    kvc.kvc_paged_append(t.cache, k[:10], k[:10], _dev_i32([0, 10]), 10, idx=idx, dev_err=t.err)
    torch.cuda.synchronize()
    page = int(t.pool.table[0, 0])
    assert t.err.item() == kvc.KVC_DEV_ERR_INDEX and t.cache.pos[page, 0, :3].tolist() == [3, -1, -1]
    assert (t.cache.k[page, 0, 1:3] == 0).all() and torch.equal(t.cache.k[page, 0, 0], k[0, 0])


@pytest.mark.parametrize("lens,budget,recent,page", [
    ([5, 17, 16, 0, 1], 4, 2, 16), ([17, 18, 33], 17, 0, 16), ([100, 64, 65, 130], 64, 8, 32),
    ([1025], 1024, 32, 64), ([3000, 1500, 7], 700, 700, 128), ([2100], 1, 1, 256), ([2047, 2049], 2048, 1, 16),
    ([60000], 2000, 32, 128), ([300], 299, 0, 16), ([4500, 4097], 4096, 16, 32), ([16385, 9000], 16384, 100, 64),
    ([9001, 12000], 8192, 1000, 32), ([420000], 300, 10, 256)])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_evict_matches_the_form(lens, budget, recent, page, kind):
    rng = np.random.default_rng(sum(lens) + budget)
    t = Paged(rng, lens, 2, 64, page)
    if kind == "ties":
        w = rng.integers(0, 3, t.pool.weights.shape).astype(np.float32)
    elif kind == "odd":  # zeros of both signs, infinities, NaN, denormals, negatives
        w = rng.choice(np.array([0.0, -0.0, 1e-42, -1e-42, np.inf, -np.inf, np.nan, -1.5, 2.0, 1e30], np.float32),
                       t.pool.weights.shape)
    else:
        w = t.pool.weights
    t.pool.weights[...] = w
    t.cache.weights.copy_(torch.from_numpy(w))
    for b, n in enumerate(lens):  # positions: every head its own order
        t.pool.next_pos[b] = max(1, n)
    t.cache.next_pos.copy_(_dev_i32(t.pool.next_pos))
    kvc.kvc_paged_evict(t.cache, budget, recent, dev_err=t.err)
    ref.evict(t.pool, budget, recent)
    t.check_state(kind)
    kvc.kvc_paged_evict(t.cache, budget, recent, dev_err=t.err)  # at the budget: nothing to do
    t.check_state(kind)


def test_evict_flags_bad_pages_and_lengths():
    rng = np.random.default_rng(51)
    for kind in ("page", "long", "negative"):
        t = Paged(rng, [200, 90], 2, 64, 16)
        if kind == "page":
            t.cache.block_table[0, 5] = -1
        else:
            t.cache.seq_lens[0] = 100000 if kind == "long" else -1
        held = t.cache.seq_lens[0].item()
        k, w = t.cache.k.clone(), t.cache.weights.clone()
        kvc.kvc_paged_evict(t.cache, 64, 4, dev_err=t.err)
        torch.cuda.synchronize()
        assert t.err.item() == kvc.KVC_DEV_ERR_PAGES
        assert t.cache.seq_lens.tolist() == [held, 64]
        mine = [int(p) for p in t.pool.table[0, :13]]
        assert torch.equal(t.cache.k[mine], k[mine]) and torch.equal(t.cache.weights[mine], w[mine])


# --------------------------------------------------------------------------- #
# together, as they are used
# --------------------------------------------------------------------------- #
def _serve(graph):
    """Prompts -> packed prefill -> window scores -> selection -> paged cache ->
    decoding steps (append, attend and accumulate, evict)."""
    rng = np.random.default_rng(61)
    lens, H, Hkv, d, w, kk, budget = [200, 333, 64], 8, 2, 128, 16, 48, 52
    n, B = sum(lens), 3
    cu, cu_np = _dev_i32(_cu(lens)), _cu(lens)
    q, qd = _bf16(rng, n, H, d)
    k, kd = _bf16(rng, n, Hkv, d)
    v, vd = _bf16(rng, n, Hkv, d)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvc.kvc_prefill_attention_varlen(qd, kd, vd, cu, cu, max(lens), max(lens), dev_err=err)
    q_win = torch.stack([qd[e - w:e] for e in cu_np[1:]])
    scores = kvc.kvc_score_varlen(q_win, kd, cu, max(lens), dev_err=err)
    idx, _ = kvc.kvc_select_topk_varlen(scores, cu, max(lens), w, 7, kk, dev_err=err)
    cache = kvc.PagedCache.allocate(24, 16, Hkv, d, B, 4, "cuda")
    table = rng.permutation(24)[:12].reshape(B, 4)
    cache.block_table.copy_(_dev_i32(table))
    kvc.kvc_paged_append(cache, kd, vd, cu, max(lens), idx=idx, scores=scores, dev_err=err)
    pool = ref.Pool(np.zeros((24, Hkv, 16, d)), np.zeros((24, Hkv, 16, d)), np.zeros((24, Hkv, 16), np.float32),
                    np.zeros((24, Hkv, 16), np.int32), table, np.zeros(B, np.int32), np.zeros(B, np.int32))
    ref.append(pool, k, v, cu_np, idx.cpu().numpy(), scores.cpu().numpy())
    tok = [torch.empty((B, x, d), dtype=torch.bfloat16, device="cuda") for x in (H, Hkv, Hkv)]
    out, lse = torch.empty((B, H, d), device="cuda"), torch.empty((B, H), device="cuda")

    def step():
        kvc.kvc_paged_append(cache, tok[1], tok[2], dev_err=err)
        kvc.kvc_paged_decode_attention(tok[0], cache, accumulate=True, out=out, lse=lse, dev_err=err)
        kvc.kvc_paged_evict(cache, budget, w, dev_err=err)

    run = step
    if graph:
        state = [x.clone() for x in (cache.k, cache.v, cache.weights, cache.pos, cache.seq_lens, cache.next_pos)]
        for x in tok:
            x.zero_()
        step()  # the kernels' attributes are set before the capture
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for x, s in zip((cache.k, cache.v, cache.weights, cache.pos, cache.seq_lens, cache.next_pos), state):
            x.copy_(s)
        run = g.replay
    results = []
    for i in range(9):
        new = [_bf16(rng, *x.shape) for x in tok]
        for x, (_, dev) in zip(tok, new):
            x.copy_(dev)
        run()
        ref.append(pool, new[1][0], new[2][0], np.arange(B + 1))
        w_out, w_lse, add, tol, tol_lse, _ = ref.paged_decode(pool, new[0][0], 1 / math.sqrt(d))
        torch.cuda.synchronize()
        assert err.item() == 0
        _close(_np(out), w_out, tol, f"step {i} out")
        _close(_np(lse), w_lse, tol_lse, f"step {i} lse")
        for (b, g_), a in add.items():
            pool.weights[pool.at(b, g_, np.arange(len(a)))] += a.astype(np.float32)
        ref.evict(pool, budget, w)
        np.testing.assert_array_equal(cache.seq_lens.cpu().numpy(), pool.seq_lens)
        pos = cache.pos.cpu().numpy()
        for b in range(B):
            for g_ in range(Hkv):
                at = pool.at(b, g_, np.arange(pool.seq_lens[b]))
                np.testing.assert_array_equal(pos[at], pool.pos[at], err_msg=f"step {i}")
        results.append(out.clone())
    return results


def test_a_prompt_is_compacted_and_decoded():
    _serve(graph=False)


def test_decoding_steps_replayed_from_a_graph():
    eager, replayed = _serve(graph=False), _serve(graph=True)
    for a, b in zip(eager, replayed):
        assert torch.equal(a, b)


def test_two_streams_and_two_graphs_share_no_workspace():
    """Decode calls of one cache that overlap: on two streams, and as two
    captured graphs replayed at once."""
    rng = np.random.default_rng(71)
    t = Paged(rng, [5000, 3300], 2, 128, 16)
    qs = [_bf16(rng, 2, 8, 128)[1] for _ in range(2)]
    want = [kvc.kvc_paged_decode_attention(q, t.cache)[0].clone() for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(w) for w in want]
    lses = [torch.empty((2, 8), device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, o, l, s in zip(qs, outs, lses, streams):
            kvc.kvc_paged_decode_attention(q, t.cache, out=o, lse=l, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graphs = []
    for q, o, l in zip(qs, outs, lses):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvc.kvc_paged_decode_attention(q, t.cache, out=o, lse=l)
        graphs.append(g)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_a_captured_call_names_its_stream():
    """The stream a call is given is being captured, the current one is not: the
    workspace made then is the graph's, not one kept for later calls, which
    would find its counters unset until the graph's first replay."""
    rng = np.random.default_rng(73)
    t = Paged(rng, [900, 5, 333], 2, 64, 16)
    q = _bf16(rng, 3, 4, 64)[1]
    out, lse = torch.empty((3, 4, 64), device="cuda"), torch.empty((3, 4), device="cuda")
    want = kvc.kvc_paged_decode_attention(q, t.cache)[0]
    torch.cuda.synchronize()
    s, side, g = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        with torch.cuda.stream(side):
            kvc.kvc_paged_decode_attention(q, t.cache, out=out, lse=lse, stream=s)
    assert not any(handle == s.cuda_stream for _, handle in t.cache._ws)
    got = kvc.kvc_paged_decode_attention(q, t.cache, stream=s)[0]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_threads_accumulate_on_one_stream():
    """Accumulating calls of several host threads on one stream: each adds its
    own query's attention."""
    import threading
    rng = np.random.default_rng(79)
    t = Paged(rng, [700, 65], 2, 64, 16)
    qs = [_bf16(rng, 2, 4, 64) for _ in range(4)]
    held = [t.pool.at(b, g, np.arange(n)) for b, n in enumerate((700, 65)) for g in range(2)]
    before = t.cache.weights.cpu().numpy().astype(np.float64)
    threads = [threading.Thread(target=lambda q=q: [
        kvc.kvc_paged_decode_attention(q, t.cache, accumulate=True) for _ in range(25)]) for _, q in qs]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    want, tol = before.copy(), np.zeros_like(before)
    for q, _ in qs:
        _, _, add, _, _, tol_add = ref.paged_decode(t.pool, q, 1 / math.sqrt(64))
        for (b, g), a in add.items():
            at = t.pool.at(b, g, np.arange(len(a)))
            want[at] += 25 * a
            tol[at] += 25 * tol_add[b, g]
    got = t.cache.weights.cpu().numpy()
    for at in held:  # each of the 100 sums is rounded
        _close(got[at], want[at], tol[at] + 100 * 2.0 ** -24 * want[at] * 1.01, "weights")


# --------------------------------------------------------------------------- #
# bounded waits
# --------------------------------------------------------------------------- #
def test_wait_bounds_report_a_timeout_and_the_calls_return():
    """The same kernels with a wait bound of a nanosecond: a wait that would
    have ended soon gives up, the call records it, lets its copies and MMAs land
    and returns, and the regular calls after it are right."""
    import ctypes
    import os

    from long_context_kv_window_b200 import build as kbuild

    assert os.path.exists(kbuild.SHORTWAIT_LIB), "run `python -m long_context_kv_window_b200.build`"
    L = ctypes.CDLL(kbuild.SHORTWAIT_LIB)
    for name in ("kvc_prefill_attention_varlen", "kvc_paged_decode_attention"):
        fn = getattr(L, name)
        fn.argtypes, fn.restype = kvc._SIGS[name]
    rng = np.random.default_rng(81)
    n, H, Hkv, d = 700, 8, 2, 128
    q, qd = _bf16(rng, n, H, d)
    k, kd = _bf16(rng, n, Hkv, d)
    v, vd = _bf16(rng, n, Hkv, d)
    cu = _dev_i32([0, n])
    out, lse = torch.empty_like(qd), torch.empty((n, H), device="cuda")
    t = Paged(rng, [900, 40], Hkv, d, 16)
    # a stream long enough that loads queue: 123 MB of entries, pages shared by the sequences
    pages = torch.randn(15000, Hkv, 16, d, device="cuda").bfloat16()
    long = kvc.PagedCache(pages, pages, torch.randint(15000, (2, 3750), device="cuda").to(torch.int32),
                          _dev_i32([60000, 59000]))
    dq, dout, dlse = qd[:2].contiguous(), torch.empty((2, H, d), device="cuda"), torch.empty((2, H), device="cuda")
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        err.zero_()
        rc = L.kvc_prefill_attention_varlen(qd.data_ptr(), H * d, d, kd.data_ptr(), Hkv * d, d, vd.data_ptr(), Hkv * d, d,
                                            cu.data_ptr(), cu.data_ptr(), 1, n, n, n, n, H, Hkv, d, 0.1,
                                            out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), err.data_ptr(), st)
        torch.cuda.synchronize()
        assert rc == kvc.KVC_OK and err.item() & kvc.KVC_DEV_ERR_TIMEOUT
        err.zero_()
        rc = L.kvc_paged_decode_attention(long._ref, dq.data_ptr(), H * d, d, H, 0.1, long.capacity, 0,
                                          dout.data_ptr(), dlse.data_ptr(), ws.data_ptr(), ws.numel(), err.data_ptr(), st)
        torch.cuda.synchronize()
        assert rc == kvc.KVC_OK
        if not err.item() & kvc.KVC_DEV_ERR_TIMEOUT:  # every copy was there when it was asked for
            assert torch.equal(dout, kvc.kvc_paged_decode_attention(dq, long, scale=0.1)[0])
    out, lse = _run_prefill(qd[:60], kd[:60], vd[:60], [60], [60])
    w_out, w_lse, tol, tol_lse = ref.prefill_varlen(q[:60], k[:60], v[:60], [0, 60], [0, 60], 1 / math.sqrt(d))
    _close(_np(out), w_out, tol, "out after the short waits")
    t.decode(rng, H, True)
    # the counters went back to zero: the workspace serves on
    assert torch.equal(kvc.kvc_paged_decode_attention(dq, long, ws=ws)[0], kvc.kvc_paged_decode_attention(dq, long)[0])
