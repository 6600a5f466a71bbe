"""GPU tests of the serving operators at the edges of what their documentation
allows: workspaces that one caller shares among the calls, empty selections,
padded packed batches, rows whose logits are all -inf, streams that the calls
are given, waits that give up."""
import math

import numpy as np
import pytest
import torch

import long_context_kv_window_b200 as kvc
from tests import paged_reference as ref
from tests.test_gpu_paged import Paged, _bf16, _close, _cu, _dev_i32, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvc.lib()
    torch.cuda.set_device(0)


def test_one_workspace_serves_append_decode_and_evict_in_turn():
    """Every call leaves the first batch * num_kv_heads counters at zero, also
    where they are more than a workspace's smallest piece of 256 bytes."""
    rng = np.random.default_rng(3)
    B, Hkv, d, budget = 16, 8, 64, 500
    t = Paged(rng, [int(x) for x in rng.integers(520, 700, B)], Hkv, d, 16, room=40)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    counters = ws[:4 * B * Hkv]
    assert counters.numel() > 256
    for _ in range(2):
        k, kd = _bf16(rng, 30 * B, Hkv, d)
        v, vd = _bf16(rng, 30 * B, Hkv, d)
        cu = _cu([30] * B)
        kvc.kvc_paged_append(t.cache, kd, vd, _dev_i32(cu), 30, ws=ws, dev_err=t.err)
        ref.append(t.pool, k, v, cu)
        t.check_state("append")
        assert not counters.any(), "append"
        t.decode(rng, 2 * Hkv, True, ws=ws)
        assert not counters.any(), "decode"
        kvc.kvc_paged_evict(t.cache, budget, 10, ws=ws, dev_err=t.err)
        ref.evict(t.pool, budget, 10)
        t.check_state("evict")
        assert not counters.any(), "evict"


def test_append_of_an_empty_selection():
    """A selection of no entry keeps none: the tokens are seen, nothing is written."""
    rng = np.random.default_rng(5)
    t = Paged(rng, [7, 0, 20], 2, 64, 16, room=40)
    held = [x.clone() for x in (t.cache.k, t.cache.v, t.cache.weights, t.cache.pos)]
    lens = [5, 0, 12]
    _, kd = _bf16(rng, sum(lens), 2, 64)
    kvc.kvc_paged_append(t.cache, kd, kd, _dev_i32(_cu(lens)), 12, idx=_dev_i32(np.zeros((3, 2, 0))), dev_err=t.err,
                         scores=torch.ones((2, sum(lens)), device="cuda"))
    t.pool.next_pos += np.array(lens, np.int32)
    t.check_state()
    for x, y in zip(held, (t.cache.k, t.cache.v, t.cache.weights, t.cache.pos)):
        assert torch.equal(x, y)


def test_a_wait_that_gives_up_leaves_the_weights_alone():
    """Accumulating decode with a wait bound of a nanosecond: a KV head some of
    whose entries did not arrive in time has no result and leaves its weights as
    they were; the others, if any, are the regular call's, to the last bit."""
    import ctypes

    from long_context_kv_window_b200 import build as kbuild

    L = ctypes.CDLL(kbuild.SHORTWAIT_LIB)
    fn = L.kvc_paged_decode_attention
    fn.argtypes, fn.restype = kvc._SIGS["kvc_paged_decode_attention"]
    B, Hkv, H, d, page, n = 6, 4, 8, 128, 16, 20000
    pages = B * n // page
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((pages, Hkv, page, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(B, -1)
    lens = _dev_i32([n - 7 * b for b in range(B)])
    w0 = torch.rand((pages, Hkv, page), generator=g, device="cuda")
    q = torch.randn((B, H, d), generator=g, device="cuda").bfloat16()
    regular, short = (kvc.PagedCache(k, v, table, lens, weights=w0.clone()) for _ in range(2))
    out, lse = kvc.kvc_paged_decode_attention(q, regular, scale=0.1, accumulate=True)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    got, got_lse, err = torch.empty_like(out), torch.empty_like(lse), torch.zeros(1, dtype=torch.int32, device="cuda")
    seen = 0
    for _ in range(20):
        short.weights.copy_(w0)
        err.zero_()
        rc = fn(short._ref, q.data_ptr(), H * d, d, H, 0.1, short.capacity, 1, got.data_ptr(), got_lse.data_ptr(),
                ws.data_ptr(), ws.numel(), err.data_ptr(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert rc == kvc.KVC_OK and err.item() in (0, kvc.KVC_DEV_ERR_TIMEOUT)
        assert not ws[:4 * B * Hkv].any()
        none = (got_lse == -math.inf).view(B, Hkv, H // Hkv)
        assert (none.all(2) == none.any(2)).all() and none.any() == (err.item() != 0)
        none = none.all(2)
        rows = none.repeat_interleave(H // Hkv, 1)
        assert (got[rows] == 0).all() and torch.equal(got[~rows], out[~rows]) and torch.equal(got_lse[~rows], lse[~rows])
        kept = none[torch.arange(B, device="cuda").repeat_interleave(n // page)]  # [B * pages of a sequence][Hkv]
        by_page = torch.empty_like(kept)
        by_page[table.reshape(-1).long()] = kept
        assert torch.equal(short.weights, torch.where(by_page[:, :, None], w0, regular.weights))
        seen += err.item() != 0
        if seen == 3:
            break
    assert seen, "no wait gave up"
    kvc.kvc_paged_decode_attention(q, short, scale=0.1, out=got, lse=got_lse, ws=ws)
    assert torch.equal(got, out) and torch.equal(got_lse, lse)


@pytest.mark.parametrize("lens", [[50, 33], [3000, 700]])
def test_decode_over_entries_whose_logits_are_all_minus_infinity(lens):
    """exp(s - lse) of such a head is NaN, and so is what the entries' weights
    become: the head is not taken for one whose pages could not be read."""
    rng = np.random.default_rng(11)
    t = Paged(rng, lens, 2, 64, 16)
    q, qd = _bf16(rng, 2, 6, 64)
    qd[:, :, 9] = qd[:, :, 9].abs() + 1
    clean = [x.clone() for x in kvc.kvc_paged_decode_attention(qd, t.cache)]
    before = t.cache.weights.clone()
    at = [x.tolist() if isinstance(x, np.ndarray) else x for x in t.pool.at(0, 1, np.arange(lens[0]))]
    t.cache.k[at[0], 1, at[2], 9] = -math.inf
    out, lse = kvc.kvc_paged_decode_attention(qd, t.cache, accumulate=True, dev_err=t.err)
    torch.cuda.synchronize()
    assert t.err.item() == 0
    assert out[0, 3:].isnan().all() and (lse[0, 3:] == -math.inf).all()
    assert torch.equal(out[0, :3], clean[0][0, :3]) and torch.equal(out[1], clean[0][1])
    assert torch.equal(lse[0, :3], clean[1][0, :3]) and torch.equal(lse[1], clean[1][1])
    assert t.cache.weights[at[0], 1, at[2]].isnan().all()
    others = torch.ones_like(before, dtype=torch.bool)
    others[at[0], 1, at[2]] = False
    assert t.cache.weights[others].isfinite().all() and not torch.equal(t.cache.weights[others], before[others])


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_varlen_rows_without_a_finite_logit_split_or_not(d):
    """A row that sees keys, all at -inf, has the log-sum-exp -inf and NaN as
    output; a NaN in its query makes NaN of both.  That does not depend on how
    many CTAs share its keys, and rows that see no key stay 0 and -inf."""
    rng = np.random.default_rng(d)
    H, Hkv, lq, lk = 4, 2, 24, 2600
    _, q = _bf16(rng, lq, H, d)
    _, k = _bf16(rng, lk, Hkv, d)
    _, v = _bf16(rng, lk, Hkv, d)
    q[:, :, 3] = q[:, :, 3].abs() + 1
    k[:, 1, 3] = -math.inf  # the second KV head's logits
    q[5, 0, 7] = math.nan
    none = torch.empty((0, Hkv, d), dtype=torch.bfloat16, device="cuda")
    assert kvc.prefill_varlen_workspace_size(H, Hkv, d, 2, 2 * lq, lq, lk) > 0  # split
    many = 90
    assert kvc.prefill_varlen_workspace_size(H, Hkv, d, many, many * lq, lq, lk) == 0
    for B in (2, many):  # the last sequence has no key
        lens_k = [lk] * (B - 1) + [0]
        out, lse = (x.clone() for x in kvc.kvc_prefill_attention_varlen(
            q.repeat(B, 1, 1), torch.cat([k] * (B - 1) + [none]), torch.cat([v] * (B - 1) + [none]),
            _dev_i32(_cu([lq] * B)), _dev_i32(_cu(lens_k)), lq, lk))
        for b in range(B - 1):
            o, z = out[b * lq:(b + 1) * lq], lse[b * lq:(b + 1) * lq]
            assert o[:, 2:].isnan().all() and (z[:, 2:] == -math.inf).all(), (B, b)
            assert o[5, 0].isnan().all() and z[5, 0].isnan(), (B, b)
            rest = torch.ones((lq, 2), dtype=torch.bool, device="cuda")
            rest[5, 0] = False
            assert o[:, :2][rest].isfinite().all() and z[:, :2][rest].isfinite().all(), (B, b)
        assert (out[-lq:] == 0).all() and (lse[-lq:] == -math.inf).all()


@pytest.mark.parametrize("lq,most,H,d", [([20], 20, 8, 128), ([20, 0, 13], 20, 8, 64), ([3, 40, 17], 64, 4, 128)])
def test_prefill_varlen_split_rows_in_a_padded_batch(lq, most, H, d):
    """Few rows over many keys in a q with room for thousands: as in a tight
    one, and the room behind is left as it was."""
    rng = np.random.default_rng(sum(lq) + H)
    Hkv, lk = 2, [2900 - 150 * b for b in range(len(lq))]
    room = 5000
    q, qd = _bf16(rng, sum(lq), H, d)
    k, kd = _bf16(rng, sum(lk), Hkv, d)
    v, vd = _bf16(rng, sum(lk), Hkv, d)
    big = torch.full((room, H, d), math.nan, dtype=torch.bfloat16, device="cuda")
    big[:sum(lq)] = qd
    got = []
    for x in (qd, big):
        out = torch.full(x.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(x.shape[:2], 7.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert kvc.prefill_varlen_workspace_size(H, Hkv, d, len(lq), x.shape[0], most, max(lk)) > 0
        kvc.kvc_prefill_attention_varlen(x, kd, vd, _dev_i32(_cu(lq)), _dev_i32(_cu(lk)), most, max(lk), out=out, lse=lse,
                                         dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == 0
        got.append((out, lse))
    w_out, w_lse, tol, tol_lse = ref.prefill_varlen(q, k, v, _cu(lq), _cu(lk), 1 / math.sqrt(d))
    n = sum(lq)
    for out, lse in got:
        _close(_np(out)[:n], w_out, tol, "out")
        _close(_np(lse)[:n], w_lse, tol_lse, "lse")
        assert (out[n:] == 7).all() and (lse[n:] == 7).all()


@pytest.mark.parametrize("op", ["prefill", "decode"])
def test_results_of_a_call_on_another_stream_have_memory_of_their_own(op):
    """A tensor that was freed while work of the current stream still reads it is
    not where a call on another stream, which does not wait for that work, puts
    its results; nor is a result that the current stream still reads where the
    next call puts its own."""
    rng = np.random.default_rng(13)
    s = torch.cuda.Stream()
    if op == "prefill":
        n, H, d, dtype = 2000, 8, 128, torch.bfloat16
        _, q = _bf16(rng, n, H, d)
        _, k = _bf16(rng, n, 2, d)
        cu = _dev_i32([0, n])

        def call(stream, q=q):
            return kvc.kvc_prefill_attention_varlen(q, k, k, cu, cu, n, n, stream=stream)
    else:
        n, H, d, dtype = 256, 32, 128, torch.float32
        t = Paged(rng, [20] * n, 2, d, 16)
        _, q = _bf16(rng, n, H, d)

        def call(stream, q=q):
            return kvc.kvc_paged_decode_attention(q, t.cache, stream=stream)
    other_q = -q
    call(s)  # the cache's workspace of that stream
    want = [x.clone() for x in call(None)]
    held = torch.full((n, H, d), 3.0, dtype=dtype, device="cuda")
    copy = torch.empty_like(held)
    torch.cuda.synchronize()
    torch.cuda._sleep(300_000_000)
    copy.copy_(held)
    del held
    out, lse = call(s)
    torch.cuda.synchronize()
    assert (copy == 3.0).all()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    torch.cuda._sleep(300_000_000)
    copy.copy_(out)
    del out
    other = call(s, other_q)[0]
    torch.cuda.synchronize()
    assert torch.equal(copy, want[0]) and not torch.equal(other, want[0])


def test_a_bound_that_follows_the_lengths_keeps_few_workspaces():
    """max_len given exactly, a token longer each step: the kept workspace is made
    anew a few times, and what the cache remembers of the sizes stays small."""
    rng = np.random.default_rng(17)
    t = Paged(rng, [300, 12], 2, 64, 16, room=1400)
    _, k = _bf16(rng, 2, 2, 64)
    _, q = _bf16(rng, 2, 4, 64)
    made, n = set(), 300
    for step in range(1400):
        kvc.kvc_paged_append(t.cache, k, k, dev_err=t.err)
        n += 1
        kvc.kvc_paged_decode_attention(q, t.cache, max_len=n, accumulate=True, dev_err=t.err)
        kvc.kvc_paged_evict(t.cache, 4000, 1, max_len=n, dev_err=t.err)
        made |= {(key, kept[2]) for key, kept in t.cache._ws.items()}
        assert len(t.cache._need) <= 256
    assert len(made) < 30
    t.pool.seq_lens += 1400
    at = [t.pool.at(b, g, np.arange(m)) for b, m in enumerate(t.pool.seq_lens) for g in range(2)]
    kd, vd = _np(t.cache.k), _np(t.cache.v)
    for i in at:
        t.pool.k[i], t.pool.v[i] = kd[i], vd[i]
    t.pool.weights = t.cache.weights.cpu().numpy().copy()
    t.decode(rng, 4, True, max_len=n)


def test_prefill_varlen_queries_where_the_bound_says_none():
    """max_seqlen_q = 0: sequences without queries are fine, one with some is reported."""
    q = torch.randn((6, 4, 64), device="cuda").bfloat16()
    for cu, want in (([0, 0, 0], 0), ([0, 0, 6], kvc.KVC_DEV_ERR_SEQLENS)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = torch.full_like(q, 7.0), torch.full((6, 4), 7.0, device="cuda")
        kvc.kvc_prefill_attention_varlen(q, q[:, :2], q[:, :2], _dev_i32(cu), _dev_i32([0, 3, 6]), 0, 3, out=out, lse=lse,
                                         dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == want and (out == 7).all() and (lse == 7).all()


def test_append_with_a_bound_far_above_the_tokens():
    rng = np.random.default_rng(19)
    lens = [1, 0, 40]
    t = Paged(rng, [5, 6, 7], 2, 64, 16, room=50)
    k, kd = _bf16(rng, sum(lens), 2, 64)
    kvc.kvc_paged_append(t.cache, kd, kd, _dev_i32(_cu(lens)), (1 << 30) - 1, dev_err=t.err)
    ref.append(t.pool, k, k, _cu(lens))
    t.check_state()
    kvc.kvc_paged_append(t.cache, kd[:0], kd[:0], _dev_i32(_cu([0, 0, 0])), 9, dev_err=t.err)
    t.check_state()


def test_prefill_varlen_calls_that_overlap():
    """Split and unsplit calls on two streams at once, eager and as two graphs
    replayed at once: each as it is alone, to the last bit."""
    rng = np.random.default_rng(23)
    H, Hkv, d = 8, 2, 128
    plans = [([900, 40, 2000, 3], [900, 40, 2000, 3]), ([16, 30], [5000, 4000])]
    calls, want = [], []
    for lq, lk in plans:
        q, k, v = (_bf16(rng, n, h, d)[1] for n, h in ((sum(lq), H), (sum(lk), Hkv), (sum(lk), Hkv)))
        cq, ck = _dev_i32(_cu(lq)), _dev_i32(_cu(lk))
        out, lse = torch.empty_like(q), torch.empty((sum(lq), H), device="cuda")

        def call(stream, q=q, k=k, v=v, cq=cq, ck=ck, lq=lq, lk=lk, out=out, lse=lse):
            kvc.kvc_prefill_attention_varlen(q, k, v, cq, ck, max(lq), max(lk), out=out, lse=lse, stream=stream)
            return out, lse
        want.append([x.clone() for x in call(None)])
        calls.append(call)
    split = [kvc.prefill_varlen_workspace_size(H, Hkv, d, len(lq), sum(lq), max(lq), max(lk)) > 0 for lq, lk in plans]
    assert split == [False, True]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for call in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(None)
    for replay in (False, True):
        for call in calls:
            for x in call(None):
                x.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for call, g, s in zip(calls, graphs, streams):
                if replay:
                    with torch.cuda.stream(s):
                        g.replay()
                else:
                    call(s)
        torch.cuda.synchronize()
        for call, w in zip(calls, want):
            out, lse = call.__defaults__[-2:]
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])
