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
