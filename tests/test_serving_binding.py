"""CPU tests of what the binding of the serving operators hands to the library."""
import pytest
import torch

import long_context_kv_window_b200 as kvc
from tests.test_binding_checks import lib as fake_lib  # noqa: F401  (fixture)
from tests.test_paged_checks import _tensors
from tests.test_paged_checks import lib as paged_lib  # noqa: F401  (fixture)

bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture
def calls(paged_lib, monkeypatch):  # noqa: F811
    """Every library call with its arguments."""
    made = []
    monkeypatch.setattr(kvc, "_call", lambda dev, fn, *args: made.append(args) or fn(*args))
    return made


def test_a_selection_of_no_entry_is_not_every_token(calls):
    c = kvc.PagedCache(**_tensors())
    p, cu = torch.empty((9, 2, 64), dtype=bf), torch.zeros(3, dtype=i32)
    for idx, null in ((None, True), (torch.zeros((2, 2, 4), dtype=i32), False), (torch.zeros((2, 2, 0), dtype=i32), False)):
        kvc.kvc_paged_append(c, p, p, cu, 5, idx=idx)
        sel, kk = calls[-1][8:10]
        assert (sel is None) == null and sel != 0 and kk == (0 if idx is None else idx.shape[2])


def test_prefill_workspace_does_not_grow_with_room_behind_the_sequences():
    """A few rows over many keys in a q with room for many more rows."""
    from long_context_kv_window_b200 import build
    build.build()
    size = kvc.prefill_varlen_workspace_size
    tight = size(32, 8, 128, 3, 60, 20, 30000)
    assert tight > 0
    assert size(32, 8, 128, 3, 1 << 20, 20, 30000) == tight
    # at most three CTAs per SM (148 of them) with 256 rows each, of d + 1 floats
    for H, Hkv, d, B, tq, mq, mk in ((32, 8, 128, 1, 1 << 30, 32, 1 << 17), (8, 1, 64, 5, 1 << 20, 100, 1 << 20),
                                     (1, 1, 128, 200, 300, 101, 1 << 20), (40, 8, 128, 4, 7, 7, 1 << 15)):
        assert size(H, Hkv, d, B, tq, mq, mk) <= 3 * 148 * 256 * (d + 1) * 4 + 512


def test_prefill_workspace_is_that_of_the_tensors_device(monkeypatch):
    """The size hangs on the SMs of the device that the tensors are on, which
    need not be the current one."""
    current = [0]

    def call(dev, fn, *args):
        before, current[0] = current[0], dev.index
        try:
            return fn(*args)
        finally:
            current[0] = before

    class Lib:
        @staticmethod
        def kvc_prefill_varlen_workspace_size(*args):
            args[-1]._obj.value = 1000 + current[0]
            return kvc.KVC_OK

    monkeypatch.setattr(kvc, "_call", call)
    monkeypatch.setattr(kvc, "lib", Lib)
    shape = (6, 2, 64, 11, 977, 131, 8191)  # of no other test
    for _ in range(2):
        assert [kvc.prefill_varlen_workspace_size(*shape, torch.device("cuda", i)) for i in (0, 1, 0, 2)] == [
            1000, 1001, 1000, 1002]
    kvc._prefill_varlen_bytes.cache_clear()


def test_append_beyond_the_counter_of_its_ctas_is_refused():
    import ctypes

    from long_context_kv_window_b200 import build
    from tests.test_paged_checks import PTR, _cache
    build.build()

    def call(batch, total, most):
        c = _cache(batch=batch, page_size=256, max_pages=1 << 22, table_stride=1 << 22, page_stride=1 << 15)
        return kvc.lib().kvc_paged_append(ctypes.byref(c), PTR, PTR, 128, 64, PTR, total, most, None, 0, None, PTR, 256,
                                          None, None)

    before = kvc.launch_count()
    assert call(1024, (1 << 31) - 1, (1 << 30) - 1) == 1 and "2^38" in kvc.last_error()
    assert call(1024, 1 << 27, 1 << 28) == 1  # 2^28 entries of two heads, 1024 times
    assert kvc.launch_count() == before
