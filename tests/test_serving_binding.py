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
