"""CPU tests of what the serving operators refuse: the C entry points, which
validate before any launch, and the Python binding, which checks every
tensor's extent (the CUDA-only steps replaced by stand-ins)."""
import ctypes

import pytest
import torch

import long_context_kv_window_b200 as kvc
from tests.test_binding_checks import lib as fake_lib  # noqa: F401  (fixture)

f32, i32, bf = torch.float32, torch.int32, torch.bfloat16
PTR = ctypes.c_void_p(256)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def clib():
    from long_context_kv_window_b200 import build
    build.build()
    return kvc.lib()


def _cache(**kw):
    f = dict(k=256, v=256, weights=256, pos=256, block_table=256, seq_lens=256, next_pos=256, page_stride=2 * 16 * 64,
             table_stride=4, num_pages=8, page_size=16, max_pages=4, batch=2, num_kv_heads=2, head_dim=64)
    f.update(kw)
    return kvc.PagedCacheStruct(*(f[n] for n, _ in kvc.PagedCacheStruct._fields_))


SHAPES = [(dict(head_dim=96), 2), (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=512), 2),
          (dict(batch=0), 1), (dict(batch=1025), 1), (dict(num_kv_heads=0), 1), (dict(num_pages=0), 1),
          (dict(max_pages=0), 1), (dict(max_pages=1 << 28), 1), (dict(table_stride=3), 1),
          (dict(page_stride=2 * 16 * 64 - 8), 1), (dict(page_stride=2 * 16 * 64 + 4), 1)]
POINTERS = [(dict(k=0), 1), (dict(v=0), 1), (dict(block_table=0), 1), (dict(seq_lens=0), 1), (dict(k=264), 1),
            (dict(pos=0), 1), (dict(next_pos=0), 1)]


@pytest.mark.parametrize("fields,status", SHAPES + POINTERS)
def test_every_paged_call_checks_the_cache(clib, fields, status):
    c = ctypes.byref(_cache(**fields))
    n = ctypes.c_size_t()
    before = kvc.launch_count()
    shape = (fields, status) in SHAPES
    if shape:
        assert clib.kvc_paged_append_workspace_size(c, ctypes.byref(n)) == status
        assert clib.kvc_paged_decode_workspace_size(c, 4, 64, 1, ctypes.byref(n)) == status
        assert clib.kvc_paged_evict_workspace_size(c, 64, 8, ctypes.byref(n)) == status
    assert clib.kvc_paged_append(c, PTR, PTR, 128, 64, None, 2, 1, None, 0, None, PTR, 1 << 20, None, None) == status
    assert clib.kvc_paged_decode_attention(c, PTR, 256, 64, 4, 0.125, 64, 0, PTR, None, PTR, 1 << 30, None,
                                           None) == status
    assert clib.kvc_paged_evict(c, 64, 8, 2, PTR, 1 << 30, None, None) == status
    assert kvc.last_error() != "" and kvc.launch_count() == before


def test_append_refusals(clib):
    c = ctypes.byref(_cache())

    def call(k=PTR, sn=128, sh=64, cu=None, total=2, most=1, idx=None, kk=0, ws=PTR, nbytes=256):
        return clib.kvc_paged_append(c, k, PTR, sn, sh, cu, total, most, idx, kk, None, ws, nbytes, None, None)

    assert call(k=None) == 1 and call(k=ctypes.c_void_p(264)) == 1
    assert call(sn=130) == 1 and call(sh=-64) == 1
    assert call(total=3) == 1 and call(most=2) == 1            # one token per sequence without cu_seqlens
    assert call(cu=PTR, total=-1) == 1 and call(cu=PTR, total=9, most=-1) == 1
    assert call(cu=PTR, total=9, most=5, idx=PTR, kk=-1) == 1
    assert call(ws=None) == 4 and call(nbytes=16) == 4 and call(ws=ctypes.c_void_p(128)) == 4
    assert call(cu=PTR, total=9, most=1 << 30, nbytes=256) == 1  # 2^30 entries of two heads
    assert call(cu=PTR, k=None, total=0, most=0) == 0            # nothing to append


def test_decode_refusals(clib):
    def call(q=PTR, sb=256, sh=64, H=4, scale=0.125, most=64, acc=0, out=PTR, ws=PTR, nbytes=1 << 30, **fields):
        return clib.kvc_paged_decode_attention(ctypes.byref(_cache(**fields)), q, sb, sh, H, scale, most, acc, out,
                                               None, ws, nbytes, None, None)

    assert call(q=None) == 1 and call(out=None) == 1 and call(q=ctypes.c_void_p(258)) == 1
    assert call(sb=260) == 1 and call(sh=-8) == 1
    assert call(H=3) == 1 and call(H=0) == 1 and call(H=34) == 2  # 17 heads per KV head
    assert call(scale=0.0) == 1 and call(scale=float("inf")) == 1 and call(scale=float("nan")) == 1
    assert call(most=0) == 1 and call(most=65) == 1               # past the block table's room
    assert call(acc=1, weights=0) == 1
    assert call(ws=None) == 4 and call(acc=1, nbytes=256) == 4 and call(ws=ctypes.c_void_p(128)) == 4


def test_evict_refusals(clib):
    def call(most=64, budget=8, recent=2, ws=PTR, nbytes=1 << 30, **fields):
        return clib.kvc_paged_evict(ctypes.byref(_cache(**fields)), most, budget, recent, ws, nbytes, None, None)

    assert call(most=0) == 1 and call(most=65) == 1
    assert call(budget=0) == 1 and call(budget=1 << 31) == 1
    assert call(recent=-1) == 1 and call(recent=9) == 1
    assert call(weights=0) == 1 and call(pos=0, next_pos=0) == 1  # recent entries need positions
    assert call(ws=None) == 4 and call(nbytes=256) == 4 and call(ws=ctypes.c_void_p(128)) == 4


def test_prefill_varlen_refusals(clib):
    def call(q=PTR, k=PTR, st=(512, 128, 256, 128, 256, 128), cu=PTR, B=2, tq=10, tk=10, mq=8, mk=8, H=4, Hkv=2,
             d=128, scale=0.1, out=PTR, ws=PTR, nbytes=1 << 30):
        return clib.kvc_prefill_attention_varlen(q, st[0], st[1], k, st[2], st[3], PTR, st[4], st[5], cu, PTR, B, tq,
                                                 tk, mq, mk, H, Hkv, d, scale, out, None, ws, nbytes, None, None)

    before = kvc.launch_count()
    assert call(q=None) == 1 and call(k=None) == 1 and call(cu=None) == 1
    assert call(q=ctypes.c_void_p(264)) == 1 and call(out=ctypes.c_void_p(264)) == 1
    assert call(d=96) == 2 and call(H=3) == 1 and call(Hkv=0) == 1 and call(H=258) == 2  # 129 heads per KV head
    assert call(B=0) == 1 and call(B=1025) == 1
    assert call(tq=-1) == 1 and call(tk=-1) == 1 and call(tk=1 << 31) == 1
    assert call(mq=-1) == 1 and call(mk=1 << 31) == 1
    assert call(scale=0.0) == 1 and call(scale=float("nan")) == 1
    assert call(st=(516, 128, 256, 128, 256, 128)) == 1 and call(st=(512, 64, 256, 128, 256, 128)) == 1
    # few rows over many keys use a workspace
    assert call(mk=8000, tk=9000, ws=None) == 4 and call(mk=8000, tk=9000, nbytes=64) == 4
    assert call(mk=8000, tk=9000, ws=ctypes.c_void_p(128)) == 4
    assert call(tq=0) == 0  # nothing to do is not an error, and launches nothing
    assert kvc.launch_count() == before
    n = ctypes.c_size_t()
    assert clib.kvc_prefill_varlen_workspace_size(4, 2, 96, 2, 10, 8, 8, ctypes.byref(n)) == 2
    assert clib.kvc_prefill_varlen_workspace_size(4, 2, 128, 2, 10, 8, 8, None) == 1


# --------------------------------------------------------------------------- #
# the binding
# --------------------------------------------------------------------------- #
@pytest.fixture
def lib(fake_lib, monkeypatch):  # noqa: F811
    monkeypatch.setattr(kvc, "_raw_stream", lambda stream, dev: 0)
    monkeypatch.setattr(kvc.PagedCache, "_workspace",
                        lambda self, ws, *a: (0, 16 if ws is None else kvc._ws_bytes(ws, self.device)))
    monkeypatch.setattr(kvc, "_used_on", lambda stream, *made: None)
    return fake_lib


def _tensors(P=6, Hkv=2, page=16, d=64, B=2, mp=3):
    return dict(k=torch.empty((P, Hkv, page, d), dtype=bf), v=torch.empty((P, Hkv, page, d), dtype=bf),
                block_table=torch.zeros((B, mp), dtype=i32), seq_lens=torch.zeros(B, dtype=i32),
                weights=torch.zeros((P, Hkv, page), dtype=f32), pos=torch.zeros((P, Hkv, page), dtype=i32),
                next_pos=torch.zeros(B, dtype=i32))


def test_paged_cache_checks_its_tensors(lib):
    ok = _tensors()
    c = kvc.PagedCache(**ok)
    assert c.capacity == 48 and c._c.page_stride == 2 * 16 * 64 and c._c.table_stride == 3
    both = torch.empty((6, 2, 2, 16, 64), dtype=bf)
    assert kvc.PagedCache(**{**ok, "k": both[:, 0], "v": both[:, 1]})._c.page_stride == 4 * 16 * 64
    one = torch.empty((6, 16, 1, 64), dtype=bf).transpose(1, 2)  # one head: its stride is not a dense tensor's
    heads1 = {n: torch.zeros((6, 1, 16), dtype=t) for n, t in (("weights", f32), ("pos", i32))}
    assert kvc.PagedCache(**{**ok, **heads1, "k": one, "v": one})._c.page_stride == 16 * 64
    wide = torch.zeros((2, 9), dtype=i32)
    assert kvc.PagedCache(**{**ok, "block_table": wide[:, :3]})._c.table_stride == 9
    for b in (dict(k=torch.empty((6, 2, 16, 64), dtype=f32)), dict(v=torch.empty((6, 2, 16, 128), dtype=bf)),
              dict(v=both[:, 1]), dict(k=both[:, 0].transpose(1, 2), v=both[:, 1].transpose(1, 2)),
              dict(block_table=torch.zeros((3, 3), dtype=i32)), dict(block_table=torch.zeros((2, 3), dtype=torch.int64)),
              dict(block_table=torch.zeros((3, 2), dtype=i32).t()), dict(seq_lens=torch.zeros(2, dtype=torch.int64)),
              dict(weights=torch.zeros((6, 2, 15), dtype=f32)), dict(weights=torch.zeros((6, 2, 16), dtype=torch.float64)),
              dict(pos=None), dict(next_pos=None), dict(next_pos=torch.zeros(3, dtype=i32)),
              dict(seq_lens=torch.zeros(2, dtype=i32, device="meta"))):
        with pytest.raises((ValueError, TypeError)):
            kvc.PagedCache(**{**ok, **b})


def test_append_binding(lib):
    c = kvc.PagedCache(**_tensors())
    k = torch.empty((2, 2, 64), dtype=bf)
    p, cu = torch.empty((9, 2, 64), dtype=bf), torch.zeros(3, dtype=i32)
    kvc.kvc_paged_append(c, k, k)
    kvc.kvc_paged_append(c, p, p, cu, 5, idx=torch.zeros((2, 2, 4), dtype=i32), scores=torch.zeros((2, 9), dtype=f32))
    assert lib.calls == ["kvc_paged_append"] * 2
    for a, kw in (((p, p), {}), ((k, None), {}), ((k, p), {}), ((p, p, cu), {}), ((p, p, cu[:2], 5), {}),
                  ((torch.empty((2, 3, 64), dtype=bf),) * 2, {}), ((k, k), dict(idx=torch.zeros((2, 2, 1), dtype=i32))),
                  ((p, p, cu, 5), dict(idx=torch.zeros((2, 4), dtype=i32))),
                  ((p, p, cu, 5), dict(idx=torch.zeros((2, 3, 4), dtype=i32))),
                  ((p, p, cu, 5), dict(scores=torch.zeros((2, 8), dtype=f32))),
                  ((k, k), dict(dev_err=torch.zeros(1, dtype=torch.int64)))):
        with pytest.raises((ValueError, TypeError)):
            kvc.kvc_paged_append(c, *a, **kw)


def test_decode_and_evict_bindings(lib):
    c = kvc.PagedCache(**_tensors())
    q = torch.empty((2, 4, 64), dtype=bf)
    out, lse = kvc.kvc_paged_decode_attention(q, c, accumulate=True)
    assert out.shape == (2, 4, 64) and out.dtype == f32 and lse.shape == (2, 4)
    kvc.kvc_paged_evict(c, 8, 2)
    assert lib.calls == ["kvc_paged_decode_attention", "kvc_paged_evict"]
    bare = kvc.PagedCache(**{**_tensors(), "weights": None, "pos": None, "next_pos": None})
    for f, a, kw in ((kvc.kvc_paged_decode_attention, (q[:1], c), {}),
                     (kvc.kvc_paged_decode_attention, (torch.empty((2, 4, 128), dtype=bf), c), {}),
                     (kvc.kvc_paged_decode_attention, (q.float(), c), {}),
                     (kvc.kvc_paged_decode_attention, (q, bare), dict(accumulate=True)),
                     (kvc.kvc_paged_decode_attention, (q, c), dict(out=torch.empty((2, 4, 64), dtype=bf))),
                     (kvc.kvc_paged_decode_attention, (q, c), dict(lse=torch.empty((4, 2), dtype=f32))),
                     (kvc.kvc_paged_decode_attention, (q, c), dict(ws=torch.empty(32, dtype=torch.uint8)[::2])),
                     (kvc.kvc_paged_evict, (bare, 8, 0), {}),
                     (kvc.kvc_paged_evict, (kvc.PagedCache(**{**_tensors(), "pos": None, "next_pos": None}), 8, 2), {}),
                     (kvc.kvc_paged_evict, (c, 8, 2), dict(dev_err=torch.zeros(1, dtype=f32)))):
        with pytest.raises((ValueError, TypeError)):
            f(*a, **kw)


def test_prefill_varlen_binding(lib, monkeypatch):
    monkeypatch.setattr(kvc, "prefill_varlen_workspace_size", lambda *a: 0)
    q, k = torch.empty((9, 4, 64), dtype=bf), torch.empty((12, 2, 64), dtype=bf)
    cu = torch.zeros(3, dtype=i32)
    out, lse = kvc.kvc_prefill_attention_varlen(q, k, k, cu, cu, 5, 6)
    assert out.shape == (9, 4, 64) and out.dtype == bf and lse.shape == (9, 4)
    assert kvc.kvc_prefill_attention_varlen(q, k, k, cu, cu, 5, 6, want_out=False)[0] is None
    for a, kw in (((q, k, k[:11], cu, cu, 5, 6), {}), ((q, k.float(), k, cu, cu, 5, 6), {}),
                  ((q, torch.empty((12, 2, 128), dtype=bf), k, cu, cu, 5, 6), {}), ((q, k, k, cu, cu[:2], 5, 6), {}),
                  ((q, k, k, cu.long(), cu, 5, 6), {}), ((q, k, k, cu, cu, 5, 6), dict(out=torch.empty((9, 4, 64)))),
                  ((q, k, k, cu, cu, 5, 6), dict(lse=torch.empty((4, 9)))),
                  ((q[:, :, ::2], k[:, :, ::2], k[:, :, ::2], cu, cu, 5, 6), {})):
        with pytest.raises((ValueError, TypeError)):
            kvc.kvc_prefill_attention_varlen(*a, **kw)


def test_paged_sizes_beyond_the_kernels_counters(clib):
    n = ctypes.byref(ctypes.c_size_t())
    big = _cache(batch=1024, page_size=256, max_pages=1 << 22, table_stride=1 << 22,  # room for 2^30 entries each
                 page_stride=1 << 15)
    c = ctypes.byref(big)
    assert clib.kvc_paged_decode_workspace_size(c, 2, (1 << 26) - 1024, 0, n) == 0
    assert clib.kvc_paged_decode_workspace_size(c, 2, (1 << 27), 0, n) == 1  # 2^37 entries
    assert clib.kvc_paged_decode_attention(c, PTR, 128, 64, 2, 0.125, 1 << 27, 0, PTR, None, PTR, 1 << 40, None,
                                           None) == 1
    wide = _cache(batch=1024, page_size=256, max_pages=1 << 22, table_stride=1 << 22, num_kv_heads=1 << 15,
                  page_stride=256 << 21)
    assert clib.kvc_paged_decode_workspace_size(ctypes.byref(wide), 1 << 15, 1 << 16, 0, n) == 1  # 2^41 of all heads
    over = ctypes.byref(_cache(page_size=256, max_pages=(1 << 22) + 1, table_stride=1 << 23, page_stride=1 << 15))
    assert clib.kvc_paged_append_workspace_size(over, n) == 1 and "2^30" in kvc.last_error()
