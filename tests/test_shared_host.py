"""Refusals of the shared-prefix calls, checked before anything is launched, and their
workspace sizes."""

import ctypes

import numpy as np
import pytest

from mixed_precision_bit_gb300 import kitty as K

A = 1 << 20  # a device address that is never used


@pytest.fixture(scope="module")
def lib():
    return K.load()


def _cfg(**kw):
    return K.Config(**{**dict(num_kv_heads=2, num_q_heads=8), **kw})


def _packed(lib, cfg=None, **kw):
    a = dict(q=A, pool=A, pp=4, pt=A, npre=3, pre=A, bt=A, mp=2, np=A, tk=A, tv=A, tl=A, sm=0.1, out=A, od=0,
             ws=A, wb=1 << 30, B=2, st=None, stream=None)
    a.update(kw)
    return lib.kitty_decode_attention_shared(ctypes.byref((cfg or _cfg()).c()), *a.values())


def _plain(lib, cfg=None, **kw):
    a = dict(q=A, pool=A, pp=4, pt=A, npre=3, pre=A, bt=A, mp=2, ln=A, sm=0.1, out=A, od=0, ws=A, wb=1 << 30,
             B=2, st=None, stream=None)
    a.update(kw)
    return lib.kitty_f16kv_decode_shared(ctypes.byref((cfg or _cfg()).c()), *a.values())


def test_refusals(lib):
    for call, extra in ((_packed, [dict(np=None), dict(tk=None), dict(tl=None), dict(tv=A + 8)]),
                        (_plain, [dict(ln=None)])):
        assert call(lib, B=0) == 0
        for kw in [dict(B=-1), dict(npre=-1), dict(mp=-1), dict(pp=-1), dict(q=None), dict(out=None), dict(pool=None),
                   dict(pool=A + 8), dict(pt=None), dict(bt=None), dict(od=3), dict(sm=float("nan")),
                   dict(sm=float("inf")), dict(q=A + 8)] + extra:
            assert call(lib, **kw) == -1, kw
        for kw in (dict(ws=None), dict(ws=A + 4), dict(wb=0), dict(wb=100)):
            assert call(lib, **kw) == -4, kw
        assert call(lib, cfg=_cfg(head_dim=64)) == -2
        assert call(lib, B=70000, wb=1 << 60) == -2
    assert _packed(lib, cfg=_cfg(num_kv_heads=1, num_q_heads=33)) == -2
    assert _plain(lib, cfg=_cfg(num_kv_heads=1, num_q_heads=5)) == -2


def test_workspace_bytes(lib):
    for size in (K.shared_workspace_bytes, K.f16kv_shared_workspace_bytes):
        cfg = _cfg()
        assert size(cfg, 0, 10, 10) == 0
        rows = 5 * 8 * 132 * 4
        n0 = size(cfg, 5, 0, 10)                      # no prefix: the own partials
        assert n0 >= 2 * rows and n0 % rows == 0
        n1 = size(cfg, 5, 100, 10)
        assert n1 > n0 and (n1 - n0) % rows == 0
        for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, -1)):
            with pytest.raises(K.KittyError) as e:
                size(cfg, *bad)
            assert e.value.code == -1


def test_binding_checks_shapes():
    import torch
    cfg = _cfg()
    out = torch.zeros(2, 8, 128)
    with pytest.raises(ValueError, match="must be"):
        K._attended(cfg, torch.zeros(2, 7, 128, dtype=torch.int16), out, 2, 0)
    with pytest.raises(ValueError, match="must be"):
        K._attended(cfg, torch.zeros(2, 8, 128), out, 2, 0)
    with pytest.raises(ValueError, match="block table"):
        K._table(torch.zeros(1, 4, dtype=torch.int32), 2, 0)
    with pytest.raises(ValueError, match="device memory"):
        K._attended(cfg, torch.zeros(2, 8, 128, dtype=torch.int16), out, 2, 0)


def _caches():
    from mixed_precision_bit_gb300.cache import F16LayerCache, LayerCache
    return [c(_cfg(), 3, 4, 16, device="cpu") for c in (LayerCache, F16LayerCache)]


def test_cache_refuses_a_bad_prefix_and_keeps_its_pages():
    import torch
    rows = lambda n, h=2, t=torch.int16: torch.zeros(n, h, 128, dtype=t)  # noqa: E731
    for lc in _caches():
        for k, v, of in ((rows(33), rows(33), None), (rows(32), rows(64), None), (rows(32, 3), rows(32, 3), None),
                         (rows(32, 2, torch.float32), rows(32), None), (rows(32), rows(32), [1, 1]),
                         (rows(32), rows(32), [0, 1, 2]), (rows(32), rows(32), [-1, 1, 1])):
            with pytest.raises(ValueError):
                lc.share_prefix(k, v, pages_of=of)
            assert lc.alloc.free_count == 16 and lc.prefix is None
        lc.plan_flush()                                   # the sequences hold a token now
        with pytest.raises(ValueError, match="hold tokens"):
            lc.share_prefix(rows(32), rows(32))
    from mixed_precision_bit_gb300.cache import LayerCache
    lc = LayerCache(_cfg(rank_mode=K.RANK_RUNNING), 3, 4, 16, device="cpu")
    with pytest.raises(ValueError, match="all of the prefix or none"):
        lc.share_prefix(rows(64), rows(64), pages_of=[2, 1, 0])
    assert lc.alloc.free_count == 16


def test_cache_plans_of_several_tokens():
    lc = _caches()[1]
    ids, start = lc.plan_extend([40, 0, 32])
    assert list(start) == [0, 40, 40, 72] and list(np.nonzero(ids >= 0)[0]) == [0, 32, 40]
    ids, start = lc.plan_extend([24, 1, 1])               # up to a page's end; a first token; a new page
    assert list(np.nonzero(ids >= 0)[0]) == [24, 25] and list(lc.h_len) == [64, 1, 33]
    free = lc.alloc.free_count
    for lens in ([65, 0, 0], [1, 1], [1, -1, 1]):
        with pytest.raises(ValueError):
            lc.plan_extend(lens)
    with pytest.raises(ValueError):
        lc.extend_rope(None, None, torch_rows(4), torch_rows(5), [1, 1, 2], None)
    assert lc.alloc.free_count == free and list(lc.h_len) == [64, 1, 33]


def torch_rows(n):
    import torch
    return torch.zeros(n, 2, 128, dtype=torch.int16)


def test_prefill_refuses_lengths_that_do_not_fit():
    lc = _caches()[0]
    for k, v, lens in ((torch_rows(3), torch_rows(3), [1, 1]), (torch_rows(3), torch_rows(3), [1, 1, 2]),
                       (torch_rows(3), torch_rows(2), [1, 1, 1]), (torch_rows(160), torch_rows(160), [160, 0, 0]),
                       (torch_rows(1), torch_rows(1), [2, -1, 0])):
        with pytest.raises(ValueError):
            lc.prefill_rope(None, None, k, v, lens, None)
    assert lc.alloc.free_count == 16


def test_caches_refuse_rows_of_the_other_16_bit_type():
    import torch
    from mixed_precision_bit_gb300.cache import F16LayerCache, LayerCache
    rows = lambda n, t: torch.zeros(n, 2, 128, dtype=t)  # noqa: E731
    for kind in (LayerCache, F16LayerCache):
        lc = kind(_cfg(in_dtype=K.BF16), 3, 4, 16, device="cpu")
        for k, v in ((torch.float16, torch.bfloat16), (torch.bfloat16, torch.float16)):
            with pytest.raises(ValueError, match="configuration has"):
                lc.share_prefix(rows(32, k), rows(32, v))
        assert lc.alloc.free_count == 16 and lc.prefix is None
    lc = LayerCache(_cfg(in_dtype=K.F16), 3, 4, 16, device="cpu")
    for t, match in ((torch.bfloat16, "configuration has"), (torch.float32, "16-bit")):
        with pytest.raises(ValueError, match=match):
            lc.prefill_rope(None, None, rows(3, torch.float16), rows(3, t), [1, 1, 1], None)
    assert lc.alloc.free_count == 16


def test_cleared_caches_have_their_pages_and_no_tokens():
    """clear gives back the pages of the sequences, of flushes that were planned and not made, and
    of a prefill over another; the prefix keeps its own."""
    import torch
    from mixed_precision_bit_gb300.cache import F16LayerCache, LayerCache
    for rank in (K.RANK_PAGE, K.RANK_RUNNING):
        for kind in (LayerCache, F16LayerCache):
            lc = kind(_cfg(rank_mode=rank), 3, 4, 16, device="cpu")
            packed = kind is LayerCache
            ids = lc.alloc.alloc(2)
            lc._set_prefix(ids, np.array([2, 0, 2], np.int32), True)
            if packed and rank:
                lc._prefix_stats = [torch.full((1,) + t.shape[1:], 3, dtype=t.dtype) for t in lc._stats()]
            lc.alloc.alloc(3)                             # an earlier prefill's, and a planned flush's
            lc.block_table[1, :2] = 7
            if packed:
                lc.h_pages[:], lc.h_tail[:] = [0, 2, 0], [31, 5, 0]
                lc.num_pages[1], lc.tail_len[0] = 2, 31
                for t in lc._stats():
                    t.fill_(9)
                lc.plan_flush()
            else:
                lc.h_len[:] = [64, 5, 0]
                lc.ctx_len[0] = 64
                lc.plan_flush()
            lc.clear()
            assert lc.alloc.free_count == 14 and lc.kv_tokens() == lc._prefix_tokens() == 4 * 32
            assert (lc.block_table == -1).all()
            assert sorted(lc.alloc.alloc(14).tolist() + ids.tolist()) == list(range(16))
            lc.alloc.free(np.setdiff1d(np.arange(16), ids))
            if packed:
                assert not lc.num_pages.any() and not lc.tail_len.any()
                for t in lc._stats():
                    assert (t[0] == 3).all() and (t[1] == 0).all() and (t[2] == 3).all()
                    t.fill_(9)
            else:
                assert not lc.ctx_len.any()
            lc.drop_prefix()
            assert lc.alloc.free_count == 16 and lc.kv_tokens() == 0
            if packed:
                for t in lc._stats():                     # of those that saw it
                    assert (t[0] == 0).all() and (t[1] == 9).all() and (t[2] == 0).all()
            lc.clear()
            assert lc.alloc.free_count == 16 and not (packed and any(t.any() for t in lc._stats()))


@pytest.mark.parametrize("rank", [K.RANK_PAGE, K.RANK_RUNNING])
def test_a_prefix_that_the_page_write_refuses_is_not_installed(rank):
    """The binding refuses host memory and rows with gaps (here everything is on the host): the
    cache is as before, and a corrected call is not refused for a prefix that is not there."""
    import torch
    from mixed_precision_bit_gb300.cache import F16LayerCache, LayerCache
    rows = torch.zeros(32, 4, 128, dtype=torch.int16)
    for kind in (LayerCache, F16LayerCache):
        lc = kind(_cfg(rank_mode=rank), 3, 4, 16, device="cpu")
        for k in (rows[:, :2].contiguous(), rows[:, :2]):  # a slice of a joint projection, too
            for _ in range(2):
                with pytest.raises(ValueError, match="tensor arguments must be"):
                    lc.share_prefix(k, k, pages_of=[1, 0, 1])
                assert lc.alloc.free_count == 16 and lc.kv_tokens() == 0
                assert lc.prefix is None and lc.prefix_pages is None and lc.pos_base is None
                assert np.sum(lc.h_prefix) == 0


def test_a_refused_extension_takes_no_pages():
    import torch
    lc = _caches()[1]
    rows = lambda h, t=torch.int16: torch.zeros(40, h, 128, dtype=t)  # noqa: E731
    rope = K.Rope(K.rope_frequencies(64)[0], device="cpu")
    for q, k, v, q_out in ((rows(8), rows(2), rows(2), rows(8)),              # host memory
                           (None, rows(2), rows(2, torch.float32), None),     # not 16-bit
                           (None, rows(4)[:, ::2], rows(2), None)):           # heads with gaps
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            lc.extend_rope(rope, q, k, v, [33, 0, 7], q_out)
        assert lc.alloc.free_count == 16 and list(lc.h_len) == [0, 0, 0]


def test_outgrown_workspaces_stay_allocated():
    """A captured step holds the addresses of the workspaces that it was captured with: a plan
    that needs more gets new ones beside them, few and not much larger than needed."""
    import gc
    import weakref
    import torch
    from mixed_precision_bit_gb300.cache import LayerCache
    lc = LayerCache(_cfg(), 3, 400, 1300, device="cpu")
    lc._set_prefix(lc.alloc.alloc(40), np.full(3, 40, np.int32), None)
    lc.set_plan_hint(3, 1)
    old = {}
    for total, most in ((3, 1), (30, 10), (300, 100), (900, 300), (30, 10), (1200, 400)):
        for ws in (lc.workspace, lc.shared_workspace):
            old[ws.data_ptr()] = weakref.ref(ws)
        del ws
        lc.set_plan_hint(total, most)
        cfg = _cfg(decode_total_pages=total, decode_max_pages=most)
        for ws, need in ((lc.workspace, K.decode_workspace_bytes(cfg, 3, 400)),
                         (lc.shared_workspace, K.shared_workspace_bytes(cfg, 3, 40, 400))):
            assert ws.numel() * ws.element_size() >= need
        del ws
        gc.collect()
        assert all(r() is not None for r in old.values())
    largest = lc.workspace.numel() + lc.shared_workspace.numel()
    assert len(lc._outgrown) >= 2 and sum(w.numel() for w in lc._outgrown) < largest
