"""Masks and positions of drafted trees, page tables on the device, and accepted paths into both
caches, against plain computations; whole numbers and bytes have to be equal."""

import numpy as np
import pytest

import oracle
from mixed_precision_bit_gb300 import synth
from tests.kitty_cases import dev16, dev32
from tests.tree_cases import D, P, dev64, masks_of, random_parents, starts

pytestmark = pytest.mark.gpu
BF16, F16 = synth.BF16, synth.F16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


def status0():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def host(t):
    return t.cpu().numpy()


# ------------------------------------------------------------------ masks and positions
def plan(parents, counts, pages, lens, base, pad=0, status=None, **kw):
    import torch
    from mixed_precision_bit_gb300 import kitty
    T = len(parents) + pad
    vis = torch.full((T,), 77, dtype=torch.int64, device="cuda")
    pos = torch.full((T,), 77, dtype=torch.int32, device="cuda")
    kitty.tree_plan(dev32(np.concatenate([parents, np.full(pad, -9)])), dev32(starts(counts)), dev32(lens), vis, pos,
                    num_pages=None if pages is None else dev32(pages), pos_base=None if base is None else dev32(base),
                    status=status, **kw)
    return host(vis).view(np.uint64), host(pos)


@pytest.mark.parametrize("counts,pad", [([1], 0), ([64], 0), ([0, 5, 64, 33, 1, 32, 0], 3), ([7] * 130, 5)])
@pytest.mark.parametrize("shape", ["random", "chain", "roots"])
def test_plan(counts, pad, shape):
    r = np.random.default_rng(1)
    make = dict(random=lambda n: random_parents(r, n), chain=lambda n: np.arange(-1, n - 1), roots=lambda n: np.full(n, -1))[shape]
    trees = [np.asarray(make(n), np.int32) for n in counts]
    B = len(counts)
    pages, lens, base = r.integers(0, 1000, B), r.integers(0, 32, B), r.integers(0, 5000, B)
    for pg, ba in ((pages, base), (None, None)):
        st = status0()
        vis, pos = plan(np.concatenate(trees), counts, pg, lens, ba, pad, st)
        at = 0
        for b, tree in enumerate(trees):
            m = masks_of(tree)
            held = lens[b] + (0 if pg is None else 32 * pages[b] + base[b])
            assert np.array_equal(vis[at:at + len(m)], m)
            assert np.array_equal(pos[at:at + len(m)], [held + bin(int(x)).count("1") - 1 for x in m])
            at += len(m)
        assert (vis[at:] == 77).all() and (pos[at:] == 77).all() and int(st.item()) == 0


def test_plan_bad_parents_and_starts():
    st = status0()
    vis, pos = plan(np.array([-1, 1, 0, 7, -2, 0], np.int32), [6], None, [10], None, 0, st)
    assert int(st.item()) == 12
    assert list(vis) == [1, 2, 5, 8, 16, 33] and list(pos) == [10, 10, 11, 10, 10, 11]
    from mixed_precision_bit_gb300 import kitty
    import torch
    for start, code in (([0, 4, 2, 6], 9), ([0, 2, 7, 9], 9), ([0, 2, -1, 6], 9)):
        st.zero_()
        vis = torch.zeros(6, dtype=torch.int64, device="cuda")
        kitty.tree_plan(dev32([-1] * 6), dev32(start), dev32([0, 0, 0]), vis, None, status=st)
        assert int(st.item()) == code and host(vis)[0] == 1
    st.zero_()
    vis = torch.zeros(70, dtype=torch.int64, device="cuda")
    kitty.tree_plan(dev32([-1] * 70), dev32([0, 65, 70]), dev32([0, 0]), vis, None, status=st)
    assert int(st.item()) == 5 and (host(vis)[:65] == 0).all() and (host(vis)[65:] != 0).all()


# ------------------------------------------------------------------ page tables
class Tables:
    """The operator's rules, one page at a time."""

    def __init__(self, pool, B, M, r=None):
        self.free = list(range(pool)) if r is None else [int(x) for x in r.permutation(pool)]
        self.pool, self.M = pool, M
        self.bt, self.held = np.full((B, M), -1, np.int32), np.zeros(B, np.int32)

    def step(self, tokens, partial, shrink):
        want = [(t + 31) // 32 if partial else t // 32 for t in tokens]
        ok = [w <= self.M for w in want]
        if shrink:
            for b in reversed(range(len(want))):
                while ok[b] and self.held[b] > want[b]:
                    self.held[b] -= 1
                    self.free.append(int(self.bt[b, self.held[b]]))
                    self.bt[b, self.held[b]] = -1
        left, out = len(self.free), True
        for b, w in enumerate(want):
            more = w - int(self.held[b])
            if not ok[b] or more <= 0:
                continue
            left -= more
            if left < 0:
                out = False
                continue
            for _ in range(more):
                self.bt[b, self.held[b]] = self.free.pop()
                self.held[b] += 1
        return 8 if not all(ok) else 0 if out else 11


def device_tables(h):
    import torch
    ids = np.zeros(h.pool, np.int32)
    ids[:len(h.free)] = h.free
    return dict(held=dev32(h.held), block_table=dev32(h.bt), free_ids=dev32(ids),
                free_count=torch.tensor([len(h.free)], dtype=torch.int32, device="cuda"))


def same_tables(t, h):
    n = int(t["free_count"].item())
    assert n == len(h.free) and list(host(t["free_ids"])[:n]) == h.free
    assert np.array_equal(host(t["held"]), h.held) and np.array_equal(host(t["block_table"]), h.bt)


@pytest.mark.parametrize("B,M,pool", [(1, 9, 9), (5, 40, 150), (64, 33, 1500), (1500, 6, 7000), (3, 700, 1500)])
@pytest.mark.parametrize("partial", [True, False])
def test_page_tables(B, M, pool, partial):
    """Random growth and shrinking, with and without enough free pages, against the rules."""
    from mixed_precision_bit_gb300 import kitty
    r = np.random.default_rng(B)
    h = Tables(pool, B, M, r)
    t = device_tables(h)
    lens = np.zeros(B, np.int64)
    seen = set()
    for step in range(14):
        lens = np.clip(lens + r.integers(-200, 260, B) * (r.random(B) < 0.7), 0, 32 * M + (40 if step == 9 else 0))
        new = np.minimum(r.integers(0, 40, B), np.maximum(32 * M - lens, 0))
        shrink = bool(step % 2)
        st = status0()
        split = r.integers(0, 2) == 0
        kitty.page_tables(dev32(lens % 32 if split else lens), num_pages=dev32(lens // 32) if split else None,
                          seq_start=dev32(starts(new)), partial=partial, shrink=shrink, status=st, **t)
        code = h.step(lens + new, partial, shrink)
        if code == 8:  # beside it pages may run out: the first to be seen is reported
            assert int(st.item()) in (8, 11)
        else:
            assert int(st.item()) == code
        seen.add(code)
        same_tables(t, h)
        lens = np.minimum(lens, 32 * M)
    assert 0 in seen


def test_page_tables_slots():
    from mixed_precision_bit_gb300 import kitty
    import torch
    r = np.random.default_rng(3)
    B, M = 9, 20
    h = Tables(100, B, M, r)
    t = device_tables(h)
    lens, new = r.integers(0, 300, B), r.integers(0, 150, B)
    new[4] = 0
    start = starts(new)
    T = int(start[-1]) + 6
    slots = torch.full((T,), -7, dtype=torch.int64, device="cuda")
    ids = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    st = status0()
    kitty.page_tables(dev32(lens), seq_start=dev32(start), slots=slots, new_page_ids=ids, status=st, **t)
    code = h.step(lens + new, True, False)
    assert int(st.item()) == code
    same_tables(t, h)
    s, i = host(slots), host(ids)
    for b in range(B):
        for k in range(new[b]):
            pos, at = lens[b] + k, start[b] + k
            page = h.bt[b, pos // 32] if pos // 32 < h.held[b] else -1
            assert s[at] == (-1 if page < 0 else 32 * page + pos % 32)
            assert i[at] == (page if pos % 32 == 0 else -1)
    assert (s[start[-1]:] == -7).all() and (i[start[-1]:] == -7).all()
    # a take and its give-back leave the stack as it was
    before = {k: v.clone() for k, v in t.items()}
    kitty.page_tables(dev32(lens), seq_start=dev32(start), extra=64, **t)
    kitty.page_tables(dev32(lens), seq_start=dev32(start), shrink=True, **t)
    n = int(t["free_count"].item())
    assert n == int(before["free_count"].item())
    assert torch.equal(t["free_ids"][:n], before["free_ids"][:n]) and torch.equal(t["block_table"], before["block_table"])


def test_page_tables_bad_state():
    from mixed_precision_bit_gb300 import kitty
    h = Tables(20, 4, 5)
    h.step([64, 64, 64, 64], True, False)
    t = device_tables(h)
    t["block_table"][1, 1] = 20           # an id out of range: sequence 1 keeps its row
    st = status0()
    kitty.page_tables(dev32([0, 0, 0, 64]), shrink=True, status=st, **t)
    assert int(st.item()) == 4
    assert list(host(t["held"])) == [0, 2, 0, 2] and list(host(t["block_table"])[1, :2]) == [h.bt[1, 0], 20]
    assert list(host(t["free_ids"])[:16]) == h.free + [int(x) for x in (h.bt[2, 1], h.bt[2, 0], h.bt[0, 1], h.bt[0, 0])]
    for name, value, code in (("held", 6, 5), ("held", -1, 5)):
        t = device_tables(h)
        t[name][2] = value
        st.zero_()
        kitty.page_tables(dev32([96] * 4), status=st, **t)
        assert int(st.item()) == code and list(host(t["held"])) == [3, 3, value, 3]
    for n in (-1, 21):
        t = device_tables(h)
        t["free_count"].fill_(n)
        st.zero_()
        kitty.page_tables(dev32([96] * 4), status=st, **t)
        assert int(st.item()) == 5 and np.array_equal(host(t["block_table"]), h.bt)
    t = device_tables(h)
    st.zero_()
    kitty.page_tables(dev32([96, -5, 96, 161]), status=st, **t)
    assert int(st.item()) in (5, 8) and list(host(t["held"])) == [3, 2, 3, 2]


# ------------------------------------------------------------------ accepted paths
def commit_inputs(r, dt, Hkv, Hq, counts, width, before, pad=2):
    rows = synth.to_bits(r.standard_normal((sum(counts) + pad, Hq + 2 * Hkv, D)), dt)
    n = np.array([int(r.integers(0, min(c, width) + 1)) for c in counts], np.int32)
    path = np.full((len(counts), width), 99, np.int32)
    for b, c in enumerate(counts):
        path[b, :n[b]] = np.sort(r.permutation(c)[:n[b]])
    return rows, path, n


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("n_hi,lo_bit,v_bit,dt", [(32, 2, 2, BF16), (0, 2, 2, F16), (16, 4, 2, BF16), (48, 4, 4, F16)])
@pytest.mark.parametrize("counted", [False, True])
def test_commit_packed(mode, n_hi, lo_bit, v_bit, dt, counted):
    """Every byte of the cache as token-by-token appends leave it, over several steps."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    r = np.random.default_rng(5)
    Hkv, Hq, M = 2, 4, 12
    counts = [64, 9, 1, 33, 0, 64]
    B = len(counts)
    cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, n_hi=n_hi, in_dtype=dt, hi_bit=2 * lo_bit, lo_bit=lo_bit,
                       v_bit=v_bit, rank_mode=mode)
    blob, per_page = kitty.page_bytes(cfg)
    pool_pages = B * M
    bt = r.permutation(pool_pages).reshape(B, M).astype(np.int32)   # every page reserved
    st = dict(pool=np.zeros(pool_pages * per_page, np.uint8), num_pages=np.zeros(B, np.int32),
              tail_k=np.zeros((B, Hkv, P, D), np.uint16), tail_v=np.zeros((B, Hkv, P, D), np.uint16),
              tail_len=np.array([31, 30, 0, 5, 17, 0], np.int32), run=np.zeros((B, Hkv, D), np.float32),
              run2=np.zeros((B, Hkv, D), np.float32), cnt=np.zeros((B, Hkv), np.int32))
    dev = {k: torch.from_numpy((v.view(np.int16) if v.dtype == np.uint16 else v).copy()).cuda() for k, v in st.items()}
    status = status0()
    for step in range(4):
        rows, path, n = commit_inputs(r, dt, Hkv, Hq, counts, 64, st["tail_len"])
        if step == 0:
            n[0] = 64
            path[0] = np.arange(64)
        start = starts(counts)
        d = dev16(rows)
        old = st["num_pages"].copy(), st["tail_len"].copy()
        # the oracle, token by token; a sequence without one more token sits that step out
        for i in range(64):
            for b in np.nonzero(n > i)[0]:
                row = start[b] + path[b, i]
                fl = np.array([bt[b, st["num_pages"][b]] if st["tail_len"][b] == 31 else -1], np.int32)
                part = {k: (v if k == "pool" else v[b:b + 1]) for k, v in st.items()}
                table = bt[b:b + 1].copy()
                rc = oracle.append_token(Hkv, n_hi, mode, dt, rows[row:row + 1, Hq:Hq + Hkv].copy(),
                                         rows[row:row + 1, Hq + Hkv:].copy(), part["tail_k"], part["tail_v"],
                                         part["tail_len"], part["run"], part["run2"], part["cnt"], fl, table, M,
                                         part["num_pages"], part["pool"], pool_pages, lo_bit=lo_bit, v_bit=v_bit)
                assert rc == 0
        if counted:
            dev["num_pages"].copy_(torch.from_numpy(st["num_pages"]))
            dev["tail_len"].copy_(torch.from_numpy(st["tail_len"]))
        run = (dev["run"], dev["run2"], dev["cnt"]) if mode else (None, None, None)
        kitty.tree_commit(cfg, d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], dev32(start), dev32(path), dev32(n), dev["tail_k"],
                          dev["tail_v"], dev["tail_len"], *run, dev32(bt), dev["num_pages"], dev["pool"], pool_pages,
                          counted=counted, status=status)
        assert int(status.item()) == 0
        for k, v in st.items():
            if mode or k not in ("run", "run2", "cnt"):
                assert np.array_equal(host(dev[k]).view(np.uint8), v.view(np.uint8)), (step, k)
        assert not np.array_equal(old[0], st["num_pages"]) or not np.array_equal(old[1], st["tail_len"])


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("counted", [False, True])
def test_commit_plain16(dt, counted):
    import torch
    from mixed_precision_bit_gb300 import kitty
    r = np.random.default_rng(6)
    Hkv, Hq, M = 3, 6, 9
    counts = [64, 9, 1, 33, 0, 64]
    B = len(counts)
    cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, in_dtype=dt)
    pool_pages = B * M
    bt = r.permutation(pool_pages).reshape(B, M).astype(np.int32)
    lens = np.array([31, 30, 0, 65, 17, 0], np.int64)
    pool = synth.to_bits(r.standard_normal((pool_pages, Hkv, 2, P, D)), dt)
    d_pool, d_lens, status = dev16(pool), dev32(lens), status0()
    for step in range(3):
        rows, path, n = commit_inputs(r, dt, Hkv, Hq, counts, 40, None)
        if step == 1:
            path[3, :3], n[3] = [5, 5, 2], 3                      # the same node twice, any order
        start = starts(counts)
        for b in range(B):
            for i in range(n[b]):
                pos = lens[b] + i
                row = rows[start[b] + path[b, i]]
                pool[bt[b, pos // 32], :, 0, pos % 32] = row[Hq:Hq + Hkv]
                pool[bt[b, pos // 32], :, 1, pos % 32] = row[Hq + Hkv:]
        lens = lens + n
        if counted:
            d_lens.copy_(dev32(lens))
        d = dev16(rows)
        kitty.f16kv_tree_commit(cfg, d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], dev32(start), dev32(path), dev32(n), d_pool,
                                pool_pages, dev32(bt), d_lens, counted=counted, status=status)
        assert int(status.item()) == 0
        assert np.array_equal(host(d_pool).view(np.uint16), pool) and np.array_equal(host(d_lens), lens)


def test_commit_refuses_whole_sequences():
    """Each fault is that of sequence 1: it keeps everything, the others are appended to."""
    import torch
    from mixed_precision_bit_gb300 import kitty
    r = np.random.default_rng(7)
    Hkv, Hq, M, B = 1, 2, 4, 3
    for packed in (True, False):
        cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq)
        blob, per_page = (kitty.page_bytes if packed else kitty.f16kv_page_bytes)(cfg)
        for fault, code in (("node", 12), ("count", 12), ("page", 4), ("full", 8), ("length", 5), ("starts", 9)):
            rows = dev16(synth.to_bits(r.standard_normal((15, Hq + 2 * Hkv, D)), BF16))
            start, n = np.array([0, 5, 10, 15], np.int32), np.array([3, 4, 5], np.int32)
            path = np.tile(np.arange(5, dtype=np.int32), (B, 1))
            bt = np.arange(B * M, dtype=np.int32).reshape(B, M)
            pages, tail, lens = np.array([1, 1, 1]), np.array([30, 30, 3]), np.array([62, 62, 35])
            if fault == "node":
                path[1, 2] = 5
            if fault == "count":
                n[1] = 6
            if fault == "page":
                bt[1, 1] = B * M
            if fault == "full":
                pages[1], lens[1] = 4, 126
            if fault == "length":
                pages[1], lens[1] = 5, 130
            if fault == "starts":
                start[2] = 4
            pool = torch.zeros(B * M * per_page, dtype=torch.uint8, device="cuda")
            tk = torch.zeros((B, Hkv, P, D), dtype=torch.int16, device="cuda")
            tv, st = torch.zeros_like(tk), status0()
            d_pages, d_tail, d_lens = dev32(pages), dev32(tail), dev32(lens)
            if packed:
                kitty.tree_commit(cfg, rows[:, 2:3], rows[:, 3:], dev32(start), dev32(path), dev32(n), tk, tv, d_tail,
                                  None, None, None, dev32(bt), d_pages, pool, B * M, status=st)
                want = [(2, 1), (pages[1], tail[1]), (1, 8)]
                assert [tuple(x) for x in zip(host(d_pages), host(d_tail))] == want, fault
                assert not tk[1].any() and tk[0].any() and tk[2].any()
            else:
                kitty.f16kv_tree_commit(cfg, rows[:, 2:3], rows[:, 3:], dev32(start), dev32(path), dev32(n), pool,
                                        B * M, dev32(bt), d_lens, status=st)
                assert list(host(d_lens)) == [65, lens[1], 40], fault
                assert not pool.view(B, -1)[1].any() and pool.view(B, -1)[0].any()
            assert int(st.item()) == code, (packed, fault)
