"""The operators on drafted trees together, as a server uses them: prompts from the projections, then
steps of drafting (masks and positions, norm and rotation, attention, pages, the accepted path), whole
steps captured into a graph or not, against caches that append the accepted tokens one by one.  Pages,
tails, statistics and lengths have to be the same bytes.

Outputs: the weights of a row sum to 1, so rounding each p to fp16 (2^-11) moves an output by at most
2^-11 max|v - out| <= 2^-10 max|v|, and rounding the middles of groups of Values by 2^-11 max|v|; scores
are off by what fp32 sums of fp16 products are (2^-19 of |q||k| here, below 2^-11): in all 2^-9 max|v|.
The decode that it is compared with is within 2e-3 of the outputs' RMS."""

import numpy as np
import pytest

from mixed_precision_bit_gb300 import synth
from tests.test_gpu_prefix_cache import _rope
from tests.tree_cases import masks_of, random_parents

pytestmark = pytest.mark.gpu
P, D = 32, 128
B, Hkv, Hq, NP, NODES, WIDTH = 4, 2, 8, 3, 11, 6
OWN = np.array([40, 0, 95, 31])


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_bit_gb300 import kitty
    kitty.load()


def _make(kind, cfg, n, max_pages, pool):
    from mixed_precision_bit_gb300 import cache
    return (cache.LayerCache if kind == "packed" else cache.F16LayerCache)(cfg, n, max_pages, pool)


def _prompt(c, rope, q, k, v, lens):
    import torch
    if lens.sum() == 0:
        return
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    (c.prefill_rope if hasattr(c, "tail_k") else c.extend_rope)(rope, q, k, v, lens, out)


def _path(r, tree):
    """A random way from a root down: places in the tree."""
    at, path = -1, []
    while len(path) < WIDTH:
        below = np.nonzero(tree == at)[0]
        if below.size == 0 or (path and r.random() < 0.15):
            break
        at = int(r.choice(below))
        path.append(at)
    return path if r.random() < 0.85 else []


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("shared", [0, NP], ids=["alone", "shared"])
@pytest.mark.parametrize("kind,rank", [("packed", 0), ("packed", 1), ("plain", 0)], ids=["page", "running", "16"])
def test_steps_of_drafting(kind, rank, shared, graph):
    import torch
    from mixed_precision_bit_gb300 import kitty
    torch.manual_seed(3)
    r = np.random.default_rng(17)
    rope, t = _rope(synth.BF16)
    cfg = kitty.Config(num_kv_heads=Hkv, num_q_heads=Hq, in_dtype=synth.BF16, rank_mode=rank, n_hi=16)
    max_pages = 8
    a = _make(kind, cfg, B, max_pages, shared + B * max_pages)
    alone = [_make(kind, cfg, 1, max_pages, shared + max_pages) for _ in range(B)]

    def rows(n):
        x = torch.randn(n, Hq + 2 * Hkv, D, device="cuda").to(t)
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]

    if shared:
        _, pk, pv = rows(shared * P)
        rot = torch.empty(shared * P, Hkv, D, dtype=t, device="cuda")
        kitty.norm_rope(cfg, rope, None, pk, torch.arange(shared * P, dtype=torch.int32, device="cuda"), None, rot)
        for c in (a, *alone):
            c.share_prefix(rot, pv.contiguous())
    q, k, v = rows(int(OWN.sum()))
    _prompt(a, rope, q, k, v, OWN)
    at = 0
    for b, c in enumerate(alone):
        _prompt(c, rope, q[at:at + OWN[b]], k[at:at + OWN[b]], v[at:at + OWN[b]], OWN[b:b + 1])
        at += OWN[b]

    a.pages_to_device()
    with pytest.raises(ValueError, match="on the device"):
        a.plan_flush()
    n = B * NODES
    ints = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device="cuda")
    parents, start, pos, path, length = ints(n), ints(B + 1), ints(n), ints(B, WIDTH), ints(B)
    visible = torch.zeros(n, dtype=torch.int64, device="cuda")
    buf = torch.zeros(n, Hq + 2 * Hkv, D, dtype=t, device="cuda")
    q_rot, k_rot = (torch.empty(n, h, D, dtype=t, device="cuda") for h in (Hq, Hkv))
    out = torch.zeros(n, Hq, D, device="cuda")

    def step():
        a.plan_trees(parents, start, visible, pos)
        kitty.norm_rope(cfg, rope, buf[:, :Hq], buf[:, Hq:Hq + Hkv], pos, q_rot, k_rot)
        a.attend_tree(q_rot, k_rot, buf[:, Hq + Hkv:], start, visible, NODES, out)
        a.reserve(WIDTH)
        a.commit_tree(k_rot, buf[:, Hq + Hkv:], start, path, length)

    captured = None
    for turn in range(14):
        counts = r.integers(1, NODES + 1, B)
        trees = [random_parents(r, c) for c in counts]
        first = np.concatenate([[0], np.cumsum(counts)])
        paths = [_path(r, tree) for tree in trees]
        flat = np.full(n, -1, np.int32)
        flat[:first[-1]] = np.concatenate(trees)
        table = np.zeros((B, WIDTH), np.int32)
        for b in range(B):
            table[b, :len(paths[b])] = paths[b]
        for dev, val in ((parents, flat), (start, first), (path, table), (length, [len(x) for x in paths])):
            dev.copy_(torch.from_numpy(np.asarray(val, np.int32)))
        buf.copy_(torch.randn(n, Hq + 2 * Hkv, D, device="cuda").to(t))
        held = [int(c.h_tail[0]) if kind == "packed" else 0 for c in alone]
        if not graph or turn == 0:
            step()  # (the workspace is made here)
        else:
            if captured is None:
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured):
                    step()
            captured.replay()
        seen = visible.cpu().numpy().view(np.uint64)
        for b, c in enumerate(alone):
            assert np.array_equal(seen[first[b]:first[b + 1]], masks_of(trees[b]))
            for i, node in enumerate(paths[b]):
                row = buf[first[b] + node:first[b] + node + 1]
                one, got = torch.empty(1, Hq, D, dtype=t, device="cuda"), torch.empty(1, Hq, D, device="cuda")
                ids = torch.from_numpy(c.plan_flush()).cuda()
                c.step_rope(rope, row[:, :Hq], row[:, Hq:Hq + Hkv].contiguous(), row[:, Hq + Hkv:].contiguous(), ids, one, got)
                assert torch.equal(one[0], q_rot[first[b] + node])
                if held[b] + i + 1 < P or kind == "plain":  # (from there on its page is quantized)
                    off = (out[first[b] + node] - got[0]).abs().max().item()
                    assert off <= 2 ** -9 * 5.5 + 2e-3 * got.square().mean().sqrt().item(), (turn, b, i, off)
    assert buf.abs().max().item() < 5.5 and int(a.status.item()) == 0 and all(int(c.status.item()) == 0 for c in alone)

    a.pages_to_host()
    with pytest.raises(ValueError, match="on the host"):
        a.reserve(1)
    used, pool = shared, a.pool.view(-1, a.per_page)
    for b, c in enumerate(alone):
        if kind == "packed":
            assert a.h_pages[b] == c.h_pages[0] and a.h_tail[b] == c.h_tail[0]
            full, m = int(c.h_pages[0]), int(c.h_tail[0])
            assert torch.equal(a.tail_k[b, :, :m], c.tail_k[0, :, :m]) and torch.equal(a.tail_v[b, :, :m], c.tail_v[0, :, :m])
            for x, y in ((a.run_sum, c.run_sum), (a.run_sumsq, c.run_sumsq), (a.run_count, c.run_count)):
                assert x is None or torch.equal(x[b], y[0])
            mine = pool[a.block_table[b, :full].long()]
            assert torch.equal(mine, c.pool.view(-1, c.per_page)[c.block_table[0, :full].long()])
            used += full
        else:
            assert a.h_len[b] == c.h_len[0]
            size = int(c.h_len[0])
            full = (size + P - 1) // P
            x, y = (z.pool.view(-1, z.per_page)[z.block_table[i, :full].long()].view(full, Hkv, 2, P, -1).transpose(1, 3)
                    .reshape(full * P, -1)[:size] for z, i in ((a, b), (c, 0)))
            assert torch.equal(x, y)
            used += full
    assert a.alloc.free_count == a.pool_pages - used
    # and the host goes on
    q, k, v = rows(B)
    one, got = torch.empty(B, Hq, D, dtype=t, device="cuda"), torch.empty(B, Hq, D, device="cuda")
    a.step_rope(rope, q, k.contiguous(), v.contiguous(), torch.from_numpy(a.plan_flush()).cuda(), one, got)
    for b, c in enumerate(alone):
        mine = torch.empty(1, Hq, D, device="cuda")
        c.step_rope(rope, q[b:b + 1], k[b:b + 1].contiguous(), v[b:b + 1].contiguous(), torch.from_numpy(c.plan_flush()).cuda(),
                    one[:1], mine)
        assert (got[b] - mine[0]).abs().max().item() <= 4e-3 * mine.square().mean().sqrt().item()
    if captured is None:
        return
    # the captured step after another hand-over: the last paths once more, behind what the host appended
    before = [int(x) for x in (a.h_len if kind == "plain" else a.h_pages * P + a.h_tail)]
    a.pages_to_device()
    captured.replay()
    a.pages_to_host()
    after = [int(x) for x in (a.h_len if kind == "plain" else a.h_pages * P + a.h_tail)]
    assert after == [x + len(y) for x, y in zip(before, paths)] and int(a.status.item()) == 0
    held = a.h_pages if kind == "packed" else (a.h_len + P - 1) // P
    assert a.alloc.free_count == a.pool_pages - shared - int(held.sum())
    ids = np.concatenate([a.block_table[b, :held[b]].cpu().numpy() for b in range(B)])
    assert (ids >= 0).all() and np.unique(ids).size == ids.size
