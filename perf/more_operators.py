"""Cases of the operators of a step of drafted tokens on the paged caches.

* ``plan``: ancestor masks and positions of trees of drafted tokens (``kitty.tree_plan``);
* ``pages``: block tables and slot maps from lengths, with the free pages on the device: room for a
  step's new tokens, then what the step did not keep given back (``kitty.page_tables``);
* ``tree``: attention of the drafted tokens to the packed cache and to each other
  (``kitty.tree_attention``), also behind a shared prefix;
* ``tree16``: the same on 16-bit pages (``kitty.f16kv_tree_attention``);
* ``commit``: the accepted path's keys and values into the packed cache, full tails quantized
  (``kitty.tree_commit``);
* ``commit16``: the same into 16-bit pages (``kitty.f16kv_tree_commit``).

``run`` computes each in elementary torch operations, or, with ``own``, by the framework's calls.
"""

import math

import torch

own = False

D = 128     # channels of a head
PAGE = 32   # tokens of a page
MOST = 64   # nodes of a tree
SCALE = 1.0 / math.sqrt(D)

_CASES = [
    # 16 small trees between the draft's pass and the verification: latency
    dict(name="plan 16x8", op="plan", B=16, nodes=8, ragged=False, kind="tree", pad=0),
    # a large batch of ragged trees, padding rows behind the last
    dict(name="plan 512x64", op="plan", B=512, nodes=64, ragged=True, kind="tree", pad=37),
    # a decode step of 64 sequences with 16 drafted tokens each
    dict(name="pages step 64", op="pages", B=64, far=8192, new=16, ragged=False, spare=64, pad=0),
    # a batch that admits 256 ragged prompts of up to 2048 tokens
    dict(name="pages prompts 256", op="pages", B=256, far=64, new=2048, ragged=True, spare=1024, pad=5),
    # four short chats, a chain of up to five drafted tokens each: the smallest call
    dict(name="tree chain 4x1024", op="tree", B=4, nodes=5, ragged=True, kind="chain", ctx=1024, prefix=0,
         Hq=32, Hkv=8, n_hi=32, dtype="bf16", pad=0),
    # 64 sequences near 8192 tokens, a tree of 16 nodes each
    dict(name="tree 64x8192", op="tree", B=64, nodes=16, ragged=False, kind="tree", ctx=8192, prefix=0,
         Hq=32, Hkv=8, n_hi=16, dtype="bf16", pad=0),
    # eight documents of up to 32768 tokens, trees of 64 nodes, a 64/8-head layer
    dict(name="tree 8x32768", op="tree", B=8, nodes=64, ragged=False, kind="tree", ctx=32768, prefix=0,
         Hq=64, Hkv=8, n_hi=32, dtype="bf16", pad=0),
    # 32 answers of a few hundred tokens behind one 4096-token prompt, ragged trees
    dict(name="tree 32 behind 4096", op="tree", B=32, nodes=12, ragged=True, kind="tree", ctx=320,
         prefix=128, Hq=32, Hkv=8, n_hi=32, dtype="fp16", pad=3),
    # 32 sequences near 8192 tokens in 16-bit pages, a tree of 16 nodes each
    dict(name="tree16 32x8192", op="tree16", B=32, nodes=16, ragged=False, kind="tree", ctx=8192, prefix=0,
         Hq=32, Hkv=8, dtype="bf16", pad=0),
    # an odd batch of a small layer in 16-bit pages, any masks (rows that see nothing among the drafts)
    dict(name="tree16 33x1950", op="tree16", B=33, nodes=27, ragged=True, kind="any", ctx=1950, prefix=0,
         Hq=6, Hkv=2, dtype="fp16", pad=2),
    # up to 8 accepted of 16 drafted tokens of 64 sequences, into the packed cache
    dict(name="commit 64", op="commit", B=64, nodes=16, accept=8, far=8192, Hq=32, Hkv=8, n_hi=32,
         dtype="bf16", pad=0),
    # the same of 128 sequences of trees of 64 nodes, into 16-bit pages
    dict(name="commit16 128", op="commit16", B=128, nodes=64, accept=12, far=8192, Hq=32, Hkv=8,
         dtype="bf16", pad=0),
]


def listed():
    return [dict(c) for c in _CASES]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "pages", "tree", "tree", "tree", "tree16", "tree16", "commit", "commit16"])
    c = dict(op=op, B=_log(rng, 1, 256), pad=rng.choice([0, 5]))
    if op == "pages":
        c.update(far=_log(rng, 32, 16384), new=rng.choice([1, _log(rng, 2, 2048)]), ragged=rng.random() < 0.5,
                 spare=rng.randint(0, 2048))
        return c
    c.update(nodes=_log(rng, 1, MOST))
    if op == "plan":
        c.update(ragged=rng.random() < 0.5, kind="tree")
        return c
    Hkv = rng.choice([1, 2, 4, 5, 8])
    c.update(Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 3, 4, 6, 8]), dtype=rng.choice(["bf16", "fp16"]))
    if op in ("tree", "commit"):
        c["n_hi"] = rng.choice([0, 16, 32, 64, 128])
    if op in ("commit", "commit16"):
        c.update(accept=rng.randint(1, c["nodes"]), far=_log(rng, 32, 16384))
        return c
    c.update(B=_log(rng, 1, 64), ragged=rng.random() < 0.5, kind=rng.choice(["tree", "chain", "any"]),
             ctx=_log(rng, 1, 16384), prefix=rng.choice([0, 0, _log(rng, 1, 128)]))
    # no more tokens than the largest listed cases hold, and no more products
    c["ctx"] = max(1, min(c["ctx"], (1 << 22) // (c["B"] * Hkv), (1 << 27) // (c["B"] * c["nodes"] * c["Hq"])))
    return c


# ------------------------------------------------------------------ inputs
def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _int(gen, lo, hi, *shape):
    """Whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda")


def _i32(x):
    return x.to(torch.int32).contiguous()


def _trees(case, gen):
    """Ragged trees: starts of the rows, parents, and ancestor masks (None: every tree is a chain)."""
    B, N = case["B"], case["nodes"]
    n = _int(gen, 0, N, B) if case.get("ragged") else torch.full((B,), N, device="cuda")
    n[0] = N
    start = torch.cat([n.new_zeros(1), n.cumsum(0)])
    T = B * N + case["pad"]
    node = torch.arange(N, device="cuda")
    straight = torch.rand((B, N), generator=gen, device="cuda") < 0.6
    some = (torch.rand((B, N), generator=gen, device="cuda") * (node + 1)).long().minimum(node) - 1
    parent = torch.where(straight, node - 1, some)
    kind = case.get("kind", "tree")
    if kind == "chain":
        parent = (node - 1).expand(B, N)
    mask = torch.zeros((B, N), dtype=torch.int64, device="cuda")
    rows = torch.arange(B, device="cuda")
    for i in range(N):
        above = torch.where(parent[:, i] >= 0, mask[rows, parent[:, i].clamp(min=0)], 0)
        mask[:, i] = above | (-1 << 63 if i == 63 else 1 << i)
    if kind == "any":  # any bits, a quarter of the rows none
        bits = (torch.rand((B, N, MOST), generator=gen, device="cuda") < 0.4).long()
        some = (bits << torch.arange(MOST, device="cuda")).sum(-1)
        mask = torch.where(torch.rand((B, N), generator=gen, device="cuda") < 0.25, 0, some)
    b, i, real = _places(start, T, B, N)
    where = lambda x, other: torch.where(real, x[b, i], other)  # noqa: E731
    return dict(start=_i32(start), parents=_i32(where(parent, -1)),
                visible=None if kind == "chain" else where(mask, 0).contiguous())


def _places(start, T, B, N):
    """Of T rows: their sequence, their place in it, and whether they are one's at all."""
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(start[1:].long().contiguous(), t, right=True)
    real = b < B
    b = b.clamp(max=B - 1)
    return b, (t - start[b].long()).clamp(0, N - 1), real


def _rows(gen, case, T, sigma):
    """The projections of T tokens, as one matrix: query, key and value heads side by side."""
    Hq, Hkv = case["Hq"], case["Hkv"]
    x = torch.randn((T, Hq + 2 * Hkv, D), generator=gen, device="cuda")
    x[:, Hq:Hq + Hkv] *= sigma
    x = x.to(_type(case))
    return x, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _pack(codes):
    """32-bit words of 16 two-bit codes: [.., e, half, tau] (2, 2, 4) at bit 16e + 8half + 2tau + 2."""
    e, h, t = (torch.arange(n, device="cuda") for n in (2, 2, 4))
    bit = (16 * e[:, None, None] + 8 * h[None, :, None] + 2 * t[None, None, :] + 2) % 32
    w = (codes.long() << bit).flatten(-3).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _steps(s):
    """Quantization steps rounded up to seven significant bits and to what fp16 holds."""
    v = ((s.contiguous().view(torch.int32) + 0x1FFFF) & ~0x1FFFF).view(torch.float32)
    h = v.half()
    return torch.where(h.float() < v, (h.view(torch.int16) + 1).view(torch.float16), h)


def _halved(x):
    n = x.shape[1] // 2
    return x[:, :n] + x[:, n:]


def _total(x):
    """Sums over the 32 tokens of dimension 1, the upper half onto the lower, and so on."""
    return _halved(_halved(_halved(_halved(_halved(x)))))[:, 0]


def _codes(x, M, unit, levels):
    code = torch.round((x - M.float()) * (1.0 / unit)).clamp(min=0).minimum(levels)
    return torch.where(unit == 0, 0.0, code).to(torch.int32)


def _quantized(k, v, n_hi):
    """Packed pages, uint8 [n, blob], of fp32 Keys and Values [n, 32, 128]: 2-bit Key channels with
    the n_hi of largest variance at 4 bits (two planes), 2-bit Values in groups of 32 channels.
    Every step in fp32, rounded once."""
    n = k.shape[0]
    mn, mx = k.amin(1), k.amax(1)
    mean = _total(k) / 32.0
    order = (_total(k * k) / 32.0 - mean * mean).argsort(dim=1, descending=True, stable=True)
    ch = order[:, :n_hi].sort(dim=1).values
    boost = torch.zeros((n, D), dtype=torch.bool, device="cuda").scatter_(1, ch, True)
    levels = torch.where(boost, 15.0, 3.0)
    S = _steps((mx - mn) / levels * torch.where(boost, 4.0, 1.0))
    unit = S.float() * torch.where(boost, 0.25, 1.0)
    M = mn.half()
    code = _codes(k, M[:, None], unit[:, None], levels[:, None])
    hi = torch.where(boost[:, None], code >> 2, code)
    key = lambda x: _pack(x.view(n, 4, 8, -1, 2, 4, 2).permute(0, 2, 5, 3, 6, 4, 1)).flatten(1)  # noqa: E731
    base = key(hi)
    lo = (code & 3).gather(2, ch[:, None].expand(n, PAGE, n_hi))
    extra = key(lo) if n_hi else base[:, :0]
    vg = v.view(n, PAGE, 4, 32)
    vmin, vmax = vg.amin(3), vg.amax(3)
    vS, vM = _steps((vmax - vmin) / 3.0), vmin.half()
    vcode = _codes(vg, vM[..., None], vS.float()[..., None], torch.full_like(vS.float()[..., None], 3.0))
    val = _pack(vcode.view(n, 2, 2, 4, 2, 4, 4, 8).permute(0, 7, 3, 5, 1, 4, 2, 6)).flatten(1)
    chan = lambda x: x.view(n, 8, 2, 4, 2).permute(0, 3, 1, 2, 4).flatten(1)  # noqa: E731
    meta = lambda x: x.permute(0, 2, 1).reshape(n, 4, 2, 2, 4, 2).permute(0, 1, 4, 2, 3, 5).flatten(1)  # noqa: E731
    ids = ch.to(torch.uint8).view(n, n_hi // 16, 2, 4, 2).permute(0, 1, 3, 2, 4).flatten(1)
    parts = [base, extra, S, chan(M), ids, val, meta(vS), meta(vM)]
    return torch.cat([p.contiguous().view(torch.uint8).view(n, -1) for p in parts], 1)


def _blob(n_hi):
    """Bytes of one (page, kv head): two code planes of 1024, four rows of 256, and 9 a boosted channel."""
    return 2 * 1024 + 4 * 256 + 9 * n_hi


def _sigma(gen, case):
    """The spread of each Key channel: some are far wider than the rest."""
    return torch.exp(torch.randn((case["Hkv"], D), generator=gen, device="cuda"))


def _table(gen, held, first, total=None):
    """A shuffled pool's block table [B, most + 1] of held[b] pages a row, behind `first` pages that
    no row has, of `total` pages (default: no others); -1 elsewhere.  (table, all the ids in order)."""
    most = int(held.max())
    total = first + int(held.sum()) if total is None else total
    ids = torch.randperm(max(total, 1), generator=gen, device="cuda")
    at = torch.arange(most + 1, device="cuda")[None]
    place = (first + held.cumsum(0) - held)[:, None] + at
    table = torch.where(at < held[:, None], ids[place.clamp(max=max(total, 1) - 1)], -1)
    return _i32(table), _i32(ids)


def _prepare_attention(case, gen):
    B, Hkv, P = case["B"], case["Hkv"], case["prefix"]
    packed, dt = case["op"] == "tree", _type(case)
    st = dict(case=case, **_trees(case, gen))
    T = st["parents"].numel()
    sigma = _sigma(gen, case)
    st["rows"], st["q"], st["k"], st["v"] = _rows(gen, case, T, sigma)
    st["out"] = torch.zeros((T, case["Hq"], D), dtype=dt, device="cuda")
    # lengths of a batch: half to all of ctx, one in eight a request that has just come
    ctx = _int(gen, (case["ctx"] + 1) // 2, case["ctx"], B)
    ctx[7::8] = 0
    held = ctx // PAGE if packed else (ctx + PAGE - 1) // PAGE
    bt, ids = _table(gen, held, P)
    total = ids.numel()
    st.update(block_table=bt, pool_pages=total, prefix_table=ids[:P].contiguous() if P else None)

    def tokens(*shape):
        k = torch.randn(shape, generator=gen, device="cuda") * sigma[:, None]
        return k.to(dt), torch.randn(shape, generator=gen, device="cuda").to(dt)

    k, v = tokens(total, Hkv, PAGE, D)
    if packed:
        blobs = _quantized(k.float().view(-1, PAGE, D), v.float().view(-1, PAGE, D), case["n_hi"])
        st["tail_k"], st["tail_v"] = tokens(B, Hkv, PAGE, D)
        st.update(pool=blobs.view(total, Hkv, -1), num_pages=_i32(held), tail_len=_i32(ctx % PAGE))
    else:
        st.update(pool=torch.stack([k, v], 2), ctx_len=_i32(ctx))
    return st


def _prepare_commit(case, gen):
    """Lengths that count the accepted tokens already, as every layer after the first finds them."""
    B, N, Hkv, dt = case["B"], case["nodes"], case["Hkv"], _type(case)
    packed = case["op"] == "commit"
    st = dict(case=case, **_trees(dict(case, kind="tree", ragged=False), gen))
    T = st["parents"].numel()
    _, _, st["k"], st["v"] = _rows(gen, case, T, _sigma(gen, case))
    W = min(N, case["accept"])
    n = _int(gen, 0, W, B)
    path = torch.rand((B, N), generator=gen, device="cuda").argsort(1)[:, :W].sort(1).values
    have = _int(gen, 0, case["far"], B)
    before, after = have % PAGE, have % PAGE + n
    if not packed:
        # the pages that the new tokens lie in; what is before them is not touched
        first, last = have // PAGE, (have + n + PAGE - 1) // PAGE
        M = int(last.max()) + 1
        here, ids = _table(gen, last - first, 1, 1 + B * (W // PAGE + 2))
        at = torch.arange(M, device="cuda")[None] - first[:, None]
        bt = torch.where((at >= 0) & (at < (last - first)[:, None]), here.gather(1, at.clamp(0, here.shape[1] - 1)), ids[0])
        st.update(path=_i32(path), path_len=_i32(n), ctx_len=_i32(have + n), block_table=_i32(bt),
                  pool_pages=ids.numel(), pool=torch.zeros((ids.numel(), Hkv, 2, PAGE, D), dtype=dt, device="cuda"))
        return st
    flushed = after // PAGE
    np0 = have // PAGE
    M = int((np0 + flushed).max()) + 1
    here, ids = _table(gen, flushed, 0, 2 * B)
    at = torch.arange(M, device="cuda")[None] - np0[:, None]
    bt = torch.where((at >= 0) & (at < flushed[:, None]), here.gather(1, at.clamp(0, here.shape[1] - 1)), 0)
    blob = _blob(case["n_hi"])
    st.update(path=_i32(path), path_len=_i32(n), num_pages=_i32(np0 + flushed), tail_len=_i32(after % PAGE),
              block_table=_i32(bt), pool_pages=ids.numel(),
              pool=torch.zeros((ids.numel(), Hkv, blob), dtype=torch.uint8, device="cuda"))
    sigma = _sigma(gen, case)
    st["tail_k"] = (torch.randn((B, Hkv, PAGE, D), generator=gen, device="cuda") * sigma[:, None]).to(dt)
    st["tail_v"] = torch.randn((B, Hkv, PAGE, D), generator=gen, device="cuda").to(dt)
    # accepted tokens that end where the tail's first ones were hold the same, so that a pass can be
    # repeated: token i of them is the last one written to row j
    j = torch.arange(PAGE, device="cuda")[None]
    i = PAGE * (flushed[:, None] - (j >= (after % PAGE)[:, None]).long()) + j - before[:, None]
    again = (j < before[:, None]) & (i >= 0)
    row = st["start"][:-1].long()[:, None] + path.gather(1, i.clamp(0, W - 1))
    row = torch.where(again, row, T)
    for x, tail in (("k", "tail_k"), ("v", "tail_v")):
        more = torch.cat([st[x], st[x][:1]])
        more[row.flatten()] = st[tail].transpose(1, 2).reshape(-1, Hkv, D)
        st[x] = more[:T]
    return st


def _prepare_pages(case, gen):
    """Lengths before a step (a whole batch of running sequences, or prompts that are admitted), and
    what is kept of each after it."""
    B = case["B"]
    have = _int(gen, case["far"] // 2, case["far"], B)
    new = _int(gen, 0, case["new"], B) if case["ragged"] else torch.full((B,), case["new"], device="cuda")
    kept = have + (torch.rand((B,), generator=gen, device="cuda") * (new + 1)).long().minimum(new)
    held = (kept + PAGE - 1) // PAGE
    M = (case["far"] + case["new"]) // PAGE + 2
    table, ids = _table(gen, held, 0, B * M + case["spare"])
    bt = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    bt[:, :table.shape[1]] = table[:, :M]
    free = ids[int(held.sum()):]
    stack = torch.zeros(ids.numel(), dtype=torch.int32, device="cuda")
    stack[:free.numel()] = free
    T = B * case["new"] + case["pad"]
    start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    return dict(case=case, lens=_i32(have), start=_i32(start), kept=_i32(kept), held=_i32(held), block_table=bt,
                free_ids=stack, free_count=_i32(torch.tensor([free.numel()], device="cuda")),
                slots=torch.full((T,), -1, dtype=torch.int64, device="cuda"),
                new_pages=torch.full((T,), -1, dtype=torch.int32, device="cuda"))


def _prepare_plan(case, gen):
    st = dict(case=case, **_trees(case, gen))
    T = st["parents"].numel()
    have = _int(gen, 0, 16384, case["B"])
    st.update(num_pages=_i32(have // PAGE), tail_len=_i32(have % PAGE),
              positions=torch.zeros((T,), dtype=torch.int32, device="cuda"),
              masks=torch.zeros((T,), dtype=torch.int64, device="cuda"))
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op in ("tree", "tree16"):
        return _prepare_attention(case, gen)
    if op in ("commit", "commit16"):
        return _prepare_commit(case, gen)
    return (_prepare_plan if op == "plan" else _prepare_pages)(case, gen)


# ------------------------------------------------------------------ plain forms
def _maps():
    """Where the codes of a page sit: word and bit of Key (token, channel) and Value (token, channel)."""
    t, c = torch.arange(PAGE, device="cuda")[:, None], torch.arange(D, device="cuda")[None]
    bit = lambda e, half, tau: (16 * e + 8 * half + 2 * tau + 2) % 32  # noqa: E731
    lane = 4 * (t % 8) + c % 8 // 2
    key = (lane, c // 16, bit(c % 2, c % 16 // 8, t // 8))
    lane = 4 * (c % 8) + t % 8 // 2
    val = (lane * 8 + c // 32 * 2 + t // 16, bit(t % 2, t % 16 // 8, c % 32 // 8))
    return key, val


def _unpacked(blobs, n_hi):
    """Keys and Values, fp32 [.., 32, 128], of packed pages [.., blob]."""
    (lane, word, kbit), (vword, vbit) = _maps()
    ints = lambda a, b: blobs[..., a:b].contiguous().view(torch.int32)  # noqa: E731
    halves = lambda a: blobs[..., a:a + 256].contiguous().view(torch.float16).float()  # noqa: E731
    ks = 1024 + 8 * n_hi
    S = halves(ks)
    c = torch.arange(D, device="cuda")
    M = halves(ks + 256)[..., (c % 8 // 2 * 8 + c // 16) * 4 + c % 16 // 8 * 2 + c % 2]
    code = (ints(0, 1024)[..., lane * 8 + word] >> kbit) & 3
    k = M[..., None, :] + S[..., None, :] * code
    if n_hi:
        j = torch.arange(n_hi, device="cuda")
        ch = blobs[..., ks + 512 + j // 16 * 16 + j % 8 // 2 * 4 + j % 16 // 8 * 2 + j % 2].long()
        lo = (ints(1024, ks)[..., lane[:, :n_hi] * (n_hi // 16) + word[:, :n_hi]] >> kbit[:, :n_hi]) & 3
        k.scatter_add_(-1, ch[..., None, :].expand(lo.shape), 0.25 * S.gather(-1, ch)[..., None, :] * lo)
    vb = ks + 512 + n_hi
    t, g = torch.arange(PAGE, device="cuda")[:, None], c[None] // 32
    at = g * 32 + t % 8 // 2 * 8 + t // 16 * 4 + t % 16 // 8 * 2 + t % 2
    vcode = (ints(vb, vb + 1024)[..., vword] >> vbit) & 3
    return k, halves(vb + 1280)[..., at] + halves(vb + 1024)[..., at] * vcode


def _pages16(pages):
    return pages[..., 0, :, :].float(), pages[..., 1, :, :].float()


def _attend_plain(st):
    """softmax(q K^T / sqrt(128)) V over what each drafted token sees: the prefix, its sequence's
    cached tokens, and the drafted tokens of its mask."""
    case = st["case"]
    B, N, Hq, Hkv, P = case["B"], case["nodes"], case["Hq"], case["Hkv"], case["prefix"]
    g, T = Hq // Hkv, st["q"].shape[0]
    packed = case["op"] == "tree"
    unpack = (lambda x: _unpacked(x, case["n_hi"])) if packed else _pages16
    start, node = st["start"].long(), torch.arange(N, device="cuda")
    at = (start[:-1, None] + node).clamp(max=T - 1)                     # [B, N]
    count = (start[1:] - start[:-1])[:, None]
    q = st["q"][at].float().view(B, N, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * g, D) * SCALE
    bt = st["block_table"]
    k, v = unpack(st["pool"][bt.clamp(min=0).long()])                   # [B, M, Hkv, 32, 128]
    k, v = (x.transpose(1, 2).reshape(B, Hkv, -1, D) for x in (k, v))
    t = torch.arange(k.shape[2], device="cuda")[None]
    if packed:
        off = t >= PAGE * st["num_pages"][:, None]
        k, v = (torch.cat([x, st[y].float()], 2) for x, y in ((k, "tail_k"), (v, "tail_v")))
        off = torch.cat([off, torch.arange(PAGE, device="cuda")[None] >= st["tail_len"][:, None]], 1)
    else:
        off = t >= st["ctx_len"][:, None]
    k, v = (torch.cat([x, st[y][at].float().transpose(1, 2)], 2) for x, y in ((k, "k"), (v, "v")))
    if st["visible"] is None:
        sees = (node[:, None] >= node).expand(B, N, N)
    else:
        sees = (st["visible"][at][..., None] >> node) & 1 != 0
    sees = sees & (node < count)[:, None] & (node < count)[:, :, None]
    off = torch.cat([off[:, None].expand(B, N, -1), ~sees], 2)          # [B, N, cached + N]
    s = q @ k.transpose(2, 3)
    s.masked_fill_(off.repeat_interleave(g, 1)[:, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    if P:
        pk, pv = unpack(st["pool"][st["prefix_table"].long()])          # [P, Hkv, 32, 128]
        pk, pv = (x.transpose(0, 1).reshape(1, Hkv, P * PAGE, D) for x in (pk, pv))
        s1 = q @ pk.transpose(2, 3)
        m = torch.maximum(m, s1.amax(-1, keepdim=True))
    s = s.sub_(m).exp_()
    o, total = s @ v, s.sum(-1, keepdim=True)
    if P:
        s1 = s1.sub_(m).exp_()
        o, total = o + s1 @ pv, total + s1.sum(-1, keepdim=True)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.view(B, Hkv, N, g, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(st["out"].dtype)
    b, i, real = _places(st["start"], T, B, N)
    return torch.where(real[:, None, None], o[b, i], st["out"])


def _squared(x):
    return (x @ x).clamp_(max=1.0)


def _plan_plain(st):
    case = st["case"]
    B, N = case["B"], case["nodes"]
    T = st["parents"].numel()
    start, node = st["start"].long(), torch.arange(N, device="cuda")
    at = (start[:-1, None] + node).clamp(max=T - 1)
    # ancestors of up to 64 steps: the parents' matrix and the identity, squared six times
    a = (st["parents"][at][..., None] == node).float() + torch.eye(N, device="cuda")
    a = _squared(_squared(_squared(_squared(_squared(_squared(a)))))).long()
    base = PAGE * st["num_pages"].long() + st["tail_len"]
    pos = base[:, None] + a.sum(-1) - 1
    bits = (a << node).sum(-1)
    b, i, real = _places(st["start"], T, B, N)
    return (torch.where(real, bits[b, i], st["masks"]),
            torch.where(real, pos[b, i].to(torch.int32), st["positions"]))


def _pages_plain(st):
    """Pages for lens + new tokens, in order from the top of the stack, and their slots; then down to
    the kept tokens' pages, given back in the reverse order."""
    case = st["case"]
    B, new = case["B"], max(case["new"], 1)
    bt, held, stack, count = st["block_table"], st["held"].long(), st["free_ids"], st["free_count"].long()
    start, lens = st["start"].long(), st["lens"].long()
    col = torch.arange(bt.shape[1], device="cuda")[None]
    need = ((lens + start[1:] - start[:-1] + PAGE - 1) // PAGE).maximum(held)
    grow = need - held
    before = (grow.cumsum(0) - grow)[:, None] + col - held[:, None]
    fresh = (col >= held[:, None]) & (col < need[:, None])
    taken = stack[(count - 1 - before).clamp(0, stack.numel() - 1)]
    bt.copy_(torch.where(fresh, taken, bt))
    count = count - grow.sum()
    b, i, real = _places(st["start"], st["slots"].numel(), B, new)
    pos = lens[b] + i
    page = bt[b, (pos // PAGE).clamp(max=bt.shape[1] - 1)]
    st["slots"].copy_(torch.where(real, page.long() * PAGE + pos % PAGE, st["slots"]))
    st["new_pages"].copy_(torch.where(real, torch.where(pos % PAGE == 0, page, -1), st["new_pages"]))
    keep = ((st["kept"].long() + PAGE - 1) // PAGE).minimum(need)
    gone = (col >= keep[:, None]) & (col < need[:, None])
    cut = need - keep
    total = cut.sum()
    behind = total - 1 - ((cut.cumsum(0) - cut)[:, None] + col - keep[:, None])  # place above the stack
    n = stack.numel()
    more = torch.cat([stack, stack[:1]])  # entries that are not given back all go behind the stack
    more[torch.where(gone, count + behind, n).clamp(0, n).flatten()] = bt.flatten()
    stack.copy_(more[:n])
    bt.masked_fill_(gone, -1)
    st["held"].copy_(keep)
    st["free_count"].copy_(count + total)
    return st["slots"], st["new_pages"], bt, st["held"], stack, st["free_count"]


def _commit_plain(st):
    case = st["case"]
    B, Hkv, W = case["B"], case["Hkv"], st["path"].shape[1]
    n = st["path_len"].long()
    total = PAGE * st["num_pages"].long() + st["tail_len"] - n  # tokens before
    before, np0 = total % PAGE, total // PAGE
    full, left = (before + n) // PAGE, (before + n) % PAGE
    # tail rows, then the accepted ones: [B, 96, Hkv, 128]
    place = torch.arange(3 * PAGE, device="cuda")[None]
    i = (place - before[:, None]).clamp(0, W - 1)
    row = st["start"][:-1].long()[:, None] + st["path"].long().gather(1, i)
    mine = (place < before[:, None])[..., None, None]
    j = torch.arange(PAGE, device="cuda")[None]
    # a row of the tail: what is left, else what the last full page held there, else what it was
    at = torch.where(j < left[:, None], PAGE * full[:, None] + j, PAGE * (full[:, None] - 1) + j)
    keep = (j >= left[:, None]) & (full[:, None] == 0)
    f = torch.arange(2, device="cuda")[None]
    real = f < full[:, None]
    page = st["block_table"].long().gather(1, (np0[:, None] + f).clamp(max=st["block_table"].shape[1] - 1))
    last = st["pool_pages"]
    page = torch.where(real, page, last).flatten()
    cut = {}
    for x, tail in (("k", "tail_k"), ("v", "tail_v")):
        old = st[tail].transpose(1, 2)
        rows = torch.where(mine, torch.cat([old, old, old], 1), st[x][row])
        cut[x] = rows[:, :2 * PAGE].float().view(B, 2, PAGE, Hkv, D).transpose(2, 3).reshape(-1, PAGE, D)
        new = rows.gather(1, at.clamp(min=0)[..., None, None].expand(B, PAGE, Hkv, D))
        st[tail].copy_(torch.where(keep[..., None, None], old, new).transpose(1, 2))
    blobs = _quantized(cut["k"], cut["v"], case["n_hi"]).view(2 * B, Hkv, -1)
    more = torch.cat([st["pool"], st["pool"][:1]])
    more[page] = blobs
    st["pool"].copy_(more[:last])
    return st["tail_k"], st["tail_v"], st["pool"], st["num_pages"], st["tail_len"]


def _commit16_plain(st):
    W, n = st["path"].shape[1], st["path_len"].long()
    i = torch.arange(W, device="cuda")[None]
    real = i < n[:, None]
    pos = st["ctx_len"].long()[:, None] - n[:, None] + i
    page = st["block_table"].long().gather(1, (pos // PAGE).clamp(0, st["block_table"].shape[1] - 1))
    page = torch.where(real, page, st["pool_pages"]).flatten()
    slot, row = (pos % PAGE).flatten(), (st["start"][:-1].long()[:, None] + st["path"]).flatten()
    more = torch.cat([st["pool"], st["pool"][:1]])
    more[page, :, 0, slot], more[page, :, 1, slot] = st["k"][row], st["v"][row]
    st["pool"].copy_(more[:st["pool_pages"]])
    return st["pool"], st["ctx_len"]


# ------------------------------------------------------------------ the framework's calls
def _handles(st):
    """The configuration and workspace that a program makes once."""
    from mixed_precision_bit_gb300 import kitty
    c = st["case"]
    if "cfg" not in st and "Hq" in c:
        dt = kitty.BF16 if c["dtype"] == "bf16" else kitty.F16
        st["cfg"] = cfg = kitty.Config(num_kv_heads=c["Hkv"], num_q_heads=c["Hq"], n_hi=c.get("n_hi", 32), in_dtype=dt)
        if c["op"] in ("tree", "tree16"):
            size = kitty.tree_workspace_bytes if c["op"] == "tree" else kitty.f16kv_tree_workspace_bytes
            n = size(cfg, c["B"], st["q"].shape[0], c["nodes"], st["block_table"].shape[1], c["prefix"])
            st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return kitty, st.get("cfg")


def _run_own(st):
    kitty, cfg = _handles(st)
    op = st["case"]["op"]
    if op == "plan":
        kitty.tree_plan(st["parents"], st["start"], st["tail_len"], st["masks"], st["positions"],
                        num_pages=st["num_pages"])
        return st["masks"], st["positions"]
    if op == "pages":
        kitty.page_tables(st["lens"], st["held"], st["block_table"], st["free_ids"], st["free_count"],
                          seq_start=st["start"], slots=st["slots"], new_page_ids=st["new_pages"])
        kitty.page_tables(st["kept"], st["held"], st["block_table"], st["free_ids"], st["free_count"], shrink=True)
        return st["slots"], st["new_pages"], st["block_table"], st["held"], st["free_ids"], st["free_count"]
    if op == "tree":
        kitty.tree_attention(cfg, st["q"], st["k"], st["v"], st["start"], st["visible"], st["case"]["nodes"],
                             st["pool"], st["pool_pages"], st["block_table"], st["num_pages"], st["tail_k"],
                             st["tail_v"], st["tail_len"], SCALE, st["out"], prefix_table=st["prefix_table"],
                             workspace=st["ws"])
        return st["out"]
    if op == "tree16":
        kitty.f16kv_tree_attention(cfg, st["q"], st["k"], st["v"], st["start"], st["visible"], st["case"]["nodes"],
                                   st["pool"], st["pool_pages"], st["block_table"], st["ctx_len"], SCALE,
                                   st["out"], prefix_table=st["prefix_table"], workspace=st["ws"])
        return st["out"]
    if op == "commit":
        kitty.tree_commit(cfg, st["k"], st["v"], st["start"], st["path"], st["path_len"], st["tail_k"],
                          st["tail_v"], st["tail_len"], None, None, None, st["block_table"], st["num_pages"],
                          st["pool"], st["pool_pages"], counted=True)
        return st["tail_k"], st["tail_v"], st["pool"], st["num_pages"], st["tail_len"]
    kitty.f16kv_tree_commit(cfg, st["k"], st["v"], st["start"], st["path"], st["path_len"], st["pool"],
                            st["pool_pages"], st["block_table"], st["ctx_len"], counted=True)
    return st["pool"], st["ctx_len"]


def run(st):
    if own:
        return _run_own(st)
    op = st["case"]["op"]
    if op in ("tree", "tree16"):
        return _attend_plain(st)
    if op == "plan":
        return _plan_plain(st)
    if op == "pages":
        return _pages_plain(st)
    return _commit_plain(st) if op == "commit" else _commit16_plain(st)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    B, op = case["B"], case["op"]
    if op == "pages":
        # lengths, starts, counts; pages taken and given back (an id read and written each, and the
        # table's entry); a slot and a page id for each new token
        new = case["new"] * (0.5 if case["ragged"] else 1.0)
        moved = 2.0 * B * new / 2 / PAGE
        return {"bytes": 24.0 * B + 8 * moved + 12.0 * B * new, "flops": 0.0}
    N = case["nodes"]
    n = N * (0.5 if case.get("ragged") else 1.0)
    if op == "plan":
        return {"bytes": B * (16.0 * n + 12), "flops": 0.0}
    Hq, Hkv = case["Hq"], case["Hkv"]
    if op in ("commit", "commit16"):
        # accepted rows read and written; each full page's rows before them read, its blob written
        accepted = B * min(N, case["accept"]) / 2
        bytes_ = accepted * Hkv * D * 2 * 2 * 2
        if op == "commit":
            bytes_ += accepted / PAGE * Hkv * (PAGE * D * 2 * 2 / 2 + _blob(case["n_hi"]))
        return {"bytes": bytes_ + 16.0 * B, "flops": 0.0}
    # three quarters of ctx in seven of eight sequences; the prefix once; rows and outputs
    cached = B * 0.75 * case["ctx"] * (B - B // 8) / B
    token = 2 * D * 2 if op == "tree16" else _blob(case["n_hi"]) / PAGE
    rows = B * n * (2 * Hq + 2 * Hkv) * D * 2
    seen = cached / B + PAGE * case["prefix"] + n / 2
    return {"bytes": (cached + PAGE * case["prefix"]) * Hkv * token + rows,
            "flops": 4.0 * B * n * Hq * D * seen}


# ------------------------------------------------------------------ 64 bits, from the definitions
def _codes_exact(words):
    """[.., n] 32-bit words -> [.., n, 2, 2, 4]: their codes by (column parity, column half, row block)."""
    u = words.long() & 0xFFFFFFFF
    u = ((u >> 2) | (u << 30)) & 0xFFFFFFFF
    return torch.stack([(u // 4 ** i) % 4 for i in range(16)], -1).unflatten(-1, (2, 2, 4))


def _unpacked_exact(blobs, n_hi):
    """Keys and Values [n, 32, 128] in 64 bits of packed pages [n, blob]."""
    n, nx = blobs.shape[0], n_hi // 16
    cut = torch.split(blobs, [1024, 8 * n_hi, 256, 256, n_hi, 1024, 256, 256], 1)
    base, extra, S, M, ids, val, vS, vM = (x.contiguous() for x in cut)
    tokens = lambda w, j: _codes_exact(w.view(torch.int32).view(n, 8, 4, j)).permute(0, 6, 1, 3, 5, 2, 4).reshape(n, PAGE, 16 * j)  # noqa: E731
    S = S.view(torch.float16).double()
    M = M.view(torch.float16).double().view(n, 4, 8, 2, 2).permute(0, 2, 3, 1, 4).reshape(n, D)
    code = 4.0 * tokens(base, 8).double()
    if nx:
        ids = ids.long().view(n, nx, 4, 2, 2).permute(0, 1, 3, 2, 4).reshape(n, n_hi)
        code.scatter_add_(2, ids[:, None].expand(n, PAGE, n_hi), tokens(extra, nx).double())
    k = M[:, None] + S[:, None] / 4.0 * code
    vc = _codes_exact(val.view(torch.int32).view(n, 8, 4, 4, 2)).permute(0, 4, 6, 2, 5, 3, 7, 1).reshape(n, PAGE, D)
    meta = lambda x: x.view(torch.float16).double().view(n, 4, 4, 2, 2, 2).permute(0, 3, 4, 2, 5, 1).reshape(n, PAGE, 4).repeat_interleave(32, 2)  # noqa: E731
    return k, meta(vM) + meta(vS) * vc


def _cached_exact(st, pages):
    """Keys and Values [Hkv, tokens, 128] of a list of pages, in 64 bits."""
    case, got = st["case"], st["pool"][pages]
    if case["op"] == "tree":
        k, v = (x.view(pages.numel(), case["Hkv"], PAGE, D) for x in _unpacked_exact(got.flatten(0, 1), case["n_hi"]))
    else:
        k, v = got[:, :, 0].double(), got[:, :, 1].double()
    return (x.transpose(0, 1).reshape(case["Hkv"], -1, D) for x in (k, v))


def _attend_exact(st):
    case = st["case"]
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    start, bt = st["start"].tolist(), st["block_table"].long()
    out = st["out"].double()
    shared = bt.new_zeros(0) if st["prefix_table"] is None else st["prefix_table"].long()
    for b in range(B):
        lo, n = start[b], start[b + 1] - start[b]
        if n == 0:
            continue
        if case["op"] == "tree":
            held, tail = int(st["num_pages"][b]), int(st["tail_len"][b])
            k, v = _cached_exact(st, torch.cat([shared, bt[b, :held]]))
            k, v = (torch.cat([x, st[y][b, :, :tail].double()], 1) for x, y in ((k, "tail_k"), (v, "tail_v")))
        else:
            length = int(st["ctx_len"][b])
            k, v = _cached_exact(st, torch.cat([shared, bt[b, :(length + PAGE - 1) // PAGE]]))
            k, v = (x[:, :PAGE * shared.numel() + length] for x in (k, v))
        cached = k.shape[1]
        k, v = (torch.cat([x, st[y][lo:lo + n].double().transpose(0, 1)], 1) for x, y in ((k, "k"), (v, "v")))
        seen = torch.ones((n, cached + n), dtype=torch.bool, device="cuda")
        if st["visible"] is None:
            seen[:, cached:] = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
        else:
            seen[:, cached:] = (st["visible"][lo:lo + n, None] // 2 ** torch.arange(n, device="cuda").clamp(max=62)) % 2 == 1
            if n == 64:
                seen[:, -1] = st["visible"][lo:lo + n] < 0
        q = st["q"][lo:lo + n].double().view(n, Hkv, Hq // Hkv, D)
        s = torch.einsum("nhgd,htd->nhgt", q, k) / math.sqrt(D)
        s.masked_fill_(~seen[:, None, None], -math.inf)
        p = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)
        out[lo:lo + n] = torch.einsum("nhgt,htd->nhgd", p, v).reshape(n, Hq, D)
    return out


def exact(case, seed):
    op = case["op"]
    if op in ("plan", "pages"):
        return None
    st = prepare(case, seed)
    if op in ("tree", "tree16"):
        return _attend_exact(st)
    start, path = st["start"].tolist(), st["path"].tolist()
    count = st["path_len"].tolist()
    if op == "commit16":
        pool, length = st["pool"].double(), st["ctx_len"].tolist()
        for b in range(case["B"]):
            for i in range(count[b]):
                at = length[b] - count[b] + i
                page = int(st["block_table"][b, at // PAGE])
                pool[page, :, 0, at % PAGE] = st["k"][start[b] + path[b][i]].double()
                pool[page, :, 1, at % PAGE] = st["v"][start[b] + path[b][i]].double()
        return pool, None
    tail_k, tail_v = st["tail_k"].double(), st["tail_v"].double()
    after = (PAGE * st["num_pages"].long() + st["tail_len"]).tolist()
    for b in range(case["B"]):
        for i in range(count[b]):
            at = after[b] - count[b] + i
            tail_k[b, :, at % PAGE] = st["k"][start[b] + path[b][i]].double()
            tail_v[b, :, at % PAGE] = st["v"][start[b] + path[b][i]].double()
    return tail_k, tail_v, None, None, None
