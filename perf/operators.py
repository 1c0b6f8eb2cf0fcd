"""Cases of the operators around a shared, position-rotated KV cache.

* ``rotate``: the RMS norm of every query and key head and the position rotation, in one pass
  (``kitty.norm_rope``);
* ``append16``: the same on the way into the 16-bit paged cache, one token or a ragged prompt a
  sequence (``kitty.f16kv_append_rope``);
* ``append``: the same on the way into the packed cache's tails (``kitty.append_rope``);
* ``shared``: decode attention of a batch whose sequences share a prefix, on packed pages
  (``kitty.decode_attention_shared``);
* ``shared16``: the same on 16-bit pages (``kitty.f16kv_decode_shared``).

``run`` computes each in elementary torch operations, or, with ``own``, by the framework's calls.
"""

import math

import numpy as np
import torch

own = False

D = 128     # channels of a head
PAGE = 32   # tokens of a page
EPS = 1e-6
SCALE = 1.0 / math.sqrt(D)

_CASES = [
    # a decode step's 64 tokens of a 32/8-head layer with per-head norms: latency
    dict(name="rotate decode 64", op="rotate", T=64, Hq=32, Hkv=8, rot=128, pairs="half", norm=True,
         freq="plain", far=8192, dtype="bf16"),
    # a prompt of 8192 tokens of the same layer, frequencies stretched by 4, positions up to 131072
    dict(name="rotate prompt 8192", op="rotate", T=8192, Hq=32, Hkv=8, rot=128, pairs="half",
         norm=True, freq="ramp", far=131072, dtype="bf16"),
    # an odd chunk of a 64/8-head layer that rotates neighbouring pairs of half of each head
    dict(name="rotate half-head 4095", op="rotate", T=4095, Hq=64, Hkv=8, rot=64,
         pairs="neighbours", norm=False, freq="plain", far=65536, dtype="fp16"),
    # one token a sequence into 16-bit pages, 64 sequences near 8192 tokens
    dict(name="append16 step 64", op="append16", B=64, new=1, far=8192, Hq=32, Hkv=8, rot=128,
         pairs="half", norm=True, freq="plain", dtype="bf16", pad=0),
    # eight ragged prompts, about 8192 tokens, into 16-bit pages, three padding rows behind them
    dict(name="append16 prompts 8", op="append16", B=8, new=2047, far=4096, Hq=32, Hkv=8, rot=128,
         pairs="half", norm=True, freq="plain", dtype="bf16", pad=3),
    # one token a sequence into the packed cache's tails, the batch of a 40 GB cache budget; no
    # tail fills in this step
    dict(name="append step 177", op="append", B=177, far=8192, Hq=32, Hkv=8, rot=128, pairs="half",
         norm=True, freq="plain", dtype="bf16"),
    # 16 sequences of a 64/8-head layer, neighbouring pairs of half of each head, no norm
    dict(name="append step 16", op="append", B=16, far=8192, Hq=64, Hkv=8, rot=64,
         pairs="neighbours", norm=False, freq="plain", dtype="fp16"),
    # 16 sequences behind one 4096-token prompt, short answers: the smallest shared decode
    dict(name="shared 16x4096", op="shared", B=16, pages=128, fork=False, own_pages=3, Hq=32, Hkv=8,
         n_hi=32, dtype="bf16"),
    # 64 sequences behind an 8192-token prompt, some of them forked off before its end
    dict(name="shared 64x8192 forked", op="shared", B=64, pages=256, fork=True, own_pages=8, Hq=32,
         Hkv=8, n_hi=16, dtype="bf16"),
    # 128 sequences of a 64/8-head layer behind a 32768-token document
    dict(name="shared 128x32768", op="shared", B=128, pages=1024, fork=False, own_pages=4, Hq=64,
         Hkv=8, n_hi=32, dtype="bf16"),
    # 64 sequences behind an 8192-token prompt in 16-bit pages
    dict(name="shared16 64x8192", op="shared16", B=64, pages=256, fork=False, own_pages=8, Hq=32,
         Hkv=8, dtype="bf16"),
    # an odd batch and an odd prefix in 16-bit pages of a small layer, forked
    dict(name="shared16 33x1952 forked", op="shared16", B=33, pages=61, fork=True, own_pages=5,
         Hq=6, Hkv=2, dtype="fp16"),
]


def listed():
    return [dict(c) for c in _CASES]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append16", "append", "shared", "shared", "shared16"])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    g = rng.choice([1, 2, 3, 4] if op == "shared16" else [1, 2, 3, 4, 6, 8])
    c = dict(op=op, Hq=Hkv * g, Hkv=Hkv, dtype=rng.choice(["bf16", "fp16"]))
    if op in ("shared", "shared16"):
        c.update(B=_log(rng, 1, 128), pages=_log(rng, 4, 512), fork=rng.random() < 0.5,
                 own_pages=rng.randint(0, 8))
        if op == "shared":
            c["n_hi"] = rng.choice([0, 16, 32, 64, 128])
        return c
    c.update(rot=rng.choice([16, 32, 64, 96, 128]), pairs=rng.choice(["half", "neighbours"]),
             norm=rng.random() < 0.5, freq=rng.choice(["plain", "ramp"]),
             far=_log(rng, 256, 131072))
    if op == "rotate":
        c["T"] = _log(rng, 1, 8192)
    elif op == "append":
        c["B"] = _log(rng, 1, 256)
    else:
        c.update(B=_log(rng, 1, 64), new=rng.choice([1, _log(rng, 2, 512)]), pad=rng.choice([0, 5]))
    return c


# ------------------------------------------------------------------ inputs
def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _frequencies(case):
    """Radians a position of each pair, in 64 bits, and the factor on the rotated channels."""
    n, base = case["rot"] // 2, 500000.0
    f = base ** (-np.arange(n, dtype=np.float64) / n)
    if case["freq"] == "plain":
        return f, 1.0
    # stretched by 4: pairs that turn over 32 times in 8192 positions stay, those under once are
    # slowed by 4, a linear ramp between them
    turns = 8192 * f / (2 * math.pi)
    keep = np.clip((turns - 1.0) / 31.0, 0.0, 1.0)
    return f * keep + f / 4.0 * (1.0 - keep), 0.1 * math.log(4.0) + 1.0


def _rows(gen, case, n):
    """The projections of n tokens, as one matrix: query, key and value heads side by side."""
    H = case["Hq"] + 2 * case["Hkv"]
    x = torch.randn((n, H, D), generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn((1, H, D), generator=gen, device="cuda"))
    x = x.to(_type(case))
    Hq, Hkv = case["Hq"], case["Hkv"]
    return x, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _prepare_rotation(case, gen, n):
    x, q, k, v = _rows(gen, case, n)
    f, amplitude = _frequencies(case)
    st = dict(case=case, rows=x, q=q, k=k, v=v, freq=torch.from_numpy(f).cuda(),
              amplitude=amplitude, q_out=torch.zeros((n, case["Hq"], D), dtype=_type(case), device="cuda"))
    for name in ("q_weight", "k_weight"):
        w = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
        st[name] = w.to(_type(case)) if case["norm"] else None
    return st


def _pack(codes_r_w):
    """32-bit words of 16 two-bit codes: [.., e, half, tau] (2, 2, 4) at bit 16e + 8half + 2tau + 2."""
    e, h, t = (torch.arange(n, device="cuda") for n in (2, 2, 4))
    bit = (16 * e[:, None, None] + 8 * h[None, :, None] + 2 * t[None, None, :] + 2) % 32
    w = (codes_r_w.long() << bit).flatten(-3).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _steps(s):
    """Quantization steps rounded up to seven significant bits."""
    return ((s.contiguous().view(torch.int32) + 0x1FFFF) & ~0x1FFFF).view(torch.float32).half()


def _quantized(k, v, n_hi):
    """Packed pages, uint8 [n, blob], of fp32 Keys and Values [n, 32, 128]: 2-bit Key channels with
    the n_hi of largest variance at 4 bits (two planes), 2-bit Values in groups of 32 channels."""
    n = k.shape[0]
    mn, mx = k.amin(1), k.amax(1)
    order = k.var(1, unbiased=False).argsort(dim=1, descending=True, stable=True)
    ch = order[:, :n_hi].sort(dim=1).values
    boost = torch.zeros((n, D), dtype=torch.bool, device="cuda").scatter_(1, ch, True)
    levels = torch.where(boost, 15.0, 3.0)
    S = _steps((mx - mn) / levels * torch.where(boost, 4.0, 1.0))
    unit = S.float() / torch.where(boost, 4.0, 1.0)
    M = mn.half()
    code = torch.round((k - M.float()[:, None]) / unit[:, None]).clamp_(min=0).minimum(levels[:, None])
    code = code.to(torch.int32)
    hi = torch.where(boost[:, None], code >> 2, code)
    key = lambda x: _pack(x.view(n, 4, 8, -1, 2, 4, 2).permute(0, 2, 5, 3, 6, 4, 1)).flatten(1)  # noqa: E731
    base = key(hi)
    lo = (code & 3).gather(2, ch[:, None].expand(n, PAGE, n_hi))
    extra = key(lo) if n_hi else base[:, :0]
    vg = v.view(n, PAGE, 4, 32)
    vmin, vmax = vg.amin(3), vg.amax(3)
    vS, vM = _steps((vmax - vmin) / 3.0), vmin.half()
    vcode = torch.round((vg - vM.float()[..., None]) / vS.float()[..., None]).clamp_(0, 3).to(torch.int32)
    val = _pack(vcode.view(n, 2, 2, 4, 2, 4, 4, 8).permute(0, 7, 3, 5, 1, 4, 2, 6)).flatten(1)
    chan = lambda x: x.view(n, 8, 2, 4, 2).permute(0, 3, 1, 2, 4).flatten(1)  # noqa: E731
    meta = lambda x: x.permute(0, 2, 1).reshape(n, 4, 2, 2, 4, 2).permute(0, 1, 4, 2, 3, 5).flatten(1)  # noqa: E731
    ids = ch.to(torch.uint8).view(n, n_hi // 16, 2, 4, 2).permute(0, 1, 3, 2, 4).flatten(1)
    parts = [base, extra, S, chan(M), ids, val, meta(vS), meta(vM)]
    return torch.cat([p.contiguous().view(torch.uint8).view(n, -1) for p in parts], 1)


def _prepare_shared(case, gen):
    B, Hq, Hkv, P = case["B"], case["Hq"], case["Hkv"], case["pages"]
    packed = case["op"] == "shared"
    dt = _type(case)
    own_pages = torch.randint(0, case["own_pages"] + 1, (B,), generator=gen, device="cuda")
    tails = torch.randint(0, PAGE, (B,), generator=gen, device="cuda")
    slots = own_pages if packed else own_pages + (tails > 0).long()
    M = max(case["own_pages"] + 1, 1)
    at = torch.arange(M, device="cuda")[None]
    total = P + int(slots.sum())
    ids = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    first = P + slots.cumsum(0) - slots
    where = (first[:, None] + at).clamp(max=total - 1)
    bt = torch.where(at < slots[:, None], ids[where], torch.tensor(-1, dtype=torch.int32, device="cuda"))
    pages = torch.full((B,), P, dtype=torch.int32, device="cuda")
    if case["fork"]:
        pages = torch.randint(0, P + 1, (B,), generator=gen, device="cuda").to(torch.int32)
        pages[::2] = P
    sigma = torch.exp(torch.randn((Hkv, 1, D), generator=gen, device="cuda"))

    def tokens(*shape):
        k = torch.randn(shape, generator=gen, device="cuda") * sigma
        return k.to(dt), torch.randn(shape, generator=gen, device="cuda").to(dt)

    st = dict(case=case, q=torch.randn((B, Hq, D), generator=gen, device="cuda").to(dt),
              out=torch.empty((B, Hq, D), dtype=dt, device="cuda"), pool_pages=total,
              prefix_table=ids[:P].contiguous(), prefix_pages=pages, block_table=bt.contiguous())
    k, v = tokens(total, Hkv, PAGE, D)
    if packed:
        blobs = _quantized(k.float().view(-1, PAGE, D), v.float().view(-1, PAGE, D), case["n_hi"])
        st["tail_k"], st["tail_v"] = tokens(B, Hkv, PAGE, D)
        st.update(pool=blobs.view(total, Hkv, -1), num_pages=own_pages.to(torch.int32),
                  tail_len=tails.to(torch.int32))
    else:
        st.update(pool=torch.stack([k, v], 2), ctx_len=(own_pages * PAGE + tails).to(torch.int32))
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op in ("shared", "shared16"):
        return _prepare_shared(case, gen)
    if op == "rotate":
        st = _prepare_rotation(case, gen, case["T"])
        st["pos"] = torch.randint(0, case["far"], (case["T"],), generator=gen, device="cuda").to(torch.int32)
        st["k_out"] = torch.zeros((case["T"], case["Hkv"], D), dtype=_type(case), device="cuda")
        return st
    B, Hkv = case["B"], case["Hkv"]
    have = torch.randint(0, case["far"], (B,), generator=gen, device="cuda")
    if op == "append":
        # lengths that already count the new token, as every layer after the first finds them
        st = _prepare_rotation(case, gen, B)
        tail = 1 + have % (PAGE - 1)
        st.update(num_pages=(have // PAGE).to(torch.int32), tail_len=tail.to(torch.int32),
                  flush=torch.full((B,), -1, dtype=torch.int32, device="cuda"), pool_pages=B,
                  pool=torch.zeros((B, Hkv, 3072 + 9 * 32), dtype=torch.uint8, device="cuda"),
                  block_table=torch.zeros((B, case["far"] // PAGE + 1), dtype=torch.int32, device="cuda"))
        for name in ("tail_k", "tail_v"):
            st[name] = torch.zeros((B, Hkv, PAGE, D), dtype=_type(case), device="cuda")
        return st
    new, most = torch.full((B,), 1, device="cuda"), B
    if case["new"] > 1:
        # ragged: shares of B * new / 2 tokens, one sequence without any; what rounding leaves over
        # joins the padding rows
        most = (B * case["new"] + 1) // 2
        share = torch.rand((B,), generator=gen, device="cuda")
        share[int(torch.randint(0, B, (1,), generator=gen, device="cuda"))] = 0.0 if B > 1 else 1.0
        new = (share / share.sum() * most).long().clamp(max=most)
    start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    T = most + case["pad"]
    st = _prepare_rotation(case, gen, T)
    # a pool of the pages that this step touches; the pages before them all name page 0
    first, last = have // PAGE, (have + new + PAGE - 1) // PAGE
    touched = last - first
    M = int(last.max()) + 1
    at = torch.arange(M, device="cuda")[None]
    total = 1 + most // PAGE + 2 * B
    ids = torch.cat([have.new_zeros(1), 1 + torch.randperm(total - 1, generator=gen, device="cuda")])
    slot = (1 + touched.cumsum(0) - touched)[:, None] + at - first[:, None]
    inside = (at >= first[:, None]) & (at < last[:, None])
    bt = torch.where(inside, ids[slot.clamp(0, total - 1)], torch.zeros_like(slot)).to(torch.int32)
    st.update(start=start.to(torch.int32), ctx_len=(have + new).to(torch.int32), block_table=bt,
              pool_pages=total, pool=torch.zeros((total, Hkv, 2, PAGE, D), dtype=_type(case), device="cuda"))
    # the page of each token that begins one
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(st["start"][1:].contiguous(), t.to(torch.int32), right=True).clamp(max=B - 1)
    pos = (have[b] + t - start[b]).clamp(max=M * PAGE - 1)
    st["new_page"] = torch.where((pos % PAGE == 0) & (t < start[-1]), bt[b, pos // PAGE],
                                 torch.tensor(-1, dtype=torch.int32, device="cuda"))
    return st


# ------------------------------------------------------------------ plain forms
def _turned(st, x, weight, pos):
    """Rows [T, H, 128] at positions [T], normed and rotated, in 32 bits (angles in 64)."""
    case = st["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    angle = pos.double()[:, None, None] * st["freq"]
    c, s = (angle.cos() * st["amplitude"]).float(), (angle.sin() * st["amplitude"]).float()
    rot, h = case["rot"], case["rot"] // 2
    if case["pairs"] == "half":
        a, b = x[..., :h], x[..., h:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1).to(st["q"].dtype)


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
    """softmax(q K^T / sqrt(128)) V over the shared pages that a sequence has and its own."""
    case = st["case"]
    B, Hq, Hkv, P = case["B"], case["Hq"], case["Hkv"], case["pages"]
    g = Hq // Hkv
    unpack = (lambda x: _unpacked(x, case["n_hi"])) if case["op"] == "shared" else _pages16
    q = st["q"].float().view(B, Hkv, g, D) * SCALE
    pk, pv = unpack(st["pool"][st["prefix_table"].long()])              # [P, Hkv, 32, 128]
    pk, pv = (x.transpose(0, 1).reshape(Hkv, P * PAGE, D) for x in (pk, pv))
    s1 = q.transpose(0, 1).reshape(Hkv, B * g, D) @ pk.transpose(1, 2)  # [Hkv, B g, P 32]
    s1 = s1.view(Hkv, B, g, P * PAGE)
    t = torch.arange(P * PAGE, device="cuda")
    s1.masked_fill_((t[None] >= PAGE * st["prefix_pages"][:, None])[None, :, None], -math.inf)
    bt = st["block_table"]
    ok, ov = unpack(st["pool"][bt.clamp(min=0).long()])                 # [B, M, Hkv, 32, 128]
    ok, ov = (x.transpose(1, 2).reshape(B, Hkv, -1, D) for x in (ok, ov))
    n = torch.arange(ok.shape[2], device="cuda")[None]
    if case["op"] == "shared":
        off = n >= PAGE * st["num_pages"][:, None]
        ok, ov = (torch.cat([x, st[y].float()], 2) for x, y in ((ok, "tail_k"), (ov, "tail_v")))
        off = torch.cat([off, torch.arange(PAGE, device="cuda")[None] >= st["tail_len"][:, None]], 1)
    else:
        off = n >= st["ctx_len"][:, None]
    s2 = (q @ ok.transpose(2, 3)).masked_fill_(off[:, None, None], -math.inf).transpose(0, 1)
    m = torch.maximum(s1.amax(-1), s2.amax(-1)).clamp(min=-1e30)[..., None]
    s1, s2 = s1.sub_(m).exp_(), (s2 - m).exp()
    o = (s1.view(Hkv, B * g, -1) @ pv).view(Hkv, B, g, D) + (s2.transpose(0, 1) @ ov).transpose(0, 1)
    total = s1.sum(-1, keepdim=True) + s2.sum(-1, keepdim=True)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.transpose(0, 1).reshape(B, Hq, D).to(st["q"].dtype)


def _append_plain(st):
    pos = PAGE * st["num_pages"].long() + st["tail_len"] - 1
    q = _turned(st, st["q"], st["q_weight"], pos)
    at = (torch.arange(st["case"]["B"], device="cuda"), slice(None), (st["tail_len"].long() - 1))
    st["tail_k"][at] = _turned(st, st["k"], st["k_weight"], pos)
    st["tail_v"][at] = st["v"]
    return q, st["tail_k"], st["tail_v"]


def _append16_plain(st):
    start, T = st["start"].long(), st["q"].shape[0]
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    real = b < st["case"]["B"]
    b = b.clamp(max=st["case"]["B"] - 1)
    pos = st["ctx_len"].long()[b] - (start[b + 1] - t)
    q = _turned(st, st["q"], st["q_weight"], pos)
    k = _turned(st, st["k"], st["k_weight"], pos)
    q = torch.where(real[:, None, None], q, st["q_out"])
    # padding rows write to the page that no sequence appends to, what is there already
    pos = torch.where(real, pos, torch.zeros_like(pos))
    page = torch.where(real, st["block_table"].long()[b, pos // PAGE], torch.zeros_like(pos))
    here = lambda x, i: torch.where(real[:, None, None], x, st["pool"][page, :, i, pos % PAGE])  # noqa: E731
    st["pool"][page, :, 0, pos % PAGE] = here(k, 0)
    st["pool"][page, :, 1, pos % PAGE] = here(st["v"], 1)
    return q, st["pool"]


# ------------------------------------------------------------------ the framework's calls
def _handles(st):
    """The configuration, rotation table and workspace that a program makes once."""
    from mixed_precision_bit_gb300 import kitty
    if "cfg" not in st:
        c = st["case"]
        dt = kitty.BF16 if c["dtype"] == "bf16" else kitty.F16
        st["cfg"] = kitty.Config(num_kv_heads=c["Hkv"], num_q_heads=c["Hq"], n_hi=c.get("n_hi", 32), in_dtype=dt)
        if "freq" in st:
            layout = kitty.ROPE_HALF if c["pairs"] == "half" else kitty.ROPE_INTERLEAVED
            st["rope"] = kitty.Rope(st["freq"].cpu().numpy(), layout=layout, amplitude=st["amplitude"],
                                    q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS)
        else:
            size = kitty.shared_workspace_bytes if c["op"] == "shared" else kitty.f16kv_shared_workspace_bytes
            n = size(st["cfg"], c["B"], c["pages"], st["block_table"].shape[1])
            st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return kitty, st["cfg"]


def _run_own(st):
    kitty, cfg = _handles(st)
    op = st["case"]["op"]
    if op == "rotate":
        kitty.norm_rope(cfg, st["rope"], st["q"], st["k"], st["pos"], st["q_out"], st["k_out"])
        return st["q_out"], st["k_out"]
    if op == "append":
        kitty.append_rope(cfg, st["rope"], st["q"], st["k"], st["v"], st["q_out"], st["tail_k"],
                          st["tail_v"], st["tail_len"], None, None, None, st["flush"], st["block_table"],
                          st["num_pages"], st["pool"], st["pool_pages"], counted=True)
        return st["q_out"], st["tail_k"], st["tail_v"]
    if op == "append16":
        kitty.f16kv_append_rope(cfg, st["rope"], st["q"], st["k"], st["v"], st["q_out"], st["pool"],
                                st["pool_pages"], st["block_table"], st["ctx_len"], st["new_page"],
                                seq_start=st["start"], counted=True)
        return st["q_out"], st["pool"]
    if op == "shared":
        kitty.decode_attention_shared(cfg, st["q"], st["pool"], st["pool_pages"], st["prefix_table"],
                                      st["prefix_pages"], st["block_table"], st["num_pages"],
                                      st["tail_k"], st["tail_v"], st["tail_len"], SCALE, st["out"],
                                      workspace=st["ws"])
    else:
        kitty.f16kv_decode_shared(cfg, st["q"], st["pool"], st["pool_pages"], st["prefix_table"],
                                  st["prefix_pages"], st["block_table"], st["ctx_len"], SCALE, st["out"],
                                  workspace=st["ws"])
    return st["out"]


def run(st):
    if own:
        return _run_own(st)
    op = st["case"]["op"]
    if op == "rotate":
        return (_turned(st, st["q"], st["q_weight"], st["pos"]),
                _turned(st, st["k"], st["k_weight"], st["pos"]))
    if op == "append":
        return _append_plain(st)
    if op == "append16":
        return _append16_plain(st)
    return _attend_plain(st)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] in ("shared", "shared16"):
        # prefix pages once for all, each sequence's own pages and tails (half of the most, on
        # average), queries and outputs; two products over every cached token
        B, P, n = case["B"], case["pages"], case["own_pages"]
        blob = 3072 + 9 * case["n_hi"] if case["op"] == "shared" else 2 * PAGE * D * 2
        mean = P * (0.75 if case["fork"] else 1.0)
        own_bytes = B * Hkv * (n / 2 * blob + (PAGE - 1) / 2 * D * 4)
        return {"bytes": P * Hkv * blob + own_bytes + 2 * B * Hq * D * 2,
                "flops": 4.0 * B * Hq * D * (PAGE * (mean + n / 2) + (PAGE - 1) / 2)}
    if case["op"] == "rotate":
        n, heads = case["T"], Hq + Hkv
    else:
        n = case["B"] * (1 if case["op"] == "append" or case["new"] == 1 else (case["new"] + 1) / 2)
        heads = Hq + 2 * Hkv
    return {"bytes": 2.0 * n * heads * D * 2 + 8 * n, "flops": 10.0 * n * (Hq + Hkv) * D}


# ------------------------------------------------------------------ 64 bits, from the definitions
def _turned_exact(st, x, weight, pos):
    case = st["case"]
    x = x.double()
    if weight is not None:
        x = x * weight.double() / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS)
    n = case["rot"] // 2
    turn = torch.polar(torch.full((pos.numel(), 1, n), st["amplitude"], dtype=torch.float64, device="cuda"),
                       (pos.double()[:, None] * st["freq"][None])[:, None])
    idx = torch.arange(n, device="cuda")
    ia, ib = (idx, idx + n) if case["pairs"] == "half" else (2 * idx, 2 * idx + 1)
    z = torch.complex(x[..., ia], x[..., ib]) * turn
    y = x.clone()
    y[..., ia], y[..., ib] = z.real, z.imag
    return y


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


def _attend_exact(st):
    case = st["case"]
    B, Hq, Hkv, P = case["B"], case["Hq"], case["Hkv"], case["pages"]
    g = Hq // Hkv
    total = st["pool_pages"]
    if case["op"] == "shared":
        k, v = (x.view(total, Hkv, PAGE, D) for x in _unpacked_exact(st["pool"].view(total * Hkv, -1), case["n_hi"]))
        counts, tails = st["num_pages"].tolist(), st["tail_len"].tolist()
    else:
        k, v = st["pool"][:, :, 0].double(), st["pool"][:, :, 1].double()
        counts, tails = st["ctx_len"].tolist(), None
    pre, shared, bt = st["prefix_table"].long(), st["prefix_pages"].tolist(), st["block_table"].long()
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    for b in range(B):
        if case["op"] == "shared":
            mine = torch.cat([pre[:shared[b]], bt[b, :counts[b]]])
        else:
            mine = torch.cat([pre[:shared[b]], bt[b, :(counts[b] + PAGE - 1) // PAGE]])
        kb, vb = (x[mine].transpose(0, 1).reshape(Hkv, -1, D) for x in (k, v))
        if tails is not None:
            kb = torch.cat([kb, st["tail_k"][b, :, :tails[b]].double()], 1)
            vb = torch.cat([vb, st["tail_v"][b, :, :tails[b]].double()], 1)
        else:
            n = PAGE * shared[b] + counts[b]
            kb, vb = kb[:, :n], vb[:, :n]
        if kb.shape[1]:
            s = torch.einsum("hgd,htd->hgt", st["q"][b].double().view(Hkv, g, D), kb) / math.sqrt(D)
            out[b] = torch.einsum("hgt,htd->hgd", torch.softmax(s, -1), vb).reshape(Hq, D)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rotate":
        return (_turned_exact(st, st["q"], st["q_weight"], st["pos"]),
                _turned_exact(st, st["k"], st["k_weight"], st["pos"]))
    if op in ("shared", "shared16"):
        return _attend_exact(st)
    B, Hkv = case["B"], case["Hkv"]
    if op == "append":
        pos = st["num_pages"].long() * PAGE + st["tail_len"].long() - 1
        k = _turned_exact(st, st["k"], st["k_weight"], pos)
        tail_k, tail_v = st["tail_k"].double(), st["tail_v"].double()
        for b, n in enumerate(st["tail_len"].tolist()):
            tail_k[b, :, n - 1], tail_v[b, :, n - 1] = k[b], st["v"][b].double()
        return _turned_exact(st, st["q"], st["q_weight"], pos), tail_k, tail_v
    start, after = st["start"].tolist(), st["ctx_len"].tolist()
    q, pool = st["q_out"].double(), st["pool"].double()
    for b in range(B):
        lo, hi = start[b], start[b + 1]
        if hi == lo:
            continue
        pos = torch.arange(after[b] - (hi - lo), after[b], device="cuda")
        q[lo:hi] = _turned_exact(st, st["q"][lo:hi], st["q_weight"], pos)
        page, slot = st["block_table"][b].long()[pos // PAGE], pos % PAGE
        pool[page, :, 0, slot] = _turned_exact(st, st["k"][lo:hi], st["k_weight"], pos)
        pool[page, :, 1, slot] = st["v"][lo:hi].double()
    return q, pool
