"""Serving a hybrid decoder with beams, measured: the paged cache held in 8 bits, attention over
it, and the beams' selection and reordering.

A case is a dict of plain values.  `op` names the operator:

* "append":  rotate new queries and keys, hold keys and values in 8 bits in the sequences' pages,
             and read the last tokens back as the values that the cache holds;
* "attn":    attention of new queries over the sequences' cached tokens;
* "select":  the best continuations of every group of beams over the vocabulary;
* "reorder": recurrent states, page tables and pages after such a selection.

The cache is uint8 [n_pages, heads, page_bytes]; one (page, head) block holds, one after the other,
the codes of `page` keys (d bytes each), the codes of `page` values, and 16 bytes of exponents for
every 128 places (one group for smaller pages): eight for the keys' blocks of 16 places, eight for
the values'.  A code is an e4m3 number, an exponent byte e stands for 2^(e - 15), 0 <= e <= 22, and
a head may have a further fp32 scale: value = e4m3 * 2^(e - 15) * scale[head].
"""
import math
import random

import torch

own = False

BLOCK = 16          # places that share an exponent
MOST_E = 22         # the largest exponent byte
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases


def listed():
    return [
        # -- append to the cache ------------------------------------------------------
        # a decode step of 64 sequences at their own lengths; the blocks that the new tokens
        # joined are read back
        dict(name="append8_token_b64", op="append", B=64, new_min=1, new_max=1, len_min=128,
             len_max=16384, lens_seed=1, idle=0, read=16, Hq=32, Hk=8, d=128, rot=128, page=64,
             axes=1, adjacent=False, head_scale=False, layout="thd", dt="bf16"),
        # prompts of twelve sequences packed together, with images among the text
        dict(name="append8_prompts_n12", op="append", B=12, new_min=700, new_max=8192, len_min=700,
             len_max=8192, lens_seed=2, idle=0, read=0, Hq=32, Hk=8, d=128, rot=128, page=64,
             axes=3, adjacent=False, head_scale=True, layout="thd", dt="bf16"),
        # fp32, small pages, several tokens each, odd offsets, heads outermost
        dict(name="append8_few_b5_f32", op="append", B=5, new_min=1, new_max=37, len_min=37,
             len_max=500, lens_seed=3, idle=0, read=0, Hq=8, Hk=8, d=64, rot=32, page=16, axes=1,
             adjacent=True, head_scale=True, layout="htd", dt="f32"),
        # -- attention over the cache -------------------------------------------------
        # one token of one short sequence: latency
        dict(name="attn8_token_b1_len77_f32", op="attn", B=1, new_min=1, new_max=1, len_min=77,
             len_max=77, lens_seed=4, idle=0, Hq=16, Hk=2, d=64, page=16, window=0, causal=True,
             head_scale=False, layout="thd", dt="f32"),
        # a decode step of 64 sequences of mixed lengths, one slot of the batch idle
        dict(name="attn8_token_b64_ragged", op="attn", B=64, new_min=1, new_max=1, len_min=128,
             len_max=16384, lens_seed=1, idle=1, Hq=32, Hk=8, d=128, page=64, window=0,
             causal=True, head_scale=True, layout="thd", dt="bf16"),
        # a large decode batch: 4.3 GB of cache
        dict(name="attn8_token_b256_len8192", op="attn", B=256, new_min=1, new_max=1, len_min=8001,
             len_max=8192, lens_seed=6, idle=0, Hq=16, Hk=8, d=128, page=128, window=0,
             causal=True, head_scale=False, layout="thd", dt="bf16"),
        # a chunk of a long prompt on top of what is cached already
        dict(name="attn8_chunk_b2_q2048", op="attn", B=2, new_min=2048, new_max=2048,
             len_min=12001, len_max=16384, lens_seed=8, idle=0, Hq=16, Hk=4, d=128, page=64,
             window=0, causal=True, head_scale=True, layout="thd", dt="bf16"),
        # -- selection ----------------------------------------------------------------
        # the first step of one request: four beams alike, the first alone alive
        dict(name="select_first_b1_w4_f32", op="select", B=1, W=4, V=32000, n=4, first=True,
             done=False, banned=0, dt="f32"),
        # a step of eight requests, some beams finished, an odd vocabulary, some of it banned
        dict(name="select_done_b8_w5", op="select", B=8, W=5, V=50257, n=5, first=False,
             done=True, banned=100, dt="bf16"),
        # a large batch; twice the beams' number of candidates, as a search that ends
        # sequences on the host wants them
        dict(name="select_b64_w8_n16", op="select", B=64, W=8, V=128256, n=16, first=False,
             done=False, banned=0, dt="bf16"),
        # -- reordering ---------------------------------------------------------------
        # one request: one recurrent and one attention layer
        dict(name="reorder_b1_w4", op="reorder", B=1, W=4, states=1, H=4, d=64, caches=1, Hk=2,
             page=16, len_min=77, len_max=77, lens_seed=9, skew=1.0),
        # sixteen requests: six recurrent layers, two attention layers
        dict(name="reorder_b16_w6", op="reorder", B=16, W=6, states=6, H=16, d=128, caches=2, Hk=4,
             page=64, len_min=33, len_max=2048, lens_seed=10, skew=1.0),
    ]


def _log(rng, lo, hi):
    """A whole number from [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "select", "reorder"])
    d = rng.choice([64, 128, 128, 256])
    Hq, Hk = rng.choice([(16, 2), (16, 4), (16, 16), (32, 8), (8, 1), (24, 8), (12, 4)])
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "select":
        V = _log(rng, 1000, 262144)
        W = rng.randint(1, 16)
        B = _log(rng, 1, max(1, min(64, (1 << 25) // (V * W))))
        done = rng.random() < 0.3
        return dict(op=op, B=B, W=W, V=V, n=W if done else rng.choice([W, rng.randint(1, 2 * W), 2 * W]),
                    first=rng.random() < 0.2, done=done, banned=rng.choice([0, 0, V // 50]), dt=dt)
    if op == "reorder":
        W, caches = rng.randint(2, 12), rng.randint(0, 2)
        H, d = rng.choice([4, 8, 16]), rng.choice([64, 128])
        states = rng.randint(0 if caches else 1, 4)
        B = _log(rng, 1, max(1, min(32, (1 << 27) // (W * 4 * H * d * d))))
        top = _log(rng, 1, 2048)
        return dict(op=op, B=B, W=W, states=states, H=H, d=d, caches=caches, Hk=rng.choice([1, 2, 4]),
                    page=page, len_min=max(1, top // rng.choice([1, 3, 20])), len_max=top,
                    lens_seed=rng.randrange(1 << 20), skew=rng.choice([0.0, 1.0, 3.0]))
    if op == "append":
        B = _log(rng, 1, 64)
        top = _log(rng, 1, max(1, min(8192, (1 << 26) // ((Hq + 2 * Hk) * d * B))))
        low = rng.choice([top, max(1, top // 7)])
        return dict(op=op, B=B, new_min=low, new_max=top, len_min=top, len_max=top + _log(rng, 1, 8192),
                    lens_seed=rng.randrange(1 << 20), idle=rng.choice([0, 0, 1]) if B > 2 else 0,
                    read=rng.choice([0, 16, 40]), Hq=Hq, Hk=Hk, d=d, rot=rng.choice([d, d, d // 2]),
                    page=page, axes=rng.choice([1, 1, 3]), adjacent=rng.random() < 0.3,
                    head_scale=rng.random() < 0.5, layout=rng.choice(["thd", "htd"]), dt=dt)
    form = rng.choice(["token", "token", "draft", "chunk"])
    if form == "token":
        new, low, top_b = 1, 1, 256
    elif form == "draft":
        new, low, top_b = rng.randint(2, 9), 2, 64
    else:
        new, low, top_b = _log(rng, 16, 2048), 16, 4
    B = _log(rng, 1, top_b)
    # at most the largest listed cases' cache bytes, and their products
    most = min(131072, (1 << 30) // (B * Hk * d), (1 << 38) // (4 * B * Hq * d * new))
    if form == "chunk" and dt == "f32":
        most = min(most, 4096)
    hi = _log(rng, min(max(new, 17), most), most)
    return dict(op=op, B=B, new_min=rng.choice([new, low]), new_max=new, len_min=max(new, hi // rng.choice([1, 2, 50])),
                len_max=max(new, hi), lens_seed=rng.randrange(1 << 20),
                idle=rng.choice([0, 0, 1]) if B > 2 else 0, Hq=Hq, Hk=Hk, d=d, page=page,
                window=rng.choice([0, 0, _log(rng, 16, 8192)]), causal=new == 1 or rng.random() < 0.8,
                head_scale=rng.random() < 0.5, layout=rng.choice(["thd", "htd"]), dt=dt)


def _lens(case):
    """(new tokens, cached tokens with them) of each sequence: the same for every seed."""
    r = random.Random(case["lens_seed"])
    new, length = [], []
    for b in range(case["B"]):
        n = r.randint(case["new_min"], case["new_max"])
        new.append(n)
        length.append(max(n, r.randint(case["len_min"], case["len_max"])))
        if b < case["idle"]:
            length[b] = 0    # an idle slot of the batch: its rows see nothing
    return new, length


def _parents(case):
    """(the beam that each beam of a group goes on from, tokens cached by each group): the same for
    every seed.  skew: how much more the better beams are gone on from."""
    r = random.Random(case["lens_seed"])
    W = case["W"]
    weight = [math.exp(-case["skew"] * i / W) for i in range(W)]
    parent, length = [], []
    for _ in range(case["B"]):
        length.append(r.randint(case["len_min"], case["len_max"]))
        parent.append(r.choices(range(W), weight, k=W))
    return parent, length


def _visible(case):
    """Per sequence: (pairs of a query token and a token that it sees, tokens seen by any)."""
    out = []
    for n, length in zip(*_lens(case)):
        if length == 0:
            out.append((0, 0))
            continue
        pairs, first, last = 0, length, 0
        for j in range(n):
            p = length - n + j
            hi = p + 1 if case["causal"] else length
            lo = max(0, p + 1 - case["window"]) if case["window"] else 0
            pairs += max(0, hi - lo)
            first, last = min(first, lo), max(last, hi)
        out.append((pairs, last - first))
    return out


def _page_bytes(page, d):
    return 2 * page * d + 16 * max(1, page // 128)


def work(case):
    d = case.get("d", 0)
    if case["op"] == "select":
        rows, size = case["B"] * case["W"], 2 if case["dt"] == "bf16" else 4
        return {"bytes": rows * (case["V"] * size + 4) + 12 * case["B"] * case["n"],
                "flops": 3 * rows * case["V"]}
    if case["op"] == "reorder":
        parent, length = _parents(case)
        lane = case["states"] * case["H"] * d * d * 4
        byte = 0
        for p, n in zip(parent, length):
            twins = case["W"] - len(set(p))     # beams whose parent goes on in another one already
            page = case["caches"] * case["Hk"] * _page_bytes(case["page"], d) if n % case["page"] else 0
            table = 4 * -(-case["len_max"] // case["page"]) + 4 if case["caches"] else 0
            byte += 2 * twins * (lane + page) + case["W"] * (12 + 2 * table)
        return {"bytes": byte, "flops": 0}
    size = 2 if case["dt"] == "bf16" else 4
    Hq, Hk = case["Hq"], case["Hk"]
    new, length = _lens(case)
    n = sum(a for a, b in zip(new, length) if b)
    if case["op"] == "append":
        # q in and out, k and v in and written, what is read back in and out
        back = sum(case["read"] or a for a, b in zip(new, length) if b)
        rows = n * case["rot"] * 4 + n * 4 * case["axes"]
        byte = n * (2 * Hq * d * size + 2 * Hk * d * size + 2 * Hk * d) + back * 2 * Hk * d * (1 + size) + rows
        return {"bytes": byte, "flops": 3 * n * (Hq + Hk) * case["rot"] + 2 * (n + back) * Hk * d}
    vis = _visible(case)
    byte = sum(seen for _, seen in vis) * Hk * (2 * d + 1 / 8) + 2 * sum(new) * Hq * d * size
    return {"bytes": int(byte), "flops": 4 * d * Hq * sum(pairs for pairs, _ in vis)}


# ------------------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _table(n, rot):
    """cos and sin of position * base^(-2 i / rot), fp32 [n, rot / 2]."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return a.cos().float().contiguous(), a.sin().float().contiguous()


def _axes(case):
    """The axis of each pair: one, or time, height and width in turn."""
    return [i % case["axes"] for i in range(case["rot"] // 2)]


def _positions(case, n, g):
    """int32 [axes, n]: counting up for text; a time, a row and a column for patches."""
    if case["axes"] == 1:
        return torch.arange(n, dtype=torch.int32, device="cuda")[None]
    t = torch.arange(n, dtype=torch.int32, device="cuda")
    wide = 17 + int(torch.randint(0, 16, (1,), generator=g, device="cuda"))
    return torch.stack([t // (wide * wide), t // wide % wide, t % wide]).contiguous()


def _rows(shape, layout, g, dt, scale=None):
    """Normal rows, seen as [tokens, heads, d] whichever axis is outermost."""
    x = torch.randn(shape, generator=g, device="cuda")
    if scale is not None:
        x = x * scale
    x = x.to(dt)
    if layout == "htd":      # heads outermost in memory
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    return x


def _parts(pages, page, d):
    """Views of the cache: codes of keys and values [n, H, page, d], exponents [n, H, page / 16]."""
    n, H, _ = pages.shape
    cut = lambda at: pages[:, :, at:at + page * d].unflatten(-1, (page, d))  # noqa: E731
    e = pages[:, :, 2 * page * d:].unflatten(-1, (-1, 2, 8))[..., :min(page, 128) // BLOCK]
    return cut(0), cut(page * d), e[..., 0, :], e[..., 1, :]


def _put_exponents(part, which, block, e):
    """part as _parts gives it, [n, H, groups, up to 8]: exponents e [*, H] of block `block` [*] of
    pages `which` [*]."""
    part[which, :, block // 8, block % 8] = e


def _fill(pages, page, d, H, inverse, g):
    """Fills the cache with held normal keys (channels of different size) and values."""
    kc, vc, ke, ve = _parts(pages, page, d)
    wide = torch.exp(0.5 * torch.randn(H, 1, d, generator=g, device="cuda"))
    step = max(1, (1 << 27) // (H * page * d))
    for at in range(0, pages.shape[0], step):
        n = min(step, pages.shape[0] - at)
        for codes, exps, i in ((kc, ke, 0), (vc, ve, 1)):
            x = torch.randn(n, H, page, d, generator=g, device="cuda")
            if i == 0:
                x = x * wide
            if inverse is not None:
                x = x * inverse[i][:, None, None]
            e = _exponent(x.abs().unflatten(2, (-1, BLOCK)).amax((3, 4)))
            codes[at:at + n] = _codes(x.unflatten(2, (-1, BLOCK)), e[..., None, None]).flatten(2, 3)
            exps[at:at + n] = e.view(n, H, exps.shape[2], exps.shape[3])


def _prepare_select(case, g):
    B, W, V, dt = case["B"], case["W"], case["V"], _DT[case["dt"]]
    # logits as a model leaves them: most of the weight on few tokens
    x = 2.0 * torch.randn(B, W, V, generator=g, device="cuda")
    likely = torch.randint(0, V, (B, W, 20), generator=g, device="cuda")
    x.scatter_add_(2, likely, 10.0 * torch.rand(B, W, 20, generator=g, device="cuda"))
    if case["banned"]:
        x[:, :, torch.randint(0, V, (case["banned"],), generator=g, device="cuda")] = -math.inf
    scores = -20.0 * torch.rand(B, W, generator=g, device="cuda")
    scores = scores.sort(-1, descending=True).values
    if case["first"]:       # one prompt each: its beams are alike and only the first counts
        x[:, 1:] = x[:, :1]
        scores.fill_(-math.inf)
        scores[:, 0] = 0.0
    done = None
    if case["done"]:
        done = torch.rand(B, W, generator=g, device="cuda") < 0.3
    return dict(case=case, logits=x.to(dt), scores=scores.contiguous(), done=done)


def _prepare_reorder(case, g):
    parent, length = _parents(case)
    B, W, H, d, page = case["B"], case["W"], case["H"], case["d"], case["page"]
    lanes = B * W + 2                          # two that no beam has
    state = dict(case=case, parent=torch.tensor(parent, dtype=torch.int32, device="cuda"),
                 slots=torch.randperm(lanes, generator=g, device="cuda")[:B * W].int().view(B, W),
                 states=[torch.randn(lanes, H, d, d, generator=g, device="cuda")
                         for _ in range(case["states"])], caches=[])
    if case["caches"]:
        per = -(-case["len_max"] // page) + 1
        # every lane has pages of its own; what lies behind the groups' first tokens is shared
        # by beams that went on from the same one
        state["own_pages"] = torch.randperm(lanes * per, generator=g, device="cuda").int().view(lanes, per)
        n = torch.tensor(length, dtype=torch.int32, device="cuda").repeat_interleave(W)
        state["len"] = n
        # (a full page may be any beam's of the group, the last one is the beam's own)
        beam = torch.randint(0, W, (B, W, per), generator=g, device="cuda")
        mine = torch.arange(W, device="cuda")[None, :, None]
        full = torch.arange(per, device="cuda") < (n.view(B, W, 1) // page)
        lane = state["slots"].long().gather(1, torch.where(full, beam, mine).flatten(1)).view(B, W, per)
        state["table"] = state["own_pages"][lane, torch.arange(per, device="cuda")].reshape(B * W, per).contiguous()
        state["caches"] = [torch.randint(0, 256, (lanes * per, case["Hk"], _page_bytes(page, d)), generator=g,
                                         device="cuda", dtype=torch.uint8) for _ in range(case["caches"])]
    return state


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "select":
        return _prepare_select(case, g)
    if case["op"] == "reorder":
        return _prepare_reorder(case, g)
    dt, d, Hq, Hk = _DT[case["dt"]], case["d"], case["Hq"], case["Hk"]
    new, length = _lens(case)
    page, B = case["page"], case["B"]
    counts = [-(-n // page) for n in length]
    total, most = sum(counts) + 3, max(1, max(counts))
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = [sum(counts[:b]) for b in range(B)]
    table = torch.zeros(B, most, dtype=torch.int32, device="cuda")
    i = torch.arange(most, device="cuda")
    n_pages = torch.tensor(counts, device="cuda")
    used = i[None] < n_pages[:, None]
    table[used] = order[(torch.tensor(at, device="cuda")[:, None] + i)[used]]
    scale = None
    if case["head_scale"]:
        scale = torch.rand(2, Hk, generator=g, device="cuda") * 0.5 + 0.05
    pages = torch.zeros(total, Hk, _page_bytes(page, d), device="cuda", dtype=torch.uint8)
    _fill(pages, page, d, Hk, None if scale is None else 1 / scale, g)
    N = sum(new)
    cu = [sum(new[:b]) for b in range(B + 1)]
    state = dict(case=case, pages=pages, table=table, scale=scale,
                 len=torch.tensor(length, dtype=torch.int32, device="cuda"),
                 cu=torch.tensor(cu, dtype=torch.int32, device="cuda") if min(new) < max(new) else None,
                 spare=order[sum(counts)].long(), q=_rows((N, Hq, d), case["layout"], g, dt),
                 max_len=max(length), max_new=max(new))
    if case["op"] == "append":
        state["k"] = _rows((N, Hk, d), case["layout"], g, dt, torch.exp(0.5 * torch.randn(Hk, d, generator=g, device="cuda")))
        state["v"] = _rows((N, Hk, d), case["layout"], g, dt)
        if case["axes"] == 1:     # text: a token's position is its place in the cache
            at = [max(0, a - b) + j for a, b in zip(length, new) for j in range(b)]
            pos = torch.tensor([at], dtype=torch.int32, device="cuda")
        else:
            pos = _positions(case, N, g)
        state["pos"], state["axes"] = pos, _axes(case)
        state["cos"], state["sin"] = _table(int(pos.max()) + 1, case["rot"])
        return state
    # what lies behind a sequence's end in its last page is left over from other tokens
    last = (state["len"].long() - 1).clamp_min(0)
    behind = torch.arange(page, device="cuda")[None] > (last % page)[:, None]
    which = table[torch.arange(B, device="cuda"), last // page].long()
    for part in _parts(pages, page, d)[:2]:
        rows = part[which]
        junk = torch.randint(0, 256, rows.shape, generator=g, device="cuda", dtype=torch.uint8)
        here = (behind & (state["len"] > 0)[:, None])[:, None, :, None]
        some = torch.nonzero(state["len"] > 0)[:, 0]
        part[which[some]] = torch.where(here, junk, rows)[some]
    return state


# --------------------------------------------------------------------- the plain forms


def _rotate(x, cos, sin, rot, adjacent):
    """Rotates the first `rot` elements of fp32 rows; cos and sin broadcast to [..., rot / 2]."""
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if adjacent else (r[..., :rot // 2], r[..., rot // 2:])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([ya, yb], -1).flatten(-2) if adjacent else torch.cat([ya, yb], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _angles(state, dtype=torch.float32):
    """cos and sin of each token's pairs, [tokens, rot / 2]."""
    axis = torch.tensor(state["axes"], device="cuda")
    pos = state["pos"].long()[axis].movedim(0, -1)
    pair = torch.arange(len(state["axes"]), device="cuda")
    return state["cos"][pos, pair].to(dtype), state["sin"][pos, pair].to(dtype)


def _exponent(m):
    """The exponent byte of a block whose largest magnitude is m: the least with m <= 448 * 2^(e - 15)."""
    f, x = torch.frexp(m)                      # m = f * 2^x, 1/2 <= f < 1; 448 = 7/8 * 2^9
    e = x.int() - 9 + (f > 0.875).int() + 15
    return torch.where(torch.isinf(m), MOST_E, torch.where(m == 0, 0, e)).clamp(0, MOST_E).to(torch.uint8)


def _power(e):
    """2^(15 - e)"""
    return torch.ldexp(torch.ones((), device="cuda"), 15 - e.int())


def _codes(x, e):
    """fp32 numbers as e4m3 bytes under exponents e; a NaN makes its 16 neighbours along d NaN."""
    y = (x * _power(e)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    bad = x.unflatten(-1, (-1, 16)).isnan().any(-1, keepdim=True).expand(*x.shape[:-1], -1, 16).flatten(-2)
    return torch.where(bad, 0x7F, y)


def _values(codes, e, head, dtype=torch.float32):
    """What codes stand for under exponents e; `head` broadcasts to the rows, or is None."""
    v = codes.view(torch.float8_e4m3fn).to(dtype) * torch.ldexp(torch.ones((), dtype=dtype, device="cuda"), e.int() - 15)
    return v if head is None else v * head


def _places(state, n=0):
    """(sequence, place in the cache) of every new token; n: of the last n of every sequence."""
    B = state["len"].shape[0]
    N = n * B or state["q"].shape[0]
    t = torch.arange(N, device="cuda")
    if n or state["cu"] is None:
        each = n or N // B
        seq = t // each
        return seq, state["len"].long()[seq] - each + t % each
    cu = state["cu"].long()
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq, state["len"].long()[seq] - (cu[seq + 1] - cu[seq]) + (t - cu[seq])


def _plain_append(s):
    c, dt = s["case"], s["q"].dtype
    page, d, B = c["page"], c["d"], c["B"]
    cos, sin = _angles(s)
    turn = lambda x: _rotate(x.float(), cos[:, None], sin[:, None], c["rot"], c["adjacent"])  # noqa: E731
    seq, place = _places(s)
    live = place >= 0
    row = place.clamp_min(0)
    table = s["table"].long()
    # a token of an idle slot is not written: here it goes to a page that nobody has
    which = torch.where(live, table[seq, row // page], s["spare"])
    # the call's blocks of 16 places, and the rows of each sequence's first one that were there
    blocks = table.shape[1] * (page // BLOCK)
    gid = torch.where(live, seq * blocks + row // BLOCK, B * blocks)
    start = torch.full((B,), blocks * BLOCK, device="cuda").scatter_reduce(0, seq, torch.where(live, place, blocks * BLOCK), "amin")
    had = torch.where(start < blocks * BLOCK, start % BLOCK, 0)
    first = (start // BLOCK).clamp_max(blocks - 1)
    page0 = torch.where(had > 0, table[torch.arange(B, device="cuda"), first * BLOCK // page], s["spare"])
    block0 = first % (page // BLOCK)
    kc, vc, ke, ve = _parts(s["pages"], page, d)
    for x, codes, exps, i in ((turn(s["k"]), kc, ke, 0), (s["v"].float(), vc, ve, 1)):
        if s["scale"] is not None:
            x = x * (1.0 / s["scale"][i])[:, None]
        y = x.abs().unflatten(-1, (-1, 16))
        m = torch.where(y.isnan().any(-1), 0.0, y.amax(-1)).amax(-1)          # [N, H]
        most = torch.zeros(B * blocks + 1, x.shape[1], device="cuda").scatter_reduce(
            0, gid[:, None].expand_as(m), m, "amax")
        e = _exponent(most)
        # a block that had rows keeps its exponent at least, and they move to a larger one
        old = exps[page0, :, block0 // 8, block0 % 8]                          # [B, H]
        at0 = torch.where(had > 0, torch.arange(B, device="cuda") * blocks + first, B * blocks)
        e = e.scatter_reduce(0, at0[:, None].expand_as(old), old, "amax")
        grown = e[at0]
        r0 = (block0 * BLOCK)[:, None] + torch.arange(BLOCK, device="cuda")   # [B, 16]
        rows = codes[page0[:, None], :, r0]                                    # [B, 16, H, d]
        moved = _codes(_values(rows, old[:, None, :, None], None), grown[:, None, :, None])
        keep = (torch.arange(BLOCK, device="cuda") < had[:, None])[..., None, None]
        codes[page0[:, None], :, r0] = torch.where(keep, torch.where((rows & 0x7F) == 0x7F, rows, moved), rows)
        e = e[gid]
        codes[which, :, row % page] = _codes(x, e[..., None])
        _put_exponents(exps, which, row % page // BLOCK, e)
    out = {"q": turn(s["q"]).to(dt)}
    if c["read"]:
        seq, place = _places(s, c["read"])
        live = place >= 0
        row = place.clamp_min(0)
        which = torch.where(live, table[seq, row // page], s["spare"])
    for name, codes, exps, i in (("k", kc, ke, 0), ("v", vc, ve, 1)):
        e = exps[which, :, row % page // BLOCK // 8, row % page // BLOCK % 8]
        back = _values(codes[which, :, row % page], e[..., None], None if s["scale"] is None else s["scale"][i][:, None])
        out[name] = torch.where(live[:, None, None], back, 0.0).to(dt)
    return out


def _plain_attn(s):
    c, q = s["case"], s["q"]
    N, Hq, d = q.shape
    B, Hk, page = c["B"], c["Hk"], c["page"]
    seq, place = _places(s)
    first = torch.cat([torch.ones(1, dtype=torch.bool, device="cuda"), seq[1:] != seq[:-1]])
    start = torch.cummax(torch.where(first, torch.arange(N, device="cuda"), 0), 0).values
    j = torch.arange(N, device="cuda") - start
    rows = torch.zeros(B, s["max_new"], Hq, d, device="cuda")
    rows[seq, j] = q.float()
    at = torch.full((B, s["max_new"]), -1, dtype=torch.long, device="cuda")
    at[seq, j] = place
    # every sequence's pages, one after the other: [B, Hk, tokens, d]
    L = s["table"].shape[1] * page
    t = torch.arange(L, device="cuda")
    there = (t[None] < s["len"][:, None])[:, None, :, None]
    kc, vc, ke, ve = _parts(s["pages"], page, d)
    table = s["table"].long()

    def whole(codes, exps, head):
        e = exps[table].flatten(3).transpose(1, 2).flatten(2, 3).repeat_interleave(BLOCK, 2)
        v = _values(codes[table].transpose(1, 2).flatten(2, 3), e[..., None], None if head is None else head[:, None, None])
        return torch.where(there, v, 0.0)

    head = (None, None) if s["scale"] is None else s["scale"]
    rows = rows.view(B, s["max_new"], Hk, Hq // Hk, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, d)
    scores = rows @ whole(kc, ke, head[0]).transpose(-1, -2) * (1.0 / math.sqrt(d))
    hi = (at + 1 if c["causal"] else torch.where(at >= 0, s["len"][:, None].long(), 0))[..., None]
    lo = (at + 1 - c["window"] if c["window"] else torch.zeros_like(at))[..., None]
    seen = ((t >= lo) & (t < hi))[:, None, None]
    scores = scores.view(B, Hk, Hq // Hk, s["max_new"], L).masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = (scores - torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hk, -1, L) @ whole(vc, ve, head[1])).view(B, Hk, Hq // Hk, s["max_new"], d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B, s["max_new"], Hq, d)
    return o[seq, j].to(q.dtype)


EOS = 1     # the token that a finished beam goes on with


def _plain_select(s):
    c = s["case"]
    B, W, V, n = c["B"], c["W"], c["V"], c["n"]
    # in 64 bits: beams are told apart by sums of many terms
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    lse = (x - top).exp_().sum(-1, keepdim=True).log_() + top
    x.sub_(lse).add_(s["scores"].double()[..., None])
    if s["done"] is not None:
        d = s["done"][..., None]
        x.masked_fill_(d, -math.inf)
        x[..., EOS] = torch.where(s["done"], s["scores"].double(), x[..., EOS])
    v, i = x.view(B, -1).sort(dim=-1, descending=True, stable=True)
    v, i = v[:, :n], i[:, :n]
    return {"scores": v.float(), "beam": (i // V).int(), "token": (i % V).int()}


def _plain_reorder(s):
    c = s["case"]
    B, W, page = c["B"], c["W"], c["page"]
    parent, slots = s["parent"].long(), s["slots"].long()
    i = torch.arange(W, device="cuda")
    twin = ((parent[:, :, None] == parent[:, None]) & (i < i[:, None])).any(-1)     # an earlier beam has its lane
    childless = ~(parent[:, None] == i[:, None]).any(-1)
    free = torch.sort((~childless).int(), dim=-1, stable=True).indices                  # childless beams first, in order
    rank = (twin.cumsum(-1) - 1).clamp_min(0)
    lane0 = slots.gather(1, parent)
    lane = torch.where(twin, slots.gather(1, free.gather(1, rank)), lane0)
    for x in s["states"]:
        x[lane.flatten()] = x[lane0.flatten()]
    out = {"slots": lane.int(), "states": s["states"], "caches": s["caches"]}
    if s["caches"]:
        table = s["table"].view(B, W, -1)
        full = (s["len"].long() // page).view(B, W, 1)
        from_ = table.gather(1, parent[..., None].expand_as(table))
        j = torch.arange(table.shape[-1], device="cuda")
        new = torch.where((j >= full) & twin[..., None], s["own_pages"][lane], from_)
        part = (s["len"].view(B, W, 1) % page) > 0
        a = from_.gather(2, full).long()
        b = torch.where(part, new.gather(2, full).long(), a)     # (nothing in it yet: onto itself)
        for x in s["caches"]:
            x[b.flatten()] = x[a.flatten()]
        out["table"] = new.reshape(B * W, -1)
    return out


def run(state):
    c = state["case"]
    if not own:
        return {"append": _plain_append, "attn": _plain_attn, "select": _plain_select,
                "reorder": _plain_reorder}[c["op"]](state)
    import gated_deltanet_recurrence_gdn_gb300 as gdn
    if c["op"] == "append":
        q = gdn.gdn_kv8_append(state["pages"], state["k"], state["v"], state["table"], state["len"],
                               q=state["q"], cu_seqlens=state["cu"], kv_scale=state["scale"],
                               cos=state["cos"], sin=state["sin"], pos=state["pos"], axes=state["axes"],
                               adjacent=c["adjacent"])
        k, v = gdn.gdn_kv8_read(state["pages"], state["table"], state["len"],
                                c["read"] * c["B"] or state["q"].shape[0], c["d"],
                                cu_seqlens=None if c["read"] else state["cu"], kv_scale=state["scale"],
                                dtype=state["q"].dtype)
        return {"q": q, "k": k, "v": v}
    if c["op"] == "attn":
        return gdn.gdn_kv8_attn(state["q"], state["pages"], state["table"], state["len"],
                                cu_seqlens=state["cu"], kv_scale=state["scale"], max_len=state["max_len"],
                                max_new=state["max_new"], causal=c["causal"], window=c["window"])
    if c["op"] == "select":
        scores, beam, token = gdn.gdn_beam_select(state["logits"], state["scores"], c["n"], done=state["done"],
                                                  eos=EOS if c["done"] else None)
        return {"scores": scores, "beam": beam, "token": token}
    if not c["caches"]:
        slots = gdn.gdn_beam_reorder(state["parent"], state["slots"], states=state["states"])
        return {"slots": slots, "states": state["states"], "caches": []}
    slots, table = gdn.gdn_beam_reorder(state["parent"], state["slots"], states=state["states"],
                                        caches=state["caches"], page_table=state["table"],
                                        own_pages=state["own_pages"], kv_len=state["len"],
                                        page_size=c["page"])
    return {"slots": slots, "states": state["states"], "caches": state["caches"], "table": table}


# ------------------------------------------------------------- the definition in 64 bits


def _turn64(x, state):
    """Each pair (a, b) of a row as the complex number a + i b, times cos + i sin."""
    c = state["case"]
    half = c["rot"] // 2
    angle = torch.empty(state["pos"].shape[1], half, dtype=torch.complex128, device="cuda")
    for i, axis in enumerate(state["axes"]):
        p = state["pos"][axis].long()
        angle[..., i] = torch.complex(state["cos"][p, i].double(), state["sin"][p, i].double())
    angle = angle.unsqueeze(1)      # one for all heads
    y = x.double().clone()
    a = slice(0, c["rot"], 2) if c["adjacent"] else slice(0, half)
    b = slice(1, c["rot"], 2) if c["adjacent"] else slice(half, c["rot"])
    z = torch.complex(y[..., a], y[..., b]) * angle
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _e4m3_grid():
    e4m3 = [m / 512.0 for m in range(8)] + [(1 + m / 8.0) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    return torch.tensor(e4m3[:127], dtype=torch.float64, device="cuda")


def _nearest64(x):
    """The nearest e4m3 number, at most 448; a tie goes to the one of even code."""
    grid = _e4m3_grid()
    a = x.abs().contiguous()
    i = torch.searchsorted(grid, a).clamp(1, len(grid) - 1)
    low, high = a - grid[i - 1], grid[i] - a
    up = (high < low) | ((high == low) & (i % 2 == 0))
    return grid[torch.where(up, i, i - 1)] * x.sign()


def _e4m3_64(byte):
    i = (byte & 127).long()
    v = torch.where(i == 127, math.nan, _e4m3_grid()[i.clamp_max(126)])
    return torch.where(byte >= 128, -v, v)


def _least64(m):
    """The least exponent under which magnitude m is at most 448."""
    bound = 448.0 * 2.0 ** torch.arange(-15, MOST_E - 15, dtype=torch.float64, device="cuda")
    return torch.searchsorted(bound, m.contiguous())


def _read64(block, page, d, which):
    """Keys (0) or values (1) of some pages of one head, uint8 [n, page_bytes]: ([n, page, d] without
    their exponents, exponents [n, page / 16])."""
    v = _e4m3_64(block[:, which * page * d:(which + 1) * page * d]).view(-1, page, d)
    e = [2 * page * d + 16 * (i // 8) + 8 * which + i % 8 for i in range(page // BLOCK)]
    return v, block[:, e].long()


def _exact_append(case, s):
    new, length = _lens(case)
    d, page, Hk = case["d"], case["page"], case["Hk"]
    rows = {"k": _turn64(s["k"], s), "v": s["v"].double()}
    out = {"q": _turn64(s["q"], s)}
    for i, name in enumerate(("k", "v")):
        got, at = [], 0
        for b, (n, L) in enumerate(zip(new, length)):
            back = case["read"] or n
            x = rows[name][at:at + n]
            at += n
            if L == 0:
                got.append(torch.zeros(back, Hk, d, dtype=torch.float64, device="cuda"))
                continue
            g = torch.ones(Hk, 1, dtype=torch.float64, device="cuda") if s["scale"] is None else s["scale"][i].double()[:, None]
            # the sequence as it was, a whole number of blocks
            ids = s["table"][b, :-(-L // page)].long()
            held = [_read64(s["pages"][ids, h], page, d, i) for h in range(Hk)]
            v = torch.stack([a.reshape(-1, BLOCK, d) for a, _ in held], 1)             # [blocks, H, 16, d]
            e = torch.stack([a.reshape(-1) for _, a in held], 1)
            t = torch.arange(v.shape[0] * BLOCK, device="cuda").view(-1, 1, BLOCK, 1)
            is_new = (t >= L - n) & (t < L)
            z = torch.zeros(v.shape[0] * BLOCK, Hk, d, dtype=torch.float64, device="cuda")
            z[L - n:L] = x / g
            z = z.view(-1, BLOCK, Hk, d).transpose(1, 2)
            there = t < L - n
            old = torch.where(there.any(2)[..., 0], e, 0)
            now = torch.maximum(old, torch.where(is_new.any(2)[..., 0], _least64(torch.where(is_new, z, 0.0).abs().amax((2, 3))), 0))
            two = lambda p: torch.pow(2.0, p.double())[..., None, None]  # noqa: E731
            moved = torch.where((now > old)[..., None, None], _nearest64(v * two(old - now)), v)
            v = torch.where(is_new, _nearest64(z * two(15 - now)), moved) * two(now - 15) * g[:, None]
            v = v.transpose(1, 2).reshape(-1, Hk, d)
            zero = torch.zeros(max(0, back - L), Hk, d, dtype=torch.float64, device="cuda")
            got.append(torch.cat([zero, v[max(0, L - back):L]]))
        out[name] = torch.cat(got)
    return out


def _exact_attn(case, s):
    new, length = _lens(case)
    d, Hq, Hk, page = case["d"], case["Hq"], case["Hk"], case["page"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, L) in enumerate(zip(new, length)):
        ids = s["table"][b, :-(-L // page)].long()
        p = L - n + torch.arange(n, device="cuda")
        t = torch.arange(L, device="cuda")
        seen = (t[None] <= p[:, None]) if case["causal"] else torch.ones(n, L, dtype=torch.bool, device="cuda")
        if case["window"]:
            seen = seen & (t[None] > p[:, None] - case["window"])
        for h in range(Hk if L else 0):
            block = s["pages"][ids, h]
            kv = []
            for i in (0, 1):
                v, e = _read64(block, page, d, i)
                v = v * torch.pow(2.0, e.double() - 15).repeat_interleave(BLOCK, 1)[..., None]
                kv.append(v.reshape(-1, d)[:L] * (1.0 if s["scale"] is None else s["scale"][i, h].double()))
            for i in range(h * (Hq // Hk), (h + 1) * (Hq // Hk)):
                w = (s["q"][at:at + n, i].double() @ kv[0].T) / math.sqrt(d)
                w = torch.softmax(w.masked_fill(~seen, -math.inf), -1).nan_to_num(0.0)
                o[at:at + n, i] = w @ kv[1]
        at += n
    return o


def _exact_select(case, s):
    W, V, n = case["W"], case["V"], case["n"]
    out = {"scores": [], "beam": [], "token": []}
    for b in range(case["B"]):
        x = torch.log_softmax(s["logits"][b].double(), -1) + s["scores"][b].double()[:, None]
        if s["done"] is not None:
            only = torch.full_like(x, -math.inf)
            only[:, EOS] = s["scores"][b].double()
            x = torch.where(s["done"][b][:, None], only, x)
        x = x.flatten()
        taken = torch.zeros(W * V, dtype=torch.bool, device="cuda")
        for _ in range(n):
            best = x.masked_fill(taken, -math.inf).max()
            i = int(torch.nonzero((x == best) & ~taken)[0])
            taken[i] = True
            out["scores"].append(float(x[i]))
            out["beam"].append(i // V)
            out["token"].append(i % V)
    shape = (case["B"], n)
    return {"scores": torch.tensor(out["scores"], dtype=torch.float64, device="cuda").view(shape),
            "beam": torch.tensor(out["beam"], dtype=torch.int32, device="cuda").view(shape),
            "token": torch.tensor(out["token"], dtype=torch.int32, device="cuda").view(shape)}


def _exact_reorder(case, s):
    W, page = case["W"], case["page"]
    slots, moves = s["slots"].tolist(), []
    table = s["table"].clone() if s["caches"] else None
    for b, (parent, length) in enumerate(zip(*_parents(case))):
        old = list(slots[b])
        free = [old[i] for i in range(W) if i not in parent]
        used = set()
        for i, p in enumerate(parent):
            twin = p in used
            used.add(p)
            lane = free.pop(0) if twin else old[p]
            slots[b][i] = lane
            if table is not None:
                table[b * W + i] = s["table"][b * W + p]
                if twin:
                    at = length // page
                    table[b * W + i, at:] = s["own_pages"][lane, at:]
            if twin:
                at = length // page
                part = table is not None and length % page > 0
                moves.append((old[p], lane, int(s["table"][b * W + p, at]) if part else 0,
                              int(s["own_pages"][lane, at]) if part else 0))
    states, caches = [x.clone() for x in s["states"]], [x.clone() for x in s["caches"]]
    for a, z, pa, pz in moves:
        for x, y in zip(states, s["states"]):
            x[z] = y[a]
        if pa != pz:
            for x, y in zip(caches, s["caches"]):
                x[pz] = y[pa]
    out = {"slots": torch.tensor(slots, dtype=torch.int32, device="cuda"), "states": [x.double() for x in states],
           "caches": caches}
    if table is not None:
        out["table"] = table
    return out


def exact(case, seed):
    if case["op"] == "attn" and work(case)["flops"] > 1.2e12:
        return None
    if case["op"] == "select" and case["B"] * case["n"] * case["W"] * case["V"] > 1.5e10:
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "select": _exact_select,
            "reorder": _exact_reorder}[case["op"]](case, s)
