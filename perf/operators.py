"""The 4-bit cache and page operators as calls of one pass each: their plain
form in elementary torch operations, and the library's calls of them.

``own`` selects which of the two ``run`` computes.  A case is one shape of one
operator; ``listed`` gives the fixed ones and ``draw`` more of the same ranges.

Operators
* decode: attention of a few query rows over a cache held in 4 bits (e2m1
  codes, two per byte, and one e4m3 scale per 16 values), flat or paged;
* append: new K/V rows quantised into such a cache, then read back as bf16 (a
  prompt chunk is written once and read by the next chunk's attention);
* fork, admit, compact: page bookkeeping of a paged cache with reference
  counts, and the copies of pages it asks for.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases
def _decode(name, B, n_q, Hq, Hkv, d, cap, lo, hi, causal, page=0, token_major=False, k_global=1.0, v_global=1.0):
    return dict(name=name, op="decode", B=B, n_q=n_q, Hq=Hq, Hkv=Hkv, d=d, cap=cap, lo=lo, hi=hi, causal=causal,
                page=page, token_major=token_major, k_global=k_global, v_global=v_global)


def _append(name, B, n, lo, Hkv, d, cap, page=0, token_major=False, k_global=1.0, v_global=1.0):
    return dict(name=name, op="append", B=B, n=n, lo=lo, Hkv=Hkv, d=d, cap=cap, page=page, token_major=token_major,
                k_global=k_global, v_global=v_global)


def _fork(name, parents, children, n_new, page, max_pages, layers, Hkv, d):
    return dict(name=name, op="fork", parents=parents, children=children, n_new=n_new, page=page, max_pages=max_pages,
                layers=layers, Hkv=Hkv, d=d)


def _admit(name, B, leaving, hi, page, max_pages):
    return dict(name=name, op="admit", B=B, leaving=leaving, hi=hi, page=page, max_pages=max_pages)


def _compact(name, B, max_pages, spare, layers, Hkv, page, d):
    return dict(name=name, op="compact", B=B, max_pages=max_pages, spare=spare, layers=layers, Hkv=Hkv, page=page, d=d)


def listed():
    return [
        # one short chat: the smallest decode call, where latency counts
        _decode("decode one short", 1, 1, 8, 2, 128, 4096, 1000, 1000, False),
        # a token and three drafts verified over a quarter-filled preallocated cache
        _decode("decode verify", 1, 4, 16, 4, 256, 24007, 3000, 3000, True),
        # a served batch of ragged lengths, six-row speculative windows
        _decode("decode ragged", 8, 6, 16, 4, 256, 32768, 1024, 32768, True, k_global=0.5),
        # long contexts: what a 4-bit cache is for
        _decode("decode long", 4, 1, 32, 8, 128, 131072, 131072, 131072, False),
        # many short sequences over 16-position pages stored token by token
        _decode("decode paged", 64, 1, 32, 8, 128, 4096, 1, 4096, False, page=16, token_major=True, v_global=0.25),
        # one decode step's rows of a served batch
        _append("append token", 64, 1, 1, 8, 128, 4096, page=16, token_major=True),
        # ragged prompts of up to 8192 positions into 64-position pages
        _append("append prompts", 4, 8192, 1000, 8, 128, 16384, page=64, k_global=0.5),
        # one request sampled four ways: a latency-bound scheduler step
        _fork("fork small", 1, 3, 1, 16, 64, 2, 2, 128),
        # eight requests of eight beams each, a cache of eight layers
        _fork("fork beams", 8, 7, 1, 16, 64, 8, 8, 128),
        # requests that finish make room for prompts that arrive
        _admit("admit prompts", 256, 64, 4096, 16, 512),
        # a small pool tightened so that its end can be handed back
        _compact("compact small", 16, 32, 100, 2, 2, 16, 128),
        # a large one
        _compact("compact large", 64, 128, 2000, 2, 4, 16, 128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "fork", "admit", "compact"])
    d = rng.choice([128, 256])
    if op in ("decode", "append"):
        page = rng.choice([0, 0, 16, 64, 48, 128])
        tm = rng.random() < 0.4
        kg, vg = rng.choice([1.0, 0.5, 0.125]), rng.choice([1.0, 0.25, 2.0])
    if op == "decode":
        B, n_q, g, Hkv = _log(rng, 1, 64), rng.choice([1, 1, 2, 3, 4, 6]), rng.choice([1, 2, 4, 5, 8, 10]), rng.choice([1, 2, 4, 8])
        # at most an eighth of the largest listed case's positions x heads
        hi = _log(rng, 1, max(2, min(131072, (1 << 19) // (B * Hkv))))
        hi = max(hi, n_q)
        lo = rng.randint(0, hi)
        cap = hi + rng.choice([0, 7, 1000])
        if page:
            cap = (cap + page - 1) // page * page
        return dict(_decode("", B, n_q, Hkv * g, Hkv, d, cap, lo, hi, n_q > 1 or rng.random() < 0.3, page, tm, kg, vg))
    if op == "append":
        Hkv, B = rng.choice([1, 2, 4, 8]), _log(rng, 1, 64)
        n = _log(rng, 1, max(1, min(8192, (1 << 17) // (B * Hkv))))
        cap = n + rng.randint(0, 600)
        if page:
            cap = (cap + page - 1) // page * page
        return dict(_append("", B, n, rng.randint(0, n), Hkv, d, cap, page, tm, kg, vg))
    if op == "fork":
        parents = _log(rng, 1, 16)
        return dict(_fork("", parents, rng.randint(1, max(1, 63 // parents)), rng.randint(1, 6), rng.choice([8, 16, 32]),
                          rng.randint(4, 40), rng.randint(1, 4), rng.choice([1, 2, 4]), d))
    if op == "admit":
        B = _log(rng, 4, 256)
        page, mp = rng.choice([16, 32, 64]), _log(rng, 8, 512)
        return dict(_admit("", B, rng.randint(1, B // 2), rng.randint(page, page * mp), page, mp))
    return dict(_compact("", _log(rng, 2, 64), _log(rng, 4, 100), rng.randint(8, 1500), rng.randint(1, 2), rng.choice([1, 2, 4]), 16, d))


# ------------------------------------------------------------------ format
def _codes_of(x, g):
    """Plain quantisation of x [..., d] (float): e2m1 codes as numbers 0..15
    (uint8, [..., d]) and e4m3 scales [..., d/16].  fp32 throughout."""
    xg = x.float().unflatten(-1, (-1, 16))
    amax = xg.abs().amax(-1)
    finite = amax < math.inf                       # false for NaN too
    s = (amax / (6.0 * g)).clamp(max=448.0)
    s = torch.where(finite, s, math.nan).to(torch.float8_e4m3fn)
    sg = s.float() * g
    y = xg.abs() / sg.unsqueeze(-1)
    y = torch.where((sg > 0).unsqueeze(-1), y, 0.0)   # scale 0 or NaN: zero codes
    # nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code
    n = (y > 0.25).to(torch.uint8)
    n += y >= 0.75
    n += y > 1.25
    n += y >= 1.75
    n += y > 2.5
    n += y >= 3.5
    n += y > 5.0
    n += torch.where(finite.unsqueeze(-1), torch.signbit(xg), False).to(torch.uint8) * 8
    return n.flatten(-2), s


def _pack(n):
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _values(codes, scale, g, dtype=torch.float32):
    """The values that packed codes [..., d/2] and scales [..., d/16] stand for."""
    mags = torch.tensor(E2M1, dtype=dtype, device=codes.device)
    lut = torch.cat([mags, -mags])
    byte = torch.arange(256, device=codes.device)
    pairs = torch.stack([lut[byte & 15], lut[byte >> 4]], -1)
    v = pairs[codes.int()].flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * (scale.to(dtype) * g).unsqueeze(-1)).flatten(-2)


# ------------------------------------------------------------------ inputs
def _lengths(case, seed, most):
    g = torch.Generator().manual_seed(seed * 7 + 1)
    lo, hi = case["lo"], most
    n = torch.randint(lo, hi + 1, (case["B"],), generator=g)
    n[0] = hi
    return n.to(torch.int32)


def _cache_values(shape, gen):
    """Keys and values as projections give them: channels of unequal size."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return x * torch.exp(0.5 * torch.randn(shape[-1], generator=gen, device="cuda"))


def _paged_shape(case):
    max_pages = case["cap"] // case["page"]
    return case["B"] * max_pages + 5, max_pages


def _make_cache(case, gen, seed, filled):
    """k, v codes and scales (flat [B, Hkv, cap, .] or pools [pages, Hkv, page, .]) and the block table."""
    B, Hkv, d, cap, page = case["B"], case["Hkv"], case["d"], case["cap"], case["page"]
    table = None
    if page:
        pages, max_pages = _paged_shape(case)
        table = torch.randperm(pages, generator=torch.Generator().manual_seed(seed + 3))[:B * max_pages]
        table = table.view(B, max_pages).to(torch.int32).cuda()
        lead, rows = pages, page
    else:
        lead, rows = B, cap
    got = []
    for g in (case["k_global"], case["v_global"]):
        shape = (lead, rows, Hkv, d) if case["token_major"] else (lead, Hkv, rows, d)
        if filled:
            n, s = _codes_of(_cache_values(shape, gen), g)
            c = _pack(n)
            del n
        else:
            c = torch.zeros((*shape[:-1], d // 2), dtype=torch.uint8, device="cuda")
            s = torch.zeros((*shape[:-1], d // 16), device="cuda").to(torch.float8_e4m3fn)
        got.append((c.transpose(1, 2), s.transpose(1, 2)) if case["token_major"] else (c, s))
    (k, ks), (v, vs) = got
    return k, v, ks, vs, table


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def prepare(case, seed):
    return {"decode": _prepare_decode, "append": _prepare_append, "fork": _prepare_fork, "admit": _prepare_admit,
            "compact": _prepare_compact}[case["op"]](case, seed)


def _prepare_decode(case, seed):
    gen = _gen(seed)
    k, v, ks, vs, table = _make_cache(case, gen, seed, True)
    lens = _lengths(case, seed, case["hi"])
    q = torch.randn((case["B"], case["n_q"], case["Hq"], case["d"]), generator=gen, device="cuda").to(torch.bfloat16)
    return dict(case=case, q=q, k=k, v=v, ks=ks, vs=vs, table=table, lens=lens.cuda(), longest=int(lens.max()),
                scale=1.0 / math.sqrt(case["d"]))


def _prepare_append(case, seed):
    gen = _gen(seed)
    k, v, ks, vs, table = _make_cache(case, gen, seed, False)
    shape = (case["B"], case["n"], case["Hkv"], case["d"])
    k_new, v_new = (_cache_values(shape, gen).to(torch.bfloat16) for _ in range(2))
    new = _lengths(case, seed, case["n"])
    start = torch.randint(0, case["cap"] - case["n"] + 1, (case["B"],), generator=torch.Generator().manual_seed(seed + 5))
    return dict(case=case, k=k, v=v, ks=ks, vs=vs, table=table, k_new=k_new, v_new=v_new, new=new.cuda(),
                start=start.to(torch.int32).cuda(), after=torch.zeros_like(new).cuda())


def _pools(layers, pages, Hkv, page, d, gen):
    """K and V pools of every layer, in 4 bits: codes and scales."""
    codes = [torch.randint(0, 256, (layers, pages, Hkv, page, d // 2), generator=gen, device="cuda").to(torch.uint8) for _ in range(2)]
    scales = [torch.rand((layers, pages, Hkv, page, d // 16), generator=gen, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    return codes + scales


def _plan(pools):
    """The handle that the library's copies go by, kept with the pools."""
    from decode_attention_preallocated_gb300 import fd
    return fd.PagePools([t for p in pools for t in p.unbind(0)])


def _prepare_fork(case, seed):
    """Parents hold pages; the rows of their children are still empty."""
    gen, host = _gen(seed), torch.Generator().manual_seed(seed + 11)
    P, c, page, mp = case["parents"], case["children"], case["page"], case["max_pages"]
    B, n_new = P * (1 + c), case["n_new"]
    room = page * mp - n_new
    lens = torch.zeros(B, dtype=torch.int32)
    lens[:P] = torch.randint(1, room + 1, (P,), generator=host)
    held = (lens[:P].long() + page - 1) // page
    extra = (n_new + page - 1) // page + 1
    pages = P * mp + B * extra + 9
    order = torch.randperm(pages, generator=host).to(torch.int32)
    j = torch.arange(mp)
    first = torch.cumsum(held, 0) - held
    table = torch.full((B, mp), -1, dtype=torch.int32)
    table[:P] = torch.where(j < held[:, None], order[(first[:, None] + j).clamp(max=pages - 1)], -1)
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[order[:int(held.sum())].long()] = 1
    src = torch.arange(P).repeat_interleave(c).to(torch.int32)
    dst = torch.arange(P, B).to(torch.int32)
    copies = int(((lens[:P] % page != 0).sum()) * c)    # each child of a parent whose last page is part-filled
    pools = _pools(case["layers"], pages, case["Hkv"], page, case["d"], gen)
    return dict(case=case, table=table.cuda(), refs=refs.cuda(), lens=lens.cuda(), src=src.cuda(), dst=dst.cuda(), pools=pools,
                plan=_plan(pools) if own else None, copies=copies, pairs=torch.full((B, 2), -1, dtype=torch.int32, device="cuda"),
                count=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_admit(case, seed):
    """Every sequence holds pages; some have finished and their places get prompts."""
    host = torch.Generator().manual_seed(seed + 13)
    B, page, mp = case["B"], case["page"], case["max_pages"]
    lens = torch.randint(1, case["hi"] + 1, (B,), generator=host)
    held = (lens + page - 1) // page
    leaving = torch.randperm(B, generator=host)[:case["leaving"]]
    new = torch.zeros(B, dtype=torch.int64)
    new[leaving] = torch.randint(1, case["hi"] + 1, (case["leaving"],), generator=host)
    pages = (B + case["leaving"]) * ((case["hi"] + page - 1) // page) + 7
    order = torch.randperm(pages, generator=host).to(torch.int32)
    first = torch.cumsum(held, 0) - held
    j = torch.arange(mp)
    table = torch.where(j < held[:, None], order[(first[:, None] + j).clamp(max=pages - 1)], -1).to(torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[order[:int(held.sum())].long()] = 1
    return dict(case=case, table=table.cuda(), refs=refs.cuda(), lens=lens.to(torch.int32).cuda(), new=new.to(torch.int32).cuda(),
                leaving=leaving.to(torch.int32).cuda(), pairs=torch.full((B, 2), -1, dtype=torch.int32, device="cuda"),
                count=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_compact(case, seed):
    """Pages in use are scattered over a pool that has shrunk in use; some are shared."""
    gen, host = _gen(seed), torch.Generator().manual_seed(seed + 17)
    B, mp = case["B"], case["max_pages"]
    held = torch.randint(0, mp + 1, (B,), generator=host)
    pages = B * mp + case["spare"]
    order = torch.randperm(pages, generator=host).to(torch.int32)
    first = torch.cumsum(held, 0) - held
    j = torch.arange(mp)
    table = torch.where(j < held[:, None], order[(first[:, None] + j).clamp(max=pages - 1)], -1).to(torch.int32)
    table[-1] = torch.where(j < held[0], table[0], -1)          # the last sequence shares the first one's pages
    named = table[table >= 0].long()
    refs = torch.zeros(pages, dtype=torch.int32).index_add_(0, named, torch.ones(len(named), dtype=torch.int32))
    used = int((refs > 0).sum())
    moves = int((refs[used:] > 0).sum())
    pools = _pools(case["layers"], pages, case["Hkv"], case["page"], case["d"], gen)
    return dict(case=case, table=table.cuda(), refs=refs.cuda(), table0=table.cuda(), refs0=refs.cuda(), pools=pools,
                plan=_plan(pools) if own else None, moves=moves,
                pairs=torch.full((max(1, pages // 2), 2), -1, dtype=torch.int32, device="cuda"),
                count=torch.zeros(1, dtype=torch.int32, device="cuda"))


# -------------------------------------------------------------------- runs
def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


def _rows(t, table, n):
    """Positions 0..n-1 of every sequence of a cache: [B, Hkv, n, .]"""
    if table is None:
        return t[:, :, :n]
    page = t.shape[2]
    need = (n + page - 1) // page
    r = t.view(torch.uint8)[table[:, :need].long()]             # [B, need, Hkv, page, .]
    return r.transpose(1, 2).flatten(2, 3)[:, :, :n].view(t.dtype)


def _plain_decode(st):
    case, n = st["case"], st["longest"]
    B, n_q, Hq, Hkv, d = (case[x] for x in ("B", "n_q", "Hq", "Hkv", "d"))
    k = _values(_rows(st["k"], st["table"], n), _rows(st["ks"], st["table"], n), case["k_global"])
    q = st["q"].float().view(B, n_q, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    s = (q @ k.transpose(-1, -2)).view(B, Hkv, -1, n_q, n) * st["scale"]
    del k
    pos, L = torch.arange(n, device="cuda"), st["lens"].view(B, 1, 1, 1, 1)
    last = L - n_q + torch.arange(n_q, device="cuda").view(n_q, 1) if case["causal"] else L - 1
    seen = pos <= last
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    v = _values(_rows(st["v"], st["table"], n), _rows(st["vs"], st["table"], n), case["v_global"])
    o = (p.view(B, Hkv, -1, n) @ v).view(B, Hkv, Hq // Hkv, n_q, d)
    return o.permute(0, 3, 1, 2, 4).reshape(B, n_q, Hq, d).to(torch.bfloat16)


def _own_decode(st):
    from decode_attention_preallocated_gb300 import fd
    case = st["case"]
    return fd.decode_fp4(st["q"], st["k"], st["v"], st["ks"], st["vs"], st["lens"], causal=case["causal"], scale=st["scale"],
                         k_global=case["k_global"], v_global=case["v_global"], block_table=st["table"])


def _plain_append(st):
    case, table = st["case"], st["table"]
    B, n, Hkv, d = case["B"], case["n"], case["Hkv"], case["d"]
    i = torch.arange(n, device="cuda")
    pos = st["start"].view(B, 1) + i
    real = i < st["new"].view(B, 1)
    after = (st["start"] + st["new"]).clamp(max=case["cap"])
    lead, row = torch.arange(B, device="cuda").view(B, 1).expand(B, n), pos.long()
    if table is not None:
        page = st["k"].shape[2]
        lead, row = table.gather(1, (pos // page).long()).long(), (pos % page).long()
    out = []
    for new, c, s, g in ((st["k_new"], st["k"], st["ks"], case["k_global"]), (st["v_new"], st["v"], st["vs"], case["v_global"])):
        codes, scale = _codes_of(new, g)
        codes, scale, sb = _pack(codes), scale.view(torch.uint8), s.view(torch.uint8)
        # rows that are only padding keep what the cache held there
        keep = real.view(B, n, 1, 1)
        c.transpose(1, 2)[lead, row] = torch.where(keep, codes, c.transpose(1, 2)[lead, row])
        sb.transpose(1, 2)[lead, row] = torch.where(keep, scale, sb.transpose(1, 2)[lead, row])
        back = _values(c.transpose(1, 2)[lead, row], sb.transpose(1, 2)[lead, row].view(torch.float8_e4m3fn), g)
        out.append(torch.where(keep, back, 0.0).to(torch.bfloat16))
    return {"k": out[0], "v": out[1], "lengths": after}


def _own_append(st):
    from decode_attention_preallocated_gb300 import fd
    case = st["case"]
    kw = dict(k_global=case["k_global"], v_global=case["v_global"], block_table=st["table"])
    fd.append_fp4(st["k_new"], st["v_new"], st["k"], st["v"], st["ks"], st["vs"], st["start"], new_lengths=st["new"],
                  lengths_out=st["after"], **kw)
    k, v = fd.read_fp4(st["k"], st["v"], st["ks"], st["vs"], st["after"], case["n"], start=st["start"], **kw)
    return {"k": k, "v": v, "lengths": st["after"]}


def _plain_free(st, seqs):
    table, refs, mp = st["table"], st["refs"], st["table"].shape[1]
    seqs = seqs.long()
    rows = table[seqs]
    named = rows >= 0
    refs.index_add_(0, rows.clamp(min=0).long().flatten(), -named.int().flatten())
    table[seqs] = torch.full((len(seqs), mp), -1, dtype=torch.int32, device="cuda")
    st["lens"][seqs] = torch.zeros(len(seqs), dtype=torch.int32, device="cuda")


def _plain_reserve(st, page, n_new):
    """Pages for the next n_new positions of every sequence, in order."""
    table, refs, lens = st["table"], st["refs"], st["lens"]
    B, mp = table.shape
    j = torch.arange(mp, device="cuda")
    L = lens.view(B, 1).long()
    n = n_new.view(-1, 1).long() if torch.is_tensor(n_new) else n_new
    writes = (j >= L // page) & (j < (L + n + page - 1) // page) & (torch.as_tensor(n, device="cuda") > 0)
    e = table.clamp(min=0).long()
    shared = writes & (table >= 0) & (refs[e] > 1)
    slot = torch.arange(B * mp, device="cuda").view(B, mp)
    flat_e, flat_s = e.flatten(), shared.flatten()
    writers = torch.zeros_like(refs).index_add_(0, flat_e, flat_s.int())
    first = torch.full(refs.shape, B * mp, device="cuda").scatter_reduce_(0, flat_e, torch.where(shared, slot, B * mp).flatten(), "amin")
    keeps = shared & (writers[e] == refs[e]) & (first[e] == slot)
    need = writes & ((table < 0) | (shared & ~keeps))
    free = refs == 0
    rank = torch.cumsum(need.flatten(), 0).view(B, mp) - 1
    place = torch.where(free, torch.cumsum(free, 0) - 1, len(refs))
    pages = torch.zeros(len(refs) + 1, dtype=torch.int32, device="cuda").scatter_(0, place, torch.arange(len(refs), dtype=torch.int32, device="cuda"))
    new = pages[rank.clamp(min=0, max=len(refs))]
    leaves = need & (table >= 0)
    copy = leaves & (j * page < L)
    prank = torch.where(copy, torch.cumsum(copy.flatten(), 0).view(B, mp) - 1, B)
    room = torch.cat([st["pairs"], st["pairs"][:1]])
    room.index_copy_(0, prank.flatten(), torch.stack([table, new], -1).view(-1, 2))
    st["pairs"].copy_(room[:B])
    st["count"].copy_(copy.sum().int().view(1))
    refs.index_add_(0, flat_e, -leaves.int().flatten())
    refs.index_add_(0, torch.where(need, new, 0).long().flatten(), need.int().flatten())
    table.copy_(torch.where(need, new, table))


def _plain_fork(st, page):
    table, refs = st["table"], st["refs"]
    src, dst = st["src"].long(), st["dst"].long()
    rows = table[src]
    j = torch.arange(table.shape[1], device="cuda")
    rows = torch.where(j * page < st["lens"][src].view(-1, 1), rows, -1)
    refs.index_add_(0, rows.clamp(min=0).long().flatten(), (rows >= 0).int().flatten())
    table[dst] = rows
    st["lens"][dst] = st["lens"][src]


def _plain_copy(st, n):
    src, dst = st["pairs"][:n, 0].long(), st["pairs"][:n, 1].long()
    k, v, ks, vs = (p.view(torch.uint8) for p in st["pools"])
    k[:, dst] = k[:, src]
    v[:, dst] = v[:, src]
    ks[:, dst] = ks[:, src]
    vs[:, dst] = vs[:, src]


def _books(st):
    return {"table": st["table"], "refs": st["refs"], "lens": st.get("lens"), "pairs": st["pairs"], "count": st["count"],
            "pools": st.get("pools")}


def _plain_fork_pass(st):
    case = st["case"]
    _plain_free(st, st["dst"])
    _plain_fork(st, case["page"])
    _plain_reserve(st, case["page"], case["n_new"])
    _plain_copy(st, st["copies"])
    return _books(st)


def _own_fork_pass(st):
    from decode_attention_preallocated_gb300 import fd
    case = st["case"]
    books = (st["table"], st["lens"], st["refs"], case["page"])
    fd.pages_free(*books, seqs=st["dst"])
    fd.pages_fork(*books, st["src"], st["dst"])
    fd.pages_reserve(*books, case["n_new"], pairs=st["pairs"], count=st["count"])
    fd.pages_copy(st["plan"], st["pairs"], st["count"])
    return _books(st)


def _plain_admit(st):
    _plain_free(st, st["leaving"])
    _plain_reserve(st, st["case"]["page"], st["new"])
    return _books(st)


def _own_admit(st):
    from decode_attention_preallocated_gb300 import fd
    books = (st["table"], st["lens"], st["refs"], st["case"]["page"])
    fd.pages_free(*books, seqs=st["leaving"])
    fd.pages_reserve(*books, st["new"], pairs=st["pairs"], count=st["count"])
    return _books(st)


def _plain_compact(st):
    table, refs = st["table"], st["refs"]
    table.copy_(st["table0"])                  # the books as requests left them
    refs.copy_(st["refs0"])
    P, half = len(refs), len(st["pairs"])
    used = refs > 0
    n_used = used.sum()
    idx = torch.arange(P, dtype=torch.int32, device="cuda")
    hole, mover = ~used & (idx < n_used), used & (idx >= n_used)
    hole_at = torch.where(hole, torch.cumsum(hole, 0) - 1, half)
    mover_at = torch.where(mover, torch.cumsum(mover, 0) - 1, half)
    room = torch.cat([st["pairs"], st["pairs"][:1]])
    room[:, 0].scatter_(0, mover_at, idx)
    room[:, 1].scatter_(0, hole_at, idx)
    st["pairs"].copy_(room[:half])
    count = mover.sum()
    st["count"].copy_(count.int().view(1))
    goes = torch.where(mover, st["pairs"][:, 1][mover_at.clamp(max=half - 1)], idx)
    refs.copy_(torch.zeros_like(refs).index_add_(0, goes.long(), torch.where(used, refs, 0)))
    table.copy_(torch.where(table >= 0, goes[table.clamp(min=0).long()], table))
    _plain_copy(st, st["moves"])
    return _books(st)


def _own_compact(st):
    from decode_attention_preallocated_gb300 import fd
    st["table"].copy_(st["table0"])
    st["refs"].copy_(st["refs0"])
    fd.pages_compact(st["table"], st["refs"], pairs=st["pairs"], count=st["count"])
    fd.pages_copy(st["plan"], st["pairs"], st["count"])
    return _books(st)


_PLAIN = {"decode": _plain_decode, "append": _plain_append, "fork": _plain_fork_pass, "admit": _plain_admit, "compact": _plain_compact}
_OWN = {"decode": _own_decode, "append": _own_append, "fork": _own_fork_pass, "admit": _own_admit, "compact": _own_compact}


# ------------------------------------------------------------- floor, exact
def work(case):
    op = case["op"]
    if op == "decode":
        # the mean length; each sequence's K and V read once: codes d/2 bytes and scales d/16 bytes a row each
        positions = case["B"] * (case["lo"] + case["hi"]) / 2
        rows = case["B"] * case["n_q"] * case["Hq"] * case["d"]
        return {"bytes": positions * case["Hkv"] * (case["d"] + case["d"] / 8) + 4 * rows,
                "flops": 4 * positions * case["Hq"] * case["n_q"] * case["d"]}
    if op == "append":
        # bf16 rows read, codes and scales written, read again, bf16 rows written
        values = case["B"] * (case["lo"] + case["n"]) / 2 * case["Hkv"] * case["d"] * 2
        return {"bytes": values * (2 + 0.5625 + 0.5625 + 2), "flops": values * 4}
    table = 4 * case["max_pages"]
    if op == "fork":
        B = case["parents"] * (1 + case["children"])
        page_bytes = case["layers"] * case["Hkv"] * case["page"] * case["d"] * 1.125
        copies = case["parents"] * case["children"] * (1 - 1 / case["page"])
        return {"bytes": 2 * copies * page_bytes + 3 * B * table, "flops": 0}
    if op == "admit":
        named = case["leaving"] * (case["hi"] / 2 / case["page"])
        return {"bytes": 4 * named * 6 + 4 * case["B"] * case["hi"] / 2 / case["page"], "flops": 0}
    used = case["B"] * case["max_pages"] / 2
    moves = used * (used + case["spare"]) / (2 * used + case["spare"])
    page_bytes = case["layers"] * case["Hkv"] * case["page"] * case["d"] * 1.125
    return {"bytes": 2 * moves * page_bytes + 4 * (2 * used + case["spare"]) + 2 * case["B"] * table, "flops": 0}


def exact(case, seed):
    if case["op"] == "decode":
        return _exact_decode(case, seed)
    if case["op"] == "append":
        return _exact_append(case, seed)
    return None          # whole numbers and copies


def _exact_value_table():
    """e2m1: sign, two exponent bits with bias 1, one mantissa bit."""
    vals = []
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        mag = m * 0.5 if e == 0 else 2.0 ** (e - 1) * (1 + m * 0.5)
        vals.append(-mag if c & 8 else mag)
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _exact_rows(codes, scale, g):
    """[n, d/2] bytes and [n, d/16] scales -> [n, d] in 64 bits."""
    t = _exact_value_table()
    out = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=torch.float64, device="cuda")
    out[:, 0::2] = t[(codes % 16).int()]
    out[:, 1::2] = t[(codes // 16).int()]
    return out * (scale.double() * g).repeat_interleave(16, dim=1)


def _exact_decode(case, seed):
    st = prepare(case, seed)
    group = case["Hq"] // case["Hkv"]
    out = torch.zeros((case["B"], case["n_q"], case["Hq"], case["d"]), dtype=torch.float64, device="cuda")
    lens = st["lens"].tolist()
    for b in range(case["B"]):
        L = lens[b]
        if L == 0:
            continue
        for h in range(case["Hkv"]):
            def rows(t):
                if st["table"] is None:
                    return t[b, h, :L]
                pages = st["table"][b, :-(-L // case["page"])].long()
                return t.view(torch.uint8)[pages, h].reshape(-1, t.shape[-1])[:L].view(t.dtype)
            k = _exact_rows(rows(st["k"]), rows(st["ks"]), case["k_global"])
            v = _exact_rows(rows(st["v"]), rows(st["vs"]), case["v_global"])
            q = st["q"][b, :, h * group:(h + 1) * group].double()          # [n_q, group, d]
            s = torch.einsum("igd,jd->igj", q, k) * st["scale"]
            if case["causal"]:
                seen = torch.arange(L, device="cuda") <= (L - case["n_q"] + torch.arange(case["n_q"], device="cuda")).view(-1, 1)
                s = s.masked_fill(~seen.unsqueeze(1), -math.inf)
            w = torch.softmax(s, -1).nan_to_num(0.0)                        # a row that sees nothing gives 0
            out[b, :, h * group:(h + 1) * group] = torch.einsum("igj,jd->igd", w, v)
    return out


def _exact_append(case, seed):
    st = prepare(case, seed)
    table = _exact_value_table()[:8]
    mids = (table[1:] + table[:-1]) / 2
    res = []
    for x, g in ((st["k_new"], case["k_global"]), (st["v_new"], case["v_global"])):
        x = x.double().unflatten(-1, (-1, 16))
        want = x.abs().amax(-1) / (6.0 * g)
        # nearest e4m3: three mantissa bits, least exponent -6
        e = torch.floor(torch.log2(want.clamp(min=2.0 ** -20))).clamp(min=-6.0)
        step = torch.exp2(e - 3)
        s = (torch.round(want / step) * step).clamp(max=448.0)
        y = torch.where(s.unsqueeze(-1) > 0, x.abs() / (s * g).unsqueeze(-1), 0.0)
        low = torch.searchsorted(mids, y)                                   # mids below y
        at = mids[low.clamp(max=6)] == y
        code = low + (at & (low % 2 == 1)).long()                           # a tie goes to the even code
        val = torch.sign(x) * table[code] * (s * g).unsqueeze(-1)
        real = torch.arange(case["n"], device="cuda") < st["new"].view(-1, 1)
        res.append(val.flatten(-2) * real.view(case["B"], case["n"], 1, 1))
    return {"k": res[0], "v": res[1], "lengths": None}
