"""Writing and attending a prompt chunk over a paged cache, and a beam search's
step over the same pages, as calls of one pass each: their plain form in
elementary torch operations, and the library's calls of them.

``own`` selects which of the two ``run`` computes.  A case is one shape of one
operator; ``listed`` gives the fixed ones and ``draw`` more of the same ranges.

Operators
* append: new K/V rows written into a bf16 or int8 cache, flat or paged, keys
  and queries rotated to their positions on the way;
* prefill: attention of a chunk of new tokens over such a cache;
* select: the best continuations of a beam search over beams and vocabulary;
* reorder: the block table's rows follow the beams that were selected.
"""
import math

import torch

own = False


# ------------------------------------------------------------------- cases
def _append(name, B, n, lo, Hq, Hkv, d, cap, page=0, int8=False, r=0, interleaved=False, token_major=False):
    return dict(name=name, op="append", B=B, n=n, lo=lo, Hq=Hq, Hkv=Hkv, d=d, cap=cap, page=page, int8=int8, r=r or d,
                interleaved=interleaved, token_major=token_major)


def _prefill(name, B, n, new_lo, before_lo, before_hi, Hq, Hkv, d, page=0, int8=False, causal=True, token_major=False):
    """new_lo .. n new tokens a sequence behind before_lo .. before_hi cached ones."""
    return dict(name=name, op="prefill", B=B, n=n, new_lo=new_lo, before_lo=before_lo, before_hi=before_hi, Hq=Hq, Hkv=Hkv,
                d=d, page=page, int8=int8, causal=causal, token_major=token_major)


def _select(name, B, K, V, n_out, bf16, ended=0.0):
    return dict(name=name, op="select", B=B, K=K, V=V, n_out=n_out, bf16=bf16, ended=ended)


def _reorder(name, groups, K, page, max_pages):
    return dict(name=name, op="reorder", groups=groups, K=K, page=page, max_pages=max_pages)


def listed():
    return [
        # one decode step's rows of a served batch: latency counts
        _append("append token", 64, 1, 1, 32, 8, 128, 4096, page=16, token_major=True),
        # ragged prompt chunks of up to 2048 positions into 64-position pages
        _append("append prompts", 8, 2048, 300, 32, 8, 128, 4096, page=64),
        # the same into an int8 cache, a quarter of each head rotated
        _append("append int8", 4, 1024, 100, 16, 4, 256, 1040, page=16, int8=True, r=64),
        # a short question behind a short chat: the smallest call
        _prefill("prefill short", 1, 37, 37, 963, 963, 8, 2, 128),
        # a question of a few tokens about a long document, per sequence
        _prefill("prefill question", 4, 16, 5, 30000, 65536, 32, 8, 128, page=16, token_major=True),
        # one chunk of a long prompt: the serving engine's ordinary step
        _prefill("prefill chunk", 1, 2048, 2048, 30720, 30720, 32, 8, 128, page=64),
        # a batch of ragged prompts from their first token, wide heads, flat cache
        _prefill("prefill prompts", 8, 4096, 500, 0, 0, 16, 4, 256),
        # ragged chunks over an int8 cache
        _prefill("prefill int8", 4, 512, 200, 1000, 8000, 32, 8, 128, page=64, int8=True),
        # one request's four beams: the smallest selection
        _select("select one", 1, 4, 32000, 8, False),
        # many requests of eight beams over a large vocabulary, some beams ended
        _select("select batch", 32, 8, 128000, 16, True, 0.2),
        # four beams change places
        _reorder("reorder one", 1, 4, 16, 128),
        # the beams of many requests, long contexts
        _reorder("reorder batch", 32, 8, 16, 2048),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "append", "prefill", "prefill", "prefill", "select", "reorder"])
    d, Hkv, page = rng.choice([128, 256]), rng.choice([1, 2, 4, 8]), rng.choice([0, 0, 16, 64, 48, 128, 20])
    tm, int8 = rng.random() < 0.4, rng.random() < 0.35
    Hq = Hkv * rng.choice([1, 2, 4, 4, 5, 6, 8])
    if op == "append":
        B = _log(rng, 1, 64)
        n = _log(rng, 1, max(1, min(4096, (1 << 22) // (B * Hq * d))))
        cap = n + rng.randint(0, 600)
        if page:
            cap = (cap + page - 1) // page * page
        return dict(_append("", B, n, rng.randint(0, n), Hq, Hkv, d, cap, page, int8, rng.choice([d, d, d // 2, 64]),
                            rng.random() < 0.4, tm))
    if op == "prefill":
        B, n = _log(rng, 1, 16), _log(rng, 1, 4096)
        n = min(n, max(1, 8192 // B))
        # at most half the largest listed case's pairs of positions and heads
        room = max(1, (1 << 30) // (B * n * Hq * d // 128))
        hi = _log(rng, 1, max(2, min(65536, room)))
        return dict(_prefill("", B, n, rng.randint(0, n), rng.randint(0, hi), hi, Hq, Hkv, d, page, int8, rng.random() < 0.8, tm))
    if op == "select":
        B, K = _log(rng, 1, 48), rng.choice([1, 2, 3, 4, 5, 8, 10, 16])
        V = _log(rng, 500, min(160000, (1 << 25) // (B * K)))
        return dict(_select("", B, K, V, rng.choice([K, 2 * K]), rng.random() < 0.5, rng.choice([0.0, 0.25])))
    return dict(_reorder("", _log(rng, 1, 48), rng.choice([2, 3, 4, 5, 8]), rng.choice([8, 16, 32, 64]), _log(rng, 4, 1500)))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _host(seed, salt):
    return torch.Generator().manual_seed(seed * 13 + salt)


def _between(lo, hi, B, gen):
    """B whole numbers of lo .. hi, the first of them hi."""
    x = torch.randint(lo, hi + 1, (B,), generator=gen)
    x[0] = hi
    return x.to(torch.int32)


def _values(shape, gen):
    """Keys and values as projections give them: channels of unequal size."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return x * torch.exp(0.3 * torch.randn(shape[-1], generator=gen, device="cuda"))


def _int8_of(x):
    """Codes and scales of x [..., d] (fp32), one scale a row."""
    s = x.abs().amax(-1) / 127.0
    y = torch.where((s > 0).unsqueeze(-1), x / s.unsqueeze(-1), 0.0)
    return torch.round(y).to(torch.int8), s


def _cache(case, B, cap, gen, host, filled):
    """k, v (and the scales of int8 ones): flat [B, Hkv, cap, d] or pools [pages, Hkv, page, d] with a block table."""
    Hkv, d, page, table = case["Hkv"], case["d"], case["page"], None
    lead, rows = B, cap
    if page:
        max_pages = (cap + page - 1) // page
        lead, rows = B * max_pages + 3, page
        table = torch.randperm(lead, generator=host)[:B * max_pages].view(B, max_pages).to(torch.int32).cuda()
    got = []
    for _ in range(2):
        shape = (lead, rows, Hkv, d) if case["token_major"] else (lead, Hkv, rows, d)
        x = _values(shape, gen) if filled else torch.zeros(shape, device="cuda")
        pair = _int8_of(x) if case["int8"] else (x.to(torch.bfloat16), None)
        got.append(tuple(t.transpose(1, 2) if t is not None and case["token_major"] else t for t in pair))
    return got[0][0], got[1][0], got[0][1], got[1][1], table


def prepare(case, seed):
    return {"append": _prepare_append, "prefill": _prepare_prefill, "select": _prepare_select, "reorder": _prepare_reorder}[case["op"]](case, seed)


def _prepare_append(case, seed):
    gen, host = _gen(seed), _host(seed, 1)
    B, n, Hq, Hkv, d, r = (case[x] for x in ("B", "n", "Hq", "Hkv", "d", "r"))
    k, v, ks, vs, table = _cache(case, B, case["cap"], gen, host, False)
    # one projection gives queries, keys and values side by side
    qkv = _values((B, n, Hq + 2 * Hkv, d), gen).to(torch.bfloat16)
    q, k_new, v_new = qkv.split([Hq, Hkv, Hkv], 2)
    angle = torch.arange(case["cap"], dtype=torch.float64, device="cuda").view(-1, 1) * \
        10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    new = _between(case["lo"], n, B, host)
    start = torch.randint(0, case["cap"] - n + 1, (B,), generator=host).to(torch.int32)
    values = [torch.zeros_like(x, dtype=torch.bfloat16) for x in (k, v)] if case["int8"] else None
    return dict(case=case, k=k, v=v, ks=ks, vs=vs, table=table, q=q, k_new=k_new, v_new=v_new,
                rope=torch.cat([angle.cos(), angle.sin()], 1).float(), new=new.cuda(), start=start.cuda(),
                after=torch.zeros(B, dtype=torch.int32, device="cuda"), q_out=torch.zeros((B, n, Hq, d), dtype=torch.bfloat16, device="cuda"),
                values=values)


def _prepare_prefill(case, seed):
    gen, host = _gen(seed), _host(seed, 2)
    B, n, Hq, d = (case[x] for x in ("B", "n", "Hq", "d"))
    new = _between(case["new_lo"], n, B, host)
    lens = new + _between(case["before_lo"], case["before_hi"], B, host)
    k, v, ks, vs, table = _cache(case, B, n + case["before_hi"], gen, host, True)
    q = torch.randn((B, n, Hq, d), generator=gen, device="cuda").to(torch.bfloat16)
    return dict(case=case, k=k, v=v, ks=ks, vs=vs, table=table, q=q, new=new.cuda(), lens=lens.cuda(), longest=int(lens.max()),
                scale=1.0 / math.sqrt(d), out=torch.zeros_like(q))


def _prepare_select(case, seed):
    gen, host = _gen(seed), _host(seed, 3)
    B, K, V = case["B"], case["K"], case["V"]
    # logits of a language model: most words far below a few likely ones
    logits = 2.5 * torch.randn((B, K, V), generator=gen, device="cuda")
    logits += 6.0 * (torch.rand((B, K, V), generator=gen, device="cuda") < 40.0 / V)
    if case["bf16"]:
        logits = logits.to(torch.bfloat16)
    scores = -20.0 * torch.rand((B, K), generator=gen, device="cuda") - 1.0
    ended = (torch.rand((B, K), generator=host) < case["ended"]).to(torch.int32).cuda()
    return dict(case=case, logits=logits, scores=scores, ended=ended, end=2)


def _prepare_reorder(case, seed):
    """Each group's beams hold a shared prefix and pages of their own; some beams go on twice, some end."""
    host = _host(seed, 4)
    G, K, page, mp = (case[x] for x in ("groups", "K", "page", "max_pages"))
    B = G * K
    shared = torch.randint(0, mp, (G,), generator=host).repeat_interleave(K)
    lens = torch.randint(1, page * mp + 1, (G,), generator=host).repeat_interleave(K)
    held = (lens + page - 1) // page
    shared = torch.minimum(shared, held - 1)
    j = torch.arange(mp)
    common = j < shared[:, None]
    fresh = (j < held[:, None]) & (~common | (torch.arange(B) % K == 0)[:, None])
    pages = B * mp + 7
    order = torch.randperm(pages, generator=host).to(torch.int32)
    table = torch.full((B, mp), -1, dtype=torch.int32)
    table[fresh] = order[:int(fresh.sum())]
    first = table.view(G, K, mp)[:, :1].expand(G, K, mp).reshape(B, mp)
    table = torch.where(common, first, table)
    named = table[table >= 0].long()
    refs = torch.zeros(pages, dtype=torch.int32).index_add_(0, named, torch.ones(len(named), dtype=torch.int32))
    src = (torch.randint(0, K, (G, K), generator=host) + K * torch.arange(G).view(G, 1)).flatten().to(torch.int32)
    kept = torch.cat([table.flatten(), refs, lens.to(torch.int32)]).cuda()
    books = kept.clone()
    return dict(case=case, kept=kept, books=books, table=books[:B * mp].view(B, mp), refs=books[B * mp:B * mp + pages],
                lens=books[B * mp + pages:], src=src.cuda())


# -------------------------------------------------------------------- runs
def run(state):
    if own:
        return _OWN[state["case"]["op"]](state)
    return _PLAIN[state["case"]["op"]](state)


def _rotated(x, st, pos):
    """x [B, n, H, d] in fp32 with its first r dimensions rotated by the table's rows pos [B, n]."""
    case, x = st["case"], x.float()
    r = case["r"]
    at = st["rope"][pos.long()].unsqueeze(2)
    cos, sin = at[..., :r // 2], at[..., r // 2:]
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_append(st):
    case, table = st["case"], st["table"]
    B, n = case["B"], case["n"]
    i = torch.arange(n, device="cuda")
    pos = st["start"].view(B, 1) + i
    real = (i < st["new"].view(B, 1)).view(B, n, 1, 1)
    lead, row = torch.arange(B, device="cuda").view(B, 1).expand(B, n), pos.long()
    if table is not None:
        page = case["page"]
        lead, row = table.gather(1, (pos // page).long()).long(), (pos % page).long()

    def put(cache, rows):
        # rows that are only padding keep what the cache held there
        at = cache.transpose(1, 2)
        at[lead, row] = torch.where(real if rows.dim() == 4 else real[..., 0], rows, at[lead, row])

    st["q_out"].copy_(torch.where(real, _rotated(st["q"], st, pos).to(torch.bfloat16), st["q_out"]))
    new = {"k": _rotated(st["k_new"], st, pos), "v": st["v_new"].float()}
    if case["int8"]:
        (kc, ks), (vc, vs) = _int8_of(new["k"]), _int8_of(new["v"])
        put(st["k"], kc)
        put(st["v"], vc)
        put(st["ks"], ks)
        put(st["vs"], vs)
    else:
        put(st["k"], new["k"].to(torch.bfloat16))
        put(st["v"], new["v"].to(torch.bfloat16))
    st["after"].copy_((st["start"] + st["new"]).clamp(max=case["cap"]))
    return _written(st)


def _written(st):
    if not st["case"]["int8"]:
        return {"q": st["q_out"], "k": st["k"], "v": st["v"], "lengths": st["after"]}
    k, v = st["values"]              # what the codes stand for
    torch.mul(st["k"], st["ks"].unsqueeze(-1), out=k)
    torch.mul(st["v"], st["vs"].unsqueeze(-1), out=v)
    return {"q": st["q_out"], "k": k, "v": v, "k_scale": st["ks"], "v_scale": st["vs"], "lengths": st["after"]}


def _own_append(st):
    from decode_attention_preallocated_gb300 import fd
    case = st["case"]
    fd.append(st["k_new"], st["v_new"], st["k"], st["v"], st["start"], new_lengths=st["new"], lengths_out=st["after"], q=st["q"],
              q_out=st["q_out"], rope=st["rope"], interleaved=case["interleaved"], k_scale=st["ks"], v_scale=st["vs"],
              block_table=st["table"])
    return _written(st)


def _rows(t, table, n):
    """Positions 0..n-1 of every sequence of a cache: [B, Hkv, n, ...]"""
    if table is None:
        return t[:, :, :n]
    page = t.shape[2]
    return t[table[:, :(n + page - 1) // page].long()].transpose(1, 2).flatten(2, 3)[:, :, :n]


def _plain_prefill(st):
    case, L = st["case"], st["longest"]
    B, n, Hq, Hkv, d = (case[x] for x in ("B", "n", "Hq", "Hkv", "d"))
    g = Hq // Hkv

    def numbers(cache, scale):
        x = _rows(cache, st["table"], L).float()
        return x if scale is None else x * _rows(scale, st["table"], L).unsqueeze(-1)

    q = st["q"].float().view(B, n, Hkv, g, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * n, d)
    s = (q @ numbers(st["k"], st["ks"]).transpose(-1, -2)).view(B, Hkv, g, n, L)
    i, j = torch.arange(n, device="cuda").view(n, 1), torch.arange(L, device="cuda")
    lens, new = st["lens"].view(B, 1, 1), st["new"].view(B, 1, 1)
    seen = j <= lens - new + i if case["causal"] else j < lens.expand(B, n, 1)
    s = s.mul_(st["scale"]).masked_fill_(~seen.view(B, 1, 1, n, L), -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, g * n, L) @ numbers(st["v"], st["vs"])).view(B, Hkv, g, n, d) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, d).to(torch.bfloat16)
    # rows that are only padding are left as they were
    st["out"].copy_(torch.where((i.view(1, n) < st["new"].view(B, 1)).view(B, n, 1, 1), o, st["out"]))
    return st["out"]


def _own_prefill(st):
    from decode_attention_preallocated_gb300 import fd
    return fd.prefill(st["q"], st["k"], st["v"], st["lens"], new_lengths=st["new"], causal=st["case"]["causal"], scale=st["scale"],
                      k_scale=st["ks"], v_scale=st["vs"], block_table=st["table"], out=st["out"])


def _plain_select(st):
    case = st["case"]
    B, K, V, n = (case[x] for x in ("B", "K", "V", "n_out"))
    x = st["logits"].float()
    token = torch.arange(V, device="cuda")
    ended = (st["ended"] != 0).unsqueeze(-1)
    # a beam that has ended goes on by its end token alone, at no cost
    x = torch.where(ended, torch.where(token == st["end"], 0.0, -math.inf), x)
    m = x.amax(-1, keepdim=True).double()
    m = torch.where(m == -math.inf, 0.0, m)
    lse = (m + torch.exp(x.double() - m).sum(-1, keepdim=True).log()).float()
    # each beam's best: by logit, then by lower token; the key is the number's
    # bits in the order of the numbers, and the token below them
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7fffffff), bits) * (1 << 32) + (V - 1 - token)
    best = key.topk(min(n, V), -1).values
    token = V - 1 - (best & 0xffffffff)
    logit = x.gather(-1, token)
    score = st["scores"].double().unsqueeze(-1) + (logit.double() - lse.double())
    # the best of all beams; equal ones in the order of beams
    score, at = score.flatten(1).sort(stable=True, dim=-1, descending=True)
    score, at = score[:, :n], at[:, :n]
    there = score > -math.inf
    beam = at // token.shape[-1] + K * torch.arange(B, device="cuda").view(B, 1)
    token = token.flatten(1).gather(1, at)
    none = torch.full((), -1, dtype=torch.int64, device="cuda")
    return {"scores": score.float(), "beams": torch.where(there, beam, none).int(), "tokens": torch.where(there, token, none).int()}


def _own_select(st):
    from decode_attention_preallocated_gb300 import fd
    scores, beams, tokens = fd.beam_select(st["logits"], st["scores"], st["case"]["n_out"], finished=st["ended"], end_token=st["end"])
    return {"scores": scores, "beams": beams, "tokens": tokens}


def _books(st):
    return {"table": st["table"], "refs": st["refs"], "lens": st["lens"]}


def _plain_reorder(st):
    st["books"].copy_(st["kept"])        # the books as the step before left them
    table, refs, lens, page = st["table"], st["refs"], st["lens"], st["case"]["page"]
    B, mp = table.shape
    src, b = st["src"].long(), torch.arange(B, device="cuda")
    length = lens[src]
    j = torch.arange(mp, device="cuda")
    taken = torch.where(j * page < length.view(B, 1), table[src], -1)
    taken = torch.where((src == b).view(B, 1), table, taken)
    refs.index_add_(0, table.clamp(min=0).long().flatten(), -(table >= 0).int().flatten())
    refs.index_add_(0, taken.clamp(min=0).long().flatten(), (taken >= 0).int().flatten())
    table.copy_(taken)
    lens.copy_(length)
    return _books(st)


def _own_reorder(st):
    from decode_attention_preallocated_gb300 import fd
    st["books"].copy_(st["kept"])
    fd.pages_reorder(st["table"], st["lens"], st["refs"], st["case"]["page"], st["src"])
    return _books(st)


_PLAIN = {"append": _plain_append, "prefill": _plain_prefill, "select": _plain_select, "reorder": _plain_reorder}
_OWN = {"append": _own_append, "prefill": _own_prefill, "select": _own_select, "reorder": _own_reorder}


# ------------------------------------------------------------- floor, exact
def work(case):
    op = case["op"]
    if op == "append":
        # the mean count of new rows: q, k and v read, q, k and v written; the table's rows of cosines and sines
        rows = case["B"] * (case["lo"] + case["n"]) / 2
        kv = 2 * case["Hkv"] * case["d"]
        held = kv * (1 if case["int8"] else 2) + (8 * case["Hkv"] if case["int8"] else 0)
        return {"bytes": rows * (4 * case["Hq"] * case["d"] + 2 * kv + held + 4 * case["r"]),
                "flops": rows * (3 * case["r"] * (case["Hq"] + case["Hkv"]) + (4 * kv if case["int8"] else 0))}
    if op == "prefill":
        new = (case["new_lo"] + case["n"]) / 2
        before = (case["before_lo"] + case["before_hi"]) / 2
        seen = before + (new / 2 if case["causal"] else new)
        row = case["d"] * (1 if case["int8"] else 2) + (4 if case["int8"] else 0)
        return {"bytes": case["B"] * (2 * (before + new) * case["Hkv"] * row + 4 * new * case["Hq"] * case["d"]),
                "flops": 4.0 * case["B"] * new * seen * case["Hq"] * case["d"]}
    if op == "select":
        n = case["B"] * case["K"] * case["V"]
        return {"bytes": n * (2 if case["bf16"] else 4) + 12 * case["B"] * case["n_out"], "flops": 4 * n}
    # half of the table's entries name pages: read, written, and their counts changed
    return {"bytes": 4 * case["groups"] * case["K"] * case["max_pages"] * 2, "flops": 0}


def exact(case, seed):
    return {"append": _exact_append, "prefill": _exact_prefill, "select": _exact_select, "reorder": lambda c, s: None}[case["op"]](case, seed)


def _exact_append(case, seed):
    st = prepare(case, seed)
    half, r = case["r"] // 2, case["r"]
    after = (st["start"] + st["new"]).clamp(max=case["cap"]).tolist()
    start = st["start"].tolist()
    q_out = st["q_out"].double()
    caches = {x: st[x].double() for x in "kv"}
    scales = {x: st[x + "s"].double() for x in "kv"} if case["int8"] else None
    one = torch.arange(half, device="cuda")
    first, second = (2 * one, 2 * one + 1) if case["interleaved"] else (one, one + half)
    for b in range(case["B"]):
        p = torch.arange(start[b], after[b], device="cuda")
        cos, sin = st["rope"][p, :half].double().unsqueeze(1), st["rope"][p, half:].double().unsqueeze(1)

        def turn(x):
            x = x[b, :len(p)].double()
            y = x.clone()
            y[..., first] = x[..., first] * cos - x[..., second] * sin
            y[..., second] = x[..., second] * cos + x[..., first] * sin
            return y
        q_out[b, :len(p)] = turn(st["q"])
        lead, row = (p * 0 + b, p) if st["table"] is None else (st["table"][b, p // case["page"]].long(), p % case["page"])
        for x, rows in (("k", turn(st["k_new"])), ("v", st["v_new"][b, :len(p)].double())):
            if case["int8"]:
                s = rows.abs().amax(-1, keepdim=True) / 127
                scales[x][lead, :, row] = s.squeeze(-1)
                rows = torch.where(s > 0, torch.round(rows / s) * s, 0.0)
            caches[x][lead, :, row] = rows
    res = {"q": q_out, "k": caches["k"], "v": caches["v"], "lengths": None}
    if case["int8"]:
        res.update(k_scale=scales["k"], v_scale=scales["v"])
    return res


def _exact_prefill(case, seed):
    st = prepare(case, seed)
    group = case["Hq"] // case["Hkv"]
    out = torch.zeros((case["B"], case["n"], case["Hq"], case["d"]), dtype=torch.float64, device="cuda")
    lens, new = st["lens"].tolist(), st["new"].tolist()
    for b in range(case["B"]):
        L, t = lens[b], new[b]
        for h in range(case["Hkv"] if t and L else 0):
            def rows(cache, scale):
                if st["table"] is None:
                    x, s = cache[b, h, :L], None if scale is None else scale[b, h, :L]
                else:
                    pages = st["table"][b, :-(-L // case["page"])].long()
                    x = cache[pages, h].reshape(-1, case["d"])[:L]
                    s = None if scale is None else scale[pages, h].reshape(-1)[:L]
                return x.double() if s is None else x.double() * s.double().unsqueeze(-1)
            k, v = rows(st["k"], st["ks"]), rows(st["v"], st["vs"])
            for first in range(0, t, 512):
                q = st["q"][b, first:min(t, first + 512), h * group:(h + 1) * group].double()
                s = torch.einsum("igd,jd->igj", q, k) * st["scale"]
                if case["causal"]:
                    last = L - t + first + torch.arange(len(q), device="cuda")
                    s = s.masked_fill((torch.arange(L, device="cuda") > last.view(-1, 1)).unsqueeze(1), -math.inf)
                w = torch.softmax(s, -1).nan_to_num(0.0)
                out[b, first:first + len(q), h * group:(h + 1) * group] = torch.einsum("igj,jd->igd", w, v)
    return out


def _exact_select(case, seed):
    st = prepare(case, seed)
    logp = torch.log_softmax(st["logits"].double(), -1)
    ended = st["ended"].bool()
    logp[ended] = -math.inf
    logp[..., st["end"]] = torch.where(ended, 0.0, logp[..., st["end"]])
    score = (logp + st["scores"].double().unsqueeze(-1)).flatten(1)
    best = score.topk(min(case["n_out"], score.shape[1]), -1).values
    return {"scores": best, "beams": None, "tokens": None}
