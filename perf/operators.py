"""Cases, plain forms and exact forms of the decoder-serving operators: causal prompt attention over packed
sequences, the paged key-value cache (reserve, append, fork, free, compact) and the attention of one new token
over it.

The cache of every case is laid out as the library's: pool [layers, pages, 2, kv heads, page rows, head size]
(index 0 of the third axis K, 1 V), table int32 [slots, max_pages], lens int32 [slots], refs int32 [pages].  A page
is free where refs is 0, and pages are taken lowest number first.
"""
import math
import random

import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a short question of one user, heads as in BERT-base: latency of the smallest prompt
        dict(name="prompt_short", op="prompt", dtype="fp16", B=1, lo=97, hi=97, nh=12, nkv=12, d=64),
        # a batch of prompts with the BERT-large lengths and heads of this repository's benchmark
        dict(name="prompt_batch", op="prompt", dtype="bf16", B=64, lo=32, hi=384, nh=16, nkv=16, d=64),
        # documents of two users, grouped heads: the largest prompt
        dict(name="prompt_long", op="prompt", dtype="bf16", B=2, lo=7001, hi=8192, nh=32, nkv=8, d=128),
        # one user's chat: latency of the smallest step
        dict(name="decode_one", op="decode", dtype="bf16", B=1, lo=1043, hi=1043, nh=32, nkv=8, d=128, ps=16),
        # a full serving batch of mixed lengths
        dict(name="decode_batch", op="decode", dtype="bf16", B=128, lo=200, hi=8192, nh=32, nkv=8, d=128, ps=16),
        # one sequence over a long context, every head its own keys
        dict(name="decode_long", op="decode", dtype="fp16", B=1, lo=131000, hi=131000, nh=16, nkv=16, d=64, ps=64),
        # the keys and values of one new token per sequence
        dict(name="append_step", op="append", dtype="bf16", B=96, lo=10, hi=500, nkv=8, d=128, ps=16),
        # prompts take over the slots of finished sequences: free, reserve, append
        dict(name="admit_prompts", op="admit", dtype="bf16", B=24, lo=100, hi=2048, nkv=8, d=128, ps=16),
        # beams of one step: the losing beams are freed, the winning ones forked
        dict(name="fork_beams", op="fork", dtype="bf16", layers=24, src=4, fan=2, lo=50, hi=900, nkv=8, d=128, ps=16),
        # samples of several prompts, heads of BERT-large, larger pages
        dict(name="fork_samples", op="fork", dtype="fp16", layers=12, src=16, fan=8, lo=100, hi=1500, nkv=16, d=64, ps=64),
        # a small cache after a few sequences have left
        dict(name="compact_small", op="compact", dtype="fp16", layers=4, pages=300, live=0.7, B=9, nkv=4, d=64, ps=16),
        # a cache of many layers before a part of its memory is given back
        dict(name="compact_large", op="compact", dtype="bf16", layers=24, pages=1000, live=0.6, B=40, nkv=8, d=128, ps=16),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "decode", "decode", "append", "admit", "fork", "compact"])
    d = rng.choice([64, 128])
    nkv = rng.choice([1, 2, 3, 4, 8, 12, 16])
    c = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), nkv=nkv, d=d)
    if op in ("prompt", "decode"):
        c["nh"] = nkv * rng.choice([g for g in (1, 2, 3, 4, 5, 8, 12, 16) if g * nkv <= 48])
    if op != "prompt":
        c["ps"] = rng.choice([16, 16, 32, 48, 64, 128])
    if op == "prompt":
        c["hi"] = _spread(rng, 1, 6000)
        room = 2 * 32 * 6000 * 6000 // (c["nh"] * c["hi"] * c["hi"])    # scores of the plain form
        c["B"] = _spread(rng, 1, max(1, min(96, room, 120000 // c["hi"])))
        c["lo"] = rng.randint(1, c["hi"])
    elif op == "decode":
        c["hi"] = _spread(rng, 1, 100000)
        room = 128 * 4200 * 8 * 128 // (c["hi"] * nkv * d)
        c["B"] = _spread(rng, 1, max(1, min(300, room)))
        c["lo"] = rng.randint(1, c["hi"])
    elif op in ("append", "admit"):
        c["hi"] = _spread(rng, 3, 3000)
        c["lo"] = rng.randint(1, c["hi"])
        c["B"] = _spread(rng, 1, max(1, min(200, 24 * 2048 * 8 * 128 // (max(c["hi"], c["ps"]) * nkv * d))))
    elif op == "fork":
        c["hi"] = _spread(rng, 2, 2000)
        c["lo"] = rng.randint(1, c["hi"])
        c["src"], c["fan"] = _spread(rng, 1, 16), _spread(rng, 1, 8)
        rows = c["src"] * (max(c["hi"], c["ps"]) + 2 * c["fan"] * c["ps"])
        c["layers"] = max(1, min(rng.randint(1, 32), 500_000_000 // (rows * 2 * nkv * d)))
    else:
        c["live"] = round(rng.uniform(0.05, 0.95), 3)
        c["pages"], c["B"] = _spread(rng, 3, 4000), _spread(rng, 1, 60)
        c["layers"] = max(1, min(rng.randint(1, 32), 500_000_000 // (c["pages"] * 2 * nkv * d * c["ps"])))
    return c


def _rng(c):
    """The sizes inside a case (lengths, which pages are in use) go by the case alone."""
    return random.Random(" ".join("%s=%s" % kv for kv in sorted(c.items()) if kv[0] != "name"))


def _lengths(c, n, rng):
    got = [rng.randint(c["lo"], c["hi"]) for _ in range(n)]
    got[0] = c["hi"]
    return got


def _up(n, m):
    return -(-n // m)


# ---------------------------------------------------------------- inputs
def _fill(c, pages, layers, g):
    shape = (layers, pages, 2, c["nkv"], c["ps"], c["d"])
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(_DT[c["dtype"]]) if math.prod(shape) < 1 << 28 else \
        torch.randn(shape, generator=g, device="cuda", dtype=_DT[c["dtype"]])


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(c, lens, pages, slots, max_pages, layers, g, rng):
    """A cache whose first len(lens) slots hold sequences on pages scattered over the pool."""
    order = list(range(pages))
    rng.shuffle(order)
    table = [[-1] * max_pages for _ in range(slots)]
    refs = [0] * pages
    for s, n in enumerate(lens):
        for j in range(_up(n, c["ps"])):
            table[s][j] = order.pop()
            refs[table[s][j]] = 1
    return dict(pool=_fill(c, pages, layers, g), table=_ints(table), lens=_ints(lens + [0] * (slots - len(lens))), refs=_ints(refs))


def prepare(case, seed):
    c, rng = case, _rng(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, op, nkv, d = _DT[c["dtype"]], c["op"], c["nkv"], c["d"]

    def rows(n, heads, scale=1.0):
        return (scale * torch.randn((n, heads * d), generator=g, device="cuda")).to(dt)

    st = dict(case=c)
    if op == "prompt":
        lens = _lengths(c, c["B"], rng)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        # the QKV projection's output: rows of Q | K | V; queries of twice the keys' size, so that weights are uneven
        st["qkv"] = torch.cat([rows(cu[-1], c["nh"], 2.0), rows(cu[-1], 2 * nkv)], 1)
        st["cu"] = _ints(cu)
        st["max_len"] = max(lens)
    elif op == "decode":
        lens = _lengths(c, c["B"], rng)
        need = sum(_up(n, c["ps"]) for n in lens)
        st |= _cache(c, lens, need + need // 8 + 1, c["B"] + 3, _up(max(lens), c["ps"]) + 1, 1, g, rng)
        slots = list(range(c["B"]))
        rng.shuffle(slots)
        st["slots"] = _ints(slots)
        st["max_len"] = max(lens)
        st["qkv"] = torch.cat([rows(c["B"], c["nh"], 2.0), rows(c["B"], 2 * nkv)], 1)
    elif op in ("append", "admit"):
        lens = _lengths(c, c["B"], rng)
        new = [1] * c["B"] if op == "append" else _lengths(c, c["B"], rng)
        need = sum(max(_up(a, c["ps"]), _up(b, c["ps"])) for a, b in zip(lens, new))
        st |= _cache(c, lens, need + sum(_up(b, c["ps"]) for b in new), c["B"] + 1, _up(c["hi"], c["ps"]) + 1, 1, g, rng)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        st["cu"], st["new"] = _ints(cu), _ints(new)
        slots = list(range(c["B"]))
        rng.shuffle(slots)
        st["slots"] = _ints(slots)
        st["kv"] = rows(cu[-1], 2 * nkv)
    elif op == "fork":
        n = c["src"] * c["fan"]
        lens = _lengths(c, c["src"] + n, rng)
        mp = _up(c["hi"], c["ps"])
        lens[c["src"]:] = [min(m, 2 * c["ps"]) for m in lens[c["src"]:]]
        st |= _cache(c, lens, sum(_up(m, c["ps"]) for m in lens) + n, len(lens) + 1, mp, c["layers"], g, rng)
        st["src"] = _ints([i // c["fan"] for i in range(n)])
        st["dst"] = _ints([c["src"] + i for i in range(n)])
    else:
        lens = _compact_lengths(c, rng)
        st |= _cache(c, lens, c["pages"], len(lens) + 1, max(_up(m, c["ps"]) for m in lens) + 1, c["layers"], g, rng)
        st["table_out"], st["refs_out"] = torch.empty_like(st["table"]), torch.empty_like(st["refs"])
    if own:
        import remove_padding_prefix_gb300 as rpp
        if op != "prompt":
            st["cache"] = rpp.KvCache.from_tensors(st["pool"], st["table"], st["lens"], st["refs"])
            st["err"] = rpp.new_error_word()
        if op == "decode":
            st["ws"] = rpp.attention_decode_workspace(st["cache"], c["B"], c["nh"])
    return st


def _compact_lengths(c, rng):
    left, lens = max(1, min(c["pages"] - 1, int(c["pages"] * c["live"]))), []
    for i in range(c["B"]):
        n = min(left, max(1, int(rng.uniform(0.5, 1.5) * c["pages"] * c["live"] / c["B"])))
        if i == c["B"] - 1:
            n = left
        if n:
            lens.append((n - 1) * c["ps"] + rng.randint(1, c["ps"]))
            left -= n
    return lens


# ---------------------------------------------------------------- plain forms
def _softmax_rows(s):
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _plain_prompt(st):
    c, cu, qkv = st["case"], st["cu"].long(), st["qkv"]
    nh, nkv, d, L, B = c["nh"], c["nkv"], c["d"], st["max_len"], c["B"]
    at = torch.arange(L, device="cuda")
    length = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + at).clamp(max=qkv.shape[0] - 1)                      # [B, L]
    x = qkv[row].float()                                                        # padded rows
    q = x[..., :nh * d].view(B, L, nkv, nh // nkv, d).permute(0, 2, 3, 1, 4)    # [B, nkv, g, L, d]
    k = x[..., nh * d:(nh + nkv) * d].view(B, L, nkv, 1, d).permute(0, 2, 3, 4, 1)
    v = x[..., (nh + nkv) * d:].view(B, L, nkv, 1, d).permute(0, 2, 3, 1, 4)
    seen = (at[None, :] <= at[:, None])[None] & (at[None, None, :] < length[:, None, None])
    s = torch.matmul(q, k).mul_(d ** -0.5)
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(s, v) / s.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(B * L, nh * d)
    t = torch.arange(qkv.shape[0], device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    return o[b * L + t - cu[b]].to(qkv.dtype)


def _plain_decode(st):
    c = st["case"]
    nh, nkv, d, ps, B = c["nh"], c["nkv"], c["d"], c["ps"], c["B"]
    n = _up(st["max_len"], ps)
    slots = st["slots"].long()
    page = st["table"][slots, :n].long().clamp(min=0)                           # [B, n]
    kv = st["pool"][0][page].permute(2, 0, 3, 1, 4, 5).reshape(2, B, nkv, n * ps, d).float()
    q = st["qkv"][:, :nh * d].float().view(B, nkv, nh // nkv, d)
    s = torch.matmul(q, kv[0].transpose(-1, -2)) * d ** -0.5                     # [B, nkv, g, n ps]
    past = torch.arange(n * ps, device="cuda") >= st["lens"].long()[slots][:, None]
    s = s.masked_fill(past[:, None, None], float("-inf"))
    return torch.matmul(_softmax_rows(s), kv[1]).reshape(B, nh * d).to(st["qkv"].dtype)


def _plain_free(st, slots):
    ps, table = st["case"]["ps"], st["table"]
    pages = table[slots]
    used = torch.arange(table.shape[1], device="cuda") < ((st["lens"][slots].long() + ps - 1) // ps)[:, None]
    st["refs"].index_add_(0, pages.clamp(min=0).long().flatten(), -used.flatten().int())
    table[slots] = -1
    st["lens"][slots] = 0


def _plain_pages(st, need):
    """For sequence i and j < need[i]: the next free page, lowest number first; -1 elsewhere."""
    rank = (st["refs"] == 0).long().cumsum(0)
    j = torch.arange(st["table"].shape[1], device="cuda")
    k = (need.cumsum(0) - need)[:, None] + j + 1
    page = torch.searchsorted(rank, k.clamp(max=rank.numel()))
    wanted = j < need[:, None]
    return torch.where(wanted, page, torch.full_like(page, -1)), wanted


def _plain_append(st, k, v, slots, cu):
    c, t = st["case"], torch.arange(k.shape[0], device="cuda")
    cu = cu.long()
    i = torch.searchsorted(cu[1:], t, right=True)
    pos = st["lens"].long()[slots[i]] - cu[i + 1] + t
    page = st["table"][slots[i], pos // c["ps"]].long()
    pool = st["pool"][0]
    pool[page, 0, :, pos % c["ps"]] = k.view(-1, c["nkv"], c["d"])
    pool[page, 1, :, pos % c["ps"]] = v.view(-1, c["nkv"], c["d"])


def _state(st):
    return {"pool": st["pool"], "table": st["table"], "lens": st["lens"], "refs": st["refs"]}


def _plain_cache(st):
    c, op = st["case"], st["case"]["op"]
    ps = c["ps"]
    if op in ("append", "admit"):
        slots, w = st["slots"].long(), c["nkv"] * c["d"]
        if op == "admit":
            _plain_free(st, slots)
            page, wanted = _plain_pages(st, (st["new"].long() + ps - 1) // ps)
            st["table"][slots] = page.int()
            st["refs"].index_add_(0, page.clamp(min=0).flatten(), wanted.flatten().int())
            st["lens"][slots] = st["new"]
        _plain_append(st, st["kv"][:, :w], st["kv"][:, w:], slots, st["cu"])
        return _state(st) if op == "admit" else st["pool"]
    if op == "fork":
        src, dst, pool = st["src"].long(), st["dst"].long(), st["pool"]
        _plain_free(st, dst)
        length = st["lens"][src].long()
        rows, full = length % ps, length // ps
        page, _ = _plain_pages(st, (rows > 0).long())
        j = torch.arange(st["table"].shape[1], device="cuda")
        old = st["table"][src].long()
        last = (j == full[:, None]) & (rows > 0)[:, None]
        fresh = torch.where(last, page[:, :1], torch.where(j < full[:, None], old, torch.full_like(old, -1)))
        st["table"][dst] = fresh.int()
        st["refs"].index_add_(0, fresh.clamp(min=0).flatten(), (fresh >= 0).flatten().int())
        st["lens"][dst] = length.int()
        a, b = old[last], fresh[last]
        keep = (torch.arange(ps, device="cuda") < rows[rows > 0][:, None])[None, :, None, None, :, None]
        pool[:, b] = torch.where(keep, pool[:, a], pool[:, b])
        return _state(st)
    refs, pool = st["refs"], st["pool"]
    at, alive = torch.arange(refs.numel(), device="cuda"), refs > 0
    live = alive.sum()
    a, b = (alive & (at >= live)).nonzero().flatten(), (~alive & (at < live)).nonzero().flatten()
    new = torch.where(alive, at, torch.full_like(at, -1))
    new[a] = b
    pool[:, b] = pool[:, a]
    used = torch.arange(st["table"].shape[1], device="cuda") < ((st["lens"].long() + ps - 1) // ps)[:, None]
    table = torch.where(used, new[st["table"].clamp(min=0).long()], -1).int()
    out = torch.zeros_like(refs)
    out[new[alive]] = refs[alive]
    return {"pool": pool, "table": table, "refs": out, "live": live.int()}


# ---------------------------------------------------------------- one pass
def _own(st):
    import remove_padding_prefix_gb300 as rpp
    c, op = st["case"], st["case"]["op"]
    if op == "prompt":
        w, n = c["nh"] * c["d"], c["nkv"] * c["d"]
        qkv = st["qkv"]
        return rpp.attention_causal_varlen(qkv[:, :w], qkv[:, w:w + n], qkv[:, w + n:], st["cu"], c["B"], st["max_len"],
                                           c["nh"], c["nkv"], c["d"])
    cache, err = st["cache"], st["err"]
    if op == "decode":
        return rpp.attention_decode(cache, 0, st["qkv"][:, :c["nh"] * c["d"]], st["slots"], workspace=st["ws"], err=err)
    if op in ("append", "admit"):
        w = c["nkv"] * c["d"]
        if op == "admit":
            rpp.kv_free(cache, st["slots"], err=err)
            rpp.kv_reserve(cache, st["slots"], st["new"], err=err)
        rpp.kv_append(cache, 0, st["kv"][:, :w], st["kv"][:, w:], st["slots"], None if op == "append" else st["cu"], err=err)
        return _state(st) if op == "admit" else st["pool"]
    if op == "fork":
        rpp.kv_free(cache, st["dst"], err=err)
        rpp.kv_fork(cache, st["src"], st["dst"], err=err)
        return _state(st)
    table, refs, live = rpp.kv_compact(cache, table_out=st["table_out"], refs_out=st["refs_out"], err=err)
    return {"pool": st["pool"], "table": table, "refs": refs, "live": live[0]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_prompt(state) if op == "prompt" else _plain_decode(state) if op == "decode" else _plain_cache(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c, rng, e = case, _rng(case), 2
    op, nkv, d = c["op"], c["nkv"], c["d"]
    if op == "prompt":
        lens = _lengths(c, c["B"], rng)
        return {"bytes": sum(lens) * (2 * c["nh"] + 2 * nkv) * d * e + 4 * (c["B"] + 1),
                "flops": 4 * d * c["nh"] * sum(n * (n + 1) // 2 for n in lens)}
    if op == "decode":
        lens = _lengths(c, c["B"], rng)
        return {"bytes": sum(lens) * 2 * nkv * d * e + 2 * c["B"] * c["nh"] * d * e + 4 * sum(_up(n, c["ps"]) + 2 for n in lens),
                "flops": 4 * d * c["nh"] * sum(lens)}
    row = 2 * nkv * d * e                                                       # K and V of one token in one layer
    if op == "append":
        return {"bytes": c["B"] * (2 * row + 12), "flops": 0}
    if op == "admit":
        lens = _lengths(c, c["B"], rng)
        new = _lengths(c, c["B"], rng)
        pages = sum(_up(a, c["ps"]) + _up(b, c["ps"]) for a, b in zip(lens, new))
        return {"bytes": sum(new) * 2 * row + 16 * pages, "flops": 0}
    if op == "fork":
        n = c["src"] * c["fan"]
        lens = _lengths(c, c["src"] + n, rng)
        at = [lens[i // c["fan"]] for i in range(n)]
        return {"bytes": c["layers"] * row * 2 * sum(m % c["ps"] for m in at) + 16 * sum(_up(m, c["ps"]) for m in at), "flops": 0}
    lens = _compact_lengths(c, rng)
    order = list(range(c["pages"]))
    rng.shuffle(order)
    live = sum(_up(n, c["ps"]) for n in lens)
    moved = sum(p >= live for p in order[c["pages"] - live:])
    return {"bytes": 2 * moved * c["layers"] * row * c["ps"] + 8 * c["pages"] + 8 * live, "flops": 0}


# ---------------------------------------------------------------- in 64 bits, from the definition
def exact(case, seed):
    c = case
    if c["op"] not in ("prompt", "decode"):
        return None    # these move values and count pages
    st = prepare(case, seed)
    nh, nkv, d = c["nh"], c["nkv"], c["d"]
    per = nh // nkv
    if c["op"] == "prompt":
        qkv, cu = st["qkv"], st["cu"].tolist()
        out = torch.zeros((qkv.shape[0], nh * d), dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            x = qkv[cu[b]:cu[b + 1]].double()
            hide = torch.ones((x.shape[0], x.shape[0]), dtype=torch.bool, device="cuda").triu(1)
            for h in range(nh):
                kh = nh + h // per
                z = x[:, h * d:(h + 1) * d] @ x[:, kh * d:(kh + 1) * d].T / math.sqrt(d)
                w = torch.softmax(z.masked_fill_(hide, -math.inf), dim=1)
                out[cu[b]:cu[b + 1], h * d:(h + 1) * d] = w @ x[:, (kh + nkv) * d:(kh + nkv + 1) * d]
        return out
    out = torch.zeros((c["B"], nh * d), dtype=torch.float64, device="cuda")
    lens, table = st["lens"].tolist(), st["table"].tolist()
    for i, s in enumerate(st["slots"].tolist()):
        n = lens[s]
        pages = torch.tensor(table[s][:_up(n, c["ps"])], device="cuda")
        for h in range(nkv):
            k, v = (st["pool"][0, pages, x, h].reshape(-1, d)[:n].double() for x in (0, 1))
            q = st["qkv"][i, h * per * d:(h + 1) * per * d].double().view(per, d)
            out[i, h * per * d:(h + 1) * per * d] = (torch.softmax(q @ k.T / math.sqrt(d), dim=1) @ v).flatten()
    return out
