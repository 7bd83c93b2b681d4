"""Cases, plain forms and exact forms of the key-value cache held in 8 bits: quantising rows as they are written, reading
them back, and the attention of one new token over them.

The cache of every case: pool [layers, pages, 2, kv heads, page rows, head size] of int8 or e4m3 codes (index 0 of the
third axis K, 1 V), scales uint8 [layers, pages, 2, kv heads, page rows / block], table int32 [slots, max_pages], lens
int32 [slots], refs int32 [pages].  A code stands for code * 2^(b - 127), b its block's scale byte; 255 makes the block NaN.
The scale of rows with largest magnitude a is the smallest power of two at which a is no more than half a step past the
largest code; a block that has rows already keeps its scale or takes the larger one, and then its codes are rounded again.
"""
import math
import random

import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
_CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_TOP = {"int8": 127.0, "e4m3": 448.0}       # the largest code
_PAST = {"int8": 127.5, "e4m3": 464.0}      # and half a step past it
_LOG = {"int8": 6, "e4m3": 8}               # its exponent


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the keys and values of one new token per sequence, written and their blocks fetched: the smallest write
        dict(name="write_step", op="write", code="e4m3", dtype="bf16", B=96, lo=10, hi=500, one=True, nkv=8, d=128, ps=16, block=16),
        # one user's new token, heads of BERT-base: latency
        dict(name="write_one", op="write", code="int8", dtype="fp16", B=1, lo=777, hi=777, one=True, nkv=12, d=64, ps=16, block=16),
        # prompts of a batch taken in and swapped out
        dict(name="write_prompts", op="write", code="e4m3", dtype="bf16", B=24, lo=100, hi=2048, one=False, nkv=8, d=128, ps=16, block=16),
        # chunks of long prompts, a scale of each token's own, heads of BERT-large
        dict(name="write_chunks", op="write", code="int8", dtype="fp16", B=40, lo=33, hi=1500, one=False, nkv=16, d=64, ps=64, block=1),
        # one short prefix on its way to another sequence: latency
        dict(name="read_one", op="read", code="e4m3", dtype="bf16", B=1, lo=97, hi=97, nkv=8, d=128, ps=16, block=16),
        # prefixes of a full batch for a prompt attention that takes packed rows
        dict(name="read_prefixes", op="read", code="e4m3", dtype="bf16", B=32, lo=300, hi=4096, nkv=8, d=128, ps=16, block=16),
        # the same of a cache with one scale for a page of 64 tokens
        dict(name="read_pages", op="read", code="int8", dtype="fp16", B=16, lo=1, hi=2500, nkv=16, d=64, ps=64, block=64),
        # one user's chat: latency of the smallest step
        dict(name="attend_one", op="attend", code="e4m3", dtype="bf16", B=1, lo=1043, hi=1043, nh=32, nkv=8, d=128, ps=16, block=16),
        # a full serving batch of mixed lengths
        dict(name="attend_batch", op="attend", code="e4m3", dtype="bf16", B=128, lo=200, hi=8192, nh=32, nkv=8, d=128, ps=16, block=16),
        # the same in int8 with a scale of each token's own
        dict(name="attend_tokens", op="attend", code="int8", dtype="bf16", B=64, lo=200, hi=8192, nh=32, nkv=8, d=128, ps=16, block=1),
        # one sequence over a long context, every head its own keys
        dict(name="attend_long", op="attend", code="int8", dtype="fp16", B=1, lo=131000, hi=131000, nh=16, nkv=16, d=64, ps=64, block=64),
        # many queries of one key head
        dict(name="attend_shared", op="attend", code="e4m3", dtype="fp16", B=48, lo=1000, hi=6000, nh=32, nkv=2, d=128, ps=32, block=32),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["write", "write", "read", "attend", "attend", "attend"])
    d, nkv = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8, 12, 16])
    ps = rng.choice([16, 16, 32, 48, 64, 128])
    c = dict(op=op, code=rng.choice(["e4m3", "int8"]), dtype=rng.choice(["fp16", "bf16"]), nkv=nkv, d=d, ps=ps,
             block=rng.choice([b for b in (1, 2, 4, 8, 16, 16, 16, 32, 64, 128) if ps % b == 0]))
    if op == "attend":
        c["nh"] = nkv * rng.choice([g for g in (1, 2, 3, 4, 5, 8, 12, 16) if g * nkv <= 48])
        c["hi"] = _spread(rng, 1, 100000)
        room = 128 * 4200 * 8 * 128 // (c["hi"] * nkv * d)
        c["B"] = _spread(rng, 1, max(1, min(300, room)))
    else:
        c["hi"] = _spread(rng, 3, 3000)
        c["B"] = _spread(rng, 1, max(1, min(200, 24 * 2048 * 8 * 128 // (max(c["hi"], ps) * nkv * d))))
        if op == "write":
            c["one"] = rng.random() < 0.4
    c["lo"] = rng.randint(1, c["hi"])
    return c


def _rng(c):
    """The sizes inside a case (lengths, which pages are in use) go by the case alone."""
    return random.Random(" ".join("%s=%s" % kv for kv in sorted(c.items()) if kv[0] != "name"))


def _lengths(c, rng):
    got = [rng.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    got[0] = c["hi"]
    return got


def _new_rows(c, lens, rng):
    """How many of each sequence's tokens a write brings: one, the whole prompt, or what comes after a chunk."""
    return [1 if c["one"] else n if rng.random() < 0.5 else rng.randint(1, n) for n in lens]


def _read_from(c, lens, rng):
    """Where a read begins: mostly at the first token."""
    return [0 if rng.random() < 0.7 else rng.randint(0, n - 1) for n in lens]


def _up(n, m):
    return -(-n // m)


def _sums(v):
    got = [0]
    for n in v:
        got.append(got[-1] + n)
    return got


# ---------------------------------------------------------------- inputs
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(c, lens, pages, max_pages, g, rng):
    """A cache of sequences on pages scattered over the pool, codes spread as those of blocks whose largest is near the top."""
    order = list(range(pages))
    rng.shuffle(order)
    table = [[-1] * max_pages for _ in range(len(lens) + 1)]
    refs = [0] * pages
    for s, n in enumerate(lens):
        for j in range(_up(n, c["ps"])):
            table[s][j] = order.pop()
            refs[table[s][j]] = 1
    top = _TOP[c["code"]]
    x = torch.randn((1, pages, 2, c["nkv"], c["ps"], c["d"]), generator=g, device="cuda").mul_(top / 3.5).clamp_(-top, top)
    pool = (x.round_() if c["code"] == "int8" else x).to(_CODE[c["code"]])
    base = 127 + 1 - _LOG[c["code"]]
    scales = torch.randint(base - 1, base + 2, (1, pages, 2, c["nkv"], c["ps"] // c["block"]), generator=g, device="cuda", dtype=torch.uint8)
    return dict(pool=pool, scales=scales, table=_ints(table), lens=_ints(lens + [0]), refs=_ints(refs))


def prepare(case, seed):
    c, rng = case, _rng(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, op, nkv, d = _DT[c["dtype"]], c["op"], c["nkv"], c["d"]
    lens = _lengths(c, rng)
    need = sum(_up(n, c["ps"]) for n in lens)
    st = dict(case=c) | _cache(c, lens, need + need // 8 + 1, _up(max(lens), c["ps"]) + 1, g, rng)
    slots = list(range(c["B"]))
    rng.shuffle(slots)
    st["slots"] = _ints(slots)
    st["max_len"] = max(lens)
    at = [lens[s] for s in slots]
    if op == "write":
        new = _new_rows(c, at, rng)
        st["cu"] = _ints(_sums(new))
        # a few channels of the keys carry most of their size
        loud = torch.exp(0.7 * torch.randn((2 * nkv * d,), generator=g, device="cuda"))
        st["kv"] = (loud * torch.randn((sum(new), 2 * nkv * d), generator=g, device="cuda")).to(dt)
        # what is fetched: every token of the blocks that took one
        first = [(n - m) // c["block"] * c["block"] for n, m in zip(at, new)]
    elif op == "read":
        first = _read_from(c, at, rng)
    else:
        # queries of twice the keys' size, so that weights are uneven
        st["qkv"] = torch.cat([(z * torch.randn((c["B"], h * d), generator=g, device="cuda")).to(dt) for z, h in ((2.0, c["nh"]), (1.0, 2 * nkv))], 1)
    if op != "attend":
        count = [n - a for n, a in zip(at, first)]
        st["starts"], st["read_cu"], st["rows"] = _ints(first), _ints(_sums(count)), sum(count)
    if own:
        import remove_padding_prefix_gb300 as rpp
        st["cache"] = rpp.KvCache8.from_tensors(st["pool"], st["scales"], st["table"], st["lens"], st["refs"])
        st["err"] = rpp.new_error_word()
        if op == "attend":
            st["ws"] = rpp.attention_decode_workspace(st["cache"], c["B"], c["nh"])
    return st


# ---------------------------------------------------------------- plain forms
def _scale(b):
    """2^(b - 127) of scale bytes in 32 bits, NaN of 255."""
    b = b.int()
    f = torch.where(b > 0, b << 23, torch.full_like(b, 1 << 22)).view(torch.float32)
    return torch.where(b == 255, torch.full_like(f, float("nan")), f)


def _encode(c, x):
    """Codes of values that are already in steps."""
    top = _TOP[c["code"]]
    return (x.round() if c["code"] == "int8" else x).clamp(-top, top).to(_CODE[c["code"]])


def _places(st, cu, starts, rows):
    """Sequence, page and row in the page of each packed row."""
    c, t = st["case"], torch.arange(rows, device="cuda")
    cu = cu.long()
    i = torch.searchsorted(cu[1:], t, right=True)
    pos = starts.long()[i] + t - cu[i]
    return i, pos, st["table"].long()[st["slots"].long()[i], pos // c["ps"]], pos % c["ps"]


def _bytes(t):
    return t.view(torch.uint8)


def _plain_read(st):
    c = st["case"]
    _, _, page, row = _places(st, st["read_cu"], st["starts"], st["rows"])
    code = _bytes(st["pool"])[0, page, :, :, row].view(_CODE[c["code"]]).float()        # [rows, 2, nkv, d]
    x = code * _scale(st["scales"][0, page, :, :, row // c["block"]])[..., None]
    top = torch.finfo(_DT[c["dtype"]]).max
    return x.clamp(-top, top).to(_DT[c["dtype"]]).flatten(2).unbind(1)


def _plain_write(st):
    c = st["case"]
    nkv, d, block, ps = c["nkv"], c["d"], c["block"], c["ps"]
    rows = st["kv"].shape[0]
    cu = st["cu"].long()
    begin = st["lens"].long()[st["slots"].long()] - (cu[1:] - cu[:-1])                  # each sequence's first new token
    i, pos, page, row = _places(st, st["cu"], begin, rows)
    x = st["kv"].float().view(rows, 2, nkv, d)
    per = ps // block
    at = page * per + row // block                                                      # the block, over all pages
    pages = st["refs"].numel()
    most = torch.zeros((pages * per, 2, nkv), device="cuda")
    most.scatter_reduce_(0, at[:, None, None].expand(rows, 2, nkv), x.abs().amax(-1), "amax")
    used, first = torch.unique(at, return_inverse=True)
    a = most[used]
    b = ((a.view(torch.int32) >> 23) - _LOG[c["code"]]).clamp(min=0)
    b = b + (a > _PAST[c["code"]] * _scale(b)).int()
    b = torch.where(torch.isfinite(a), b, torch.full_like(b, 255))
    # blocks that have tokens already: the first new token of a sequence is not the block's first
    scales = st["scales"][0].permute(0, 3, 1, 2).reshape(pages * per, 2, nkv)           # [block, 2, nkv]
    old_rows = torch.zeros(used.numel(), dtype=torch.long, device="cuda")
    new_seq = torch.where(pos == begin[i], row % block, torch.zeros_like(row))
    old_rows.scatter_reduce_(0, first, new_seq, "amax")
    had = scales[used].int()
    b = torch.where((old_rows > 0)[:, None, None], torch.maximum(b, had), b)
    # their codes, rounded to the new step
    pg, lo = used // per, used % per * block
    r = torch.arange(block, device="cuda")
    codes = _bytes(st["pool"])[0]
    was = codes[pg[:, None], :, :, lo[:, None] + r]                                     # [used, block, 2, nkv, d]
    value = was.view(_CODE[c["code"]]).float() * _scale((127 + had - b).clamp(0, 127))[:, None, :, :, None]
    again = ((r < old_rows[:, None])[:, :, None, None] & (b > had)[:, None] & (b < 255)[:, None])[..., None]
    now = torch.where(again, _bytes(_encode(c, value)), was)
    codes[pg[:, None], :, :, lo[:, None] + r] = now
    # the new rows
    step = _scale(254 - b.clamp(max=254))[first]
    new = _encode(c, torch.where((b < 255)[first][..., None], x * step[..., None], torch.zeros_like(x)))
    codes[page, :, :, row] = _bytes(new)
    st["scales"][0, pg, :, :, used % per] = b.to(torch.uint8)
    return _plain_read(st) + (st["scales"],)


def _plain_attend(st):
    c = st["case"]
    nh, nkv, d, ps, B = c["nh"], c["nkv"], c["d"], c["ps"], c["B"]
    n = _up(st["max_len"], ps)
    slots = st["slots"].long()
    page = st["table"][slots, :n].long().clamp(min=0)                                   # [B, n]
    kv = _bytes(st["pool"])[0][page].view(_CODE[c["code"]]).float()                     # [B, n, 2, nkv, ps, d]
    kv.mul_(_scale(st["scales"][0][page]).repeat_interleave(c["block"], -1)[..., None])
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, B, nkv, n * ps, d)
    q = st["qkv"][:, :nh * d].float().view(B, nkv, nh // nkv, d)
    s = torch.matmul(q, kv[0].transpose(-1, -2)) * d ** -0.5                             # [B, nkv, g, n ps]
    past = torch.arange(n * ps, device="cuda") >= st["lens"].long()[slots][:, None]
    s = s.masked_fill(past[:, None, None], float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return torch.matmul(p / p.sum(-1, keepdim=True), kv[1]).reshape(B, nh * d).to(st["qkv"].dtype)


# ---------------------------------------------------------------- one pass
def _own(st):
    import remove_padding_prefix_gb300 as rpp
    c, cache, err = st["case"], st["cache"], st["err"]
    if c["op"] == "attend":
        return rpp.attention_decode(cache, 0, st["qkv"][:, :c["nh"] * c["d"]], st["slots"], workspace=st["ws"], err=err)
    w = c["nkv"] * c["d"]
    if c["op"] == "write":
        rpp.kv_append(cache, 0, st["kv"][:, :w], st["kv"][:, w:], st["slots"], st["cu"], err=err)
    out = rpp.kv_read(cache, 0, st["slots"], st["read_cu"], starts=st["starts"], rows=st["rows"], dtype=c["dtype"], err=err)
    return out + (st["scales"],) if c["op"] == "write" else out


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_write(state) if op == "write" else _plain_read(state) if op == "read" else _plain_attend(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c, rng = case, _rng(case)
    lens = _lengths(c, rng)
    need = sum(_up(n, c["ps"]) for n in lens)
    order = list(range(need + need // 8 + 1))
    rng.shuffle(order)
    slots = list(range(c["B"]))
    rng.shuffle(slots)
    at = [lens[s] for s in slots]
    w, block = 2 * c["nkv"] * c["d"], c["block"]
    if c["op"] == "attend":
        row = w + 2 * c["nkv"] / block
        return {"bytes": sum(lens) * row + 2 * c["B"] * c["nh"] * c["d"] * 2 + 4 * sum(_up(n, c["ps"]) + 2 for n in lens),
                "flops": 4 * c["d"] * c["nh"] * sum(lens)}
    if c["op"] == "read":
        count = [n - a for n, a in zip(at, _read_from(c, at, rng))]
        return {"bytes": sum(count) * (3 * w + 2 * c["nkv"] / block) + 16 * c["B"], "flops": sum(count) * w}
    new = _new_rows(c, at, rng)
    count = [n - (n - m) // block * block for n, m in zip(at, new)]
    # rows in, codes out; the fetched blocks' codes in (those just written are read from near by), rows out
    return {"bytes": sum(new) * 3 * w + sum(count) * 3 * w + 2 * sum(count) * 2 * c["nkv"] / block + 16 * c["B"],
            "flops": 4 * sum(new) * w + sum(count) * w}


# ---------------------------------------------------------------- in 64 bits, from the definition
def _pow2(e):
    """2^e of whole numbers, to the bit (a library's power need not be)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    nkv, d, ps, block = c["nkv"], c["d"], c["ps"], c["block"]
    kind = _CODE[c["code"]]
    pool, scales, table = st["pool"][0], st["scales"][0], st["table"].tolist()
    lens, slots = st["lens"].tolist(), st["slots"].tolist()

    def held(s):
        """All values of a sequence: [2, nkv, rows of its pages, d]."""
        pages = torch.tensor(table[s][:_up(lens[s], ps)], device="cuda")
        x = pool.view(torch.uint8)[pages].view(kind).double()                           # [pages, 2, nkv, ps, d]
        x = x.unflatten(3, (-1, block)) * _pow2(scales[pages].double() - 127.0)[..., None, None]
        return x.permute(1, 2, 0, 3, 4, 5).reshape(2, nkv, -1, d)

    if c["op"] == "attend":
        nh, per = c["nh"], c["nh"] // nkv
        out = torch.zeros((c["B"], nh * d), dtype=torch.float64, device="cuda")
        for i, s in enumerate(slots):
            k, v = held(s)[:, :, :lens[s]]
            q = st["qkv"][i, :nh * d].double().view(nkv, per, d)
            out[i] = (torch.softmax(q @ k.transpose(1, 2) / math.sqrt(d), dim=-1) @ v).flatten()
        return out
    begin, cut = st["starts"].tolist(), st["read_cu"].tolist()
    out = torch.zeros((2, st["rows"], nkv * d), dtype=torch.float64, device="cuda")
    for i, s in enumerate(slots):
        x = held(s)
        if c["op"] == "write":
            a, e = st["cu"][i:i + 2].tolist()
            n0 = lens[s] - (e - a)
            rows = st["kv"][a:e].double().view(e - a, 2, nkv, d).permute(1, 2, 0, 3)
            lead = n0 % block                                                           # tokens that the first block has
            z = torch.cat([x[:, :, n0 - lead:n0], rows], 2)
            z = torch.nn.functional.pad(z, (0, 0, 0, -z.shape[2] % block)).unflatten(2, (-1, block))
            # the smallest power of two whose largest code, and half a step, reach the largest magnitude
            fresh = z.clone()
            fresh[:, :, 0, :lead] = 0.0
            top = fresh.abs().amax((-1, -2))                                            # [2, nkv, blocks]
            e2 = torch.ceil(torch.log2(top / _PAST[c["code"]]))
            for nudge in (-1.0, 1.0):                                                   # log2 may round over a whole number
                better = (top <= _PAST[c["code"]] * _pow2(e2 - 1)) if nudge < 0 else (top > _PAST[c["code"]] * _pow2(e2))
                e2 = torch.where(better, e2 + nudge, e2)
            if lead:
                page = table[s][n0 // ps]
                had = scales[page, :, :, n0 % ps // block].double() - 127.0
                e2[:, :, 0] = torch.maximum(e2[:, :, 0], had)
            unit = _pow2(e2)[..., None, None]
            y = z / unit
            if c["code"] == "int8":
                y = y.round()
            else:
                step = _pow2(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1].double() - 4.0)
                y = (y / step).round() * step
            x = (y.clamp(-_TOP[c["code"]], _TOP[c["code"]]) * unit).flatten(2, 3)
            x = x[:, :, begin[i] - (n0 - lead):][:, :, :cut[i + 1] - cut[i]]
        else:
            x = x[:, :, begin[i]:lens[s]]
        out[:, cut[i]:cut[i + 1]] = x.permute(0, 2, 1, 3).reshape(2, -1, nkv * d)
    if c["op"] == "write":
        return out[0], out[1], None
    return out[0], out[1]
