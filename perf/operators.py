"""Timed cases of the paged 8-bit key/value cache: writing new tokens and
reading them back, and attention over the cache.

The cache is a pool of pages of `block` tokens.  A page holds, for every
key/value head, the e4m3 codes of its tokens' keys ([token][channel]) and
values ([token/16][channel][16 tokens]), and one power-of-two scale each for
the keys and the values; a code stands for code * scale.  A batch is a table
of pages per sequence, each sequence's length with its new tokens, and the
offsets of its new rows in the batch: row j of a sequence with m new rows and
length n sits at position n - m + j.

With `own` false, run() computes everything with elementary torch operations
in 32 bits; with `own` true it calls the framework's operators.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
EXP_MIN, EXP_MAX = -64, 120  # exponents a page's scale may have


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def _case(name, op, **kw):
    c = dict(op=op, heads=32, kv_heads=8, dim=128, block=16, seqs=0, old_min=0, old_max=0, new_min=1, new_max=1,
             singles=0, idle=0, causal=True, window=0, lens=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # four requests early in their answers: the latency of one small call
        _case("attend_decode_4", "attend", singles=4, old_min=5, old_max=300, lens=11),
        # a decode step of 32 requests, mid-sized contexts
        _case("attend_decode_32", "attend", singles=32, old_min=100, old_max=4000, lens=12),
        # a full decode batch, some of its slots idle
        _case("attend_decode_256", "attend", singles=250, idle=6, old_min=1000, old_max=8100, lens=13),
        # two requests far into long documents: few rows, a long axis
        _case("attend_decode_long", "attend", singles=2, old_min=90000, old_max=131000, block=64, lens=14),
        # sliding window, seven query heads to a key head, 64 channels
        _case("attend_window_64", "attend", heads=28, kv_heads=4, dim=64, block=32, singles=96, old_min=50,
              old_max=6000, window=1024, lens=15),
        # 4 prompts of 96 tokens that join 128 decoding requests (512 rows)
        _case("attend_mixed_512", "attend", seqs=4, new_min=96, new_max=96, singles=128, old_min=0, old_max=2000,
              lens=16),
        # prompts of 8 requests, nothing cached before
        _case("attend_prompt_8", "attend", seqs=8, new_min=64, new_max=1024, lens=17),
        # one chunk of a long prompt over what is already cached
        _case("attend_chunk_2048", "attend", seqs=1, new_min=2048, new_max=2048, old_min=16301, old_max=16301,
              block=64, lens=18),
        # one new token of each of 256 requests, then the pages it changed
        _case("write_decode_256", "write", singles=256, old_min=0, old_max=2000, lens=19),
        # 8 prompts written (page boundaries anywhere), then read back
        _case("write_prompt_8", "write", seqs=8, new_min=64, new_max=1024, old_min=0, old_max=90, lens=20),
        # a long cached prefix read back, for another replica or another cache
        _case("read_prefix_32768", "read", seqs=1, new_min=32768, new_max=32768, block=64, lens=21),
        # many short histories read back, 80 channels
        _case("read_batch_64", "read", heads=16, kv_heads=4, dim=80, seqs=64, new_min=1, new_max=1500, lens=22),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "write", "read"])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 16])
    c = _case(None, op, heads=heads, kv_heads=kv_heads, dim=rng.choice([64, 80, 96, 128, 128, 128, 192, 256]),
              block=rng.choice([16, 16, 32, 64, 128]), lens=rng.randrange(1 << 30))
    budget = 2048 * 8 * 128 // (kv_heads * c["dim"]) * 128  # tokens that the largest listed case's bytes stand for
    if op == "attend":
        kind = rng.choice(["decode", "long", "mixed", "prompt", "chunk", "window", "few"])
        if kind in ("decode", "window"):
            c["singles"] = _log_int(rng, 1, 256)
            c["old_max"] = max(1, min(_log_int(rng, 16, 16384), budget // c["singles"]))
            c["old_min"] = rng.randrange(c["old_max"])
            c["idle"] = rng.choice([0, 0, 3])
            if kind == "window":
                c["window"] = _log_int(rng, 1, 4096)
        elif kind == "long":
            c["singles"] = rng.randint(1, 4)
            c["old_max"] = _log_int(rng, 20000, 130000) // c["singles"]
            c["old_min"] = c["old_max"] // 2
        elif kind == "mixed":
            c["seqs"], c["singles"] = rng.randint(1, 6), _log_int(rng, 1, 128)
            c["new_min"], c["new_max"] = rng.randint(2, 40), rng.randint(40, 160)
            c["old_max"] = _log_int(rng, 16, 2000)
        elif kind == "prompt":
            c["seqs"] = rng.randint(1, 8)
            c["new_min"], c["new_max"] = _log_int(rng, 1, 64), _log_int(rng, 64, 1024)
            c["causal"] = rng.random() < 0.8
            if c["causal"] and rng.random() < 0.3:
                c["window"] = _log_int(rng, 1, 1024)
        elif kind == "chunk":
            c["seqs"] = 1
            c["new_min"] = c["new_max"] = _log_int(rng, 100, 1500)
            c["old_min"] = c["old_max"] = _log_int(rng, 500, 12000)
        else:  # a few tokens at a time, as when drafted tokens are checked
            c["seqs"] = _log_int(rng, 1, 64)
            c["new_min"], c["new_max"] = rng.randint(1, 3), rng.randint(3, 9)
            c["old_max"] = _log_int(rng, 16, 4000)
    elif op == "write":
        if rng.random() < 0.5:
            c["singles"] = _log_int(rng, 1, 256)
        else:
            c["seqs"] = _log_int(rng, 1, 16)
            c["new_min"], c["new_max"] = _log_int(rng, 1, 50), _log_int(rng, 50, 1000)
        c["old_max"] = _log_int(rng, 1, 1000)
    else:
        c["seqs"] = _log_int(rng, 1, 64)
        c["new_max"] = min(_log_int(rng, 8, 30000), 30000 * 8 * 128 // (kv_heads * c["dim"]) // c["seqs"])
        c["new_min"] = _log_int(rng, 1, c["new_max"])
    return c


def _lengths(case):
    """(new tokens, length with them) of every sequence, by the case alone."""
    rng = random.Random(case["lens"])
    new = [rng.randint(case["new_min"], case["new_max"]) for _ in range(case["seqs"])]
    new += [1] * case["singles"]
    total = [m + rng.randint(case["old_min"], case["old_max"]) for m in new]
    for _ in range(case["idle"]):
        at = rng.randrange(len(new) + 1)
        new.insert(at, 0)
        total.insert(at, 0)
    return new, total


def _pages(total, block):
    return [-(-n // block) for n in total]


def work(case):
    new, total = _lengths(case)
    H, D, Hq, B = case["kv_heads"], case["dim"], case["heads"], case["block"]
    rows = sum(new)
    if case["op"] == "read":  # codes and scales in, bf16 out
        return {"bytes": rows * H * D * 2 * (1 + 2) + sum(_pages(total, B)) * H * 2 * 4, "flops": 0}
    if case["op"] == "write":
        back = sum(_read_back(m, n, B) for m, n in zip(new, total))
        touched = sum(-(-n // B) - (n - m) // B for m, n in zip(new, total) if m)
        return {"bytes": rows * H * D * 2 * (2 + 1) + back * H * D * 2 * 2 + touched * H * 2 * 4, "flops": 0}
    keys = pairs = pages = 0
    w = case["window"] or 1 << 40
    for m, n in zip(new, total):
        if not m:
            continue
        first = max(0, n - m - w + 1) if case["causal"] else 0
        keys += n - first
        pages += -(-n // B) - first // B
        pairs += sum(min(w, n - m + j + 1) for j in range(m)) if case["causal"] else m * n
    return {"bytes": keys * H * D * 2 + pages * (H * 2 * 4 + 4) + rows * Hq * D * 2 * 2, "flops": 4 * Hq * D * pairs}


def _read_back(m, n, block):
    """Rows of a sequence that a write may have changed: its new ones and
    those before them in the first page that it touched."""
    return m + (n - m) % block if m else 0


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _fill(g, n_blocks, H, B, D):
    """Cached content: channels of unequal size (a few large ones), tokens of
    unequal size, as e4m3 codes with a scale for each page and head."""
    size = torch.exp(0.4 * torch.randn(1, H, 1, D, device=DEV, generator=g))
    size = size * torch.where(torch.rand(1, H, 1, D, device=DEV, generator=g) < 0.03, 6.0, 1.0)
    x = torch.randn(n_blocks, H, B, D, device=DEV, generator=g)
    x *= size
    x *= torch.exp2(0.7 * torch.randn(n_blocks, H, B, 1, device=DEV, generator=g))
    scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 440)))
    x /= scale[:, :, None, None]
    return x.to(torch.float8_e4m3fn).view(torch.uint8), scale, size


def _batch(new, total, table, rows=None):
    row_off = [0]
    for m in new:
        row_off.append(row_off[-1] + m)
    return dict(table=table, kv_len=_ints(total), row_off=_ints(row_off), n_rows=row_off[-1],
                max_new=max(new), n_seq=len(new))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    H, D, Hq, B = case["kv_heads"], case["dim"], case["heads"], case["block"]
    new, total = _lengths(case)
    pages = _pages(total, B)
    n_blocks = sum(pages) + 7
    # pages lie anywhere in the pool, as after some time of serving
    free = torch.randperm(n_blocks, device=DEV, generator=g).to(torch.int32)
    width = max(max(pages), 1)
    count = _ints(pages)
    start = torch.cumsum(count, 0) - count
    j = torch.arange(width, device=DEV)
    at = (start[:, None] + j[None, :]).clamp(max=n_blocks - 1)
    table = torch.where(j[None, :] < count[:, None], free[at], -1).to(torch.int32)
    k, k_scale, k_size = _fill(g, n_blocks, H, B, D)
    v, v_scale, v_size = _fill(g, n_blocks, H, B, D)
    v = v.view(n_blocks, H, B // 16, 16, D).transpose(3, 4).contiguous()
    st = dict(case=case, k=k[None], v=v[None], k_scale=k_scale[None], v_scale=v_scale[None])
    st["batch"] = b = _batch(new, total, table)
    if case["op"] != "read":
        # one row of a projection's output: queries, then keys, then values
        qkv = torch.randn(b["n_rows"], Hq + 2 * H, D, device=DEV, generator=g)
        qkv[:, Hq:Hq + H] *= k_size[:, :, 0]
        qkv[:, Hq + H:] *= v_size[:, :, 0]
        qkv[:, Hq:] *= torch.exp2(0.7 * torch.randn(b["n_rows"], 2 * H, 1, device=DEV, generator=g))
        qkv = qkv.to(torch.bfloat16)
        st["q"], st["new_k"], st["new_v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    if case["op"] == "write":
        st["back"] = _batch([_read_back(m, n, B) for m, n in zip(new, total)], total, table)
    if own:
        import lora_serving_mlora_amd as M
        st["cache"] = M.KVCache(1, n_blocks, H, D, B, storage=(st["k"], st["v"], st["k_scale"], st["v_scale"]))
        for name in ("batch", "back"):
            if name in st:
                c = st[name]
                st["own_" + name] = M.KVBatch(c["table"], c["kv_len"], c["row_off"], c["n_rows"], max_new=c["max_new"])
        if case["op"] == "attend":
            st["work"] = M.new_kv_work(st["cache"], st["own_batch"], Hq)
    return st


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        import lora_serving_mlora_amd as M
        if op == "attend":
            return M.kv_attention(st["cache"], 0, st["q"], st["own_batch"], causal=st["case"]["causal"],
                                  window=st["case"]["window"], work=st["work"])
        if op == "read":
            k, v = M.kv_read(st["cache"], 0, st["own_batch"])
            return {"k": k, "v": v}
        M.kv_append(st["cache"], 0, st["new_k"], st["new_v"], st["own_batch"])
        k, v = M.kv_read(st["cache"], 0, st["own_back"])
        return {"k": k, "v": v, "k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    if op == "attend":
        return _attend(st)
    if op == "read":
        k, v = _read(st, st["batch"])
        return {"k": k, "v": v}
    _write(st)
    k, v = _read(st, st["back"])
    return {"k": k, "v": v, "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _rows(b):
    """Sequence, index in it and position of every new row."""
    off = b["row_off"].long()
    new = off[1:] - off[:-1]
    seq = torch.repeat_interleave(torch.arange(b["n_seq"], device=DEV), new, output_size=b["n_rows"])
    j = torch.arange(b["n_rows"], device=DEV) - off[seq]
    return seq, j, b["kv_len"].long()[seq] - new[seq] + j


def _values(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * scale


def _read(st, b):
    B = st["case"]["block"]
    seq, _, pos = _rows(b)
    page = b["table"][seq, pos // B].long()
    t = pos % B
    k = _values(st["k"][0][page, :, t], st["k_scale"][0][page][:, :, None])
    v = _values(st["v"][0][page, :, t // 16, :, t % 16], st["v_scale"][0][page][:, :, None])
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _attend(st):
    c, b = st["case"], st["batch"]
    S, H, D, B, Hq = b["n_seq"], c["kv_heads"], c["dim"], c["block"], c["heads"]
    G, M = Hq // H, b["max_new"]
    L = b["table"].shape[1] * B
    page = b["table"].long().clamp(min=0)
    k = _values(st["k"][0][page], st["k_scale"][0][page][..., None, None])  # [S][pages][H][B][D]
    k = k.permute(0, 2, 4, 1, 3).reshape(S, H, D, L)
    v = _values(st["v"][0][page], st["v_scale"][0][page][..., None, None, None])  # [S][pages][H][B/16][D][16]
    v = v.permute(0, 2, 1, 3, 5, 4).reshape(S, H, L, D)
    seq, j, _ = _rows(b)
    q = torch.zeros(S, M, Hq, D, device=DEV)
    q[seq, j] = st["q"].float()
    q = q.view(S, M, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * M, D)
    s = torch.matmul(q, k).view(S, H, G, M, L) * (1.0 / math.sqrt(D))
    off = b["row_off"].long()
    n = b["kv_len"].long()[:, None, None]
    pos = n - (off[1:] - off[:-1])[:, None, None] + torch.arange(M, device=DEV)[None, :, None]
    key = torch.arange(L, device=DEV)[None, None, :]
    seen = key < n
    if c["causal"]:
        seen = seen & (key <= pos)
        if c["window"]:
            seen = seen & (key > pos - c["window"])
    else:
        seen = seen.expand(S, M, L)
    s = torch.where(seen[:, None, None], s, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, H, G * M, L), v).view(S, H, G, M, D)
    o = o / torch.where(total == 0, 1.0, total)
    return o.permute(0, 3, 1, 2, 4).reshape(S, M, Hq, D)[seq, j].to(torch.bfloat16)


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, within the scale's range."""
    m, e = torch.frexp(amax / E4M3_MAX)  # amax / 448 = m * 2^e, 0.5 <= m < 1
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(amax == 0, EXP_MIN, e).clamp(EXP_MIN, EXP_MAX)


def _write(st):
    c, b = st["case"], st["batch"]
    H, D, B = c["kv_heads"], c["dim"], c["block"]
    seq, _, pos = _rows(b)
    page = b["table"][seq, pos // B].long()
    t = pos % B
    # a page whose first token is among the new ones starts anew
    off = b["row_off"].long()
    first = b["kv_len"].long() - (off[1:] - off[:-1])
    tail = b["table"].long().gather(1, (first // B)[:, None])[:, 0]  # first page of each sequence that is written
    kept = first % B > 0  # it holds older tokens
    for codes, scale, x, is_v in ((st["k"][0], st["k_scale"][0], st["new_k"], False),
                                  (st["v"][0], st["v_scale"][0], st["new_v"], True)):
        x = x.float()
        amax = torch.zeros_like(scale)
        amax.scatter_reduce_(0, page[:, None].expand(-1, H), x.abs().amax(-1), "amax")
        need = _exponent(amax)
        old = (torch.frexp(scale)[1] - 1).clamp(EXP_MIN, EXP_MAX)
        floor = torch.zeros(scale.shape[0], 1, dtype=torch.bool, device=DEV)
        floor[tail] = kept[:, None]
        e = torch.where(floor, torch.maximum(old, need), need)
        wrote = torch.zeros(scale.shape[0], 1, dtype=torch.bool, device=DEV)
        wrote[page] = True
        scale_new = torch.where(wrote, torch.ldexp(torch.ones_like(scale), e), scale)
        # older tokens of a page whose scale grew are rounded to the new one
        was = codes[tail]
        shape = (-1, H, 1, 1, 1) if is_v else (-1, H, 1, 1)
        again = (_values(was, scale[tail].view(shape)) / scale_new[tail].view(shape)).to(torch.float8_e4m3fn)
        grown = (kept[:, None] & (e[tail] > old[tail])).view(shape)
        at = torch.arange(B, device=DEV)
        older = at[None, :] < (first % B)[:, None]
        older = older.view(-1, 1, B // 16, 1, 16) if is_v else older.view(-1, 1, B, 1)
        codes[tail] = torch.where(grown & older, again.view(torch.uint8), was)
        code = (x / scale_new[page][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        if is_v:
            codes[page, :, t // 16, :, t % 16] = code
        else:
            codes[page, :, t] = code
        scale.copy_(scale_new)


# ----------------------------------------------------------------------------
# 64-bit results, from the definition, a sequence (or a page) at a time
# ----------------------------------------------------------------------------

def _code_values():
    out = []
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            x = math.nan
        elif e:
            x = (8 + m) * 2.0 ** (e - 10)
        else:
            x = m * 2.0 ** -9
        out.append(-x if s else x)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _history(st, lut, i, n):
    """Keys and values [tokens][H][D] of sequence i's first n tokens."""
    c, B = st["case"], st["case"]["block"]
    ids = st["batch"]["table"][i, :-(-n // B)].long()
    k = lut[st["k"][0][ids].long()] * st["k_scale"][0][ids].double()[:, :, None, None]
    v = lut[st["v"][0][ids].long()] * st["v_scale"][0][ids].double()[:, :, None, None, None]
    k = k.transpose(1, 2).reshape(-1, c["kv_heads"], c["dim"])[:n]
    v = v.permute(0, 2, 4, 1, 3).reshape(-1, c["kv_heads"], c["dim"])[:n]
    return k, v


def _to_e4m3(x):
    """The nearest e4m3 value, ties to even."""
    a = x.abs().clamp(min=2.0 ** -60)
    step = torch.exp2((torch.floor(torch.log2(a))).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    new, total = _lengths(case)
    H, D, Hq, B = case["kv_heads"], case["dim"], case["heads"], case["block"]
    lut = _code_values()
    if case["op"] == "attend":
        out, at = [], 0
        for i, (m, n) in enumerate(zip(new, total)):
            if not m:
                continue
            k, v = _history(st, lut, i, n)
            q = st["q"][at:at + m].double()
            at += m
            key = torch.arange(n, device=DEV)[None, :]
            pos = n - m + torch.arange(m, device=DEV)[:, None]
            hidden = torch.zeros(m, n, dtype=torch.bool, device=DEV)
            if case["causal"]:
                hidden = key > pos
                if case["window"]:
                    hidden = hidden | (key <= pos - case["window"])
            o = torch.empty(m, Hq, D, dtype=torch.float64, device=DEV)
            for h in range(Hq):
                s = q[:, h] @ k[:, h * H // Hq].T / math.sqrt(D)
                s.masked_fill_(hidden, -math.inf)
                o[:, h] = torch.softmax(s, -1) @ v[:, h * H // Hq]
            out.append(o)
        return torch.cat(out)
    if case["op"] == "write":
        scales = {"k": st["k_scale"].double().clone(), "v": st["v_scale"].double().clone()}
        x = {"k": st["new_k"].double(), "v": st["new_v"].double()}
    got = {"k": [], "v": []}
    at = 0
    for i, (m, n) in enumerate(zip(new, total)):
        if not m:
            continue
        k, v = _history(st, lut, i, n)
        if case["op"] == "read":
            got["k"].append(k[n - m:])
            got["v"].append(v[n - m:])
            continue
        a = n - m
        for name, whole in (("k", k), ("v", v)):
            whole[a:] = x[name][at:at + m]
            for p in range(a // B, -(-n // B)):
                page = int(st["batch"]["table"][i, p])
                lo, hi = max(p * B, a), min((p + 1) * B, n)
                top = whole[lo:hi].abs().amax((0, 2)) / E4M3_MAX
                e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp(min=1e-300))), EXP_MIN).clamp(EXP_MIN, EXP_MAX)
                if p * B < a:
                    was = torch.log2(scales[name][0, page])
                    e = torch.maximum(e, was)
                s = torch.exp2(e)
                whole[p * B:hi] = _to_e4m3(whole[p * B:hi] / s[None, :, None]) * s[None, :, None]
                scales[name][0, page] = s
            got[name].append(whole[a - a % B:])
        at += m
    sides = {name: torch.cat(got[name]) for name in got}
    if case["op"] == "write":
        sides.update(k_scale=scales["k"], v_scale=scales["v"])
    return sides
