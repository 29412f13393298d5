"""Timed cases of the steps around the key/value cache of a served layer:
products with 4-bit weights (with each row's adapter on top), the norms of
queries and keys with the rotation of their positions, and the sampling of
the next tokens.

4-bit weights: a code is sign, 2 exponent bits, 1 fraction bit (0, 0.5, 1,
1.5, 2, 3, 4, 6), two codes a byte, the lower half first; 32 channels of a row
share the scale 2^(b - 127), b one byte.  The quantiser takes the least scale
whose 6 covers the 32 weights, and the nearest code, ties to the even one.

Sampling: w = exp((logit - largest) / temperature); tokens stand in the order
of falling logits, the lower index first; of these the first top_k are kept,
of those the shortest part from the top that holds top_p of their mass, of
those the ones with w >= min_p; the token is the first at which the running
mass exceeds u times the mass kept.

With `own` false, run() computes everything with elementary torch operations;
with `own` true it calls the framework's operators.
"""
import math
import random

import torch

own = False

DEV = "cuda"
GROUP = 32
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def _product(name, rows, din, dout, ranks="", bare=0.25):
    """ranks: "16,8,64" = three adapters of these ranks; bare: share of rows without one."""
    c = dict(op="product", rows=rows, din=din, dout=dout, ranks=ranks, bare=bare)
    return dict(c, name=name) if name else c


def _quantise(name, din, dout):
    c = dict(op="quantise", din=din, dout=dout)
    return dict(c, name=name) if name else c


def _rotate(name, **kw):
    c = dict(op="rotate", heads=32, kv_heads=8, dim=128, rot=128, base=10000.0, interleaved=False, norm=True,
             seqs=0, new_min=1, new_max=1, singles=0, idle=0, old_min=0, old_max=0, lens=1)
    c.update(kw)
    return dict(c, name=name) if name else c


def _sample(name, rows, vocab, **kw):
    c = dict(op="sample", rows=rows, vocab=vocab, type="bf16", greedy=0.0, top_k=0, top_p=True, min_p=False, spread=2.2)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request, one projection: the latency of one product
        _product("product_1", 1, 4096, 4096),
        # a decode step, 32 requests on three adapters
        _product("product_decode_32", 32, 4096, 4096, "16,16,16"),
        # a down projection, odd row count, adapters of mixed ranks
        _product("product_down_61", 61, 11008, 4096, "8,16,64"),
        # prompts of eight requests
        _product("product_prompt_4096", 4096, 4096, 11008, "8,16,64,8,16,64", 0.0),
        # a weight taken in (as after an adapter was merged into it) and read back
        _quantise("quantise_4096", 4096, 4096),
        _quantise("quantise_11008", 4096, 11008),
        # four requests early in their answers: the latency of one small call
        _rotate("rotate_decode_4", singles=4, old_min=5, old_max=300, lens=11),
        # a full decode batch far into long contexts, some of its slots idle
        _rotate("rotate_decode_256", singles=250, idle=6, old_min=1000, old_max=120000, lens=12),
        # prompts of 8 requests, a part of the 80 channels rotated, no norm
        _rotate("rotate_prompt_80", heads=32, kv_heads=32, dim=80, rot=32, norm=False, seqs=8, new_min=64,
                new_max=1024, lens=13),
        # one request, small vocabulary
        _sample("sample_1", 1, 32000, top_k=50),
        # a decode batch of mixed requests, odd vocabulary
        _sample("sample_32", 32, 50001, type="fp32", top_k=200, min_p=True, greedy=0.2),
        # a full decode batch, large vocabulary, most requests with top-p alone
        _sample("sample_256", 256, 131072),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "product", "quantise", "rotate", "rotate", "sample", "sample", "sample"])
    if op == "product":
        rows = rng.choice([_log_int(rng, 1, 16), _log_int(rng, 1, 64), _log_int(rng, 65, 1024),
                           _log_int(rng, 1025, 4096)])
        din = GROUP * _log_int(rng, 8, 512)
        dout = min(_log_int(rng, 64, 16384), 4096 * 4096 * 11008 // (din * rows))
        if rng.random() < 0.7:
            dout = max(8, dout // 8 * 8)
        ranks = ",".join(str(rng.choice([1, 4, 8, 16, 32, 64])) for _ in range(rng.choice([0, 1, 3, 6])))
        return _product(None, rows, din, dout, ranks, rng.choice([0.0, 0.25, 0.9]))
    if op == "quantise":
        return _quantise(None, GROUP * _log_int(rng, 8, 344), _log_int(rng, 1, 4096))
    if op == "rotate":
        kv_heads = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
        c = _rotate(None, heads=kv_heads * rng.choice([1, 2, 4, 5, 7, 8]), kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2 // 8 * 8, 16]), base=rng.choice([10000.0, 500000.0, 1e6]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.7, lens=rng.randrange(1 << 30))
        if rng.random() < 0.5:
            c["singles"], c["idle"] = _log_int(rng, 1, 256), rng.choice([0, 0, 3])
            c["old_max"] = _log_int(rng, 16, 130000)
            c["old_min"] = rng.randrange(c["old_max"])
        else:
            c["seqs"], c["singles"] = rng.randint(1, 8), rng.choice([0, 0, 20])
            c["new_min"], c["new_max"] = _log_int(rng, 1, 64), _log_int(rng, 64, 1024)
            c["old_max"] = _log_int(rng, 1, 4000)
        return c
    rows = _log_int(rng, 1, 256)
    vocab = min(_log_int(rng, 1000, 200000), 256 * 131072 // rows // 2)
    return _sample(None, rows, vocab, type=rng.choice(["bf16", "fp32"]), greedy=rng.choice([0.0, 0.2]),
                   top_k=rng.choice([0, 0, _log_int(rng, 1, 1000)]), top_p=rng.random() < 0.7,
                   min_p=rng.random() < 0.4, spread=rng.choice([0.5, 1.5, 2.2, 4.0]))


def _lengths(case):
    """(new tokens, length with them) of every sequence, by the case alone."""
    rng = random.Random(case["lens"])
    new = [rng.randint(case["new_min"], case["new_max"]) for _ in range(case["seqs"])] + [1] * case["singles"]
    total = [m + rng.randint(case["old_min"], case["old_max"]) for m in new]
    for _ in range(case["idle"]):
        at = rng.randrange(len(new) + 1)
        new.insert(at, 0)
        total.insert(at, 0)
    return new, total


def _ranks(case):
    return [int(r) for r in case["ranks"].split(",") if r]


def work(case):
    op = case["op"]
    if op == "product":
        n, din, dout, ranks = case["rows"], case["din"], case["dout"], _ranks(case)
        served = n * (1 - case["bare"]) if ranks else 0
        mean = sum(ranks) / len(ranks) if ranks else 0
        return {"bytes": din * dout // 2 + din * dout // GROUP + 2 * n * (din + dout) + 2 * sum(ranks) * (din + dout),
                "flops": int(2 * n * din * dout + 2 * served * mean * (din + dout))}
    if op == "quantise":  # bf16 in, codes and scales out, these in, bf16 out
        w = case["din"] * case["dout"]
        return {"bytes": 4 * w + 2 * (w // 2 + w // GROUP), "flops": 0}
    if op == "rotate":
        x = sum(_lengths(case)[0]) * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 4 * x, "flops": 7 * x}
    size = 2 if case["type"] == "bf16" else 4
    return {"bytes": case["rows"] * (case["vocab"] * size + 24), "flops": 20 * case["rows"] * case["vocab"]}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _weights(g, rows, cols):
    """A weight matrix: columns of unequal size, a few of them large."""
    size = torch.exp(0.5 * torch.randn(1, cols, device=DEV, generator=g)) / math.sqrt(cols)
    w = torch.randn(rows, cols, device=DEV, generator=g)
    w *= size
    return w


def _prepare_product(case, g):
    n, din, dout, ranks = case["rows"], case["din"], case["dout"], _ranks(case)
    codes = torch.randint(0, 256, (dout, din // 2), device=DEV, generator=g, dtype=torch.uint8)
    scales = torch.randint(118, 122, (dout, din // GROUP), device=DEV, generator=g, dtype=torch.uint8)
    x = torch.randn(n, din, device=DEV, generator=g)
    x *= torch.exp(0.5 * torch.randn(1, din, device=DEV, generator=g))
    st = dict(codes=codes, scales=scales, x=x.to(torch.bfloat16))
    if ranks:
        ids = torch.randint(0, len(ranks), (n,), device=DEV, generator=g, dtype=torch.int32)
        st["ids"] = torch.where(torch.rand(n, device=DEV, generator=g) < case["bare"], -1, ids).to(torch.int32)
        st["scale"] = [0.25 * (2 + i % 5) for i in range(len(ranks))]
        st["down"] = [_weights(g, r, din).to(torch.bfloat16) for r in ranks]
        st["up"] = [_weights(g, dout, r).to(torch.bfloat16) for r in ranks]
    if own:
        import lora_serving_mlora_amd as M
        st["w4"] = M.Q4Weight(codes, scales)
        pool = None
        if ranks:
            pool = st["pool"] = M.Pool(din, dout, 1, len(ranks), max(ranks), sum(ranks))
            for a, r in enumerate(ranks):
                pool.load(a, r, st["scale"][a], st["down"][a][None], st["up"][a][None])
            st["seg"] = M.build_segments(pool, st["ids"])
        st["work"] = M.new_q4_work(st["w4"], n, pool=pool)
    elif ranks:  # the plain form's adapters side by side
        st["owner"] = _ints([a for a, r in enumerate(ranks) for _ in range(r)])
        st["down"], st["up"] = torch.cat(st["down"]), torch.cat(st["up"], 1)
        st["factor"] = torch.tensor(st["scale"], device=DEV)[st["owner"].long()]
    return st


def _prepare_rotate(case, g):
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    new, total = _lengths(case)
    off = [0]
    for m in new:
        off.append(off[-1] + m)
    n = off[-1]
    # one row of a projection's output: queries, then keys, then values
    qkv = torch.randn(n, H + 2 * Hk, D, device=DEV, generator=g)
    qkv *= torch.exp(0.4 * torch.randn(1, H + 2 * Hk, D, device=DEV, generator=g))
    qkv = qkv.to(torch.bfloat16)
    st = dict(q=qkv[:, :H], k=qkv[:, H:H + Hk], kv_len=_ints(total), row_off=_ints(off), n=n, n_seq=len(new))
    freq = torch.arange(case["rot"] // 2, dtype=torch.float64, device=DEV)
    st["freqs"] = case["base"] ** (-2.0 * freq / case["rot"])
    if case["norm"]:
        st["qw"] = (1 + 0.3 * torch.randn(D, device=DEV, generator=g)).to(torch.bfloat16)
        st["kw"] = (1 + 0.3 * torch.randn(D, device=DEV, generator=g)).to(torch.bfloat16)
    if own:
        import lora_serving_mlora_amd as M
        table = torch.zeros(len(new), max(1, -(-max(total) // 16)), dtype=torch.int32, device=DEV)
        st["batch"] = M.KVBatch(table, st["kv_len"], st["row_off"], n, max_new=max(new))
        st["rotary"] = M.Rotary(case["rot"], base=case["base"], interleaved=case["interleaved"])
    return st


def _prepare_sample(case, g):
    n, V = case["rows"], case["vocab"]
    # a wide bulk and some tokens that stand out, as a model's logits do
    logits = case["spread"] * torch.randn(n, V, device=DEV, generator=g)
    likely = torch.randint(0, V, (n, 60), device=DEV, generator=g)
    lift = 4 * case["spread"] - 2.5 * torch.log(torch.rand(n, 60, device=DEV, generator=g) + 1e-3)
    logits.scatter_(1, likely, lift)
    st = dict(logits=logits.to(torch.bfloat16 if case["type"] == "bf16" else torch.float32))
    draw_ = lambda: torch.rand(n, device=DEV, generator=g)
    st["u"] = draw_()
    st["temperature"] = torch.where(draw_() < case["greedy"], 0.0, 0.4 + draw_())
    st["top_k"] = st["top_p"] = st["min_p"] = None
    if case["top_k"]:  # some requests without a limit
        k = torch.randint(1, 2 * case["top_k"], (n,), device=DEV, generator=g, dtype=torch.int32)
        st["top_k"] = torch.where(draw_() < 0.2, 0, k).to(torch.int32)
    if case["top_p"]:
        st["top_p"] = torch.where(draw_() < 0.2, 1.0, 0.5 + 0.49 * draw_())
    if case["min_p"]:
        st["min_p"] = torch.where(draw_() < 0.3, 0.0, 0.1 * draw_())
    if own:
        import lora_serving_mlora_amd as M
        st["work"] = M.new_sample_work(n, V)
    return st


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["op"] == "product":
        st = _prepare_product(case, g)
    elif case["op"] == "quantise":
        st = dict(w=_weights(g, case["dout"], case["din"]).to(torch.bfloat16))
    elif case["op"] == "rotate":
        st = _prepare_rotate(case, g)
    else:
        st = _prepare_sample(case, g)
    st["case"] = case
    return st


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        import lora_serving_mlora_amd as M
        if op == "product":
            if "pool" in st:
                return M.q4_apply(st["pool"], 0, st["x"], st["w4"], st["seg"], work=st["work"])
            return M.q4_gemm(st["x"], st["w4"], work=st["work"])
        if op == "quantise":
            w4 = M.q4_quantize(st["w"])
            return {"values": M.q4_dequantize(w4), "scales": w4.scales}
        if op == "rotate":
            q, k = M.qk_norm_rotary(st["q"], st["k"], st["batch"], st["rotary"], q_weight=st.get("qw"),
                                    k_weight=st.get("kw"), eps=1e-6)
            return {"q": q, "k": k}
        return M.sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                        min_p=st["min_p"], work=st["work"])
    return {"product": _run_product, "quantise": _run_quantise, "rotate": _run_rotate, "sample": _run_sample}[op](st)


def _unpack(codes, scales):
    """float [rows][channels] of codes and scale bytes."""
    half = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    values = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=DEV)[half.long()]
    return values * torch.exp2(scales.float() - 127).repeat_interleave(GROUP, -1)


def _run_product(st):
    x = st["x"].float()
    y = torch.matmul(x, _unpack(st["codes"], st["scales"]).t())
    if "ids" in st:
        t = torch.matmul(x, st["down"].float().t())
        t = torch.where(st["ids"][:, None] == st["owner"][None, :], t * st["factor"], 0.0)
        y = y + torch.matmul(t, st["up"].float().t())
    return y.to(torch.bfloat16)


def _run_quantise(st):
    w = st["w"].float()
    rows, cols = w.shape
    w = w.view(rows, cols // GROUP, GROUP)
    amax = w.abs().amax(-1)
    m, x = torch.frexp(amax)  # amax = m 2^x, 6 = 0.75 2^3
    e = torch.where(amax == 0, -125, torch.where(m <= 0.75, x - 3, x - 2)).clamp(-125, 125)
    scale = torch.ldexp(torch.ones_like(amax), e)
    a = (w / scale[..., None]).abs()
    # spacing of the codes: 0.5 below 2, 1 below 4, then 2
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.clamp(torch.round(a / step) * step, max=6.0)
    values = torch.copysign(a, w) * scale[..., None]
    return {"values": values.view(rows, cols).to(torch.bfloat16), "scales": (e + 127).to(torch.uint8)}


def _run_rotate(st):
    c = st["case"]
    off = st["row_off"].long()
    new = off[1:] - off[:-1]
    seq = torch.repeat_interleave(torch.arange(st["n_seq"], device=DEV), new, output_size=st["n"])
    pos = st["kv_len"].long()[seq] - new[seq] + torch.arange(st["n"], device=DEV) - off[seq]
    angle = pos.double()[:, None] * st["freqs"][None, :]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        r = c["rot"]
        part = x[..., :r]
        if c["interleaved"]:
            a, b = part[..., 0::2], part[..., 1::2]
            part = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = part[..., :r // 2], part[..., r // 2:]
            part = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((part, x[..., r:]), -1).to(torch.bfloat16)

    return {"q": one(st["q"], st.get("qw")), "k": one(st["k"], st.get("kw"))}


def _run_sample(st):
    n, V = st["logits"].shape
    x = st["logits"].double()
    top = x.amax(-1, keepdim=True)
    t = st["temperature"].double()[:, None]
    w = torch.where(t > 0, torch.exp((x - top) / torch.where(t > 0, t, 1.0)), (x == top).double())
    w = torch.where(x == top, 1.0, w)
    order = torch.sort(x, dim=-1, descending=True, stable=True)[1]
    w = w.gather(-1, order)
    cum = torch.cumsum(w, -1)
    kept = torch.full((n, 1), V, device=DEV)
    if st["top_k"] is not None:
        k = st["top_k"].long()[:, None]
        kept = torch.where(k > 0, k.clamp(max=V), kept)
    if st["top_p"] is not None:
        mass = cum.gather(-1, kept - 1)
        p = ((cum - w) < st["top_p"].double()[:, None] * mass).sum(-1, keepdim=True)
        kept = torch.minimum(kept, torch.where(st["top_p"][:, None] < 1, p.clamp(min=1), kept))
    if st["min_p"] is not None:
        kept = torch.minimum(kept, (w >= st["min_p"].double()[:, None]).sum(-1, keepdim=True).clamp(min=1))
    # a temperature of 0 takes the first of the largest
    kept = torch.where(t > 0, kept, 1)
    aim = st["u"].double()[:, None] * cum.gather(-1, kept - 1)
    at = torch.minimum((cum <= aim).sum(-1, keepdim=True), kept - 1)
    return order.gather(-1, at)[:, 0].to(torch.int32)


# ----------------------------------------------------------------------------
# 64-bit results, from the definitions
# ----------------------------------------------------------------------------

def _code(c):
    """Value of a 4-bit code: sign, two exponent bits (bias 1), one fraction bit."""
    e, f = (c >> 1) & 3, c & 1
    v = torch.where(e > 0, torch.exp2(e.double() - 1) * (1 + 0.5 * f), 0.5 * f.double())
    return torch.where(c >= 8, -v, v)


def _exact_product(case, st):
    dout, half = st["codes"].shape
    w = torch.empty(dout, 2 * half, dtype=torch.float64, device=DEV)
    w[:, 0::2], w[:, 1::2] = _code(st["codes"].int() & 15), _code(st["codes"].int() >> 4)
    w = (w.view(dout, -1, GROUP) * torch.exp2(st["scales"].double() - 127)[..., None]).view(dout, -1)
    x = st["x"].double()
    y = x @ w.T
    at = 0
    for a, r in enumerate(_ranks(case)):
        down, up = (st["down"][a], st["up"][a]) if own else (st["down"][at:at + r], st["up"][:, at:at + r])
        at += r
        rows = st["ids"] == a
        y[rows] += st["scale"][a] * ((x[rows] @ down.double().T) @ up.double().T)
    return y


def _exact_quantise(case, st):
    w = st["w"].double().view(case["dout"], -1, GROUP)
    e = torch.full(w.shape[:2], -125, device=DEV, dtype=torch.float64)
    for i in range(-125, 125):  # one more as long as 6 * 2^e does not cover the largest
        e += (w.abs().amax(-1) > 6 * 2.0 ** i)
    scaled = w / torch.exp2(e)[..., None]
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)
    mid = (levels[1:] + levels[:-1]) / 2
    up, down = torch.bucketize(scaled.abs(), mid, right=True), torch.bucketize(scaled.abs(), mid)
    near = torch.where(up % 2 == 0, up, down)  # they differ where the value lies between two codes: the even one
    out = torch.sign(scaled) * levels[near] * torch.exp2(e)[..., None]
    return {"values": out.view(case["dout"], -1), "scales": (e + 127).to(torch.uint8)}


def _exact_rotate(case, st):
    new, total = _lengths(case)
    pos = torch.tensor([n - m + j for m, n in zip(new, total) for j in range(m)], dtype=torch.float64, device=DEV)
    r, out = case["rot"], {}
    for name in ("q", "k"):
        x = st[name].double()
        if case["norm"]:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + 1e-6) * st[name + "w"].double()
        first = torch.arange(r // 2, device=DEV)
        first, second = (2 * first, 2 * first + 1) if case["interleaved"] else (first, first + r // 2)
        turn = torch.polar(torch.ones(1, dtype=torch.float64, device=DEV), pos[:, None] * st["freqs"])[:, None]
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out


def _exact_sample(case, st):
    """A row at a time, over its distinct logits in falling order."""
    out = []
    get = lambda name, i, off: off if st[name] is None else st[name][i].double().item()
    for i in range(case["rows"]):
        x = st["logits"][i].double()
        level, where, count = torch.unique(x, return_inverse=True, return_counts=True)
        level, count, where = level.flip(0), count.flip(0).double(), level.numel() - 1 - where
        t, u = get("temperature", i, 1.0), get("u", i, 0.0)
        if t == 0:
            out.append((x == level[0]).nonzero()[0, 0])
            continue
        w = torch.exp((level - level[0]) / t)
        before, mass = torch.cumsum(count, 0) - count, torch.cumsum(count * w, 0)

        def mass_of(first):  # of the first tokens in order
            j = torch.searchsorted(before, first, right=True) - 1
            return mass[j] - w[j] * (count[j] - (first - before[j]))

        def reach(aim, more):  # tokens until their mass is at least aim (more: above it)
            j = torch.searchsorted(mass, aim, right=more).clamp(max=level.numel() - 1)
            part = (aim - (mass[j] - w[j] * count[j])) / w[j]
            need = torch.floor(part) + 1 if more else torch.ceil(part)
            return before[j] + torch.minimum(need.clamp(min=1), count[j])

        total = torch.tensor(float(case["vocab"]), dtype=torch.float64, device=DEV)
        k = get("top_k", i, 0)
        kept = total.clamp(max=k) if k > 0 else total
        p = get("top_p", i, 1.0)
        if p < 1:
            kept = torch.minimum(kept, reach(p * mass_of(kept), False))
        kept = torch.minimum(kept, count[w >= get("min_p", i, 0.0)].sum().clamp(min=1))
        at = torch.minimum(reach(u * mass_of(kept), True), kept)
        j = torch.searchsorted(before, at, right=False) - 1  # the level that holds token number `at`
        out.append((where == j).nonzero()[(at - before[j]).long() - 1, 0])
    return torch.stack(out).to(torch.int32)


def exact(case, seed):
    st = prepare(case, seed)
    return {"product": _exact_product, "quantise": _exact_quantise, "rotate": _exact_rotate,
            "sample": _exact_sample}[case["op"]](case, st)
