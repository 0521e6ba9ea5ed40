"""Measured cases of the plain key-value cache: the append of rotated keys and values, the attention of
one new token over the pages, the selection of pages by a cheap score, and the attention over a selection.

``listed()`` and ``draw()`` give cases, ``prepare()`` their inputs, ``run()`` one pass: the plain torch form where
``own`` is false, this package's calls where it is true. ``exact()`` gives the same outputs from the formulas in
64 bits. A page holds 64 tokens: per KV head the lower and upper bounds of its keys ([2][d], 16 bits each), then
per KV head the keys [64][d] and the values [64][d] (16 bits, or 8-bit codes followed by the keys' and the values'
fp16 scales, one per token and 32 channels).
"""
import math

import torch

own = False

PAGE = 64
ACT = {"bf16": torch.bfloat16, "f16": torch.float16, "int8": torch.bfloat16}  # type of queries, keys and results
DEV = "cuda"


# ------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 32 sequences: a token each, latency is all of it
        dict(name="append step 32", op="append", fmt="bf16", heads=32, kv=8, d=128, batch=32, new=1, ctx=1024, ragged=True),
        # the last chunk of a long prompt, at far positions
        dict(name="append prompt 8192 at 131072", op="append", fmt="bf16", heads=32, kv=8, d=128, batch=1, new=8192,
             ctx=131072, ragged=False),
        # prompts of a small batch into an 8-bit cache, one KV head per query head, lengths off the page grid
        dict(name="append int8 3 x 335", op="append", fmt="int8", heads=32, kv=32, d=128, batch=3, new=335, ctx=1029,
             ragged=True),
        # one short conversation: the smallest attention call
        dict(name="decode 1 x 1000", op="decode", fmt="bf16", heads=32, kv=8, d=128, batch=1, ctx=1000, ragged=False,
             window=0, empty=False),
        # one KV head per query head
        dict(name="decode 8 x 4096 mha", op="decode", fmt="bf16", heads=32, kv=32, d=128, batch=8, ctx=4096, ragged=False,
             window=0, empty=False),
        # a serving batch at long context: the largest call
        dict(name="decode 32 x 32768", op="decode", fmt="bf16", heads=32, kv=8, d=128, batch=32, ctx=32768, ragged=False,
             window=0, empty=False),
        # one very long sequence from an 8-bit cache
        dict(name="decode int8 1 x 131072", op="decode", fmt="int8", heads=32, kv=8, d=128, batch=1, ctx=131072,
             ragged=False, window=0, empty=False),
        # a ragged batch of a layer with a sliding window, three query heads per KV head, an empty slot in the batch
        dict(name="decode f16 ragged window", op="decode", fmt="f16", heads=24, kv=8, d=64, batch=17, ctx=8191, ragged=True,
             window=2000, empty=True),
        # the selection alone, for a serving batch
        dict(name="select 32 x 32768", op="select", fmt="bf16", heads=32, kv=8, d=128, batch=32, ctx=32768, ragged=False,
             pages=64, first=1, last=2),
        # the selection alone, for one very long sequence
        dict(name="select 1 x 131000", op="select", fmt="bf16", heads=32, kv=8, d=128, batch=1, ctx=131000, ragged=False,
             pages=32, first=1, last=1),
        # selection and attention of a decode step, an eighth of the cache
        dict(name="sparse 32 x 32768", op="sparse", fmt="bf16", heads=32, kv=8, d=128, batch=32, ctx=32768, ragged=False,
             pages=64, first=1, last=2),
        # a small ragged batch, eight query heads per KV head, some sequences shorter than the budget
        dict(name="sparse f16 3 ragged", op="sparse", fmt="f16", heads=16, kv=2, d=128, batch=3, ctx=5000, ragged=True,
             pages=9, first=1, last=2),
    ]


HEADS = [(32, 8, 128), (32, 32, 128), (16, 2, 128), (16, 16, 64), (24, 8, 64), (4, 4, 64), (64, 4, 128), (10, 2, 128)]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "select", "sparse"])
    fmt = rng.choice(["bf16", "f16", "int8"])
    heads, kv, d = rng.choice(HEADS)
    c = dict(op=op, fmt=fmt, heads=heads, kv=kv, d=d)
    batch = spread(rng, 1, 48)
    if op == "append":
        new = spread(rng, 1, 8192 // batch)
        return dict(c, batch=batch, new=new, ctx=new + spread(rng, 1, 4096), ragged=rng.random() < 0.5)
    ctx = spread(rng, 1 if op == "decode" else 64, min(131072, 500000 // batch))
    if batch * ctx * kv * d > 1 << 29:  # no larger than the largest listed case
        ctx = max(64, (1 << 29) // (batch * kv * d))
    c = dict(c, batch=batch, ctx=ctx, ragged=rng.random() < 0.5)
    if op == "decode":
        return dict(c, window=spread(rng, 1, ctx) if rng.random() < 0.25 else 0, empty=rng.random() < 0.25)
    first, last = rng.randint(0, 2), rng.randint(1, 3)
    return dict(c, pages=first + last + spread(rng, 1, 120), first=first, last=last)


def lengths(c):
    """Tokens of each sequence, the new ones among them."""
    low = c.get("new", 1)
    n = [c["ctx"]] * c["batch"]
    if c["ragged"]:
        n = [low + (c["ctx"] - low) * ((37 * b + 100) % 101) // 100 for b in range(c["batch"])]
    if c.get("empty"):
        n[0 if c["batch"] == 1 else 1] = 0
    return n


def pages_of(n):
    return -(-n // PAGE)


def sizes(c):
    """Bytes of a page's bounds, of a KV head's tile, of its keys, and of a page."""
    bounds = 2 * c["d"] * 2 * c["kv"]
    keys = PAGE * c["d"] * (1 if c["fmt"] == "int8" else 2)
    tile = 2 * keys + (2 * PAGE * (c["d"] // 32) * 2 if c["fmt"] == "int8" else 0)
    return bounds, tile, keys, bounds + c["kv"] * tile


def work(c):
    lens, (bounds, tile, _, _) = lengths(c), sizes(c)
    H, kv, d, B = c["heads"], c["kv"], c["d"], c["batch"]
    token = kv * tile // PAGE
    if c["op"] == "append":
        n = B * c["new"]
        done = sum(n // PAGE - (n - c["new"]) // PAGE for n in lens)
        moved = n * (H * d * 2 * 2 + 2 * kv * d * 2 + token) + done * bounds
        return {"bytes": moved, "flops": 3 * n * (H + kv) * d + 2 * done * PAGE * kv * d}
    span = [min(n, c["window"]) if c.get("window") else n for n in lens]
    rows = B * H * (d * 2 * 2 + 4)
    if c["op"] == "decode":
        return {"bytes": sum(span) * token + rows, "flops": 4 * sum(span) * H * d}
    P = [pages_of(n) for n in lens]
    scored = sum(max(0, p - c["first"] - c["last"]) for p in P if p > c["pages"])
    choice = {"bytes": scored * bounds + B * (H * d * 2 + kv * c["pages"] * 4), "flops": 2 * scored * H * d}
    if c["op"] == "select":
        return choice
    read = sum(min(n, c["pages"] * PAGE) for n in lens)
    return {"bytes": choice["bytes"] + read * token + rows, "flops": choice["flops"] + 4 * read * H * d}


# ------------------------------------------------------------------------------------------- the inputs
def tiles_of(pool, c):
    """Views of the pool: bounds [pages][kv][2][d]; keys and values [pages][kv][64][d]; their scales or None."""
    n, (bounds, tile, keys, _), kv, d = pool.shape[0], sizes(c), c["kv"], c["d"]
    b = pool[:, :bounds].view(ACT[c["fmt"]]).unflatten(1, (kv, 2, d))
    t = pool[:, bounds:].unflatten(1, (kv, tile))
    el = torch.int8 if c["fmt"] == "int8" else ACT[c["fmt"]]
    k, v = (t[:, :, i * keys:(i + 1) * keys].view(el).unflatten(2, (PAGE, d)) for i in (0, 1))
    if c["fmt"] != "int8":
        return b, k, v, None, None
    half = PAGE * (d // 32) * 2
    ks, vs = (t[:, :, 2 * keys + i * half:2 * keys + (i + 1) * half].view(torch.float16).unflatten(2, (PAGE, d // 32))
              for i in (0, 1))
    return b, k, v, ks, vs


def prepare(c, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    kv, d, B, fmt = c["kv"], c["d"], c["batch"], c["fmt"]
    lens = lengths(c)
    width = max(1, max(pages_of(n) for n in lens))
    count = max(1, sum(pages_of(n) for n in lens))
    pool = torch.empty(count, sizes(c)[3], dtype=torch.uint8, device=DEV)
    bounds, keys, values, ks, vs = tiles_of(pool, c)
    # keys have a mean per channel, as trained ones do; the tiles are filled some pages at a time
    mean = torch.randn(kv, 1, d, device=DEV, generator=g)
    step = max(1, (1 << 26) // (kv * PAGE * d))
    for i in range(0, count, step):
        j = min(count, i + step)
        shape = (j - i, kv, PAGE, d)
        for to, scales, x in ((keys, ks, torch.randn(shape, device=DEV, generator=g) + mean),
                              (values, vs, torch.randn(shape, device=DEV, generator=g))):
            if scales is None:
                to[i:j] = x.to(to.dtype)
                continue
            s = (x.unflatten(3, (d // 32, 32)).abs().amax(-1) / 127).half()
            scales[i:j] = s
            to[i:j] = torch.round(x / s.float().repeat_interleave(32, 3)).clamp(-127, 127).to(torch.int8)
        k = keys[i:j].float() if ks is None else keys[i:j].float() * ks[i:j].float().repeat_interleave(32, 3)
        bounds[i:j, :, 0] = k.amin(2).to(bounds.dtype)
        bounds[i:j, :, 1] = k.amax(2).to(bounds.dtype)
    # pages in a random order
    order = torch.randperm(count, device=DEV, generator=g).int()
    table = torch.zeros(B, width, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(lens):
        table[b, :pages_of(n)] = order[at:at + pages_of(n)]
        at += pages_of(n)
    s = dict(c=c, pool=pool, table=table, theta=500000.0, lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    act = ACT[fmt]
    if c["op"] == "append":
        # the layer's fused projection: queries, keys and values of a token side by side
        n = B * c["new"]
        s["qkv"] = torch.randn(n, (c["heads"] + 2 * kv) * d, device=DEV, generator=g).to(act)
        s["seq"] = torch.arange(B, device=DEV, dtype=torch.int32).repeat_interleave(c["new"])
        first = (s["lens"] - c["new"]).repeat_interleave(c["new"])
        s["pos"] = first + torch.arange(c["new"], device=DEV, dtype=torch.int32).repeat(B)
        # the pages whose last slot this call fills
        s["done"] = torch.cat([table[b, (m - c["new"]) // PAGE:m // PAGE] for b, m in enumerate(lens)]).long()
        s["q_out"] = torch.empty(n, c["heads"], d, dtype=act, device=DEV)
        s["k_out"], s["v_out"] = (torch.empty(n, kv, d, dtype=act, device=DEV) for _ in range(2))
    else:
        s["q"] = (1.5 * torch.randn(B, c["heads"], d, device=DEV, generator=g)).to(act)
        s["out"] = torch.empty(B, c["heads"], d, dtype=act, device=DEV)
        s["lse"] = torch.empty(B, c["heads"], dtype=torch.float32, device=DEV)
        s["sel"] = torch.empty(B, kv, c.get("pages", 1), dtype=torch.int32, device=DEV)
    if own:  # the layout, the rotation table, the workspace and the status word that a program keeps
        from rank_quantized_kv_decode_b200 import api
        lay = api.kv_layout_init(api.make_kv_config(c["heads"], kv, d, fmt, s["theta"]))
        s["kv"] = api.KvCache.create(lay, 0, B, width)
    return s


# ------------------------------------------------------------------------------------------- one pass
def run(s):
    c = s["c"]
    return (own_form if own else plain_form)[c["op"]](s, c)


def own_append(s, c):
    from rank_quantized_kv_decode_b200 import api
    w, H, kv, d = s["kv"], c["heads"], c["kv"], c["d"]
    q, k, v = s["qkv"].unflatten(1, (H + 2 * kv, d)).split((H, kv, kv), 1)
    api.kv_append(w.layout, k, v, s["seq"], s["pos"], s["table"], s["pool"], w.rope, w.status, q=q, q_out=s["q_out"])
    if c["fmt"] != "int8":
        return s["pool"].view(ACT[c["fmt"]]), s["q_out"]
    api.kv_gather(w.layout, s["pool"], s["seq"], s["pos"], s["table"], s["k_out"], s["v_out"], w.status)
    return tiles_of(s["pool"], c)[0], s["q_out"], s["k_out"], s["v_out"]


def own_decode(s, c, sel=None):
    from rank_quantized_kv_decode_b200 import api
    w = s["kv"]
    api.kv_decode(w.layout, s["q"], s["pool"], s["table"], s["lens"], s["out"], w.decode_ws, w.status, sel=sel,
                  lse=s["lse"], window=c.get("window", 0))
    return s["out"], s["lse"]


def own_select(s, c):
    from rank_quantized_kv_decode_b200 import api
    w = s["kv"]
    api.kv_select(w.layout, s["q"], s["pool"], s["table"], s["lens"], s["sel"], w.status, keep_first=c["first"],
                  keep_last=c["last"])
    return s["sel"]


def own_sparse(s, c):
    sel = own_select(s, c)
    return (sel,) + own_decode(s, c, sel)


own_form = dict(append=own_append, decode=own_decode, select=own_select, sparse=own_sparse)


def rotate(x, pos, theta):
    """Half-split rotation of x [n][heads][d] in 32 bits; the angles in 64, for far positions."""
    h = x.shape[-1] // 2
    f = theta ** (-torch.arange(h, device=x.device, dtype=torch.float64) / h)
    a = pos.double()[:, None, None] * f
    cs, sn = a.cos().float(), a.sin().float()
    x = x.float()
    return torch.cat((x[..., :h] * cs - x[..., h:] * sn, x[..., h:] * cs + x[..., :h] * sn), -1)


def codes_of(x):
    """8-bit codes of x [...][d] and their fp16 scales [...][d / 32]."""
    g = x.float().unflatten(-1, (-1, 32))
    s = (g.abs().amax(-1) / 127).clamp(max=65504).half()
    q = torch.where(s[..., None] > 0, torch.round(g / s.float()[..., None]), 0)
    return q.clamp(-127, 127).to(torch.int8).flatten(-2), s


def values_of(q, s):
    """The values of 8-bit codes, or of 16-bit numbers as they are, in 32 bits."""
    return q.float() if s is None else (q.float().unflatten(-1, (-1, 32)) * s.float()[..., None]).flatten(-2)


def plain_append(s, c):
    H, kv, d, act = c["heads"], c["kv"], c["d"], ACT[c["fmt"]]
    q, k, v = s["qkv"].unflatten(1, (H + 2 * kv, d)).split((H, kv, kv), 1)
    q, k = rotate(q, s["pos"], s["theta"]).to(act), rotate(k, s["pos"], s["theta"])
    bounds, keys, values, ks, vs = tiles_of(s["pool"], c)
    pos, done = s["pos"].long(), s["done"]
    page, slot = s["table"][s["seq"].long(), pos // PAGE].long(), pos % PAGE
    if ks is None:
        keys[page, :, slot], values[page, :, slot] = k.to(act), v
    else:
        keys[page, :, slot], ks[page, :, slot] = codes_of(k)
        values[page, :, slot], vs[page, :, slot] = codes_of(v)
    x = values_of(keys[done], None if ks is None else ks[done])
    bounds[done] = torch.stack((x.amin(2), x.amax(2)), 2).to(act)
    if ks is None:
        return s["pool"].view(act), q
    return (bounds, q, values_of(keys[page, :, slot], ks[page, :, slot]).to(act),
            values_of(values[page, :, slot], vs[page, :, slot]).to(act))


def attend(s, c, k, v, pos):
    """Attention over k, v [B][kv][T][d] at positions pos [B or 1][kv or 1][T] (below 0: none there)."""
    B, H, d, kv = c["batch"], c["heads"], c["d"], c["kv"]
    lens = s["lens"].long()[:, None, None]
    ok = (pos >= 0) & (pos < lens)
    if c.get("window"):
        ok &= pos >= lens - c["window"]
    q = s["q"].float().view(B, kv, H // kv, d)
    x = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
    x = torch.where(ok[:, :, None], x, -math.inf)
    m = x.amax(3, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - m)
    l = p.sum(3, keepdim=True)
    v = torch.where(ok[..., None], v, 0.0)
    o = torch.where(l > 0, torch.matmul(p, v) / l, 0.0)
    return o.view(B, H, d).to(s["out"].dtype), (m + torch.log(l)).view(B, H)


def plain_decode(s, c):
    _, keys, values, ks, vs = tiles_of(s["pool"], c)
    ids = s["table"].long()
    k, v = (values_of(x[ids], None if y is None else y[ids]).permute(0, 2, 1, 3, 4).flatten(2, 3)
            for x, y in ((keys, ks), (values, vs)))
    return attend(s, c, k, v, torch.arange(k.shape[2], device=k.device)[None, None])


def plain_select(s, c):
    B, kv, H, d = c["batch"], c["kv"], c["heads"], c["d"]
    bounds = tiles_of(s["pool"], c)[0][s["table"].long()].permute(3, 0, 2, 4, 1).double()  # [2][B][kv][d][pages]
    q = s["q"].double().view(B, kv, H // kv, d)
    score = (torch.matmul(q.clamp(min=0), bounds[1]) + torch.matmul(q.clamp(max=0), bounds[0])).amax(2)
    at = torch.arange(score.shape[2], device=score.device)
    count = ((s["lens"].long() + PAGE - 1) // PAGE)[:, None, None]
    score = torch.where((at < c["first"]) | (at >= count - c["last"]), math.inf, score)
    score = torch.where(at < count, score, -math.inf)
    best = torch.sort(score, dim=2, descending=True, stable=True).indices[..., :c["pages"]]
    far = torch.iinfo(torch.int32).max
    best = torch.sort(torch.where(best < count, best, far), dim=2).values
    out = torch.full((B, kv, c["pages"]), -1, device=score.device, dtype=torch.int32)
    out[..., :best.shape[2]] = torch.where(best < far, best, -1).int()
    return out


def plain_sparse(s, c):
    sel = plain_select(s, c)
    _, keys, values, ks, vs = tiles_of(s["pool"], c)
    at = sel.long()
    table = s["table"].long()
    ids = torch.gather(table[:, None].expand(-1, c["kv"], -1), 2, at.clamp(min=0))
    g = torch.arange(c["kv"], device=at.device)[None, :, None]
    k, v = (values_of(x[ids, g], None if y is None else y[ids, g]).flatten(2, 3) for x, y in ((keys, ks), (values, vs)))
    pos = torch.where(at[..., None] >= 0, at[..., None] * PAGE + torch.arange(PAGE, device=at.device), -1).flatten(2)
    return (sel,) + attend(s, c, k, v, pos)


plain_form = dict(append=plain_append, decode=plain_decode, select=plain_select, sparse=plain_sparse)


# ------------------------------------------------------------------------------------------- in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    return {"append": exact_append, "decode": exact_attention, "select": exact_choice,
            "sparse": lambda s, c: (exact_choice(s, c),) + exact_attention(s, c, exact_choice(s, c))}[c["op"]](s, c)


def exact_tokens(s, c, b, g, pages):
    """Keys and values of one KV head in the given pages of sequence b, in 64 bits."""
    _, keys, values, ks, vs = tiles_of(s["pool"], c)
    ids = s["table"][b, pages].long()
    x, y = keys[ids, g].double(), values[ids, g].double()
    if ks is not None:
        x = x * ks[ids, g].double().repeat_interleave(32, -1)
        y = y * vs[ids, g].double().repeat_interleave(32, -1)
    return x.reshape(-1, c["d"]), y.reshape(-1, c["d"])


def exact_attention(s, c, sel=None):
    B, H, d, kv = c["batch"], c["heads"], c["d"], c["kv"]
    G = H // kv
    out = torch.zeros(B, H, d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lengths(c)):
        if n == 0:
            continue
        low = max(0, n - c["window"]) if c.get("window") else 0
        for g in range(kv):
            if sel is None:
                pages = torch.arange(low // PAGE, pages_of(n), device=DEV)
            else:
                pages = sel[b, g][sel[b, g] >= 0].long()
            k, v = exact_tokens(s, c, b, g, pages)
            pos = (pages[:, None] * PAGE + torch.arange(PAGE, device=DEV)).reshape(-1)
            in_use = (pos < n) & (pos >= low)
            x = s["q"][b, g * G:(g + 1) * G].double() @ k[in_use].T * d ** -0.5
            lse[b, g * G:(g + 1) * G] = torch.logsumexp(x, 1)
            out[b, g * G:(g + 1) * G] = torch.softmax(x, 1) @ v[in_use]
    return out, lse


def exact_choice(s, c):
    sel = torch.full((c["batch"], c["kv"], c["pages"]), -1, dtype=torch.int32)
    bounds = tiles_of(s["pool"], c)[0]
    G = c["heads"] // c["kv"]
    for b, n in enumerate(lengths(c)):
        P = pages_of(n)
        ids = s["table"][b, :P].long()
        # [kv][G][pages]: the largest product of a key inside the bounds
        lo, hi = (bounds[ids, :, i].double().transpose(0, 1)[:, None] for i in (0, 1))
        q = s["q"][b].double().view(c["kv"], G, 1, c["d"])
        score = torch.cat([torch.maximum(q * lo[:, :, i:i + 256], q * hi[:, :, i:i + 256]).sum(-1).amax(1)
                           for i in range(0, P, 256)], 1).cpu()
        for g in range(c["kv"]):
            if P <= c["pages"]:
                chosen = list(range(P))
            else:
                ends = list(range(c["first"])) + list(range(P - c["last"], P))
                rest = sorted(range(c["first"], P - c["last"]), key=lambda p: (-float(score[g, p]), p))
                chosen = sorted(ends + rest[:c["pages"] - len(ends)])
            sel[b, g, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
    return sel.to(DEV)


def exact_append(s, c):
    H, kv, d, n = c["heads"], c["kv"], c["d"], s["qkv"].shape[0]
    x = s["qkv"].double().view(n, H + 2 * kv, d)
    turn = torch.exp(-math.log(s["theta"]) * torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d)
    z = torch.polar(torch.ones(n, d // 2, device=DEV, dtype=torch.float64), s["pos"].double()[:, None] * turn)[:, None]
    x[:, :H + kv] = torch.view_as_real(torch.complex(x[:, :H + kv, :d // 2], x[:, :H + kv, d // 2:]) * z) \
        .transpose(2, 3).reshape(n, H + kv, d)
    q, k, v = x[:, :H], x[:, H:H + kv], x[:, H + kv:]
    bounds, keys, values, ks, vs = (None if t is None else t.double() for t in tiles_of(s["pool"], c))
    if ks is not None:
        def stored(t):  # the code nearest to t / scale, times the scale
            t = t.unflatten(2, (d // 32, 32))
            scale = (t.abs().amax(3, keepdim=True) / 127).clamp(max=65504).half().double()
            return torch.where(scale > 0, torch.round(t / scale).clamp(-127, 127) * scale, 0.0).flatten(2)
        keys *= ks.repeat_interleave(32, 3)
        k, v = stored(k), stored(v)
    page = s["table"][s["seq"].long(), s["pos"].long() // PAGE].long()
    slot = s["pos"].long() % PAGE
    keys[page, :, slot] = k
    for p in s["done"]:
        bounds[p, :, 0], bounds[p, :, 1] = keys[p].min(1).values, keys[p].max(1).values
    if ks is not None:
        return bounds, q, k, v
    values[page, :, slot] = v
    whole = torch.stack((keys, values), 2).flatten(1)
    return torch.cat((bounds.flatten(1), whole), 1), q
