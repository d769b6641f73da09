"""Cases of what stands between the q, k, v linears of a block and its output
linear: norms and rotation of the heads, the cache of keys and values, and one
token's attention over it.

Operators
  heads       q' = rotate(norm(q)), k' = rotate(norm(k)): a root-mean-square norm of
              each head with weights, then its first `rot` channels turned pair by
              pair by position times frequency; up to three axes of positions.
  heads_bwd   the gradients of heads: q, k and both weights.
  kv          keys and values of new tokens written to their slots of a paged cache,
              and a context read back from it.
  attend      attention of one new token a sequence over the cache in pages.
  step        heads, the write of the new token and its attention: a decode step.

A cache holds bf16, or whole numbers c of 8 bits (|c| <= 127, one scale for each
token and head) or of 4 bits (|c| <= 7, one for 32 channels of it):
s = bf16(max |x| / 127 or 7), c = x / s to the nearest, ties to even.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6
BASE = 500000.0


def heads(name, T, Hq, Hkv, D, rot, pairs, act, axes=1, fused=False, bwd=False):
    return {"name": name, "op": "heads_bwd" if bwd else "heads", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
            "pairs": pairs, "act": act, "axes": axes, "fused": fused}


def kv(name, T, context, Hkv, D, page, kind, act):
    return {"name": name, "op": "kv", "T": T, "context": context, "Hkv": Hkv, "D": D, "page": page, "kind": kind,
            "act": act}


def attend(name, B, longest, ragged, Hq, Hkv, D, page, kind, act, window=0, step=False):
    return {"name": name, "op": "step" if step else "attend", "B": B, "longest": longest, "ragged": ragged, "Hq": Hq,
            "Hkv": Hkv, "D": D, "page": page, "kind": kind, "act": act, "window": window}


def listed():
    return [
        # one token: what one call costs
        heads("heads token", 1, 64, 8, 128, 128, "halves", "bf16"),
        # a prompt of 2048 tokens, q and k parts of one linear's output
        heads("heads prompt", 2048, 64, 8, 128, 128, "halves", "bf16", fused=True),
        # tokens of pictures: time, height and width, heads of 80 channels
        heads("heads pictures", 1023, 16, 16, 80, 80, "halves", "f32", axes=3),
        # gradients of a training step of 4096 tokens
        heads("heads gradients", 4096, 64, 8, 128, 128, "halves", "bf16", bwd=True),
        # gradients of a ragged batch, odd heads, half of their channels turned in neighbouring pairs
        heads("heads gradients odd", 333, 9, 3, 100, 50, "neighbours", "f32", bwd=True),
        # a piece of a prompt is written, the context up to it read for its attention
        kv("cache prompt", 512, 8192, 8, 128, 64, "int8", "bf16"),
        # one token of each of 61 sequences
        kv("cache tokens", 61, 61, 8, 128, 16, "int4", "f32"),
        # a conversation's first tokens
        attend("step token", 1, 100, False, 64, 8, 128, 64, "bf16", "bf16", step=True),
        # 64 conversations of different lengths
        attend("step batch", 64, 4096, True, 64, 8, 128, 32, "int8", "bf16", step=True),
        # one long document
        attend("attend long", 1, 131072, False, 64, 8, 128, 64, "int8", "bf16"),
        # long conversations of different lengths
        attend("attend batch", 32, 16384, True, 64, 8, 128, 64, "bf16", "bf16"),
        # every head with keys of its own, small pages, the last 2000 tokens seen
        attend("attend window", 7, 5001, True, 12, 12, 64, 16, "int4", "f32", window=2000),
    ]


def draw(rng: random.Random):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(("heads", "heads_bwd", "kv", "attend", "attend", "step"))
    act = rng.choice(("bf16", "bf16", "f32"))
    Hkv = size(1, 16)
    Hq = Hkv * rng.choice((1, 2, 4, 5, 8, 16))
    while Hq > 96:
        Hkv = max(1, Hkv // 2)
        Hq = Hq // 2 // Hkv * Hkv or Hkv
    if op in ("heads", "heads_bwd"):
        D = rng.choice((64, 80, 96, 100, 128, 128, 192, 256))
        axes = rng.choice((1, 1, 2, 3))
        rot = rng.choice((D, D, D // 2 // 2 * 2))
        T = size(1, 8192)
        while T * (Hq + Hkv) * D > 4096 * 72 * 128:
            T = max(1, T // 2)
        c = heads("", T, Hq, Hkv, D, rot, rng.choice(("halves", "halves", "neighbours")), act, axes, rng.random() < 0.5,
                  op == "heads_bwd")
    else:
        D, page, kind = rng.choice((64, 96, 128, 128, 192, 256)), rng.choice((16, 32, 64, 128)), \
            rng.choice(("bf16", "int8", "int4"))
        if op == "kv":
            T = size(1, 4096)
            context = T + size(1, 16384)
            while context * Hkv * D > 2 ** 23:
                T, context = max(1, T // 2), max(2, context // 2)
            c = kv("", T, context, Hkv, D, page, kind, act)
        else:
            B, longest = size(1, 128), size(1, 131072)
            while B * longest * Hkv * D > 5 * 2 ** 25:
                B, longest = max(1, B // 2), max(1, longest // 2 + 1)
            window = size(1, longest) if rng.random() < 0.25 else 0
            c = attend("", B, longest, rng.random() < 0.7, Hq, Hkv, D, page, kind, "bf16" if op == "step" else act, window,
                       op == "step")
    del c["name"]
    return c


def lengths_of(case):
    """Tokens of each sequence, the new one among them: spread over their logarithm, the first the longest; where
    sequences come and go one place of the batch is empty."""
    if not case["ragged"]:
        return [case["longest"]] * case["B"]
    r = random.Random(case["B"] * 1000003 + case["longest"])
    low = max(1, case["longest"] // 16)
    some = [int(round(math.exp(r.uniform(math.log(low), math.log(case["longest"]))))) for _ in range(case["B"])]
    some[0] = case["longest"]
    if case["op"] == "attend" and case["B"] > 3:
        some[2] = 0
    return some


def sections_of(case):
    """How many of the rot / 2 frequencies go by each axis."""
    n, A = case["rot"] // 2, case["axes"]
    first = [n // A] * (A - 1)
    return first + [n - sum(first)]


# ------------------------------------------------------------------ inputs
def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def frequencies(rot):
    return BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)


def head_inputs(case, g, T, positions):
    """q, k and v of T tokens, parts of one tensor where a linear makes all three, and the norms' weights."""
    Hq, Hkv, D, act = case["Hq"], case["Hkv"], case["D"], DT[case["act"]]
    cut = [Hq * D, Hkv * D, Hkv * D]
    x = randn(g, T, sum(cut))
    x *= torch.where(torch.rand(sum(cut), generator=g, device="cuda") < 0.01, 8.0, 1.0)  # a few channels are large
    q, k, v = (p if case.get("fused") else p.contiguous() for p in x.to(act).split(cut, dim=1))
    return {"q": q.unflatten(1, (Hq, D)), "k": k.unflatten(1, (Hkv, D)), "v": v.unflatten(1, (Hkv, D)),
            "w_q": 1 + 0.2 * randn(g, D), "w_k": 1 + 0.2 * randn(g, D), "positions": positions}


def far_positions(case, g):
    """(axes, T): the first axis goes on from some place of a long context, the others stay in a picture."""
    T, at = case["T"], torch.randint(0, 131072, (1,), generator=g, device="cuda")
    rows = [at + torch.arange(T, device="cuda")]
    rows += [torch.randint(0, 64, (T,), generator=g, device="cuda") for _ in range(case["axes"] - 1)]
    return torch.stack(rows)


def cache_inputs(case, g, pages):
    """Keys and values of every slot of the cache."""
    shape = (pages * case["page"], case["Hkv"], case["D"])
    loud = torch.where(torch.rand(1, *shape[1:], generator=g, device="cuda") < 0.02, 4.0, 1.0)
    return (randn(g, *shape) * loud).to(DT[case["act"]]), randn(g, *shape).to(DT[case["act"]])


def paging(case, g):
    """Lengths, and each sequence's pages: scattered over a cache with a few pages to spare."""
    lengths = torch.tensor(lengths_of(case), device="cuda", dtype=torch.int32)
    need = [-(-n // case["page"]) for n in lengths_of(case)]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(case["B"], max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return lengths, table, pages


def step_inputs(case, g):
    lengths, table, pages = paging(case, g)
    keys, values = cache_inputs(case, g, pages)
    t = {"lengths": lengths, "table": table, "pages": pages, "keys": keys, "values": values}
    if case["op"] == "attend":
        t["q"] = (1.5 * randn(g, case["B"], case["Hq"], case["D"])).to(DT[case["act"]])
        return t
    last = lengths.long() - 1
    page = table.long().gather(1, (last // case["page"])[:, None])[:, 0]
    t["slots"] = page * case["page"] + last % case["page"]
    return t | head_inputs(case, g, case["B"], last[None])


def kv_inputs(case, g):
    pages = -(-case["context"] // case["page"]) + 2
    keys, values = cache_inputs(case, g, pages)
    order = torch.randperm(pages, generator=g, device="cuda")
    at = torch.arange(case["context"], device="cuda")
    slots = order[at // case["page"]] * case["page"] + at % case["page"]
    shape = (case["T"], case["Hkv"], case["D"])
    return {"pages": pages, "keys": keys, "values": values, "context": slots, "slots": slots[-case["T"]:],
            "k": randn(g, *shape).to(DT[case["act"]]), "v": randn(g, *shape).to(DT[case["act"]])}


def inputs(case, g):
    if case["op"] == "kv":
        return kv_inputs(case, g)
    if case["op"] in ("attend", "step"):
        return step_inputs(case, g)
    t = head_inputs(case, g, case["T"], far_positions(case, g))
    if case["op"] == "heads_bwd":
        t["dq"], t["dk"] = (randn(g, *t[n].shape).to(DT[case["act"]]) for n in ("q", "k"))
    del t["v"]
    return t


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = inputs(case, g)
    st["case"] = case
    if case["op"] != "kv" and case["op"] != "attend":
        st["rot"] = case.get("rot", case["D"])
        st["inv_freq"] = frequencies(st["rot"])
        st["sections"] = sections_of(case) if "axes" in case else [st["rot"] // 2]
    if own:
        import binary_rank_gemv_packed_amd as nq
        if "inv_freq" in st:
            st["norm"] = nq.HeadNorm(case["D"], act_dtype=DT[case["act"]], w_q=st["w_q"], w_k=st["w_k"],
                                     inv_freq=st["inv_freq"], interleaved=case.get("pairs") == "neighbours",
                                     sections=st["sections"], eps=EPS)
        if "keys" in st:
            keys, values = st.pop("keys"), st.pop("values")
            st["cache"] = nq.KvCache(st["pages"], case["Hkv"], case["D"], page=case["page"], kind=case["kind"])
            nq.kv_write(keys, values, st["cache"], torch.arange(len(keys), device="cuda"))
        if "table" in st:
            st["ws"] = nq.new_kv_workspace(case["B"], case["Hq"], st["cache"])
    elif "keys" in st:
        st["stored"] = [held(st.pop(n), case["kind"]) for n in ("keys", "values")]
    return st


# ------------------------------------------------------------------ one pass in plain form
def held(x, kind):
    """What the cache holds for x (slots, heads, D): [values], or [whole numbers, scales]."""
    if kind == "bf16":
        return [x.to(torch.bfloat16)]
    most = 127.0 if kind == "int8" else 7.0
    x = x.float().unflatten(-1, (1, -1) if kind == "int8" else (-1, 32))
    top = x.abs().amax(-1, keepdim=True)
    s = (top / torch.full_like(top, most)).bfloat16()
    c = torch.where(s == 0, 0.0, x / s.float()).round().clamp(-most, most)
    return [c.flatten(-2).to(torch.int8), s[..., 0]]


def values_of(parts):
    if len(parts) == 1:
        return parts[0].float()
    c, s = parts
    return (c.float().unflatten(-1, (s.shape[-1], -1)) * s.float()[..., None]).flatten(-2)


def put(stored, slots, x, kind):
    new = held(x, kind)
    stored[0][slots] = new[0]
    stored[-1][slots] = new[-1]


def angles(st):
    """cos and sin (T, 1, rot / 2); the angle itself in 64 bits, for positions are far."""
    axis = torch.repeat_interleave(torch.arange(len(st["sections"]), device="cuda"),
                                   torch.tensor(st["sections"], device="cuda"), output_size=st["rot"] // 2)
    phi = st["positions"].double().t()[:, axis] * st["inv_freq"]
    return phi.cos().float()[:, None], phi.sin().float()[:, None]


def pairs_of(st, x):
    """The two members of each pair of the turned channels of x, and the channels left as they are."""
    turned, rest = x[..., :st["rot"]], x[..., st["rot"]:]
    if st["case"].get("pairs") == "neighbours":
        return turned[..., 0::2], turned[..., 1::2], rest
    return *turned.chunk(2, -1), rest


def joined(st, a, b, rest):
    turned = torch.stack((a, b), -1).flatten(-2) if st["case"].get("pairs") == "neighbours" else torch.cat((a, b), -1)
    return torch.cat((turned, rest), -1)


def plain_head(st, x, w, cos, sin):
    xf = x.float()
    n = xf * torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS) * w
    a, b, rest = pairs_of(st, n)
    return joined(st, a * cos - b * sin, a * sin + b * cos, rest).to(x.dtype)


def plain_head_bwd(st, dy, x, w, cos, sin):
    a, b, rest = pairs_of(st, dy.float())
    g = joined(st, a * cos + b * sin, b * cos - a * sin, rest)
    xf = x.float()
    r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
    n, t = xf * r, g * w
    return (r * (t - n * (t * n).mean(-1, keepdim=True))).to(x.dtype), (g * n).sum((0, 1))


def plain_attend(st, q):
    case = st["case"]
    B, Hq, D = q.shape
    Hkv, page = case["Hkv"], case["page"]
    at = torch.arange(st["table"].shape[1] * page, device="cuda")
    slots = st["table"].long()[:, at // page] * page + at % page
    n = st["lengths"].long()[:, None]
    seen = at < n
    if case["window"]:
        seen = seen & (at >= n - case["window"])
    k, v = (values_of([p[slots] for p in parts]) for parts in st["stored"])  # (B, L, Hkv, D)
    x = (q.float() / math.sqrt(D)).view(B, Hkv, Hq // Hkv, D) @ k.permute(0, 2, 3, 1)
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp_min(-1e30))
    y = (p @ v.transpose(1, 2)) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    return y.view(B, Hq, D).to(q.dtype)


def plain(st):
    case = st["case"]
    op, act = case["op"], DT[case["act"]]
    if op == "kv":
        for parts, x in zip(st["stored"], (st["k"], st["v"])):
            put(parts, st["slots"], x, case["kind"])
        return [values_of([p[st["context"]] for p in parts]).to(act) for parts in st["stored"]]
    if op == "attend":
        return plain_attend(st, st["q"])
    cos, sin = angles(st)
    if op == "heads_bwd":
        dq, dw_q = plain_head_bwd(st, st["dq"], st["q"], st["w_q"], cos, sin)
        dk, dw_k = plain_head_bwd(st, st["dk"], st["k"], st["w_k"], cos, sin)
        return {"dq": dq, "dk": dk, "dw_q": dw_q, "dw_k": dw_k}
    q, k = plain_head(st, st["q"], st["w_q"], cos, sin), plain_head(st, st["k"], st["w_k"], cos, sin)
    if op == "heads":
        return q, k
    for parts, x in zip(st["stored"], (k, st["v"])):
        put(parts, st["slots"], x, case["kind"])
    new = [values_of([p[st["slots"]] for p in parts]).to(act) for parts in st["stored"]]
    return plain_attend(st, q), *new


def run(st):
    if not own:
        return plain(st)
    import binary_rank_gemv_packed_amd as nq
    case = st["case"]
    op, act = case["op"], DT[case["act"]]
    if op == "heads":
        return nq.head_norm(st["q"], st["k"], st["positions"], st["norm"])
    if op == "heads_bwd":
        return nq.head_norm_backward(st["dq"], st["dk"], st["q"], st["k"], st["positions"], st["norm"])
    if op == "kv":
        nq.kv_write(st["k"], st["v"], st["cache"], st["slots"])
        return nq.kv_read(st["cache"], st["context"], act)
    if op == "attend":
        return nq.kv_attention(st["q"], st["cache"], st["table"], st["lengths"], window=case["window"],
                               workspace=st["ws"])
    q = nq.head_norm_write(st["q"], st["k"], st["v"], st["positions"], st["norm"], st["cache"], st["slots"])
    y = nq.kv_attention(q, st["cache"], st["table"], st["lengths"], window=case["window"], workspace=st["ws"])
    return y, *nq.kv_read(st["cache"], st["slots"], act)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    Hkv, D, a = case["Hkv"], case["D"], SIZE[case["act"]]
    if case["op"] in ("heads", "heads_bwd"):
        n, bwd = case["T"] * (case["Hq"] + Hkv) * D, case["op"] == "heads_bwd"
        return {"bytes": n * a * (3 if bwd else 2) + 8 * case["T"] * case["axes"] + 2 * D * 4 * (2 if bwd else 1),
                "flops": n * (18 if bwd else 8)}
    # keys and values of one token as they are held
    slot = 2 * Hkv * {"bf16": 2 * D, "int8": D + 2, "int4": D / 2 + D / 16}[case["kind"]]
    row = 2 * Hkv * D * a
    if case["op"] == "kv":
        T, L = case["T"], case["context"]
        return {"bytes": T * (row + slot) + L * (row + slot) + 8 * (T + L), "flops": 4 * T * Hkv * D + 2 * L * Hkv * D}
    seen = sum(min(n, case["window"] or n) for n in lengths_of(case))
    B, Hq = case["B"], case["Hq"]
    pages = sum(-(-n // case["page"]) for n in lengths_of(case))
    w = {"bytes": seen * slot + 2 * B * Hq * D * a + 4 * (pages + B), "flops": 4 * seen * Hq * D}
    if case["op"] == "step":  # k and v in, the new token's place out, and read back as it is held
        w["bytes"] += B * (2 * row + slot + 16)
        w["flops"] += 8 * B * (Hq + Hkv) * D
    return w


# ------------------------------------------------------------------ the definition in 64 bits
def exact_held(x, kind):
    """The values that the cache holds for x."""
    if kind == "bf16":
        return x.bfloat16().double()
    groups = x.double().reshape(*x.shape[:-1], -1, x.shape[-1] if kind == "int8" else 32)
    top = 127 if kind == "int8" else 7
    step = (torch.linalg.vector_norm(groups, ord=math.inf, dim=-1, keepdim=True) / top).float().bfloat16().double()
    whole = torch.nan_to_num(groups / step, nan=0.0).round().clamp(-top, top)
    return (whole * step).reshape(x.shape)


def exact_turn(case, x, positions, sign=1.0):
    """x (T, H, D) with its pairs turned as complex numbers."""
    rot = case.get("rot", case["D"])
    f = frequencies(rot)
    parts, at = [], 0
    for axis, n in enumerate(sections_of(case) if "axes" in case else [rot // 2]):
        parts.append(positions[axis].double()[:, None] * f[at:at + n])
        at += n
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), sign * torch.cat(parts, 1))[:, None]
    near = case.get("pairs") == "neighbours"
    shape = (*x.shape[:-1], rot // 2, 2) if near else (*x.shape[:-1], 2, rot // 2)
    z = x[..., :rot].reshape(shape)
    z = torch.complex(*(z.unbind(-1) if near else z.unbind(-2))) * turn
    return torch.cat((torch.stack((z.real, z.imag), -1 if near else -2).reshape(*x.shape[:-1], rot), x[..., rot:]), -1)


def exact_norm(x, w):
    return x * w / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)


def exact_attend(case, t, q, keys, values):
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    r, page = case["Hq"] // case["Hkv"], case["page"]
    for b, n in enumerate(lengths_of(case)):
        at = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device="cuda")
        if not len(at):
            continue
        slots = t["table"][b].long()[at // page] * page + at % page
        for h in range(case["Hkv"]):
            k, v = keys(slots, h), values(slots, h)
            p = torch.softmax(k @ q[b, h * r:(h + 1) * r].t() * case["D"] ** -0.5, dim=0)
            out[b, h * r:(h + 1) * r] = p.t() @ v
    return out


def exact(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = inputs(case, g)
    kind = case.get("kind")
    if case["op"] == "kv":
        rows = [t["keys"], t["values"]]
        for old, new in zip(rows, (t["k"], t["v"])):
            old[t["slots"]] = new
        return [exact_held(x[t["context"]], kind) for x in rows]
    if case["op"] in ("heads", "step"):
        q, k = (exact_turn(case, exact_norm(t[n].double(), t["w_" + n].double()), t["positions"]) for n in ("q", "k"))
        if case["op"] == "heads":
            return q, k
        t["keys"][t["slots"]], t["values"][t["slots"]] = k.to(t["k"].dtype), t["v"]
    if case["op"] in ("attend", "step"):
        of = lambda x: lambda slots, h: exact_held(x[slots, h], kind)  # noqa: E731
        y = exact_attend(case, t, t["q"].double() if case["op"] == "attend" else q, of(t["keys"]), of(t["values"]))
        if case["op"] == "attend":
            return y
        return y, *(exact_held(t[n][t["slots"]], kind) for n in ("keys", "values"))
    found = {}
    for n in ("q", "k"):
        x, w = t[n].double().requires_grad_(), t["w_" + n].double().requires_grad_()
        into = exact_turn(case, t["d" + n].double(), t["positions"], -1.0)
        found["d" + n], found["dw_" + n] = torch.autograd.grad(exact_norm(x, w), (x, w), into)
    return {n: found[n] for n in ("dq", "dk", "dw_q", "dw_k")}
