"""Cases of the 4-bit linears and of the block norms: what a decode or training
step of a compressed model calls beside its binary linears.

Operators
  q4          y = x W^T, W[i, j] = s[i, j / G] (q[i, j] - z[i, j / G]): codes of
              4 bits, one scale (and, where "zeros", one zero point, else 8) for
              each row and G consecutive columns.  x is (B, n), W (m, n).
  q4_group    up to three such weights that read the same x (q, k, v; gate, up).
  norm        between two blocks of a transformer: h' = a h + b gate * post(y),
              x = pre(h'), post and pre root-mean-square norms with weights.
  norm_bwd    the gradients of norm: h, y, the norms' weights and the gate.
              The sums over the row that the forward keeps come with the state.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5


def q4(name, m, n, B, G, zeros, scale, x, y, m2=0, m3=0):
    return {"name": name, "op": "q4_group" if m2 else "q4", "m": m, "m2": m2, "m3": m3, "n": n, "B": B, "G": G,
            "zeros": zeros, "scale": scale, "x": x, "y": y}


def norm(name, rows, d, act, res, par, gate, bwd=False):
    return {"name": name, "op": "norm_bwd" if bwd else "norm", "rows": rows, "d": d, "act": act, "res": res,
            "par": par, "gate": gate}


def listed():
    return [
        # the smallest linear: what one call costs
        q4("q4 small", 256, 256, 1, 32, False, "f32", "f32", "f32"),
        # one token through a square attention projection
        q4("q4 attention token", 8192, 8192, 1, 128, False, "f16", "bf16", "bf16"),
        # four sequences decoded together, logits of a 32000 word vocabulary in fp32
        q4("q4 head", 32000, 8192, 4, 128, False, "f16", "bf16", "f32"),
        # sixteen sequences through the projection back from the wide layer
        q4("q4 down batch", 8192, 28672, 16, 128, True, "f16", "bf16", "bf16"),
        # odd sizes: a last group of three columns, a last row tile of twelve rows
        q4("q4 odd", 1100, 4099, 7, 32, True, "f32", "f32", "f32"),
        # a prompt of 2048 tokens
        q4("q4 prompt", 11008, 4096, 2048, 128, False, "f16", "bf16", "bf16"),
        # one token through the two wide linears of a block
        q4("q4 gate and up token", 28672, 8192, 1, 128, True, "f16", "bf16", "bf16", m2=28672),
        # four sequences through q, k and v with shared key heads
        q4("q4 q k v", 8192, 8192, 4, 64, True, "f16", "bf16", "bf16", m2=1024, m3=1024),
        # one token between two blocks
        norm("norm token", 1, 8192, "bf16", "bf16", "bf16", "channel"),
        # a prompt of 2048 tokens, the residual stream held in fp32
        norm("norm prompt", 2048, 8192, "bf16", "f32", "bf16", "none"),
        # gradients of a ragged batch of an odd width, one gate for each token and channel
        norm("norm gradients odd", 333, 1619, "f32", "f32", "f32", "token", bwd=True),
        # gradients of a training step of 4096 tokens
        norm("norm gradients", 4096, 8192, "bf16", "f32", "f32", "channel", bwd=True),
    ]


def draw(rng: random.Random):
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, min(hi, v if rng.random() < 0.5 else (v + 63) // 64 * 64))

    if rng.random() < 0.6:
        m, n, B = size(64, 32000), size(64, 28672), size(1, 2048) if rng.random() < 0.3 else rng.randint(1, 16)
        m2, m3 = (size(64, 8192), rng.choice((0, size(64, 8192)))) if rng.random() < 0.4 else (0, 0)
        while (m + m2 + m3) * n * B > 2 ** 36 or (m + m2 + m3) * n > 2 ** 28:
            m, m2, m3, n, B = max(64, m // 2), m2 // 2, m3 // 2, max(64, n // 2 + 1), max(1, B // 2)
        c = q4("", m, n, B, rng.choice((32, 64, 128)), rng.random() < 0.5, rng.choice(("f16", "f32")),
               rng.choice(("bf16", "bf16", "f32")), rng.choice(("bf16", "bf16", "f32")), m2, m3)
    else:
        rows, d = size(1, 16384), size(64, 16384)
        while rows * d > 2 ** 24:
            rows = max(1, rows // 2)
        act = rng.choice(("bf16", "bf16", "f32"))
        c = norm("", rows, d, act, rng.choice((act, "f32")), rng.choice(("f32", "bf16", "f16")),
                 rng.choice(("none", "channel", "token")), rng.random() < 0.5)
    del c["name"]
    return c


def heights(case):
    return [m for m in (case["m"], case["m2"], case["m3"]) if m]


# ------------------------------------------------------------------ inputs
def q4_inputs(case, g):
    n, G = case["n"], case["G"]
    ng = (n + G - 1) // G
    weights = []
    for m in heights(case):
        # codes of a normal weight: bell-shaped about the middle
        q = (torch.randn(m, n, generator=g, device="cuda") * 2.6 + 8).round_().clamp_(0, 15).to(torch.uint8)
        s = ((torch.rand(m, ng, generator=g, device="cuda") + 0.3) * (0.4 / math.sqrt(n))).to(DT[case["scale"]])
        z = torch.randint(4, 13, (m, ng), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
        weights.append((q, s, z))
    x = torch.randn(case["B"], n, generator=g, device="cuda")
    # activations have a few channels that are much larger than the others
    x *= torch.where(torch.rand(n, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return weights, x.to(DT[case["x"]])


def norm_inputs(case, g):
    rows, d = case["rows"], case["d"]
    act, res, par = DT[case["act"]], DT[case["res"]], DT[case["par"]]
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    t = {"h": (rand(rows, d) * 2).to(res), "y": (rand(rows, d) * (0.2 + rand(rows, 1).abs())).to(act),
         "w_post": (1 + 0.2 * rand(d)).to(par), "w_pre": (1 + 0.2 * rand(d)).to(par), "gate": None}
    if case["gate"] == "channel":
        t["gate"] = (0.5 * rand(d)).to(par)
    if case["gate"] == "token":
        t["gate"] = torch.sigmoid(rand(rows, d)).to(act)
    if case["op"] == "norm_bwd":
        t["dx"], t["dh"] = rand(rows, d).to(act), (0.5 * rand(rows, d)).to(res)
        # h stands for the stream behind the block here; its kept sums belong to it
        t["stats"] = torch.stack([(t[k].double().square().mean(1) + EPS).rsqrt().float() for k in ("y", "h")])
    return t


A, BS = 0.9, 0.7  # residual scale and block scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}
    if case["op"] in ("q4", "q4_group"):
        state["weights"], state["x"] = q4_inputs(case, g)
        if own:  # the packed weights, workspace and outputs that a program keeps
            import binary_rank_gemv_packed_amd as nq
            layers = [nq.q4_pack(q, s, z, group=case["G"]) for q, s, z in state.pop("weights")]
            state["y"] = [torch.empty(case["B"], L.m, dtype=DT[case["y"]], device="cuda") for L in layers]
            state["layer"] = layers[0] if case["op"] == "q4" else nq.Q4Group(layers)
            state["ws"] = nq.new_q4_workspace(state["layer"], case["B"])
    else:
        state.update(norm_inputs(case, g))
        if own:
            import binary_rank_gemv_packed_amd as nq
            state["norm"] = nq.BlockNorm(case["d"], act_dtype=DT[case["act"]], res_dtype=DT[case["res"]],
                                         w_post=state["w_post"], w_pre=state["w_pre"],
                                         gate=state["gate"] if case["gate"] == "channel" else None,
                                         res_scale=A, block_scale=BS, eps=EPS)
            state["row_gate"] = state["gate"] if case["gate"] == "token" else None
    return state


# ------------------------------------------------------------------ one pass
def plain_q4(x, weights, G, dtype):
    out = []
    for q, s, z in weights:
        n = q.shape[1]
        wide = lambda v: v.float().repeat_interleave(G, dim=1)[:, :n]  # noqa: E731
        w = (q.float() - (8.0 if z is None else wide(z))) * wide(s)
        out.append((x.float() @ w.t()).to(dtype))
    return out


def plain_norm(st):
    y, h = st["y"].float(), st["h"].float()
    u = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) * st["w_post"].float()
    if st["gate"] is not None:
        u = u * st["gate"].float()
    out = A * h + BS * u
    x = out * torch.rsqrt(out.square().mean(1, keepdim=True) + EPS) * st["w_pre"].float()
    return out.to(st["h"].dtype), x.to(st["y"].dtype)


def plain_norm_bwd(st):
    y, h, dx = st["y"].float(), st["h"].float(), st["dx"].float()
    ry, rh = st["stats"][0][:, None], st["stats"][1][:, None]
    hhat, yhat, w_post = h * rh, y * ry, st["w_post"].float()
    t = dx * st["w_pre"].float()
    g = st["dh"].float() + rh * (t - hhat * (t * hhat).mean(1, keepdim=True))
    v = BS * g
    out = {"dh": (A * g).to(st["h"].dtype), "dw_pre": (dx * hhat).sum(0)}
    if st["gate"] is not None:
        dgate = v * yhat * w_post
        out["dgate"] = dgate.sum(0) if st["gate"].dim() == 1 else dgate.to(st["gate"].dtype)
        v = v * st["gate"].float()
    out["dw_post"] = (v * yhat).sum(0)
    t = v * w_post
    out["dy"] = (ry * (t - yhat * (t * yhat).mean(1, keepdim=True))).to(st["y"].dtype)
    return out


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op in ("q4", "q4_group"):
            return plain_q4(state["x"], state["weights"], case["G"], DT[case["y"]])
        return plain_norm(state) if op == "norm" else plain_norm_bwd(state)
    import binary_rank_gemv_packed_amd as nq
    if op == "q4":
        return [nq.q4_linear_into(state["x"], state["layer"], state["y"][0], state["ws"])]
    if op == "q4_group":
        return nq.q4_linear_group_into(state["x"], state["layer"], state["y"], state["ws"])
    if op == "norm":
        return nq.block_norm(state["h"], state["y"], state["norm"], gate=state["row_gate"])
    return nq.block_norm_backward(state["dx"], state["dh"], state["h"], state["y"], state["stats"], state["norm"],
                                  gate=state["row_gate"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] in ("q4", "q4_group"):
        n, B, M = case["n"], case["B"], sum(heights(case))
        groups = M * ((n + case["G"] - 1) // case["G"])
        return {"bytes": M * n / 2 + groups * (SIZE[case["scale"]] + (0.5 if case["zeros"] else 0))
                + B * n * SIZE[case["x"]] + B * M * SIZE[case["y"]],
                "flops": 2 * B * M * n}
    rows, d = case["rows"], case["d"]
    a, r, p = SIZE[case["act"]], SIZE[case["res"]], SIZE[case["par"]]
    params = 2 + (case["gate"] == "channel")
    token = case["gate"] == "token"
    if case["op"] == "norm":  # h, y in; h', x out
        return {"bytes": rows * d * (2 * r + 2 * a + token * a) + params * d * p, "flops": 10 * rows * d}
    # dx, dh', h', y in; dh, dy out; the weights' gradients in fp32
    return {"bytes": rows * d * (3 * r + 3 * a + 2 * token * a) + 8 * rows + params * d * (p + 4),
            "flops": 24 * rows * d}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] in ("q4", "q4_group"):
        weights, x = q4_inputs(case, g)
        column_group = torch.arange(case["n"], device="cuda") // case["G"]
        out = []
        for q, s, z in weights:
            rows = []
            for lo in range(0, q.shape[0], 4096):  # in pieces of rows: the whole weight in 64 bits is large
                part = slice(lo, lo + 4096)
                step = s[part].double()[:, column_group]
                off = step * 8 if z is None else step * z[part].double()[:, column_group]
                rows.append(torch.addcmul(-off, q[part].double(), step).matmul(x.double().t()))
            out.append(torch.cat(rows).t().contiguous())
        return out
    t = {k: v.double() for k, v in norm_inputs(case, g).items() if v is not None and k != "stats"}
    length = math.sqrt(case["d"])

    def rms(v, w):  # v over its root mean square, times w
        return v / torch.sqrt((torch.linalg.vector_norm(v, dim=1, keepdim=True) / length) ** 2 + EPS) * w

    def branch(y, w, gate):
        return BS * rms(y, w) if gate is None else BS * gate * rms(y, w)

    if case["op"] == "norm":
        out = A * t["h"] + branch(t["y"], t["w_post"], t.get("gate"))
        return out, rms(out, t["w_pre"])
    leaf = {k: t[k].requires_grad_() for k in ("h", "y", "w_post", "w_pre", "gate") if k in t}
    rms(leaf["h"], leaf["w_pre"]).backward(t["dx"])
    into = leaf["h"].grad + t["dh"]
    branch(leaf["y"], leaf["w_post"], leaf.get("gate")).backward(into)
    found = {"dh": A * into, "dw_pre": leaf["w_pre"].grad}
    if "gate" in leaf:
        found["dgate"] = leaf["gate"].grad
    found["dw_post"], found["dy"] = leaf["w_post"].grad, leaf["y"].grad
    return found
