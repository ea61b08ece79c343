"""Cases of the decode and 8-bit operators: products in 8-bit integers with scales
for each token and channel, the dense gated block in that arithmetic, and the
whole MoE layer for a few tokens.

``run`` computes a case either in its plain form (elementary torch operations in
32 bits, router scores and the quantisation's borders in 64, rounded once to the
output's type) or, with ``own`` set, through the library's entry points. ``exact``
gives the same outputs in 64 bits.

A row x is quantised to codes q = rint(x / s), ties to even, with s = max |x| / 127
rounded to 32 bits (codes 0 where s is 0); a weight is held as codes [K][N] and one
scale per column. The scale's rounding belongs to the definition: values in 16 bits
often lie on a border between two codes but for it.

Operators, by the case's ``op``:

mm    y = q(x) . W: sums of products of codes, times the row's and the column's scale
ffn   o = q(h) . Wd with h = silu(q(x) . Wu) * (q(x) . Wg) in 32 bits
few   o_t = sum_j w_tj FFN_{id_tj}(x_t) (+ a shared expert), ids and w the softmax
      top-k of x Wr (+ bias), or given (an id below zero is a slot without an
      expert); ids and w are returned where they are computed. Weights in bf16, fp32
      or as codes ("i8": both products of an expert as in ffn)
"""
import math

import torch

own = False

DEV = "cuda"
MATRICES = ("up", "gate", "down", "s_up", "s_gate", "s_down")


def listed():
    return [
        # one new token through one projection: latency counts
        {"name": "mm_1", "op": "mm", "S": 1, "K": 7168, "N": 2048, "dtype": "bf16"},
        # a small decode batch, sizes off every tile
        {"name": "mm_13_odd", "op": "mm", "S": 13, "K": 2064, "N": 5128, "dtype": "bf16"},
        # a ragged prompt in single precision
        {"name": "mm_1001_f32", "op": "mm", "S": 1001, "K": 2048, "N": 776, "dtype": "f32"},
        # a prefill's projection from the widest hidden size
        {"name": "mm_prefill", "op": "mm", "S": 16384, "K": 7168, "N": 2048, "dtype": "bf16"},
        # decode: 64 new tokens through a block of the shared expert's sizes
        {"name": "ffn_decode", "op": "ffn", "S": 64, "H": 7168, "D": 2048},
        # a ragged prompt
        {"name": "ffn_1001", "op": "ffn", "S": 1001, "H": 2048, "D": 784},
        # a prefill
        {"name": "ffn_prefill", "op": "ffn", "S": 16384, "H": 2048, "D": 2048},
        # the smallest layer in single precision
        {"name": "few_tiny_f32", "op": "few", "S": 64, "H": 128, "D": 256, "E": 8, "k": 2,
         "D_shared": 0, "dtype": "f32", "routed": True, "bias": False, "padded": 0},
        # one new token through the decode layer: latency counts
        {"name": "few_1", "op": "few", "S": 1, "H": 2048, "D": 768, "E": 256, "k": 8,
         "D_shared": 0, "dtype": "bf16", "routed": True, "bias": False, "padded": 0},
        # one new token through the widest layer
        {"name": "few_1_wide", "op": "few", "S": 1, "H": 7168, "D": 2048, "E": 256, "k": 8,
         "D_shared": 2048, "dtype": "bf16", "routed": True, "bias": True, "padded": 0},
        # the decode layer, a full batch
        {"name": "few_64", "op": "few", "S": 64, "H": 2048, "D": 768, "E": 256, "k": 8,
         "D_shared": 0, "dtype": "bf16", "routed": True, "bias": False, "padded": 0},
        # a batch of 13 tokens with 8-bit experts, 2 of them padding, routed elsewhere
        {"name": "few_13_i8", "op": "few", "S": 13, "H": 2048, "D": 768, "E": 256, "k": 8,
         "D_shared": 768, "dtype": "i8", "routed": False, "bias": False, "padded": 2},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, m, lo, hi):
    return max(m, _log(rng, lo, hi) // m * m)


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 300)


def draw(rng):
    op = rng.choice(["mm", "ffn", "few", "few"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        if op == "mm":
            case = {"op": op, "S": _log(rng, 1, 16384), "K": _mult(rng, 16, 128, 8192),
                    "N": _mult(rng, 8, 128, 16384), "dtype": rng.choice(["bf16", "bf16", "f32"])}
            if _cost(case) <= most and case["K"] * case["N"] >= 1 << 18:
                return case
        elif op == "ffn":
            case = {"op": op, "S": _log(rng, 1, 16384), "H": _mult(rng, 16, 128, 7168),
                    "D": _mult(rng, 16, 128, 7168)}
            if _cost(case) <= most and case["H"] * case["D"] >= 1 << 17:
                return case
        else:
            dtype = rng.choice(["bf16", "bf16", "i8", "f32"])
            m = 16 if dtype == "i8" else 8
            case = {"op": op, "S": _log(rng, 1, 64), "H": _mult(rng, m, 128, 4096),
                    "D": _mult(rng, m, 128, 2048), "E": rng.choice([4, 6, 8, 25, 64, 100, 128, 256]),
                    "k": rng.choice([1, 2, 3, 4, 8]), "D_shared": 0, "dtype": dtype,
                    "routed": rng.random() < 0.7, "bias": False, "padded": 0}
            if rng.random() < 0.4:
                case["D_shared"] = _mult(rng, m, 128, 1024)
            if case["routed"]:
                case["bias"] = rng.random() < 0.4
            else:
                case["padded"] = rng.randrange(0, (case["S"] + 3) // 4)
            size = case["E"] * case["H"] * case["D"]
            if case["k"] <= case["E"] and 1 << 18 <= size <= 1 << 29 and _cost(case) <= most / 2:
                return case


# ------------------------------------------------------------------ inputs

def _dt(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _normal(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _codes(x, s):
    """Codes (int8) of a float tensor with scales s."""
    q = torch.round(x.double() / s.double())
    return torch.where(s > 0, q, 0.0).clamp(-127, 127).to(torch.int8)


def _quant(x, dim):
    """Codes and scales of a float tensor, one scale per vector along dim. The quotient in 64
    bits, rounded once: a device tensor over a number is a product with the number's
    reciprocal, in 32 bits an ulp off in 3 to 6% of the vectors."""
    s = (x.abs().amax(dim, keepdim=True).double() / 127).float()
    return _codes(x, s), s


def _w8(gen, E, K, N):
    """Codes [E][K][N] and scales [E][N] of normal weights of std 1 / sqrt(K)."""
    q = torch.empty((E, K, N), dtype=torch.int8, device=DEV)
    s = torch.empty((E, N), device=DEV)
    for e in range(E):
        w = _normal(gen, (K, N), 1 / math.sqrt(K), torch.bfloat16)
        s[e] = w.float().abs().amax(0) / 127.0  # an input: whatever scales the user has
        q[e] = _codes(w, s[e])
    return q, s


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    t = {}
    if case["op"] == "mm":
        S, K, N = case["S"], case["K"], case["N"]
        t["x"] = _normal(gen, (S, K), 1.0, _dt(case))
        # activations of a residual stream: a few columns are larger
        t["x"][:, torch.randint(0, K, (1 + K // 512,), generator=gen, device=DEV)] *= 4.0
        t["w"] = _w8(gen, 1, K, N)
        return t
    if case["op"] == "ffn":
        S, H, D = case["S"], case["H"], case["D"]
        t["x"] = _normal(gen, (S, H), 1.0, torch.bfloat16)
        t["up"], t["gate"], t["down"] = _w8(gen, 1, H, D), _w8(gen, 1, H, D), _w8(gen, 1, D, H)
        return t
    S, H, D, E, k, Ds = (case[n] for n in ("S", "H", "D", "E", "k", "D_shared"))
    dt = _dt(case)

    def weight(E, K, N):
        if case["dtype"] == "i8":
            return _w8(gen, E, K, N)
        return _normal(gen, (E, K, N), 1 / math.sqrt(K), dt)

    t["x"] = _normal(gen, (S, H), 1.0, dt)
    t["up"], t["gate"], t["down"] = weight(E, H, D), weight(E, H, D), weight(E, D, H)
    if Ds:
        t["s_up"], t["s_gate"], t["s_down"] = weight(1, H, Ds), weight(1, H, Ds), weight(1, Ds, H)
    if case["routed"]:
        t["wr"] = _normal(gen, (H, E), 1 / math.sqrt(H), dt)
        if case["bias"]:
            t["bias"] = torch.randn(E, generator=gen, device=DEV) * 0.3
    else:
        score, ids = torch.randn((S, E), generator=gen, device=DEV).topk(k, dim=1)
        ids, w = ids.to(torch.int32), score.softmax(dim=1)
        if case["padded"]:
            ids[S - case["padded"]:] = -1
            w[S - case["padded"]:] = 0.0
        t["ids"], t["w"] = ids.contiguous(), w.contiguous()
    return t


def prepare(case, seed):
    t = _inputs(case, seed)
    st = {"case": case, "t": t}
    if own:
        import sparse_expert_ffn_amd as moe
        from sparse_expert_ffn_amd import layer
        if case["op"] == "mm":
            st["w"] = layer.I8Weight(*t["w"])
            st["buf"] = layer.I8LinearBuffers(case["S"], case["K"], case["N"],
                                              dtype=moe.MOE_F32 if case["dtype"] == "f32"
                                              else moe.MOE_BF16, device=DEV)
        elif case["op"] == "ffn":
            st["wt"] = [layer.I8Weight(*t[n]) for n in MATRICES[:3]]
            st["buf"] = layer.I8FFNBuffers(case["S"], case["H"], case["D"], device=DEV)
        else:
            i8 = case["dtype"] == "i8"
            mat = lambda n: layer.I8Weight(*t[n]) if i8 else t[n] if n[0] != "s" else t[n][0]
            st["wt"] = [mat(n) if n in t else None for n in MATRICES]
            st["buf"] = layer.FewMoEBuffers(
                case["S"], case["H"], case["D"], case["E"], case["k"], D_shared=case["D_shared"],
                dtype=moe.MOE_F32 if case["dtype"] == "f32" else moe.MOE_BF16, i8=i8, device=DEV)
    return st


# ------------------------------------------------------------------ one pass

def _run_own(st):
    case, t, b = st["case"], st["t"], st["buf"]
    if case["op"] == "mm":
        return b.run(t["x"], st["w"])
    if case["op"] == "ffn":
        return b.forward(t["x"], *st["wt"])
    if not case["routed"]:
        return b.forward(t["x"], *st["wt"], topk_ids=t["ids"], topk_weights=t["w"])
    o = b.run(t["x"], t["wr"], *st["wt"], router_bias=t.get("bias"))
    return o, b.topk_ids, b.topk_weights


def _mm8(x, w, e=0):
    """x [..][n][K] quantised per row, times the weight's matrices e."""
    q, s = _quant(x, -1)
    return (q.float() @ w[0][e].float()) * s * w[1][e].unsqueeze(-2)


def _gated(x, up, gate, down, e, i8):
    """x [..][n][K] through the experts e (one, or one for each of a batch)."""
    mm = _mm8 if i8 else lambda x, w, e: x @ w[e].float()
    u = mm(x, up, e)
    return mm(u / (1.0 + torch.exp(-u)) * mm(x, gate, e), down, e)


def run(state):
    if own:
        return _run_own(state)
    case, t = state["case"], state["t"]
    if case["op"] == "mm":
        return _mm8(t["x"].float(), t["w"]).to(_dt(case))
    if case["op"] == "ffn":
        return _gated(t["x"].float(), t["up"], t["gate"], t["down"], 0, True).to(torch.bfloat16)
    S, H, E, k = (case[n] for n in ("S", "H", "E", "k"))
    i8 = case["dtype"] == "i8"
    x = t["x"].float()
    if case["routed"]:
        score = (t["x"].double() @ t["wr"].double()).float()
        if case["bias"]:
            score = score + t["bias"]
        # equal scores: the lower index first
        top, ids = (v[:, :k] for v in torch.sort(score, dim=1, descending=True, stable=True))
        ex = torch.exp(top.double() - top[:, :1].double())
        w = (ex / ex.sum(1, keepdim=True)).float()
    else:
        ids, w = t["ids"].long(), torch.where(t["ids"] >= 0, t["w"], 0.0)
    if S * k < E:  # fewer choices than experts: the chosen matrices, one after another
        at = ids.clamp(min=0).reshape(-1)
        y = _gated(x.repeat_interleave(k, dim=0)[:, None], t["up"], t["gate"], t["down"], at, i8)
        o = (y.view(S, k, H) * w[:, :, None]).sum(1)
    else:  # every expert on every token, weighted by the choices
        at = torch.arange(E, device=DEV)
        y = _gated(x.expand(E, S, H), t["up"], t["gate"], t["down"], at, i8)
        m = ((ids[:, :, None] == at) * w[:, :, None]).sum(1)
        o = (y * m.t()[:, :, None]).sum(0)
    if case["D_shared"]:
        o = o + _gated(x, t["s_up"], t["s_gate"], t["s_down"], 0, i8)
    o = o.to(_dt(case))
    return (o, ids.to(torch.int32), w) if case["routed"] else o


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    es = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "mm":
        S, K, N = case["S"], case["K"], case["N"]
        return {"bytes": K * N + 4 * N + es * S * (K + N), "flops": 2 * S * K * N}
    if case["op"] == "ffn":
        S, H, D = case["S"], case["H"], case["D"]
        return {"bytes": 3 * H * D + 4 * (2 * D + H) + 4 * S * H, "flops": 6 * S * H * D}
    S, H, D, E, k, Ds = (case[n] for n in ("S", "H", "D", "E", "k", "D_shared"))
    live = S - case["padded"]
    # experts that at least one of the live tokens chooses, k of E each, as expected at random
    used = E * (1.0 - (1.0 - k / E) ** live)
    ws = 1 if case["dtype"] == "i8" else es
    router = H * E if case["routed"] else 0
    return {"bytes": int(3 * H * (used * D + Ds) * ws) + es * (router + 2 * S * H) + 8 * S * k,
            "flops": 6 * H * (live * k * D + S * Ds) + 2 * S * router}


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _mm64(a, b):
    return torch.mm(a.to(torch.float64), b.to(torch.float64))


def _product64(x, w, e):
    """Row by row x = codes * scale, the scale held in 32 bits; column by column the weight."""
    x = x.to(torch.float64)
    scale = (x.abs().max(dim=1).values / 127).to(torch.float32).to(torch.float64)
    codes = torch.where(scale[:, None] > 0, x / scale[:, None], 0.0).round()
    return torch.einsum("sn,s,n->sn", _mm64(codes, w[0][e]), scale, w[1][e].double())


def _ffn64(x, up, gate, down, e, i8):
    mm = (lambda a, w: _product64(a, w, e)) if i8 else (lambda a, w: _mm64(a, w[e]))
    u = mm(x, up)
    return mm(u * torch.special.expit(u) * mm(x, gate), down)


def exact(case, seed):
    t = _inputs(case, seed)
    if case["op"] == "mm":
        return torch.cat([_product64(x, t["w"], 0) for x in t["x"].split(4096)])
    if case["op"] == "ffn":
        return torch.cat([_ffn64(x, t["up"], t["gate"], t["down"], 0, True)
                          for x in t["x"].split(4096)])
    i8, k = case["dtype"] == "i8", case["k"]
    x = t["x"]
    if case["routed"]:
        score = _mm64(x, t["wr"])
        if case["bias"]:
            score += t["bias"].double()
        ids = torch.argsort(score, dim=1, descending=True)[:, :k]
        w = torch.softmax(torch.gather(score, 1, ids), dim=1)
    else:
        ids, w = t["ids"], t["w"].double()
    o = torch.zeros((case["S"], case["H"]), dtype=torch.float64, device=DEV)
    chosen = ids.cpu()
    for e in sorted(set(chosen[chosen >= 0].tolist())):  # expert by expert
        s, j = (chosen == e).nonzero(as_tuple=True)
        s, j = s.to(DEV), j.to(DEV)
        y = _ffn64(x[s], t["up"], t["gate"], t["down"], e, i8)
        o.index_add_(0, s, y * w[s, j][:, None])
    if case["D_shared"]:
        o += _ffn64(x, t["s_up"], t["s_gate"], t["s_down"], 0, i8)
    return (o, ids.to(torch.int32), w) if case["routed"] else o
