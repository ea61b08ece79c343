"""Cases of the operators around the MoE layer: layer norm, the dense gated
feed-forward block (training and inference) and the 4-bit products of decode.

``run`` computes a case either in its plain form (elementary torch operations
in 32 bits, rounded once to the output's type) or, with ``own`` set, through
the library's entry points. ``exact`` gives the same outputs in 64 bits.

Operators, by the case's ``op``:

ln_fwd   y = (x - mean) * rstd * gamma + beta per row, mean and rstd kept
ln_bwd   dx, dgamma, dbeta from dy and the kept mean and rstd
ffn_fwd  u = x Wu, g = x Wg, o = (silu(u) * g) Wd; u and g returned too when
         they are kept for a backward pass
ffn_bwd  dx, dWu, dWg, dWd from do and the kept u and g
matvec   y = x W, W held as 4-bit codes with one scale per group of rows
w4_moe   the MoE layer's experts with 4-bit weights on routed tokens:
         o_t = sum_j w_tj FFN_{e_tj}(x_t) (+ a shared expert); an id below
         zero is a slot without an expert (a padded token has none at all)
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # a prefill's norm before the widest layer
        {"name": "ln_fwd_prefill", "op": "ln_fwd", "S": 16384, "H": 7168, "dtype": "bf16"},
        # the same in training
        {"name": "ln_bwd_prefill", "op": "ln_bwd", "S": 16384, "H": 2048, "dtype": "bf16"},
        # a ragged batch, rows of odd length that no vector load is aligned to
        {"name": "ln_bwd_odd_f32", "op": "ln_bwd", "S": 4099, "H": 1001, "dtype": "f32"},
        # the smallest layer: latency counts
        {"name": "ffn_fwd_tiny_f32", "op": "ffn_fwd", "S": 64, "H": 128, "D": 256, "dtype": "f32",
         "keep": False},
        # decode: 64 new tokens through a block of the shared expert's sizes, bound by its weights
        {"name": "ffn_fwd_decode", "op": "ffn_fwd", "S": 64, "H": 7168, "D": 2048,
         "dtype": "bf16", "keep": False},
        # training's forward pass at the prefill sizes
        {"name": "ffn_fwd_prefill", "op": "ffn_fwd", "S": 16384, "H": 2048, "D": 2048,
         "dtype": "bf16", "keep": True},
        # and its backward pass
        {"name": "ffn_bwd_prefill", "op": "ffn_bwd", "S": 16384, "H": 2048, "D": 2048,
         "dtype": "bf16"},
        # a ragged batch in single precision
        {"name": "ffn_bwd_odd_f32", "op": "ffn_bwd", "S": 1001, "H": 2048, "D": 768,
         "dtype": "f32"},
        # one new token through one projection
        {"name": "matvec_1", "op": "matvec", "S": 1, "K": 7168, "N": 2048, "group": 128},
        # a small batch, sizes off every tile, small groups
        {"name": "matvec_13_odd", "op": "matvec", "S": 13, "K": 2056, "N": 5128, "group": 32},
        # one new token through the widest layer
        {"name": "w4_moe_1", "op": "w4_moe", "S": 1, "H": 7168, "D": 2048, "E": 256, "k": 8,
         "D_shared": 2048, "group": 128, "padded": 0},
        # the decode layer, a batch with 3 padded tokens
        {"name": "w4_moe_64", "op": "w4_moe", "S": 64, "H": 2048, "D": 768, "E": 256, "k": 8,
         "D_shared": 0, "group": 64, "padded": 3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult8(rng, lo, hi):
    return max(8, _log(rng, lo, hi) // 8 * 8)


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "ffn_fwd", "ffn_bwd", "matvec", "w4_moe"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    es = 4 if dtype == "f32" else 2
    while True:
        if op in ("ln_fwd", "ln_bwd"):
            case = {"op": op, "S": _log(rng, 1, 32768), "H": _log(rng, 8, 16384), "dtype": dtype}
            if case["S"] * case["H"] * es <= 16384 * 2048 * 2 and case["S"] * case["H"] >= 4096:
                return case
        elif op in ("ffn_fwd", "ffn_bwd"):
            case = {"op": op, "S": _log(rng, 1, 16384), "H": _mult8(rng, 64, 7168),
                    "D": _mult8(rng, 64, 7168), "dtype": dtype}
            if op == "ffn_fwd":
                case["keep"] = rng.random() < 0.5
            n = case["S"] * case["H"] * case["D"]
            if n * (16 if dtype == "f32" else 1) <= 16384 * 2048 * 2048 and n >= 1 << 20:
                return case
        elif op == "matvec":
            case = {"op": op, "S": _log(rng, 1, 32), "K": _mult8(rng, 128, 8192),
                    "N": _mult8(rng, 128, 16384), "group": rng.choice([32, 64, 128])}
            if 1 << 18 <= case["K"] * case["N"] <= 1 << 25:
                return case
        else:
            case = {"op": op, "S": _log(rng, 1, 64), "H": _mult8(rng, 128, 4096),
                    "D": _mult8(rng, 128, 2048), "E": rng.choice([4, 8, 24, 64, 128]),
                    "k": rng.choice([1, 2, 3, 4]), "D_shared": 0,
                    "group": rng.choice([32, 64, 128]), "padded": 0}
            if rng.random() < 0.4:
                case["D_shared"] = _mult8(rng, 128, 1024)
            case["padded"] = rng.randrange(0, (case["S"] + 3) // 4)
            if case["S"] * case["k"] * case["H"] * case["D"] <= 64 * 8 * 2048 * 768 // 2 \
                    and case["H"] * case["D"] >= 1 << 16:
                return case


# ------------------------------------------------------------------ inputs

def _dt(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _normal(gen, shape, std, dtype, mean=0.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std + mean).to(dtype)


def _codes(gen, shape):
    """4-bit codes 0..15 (value: code - 8), small values more often than large."""
    r = torch.randint(0, 128, shape, generator=gen, device=DEV, dtype=torch.uint8)
    c = r & 7
    c += (r >> 3) & 7
    c += r >> 6
    return c


def _w4(gen, E, K, N, group):
    """Codes [E][K][N] and scales [E][ceil(K / group)][N] of weights of std 1 / sqrt(K)."""
    s = torch.rand((E, -(-K // group), N), generator=gen, device=DEV) + 0.5
    return _codes(gen, (E, K, N)), (s * (1.0 / (3.3 * math.sqrt(K)))).to(torch.bfloat16)


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    t = {}
    if op in ("ln_fwd", "ln_bwd"):
        S, H, dt = case["S"], case["H"], _dt(case)
        # activations of a residual stream: columns with offsets, a few of them large
        off = torch.randn(H, generator=gen, device=DEV) * 0.5
        off[torch.randint(0, H, (1 + H // 512,), generator=gen, device=DEV)] += 8.0
        x = torch.randn((S, H), generator=gen, device=DEV)
        t["x"] = x.add_(off).to(dt)
        t["gamma"] = _normal(gen, (H,), 0.1, dt, 1.0)
        t["beta"] = _normal(gen, (H,), 0.1, dt)
        if op == "ln_bwd":
            t["dy"] = _normal(gen, (S, H), 0.02, dt)
            x64 = t["x"].double()
            mean = x64.mean(1)
            var = (x64 - mean[:, None]).square_().mean(1)
            t["mean"], t["rstd"] = mean.float(), (var + 1e-5).rsqrt().float()
    elif op in ("ffn_fwd", "ffn_bwd"):
        S, H, D, dt = case["S"], case["H"], case["D"], _dt(case)
        t["x"] = _normal(gen, (S, H), 1.0, dt)
        t["wu"] = _normal(gen, (H, D), 1 / math.sqrt(H), dt)
        t["wg"] = _normal(gen, (H, D), 1 / math.sqrt(H), dt)
        t["wd"] = _normal(gen, (D, H), 1 / math.sqrt(D), dt)
        if op == "ffn_bwd":
            t["do"] = _normal(gen, (S, H), 0.02, dt)
            t["u"] = (t["x"].float() @ t["wu"].float()).to(dt)
            t["g"] = (t["x"].float() @ t["wg"].float()).to(dt)
    elif op == "matvec":
        t["x"] = _normal(gen, (case["S"], case["K"]), 1.0, torch.bfloat16)
        t["w"] = _w4(gen, 1, case["K"], case["N"], case["group"])
    else:
        S, H, D, E, k = (case[n] for n in ("S", "H", "D", "E", "k"))
        t["x"] = _normal(gen, (S, H), 1.0, torch.bfloat16)
        t["up"], t["gate"] = (_w4(gen, E, H, D, case["group"]) for _ in range(2))
        t["down"] = _w4(gen, E, D, H, case["group"])
        if case["D_shared"]:
            Ds = case["D_shared"]
            t["s_up"], t["s_gate"] = (_w4(gen, 1, H, Ds, case["group"]) for _ in range(2))
            t["s_down"] = _w4(gen, 1, Ds, H, case["group"])
        score, ids = torch.randn((S, E), generator=gen, device=DEV).topk(k, dim=1)
        ids = ids.to(torch.int32)
        w = score.softmax(dim=1)
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
        op = case["op"]
        dtype = moe.MOE_F32 if case.get("dtype") == "f32" else moe.MOE_BF16
        if op in ("ln_fwd", "ln_bwd"):
            st["buf"] = layer.LayerNormBuffers(case["S"], case["H"], dtype=dtype, device=DEV)
        elif op in ("ffn_fwd", "ffn_bwd"):
            st["buf"] = layer.FFNBuffers(case["S"], case["H"], case["D"], dtype=dtype,
                                         keep=case.get("keep", True), train=op == "ffn_bwd",
                                         device=DEV)
        elif op == "matvec":
            st["w"] = layer.W4Weight(*t["w"], group=case["group"])
            st["y"] = torch.empty((case["S"], case["N"]), dtype=torch.bfloat16, device=DEV)
        else:
            pack = lambda n: layer.W4Weight(*t[n], group=case["group"]) if n in t else None
            st["buf"] = layer.W4MoEBuffers(case["S"], case["H"], case["D"], case["E"], case["k"],
                                           D_shared=case["D_shared"], group=case["group"],
                                           device=DEV)
            st["wt"] = [pack(n) for n in ("up", "gate", "down", "s_up", "s_gate", "s_down")]
    return st


# ------------------------------------------------------------------ one pass

def _run_own(st):
    import sparse_expert_ffn_amd as moe
    case, t = st["case"], st["t"]
    op = case["op"]
    if op == "ln_fwd":
        b = st["buf"]
        return b.forward(t["x"], t["gamma"], t["beta"], eps=1e-5), b.mean, b.rstd
    if op == "ln_bwd":
        return st["buf"].backward(t["dy"], t["x"], t["gamma"], t["mean"], t["rstd"])
    if op == "ffn_fwd":
        b = st["buf"]
        o = b.forward(t["x"], t["wu"], t["wg"], t["wd"])
        return (o, b.U, b.G) if case["keep"] else o
    if op == "ffn_bwd":
        return st["buf"].backward(t["do"], t["x"], t["wu"], t["wg"], t["wd"], t["u"], t["g"])
    if op == "matvec":
        moe.moe_w4_matvec(t["x"], st["w"], st["y"])
        return st["y"]
    return st["buf"].forward(t["x"], *st["wt"], topk_ids=t["ids"], topk_weights=t["w"])


def _dequant(codes, scales, group, K):
    w = codes.float().sub_(8.0)
    if K % group == 0:
        *b, _, N = w.shape
        return w.view(*b, K // group, group, N).mul_(scales.float().unsqueeze(-2)).view(*b, K, N)
    return w.mul_(scales.float().repeat_interleave(group, dim=-2)[..., :K, :])


def _gated(x, wu, wg, wd):
    """x [..][n][K] through one expert's matrices (or a batch of them), all float32."""
    u = x @ wu
    return (u / (1.0 + torch.exp(-u)) * (x @ wg)) @ wd


def run(state):
    if own:
        return _run_own(state)
    case, t = state["case"], state["t"]
    op = case["op"]
    if op == "ln_fwd":
        x = t["x"].float()
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = torch.rsqrt((xc * xc).mean(1, keepdim=True) + 1e-5)
        y = xc * rstd * t["gamma"].float() + t["beta"].float()
        return y.to(t["x"].dtype), mean[:, 0], rstd[:, 0]
    if op == "ln_bwd":
        xh = (t["x"].float() - t["mean"][:, None]) * t["rstd"][:, None]
        dy = t["dy"].float()
        d = dy * t["gamma"].float()
        dx = (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True)) \
            * t["rstd"][:, None]
        return dx.to(t["x"].dtype), (dy * xh).sum(0), dy.sum(0)
    if op == "ffn_fwd":
        dt = t["x"].dtype
        x = t["x"].float()
        u = x @ t["wu"].float()
        g = x @ t["wg"].float()
        o = ((u / (1.0 + torch.exp(-u)) * g) @ t["wd"].float()).to(dt)
        return (o, u.to(dt), g.to(dt)) if case["keep"] else o
    if op == "ffn_bwd":
        dt = t["x"].dtype
        x, do, u, g = (t[n].float() for n in ("x", "do", "u", "g"))
        dh = do @ t["wd"].float().t()
        sg = 1.0 / (1.0 + torch.exp(-u))
        a = u * sg
        dg = dh * a
        du = dh * g * (sg * (1.0 + u * (1.0 - sg)))
        dx = du @ t["wu"].float().t() + dg @ t["wg"].float().t()
        return (dx.to(dt), (x.t() @ du).to(dt), (x.t() @ dg).to(dt), ((a * g).t() @ do).to(dt))
    if op == "matvec":
        w = _dequant(t["w"][0][0], t["w"][1][0], case["group"], case["K"])
        return (t["x"].float() @ w).to(torch.bfloat16)
    S, k, H, D, E = (case[n] for n in ("S", "k", "H", "D", "E"))
    gr = case["group"]
    x, ids = t["x"].float(), t["ids"].long()
    w = torch.where(ids >= 0, t["w"], 0.0)
    matrices = (("up", H), ("gate", H), ("down", D))
    if S * k < E:  # fewer choices than experts: the chosen matrices, one after another
        at = ids.clamp(min=0).view(-1)
        y = _gated(x.repeat_interleave(k, dim=0)[:, None],
                   *(_dequant(t[n][0][at], t[n][1][at], gr, K) for n, K in matrices))
        o = (y.view(S, k, H) * w[:, :, None]).sum(1)
    else:  # every expert on every token, weighted by the choices
        y = _gated(x.expand(E, S, H), *(_dequant(*t[n], gr, K) for n, K in matrices))
        m = ((ids[:, :, None] == torch.arange(E, device=DEV)) * w[:, :, None]).sum(1)
        o = (y * m.t()[:, :, None]).sum(0)
    if case["D_shared"]:
        o = o + _gated(t["x"].float(), *(
            _dequant(t[n][0][0], t[n][1][0], gr, K)
            for n, K in (("s_up", H), ("s_gate", H), ("s_down", case["D_shared"]))))
    return o.to(torch.bfloat16)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    es = 4 if case.get("dtype") == "f32" else 2
    if op == "ln_fwd":
        S, H = case["S"], case["H"]
        return {"bytes": 2 * S * H * es + 2 * H * es + 8 * S, "flops": 8 * S * H}
    if op == "ln_bwd":
        S, H = case["S"], case["H"]
        return {"bytes": 3 * S * H * es + H * es + 8 * H + 8 * S, "flops": 14 * S * H}
    if op == "ffn_fwd":
        S, H, D = case["S"], case["H"], case["D"]
        return {"bytes": es * (2 * S * H + 3 * H * D + (2 * S * D if case["keep"] else 0)),
                "flops": 6 * S * H * D}
    if op == "ffn_bwd":
        S, H, D = case["S"], case["H"], case["D"]
        return {"bytes": es * (3 * S * H + 6 * H * D + 2 * S * D), "flops": 12 * S * H * D}
    if op == "matvec":
        S, K, N = case["S"], case["K"], case["N"]
        return {"bytes": K * N // 2 + 2 * -(-K // case["group"]) * N + 2 * S * (K + N),
                "flops": 2 * S * K * N}
    S, H, D, E, k, Ds = (case[n] for n in ("S", "H", "D", "E", "k", "D_shared"))
    live = S - case["padded"]
    # experts that at least one of the live tokens chooses, k of E each, as expected at random
    used = E * (1.0 - (1.0 - k / E) ** live)
    per = 0.5 + 2.0 / case["group"]
    return {"bytes": int(3 * H * (used * D + Ds) * per) + 4 * S * H + 8 * S * k,
            "flops": 6 * H * (live * k * D + S * Ds)}


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _mm64(a, b):
    return torch.mm(a.to(torch.float64), b.to(torch.float64))


def _w64(pair, e, group):
    """Matrix e of a 4-bit weight, row by row from its group's scale."""
    codes, scales = pair[0][e], pair[1][e].to(torch.float64)
    rows = torch.arange(codes.shape[0], device=codes.device) // group
    return (codes.to(torch.float64) - 8) * scales[rows]


def _swiglu64(u, g):
    return u * torch.special.expit(u) * g


def exact(case, seed):
    t = _inputs(case, seed)
    op = case["op"]
    if op == "ln_fwd":
        y, m, r = [], [], []
        for x in t["x"].split(2048):
            x = x.double()
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rs = 1.0 / torch.sqrt(var + 1e-5)
            y.append(torch.addcmul(t["beta"].double(), (x - mean[:, None]) * rs[:, None],
                                   t["gamma"].double()))
            m.append(mean)
            r.append(rs)
        return torch.cat(y), torch.cat(m), torch.cat(r)
    if op == "ln_bwd":
        H = case["H"]
        dx, dg, db = [], 0, 0
        for x, dy, m, r in zip(*(t[n].split(2048) for n in ("x", "dy", "mean", "rstd"))):
            n = (x.double() - m.double()[:, None]) * r.double()[:, None]
            dy = dy.double()
            d = dy * t["gamma"].double()
            c0 = d.sum(1, keepdim=True) / H
            c1 = (d * n).sum(1, keepdim=True) / H
            dx.append(r.double()[:, None] * (d - (c0 + c1 * n)))
            dg = dg + (dy * n).sum(0)
            db = db + dy.sum(0)
        return torch.cat(dx), dg, db
    if op == "ffn_fwd":
        u, g = _mm64(t["x"], t["wu"]), _mm64(t["x"], t["wg"])
        o = _mm64(_swiglu64(u, g), t["wd"])
        return (o, u, g) if case["keep"] else o
    if op == "ffn_bwd":
        u, g = t["u"].double(), t["g"].double()
        dh = _mm64(t["do"], t["wd"].t())
        s = torch.special.expit(u)
        du = dh * g * (s + u * s * torch.special.expit(-u))
        dg = dh * u * s
        dx = _mm64(torch.cat([du, dg], 1), torch.cat([t["wu"], t["wg"]], 1).t())
        xt = t["x"].t()
        return dx, _mm64(xt, du), _mm64(xt, dg), _mm64(_swiglu64(u, g).t(), t["do"])
    gr = case["group"]
    if op == "matvec":
        return _mm64(t["x"], _w64(t["w"], 0, gr))
    o = torch.zeros((case["S"], case["H"]), dtype=torch.float64, device=DEV)
    ids = t["ids"].cpu()
    for e in sorted(set(ids[ids >= 0].tolist())):  # expert by expert
        s, j = (ids == e).nonzero(as_tuple=True)
        s, j = s.to(DEV), j.to(DEV)
        x = t["x"][s]
        h = _swiglu64(_mm64(x, _w64(t["up"], e, gr)), _mm64(x, _w64(t["gate"], e, gr)))
        o.index_add_(0, s, _mm64(h, _w64(t["down"], e, gr)) * t["w"][s, j].double()[:, None])
    if case["D_shared"]:
        h = _swiglu64(_mm64(t["x"], _w64(t["s_up"], 0, gr)),
                      _mm64(t["x"], _w64(t["s_gate"], 0, gr)))
        o += _mm64(h, _w64(t["s_down"], 0, gr))
    return o
