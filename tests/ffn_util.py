"""Plain 64-bit forms and derived error bounds for the GPU tests of the operators
of include/moe_ffn.h. Everything here runs on the device in float64.

Bounds are per element. u = 2^-24 is half a step of fp32, half(t) half a step of
the output's type; a sum of n terms in any order is off by at most n u times the
sum of the terms' magnitudes. Where an operand is itself rounded to bf16 (h, dU,
dG as operands of the products), each of its elements is off by at most 2^-8 of
its value, uniformly, so the sum over K of them has a standard deviation of at
most 2^-8 / sqrt(3) sqrt(sum (a w)^2); six of those bound every element of any
test (a chance of 2e-9 each).
"""
import torch

DEV = "cuda:0"
U = 2.0 ** -24


def half(t):
    return torch.finfo(t).eps / 2


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, shape, std, dtype, mean=0.0):
    return (torch.randn(shape, generator=g, device=DEV) * std + mean).to(dtype)


def check(name, got, ref, bound):
    """|got - ref| <= bound element by element, and no NaN."""
    got = got.double()
    err = (got - ref).abs()
    bad = ~(err <= bound)
    if bool(bad.any()):
        i = int(torch.argmax(torch.where(bad, err / bound.clamp(min=1e-300), 0.0).flatten()))
        raise AssertionError(
            f"{name}: {int(bad.sum())} of {bad.numel()} elements off; worst at {i}: got "
            f"{got.flatten()[i].item()!r}, reference {ref.flatten()[i].item()!r}, bound "
            f"{bound.flatten()[i].item():.3e}")


# ---------------------------------------------------------------- layer norm

def ln_ref(x, gamma, beta, eps):
    """(y, mean, rstd, bound of y before its rounding, of mean, of rstd)."""
    H = x.shape[1]
    x = x.double()
    g = torch.ones(H, device=DEV, dtype=torch.float64) if gamma is None else gamma.double()
    b = torch.zeros(H, device=DEV, dtype=torch.float64) if beta is None else beta.double()
    m = x.mean(1, keepdim=True)
    v = (x - m).square().mean(1, keepdim=True)
    r = 1 / torch.sqrt(v + eps)
    n = (x - m) * r
    d = 80 + H / 256  # longest chain of additions: a thread's, then a tree's
    em = (d + 2) * U * x.abs().mean(1, keepdim=True)       # of the mean
    # the centred squares: (x - m') with m' off by em adds em^2 to the mean of the
    # squares and nothing in first order, roundings (d + 4) u of it
    er = r * (0.5 * ((d + 4) * U * v + em * em) / (v + eps) + 4 * U)
    y = n * g + b
    ey = g.abs() * (r * em + n.abs() * (er / r + 4 * U)) + 2 * U * (b.abs() + (n * g).abs())
    return y, m[:, 0], r[:, 0], ey, em[:, 0] + U * m[:, 0].abs(), er[:, 0]


def ln_bwd_ref(dy, x, gamma, mean, rstd):
    S, H = x.shape
    x, dy = x.double(), dy.double()
    g = torch.ones(H, device=DEV, dtype=torch.float64) if gamma is None else gamma.double()
    m, r = mean.double()[:, None], rstd.double()[:, None]
    n, d = (x - m) * r, dy * g
    c0, c1 = d.mean(1, keepdim=True), (d * n).mean(1, keepdim=True)
    dx = r * (d - c0 - n * c1)
    k = 80 + H / 256
    e0 = (k + 3) * U * d.abs().mean(1, keepdim=True)
    e1 = (k + 6) * U * (d * n).abs().mean(1, keepdim=True)
    edx = r * (e0 + n.abs() * e1 + 6 * U * (d.abs() + c0.abs() + (n * c1).abs()))
    # a group's rows, then the groups' sums (four chains and their join)
    rows = min(S, S / 512 + 160)
    dg, db = (dy * n).sum(0), dy.sum(0)
    return (dx, dg, db, edx, (rows + 4) * U * (dy * n).abs().sum(0) + 1e-300,
            (rows + 2) * U * dy.abs().sum(0) + 1e-300)


# ---------------------------------------------------------------- feed-forward block

def mm(a, b):
    return torch.mm(a.double(), b.double())


def ffn_ref(x, wu, wg, wd, bf16):
    """(o, u, g, bounds before the outputs' rounding)."""
    H, D = wu.shape
    u, g = mm(x, wu), mm(x, wg)
    eu, eg = H * U * mm(x.abs(), wu.abs()), H * U * mm(x.abs(), wg.abs())
    s = torch.sigmoid(u)
    a = u * s
    h = a * g
    # d silu / du is at most 1.1; exp and rcp to 2 u, exp's argument to u of itself
    eh = 1.1 * g.abs() * eu + a.abs() * eg + 8 * U * (1 + u.abs()) * h.abs()
    o = mm(h, wd)
    eo = mm(eh, wd.abs()) + D * U * mm(h.abs(), wd.abs())
    if bf16:
        eo += 6 * half(torch.bfloat16) / 3 ** 0.5 * mm(h.square(), wd.double().square()).sqrt()
    return o, u, g, eo, eu, eg


def ffn_bwd_ref(do, x, wu, wg, wd, u, g, bf16):
    """(dx, dwu, dwg, dwd, bounds before rounding)."""
    H, D = wu.shape
    S = x.shape[0]
    u, g = u.double(), g.double()
    dh = mm(do, wd.t())
    edh = H * U * mm(do.abs(), wd.abs().t())
    s = torch.sigmoid(u)
    a, t = u * s, s * (1 + u * (1 - s))
    du, dg, h = dh * g * t, dh * a, a * g
    fu = U * (1 + u.abs())
    edu = edh * (g * t).abs() + 16 * fu * (dh * g).abs() * (s + (u * s * (1 - s)).abs())
    edg = edh * a.abs() + 8 * fu * dg.abs()
    eh = 8 * fu * h.abs()
    q = 6 * half(torch.bfloat16) / 3 ** 0.5 if bf16 else 0.0

    def prod(a, ea, b, n):
        e = mm(ea, b.abs()) + n * U * mm(a.abs(), b.abs())
        if bf16:
            e += q * mm(a.square(), b.double().square()).sqrt()
        return mm(a, b), e

    dx0, e0 = prod(du, edu, wu.t(), 2 * D)
    dx1, e1 = prod(dg, edg, wg.t(), 2 * D)
    xt = x.t().contiguous()

    def wprod(b, eb):  # X^T b, b rounded
        e = mm(xt.abs(), eb) + S * U * mm(xt.abs(), b.abs())
        if bf16:
            e += q * mm(xt.double().square(), b.square()).sqrt()
        return mm(xt, b), e

    dwu, eu = wprod(du, edu)
    dwg, eg = wprod(dg, edg)
    dwd, ed = prod(h.t(), eh.t(), do, S)
    return (dx0 + dx1, dwu, dwg, dwd), (e0 + e1, eu, eg, ed)


# ---------------------------------------------------------------- 4-bit weights

def w4(g, E, K, N, group, std=None):
    """Random codes and scales (weights of std about 1 / sqrt(K))."""
    codes = torch.randint(0, 16, (E, K, N), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.rand((E, -(-K // group), N), generator=g, device=DEV) + 0.5
    return codes, (s / (4.6 * K ** 0.5)).to(torch.bfloat16)


def dequant(codes, scales, group):
    K = codes.shape[-2]
    s = scales.double().repeat_interleave(group, dim=-2)[..., :K, :]
    return (codes.double() - 8) * s


def w4_bound(x, codes, scales, group):
    """Bound of the sums with one matrix, before rounding: a group sums x (code + 16)
    and 24 x, at most 55 |x| together, over 2 x 128 terms at most, and is scaled;
    the groups, and up to 16 shares of K, are added in chains."""
    K = codes.shape[-2]
    s = scales.double().abs().repeat_interleave(group, dim=-2)[..., :K, :]
    w = dequant(codes, scales, group).abs()
    return (2 * group + 8) * U * 55 * mm(x.abs(), s) + (K / group + 32) * U * mm(x.abs(), w)
