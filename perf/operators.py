"""The products with 4-bit group-quantized weights that are measured, in their plain form and as the library's calls.

Weights are what ``fq.quant_groups(w, group, 4, scheme)`` stores: codes packed
two to a byte (even column in the high nibble), a float32 scale and, for affine
weights, an int32 zero-point per group of consecutive columns of a row; the
weight they stand for is W = (code - zero_point) * scale.

    matmul          y = x W^T
    gated           h = act(x Wg^T) * (x Wu^T), and g = x Wg^T, u = x Wu^T where a backward pass follows
    matmul_backward dx = dy W, dW = dy^T x (the straight-through gradient of the weights)
    gated_backward  dg = dh u act'(g), du = dh act(g); dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
"""
import math

import torch

own = False

SQRT_HALF = math.sqrt(0.5)
INV_SQRT_2PI = 1.0 / math.sqrt(2.0 * math.pi)


def listed():
    def case(name, op, m, n, k, group, scheme, dtype, act="silu", save=False):
        return dict(name=name, op=op, m=m, n=n, k=k, group=group, scheme=scheme, dtype=dtype, act=act, save=save)

    return [
        # one token against a square projection: the call whose latency a decoder sees most often
        case("matmul token", "matmul", 1, 4096, 4096, 128, "sym", "bf16"),
        # one token through the long side of a feed-forward block, affine weights with fine groups
        case("matmul token long", "matmul", 1, 4096, 12288, 64, "affine", "bf16"),
        # a few float32 rows, odd sizes, a short last group
        case("matmul few f32 ragged", "matmul", 5, 1000, 1100, 32, "affine", "f32"),
        # a serving batch of single tokens
        case("matmul batch", "matmul", 48, 8192, 4096, 128, "affine", "bf16"),
        # a prompt, or a training step's forward product
        case("matmul prompt", "matmul", 4096, 4096, 4096, 128, "sym", "bf16"),
        # one token through a gated block's first half
        case("gated token", "gated", 1, 12288, 4096, 128, "sym", "bf16"),
        # a short float32 sequence, odd sizes, fine groups
        case("gated few f32 ragged", "gated", 37, 1411, 1000, 32, "affine", "f32", "gelu"),
        # a training step's forward pass, which keeps g and u
        case("gated train", "gated", 4096, 12288, 4096, 128, "sym", "bf16", "silu", True),
        # gradients of a square projection
        case("matmul backward", "matmul_backward", 4096, 4096, 4096, 128, "sym", "bf16"),
        # gradients at odd sizes: short sequence, short last group
        case("matmul backward ragged", "matmul_backward", 333, 1000, 777, 64, "affine", "bf16"),
        # a training step's backward pass, the largest case
        case("gated backward", "gated_backward", 4096, 12288, 4096, 128, "sym", "bf16"),
        # the same at odd sizes with fine groups
        case("gated backward ragged", "gated_backward", 131, 1411, 520, 32, "affine", "bf16", "gelu"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["matmul", "matmul", "gated", "gated", "matmul_backward", "gated_backward"])
    backward = op.endswith("backward")
    m = spread(1, 8) if not backward and rng.random() < 0.4 else spread(1, 4096)
    n, k = spread(64, 12288), spread(64, 12288)
    if rng.random() < 0.6:  # most layers' widths are multiples of 64
        n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
    n = min(n, max(64, 4096 * 12288 // k))
    return dict(op=op, m=m, n=n, k=k, group=rng.choice([32, 64, 128]), scheme=rng.choice(["sym", "affine"]),
                dtype="f32" if not backward and rng.random() < 0.25 else "bf16", act=rng.choice(["silu", "gelu"]),
                save=op == "gated" and rng.random() < 0.4)


def _weights(case, gen):
    """A weight matrix whose rows have lognormal sigmas, quantized group by group."""
    n, k, group = case["n"], case["k"], case["group"]
    ng = (k + group - 1) // group
    sigma = torch.exp(torch.randn(n, 1, generator=gen, device="cuda") * 0.5) / math.sqrt(k)
    w = torch.randn(n, k, generator=gen, device="cuda") * sigma
    w = torch.cat([w, w.new_zeros(n, ng * group - k)], 1).view(n, ng, group)
    if case["scheme"] == "sym":
        scale, zp = w.abs().amax(2) / 7.0, None
        code = torch.round(w / scale[..., None]).clamp(-7, 7)
    else:
        lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
        scale = (hi - lo) / 15.0
        zp = torch.round(-8.0 - lo / scale).clamp(-8, 7)
        code = (torch.round(w / scale[..., None]) + zp[..., None]).clamp(-8, 7)
    code = code.view(n, ng * group)[:, :k].to(torch.int32) & 15
    if k % 2:
        code = torch.cat([code, code.new_zeros(n, 1)], 1)
    packed = (code[:, 0::2] * 16 + code[:, 1::2]).to(torch.uint8)
    return dict(codes=packed.contiguous(), scale=scale.contiguous(), zp=None if zp is None else zp.to(torch.int32).contiguous())


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    m, n, k = case["m"], case["n"], case["k"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    x = torch.randn(m, k, generator=gen, device="cuda")
    x[:, :: 97] *= 10.0  # about one channel in a hundred is an outlier
    s = dict(case=dict(case), x=x.to(dt))
    gated = case["op"].startswith("gated")
    s["w"] = [_weights(case, gen) for _ in range(2 if gated else 1)]
    if case["op"].endswith("backward"):
        dy = torch.randn(m, n, generator=gen, device="cuda") * 1e-3
        dy[m // 2 :: 8] = 0.0  # tokens that the loss leaves out
        s["dy"] = dy.to(dt)
    if case["op"] == "gated_backward":
        s["g"], s["u"] = ((s["x"].float() @ _dense(w, k, case["group"]).t()).to(dt) for w in s["w"])
    return s


def _dense(w, k, group):
    """The float32 matrix that the stored codes stand for."""
    b = w["codes"].to(torch.int32)
    c = torch.stack([b >> 4, b & 15], 2).view(b.shape[0], -1)[:, :k]
    c = (c - 16 * (c > 7).to(torch.int32)).to(torch.float32)
    if w["zp"] is not None:
        c = c - w["zp"].to(torch.float32).repeat_interleave(group, 1)[:, :k]
    return c * w["scale"].repeat_interleave(group, 1)[:, :k]


def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * torch.erfc(-SQRT_HALF * g)


def _act_slope(g, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    return 0.5 * torch.erfc(-SQRT_HALF * g) + g * INV_SQRT_2PI * torch.exp(-0.5 * g * g)


def _plain(s):
    c, x = s["case"], s["x"]
    dt, k, group, xf = x.dtype, c["k"], c["group"], x.float()
    w = [_dense(v, k, group) for v in s["w"]]
    if c["op"] == "matmul":
        return (xf @ w[0].t()).to(dt)
    if c["op"] == "gated":
        g, u = xf @ w[0].t(), xf @ w[1].t()
        h = (_act(g, c["act"]) * u).to(dt)
        return (h, g.to(dt), u.to(dt)) if c["save"] else h
    dy = s["dy"].float()
    if c["op"] == "matmul_backward":
        return (dy @ w[0]).to(dt), dy.t() @ xf
    g, u = s["g"].float(), s["u"].float()
    dg, du = dy * u * _act_slope(g, c["act"]), dy * _act(g, c["act"])
    return (dg @ w[0] + du @ w[1]).to(dt), (dg.t() @ xf).to(dt), (du.t() @ xf).to(dt)


def run(state):
    if not own:
        return _plain(state)
    from fake_quant_amd import linear

    c, x, w = state["case"], state["x"], state["w"]
    if c["op"] == "matmul":
        return linear.w4_matmul(x, w[0], c["group"])
    if c["op"] == "gated":
        return linear.w4_gated(x, w[0], w[1], c["group"], c["act"], save=c["save"])
    if c["op"] == "matmul_backward":
        return linear.w4_matmul_backward(state["dy"], x, w[0], c["group"])
    return linear.w4_gated_backward(state["dy"], x, state["g"], state["u"], w[0], w[1], c["group"], c["act"])


def work(case):
    m, n, k = case["m"], case["n"], case["k"]
    ng = -(-k // case["group"])
    e = 4 if case["dtype"] == "f32" else 2
    weight = n * (-(-k // 2)) + n * ng * (4 if case["scheme"] == "sym" else 8)
    if case["op"] == "matmul":
        return dict(bytes=weight + e * m * (k + n), flops=2 * m * n * k)
    if case["op"] == "gated":
        return dict(bytes=2 * weight + e * m * (k + n * (3 if case["save"] else 1)), flops=4 * m * n * k)
    if case["op"] == "matmul_backward":  # reads dy, x and W, writes dx and a float32 dW
        return dict(bytes=weight + e * m * (n + 2 * k) + 4 * n * k, flops=4 * m * n * k)
    return dict(bytes=2 * weight + e * m * (3 * n + 2 * k) + 2 * e * n * k, flops=8 * m * n * k)


def exact(case, seed):
    s = prepare(case, seed)
    k, group = case["k"], case["group"]

    def dense64(w):
        # every byte's two values from a table, then the groups' zero-points and scales by column index
        byte = torch.arange(256, device="cuda")
        nib = torch.stack([byte.div(16, rounding_mode="floor"), byte.remainder(16)], 1).double()
        table = torch.where(nib >= 8.0, nib - 16.0, nib)
        v = table[w["codes"].long()].flatten(1)[:, :k]
        col = torch.arange(k, device="cuda").div(group, rounding_mode="floor")
        if w["zp"] is not None:
            v = v - w["zp"].double()[:, col]
        return v * w["scale"].double()[:, col]

    def act64(g):
        if case["act"] == "silu":
            return g * torch.sigmoid(g)
        return g * 0.5 * torch.special.erfc(-g / math.sqrt(2.0))

    def slope64(g):
        if case["act"] == "silu":
            p = torch.sigmoid(g)
            return p + g * p * torch.sigmoid(-g)
        return 0.5 * torch.special.erfc(-g / math.sqrt(2.0)) + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)

    x = s["x"].double()
    w = [dense64(v) for v in s["w"]]
    if case["op"] == "matmul":
        return torch.matmul(x, w[0].T)
    if case["op"] == "gated":
        g, u = torch.matmul(x, w[0].T), torch.matmul(x, w[1].T)
        h = act64(g) * u
        return (h, g, u) if case["save"] else h
    dy = s["dy"].double()
    if case["op"] == "matmul_backward":
        return torch.matmul(dy, w[0]), torch.matmul(dy.T, x)
    g, u = s["g"].double(), s["u"].double()
    dg, du = dy * u * slope64(g), dy * act64(g)
    return torch.matmul(dg, w[0]) + torch.matmul(du, w[1]), torch.matmul(dg.T, x), torch.matmul(du.T, x)
