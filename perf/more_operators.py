"""Measured cases of the feed-forward half of a layer whose weights are held in
microscaled 4-bit floating point.

Three families, as a serving or fine-tuning program meets them:

* e2m1 codes with a power-of-two scale per 32 values: the quantizer (rows, or
  columns for the operands of a weight gradient), the product of float
  activations with such a weight for any number of rows.
* root-mean-square norm with the residual's addition, in float or as e4m3 codes
  with a scale per 128 values, and its gradients; followed by a projection.
* the gated feed-forward block: gate and up projections with silu(gate) * up in
  one product, the down projection, and the gated product's gradients.

``run`` computes a case in elementary torch operations in fp32, or, with the
module's ``own`` set, by the library's calls.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
TOP = 448.0   # the largest e4m3 value
BLOCK = 128   # values of an e4m3 scale
MX = 32       # values of a 4-bit scale
PITCH = 512   # a row of 4-bit codes holds a multiple of this many values
EPS = 1e-6

#: cases ------------------------------------------------------------------


def listed():
    return [
        # A weight turned into 4-bit codes when a model is loaded, and read back to look at the loss.
        dict(name="quantize weight", kind="quantize", n=11008, k=4096, type="f32"),
        # One token through a square projection of a 7B-shaped layer: the smallest product, latency.
        dict(name="matmul 1 row", kind="matmul", m=1, n=4096, k=4096, type="bf16"),
        # Eight sequences decoded together, the widest 70B-shaped matrix, fp32 activations.
        dict(name="matmul 8 rows", kind="matmul", m=8, n=28672, k=8192, type="f32"),
        # A chunk of a prompt; no size is a multiple of a tile or a block.
        dict(name="matmul odd", kind="matmul", m=203, n=5003, k=4101, type="f32"),
        # A whole prompt through the 70B-shaped matrix: arithmetic.
        dict(name="matmul prompt", kind="matmul", m=2048, n=28672, k=8192, type="bf16"),
        # Weight gradient of a 7B-shaped projection over a batch of tokens: both sides are
        # quantized along the tokens, that is down their columns.
        dict(name="weight gradient", kind="wgrad", m=4096, n=11008, k=2048, type="bf16"),
        # Residual and norm of a few decoded tokens: the smallest call, latency.
        dict(name="norm decode", kind="norm", t=5, d=4096, type="bf16", out="float", residual=True),
        # The same for a long prompt, as the e4m3 codes that the next product takes.
        dict(name="norm prompt", kind="norm", t=8192, d=8192, type="bf16", out="block", residual=True),
        # Gradients of the norm over a ragged batch, odd width.
        dict(name="norm backward", kind="norm_backward", t=4099, d=5003, type="f32", residual=True),
        # A whole feed-forward block for four decoded tokens: its weights are read once.
        dict(name="mlp decode", kind="mlp", m=4, d=4096, f=11008, type="bf16"),
        # The same over a prompt: arithmetic.
        dict(name="mlp prompt", kind="mlp", m=2048, d=4096, f=11008, type="bf16"),
        # Gradients of gate and up over a training batch of odd length, recomputing the products.
        dict(name="gated backward", kind="gated_backward", m=2047, d=4096, f=11008, type="bf16"),
    ]


def _log(rng, lo, hi):
    """An integer whose logarithm is spread evenly over [lo, hi]; half of them rounded to a multiple of 128 (or of 8) where there is room."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        unit = 128 if v >= 512 else 8 if v >= 32 else 1
        v = v // unit * unit
    return max(lo, min(hi, v))


def draw(rng):
    kind = rng.choice(["matmul", "matmul", "wgrad", "quantize", "norm", "norm_backward", "project", "mlp", "mlp", "gated_backward"])
    kind_type = rng.choice(["bf16", "f32"])
    if kind in ("matmul", "project"):
        n, k = _log(rng, 256, 28672), _log(rng, 200, 8192)
        m = _log(rng, 1, max(1, min(4096, 400_000_000_000 // (n * k))))
        return dict(kind=kind, m=m, n=n, k=k, type=kind_type)
    if kind == "wgrad":
        return dict(kind=kind, m=_log(rng, 256, 4096), n=_log(rng, 256, 11008), k=_log(rng, 64, 2048), type=kind_type)
    if kind == "quantize":
        return dict(kind=kind, n=_log(rng, 128, 11008), k=_log(rng, 128, 4096), type=kind_type)
    if kind in ("norm", "norm_backward"):
        t, d = _log(rng, 1, 8192), _log(rng, 64, 8192)
        more = dict(out=rng.choice(["float", "block"])) if kind == "norm" else {}
        return dict(kind=kind, t=t, d=d, type=kind_type, residual=rng.random() < 0.7, **more)
    return dict(kind=kind, m=_log(rng, 1, 2047), d=_log(rng, 256, 4096), f=_log(rng, 128, 11008), type=kind_type)


def _pitch(k):
    return (k + PITCH - 1) // PITCH * PITCH


def work(case):
    c, s = case, 4 if case["type"] == "f32" else 2
    kind = c["kind"]
    # half a byte and a 32nd part of a scale byte for a 4-bit value
    held = lambda n, k: n * k * 17 / 32  # noqa: E731
    if kind in ("matmul", "project"):
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": held(n, k) + m * k * s + m * n * s + (m * k * s + 4 * k if kind == "project" else 0), "flops": 2.0 * m * n * k}
    if kind == "wgrad":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": (m + n) * k * s + 4 * m * n, "flops": 2.0 * m * n * k}
    if kind == "quantize":
        # to codes, and the codes back to fp32 values
        return {"bytes": c["n"] * c["k"] * (s + 4) + 2 * held(c["n"], c["k"]), "flops": 2.0 * c["n"] * c["k"]}
    if kind == "norm":
        t, d = c["t"], c["d"]
        out = s if c["out"] == "float" else 1 + 4 / BLOCK
        return {"bytes": t * d * (s + out + (2 * s if c["residual"] else 0)) + 4 * d, "flops": 5.0 * t * d}
    if kind == "norm_backward":
        t, d = c["t"], c["d"]
        return {"bytes": t * d * s * (4 if c["residual"] else 3) + 8 * d, "flops": 10.0 * t * d}
    m, d, f = c["m"], c["d"], c["f"]
    if kind == "mlp":
        return {"bytes": held(3 * f, d) + 2 * m * d * s, "flops": 6.0 * m * d * f}
    # gated_backward: the codes of x and of both weights and dh in; gate's and up's gradients and the gated values out
    return {"bytes": held(2 * f + m, d) + 4 * m * f * s, "flops": 4.0 * m * d * f}


#: inputs -----------------------------------------------------------------


def _normal(g, *shape, std=1.0, type="f32"):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).to(TYPES[type])


def _activations(g, rows, width, type):
    """Normal values with the few large channels that layers' inputs have."""
    channel = 1.0 + 15.0 * (torch.rand(width, generator=g, device=DEV) < 0.004).float()
    return (torch.randn(rows, width, generator=g, device=DEV) * channel).to(TYPES[type])


def _gain(g, d):
    return 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    kind = c["kind"]
    if kind in ("matmul", "project"):
        state = dict(case=c, w=_codes(_normal(g, c["n"], c["k"], std=0.02)), x=_activations(g, c["m"], c["k"], c["type"]))
        if kind == "project":
            state |= dict(res=_activations(g, c["m"], c["k"], c["type"]), gain=_gain(g, c["k"]))
        return state
    if kind == "wgrad":
        # a program's tensors: one row for each token
        return dict(case=c, dy=_normal(g, c["k"], c["m"], std=1e-3, type=c["type"]), x=_normal(g, c["k"], c["n"], type=c["type"]))
    if kind == "quantize":
        return dict(case=c, w=_normal(g, c["n"], c["k"], std=0.02, type=c["type"]))
    if kind in ("norm", "norm_backward"):
        state = dict(case=c, x=_activations(g, c["t"], c["d"], c["type"]), gain=_gain(g, c["d"]))
        if c["residual"]:
            state["res"] = _activations(g, c["t"], c["d"], c["type"])
        if kind == "norm_backward":
            state["dy"] = _normal(g, c["t"], c["d"], std=1e-3, type=c["type"])
        return state
    gate_up = _codes(_normal(g, 2 * c["f"], c["d"], std=c["d"] ** -0.5))
    x = _activations(g, c["m"], c["d"], c["type"])
    if kind == "mlp":
        return dict(case=c, gate_up=gate_up, down=_codes(_normal(g, c["d"], c["f"], std=c["f"] ** -0.5)), x=x)
    # the forward pass has left the codes of x
    return dict(case=c, gate_up=gate_up, x=_codes(x), dh=_normal(g, c["m"], c["f"], std=1e-3, type=c["type"]))


def _out(c):
    """The outputs' type. Behind inner values that are rounded to 4 bits the last bit of an fp32 sum decides between two codes now and then: those outputs are no fp32 values."""
    return torch.bfloat16 if c["kind"] in ("mlp", "project") else TYPES[c["type"]]


#: the plain forms --------------------------------------------------------


def _codes(w):
    """4-bit codes (two to a byte, the first in the low half, rows of whole 512s) and scale bytes of a matrix (n, k), one for 32 values of a row.

    A scale is 2^(e - 127) with e the exponent of the largest magnitude less 2, so that it lies in [4, 8) scales; codes are the nearest of
    0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code) and bit 3 the sign.
    """
    n, k = w.shape
    kp = _pitch(k)
    p = torch.zeros(n, kp, device=w.device, dtype=torch.float32)
    p[:, :k] = w
    p = p.view(n, kp // MX, MX)
    top = p.abs().amax(-1)
    ex = torch.frexp(top)[1] - 3
    ex = torch.where(top == 0, 0, ex.clamp(min=-127))
    # 2^-e as two factors: it may be beyond fp32's largest power
    a = torch.ldexp(torch.ldexp(p, -(ex // 2)[..., None]), -(ex - ex // 2)[..., None])
    v = a.abs()
    q = (v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0)
    q = (q | torch.signbit(a).to(torch.uint8) << 3).view(n, kp // 2, 2)
    return q[..., 0] | q[..., 1] << 4, (ex + 127).to(torch.uint8)


def _values(codes, scales, k):
    """The fp32 values that codes stand for, (n, k)."""
    n = codes.shape[0]
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], -1).int()].view(n, -1, MX)
    return torch.ldexp(v, scales.int()[..., None] - 127).view(n, -1)[:, :k]


def _through(x):
    """x (m, k) as the values of its codes."""
    return _values(*_codes(x), x.shape[1])


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _norm(x, res, gain):
    """The sum that the norm sees, rounded to x's type, and the norm in fp32."""
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    v = h.float()
    return h, v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * gain


def _block(y):
    """e4m3 codes (rows of whole blocks) and scales of 1 x 128 blocks."""
    t, d = y.shape
    p = torch.zeros(t, (d + BLOCK - 1) // BLOCK * BLOCK, device=y.device)
    p[:, :d] = y
    p = p.view(t, -1, BLOCK)
    s = p.abs().amax(-1)
    s = s / torch.full_like(s, TOP)
    s = torch.where(s == 0, torch.ones_like(s), s)
    return (p / s[..., None]).clamp(-TOP, TOP).to(E4M3).view(t, -1), s


def _plain(state):
    c = state["case"]
    kind, out = c["kind"], _out(c)
    if kind == "matmul":
        return (_through(state["x"]) @ _values(*state["w"], c["k"]).t()).to(out)
    if kind == "project":
        h, y = _norm(state["x"], state["res"], state["gain"])
        return h, (_through(y) @ _values(*state["w"], c["k"]).t()).to(out)
    if kind == "wgrad":
        return _through(state["dy"].t().contiguous()) @ _through(state["x"].t().contiguous()).t()
    if kind == "quantize":
        return _through(state["w"])
    if kind == "norm":
        h, y = _norm(state["x"], state.get("res"), state["gain"])
        return h, y.to(out) if c["out"] == "float" else _block(y)
    if kind == "norm_backward":
        # the gradient of the sum: the norm's, and what flows past it
        v, dy = state["x"].float(), state["dy"].float()
        r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
        u = dy * state["gain"]
        dx = r * u - v * (r * r * r * (u * v).mean(-1, keepdim=True))
        if c["residual"]:
            dx = dx + state["res"].float()
        return dx.to(out), (dy * v * r).sum(0)
    f = c["f"]
    x = _through(state["x"]) if kind == "mlp" else _values(*state["x"], c["d"])
    p = x @ _values(*state["gate_up"], c["d"]).t()
    gate, up = p[:, :f], p[:, f:]
    h = _silu(gate) * up
    if kind == "mlp":
        return (_through(h) @ _values(*state["down"], f).t()).to(out)
    dh = state["dh"].float()
    s = 1.0 / (1.0 + torch.exp(-gate))
    dgate = dh * up * s * (1.0 + gate * (1.0 - s))
    return torch.cat([dgate, dh * gate * s], 1).to(out), h.to(out)


#: the library's calls ----------------------------------------------------


def _rec(codes, n, k):
    return dict(bits=4, block=MX, shape=[n, k], codes=codes[0], scales=codes[1])


def _own(state):
    from int8_int4_dequant_amd import qw
    c = state["case"]
    kind, out = c["kind"], _out(c)
    if kind == "matmul":
        return qw.mx_matmul(_rec(state["w"], c["n"], c["k"]), state["x"], out_dtype=out)
    if kind == "project":
        y, h = qw.rms_norm(state["x"], state["gain"], residual=state["res"], eps=EPS, quantize="mx")
        return h, qw.mx_gemm(_rec(state["w"], c["n"], c["k"]), y, out_dtype=out)
    if kind == "wgrad":
        return qw.mx_gemm(qw.mx_quantize(state["x"], transpose=True), qw.mx_quantize(state["dy"], transpose=True))
    if kind == "quantize":
        return qw.mx_unpack(qw.mx_quantize(state["w"]))
    if kind == "norm":
        y, h = qw.rms_norm(state["x"], state["gain"], residual=state.get("res"), eps=EPS, quantize="block" if c["out"] == "block" else None)
        return h, y if c["out"] == "float" else (y["codes"], y["scales"])
    if kind == "norm_backward":
        return qw.rms_norm_backward(state["dy"], state["x"], state["gain"], eps=EPS, dsum=state.get("res"))
    d, f = c["d"], c["f"]
    gate_up = _rec(state["gate_up"], 2 * f, d)
    if kind == "mlp":
        return qw.mx_mlp(gate_up, _rec(state["down"], d, f), state["x"], out_dtype=out)
    return qw.mx_gated_backward(gate_up, _rec(state["x"], c["m"], d), state["dh"])


def run(state):
    return _own(state) if own else _plain(state)


#: the definition in 64 bits ----------------------------------------------


def _round_e2m1(v):
    """The nearest e2m1 value, ties to even: one bit behind the leading one, steps of a half below 1."""
    _, ex = torch.frexp(v)  # |v| = f 2^ex with f in [1/2, 1)
    step = torch.exp2((ex - 2).clamp(min=-1).double())
    return (torch.round(v / step) * step).clamp(-6.0, 6.0)


def _true4(w):
    """The values that w's 4-bit codes stand for."""
    n, k = w.shape
    b = torch.nn.functional.pad(w.double(), (0, -k % MX)).unflatten(1, (-1, MX))
    top = b.abs().amax(2, keepdim=True)
    s = torch.exp2((torch.floor(torch.log2(top.clamp(min=1e-300))) - 2).clamp(min=-127))
    s = torch.where(top >= 8 * s, 2 * s, torch.where(top < 4 * s, s / 2, s))  # log2 rounds next to a power of two
    s = torch.where(top == 0, torch.ones_like(s), s.clamp(min=2.0 ** -127))
    return (_round_e2m1(b / s) * s).flatten(1)[:, :k]


def _read4(held, k):
    """The values of codes and scale bytes."""
    codes, scales = held
    q = torch.stack((codes % 16, codes // 16), 2).flatten(1).long()
    m, e = q % 2, q // 2 % 4
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((e - 1).double()))
    v = torch.where(q >= 8, -v, v) * torch.exp2(scales.double() - 127).repeat_interleave(MX, 1)
    return v[:, :k]


def _true8(y):
    """e4m3 values and scales of 1 x 128 blocks of y, with its fp32 rounding where the format has one."""
    t, d = y.shape
    b = torch.nn.functional.pad(y.float().double(), (0, -d % BLOCK)).unflatten(1, (-1, BLOCK))
    s = (b.abs().amax(2) / TOP).float().double()
    s[s == 0] = 1.0
    v = (b / s[..., None]).float().double().clamp(-TOP, TOP)
    step = torch.exp2((torch.frexp(v)[1] - 4).clamp(min=-9).double())
    return (torch.round(v / step) * step).flatten(1), s


def exact(case, seed):
    c, st = case, prepare(case, seed)
    kind = c["kind"]
    if kind == "matmul":
        return _true4(st["x"]) @ _read4(st["w"], c["k"]).T
    if kind == "quantize":
        return _true4(st["w"])
    if kind == "wgrad":
        return _true4(st["dy"].T) @ _true4(st["x"].T).T
    if kind in ("norm", "project", "norm_backward"):
        h = st["x"].double()
        if kind != "norm_backward" and st.get("res") is not None:
            h = (h + st["res"].double()).to(st["x"].dtype).double()  # the sum is held in the inputs' type
        d, gain = h.shape[1], st["gain"].double()
        r = 1.0 / torch.sqrt((h * h).sum(1) / d + EPS)
        if kind == "norm_backward":
            dy = st["dy"].double()
            dot = ((dy * gain) * h).sum(1) / d
            dx = r[:, None] * (dy * gain - h * (r * r * dot)[:, None])
            return dx + (st["res"].double() if c["residual"] else 0.0), ((dy * h) * r[:, None]).sum(0)
        y = h * r[:, None] * gain
        if kind == "project":
            return h, _true4(y.float()) @ _read4(st["w"], c["k"]).T
        return h, y if c["out"] == "float" else _true8(y)
    f = c["f"]
    weights = _read4(st["gate_up"], c["d"])
    x = _true4(st["x"]) if kind == "mlp" else _read4(st["x"], c["d"])
    gate, up = x @ weights[:f].T, x @ weights[f:].T
    s = torch.sigmoid(gate)
    if kind == "mlp":
        return _true4((gate * s * up).float()) @ _read4(st["down"], f).T
    dh = st["dh"].double()
    return torch.cat((dh * up * (s + gate * s * (1 - s)), dh * (gate * s)), 1), gate * s * up
