"""Cases that measure the training operators around the convolutions: group norm
with an activation (forward and backward), the norm of all gradients, and the
AdamW step over many tensors.

``run`` computes a case in plain torch (``own`` false) or through the library
(``own`` true) on what ``prepare`` made; ``exact`` gives the same outputs from
the definitions in 64 bits.

Tensors of the optimizer's cases are those of a network of deformable blocks of
width C: per block the convolution's weight [C][C][3][3] and bias [C], its
offset convolution's weight [18][C][3][3] and bias [18], and the group norm's
gamma and beta [C].  They lie in one flat buffer, each tensor's start on a
multiple of 256 elements, as a program keeps them that wants few buffers; the
gaps between tensors are zero and stay zero.
"""
import math

import torch

own = False

BLOCK = 256  # elements that share one scale of an 8-bit state
TINY = 2.0 ** -126


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a first layer's 16 channels at 16x16, one image: a call whose latency counts
        dict(name="norm fwd 1x256x16 f32", op="norm_forward", n=1, s=256, c=16, groups=4, layout="channels_last",
             act="silu", dtype="f32"),
        # behind the deformable layer at its headline shape, which leaves y channels first
        dict(name="norm fwd 16x256x56x56 bf16", op="norm_forward", n=16, s=3136, c=256, groups=32,
             layout="channels_first", act="relu", dtype="bf16"),
        # few large images, channels last
        dict(name="norm fwd 2x65536x320 bf16", op="norm_forward", n=2, s=65536, c=320, groups=32,
             layout="channels_last", act="silu", dtype="bf16"),
        # ragged steps and channels behind the 1-D depthwise convolution
        dict(name="norm fwd 3x1000x36 f32", op="norm_forward", n=3, s=1000, c=36, groups=9, layout="channels_last",
             act="gelu", dtype="f32"),
        # a deep layer's training step, channels last
        dict(name="norm bwd 16x784x512 bf16", op="norm_backward", n=16, s=784, c=512, groups=32,
             layout="channels_last", act="silu", dtype="bf16"),
        # the 1-D convolutions' benchmark shape
        dict(name="norm bwd 32x1024x512 f32", op="norm_backward", n=32, s=1024, c=512, groups=16,
             layout="channels_last", act="gelu", dtype="f32"),
        # the gradient that the deformable layer's backward takes as dy
        dict(name="norm bwd 16x256x56x56 bf16", op="norm_backward", n=16, s=3136, c=256, groups=32,
             layout="channels_first", act="relu", dtype="bf16"),
        # one narrow block in f32: latency
        dict(name="adamw f32 1 block of 16", op="adamw", blocks=1, c=16, dtype="f32", master=False, bits=32,
             clip=False),
        # bf16 weights with f32 masters, f32 states, gradients clipped: a training step's end
        dict(name="adamw 32 8 blocks of 256", op="adamw", blocks=8, c=256, dtype="bf16", master=True, bits=32,
             clip=True),
        # the same with 8-bit states on a wide network, the largest
        dict(name="adamw 8 8 blocks of 1024", op="adamw", blocks=8, c=1024, dtype="bf16", master=True, bits=8,
             clip=True),
        # the gradients of one block, and of the wide network
        dict(name="grad norm 1 block of 256", op="grad_norm", blocks=1, c=256, dtype="bf16"),
        dict(name="grad norm 8 blocks of 1024", op="grad_norm", blocks=8, c=1024, dtype="bf16"),
    ]


def _spread(rng, low, high):
    """A whole number from low to high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "adamw", "grad_norm"])
    if op.startswith("norm"):
        per, groups = _spread(rng, 1, 40), _spread(rng, 1, 48)
        c, n = per * groups, _spread(rng, 1, 32)
        most = 2 * 65536 * 320
        s = _spread(rng, 1, max(1, min(70000, most // (n * c))))
        if op == "norm_backward":
            s = max(s, -(-8 // per))  # the gradient of two values is a difference that f32 does not hold
        return dict(op=op, n=n, s=s, c=c, groups=groups, layout=rng.choice(["channels_last", "channels_first"]),
                    act=rng.choice(["none", "relu", "silu", "gelu"]), dtype=rng.choice(["f32", "bf16"]))
    blocks, c = rng.randint(1, 8), 16 * _spread(rng, 1, 64)
    dtype = rng.choice(["f32", "bf16"])
    if op == "grad_norm":
        return dict(op=op, blocks=blocks, c=c, dtype=dtype)
    case = dict(op=op, blocks=blocks, c=c, dtype=dtype, master=dtype == "bf16" and rng.random() < 0.5,
                bits=rng.choice([8, 32]), clip=rng.random() < 0.5)
    while case["blocks"] > 1 and work(case)["bytes"] > 1.2e9:
        case["blocks"] -= 1
    return case


# ---------------------------------------------------------------- inputs

def _sizes(case):
    c = case["c"]
    return [c * c * 9, c, 18 * c * 9, 18, c, c] * case["blocks"]


def _decays(case):
    # weights decay; biases, gamma and beta do not
    return [0.01, 0.0, 0.01, 0.0, 0.0, 0.0] * case["blocks"]


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _norm_shape(case):
    n, s, c = case["n"], case["s"], case["c"]
    return (n, s, c) if case["layout"] == "channels_last" else (n, c, s)


def _prepare_norm(case, rand, dev):
    n, c, g = case["n"], case["c"], case["groups"]
    last = case["layout"] == "channels_last"
    per_channel = (1, 1, c) if last else (1, c, 1)
    x = rand(_norm_shape(case)) * (0.5 + rand((c,)).abs()).view(per_channel) + 0.5 * rand((c,)).view(per_channel)
    t = _type(case)
    st = dict(x=x.to(t), gamma=(1 + 0.2 * rand((c,))).to(t), beta=(0.2 * rand((c,))).to(t))
    del x
    if case["op"] == "norm_backward":
        st["dy"] = rand(_norm_shape(case)).to(t)
        # what the forward left: the groups' mean and 1/std, in f32
        xg = st["x"].view((n, -1, g, c // g) if last else (n, g, -1, 1))
        dims = (1, 3) if last else (2, 3)
        var, mean = torch.var_mean(xg.float(), dim=dims, correction=0)
        st["mean"], st["rstd"] = mean.contiguous(), torch.rsqrt(var + 1e-5)
    if own:
        from irregular_gather_cnn_amd.norm import GroupNormAct
        st["handle"] = GroupNormAct(n, c, case["s"], g, eps=1e-5, act=case["act"], layout=case["layout"],
                                    dtype=case["dtype"], training=True, device=dev)
    return st


def _prepare_tensors(case, rand, dev):
    sizes, t = _sizes(case), _type(case)
    starts, total = [], 0
    for k in sizes:
        starts.append(total)
        total += -(-k // BLOCK) * BLOCK
    per = [-(-k // BLOCK) for k in sizes]
    nb = total // BLOCK
    # for every block of 256 elements: its tensor, its place in it, and that tensor's decay
    tensor = torch.repeat_interleave(torch.arange(len(sizes)), torch.tensor(per)).view(nb, 1).to(dev)
    first = torch.cat([torch.arange(k) * BLOCK for k in per]).view(nb, 1).to(dev)
    size = torch.tensor(sizes, device=dev)[tensor]
    inside = (first + torch.arange(BLOCK, device=dev) < size).view(-1)
    decay = torch.tensor(_decays(case), dtype=torch.float64, device=dev)[tensor]

    def views(flat):
        return [flat[a:a + k] for a, k in zip(starts, sizes)]

    st = dict(tensor=tensor, first=first, decay=decay)
    st["g"] = (rand((total,)) * 1e-3 * inside).to(t)
    st["grads"] = views(st["g"])
    if case["op"] == "adamw":
        p = rand((total,)) * math.sqrt(2.0 / (9 * case["c"])) * inside
        st["p"] = p.to(t)
        if case["master"]:
            st["master"] = p
        if case["bits"] == 32:
            st["m"] = rand((total,)) * 3e-4 * inside
            st["v"] = (1e-3 * (0.3 + rand((total,)).abs())).square() * inside
        else:
            # states of a run in progress: codes in e4m3, one scale for each block, v by its root
            st["m"] = ((rand((total,)) * 120).clamp(-448, 448) * inside).to(torch.float8_e4m3fn)
            st["v"] = ((60 + rand((total,)).abs() * 120).clamp(0, 448) * inside).to(torch.float8_e4m3fn)
            st["m_scale"] = 2.5e-6 * (1 + 0.2 * rand((nb,)).abs())
            st["v_scale"] = 6e-6 * (1 + 0.2 * rand((nb,)).abs())
    if case["op"] == "adamw":
        st["step"] = 100
    if own:
        from irregular_gather_cnn_amd.optim import AdamW, GradNorm
        if case["op"] == "grad_norm":
            st["handle"] = GradNorm(st["grads"])
        else:
            scales = [[st[k][a // BLOCK:a // BLOCK + n] if k in st else None for a, n in zip(starts, per)]
                      for k in ("m_scale", "v_scale")]
            st["handle"] = AdamW(views(st["p"]), st["grads"], bits=case["bits"], weight_decay=_decays(case),
                                 masters=views(st["master"]) if case["master"] else None, step=100, seed=SEED,
                                 states=list(zip(views(st["m"]), views(st["v"]), *scales)), **HYPER)
    return st


HYPER = dict(lr=1e-4, betas=(0.9, 0.999), eps=1e-8)
SEED = 17
MAX_NORM, INV_SCALE = 0.25, 1.0


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed)

    def rand(shape):
        return torch.randn(shape, generator=gen, device=dev)

    st = (_prepare_norm if case["op"].startswith("norm") else _prepare_tensors)(case, rand, dev)
    st["case"] = dict(case)
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        h = state["handle"]
        if op == "norm_forward":
            y, mean, rstd = h.forward(state["x"], state["gamma"], state["beta"])
            return dict(y=y, mean=mean, rstd=rstd)
        if op == "norm_backward":
            return h.backward(state["x"], state["gamma"], state["beta"], state["mean"], state["rstd"], state["dy"])
        if op == "grad_norm":
            control = h(max_norm=MAX_NORM, inv_scale=INV_SCALE)
            return dict(norm=control[0], coef=control[1])
        control = None
        if state["case"]["clip"]:
            control = h.grad_norm(max_norm=MAX_NORM, inv_scale=INV_SCALE)
        h.step(control=control)
        return _updated(state, control)
    if op == "norm_forward":
        return _plain_norm_forward(state)
    if op == "norm_backward":
        return _plain_norm_backward(state)
    if op == "grad_norm":
        control = _plain_grad_norm(state["g"])
        return dict(norm=control[0], coef=control[1])
    return _plain_adamw(state)


def _updated(state, control):
    out = {k: state[k] for k in ("p", "master", "m", "v", "m_scale", "v_scale") if k in state}
    if control is not None:
        out["norm"], out["coef"] = control[0], control[1]
    return out


# ---------------------------------------------------------------- plain forms

def _grouped(case, t):
    """A view [n][s][g][c/g] or [n][g][c/g][s], what is summed over, and the shapes that broadcast a
    group's and a channel's value over it."""
    n, s, c, g = case["n"], case["s"], case["c"], case["groups"]
    if case["layout"] == "channels_last":
        return t.view(n, s, g, c // g), (1, 3), (n, 1, g, 1), (1, 1, g, c // g), (0, 1)
    return t.view(n, g, c // g, s), (2, 3), (n, g, 1, 1), (1, g, c // g, 1), (0, 3)


def _act(act, z):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(act, z):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * (math.sqrt(0.5 / math.pi) * torch.exp(-0.5 * z * z))
    return torch.ones_like(z)


def _plain_norm_forward(st):
    case = st["case"]
    x, over, per_group, per_channel, _ = _grouped(case, st["x"].float())
    mean = x.mean(over)
    d = x - mean.view(per_group)
    rstd = 1 / torch.sqrt((d * d).mean(over) + 1e-5)
    z = d * rstd.view(per_group) * st["gamma"].float().view(per_channel) + st["beta"].float().view(per_channel)
    return dict(y=_act(case["act"], z).view(st["x"].shape).to(st["x"].dtype), mean=mean, rstd=rstd)


def _plain_norm_backward(st):
    case = st["case"]
    x, over, per_group, per_channel, over_channel = _grouped(case, st["x"].float())
    gamma, rstd = st["gamma"].float().view(per_channel), st["rstd"].view(per_group)
    h = (x - st["mean"].view(per_group)) * rstd
    dz = st["dy"].float().view(x.shape) * _act_slope(case["act"], h * gamma + st["beta"].float().view(per_channel))
    dbeta, dgamma = dz.sum(over_channel).view(-1), (dz * h).sum(over_channel).view(-1)
    dh = dz * gamma
    dx = rstd * (dh - dh.mean(over).view(per_group) - h * (dh * h).mean(over).view(per_group))
    t = st["x"].dtype
    return dict(dx=dx.view(st["x"].shape).to(t), dgamma=dgamma.to(t), dbeta=dbeta.to(t))


def _plain_grad_norm(g):
    # 64 bits: a long sum
    norm = g.double().square().sum().sqrt() * INV_SCALE
    coef = INV_SCALE * (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
    return torch.stack([norm, coef]).float()


def _mix(x):
    """A 32-bit integer hash, on int64 tensors or ints."""
    x = x ^ (x >> 16)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _rounding_bits(st, seed):
    """The 16 random bits that round element i of a tensor: one half of a hash of its pair i / 2."""
    key = _mix((seed + st["tensor"] * 0x3C6EF373) & 0xFFFFFFFF)
    i = st["first"] + torch.arange(BLOCK, device=key.device)
    h = _mix(((i >> 1) * 0x6A09E667 + key) & 0xFFFFFFFF)
    return (h >> (16 * (i & 1))) & 0xFFFF


def _step_seed(step):
    return (SEED + step * 0x9E3779B9) & 0xFFFFFFFF


def _scales(a):
    """The scale of each block, a[blocks][256] >= 0, and its inverse (0 where the block holds nothing)."""
    most = a.amax(1, keepdim=True)
    s = most / 448
    s = torch.where(s >= TINY, s, torch.zeros_like(s))
    return s, torch.where(s > 0, 1 / s, torch.zeros_like(s))


def _plain_adamw(st):
    case = st["case"]
    b1, b2 = HYPER["betas"]
    st["step"] += 1
    step = st["step"]
    control = _plain_grad_norm(st["g"]) if case["clip"] else None
    g = st["g"].float()
    if control is not None:
        g = g * control[1]
    g = g.view(-1, BLOCK)
    if case["bits"] == 32:
        m, v = st["m"].view(-1, BLOCK), st["v"].view(-1, BLOCK)
    else:
        m = st["m"].float().view(-1, BLOCK) * st["m_scale"].view(-1, 1)
        v = st["v"].float().view(-1, BLOCK) * st["v_scale"].view(-1, 1)
        v = v * v
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    root = torch.sqrt(v)
    low, rate = 1 / math.sqrt(1 - b2 ** step), HYPER["lr"] / (1 - b1 ** step)
    p = (st["master"] if case["master"] else st["p"].float()).view(-1, BLOCK)
    p = p * (1 - HYPER["lr"] * st["decay"]).float() - (m / (root * low + HYPER["eps"])) * rate
    st["p"].copy_(p.view(-1))
    if case["master"]:
        st["master"].copy_(p.view(-1))
    if case["bits"] == 32:
        st["m"].copy_(m.view(-1))
        st["v"].copy_(v.view(-1))
        return _updated(st, control)
    s, inv = _scales(m.abs())
    st["m"].copy_((m * inv).clamp(-448, 448).to(torch.float8_e4m3fn).view(-1))
    st["m_scale"].copy_(s.view(-1))
    s, inv = _scales(root)
    st["v_scale"].copy_(s.view(-1))
    t = (root * inv).clamp(max=448.0)
    u = _rounding_bits(st, _step_seed(step)).to(torch.int32)
    # e4m3 keeps the upper 3 of 23 fraction bits: a random number is added below them and the rest is cut
    # off; under 2^-6 the code's step is 2^-9 throughout.  What is not zero stays at least the least code.
    normal = ((t.view(torch.int32) + (u * 16 + 8)) & -0x100000).view(torch.float32)
    small = torch.floor(t * 512 + (u.float() + 0.5) * 2.0 ** -16) / 512
    q = torch.where(t < 2.0 ** -6, torch.where(t > 0, small.clamp(min=2.0 ** -9), small), normal)
    st["v"].copy_(q.to(torch.float8_e4m3fn).view(-1))
    return _updated(st, control)


# ---------------------------------------------------------------- work

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("norm"):
        e = case["n"] * case["s"] * case["c"]
        back = case["op"] == "norm_backward"
        return dict(bytes=e * size * (3 if back else 2), flops=e * (20 if back else 10))
    e = sum(_sizes(case))
    if case["op"] == "grad_norm":
        return dict(bytes=e * size, flops=2 * e)
    states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    # a weight that has a master is only written
    weights = 8 + size if case["master"] else 2 * size
    return dict(bytes=int(e * (size + weights + states)), flops=e * (16 if case["clip"] else 14))


# ---------------------------------------------------------------- 64 bits

def _exact_norm(case, st):
    n, s, c, g = case["n"], case["s"], case["c"], case["groups"]
    last = case["layout"] == "channels_last"
    act = case["act"]

    def slabs(t):
        t = t.double()
        return (t.transpose(1, 2) if last else t).reshape(n, g, -1)

    def back(t):
        t = t.reshape(n, c, s)
        return (t.transpose(1, 2) if last else t).contiguous()

    def channels(t):
        return t.double().repeat_interleave(s).view(1, g, -1)

    x, gamma, beta = slabs(st["x"]), channels(st["gamma"]), channels(st["beta"])
    if case["op"] == "norm_forward":
        mean = x.sum(2) / x.shape[2]
        rstd = ((x - mean[:, :, None]).pow(2).sum(2) / x.shape[2] + 1e-5).pow(-0.5)
    else:
        mean, rstd = st["mean"].double(), st["rstd"].double()
    h = (x - mean[:, :, None]) * rstd[:, :, None]
    z = h * gamma + beta
    normal = 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if case["op"] == "norm_forward":
        y = {"none": lambda: z, "relu": lambda: z * (z > 0), "silu": lambda: z * torch.sigmoid(z),
             "gelu": lambda: z * normal}[act]()
        return dict(y=back(y), mean=mean, rstd=rstd)
    slope = {"none": lambda: torch.ones_like(z), "relu": lambda: (z > 0).double(),
             "silu": lambda: torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z),
             "gelu": lambda: normal + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)}[act]()
    dz = slabs(st["dy"]) * slope
    dh = dz * gamma
    k = x.shape[2]
    dx = (dh - dh.sum(2, keepdim=True) / k - h * ((dh * h).sum(2, keepdim=True) / k)) * rstd[:, :, None]
    by_channel = lambda t: t.reshape(n, c, s).sum((0, 2))  # noqa: E731
    return dict(dx=back(dx), dgamma=by_channel(dz * h), dbeta=by_channel(dz))


def _exact_norm_of(g):
    total = torch.linalg.vector_norm(g.double()) * INV_SCALE
    return total, INV_SCALE * min(1.0, MAX_NORM / (float(total) + 1e-6))


def _grid(t, up):
    """t on the e4m3 grid: cut off after `up` of a step is added, or to nearest, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(t / step) if up is None else torch.floor(t / step + up)) * step


def _exact_adamw(case, st):
    b1, b2 = HYPER["betas"]
    step = st["step"] + 1
    out = {}
    g = st["g"].double().view(-1, BLOCK)
    if case["clip"]:
        total, coef = _exact_norm_of(st["g"])
        out["norm"], out["coef"] = total, torch.tensor(coef, dtype=torch.float64)
        g = g * coef
    if case["bits"] == 32:
        m, v = st["m"].double().view(-1, BLOCK), st["v"].double().view(-1, BLOCK)
    else:
        m = st["m"].double().view(-1, BLOCK) * st["m_scale"].double().view(-1, 1)
        v = (st["v"].double().view(-1, BLOCK) * st["v_scale"].double().view(-1, 1)) ** 2
    m = m + (1 - b1) * (g - m)
    v = v + (1 - b2) * (g * g - v)
    p = (st["master"] if case["master"] else st["p"]).double().view(-1, BLOCK)
    hat_m, hat_v = m / (1 - b1 ** step), v / (1 - b2 ** step)
    p = p - HYPER["lr"] * (hat_m / (hat_v.sqrt() + HYPER["eps"]) + st["decay"] * p)
    out["p"] = p.view(-1)
    if case["master"]:
        out["master"] = p.view(-1)
    if case["bits"] == 32:
        out["m"], out["v"] = m.view(-1), v.view(-1)
        return out
    for key, a in (("m", m), ("v", v.sqrt())):
        s = a.abs().amax(1, keepdim=True) / 448
        t = torch.where(s > 0, a / s, torch.zeros_like(a)).clamp(-448, 448)
        if key == "m":
            q = _grid(t, None)
        else:
            q = _grid(t, (_rounding_bits(st, _step_seed(step)).double() + 0.5) / 65536)
            q = torch.where(t > 0, q.clamp(min=2.0 ** -9), q)
        out[key], out[key + "_scale"] = q.view(-1), s.view(-1)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, st)
    if case["op"] == "grad_norm":
        total, coef = _exact_norm_of(st["g"])
        return dict(norm=total, coef=torch.tensor(coef, dtype=torch.float64))
    return _exact_adamw(case, st)
