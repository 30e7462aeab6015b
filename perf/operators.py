"""The gated feed-forward block and the many-tensor AdamW step, as cases to time.

Each case is one call (or the few calls that belong together) of an operator
on inputs like those of a training or serving step of an FP8 MLP block:

* ``gated_fwd``   h = act(x Wg^T) * (x Wu^T) from E4M3 operands, h as E4M3 codes
                  or bf16, its amax and, for training, the pre-activations;
* ``gated_bwd``   from dh: the E5M2 gradients of both pre-activations, dX, dW;
* ``gated_dgrad`` from the E5M2 gradient of the block's output, through the down
                  projection, the E5M2 gradients of both pre-activations;
* ``few``         y = x W^T (+ b) for a few tokens (the down projection when serving);
* ``norm``        global gradient norm and overflow flag over many tensors;
* ``adamw``       AdamW over many tensors, states in 32 bits, in 8 bits or both.

``run`` computes a case with the library (``own`` true) or in plain torch
operations in fp32, rounded once at the end.
"""

import math
import random

import torch

own = False

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
BLOCK = 256  # elements that share a scale in the 8-bit states
LEVELS_V = 4228250624.0  # 255^4 in fp32
LR, BETA1, BETA2, EPS = 3e-4, 0.9, 0.95, 1e-8
INTERVAL = 2000


def listed():
    return [
        # one token through the gate and up projections of the 4096 -> 14336 MLP: serving, bound by the weights
        dict(name="fwd 1 token", kind="gated_fwd", M=1, K=4096, F=14336, act="silu", h="e4m3", gu=False),
        # the smallest call: five tokens of a small layer, ragged in every size; latency
        dict(name="fwd 5 tokens small", kind="gated_fwd", M=5, K=768, F=2064, act="gelu", h="bf16", gu=False),
        # the MLP's training batch, pre-activations kept for the backward pass
        dict(name="fwd train", kind="gated_fwd", M=16384, K=4096, F=14336, act="silu", h="e4m3", gu=True),
        # backward of a ragged batch of a small GELU layer from an fp32 gradient
        dict(name="bwd ragged", kind="gated_bwd", M=1237, K=1040, F=2736, act="gelu", dh="f32"),
        # backward of the MLP's gate and up projections at half the training batch
        dict(name="bwd train", kind="gated_bwd", M=8192, K=4096, F=14336, act="silu", dh="bf16"),
        # the same batch's gradient through the down projection and the gate
        dict(name="dgrad train", kind="gated_dgrad", M=8192, N=4096, F=14336, act="silu"),
        # one token through the down projection
        dict(name="few 1 token", kind="few", M=1, K=14336, N=4096, y="bf16", bias=False),
        # a small batch of sequences, odd sizes, with a bias
        dict(name="few 33 tokens", kind="few", M=33, K=1552, N=6000, y="bf16", bias=True),
        # gradient clipping: the norm over one transformer block's weights
        dict(name="norm block", kind="norm", set="block", grad="bf16"),
        # the optimizer step of one transformer block, fp32 moments, E4M3 weight copies
        dict(name="adamw block 32", kind="adamw", set="block", bits="32", grad="bf16", copy="e4m3", clip=1.0),
        # the same with 8-bit moments
        dict(name="adamw block 8", kind="adamw", set="block", bits="8", grad="bf16", copy="e4m3", clip=0.05),
        # many small tensors of odd sizes, both kinds of moments, fp32 gradients: latency
        dict(name="adamw small odd", kind="adamw", set="odd", tensors=61, largest=60000, pick=7, bits="mixed",
             grad="f32", copy="bf16", clip=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log16(rng, lo, hi):
    n = 16 * _log(rng, lo // 16, hi // 16)
    return n + 16 if n == 3072 else n


def draw(rng):
    kind = rng.choice(["gated_fwd", "gated_fwd", "gated_bwd", "gated_dgrad", "few", "norm", "adamw", "adamw"])
    if kind == "gated_fwd":
        M = _log(rng, 1, 64) if rng.random() < 0.5 else _log(rng, 65, 6000)
        return dict(kind=kind, M=M, K=_log16(rng, 64, 4800), F=_log16(rng, 64, 12000),
                    act=rng.choice(["silu", "gelu"]), h=rng.choice(["e4m3", "bf16"]), gu=rng.random() < 0.5)
    if kind == "gated_bwd":
        return dict(kind=kind, M=_log(rng, 1, 4000), K=_log16(rng, 64, 4800), F=_log16(rng, 64, 8000),
                    act=rng.choice(["silu", "gelu"]), dh=rng.choice(["bf16", "f32"]))
    if kind == "gated_dgrad":
        return dict(kind=kind, M=_log(rng, 1, 5000), N=_log16(rng, 64, 4800), F=_log16(rng, 64, 10000),
                    act=rng.choice(["silu", "gelu"]))
    if kind == "few":
        return dict(kind=kind, M=_log(rng, 1, 64), K=_log16(rng, 64, 14336), N=_log16(rng, 64, 14336),
                    y=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5)
    case = dict(kind=kind, set="odd", tensors=_log(rng, 1, 300), largest=_log(rng, 100, 3000000),
                pick=rng.randrange(1 << 20), grad=rng.choice(["bf16", "f32"]))
    if kind == "adamw":
        case.update(bits=rng.choice(["32", "8", "mixed"]), copy=rng.choice(["e4m3", "bf16", "none"]),
                    clip=rng.choice([0.0, 0.01, 10.0]))
    return case


# ------------------------------------------------------------------ inputs


def _sizes(case):
    if case["set"] == "block":  # QKV, attention output, gate and up, down, and the two norms' weights
        return [12288 * 4096, 4096 * 4096, 2 * 14336 * 4096, 4096 * 14336, 4096, 4096]
    rng = random.Random(case["pick"])
    return [_log(rng, 1, case["largest"]) for _ in range(case["tensors"])]


def _groups(case):
    """Ordinals of the tensors with 32-bit and with 8-bit moments: the first go first."""
    n = len(_sizes(case))
    bits = case.get("bits", "32")
    n32 = n if bits == "32" else 0 if bits == "8" else (n + 1) // 2
    return list(range(n32)), list(range(n32, n))


def _cast(x, dtype):
    top = 448.0 if dtype is E4M3 else 57344.0
    return x.clamp(-top, top).to(dtype)


def _codes(shape, std, scale, dtype, gen):
    """Codes of normal values under `scale`, and the factor that undoes it."""
    x = torch.randn(shape, generator=gen, device="cuda") * std
    return _cast(x * scale, dtype).view(torch.uint8), torch.tensor([1.0 / scale], device="cuda")


def _one(v, dtype=torch.float32):
    return torch.tensor([v], dtype=dtype, device="cuda")


def _prepare_mlp(case, gen):
    kind, M, s = case["kind"], case["M"], dict(case=case)
    bf16, u8, dev = torch.bfloat16, torch.uint8, "cuda"
    if kind == "few":
        K, N = case["K"], case["N"]
        s["x8"], s["sinv_x"] = _codes((M, K), 1.0, 64.0, E4M3, gen)
        s["w8"], s["sinv_w"] = _codes((N, K), 0.02, 4096.0, E4M3, gen)
        s["bias"] = torch.randn(N, generator=gen, device=dev) * 0.1 if case["bias"] else None
        s["y"] = torch.empty((M, N), dtype=bf16 if case["y"] == "bf16" else torch.float32, device=dev)
        return s
    F = case["F"]
    if kind in ("gated_fwd", "gated_bwd"):
        K = case["K"]
        s["x8"], s["sinv_x"] = _codes((M, K), 1.0, 64.0, E4M3, gen)
        s["w8"], s["sinv_w"] = _codes((2 * F, K), 0.02, 4096.0, E4M3, gen)
    if kind == "gated_fwd":
        std = 0.02 * math.sqrt(K)
        # a delayed scale: what the last steps' largest |h| asked for, with the odd overflow
        s["h_scale"] = _one(448.0 / (16.0 * std * std)) if case["h"] == "e4m3" else None
        s["h_amax"] = _one(0.0)
        s["h"] = torch.empty((M, F), dtype=u8 if case["h"] == "e4m3" else bf16, device=dev)
        s["gu"] = torch.empty((M, 2 * F), dtype=bf16, device=dev) if case["gu"] else None
        return s
    s["gu"] = torch.randn((M, 2 * F), generator=gen, device=dev, dtype=bf16)
    s["dgu8"] = torch.empty((M, 2 * F), dtype=u8, device=dev)
    s["dgu_amax"] = _one(0.0)
    if kind == "gated_bwd":
        s["dh"] = torch.randn((M, F), generator=gen, device=dev).mul_(1e-4)
        s["dh"] = s["dh"].to(bf16) if case["dh"] == "bf16" else s["dh"]
        s["dgu_scale"], s["dgu_sinv"] = _one(2.0 ** 25), _one(2.0 ** -25)
        s["dx"] = torch.empty((M, K), dtype=bf16, device=dev)
        s["dw"] = torch.empty((2 * F, K), dtype=bf16, device=dev)
        s["nonfinite"] = _one(0, torch.int32)
    else:
        N = case["N"]
        s["dy8"], s["sinv_dy"] = _codes((M, N), 1e-4, 2.0 ** 25, E5M2, gen)
        s["wd8"], s["sinv_wd"] = _codes((N, F), 0.02, 4096.0, E4M3, gen)
        s["dgu_scale"] = _one(2.0 ** 25)
    return s


def _padded(n):
    return (n + BLOCK - 1) // BLOCK * BLOCK


def _encode_moments(m, v):
    """Nearest codes of fp32 moments [blocks, BLOCK] and their blocks' scales."""
    sm = m.abs().amax(1) / 16129.0
    sv = v.amax(1) / LEVELS_V
    cm = (m.abs() / sm.clamp_min(1e-37)[:, None]).sqrt().round().clamp_max(127) * m.sign()
    cv = (v / sv.clamp_min(1e-37)[:, None]).sqrt().sqrt().round().clamp(0, 255)
    cv = torch.where(v > 0, cv.clamp_min(1), cv)
    return cm.to(torch.int8), cv.to(torch.uint8), sm, sv


def _prepare_tensors(case, gen):
    """Every tensor's arrays lie one after another in flat buffers, each from a
    multiple of BLOCK elements on; what is between them is zero."""
    dev, sizes, loss_scale = "cuda", _sizes(case), 65536.0
    grad_dtype = torch.bfloat16 if case["grad"] == "bf16" else torch.float32
    s = dict(case=case, groups=[])
    total = 0
    for bits, ordinals in zip((32, 8), _groups(case)):
        if not ordinals:
            continue
        n = torch.tensor([sizes[t] for t in ordinals])
        blocks = (n + BLOCK - 1) // BLOCK
        first = torch.cumsum(blocks, 0) - blocks
        nb = int(blocks.sum())
        total += int(n.sum())
        which = torch.repeat_interleave(torch.arange(len(ordinals)), blocks).to(dev)  # a block's tensor, within the group
        start = (torch.arange(nb, device=dev) - first.to(dev)[which]) * BLOCK       # its first element, within the tensor
        alive = start[:, None] + torch.arange(BLOCK, device=dev) < n.to(dev)[which][:, None]
        rand = lambda std: torch.randn((nb, BLOCK), generator=gen, device=dev).mul_(std).mul_(alive)  # noqa: E731
        g = dict(bits=bits, which=which, start=start, ordinal=which + ordinals[0], count=len(ordinals),
                 grad=rand(1e-5 * loss_scale).to(grad_dtype))
        s["groups"].append(g)
        g["sizes"], g["first"] = [sizes[t] for t in ordinals], (first * BLOCK).tolist()
        if case["kind"] == "norm":
            continue
        g["master"] = rand(0.02)
        m, v = rand(3e-6), rand(1e-5).square_() * 0.7 + alive * 3e-11
        if bits == 8:
            g["m"], g["v"], g["sm"], g["sv"] = _encode_moments(m, v)
        else:
            g["m"], g["v"] = m, v
        decay = torch.where(n > 8192, 0.1, 0.0).to(torch.float32)  # matrices decay, the norms' weights do not
        g["decay"], g["block_decay"] = decay.tolist(), decay.to(dev)[which]
        g["copy"], g["copy_scale"], g["amax"] = None, None, None
        if case["copy"] == "e4m3":
            g["copy"] = torch.zeros((nb, BLOCK), dtype=torch.uint8, device=dev)
            g["copy_scale"] = torch.full((len(ordinals),), 2048.0, device=dev)
            g["amax"] = torch.zeros(len(ordinals), device=dev)
        elif case["copy"] == "bf16":
            g["copy"] = torch.zeros((nb, BLOCK), dtype=torch.bfloat16, device=dev)
    s["norm"] = _one(0.0)
    s["found"] = _one(0, torch.int32)
    if case["kind"] == "adamw":
        # the norm of the (loss-scaled) gradients, and a clip as a multiple of what it usually is
        s["norm"].fill_(1e-5 * loss_scale * math.sqrt(total))
        s["max_norm"] = case["clip"] * 1e-5 * math.sqrt(total)
        s["loss_scale"], s["growth"] = _one(loss_scale), _one(3, torch.int32)
        s["beta_pows"] = torch.tensor([BETA1 ** 10, BETA2 ** 10], device=dev)
        s["seed"] = torch.randint(-2 ** 31, 2 ** 31, (1,), generator=gen, device=dev).to(torch.int32)
    if own:
        s["plan"], s["workspace"] = _plan(s)
    return s


def _plan(s):
    import fp8_mixed_precision_reduce_gb300 as fp8mp

    plan = fp8mp.AdamWTensors()
    for g in s["groups"]:
        flat = {k: g[k].reshape(-1) for k in ("grad", "master", "m", "v", "copy") if g.get(k) is not None}
        for t, (n, at) in enumerate(zip(g["sizes"], g["first"])):
            part = {k: x[at:at + n] for k, x in flat.items()}
            if s["case"]["kind"] == "norm":
                plan.add(part["grad"])
                continue
            of = slice(at // BLOCK, (at + _padded(n)) // BLOCK)
            eight = dict(exp_avg_scale=g["sm"][of], exp_avg_sq_scale=g["sv"][of]) if g["bits"] == 8 else {}
            scaled = dict(copy_scale=g["copy_scale"][t:], copy_amax=g["amax"][t:]) if g["amax"] is not None else {}
            plan.add(part["grad"], part["master"], part["m"], part["v"], copy=part.get("copy"),
                     weight_decay=g["decay"][t], **eight, **scaled)
    return plan, torch.zeros(fp8mp.mp_adamw_workspace_bytes() // 4, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    make = _prepare_tensors if case["kind"] in ("norm", "adamw") else _prepare_mlp
    return make(case, gen)


# ------------------------------------------------------------- plain forms


def _act(g, act):
    if act == "silu":
        return g * (1.0 / (1.0 + torch.exp(-g)))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(g, act):
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return sig * (1.0 + g * (1.0 - sig))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _value(codes, dtype):
    return codes.view(dtype).float()


def _plain_gated_fwd(s):
    case, F = s["case"], s["case"]["F"]
    pre = (_value(s["x8"], E4M3) @ _value(s["w8"], E4M3).T) * (s["sinv_x"] * s["sinv_w"])
    h = _act(pre[:, :F], case["act"]) * pre[:, F:]
    s["h_amax"].copy_(torch.maximum(s["h_amax"], h.abs().max()))
    if s["h_scale"] is not None:
        s["h"].copy_(_cast(h * s["h_scale"], E4M3).view(torch.uint8))
    else:
        s["h"].copy_(h)
    if s["gu"] is not None:
        s["gu"].copy_(pre)


def _plain_gate_back(s, dh):
    case, F = s["case"], s["case"]["F"]
    gu = s["gu"].float()
    g, u = gu[:, :F], gu[:, F:]
    dgu = torch.cat([dh * u * _act_grad(g, case["act"]), dh * _act(g, case["act"])], 1)
    s["dgu_amax"].copy_(torch.maximum(s["dgu_amax"], dgu.abs().max()))
    s["dgu8"].copy_(_cast(dgu * s["dgu_scale"], E5M2).view(torch.uint8))


def _plain_gated_bwd(s):
    _plain_gate_back(s, s["dh"].float())
    dgu = _value(s["dgu8"], E5M2)
    s["dx"].copy_((dgu @ _value(s["w8"], E4M3)) * (s["dgu_sinv"] * s["sinv_w"]))
    s["dw"].copy_((dgu.T @ _value(s["x8"], E4M3)) * (s["dgu_sinv"] * s["sinv_x"]))
    bad = torch.logical_not(torch.isfinite(s["dw"])).any()
    s["nonfinite"].copy_(torch.maximum(s["nonfinite"], bad.to(torch.int32)))


def _plain_gated_dgrad(s):
    _plain_gate_back(s, (_value(s["dy8"], E5M2) @ _value(s["wd8"], E4M3)) * (s["sinv_dy"] * s["sinv_wd"]))


def _plain_few(s):
    y = (_value(s["x8"], E4M3) @ _value(s["w8"], E4M3).T) * (s["sinv_x"] * s["sinv_w"])
    s["y"].copy_(y if s["bias"] is None else y + s["bias"])


def _sum_squares(g):
    x = g["grad"].float()
    return torch.sum(x * x)


def _plain_norm(s):
    total = torch.stack([_sum_squares(g) for g in s["groups"]]).sum()
    s["norm"].copy_(torch.sqrt(total))
    s["found"].copy_(torch.logical_not(torch.isfinite(total)).to(torch.int32))


def _mix(x):
    """A 32-bit finalizer: xor-shifts and odd multiplies, on int64 tensors."""
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random16(g, seed):
    """Two 16-bit uniform numbers in [0, 1) for each element, from the seed and its place."""
    key = _mix((seed.to(torch.int64) + (g["ordinal"] + 1) * 0x9E3779B9) & 0xFFFFFFFF)
    i = g["start"][:, None] + torch.arange(BLOCK, device=key.device)
    h = _mix((key[:, None] + (i & 0xFFFFFFFF) + (i >> 32) * 0x85EBCA77) & 0xFFFFFFFF)
    return (h & 0xFFFF).float() * 2.0 ** -16, (h >> 16).float() * 2.0 ** -16


def _quantize(y, root, power, top, r):
    """The code below or above y on the grid 0, 1, 2^power, .., top^power, so that its mean is y."""
    c = root(y).floor().clamp_max(top)
    c = torch.where(power(c + 1.0) <= y, c + 1.0, c)
    c = torch.where(power(c) > y, c - 1.0, c).clamp_max(top)
    lo = power(c)
    up = r * (power(c + 1.0) - lo) < y - lo
    return torch.where(up, c + 1.0, c).clamp_max(top)


def _square(c):
    return c * c


def _fourth(c):
    return (c * c) * (c * c)


def _plain_adamw_group(s, g):
    one = torch.ones_like(s["loss_scale"])
    inv_s = one / s["loss_scale"]
    coef = inv_s
    if s["max_norm"] > 0:
        clip = torch.full_like(one, s["max_norm"]) / (s["norm"] * inv_s + 1e-6)
        coef = torch.where(clip < 1.0, inv_s * clip, inv_s)
    b1t, b2t = s["beta_pows"][0] * BETA1, s["beta_pows"][1] * BETA2
    u = g["grad"].float() * coef
    if g["bits"] == 8:
        cm, cv = g["m"].float(), g["v"].float()
        m, v = (cm * cm.abs()) * g["sm"][:, None], _fourth(cv) * g["sv"][:, None]
    else:
        m, v = g["m"], g["v"]
    b1 = torch.tensor(BETA1).item()
    b2 = torch.tensor(BETA2).item()
    m = m * b1 + u * (1.0 - b1)
    v = v * b2 + (u * u) * (1.0 - b2)
    step = torch.full_like(one, LR) / (one - b1t)
    root = one / torch.sqrt(one - b2t)
    w = g["master"] * (1.0 - LR * g["block_decay"])[:, None] - step * (m / (torch.sqrt(v) * root + EPS))
    g["master"].copy_(w)
    if g["bits"] == 8:
        rm, rv = _random16(g, s["seed"])
        mmax, vmax = m.abs().amax(1), v.amax(1)
        mmax = torch.where(mmax >= 2.0 ** -100, mmax, torch.zeros_like(mmax))
        vmax = torch.where(vmax >= 2.0 ** -90, vmax, torch.zeros_like(vmax))
        levels_m, levels_v = torch.full_like(mmax, 16129.0), torch.full_like(vmax, LEVELS_V)
        inv_m = torch.where(mmax > 0, levels_m / mmax, torch.zeros_like(mmax))
        inv_v = torch.where(vmax > 0, levels_v / vmax, torch.zeros_like(vmax))
        c = _quantize(m.abs() * inv_m[:, None], torch.sqrt, _square, 127.0, rm)
        g["m"].copy_(torch.where(m < 0, -c, c))
        c = _quantize(v * inv_v[:, None], lambda y: torch.sqrt(torch.sqrt(y)), _fourth, 255.0, rv)
        g["v"].copy_(torch.where((v > 0) & (vmax > 0)[:, None], c.clamp_min(1.0), c))
        g["sm"].copy_(mmax / levels_m)
        g["sv"].copy_(vmax / levels_v)
    else:
        g["m"].copy_(m)
        g["v"].copy_(v)
    if g["copy"] is not None and g["amax"] is not None:
        g["copy"].copy_(_cast(w * g["copy_scale"][g["which"]][:, None], E4M3).view(torch.uint8))
        g["amax"].scatter_reduce_(0, g["which"], w.abs().amax(1), "amax")
    elif g["copy"] is not None:
        g["copy"].copy_(w)
    return b1t, b2t


def _plain_adamw(s):
    # the found flag is an input here, and clear: its skip is a host-free select in the library
    b1t, b2t = [_plain_adamw_group(s, g) for g in s["groups"]][-1]
    s["beta_pows"].copy_(torch.stack([b1t, b2t]))
    grown = s["growth"] + 1 >= INTERVAL
    s["loss_scale"].copy_(torch.where(grown, s["loss_scale"] * 2.0, s["loss_scale"]))
    s["growth"].copy_(torch.where(grown, torch.zeros_like(s["growth"]), s["growth"] + 1))
    s["seed"].add_(1)


_PLAIN = dict(gated_fwd=_plain_gated_fwd, gated_bwd=_plain_gated_bwd, gated_dgrad=_plain_gated_dgrad,
              few=_plain_few, norm=_plain_norm, adamw=_plain_adamw)


# ------------------------------------------------------- the library's calls


def _library(s):
    import fp8_mixed_precision_reduce_gb300 as fp8mp

    case, kind = s["case"], s["case"]["kind"]
    act = {"silu": fp8mp.SILU, "gelu": fp8mp.GELU_TANH}.get(case.get("act"))
    if kind == "gated_fwd":
        fp8mp.fp8_gated_fwd(s["x8"], s["w8"], s["sinv_x"], s["sinv_w"], s["h"], act=act, h_scale=s["h_scale"],
                            h_amax=s["h_amax"], gu=s["gu"])
    elif kind == "gated_bwd":
        fp8mp.fp8_gated_bwd(s["dh"], s["gu"], s["x8"], s["w8"], s["sinv_x"], s["sinv_w"], s["dgu_scale"],
                            s["dgu_sinv"], s["dgu8"], s["dx"], s["dw"], act=act, dgu_amax=s["dgu_amax"],
                            dw_nonfinite=s["nonfinite"])
    elif kind == "gated_dgrad":
        fp8mp.fp8_gated_dgrad(s["dy8"], s["wd8"], s["gu"], s["sinv_dy"], s["sinv_wd"], s["dgu_scale"], s["dgu8"],
                              act=act, dgu_amax=s["dgu_amax"])
    elif kind == "few":
        fp8mp.fp8_linear_few(s["x8"], s["w8"], s["sinv_x"], s["sinv_w"], s["y"], bias=s["bias"])
    elif kind == "norm":
        fp8mp.mp_grad_norm(s["plan"], s["norm"], s["found"], s["workspace"])
    else:
        fp8mp.mp_adamw_step(s["plan"], s["loss_scale"], s["growth"], s["found"], s["beta_pows"], s["workspace"],
                            lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, seed=s["seed"],
                            grad_norm=s["norm"] if s["max_norm"] > 0 else None, max_norm=s["max_norm"],
                            growth_interval=INTERVAL)


def _outputs(s):
    kind = s["case"]["kind"]
    if kind == "gated_fwd":
        h = s["h"].view(E4M3) if s["h_scale"] is not None else s["h"]
        return dict(h=h, amax=s["h_amax"], gu=s["gu"])
    if kind == "gated_bwd":
        return dict(dgu=s["dgu8"].view(E5M2), amax=s["dgu_amax"], dx=s["dx"], dw=s["dw"], nonfinite=s["nonfinite"])
    if kind == "gated_dgrad":
        return dict(dgu=s["dgu8"].view(E5M2), amax=s["dgu_amax"])
    if kind == "few":
        return dict(y=s["y"])
    if kind == "norm":
        return dict(norm=s["norm"], found=s["found"])
    return dict(groups=[_group_outputs(g) for g in s["groups"]], loss_scale=s["loss_scale"], growth=s["growth"],
                beta_pows=s["beta_pows"], seed=s["seed"])


def _group_outputs(g):
    # 8-bit moments: the codes are whole multiples of the block's step in |m|^(1/2) and v^(1/4), with the steps beside them
    out = dict(master=g["master"], m=g["m"], v=g["v"], amax=g["amax"], sm=g.get("sm"), sv=g.get("sv"))
    out["copy"] = g["copy"].view(E4M3) if g["amax"] is not None else g["copy"]
    return out


def run(state):
    if own:
        _library(state)
    else:
        _PLAIN[state["case"]["kind"]](state)
    return _outputs(state)


# --------------------------------------------------------------------- work


def work(case):
    kind = case["kind"]
    if kind == "gated_fwd":
        M, K, F = case["M"], case["K"], case["F"]
        h = 1 if case["h"] == "e4m3" else 2
        return dict(bytes=M * K + 2 * F * K + M * F * h + (4 * M * F if case["gu"] else 0), flops=4 * M * F * K)
    if kind == "gated_bwd":
        M, K, F = case["M"], case["K"], case["F"]
        dh = 2 if case["dh"] == "bf16" else 4
        return dict(bytes=M * F * (dh + 4 + 2) + 3 * M * K + 6 * F * K, flops=8 * M * F * K)
    if kind == "gated_dgrad":
        M, N, F = case["M"], case["N"], case["F"]
        return dict(bytes=M * N + N * F + 6 * M * F, flops=2 * M * F * N)
    if kind == "few":
        M, K, N = case["M"], case["K"], case["N"]
        y = 2 if case["y"] == "bf16" else 4
        return dict(bytes=M * K + N * K + M * N * y + (4 * N if case["bias"] else 0), flops=2 * M * N * K)
    sizes, (g32, g8) = _sizes(case), _groups(case)
    n32, n8 = sum(sizes[t] for t in g32), sum(sizes[t] for t in g8)
    grad = 2 if case["grad"] == "bf16" else 4
    if kind == "norm":
        return dict(bytes=(n32 + n8) * grad, flops=2 * (n32 + n8))
    each = grad + 8 + {"e4m3": 1, "bf16": 2, "none": 0}[case["copy"]]
    return dict(bytes=n32 * (each + 16) + n8 * (each + 4) + 16 * (n8 // BLOCK), flops=20 * n32 + 60 * n8)


# ------------------------------------------------------- 64-bit definitions


def _wide(codes, dtype):
    return codes.view(dtype).to(torch.float64)


def _narrow(x, dtype):
    """The nearest code's value, as 64-bit numbers, saturating."""
    digits, low, top = (3, -6, 448.0) if dtype is E4M3 else (2, -14, 57344.0)
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** low))).clamp_min(low)
    quantum = torch.exp2(e - digits)
    return (torch.round(x / quantum) * quantum).clamp(-top, top)


def _gate64(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        sig = torch.special.expit(g)
        return g * sig, sig + g * sig * (1 - sig)
    c = math.sqrt(2 / math.pi)
    z = c * (g + 0.044715 * g ** 3)
    phi = torch.special.expit(2 * z)  # (1 + tanh z) / 2
    return g * phi, phi + g * 2 * phi * (1 - phi) * c * (1 + 3 * 0.044715 * g * g)


def _exact_gate_back(case, s, dh):
    F = case["F"]
    g, u = s["gu"][:, :F].double(), s["gu"][:, F:].double()
    a, da = _gate64(g, case["act"])
    del g
    dgu = torch.empty((dh.shape[0], 2 * F), dtype=torch.float64, device=dh.device)
    dgu[:, :F] = dh * u * da
    dgu[:, F:] = dh * a
    amax = dgu.abs().max().reshape(1)
    return _narrow(dgu * s["dgu_scale"].double(), E5M2), amax


def _exact_adamw(case, s):
    groups = []
    inv_s = 1.0 / s["loss_scale"].double()
    coef = inv_s
    if s["max_norm"] > 0:
        coef = inv_s * (s["max_norm"] / (s["norm"].double() * inv_s + 1e-6)).clamp_max(1.0)
    pows = s["beta_pows"].double() * torch.tensor([BETA1, BETA2], dtype=torch.float64, device="cuda")
    for g in s["groups"]:
        u = g["grad"].double() * coef
        m, v = g["m"].double(), g["v"].double()
        if g["bits"] == 8:
            m, v = m.abs() * m * g["sm"].double()[:, None], v ** 4 * g["sv"].double()[:, None]
        m = BETA1 * m + (1 - BETA1) * u
        v = BETA2 * v + (1 - BETA2) * u * u
        del u
        w = g["master"].double() * (1 - LR * g["block_decay"].double())[:, None]
        w -= LR * (m / (1 - pows[0])) / (torch.sqrt(v / (1 - pows[1])) + EPS)
        out = dict(master=w, m=m, v=v, amax=None, sm=None, sv=None, copy=None)
        if g["bits"] == 8:
            out.update(m=None, v=None, sm=m.abs().amax(1) / 127 ** 2, sv=v.amax(1) / 255 ** 4)
        if g["amax"] is not None:
            out["amax"] = torch.stack([w[g["which"] == t].abs().max() for t in range(g["count"])])
            out["copy"] = _narrow(w * g["copy_scale"].double()[g["which"]][:, None], E4M3)
        elif g["copy"] is not None:
            out["copy"] = w
        groups.append(out)
    return dict(groups=groups, loss_scale=None, growth=None, beta_pows=pows, seed=None)


def exact(case, seed):
    s, kind = prepare(case, seed), case["kind"]
    if kind == "adamw":
        return _exact_adamw(case, s)
    if kind == "norm":
        total = sum(float(g["grad"].double().square().sum()) for g in s["groups"])
        return dict(norm=torch.tensor([math.sqrt(total)], dtype=torch.float64), found=None)
    if kind == "few":
        y = (_wide(s["x8"], E4M3) @ _wide(s["w8"], E4M3).T) * (s["sinv_x"].double() * s["sinv_w"].double())
        return dict(y=y if s["bias"] is None else y + s["bias"].double())
    if kind == "gated_fwd":
        F = case["F"]
        pre = _wide(s["x8"], E4M3) @ _wide(s["w8"], E4M3).T
        pre *= s["sinv_x"].double() * s["sinv_w"].double()
        h = _gate64(pre[:, :F], case["act"])[0] * pre[:, F:]
        amax = h.abs().max().reshape(1)
        if s["h_scale"] is None:
            return dict(h=h, amax=amax, gu=pre if s["gu"] is not None else None)
        return dict(h=_narrow(h * s["h_scale"].double(), E4M3), amax=amax, gu=pre if s["gu"] is not None else None)
    if kind == "gated_dgrad":
        dh = _wide(s["dy8"], E5M2) @ _wide(s["wd8"], E4M3)
        dh *= s["sinv_dy"].double() * s["sinv_wd"].double()
        dgu, amax = _exact_gate_back(case, s, dh)
        return dict(dgu=dgu, amax=amax)
    dgu, amax = _exact_gate_back(case, s, s["dh"].double())
    dx = (dgu @ _wide(s["w8"], E4M3)) * (s["dgu_sinv"].double() * s["sinv_w"].double())
    dw = (dgu.T @ _wide(s["x8"], E4M3)) * (s["dgu_sinv"].double() * s["sinv_x"].double())
    return dict(dgu=dgu, amax=amax, dx=dx, dw=dw, nonfinite=None)
