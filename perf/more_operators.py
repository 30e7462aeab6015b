"""What surrounds the FP8 blocks of a language model, as cases to time.

Each case is one call of an operator on inputs like those of a training or
serving step:

* ``norm_fwd``   t = x + r, its RMS norm as E4M3 codes with their amax, or in bf16;
* ``norm_bwd``   the gradient of x and r, and of the norm's weight;
* ``logp_fwd``   log probabilities of given tokens over a vocabulary, their
                 entropy, the most probable tokens;
* ``logp_bwd``   the gradient of the logits, in their type or as E5M2 codes;
* ``embed_fwd``  rows of an embedding table, scaled;
* ``embed_bwd``  the table's gradient.

``run`` computes a case with the library (``own`` true) or in plain torch
operations in fp32, rounded once at the end.
"""

import math

import numpy as np
import torch

own = False

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
TYPES = dict(bf16=torch.bfloat16, f32=torch.float32)
SIZE = dict(bf16=2, f32=4, e4m3=1, e5m2=1)
EPS = 1e-6


def listed():
    return [
        # one token before a block of the 4096-wide model when serving: latency
        dict(name="norm 1 token", kind="norm_fwd", M=1, K=4096, x="bf16", r="bf16", y="e4m3"),
        # the training batch before a block
        dict(name="norm train", kind="norm_fwd", M=16384, K=4096, x="bf16", r="bf16", y="e4m3"),
        # backward of a ragged batch whose residual stream is kept in fp32
        dict(name="norm bwd ragged", kind="norm_bwd", M=1237, K=2736, x="bf16", r="f32", stream=True),
        # backward of the training batch
        dict(name="norm bwd train", kind="norm_bwd", M=16384, K=4096, x="bf16", r="bf16", stream=True),
        # a few sequences being decoded, with the 20 best tokens of each
        dict(name="logprobs 7 tokens", kind="logp_fwd", M=7, V=128000, x="bf16", entropy=True, top=20, masked=0.0),
        # scoring a ragged batch over an odd vocabulary, logits in fp32, half of the vocabulary masked
        dict(name="logprobs odd", kind="logp_fwd", M=333, V=50001, x="f32", entropy=True, top=5, masked=0.5),
        # the loss of a training batch
        dict(name="logprobs train", kind="logp_fwd", M=8192, V=128000, x="bf16", entropy=False, top=0, masked=0.0),
        # its gradient, in the codes that the head's backward pass reads
        dict(name="logprobs bwd train", kind="logp_bwd", M=8192, V=128000, x="bf16", out="e5m2", entropy=False,
             masked=0.0),
        # gradient of log probabilities and entropy for a policy over an odd vocabulary
        dict(name="logprobs bwd odd", kind="logp_bwd", M=333, V=50001, x="bf16", out="bf16", entropy=True, masked=0.5),
        # the training batch's tokens looked up in the E4M3 copy of the table
        dict(name="embed train", kind="embed_fwd", M=16384, V=128000, K=4096, table="e4m3", out="bf16"),
        # the table's gradient for that batch
        dict(name="embed bwd train", kind="embed_bwd", M=16384, V=128000, K=4096, dy="bf16", out="bf16"),
        # a small table's gradient from a ragged batch: latency
        dict(name="embed bwd small", kind="embed_bwd", M=77, V=1000, K=272, dy="f32", out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log16(rng, lo, hi):
    return 16 * _log(rng, lo // 16, hi // 16)


def draw(rng):
    kind = rng.choice(["norm_fwd", "norm_bwd", "logp_fwd", "logp_fwd", "logp_bwd", "embed_fwd", "embed_bwd"])
    either = lambda *names: rng.choice(names)  # noqa: E731
    if kind in ("norm_fwd", "norm_bwd"):
        case = dict(kind=kind, K=_log16(rng, 64, 16384), x=either("bf16", "f32"), r=either("bf16", "f32"))
        case["M"] = _log(rng, 1, min(16384, 2 ** 25 // case["K"]))
        if kind == "norm_fwd":
            return dict(case, r=either("none", case["r"]), y=either("e4m3", "e4m3", "bf16", "f32"))
        return dict(case, stream=rng.random() < 0.7)
    if kind in ("logp_fwd", "logp_bwd"):
        V = _log(rng, 50, 200000)
        case = dict(kind=kind, x=either("bf16", "f32"), entropy=rng.random() < 0.5, masked=either(0.0, 0.0, 0.5, 0.99))
        case["M"] = _log(rng, 1, min(16384, 2 ** 28 // V))
        if kind == "logp_bwd":
            out = either("e5m2", case["x"])
            return dict(case, V=V // 16 * 16 if out == "e5m2" else V, out=out)
        top = either(0, 1, _log(rng, 2, 32))
        return dict(case, V=V, top=top, M=min(case["M"], 2 ** 25 // V) if top else case["M"])
    case = dict(kind=kind, V=_log(rng, 100, 150000), K=_log16(rng, 64, 8192))
    case["M"] = _log(rng, 1, min(32768, 2 ** 26 // case["K"]))
    case["V"] = min(case["V"], 2 ** 29 // case["K"])
    if kind == "embed_fwd":
        return dict(case, table=either("e4m3", "bf16", "f32"), out=either("bf16", "f32"))
    return dict(case, dy=either("bf16", "f32"), out=either("bf16", "f32"))


# ------------------------------------------------------------------ inputs


def _narrowed(x, dtype):
    top = 448.0 if dtype is E4M3 else 57344.0
    return x.clamp(-top, top).to(dtype)


def _one(v):
    return torch.tensor([v], dtype=torch.float32, device="cuda")


def _prepare_norm(case, gen):
    M, K = case["M"], case["K"]
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    channel = torch.exp(randn(K) * 0.5)  # some channels of a residual stream are much larger than others
    s = dict(case=case, w=1.0 + 0.1 * randn(K), rstd=torch.empty(M, device="cuda"))
    xt, rt = TYPES[case["x"]], TYPES.get(case["r"])
    if case["kind"] == "norm_fwd":
        s["x"] = randn(M, K).to(xt)
        s["r"] = (randn(M, K) * channel).to(rt) if rt else None
        s["t"] = torch.empty_like(s["r"]) if rt else None
        s["y"] = torch.empty((M, K), dtype=torch.uint8 if case["y"] == "e4m3" else TYPES[case["y"]], device="cuda")
        # a delayed scale: what the last steps' largest |y| asked for, with the odd overflow
        s["scale"] = _one(448.0 / 16.0) if case["y"] == "e4m3" else None
        s["amax"] = _one(0.0)
        return s
    s["t"] = (randn(M, K) * channel).to(rt)
    s["rstd"] = torch.rsqrt(s["t"].double().square().mean(1) + EPS).float()
    s["dy"] = (randn(M, K) * 1e-4).to(xt)
    s["dt"] = (randn(M, K) * 1e-4).to(rt) if case["stream"] else None
    s["dr"] = torch.empty_like(s["t"])
    s["dx"] = torch.empty_like(s["dy"]) if xt is not rt else None
    s["dw"] = torch.empty(K, device="cuda")
    if own:
        import fp8_mixed_precision_reduce_gb300 as fp8mp

        s["workspace"] = torch.empty(fp8mp.fp8_rmsnorm_bwd_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    return s


def _parts(M, V):
    """Row ranges of about 2^27 logits."""
    step = max(1, 2 ** 27 // V)
    return [(i, min(M, i + step)) for i in range(0, M, step)]


def _prepare_logp(case, gen):
    M, V, dev = case["M"], case["V"], "cuda"
    x = torch.empty((M, V), dtype=TYPES[case["x"]], device=dev)
    target = torch.randint(0, V, (M,), generator=gen, device=dev)
    rows = torch.arange(M, device=dev)
    for i, j in _parts(M, V):
        part = torch.randn((j - i, V), generator=gen, device=dev) * 2.5
        if case["masked"]:  # tokens that a grammar or a filter does not allow
            part.masked_fill_(torch.rand((j - i, V), generator=gen, device=dev) < case["masked"], -math.inf)
        x[i:j] = part
    # what a model finds likely, the token itself among it more often than not
    x[rows, target] = (torch.randn(M, generator=gen, device=dev) * 3 + 9).to(x.dtype)
    target[torch.rand(M, generator=gen, device=dev) < 0.05] = -100  # prompt and padding
    s = dict(case=case, x=x, target=target)
    if case["kind"] == "logp_fwd":
        s["logprob"], s["stats"] = torch.empty(M, device=dev), torch.empty((M, 2), device=dev)
        s["entropy"] = torch.empty(M, device=dev) if case["entropy"] else None
        s["top"] = torch.empty((M, case["top"]), device=dev) if case["top"] else None
        s["ids"] = torch.empty((M, case["top"]), dtype=torch.int64, device=dev) if case["top"] else None
        return s
    stats, entropy = torch.empty((M, 2), device=dev), torch.empty(M, device=dev)
    for i, j in _parts(M, V):
        part = x[i:j].float()
        top = part.amax(1)
        d = part - top[:, None]
        e = torch.exp(d)
        total = e.sum(1)
        stats[i:j, 0], stats[i:j, 1] = top, torch.log(total)
        entropy[i:j] = torch.log(total) - torch.where(e > 0, e * d, 0.0).sum(1) / total
    s["stats"], s["entropy"] = stats, entropy if case["entropy"] else None
    # the gradient of a mean under a loss scale, weighted from token to token
    s["da"] = torch.randn(M, generator=gen, device=dev) * (65536.0 / M)
    s["db"] = torch.randn(M, generator=gen, device=dev) * (655.36 / M) if case["entropy"] else None
    s["out"] = torch.empty((M, V), dtype=torch.uint8 if case["out"] == "e5m2" else x.dtype, device=dev)
    s["scale"] = _one(M / 8.0) if case["out"] == "e5m2" else None
    s["amax"] = _one(0.0)
    return s


def _frequencies(V):
    """Words' frequencies fall as their ranks rise."""
    p = 1.0 / (np.arange(V, dtype=np.float64) + 2.7)
    return p / p.sum()


def _prepare_embed(case, gen):
    M, V, K, dev = case["M"], case["V"], case["K"], "cuda"
    edges = torch.from_numpy(np.cumsum(_frequencies(V))).to(dev)
    rank = torch.searchsorted(edges, torch.rand(M, generator=gen, device=dev, dtype=torch.float64)).clamp_max(V - 1)
    ids = torch.randperm(V, generator=gen, device=dev)[rank]
    ids[torch.rand(M, generator=gen, device=dev) < 0.03] = -1  # padding
    s = dict(case=case, ids=ids, factor=math.sqrt(K))
    if case["kind"] == "embed_fwd":
        table = torch.randn((V, K), generator=gen, device=dev) * 0.02
        s["sinv"] = _one(2.0 ** -12) if case["table"] == "e4m3" else None
        if case["table"] == "e4m3":
            s["table"] = _narrowed(table * 2.0 ** 12, E4M3).view(torch.uint8)
        else:
            s["table"] = table.to(TYPES[case["table"]])
        s["out"] = torch.empty((M, K), dtype=TYPES[case["out"]], device=dev)
        return s
    s["dy"] = (torch.randn((M, K), generator=gen, device=dev) * 1e-4).to(TYPES[case["dy"]])
    s["dtable"] = torch.empty((V, K), dtype=TYPES[case["out"]], device=dev)
    if own:
        import fp8_mixed_precision_reduce_gb300 as fp8mp

        s["workspace"] = torch.empty(fp8mp.mp_embedding_bwd_workspace_bytes(M, V, K), dtype=torch.uint8, device=dev)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return dict(norm=_prepare_norm, logp=_prepare_logp, embed=_prepare_embed)[case["kind"].split("_")[0]](case, gen)


# ------------------------------------------------------------- plain forms


def _plain_norm_fwd(s):
    t = s["x"].float()
    if s["r"] is not None:
        s["t"].copy_(t + s["r"])
        t = s["t"].float()
    rstd = 1.0 / torch.sqrt((t * t).mean(1) + EPS)
    y = t * rstd[:, None] * s["w"]
    s["rstd"].copy_(rstd)
    s["amax"].copy_(torch.maximum(s["amax"], y.abs().max()))
    s["y"].copy_(_narrowed(y * s["scale"], E4M3).view(torch.uint8) if s["scale"] is not None else y)


def _plain_norm_bwd(s):
    n = s["t"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"]
    dr = s["rstd"][:, None] * (g - n * (g * n).mean(1, keepdim=True))
    if s["dt"] is not None:
        dr = dr + s["dt"]
    s["dr"].copy_(dr)
    if s["dx"] is not None:
        s["dx"].copy_(dr)
    s["dw"].copy_((dy * n).sum(0))


def _plain_logp_fwd(s):
    x = s["x"].float()
    top = x.amax(1)
    d = x - top[:, None]
    e = torch.exp(d)
    total = e.sum(1)
    log_total = torch.log(total)
    given = s["target"] >= 0
    at = torch.gather(d, 1, s["target"].clamp_min(0)[:, None])[:, 0]
    s["logprob"].copy_(torch.where(given, at - log_total, 0.0))
    s["stats"].copy_(torch.stack([top, log_total], 1))
    if s["entropy"] is not None:
        s["entropy"].copy_(log_total - torch.where(e > 0, e * d, 0.0).sum(1) / total)
    if s["top"] is not None:
        values, ids = torch.sort(d, dim=1, descending=True, stable=True)
        k = s["case"]["top"]
        s["top"].copy_(values[:, :k] - log_total[:, None])
        s["ids"].copy_(ids[:, :k])


def _plain_logp_bwd(s):
    given = s["target"] >= 0
    a = torch.where(given, s["da"], 0.0)
    logp = (s["x"].float() - s["stats"][:, :1]) - s["stats"][:, 1:]
    p = torch.exp(logp)
    if s["entropy"] is not None:
        g = torch.where(p > 0, -p * (a[:, None] + s["db"][:, None] * (logp + s["entropy"][:, None])), 0.0)
    else:
        g = -p * a[:, None]
    g.scatter_add_(1, s["target"].clamp_min(0)[:, None], a[:, None])
    s["amax"].copy_(torch.maximum(s["amax"], g.abs().max()))
    s["out"].copy_(_narrowed(g * s["scale"], E5M2).view(torch.uint8) if s["scale"] is not None else g)


def _plain_embed_fwd(s):
    rows = s["table"][s["ids"].clamp_min(0)]
    rows = rows.view(E4M3).float() * (s["sinv"] * s["factor"]) if s["sinv"] is not None else rows.float() * s["factor"]
    s["out"].copy_(torch.where((s["ids"] >= 0)[:, None], rows, 0.0))


def _plain_embed_bwd(s):
    total = torch.zeros(s["dtable"].shape, device="cuda")
    total.index_add_(0, s["ids"].clamp_min(0), torch.where((s["ids"] >= 0)[:, None], s["dy"].float(), 0.0))
    s["dtable"].copy_(total * s["factor"])


_PLAIN = dict(norm_fwd=_plain_norm_fwd, norm_bwd=_plain_norm_bwd, logp_fwd=_plain_logp_fwd, logp_bwd=_plain_logp_bwd,
              embed_fwd=_plain_embed_fwd, embed_bwd=_plain_embed_bwd)


# ------------------------------------------------------- the library's calls


def _library(s):
    import fp8_mixed_precision_reduce_gb300 as fp8mp

    kind = s["case"]["kind"]
    if kind == "norm_fwd":
        fp8mp.fp8_rmsnorm_fwd(s["x"], s["w"], s["y"], s["rstd"], eps=EPS, residual=s["r"], total=s["t"],
                              y_scale=s["scale"], y_amax=s["amax"])
    elif kind == "norm_bwd":
        fp8mp.fp8_rmsnorm_bwd(s["dy"], s["t"], s["w"], s["rstd"], s["dr"], s["dw"], s["workspace"], dtotal=s["dt"],
                              dx=s["dx"])
    elif kind == "logp_fwd":
        fp8mp.mp_logprobs_fwd(s["x"], s["target"], s["logprob"], s["stats"], entropy=s["entropy"],
                              top_logprob=s["top"], top_id=s["ids"])
    elif kind == "logp_bwd":
        fp8mp.mp_logprobs_bwd(s["x"], s["target"], s["stats"], s["da"], s["out"], entropy=s["entropy"],
                              dentropy=s["db"], scale=s["scale"], amax=s["amax"])
    elif kind == "embed_fwd":
        fp8mp.mp_embedding_fwd(s["ids"], s["table"], s["out"], scale=s["factor"], sinv=s["sinv"])
    else:
        fp8mp.mp_embedding_bwd(s["ids"], s["dy"], s["dtable"], s["workspace"], scale=s["factor"])


def _outputs(s):
    kind = s["case"]["kind"]
    if kind == "norm_fwd":
        return dict(t=s["t"], y=s["y"].view(E4M3) if s["scale"] is not None else s["y"], rstd=s["rstd"], amax=s["amax"])
    if kind == "norm_bwd":
        return dict(dr=s["dr"], dx=s["dx"], dw=s["dw"])
    if kind == "logp_fwd":
        return dict(logprob=s["logprob"], stats=s["stats"], entropy=s["entropy"], top=s["top"], ids=s["ids"])
    if kind == "logp_bwd":
        return dict(out=s["out"].view(E5M2) if s["scale"] is not None else s["out"], amax=s["amax"])
    return dict(out=s["out"]) if kind == "embed_fwd" else dict(dtable=s["dtable"])


def run(state):
    if own:
        _library(state)
    else:
        _PLAIN[state["case"]["kind"]](state)
    return _outputs(state)


# --------------------------------------------------------------------- work


def work(case):
    kind, M = case["kind"], case["M"]
    if kind == "norm_fwd":
        K, r = case["K"], SIZE.get(case["r"], 0)
        return dict(bytes=M * K * (SIZE[case["x"]] + 2 * r + SIZE[case["y"]]) + 4 * M + 4 * K, flops=6 * M * K)
    if kind == "norm_bwd":
        K, x, r = case["K"], SIZE[case["x"]], SIZE[case["r"]]
        each = x + 2 * r + (r if case["stream"] else 0) + (x if case["x"] != case["r"] else 0)
        return dict(bytes=M * K * each + 4 * M + 8 * K, flops=10 * M * K)
    if kind == "logp_fwd":
        return dict(bytes=M * (case["V"] * SIZE[case["x"]] + 20 + 12 * case["top"]), flops=6 * M * case["V"])
    if kind == "logp_bwd":
        return dict(bytes=M * (case["V"] * (SIZE[case["x"]] + SIZE[case["out"]]) + 24), flops=6 * M * case["V"])
    V, K = case["V"], case["K"]
    if kind == "embed_fwd":
        rows = float(-np.expm1(M * np.log1p(-0.97 * _frequencies(V))).sum())  # those that the tokens name, on average
        return dict(bytes=int(rows * K * SIZE[case["table"]]) + M * K * SIZE[case["out"]] + 8 * M, flops=M * K)
    return dict(bytes=M * K * SIZE[case["dy"]] + V * K * SIZE[case["out"]] + 8 * M, flops=M * K + V * K)


# ------------------------------------------------------- 64-bit definitions


def _nearest(x, dtype):
    """The nearest code's value, as 64-bit numbers, saturating."""
    digits, low, top = (3, -6, 448.0) if dtype is E4M3 else (2, -14, 57344.0)
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** low))).clamp_min(low)
    quantum = torch.exp2(e - digits)
    return (torch.round(x / quantum) * quantum).clamp(-top, top)


def _exact_norm(case, s):
    w = s["w"].double()
    if case["kind"] == "norm_fwd":
        t = s["x"].double()
        if s["r"] is not None:
            t = (t + s["r"].double()).to(s["r"].dtype).double()  # the norm is of the stream as it is stored
        rstd = (t.square().sum(1) / case["K"] + EPS).rsqrt()
        y = torch.einsum("mk,m,k->mk", t, rstd, w)
        q = _nearest(y * s["scale"].double(), E4M3) if s["scale"] is not None else y
        return dict(t=t if s["r"] is not None else None, y=q, rstd=rstd, amax=y.abs().max().reshape(1))
    t, dy, rstd = s["t"].double(), s["dy"].double(), s["rstd"].double()
    along = torch.einsum("mk,mk,k->m", t, dy, w) * rstd.square() / case["K"]
    dr = (dy * w - t * along[:, None]) * rstd[:, None]
    if s["dt"] is not None:
        dr += s["dt"].double()
    return dict(dr=dr, dx=dr if s["dx"] is not None else None, dw=torch.einsum("mk,mk,m->k", t, dy, rstd))


def _exact_logp(case, s):
    M, V = case["M"], case["V"]
    forward = case["kind"] == "logp_fwd"
    empty = lambda *shape: torch.empty(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out = dict(logprob=empty(M), stats=empty(M, 2), entropy=empty(M), top=empty(M, case.get("top", 0)), ids=None)
    if not forward:
        out = dict(out=empty(M, V), amax=torch.zeros(1, dtype=torch.float64, device="cuda"))
    for i, j in _parts(M, V):
        x = s["x"][i:j].double()
        target = s["target"][i:j]
        if forward:
            lse = torch.logsumexp(x, 1)
            logp = x - lse[:, None]
            at = logp[torch.arange(j - i, device="cuda"), target.clamp_min(0)]
            out["logprob"][i:j] = torch.where(target >= 0, at, 0.0)
            out["stats"][i:j, 0] = x.amax(1)
            out["stats"][i:j, 1] = lse - x.amax(1)
            out["entropy"][i:j] = torch.special.entr(torch.exp(logp)).sum(1)
            if case["top"]:
                out["top"][i:j] = torch.topk(logp, case["top"], dim=1).values
            continue
        logp = x - s["stats"][i:j].double().sum(1, keepdim=True)
        p = torch.exp(logp)
        a = s["da"][i:j].double() * (target >= 0)
        g = p * -a[:, None]
        if s["entropy"] is not None:
            tilt = torch.where(p > 0, logp, 0.0) + s["entropy"][i:j, None].double()
            g -= p * tilt * s["db"][i:j, None].double()
        g[torch.arange(j - i, device="cuda"), target.clamp_min(0)] += a
        out["amax"] = torch.maximum(out["amax"], g.abs().max())
        out["out"][i:j] = _nearest(g * s["scale"].double(), E5M2) if s["scale"] is not None else g
    if forward:
        out["entropy"] = out["entropy"] if case["entropy"] else None
        out["top"] = out["top"] if case["top"] else None
    return out


def _exact_embed(case, s):
    kept = s["ids"] >= 0
    if case["kind"] == "embed_fwd":
        out = torch.zeros((case["M"], case["K"]), dtype=torch.float64, device="cuda")
        rows = s["table"].view(E4M3)[s["ids"][kept]] if s["sinv"] is not None else s["table"][s["ids"][kept]]
        out[kept] = rows.double() * (s["factor"] * (float(s["sinv"]) if s["sinv"] is not None else 1.0))
        return dict(out=out)
    out = torch.zeros((case["V"], case["K"]), dtype=torch.float64, device="cuda")
    out.index_put_((s["ids"][kept],), s["dy"][kept].double(), accumulate=True)
    return dict(dtable=out.mul_(s["factor"]))


def exact(case, seed):
    s = prepare(case, seed)
    return dict(norm=_exact_norm, logp=_exact_logp, embed=_exact_embed)[case["kind"].split("_")[0]](case, s)
