"""More of the operators around the sharded step, as timed cases.

The gradients that do not lie in one flat buffer: their global norm over many
tensors, the clip and the copy into the rank's flat gradient.  Two operators of
the model with small parameters whose gradients are sums over everything: the
group norm with its activation, channels last, and the learned relative position
bias by buckets.  Each with its gradient.

``listed()`` holds the cases, ``draw(rng)`` makes further ones of the same
ranges, ``prepare`` the inputs, ``run`` one pass (plain torch operations in
fp32, or the library's calls when ``own`` is true), ``exact`` the same outputs
in fp64 from the definitions, ``work`` the bytes and operations of a pass.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5


def _lib():
    import fsdp_sharded_optimizer_gb300 as Z
    return Z


# --------------------------------------------------------------------- cases
def listed():
    return [
        # the gradients of a toy model of two layers, as autograd leaves them: latency only
        dict(name="clip_small", op="clip", layers=2, dim=64, kv=64, hidden=160, vocab=512,
             bias=True, grad="f32", out="f32", max_norm=1.0),
        # GPT-2-small's width and vocabulary in 12 layers, bf16 gradients into the flat buffer
        dict(name="clip_bf16", op="clip", layers=12, dim=768, kv=768, hidden=2048, vocab=50257,
             bias=True, grad="bf16", out="bf16", max_norm=1.0),
        # Llama-1.1B's 200 tensors, fp32 gradients rounded into the bf16 flat buffer
        dict(name="clip_wide", op="clip", layers=22, dim=2048, kv=256, hidden=5632, vocab=32000,
             bias=False, grad="f32", out="bf16", max_norm=1.0),
        # one picture's coarsest feature map, 8 x 8: latency only
        dict(name="group_norm_small", op="gn", samples=1, positions=64, channels=1280, groups=32,
             type="bf16", param="bf16", act="silu", ragged=False),
        # a training batch's finest feature maps, 128 x 128
        dict(name="group_norm_large", op="gn", samples=32, positions=16384, channels=320,
             groups=32, type="bf16", param="bf16", act="silu", ragged=False),
        # recordings of unequal length, 81 channels in 3 groups: rows at odd addresses
        dict(name="group_norm_grad_ragged", op="gn_grad", samples=24, positions=3001, channels=81,
             groups=3, type="bf16", param="f32", act="gelu", ragged=True),
        # the gradient for a batch of 64 x 64 feature maps
        dict(name="group_norm_grad_large", op="gn_grad", samples=32, positions=4096, channels=640,
             groups=32, type="bf16", param="bf16", act="silu", ragged=False),
        # one new token's scores of a few sequences against their caches
        dict(name="relpos_one_query", op="relpos", batch=4, heads=12, q=1, k=1021, buckets=32,
             distance=128, bidirectional=False, causal=True, ragged=True, scores=True,
             type="f32", table="bf16"),
        # the bias alone, once a step, for a library's attention to add: 32 heads, 2048 tokens
        dict(name="relpos_bias", op="relpos", batch=1, heads=32, q=2048, k=2048, buckets=32,
             distance=128, bidirectional=True, causal=False, ragged=False, scores=False,
             type="bf16", table="bf16"),
        # added to a padded batch's scores, later and padded keys masked
        dict(name="relpos_scores", op="relpos", batch=8, heads=12, q=1024, k=1024, buckets=32,
             distance=128, bidirectional=False, causal=True, ragged=True, scores=True,
             type="bf16", table="bf16"),
        # the table's gradient, short padded sequences of an odd length, many buckets
        dict(name="relpos_grad_odd", op="relpos_grad", batch=16, heads=12, q=333, k=333,
             buckets=320, distance=800, bidirectional=True, causal=False, ragged=True,
             type="bf16", table="f32"),
        # the table's gradient, 4 sequences of 2048 tokens and 32 heads
        dict(name="relpos_grad_large", op="relpos_grad", batch=4, heads=32, q=2048, k=2048,
             buckets=32, distance=128, bidirectional=True, causal=False, ragged=False,
             type="bf16", table="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["clip", "gn", "gn_grad", "relpos", "relpos_grad"])
    if op == "clip":
        dim = _log_int(rng, 33, 2048)
        dim = dim if rng.random() < 0.3 else max(32, dim // 8 * 8)
        grad, out = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        return dict(op=op, layers=_log_int(rng, 1, 22 if dim < 1024 else 12), dim=dim,
                    kv=max(1, dim // rng.choice([1, 1, 4, 8])),
                    hidden=int(dim * rng.choice([1.5, 2, 2.75])), vocab=_log_int(rng, 300, 32000),
                    bias=rng.random() < 0.5, grad=grad, out=out,
                    max_norm=rng.choice([0.1, 1.0, 10.0]))
    if op in ("gn", "gn_grad"):
        groups = rng.choice([1, 2, 3, 8, 16, 32, 32])
        per = _log_int(rng, 1, 1280 // groups)
        channels = groups * per
        samples = _log_int(rng, 1, 64)
        positions = _log_int(rng, 1, 16384)
        type = rng.choice(["bf16", "bf16", "f32"])
        most = (83_000_000 if op == "gn" else 60_000_000) // (2 if type == "f32" else 1)
        positions = max(1, min(positions, most // (samples * channels)))
        # a group of a few values has next to no gradient: the norm takes it all away
        positions = max(positions, -(-256 // per))
        return dict(op=op, samples=samples, positions=positions, channels=channels,
                    groups=groups, type=type, param=rng.choice(["bf16", "f32"]),
                    act=rng.choice(["none", "silu", "silu", "gelu"]),
                    ragged=rng.random() < 0.3)
    batch, heads = _log_int(rng, 1, 32), _log_int(rng, 1, 32)
    k = _log_int(rng, 1, 4096)
    q = rng.choice([k, k, k, 1, max(1, k // 3)])
    if rng.random() < 0.6:
        q, k = (max(8, n // 8 * 8) for n in (q, k))
    type = rng.choice(["bf16", "bf16", "f32"])
    most = 200_000_000 // (2 if type == "f32" else 1)
    heads = max(1, min(heads, most // (q * k)))
    batch = max(1, min(batch, most // (heads * q * k)))
    buckets, distance = rng.choice([(32, 128), (32, 128), (16, 64), (64, 256), (320, 800)])
    case = dict(op=op, batch=batch, heads=heads, q=q, k=k, buckets=buckets, distance=distance,
                bidirectional=rng.random() < 0.5, causal=False, ragged=rng.random() < 0.4,
                type=type, table=rng.choice(["bf16", "f32"]))
    case["causal"] = not case["bidirectional"] and rng.random() < 0.8
    if op == "relpos":
        case["scores"] = case["ragged"] or rng.random() < 0.5
    return case


# -------------------------------------------------------------------- inputs
def _randn(gen, shape, dtype, sigma=1.0, mean=0.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return x.mul_(sigma).add_(mean).to(dtype)


def _sizes(c):
    """Elements of every parameter of a decoder: table, blocks of attention, gated hidden
    layer and two norms, last norm."""
    d, h, kv = c["dim"], c["hidden"], c["kv"]
    block = [d * d, kv * d, kv * d, d * d, h * d, h * d, h * d, d, d]
    if c["bias"]:
        block += [d, kv, kv, d, h, d]
    return [c["vocab"] * d] + block * c["layers"] + [d]


def _lengths(gen, n, most, ragged):
    """Lengths of a padded batch: at least half of the longest, which is full."""
    if not ragged:
        return None
    out = torch.randint(most - most // 2, most + 1, (n,), generator=gen, device="cuda")
    out[0] = most
    return out.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 29)
    s, c, op = dict(case=case), case, case["op"]
    if op == "clip":
        sizes = _sizes(c)
        # matrices near the output have larger gradients than those before them
        s["grads"] = [_randn(gen, (n,), _TYPES[c["grad"]], 1e-3 * (1 + i % 7))
                      for i, n in enumerate(sizes)]
        s["sizes"] = sizes
        if own:
            Z = _lib()
            s["flat"] = torch.empty(sum(sizes), dtype=_TYPES[c["out"]], device="cuda")
            s["list"] = Z.zero_tensor_list(s["grads"], list(s["flat"].split(sizes)))
            s["norm_coef"] = torch.empty(2, device="cuda")
            s["scratch"] = torch.empty(Z.zero_clip_scratch_bytes(), dtype=torch.uint8,
                                       device="cuda")
    elif op in ("gn", "gn_grad"):
        N, P, C, G = c["samples"], c["positions"], c["channels"], c["groups"]
        t, par = _TYPES[c["type"]], _TYPES[c["param"]]
        x = torch.randn((N, P, C), generator=gen, device="cuda")
        x.mul_(0.5 + torch.rand(C, generator=gen, device="cuda") * 2)
        s["x"] = x.add_(torch.randn(C, generator=gen, device="cuda")).to(t)
        del x
        s["weight"] = _randn(gen, (C,), par, 0.1, 1.0)
        s["bias"] = _randn(gen, (C,), par, 0.1)
        s["lengths"] = _lengths(gen, N, P, c["ragged"])
        if op == "gn_grad":
            s["dy"] = _randn(gen, (N, P, C), t, 1e-2)
            s["stats"] = torch.stack([torch.stack(_stats(s, n), 1) for n in range(N)]).float()
        if own:
            Z = _lib()
            s["scratch"] = torch.empty(Z.zero_group_norm_scratch_bytes(N, P, C, G),
                                       dtype=torch.uint8, device="cuda")
            if op == "gn":
                s["y"] = torch.zeros_like(s["x"])
                s["stats"] = torch.empty((N, G, 2), device="cuda")
            else:
                s["dx"] = torch.zeros_like(s["x"])
                s["dweight"], s["dbias"] = (torch.empty_like(s["weight"]) for _ in range(2))
    else:
        B, H, Q, K = c["batch"], c["heads"], c["q"], c["k"]
        t, tab = _TYPES[c["type"]], _TYPES[c["table"]]
        s["k_lengths"] = _lengths(gen, B, K, c["ragged"])
        s["q_lengths"] = s["k_lengths"] if Q == K else _lengths(gen, B, Q, c["ragged"])
        # the last query stands at the last key, as where a cache holds what came before
        s["start"] = K - Q
        s["starts"] = s["k_lengths"] - s["q_lengths"] if c["ragged"] and Q != K else None
        if op == "relpos":
            s["table"] = _randn(gen, (c["buckets"], H), tab, 0.5)
            s["scores"] = _randn(gen, (B, H, Q, K), t, 2.0) if c["scores"] else None
            if own:
                s["out"] = torch.zeros((B, H, Q, K), dtype=t, device="cuda")
        else:
            s["dout"] = _randn(gen, (B, H, Q, K), t, 1e-3)
            if own:
                s["dtable"] = torch.empty((c["buckets"], H), dtype=tab, device="cuda")
                s["scratch"] = torch.empty(
                    _lib().zero_relpos_scratch_bytes(B, H, Q, K, c["buckets"]),
                    dtype=torch.uint8, device="cuda")
    return s


def _stats(s, n):
    """Mean and 1/sqrt(variance + eps) of each group of sample n, in 64 bits."""
    c = s["case"]
    P = c["positions"] if s["lengths"] is None else int(s["lengths"][n])
    v = s["x"][n, :P].double().view(P, c["groups"], -1)
    mean = v.mean((0, 2))
    return mean, 1 / torch.sqrt(((v - mean[:, None]) ** 2).mean((0, 2)) + EPS)


# ------------------------------------------------------- the library's calls
def _run_own(s):
    Z, c = _lib(), s["case"]
    op = c["op"]
    if op == "clip":
        Z.zero_tensors_clip(s["list"], c["max_norm"], s["norm_coef"], s["scratch"])
        return {"flat": s["flat"], "norm_coef": s["norm_coef"]}
    if op in ("gn", "gn_grad"):
        common = dict(weight=s["weight"], bias=s["bias"], lengths=s["lengths"], act=c["act"])
        if op == "gn":
            Z.zero_group_norm_forward(s["x"], s["y"], s["stats"], s["scratch"], eps=EPS, **common)
            return {"y": s["y"], "stats": s["stats"]}
        Z.zero_group_norm_backward(s["x"], s["dy"], s["stats"], s["dx"], s["scratch"],
                                   dweight=s["dweight"], dbias=s["dbias"], **common)
        return {k: s[k] for k in ("dx", "dweight", "dbias")}
    common = dict(q_lengths=s["q_lengths"], k_lengths=s["k_lengths"], start=s["start"],
                  starts=s["starts"], max_distance=c["distance"], bidirectional=c["bidirectional"],
                  causal=c["causal"])
    if op == "relpos":
        Z.zero_relpos_forward(s["table"], s["out"], scores=s["scores"], **common)
        return {"out": s["out"]}
    Z.zero_relpos_backward(s["dout"], s["dtable"], s["scratch"], **common)
    return {"dtable": s["dtable"]}


# ------------------------------------------------------------ the plain forms
def _clip_plain(s):
    c = s["case"]
    total = torch.stack([(g.float() ** 2).sum(dtype=torch.float64) for g in s["grads"]]).sum()
    norm = torch.sqrt(total)
    coef = torch.clamp(c["max_norm"] / (norm + 1e-6), max=1.0).float()
    flat = torch.cat([(g.float() * coef).to(_TYPES[c["out"]]) for g in s["grads"]])
    return {"flat": flat, "norm_coef": torch.stack([norm.float(), coef])}


def _counted(lengths, most):
    """[n, most, 1] truth values of the places that a sequence has, or None."""
    if lengths is None:
        return None
    return (torch.arange(most, device="cuda") < lengths[:, None])[:, :, None]


def _activated(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return z * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))))
    return z


def _slope(z, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    return torch.ones_like(z)


def _gn_plain(s):
    c = s["case"]
    N, P, C, G = c["samples"], c["positions"], c["channels"], c["groups"]
    on = _counted(s["lengths"], P)
    x = s["x"].float()
    count = (P if on is None else s["lengths"][:, None]) * float(C // G)
    part = x if on is None else torch.where(on, x, 0.0)
    mean = part.view(N, P, G, -1).sum((1, 3)) / count
    d = x.view(N, P, G, -1) - mean[:, None, :, None]
    if on is not None:
        d = torch.where(on[:, :, :, None], d, 0.0)
    rstd = torch.rsqrt((d * d).sum((1, 3)) / count + EPS)
    z = (d * rstd[:, None, :, None]).view(N, P, C) * s["weight"].float() + s["bias"].float()
    y = _activated(z, c["act"])
    if on is not None:
        y = torch.where(on, y, 0.0)
    return {"y": y.to(_TYPES[c["type"]]), "stats": torch.stack([mean, rstd], 2)}


def _gn_grad_plain(s):
    c = s["case"]
    N, P, C, G = c["samples"], c["positions"], c["channels"], c["groups"]
    on = _counted(s["lengths"], P)
    count = (P if on is None else s["lengths"][:, None, None, None]) * float(C // G)
    mean, rstd = (s["stats"][:, None, :, i, None] for i in (0, 1))
    xh = ((s["x"].float().view(N, P, G, -1) - mean) * rstd).view(N, P, C)
    w = s["weight"].float()
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _slope(xh * w + s["bias"].float(), c["act"])
    if on is not None:
        dz, xh = torch.where(on, dz, 0.0), torch.where(on, xh, 0.0)
    par = _TYPES[c["param"]]
    out = {"dweight": (dz * xh).sum((0, 1)).to(par), "dbias": dz.sum((0, 1)).to(par)}
    dw, xg = (dz * w).view(N, P, G, -1), xh.view(N, P, G, -1)
    a = dw.sum((1, 3), keepdim=True) / count
    b = (dw * xg).sum((1, 3), keepdim=True) / count
    dx = ((dw - a - xg * b) * rstd).view(N, P, C)
    if on is not None:
        dx = torch.where(on, dx, 0.0)
    return dict(dx=dx.to(_TYPES[c["type"]]), **out)


def _borders(buckets, distance):
    """The distances at which the buckets of one direction begin: half of them hold one
    distance each, the others parts of equal size on a logarithmic scale, whose borders are
    found in whole numbers (a logarithm may round a distance into the bucket before its own)."""
    exact_ones = buckets // 2
    parts = buckets - exact_ones
    out, n = list(range(exact_ones)), exact_ones
    for j in range(parts):
        while n ** parts * exact_ones ** j < distance ** j * exact_ones ** parts:
            n += 1
        out.append(n)
    return out


def _positions(s):
    """[1 or batch, q] positions of the queries among the keys."""
    q = torch.arange(s["case"]["q"], device="cuda")[None]
    return q + (s["start"] if s["starts"] is None else s["starts"][:, None])


def _bucket_plain(s):
    """[1 or batch, q, k] bucket of every pair: a direction's own half of the buckets, or 0 for
    later keys."""
    c = s["case"]
    ahead = torch.arange(c["k"], device="cuda") - _positions(s)[:, :, None]
    buckets = c["buckets"] // 2 if c["bidirectional"] else c["buckets"]
    n = ahead.abs() if c["bidirectional"] else (-ahead).clamp(min=0)
    at = torch.tensor(_borders(buckets, c["distance"]), device="cuda")
    b = torch.searchsorted(at, n, right=True) - 1
    return torch.where(ahead > 0, b + buckets, b) if c["bidirectional"] else b


def _allowed(s):
    """Truth values of the places that count, and of the rows that are written; None: all."""
    c = s["case"]
    Q, K = c["q"], c["k"]
    keys = torch.arange(K, device="cuda")
    on = rows = None
    if c["causal"]:
        on = (keys <= _positions(s)[:, :, None])[:, None]
    if s["k_lengths"] is not None:
        inside = (keys < s["k_lengths"][:, None])[:, None, None, :]
        on = inside if on is None else on & inside
    if s["q_lengths"] is not None:
        rows = (torch.arange(Q, device="cuda") < s["q_lengths"][:, None])[:, None, :, None]
    return on, rows


def _relpos_plain(s):
    c = s["case"]
    bias = s["table"].float()[_bucket_plain(s)].permute(0, 3, 1, 2)
    out = bias.expand(c["batch"], -1, -1, -1) if s["scores"] is None else s["scores"].float() + bias
    on, rows = _allowed(s)
    if on is not None:
        out = torch.where(on, out, -math.inf)
    if rows is not None:
        out = torch.where(rows, out, 0.0)
    return {"out": out.to(_TYPES[c["type"]]).contiguous()}


def _relpos_grad_plain(s):
    c = s["case"]
    on, rows = _allowed(s)
    g = s["dout"].float()
    for mask in (on, rows):
        if mask is not None:
            g = torch.where(mask, g, 0.0)
    if s["starts"] is None:
        g = g.sum(0, keepdim=True)
    bucket = _bucket_plain(s)[:, None]
    out = [torch.where(bucket == b, g, 0.0).sum((0, 2, 3)) for b in range(c["buckets"])]
    return {"dtable": torch.stack(out).to(_TYPES[c["table"]])}


def _run_plain(s):
    return {"clip": _clip_plain, "gn": _gn_plain, "gn_grad": _gn_grad_plain,
            "relpos": _relpos_plain, "relpos_grad": _relpos_grad_plain}[s["case"]["op"]](s)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------- definitions in fp64
def exact(case, seed):
    s = prepare(case, seed)
    return {"clip": _exact_clip, "gn": _exact_gn, "gn_grad": _exact_gn_grad,
            "relpos": _exact_relpos, "relpos_grad": _exact_relpos_grad}[case["op"]](s)


def _exact_clip(s):
    norm = math.sqrt(math.fsum(float(g.double().square().sum()) for g in s["grads"]))
    coef = min(1.0, s["case"]["max_norm"] / (norm + 1e-6))
    flat = torch.empty(sum(s["sizes"]), dtype=torch.float64, device="cuda")
    at = 0
    for g in s["grads"]:
        flat[at:at + g.numel()] = g.double() * coef
        at += g.numel()
    return {"flat": flat, "norm_coef": torch.tensor([norm, coef], dtype=torch.float64)}


def _exact_gn(s):
    c = s["case"]
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    stats = []
    for n in range(c["samples"]):
        P = c["positions"] if s["lengths"] is None else int(s["lengths"][n])
        mean, rstd = _stats(s, n)
        stats.append(torch.stack([mean, rstd], 1))
        per = c["channels"] // c["groups"]
        z = ((s["x"][n, :P].double() - mean.repeat_interleave(per))
             * (rstd.repeat_interleave(per) * s["weight"].double()) + s["bias"].double())
        y[n, :P] = _exact_act(z, c["act"])[0]
    return {"y": y, "stats": torch.stack(stats)}


def _exact_act(z, act):
    """The activation and its derivative."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z)
    cdf = torch.special.ndtr(z)
    return z * cdf, cdf + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)


def _exact_gn_grad(s):
    c = s["case"]
    C, per = c["channels"], c["channels"] // c["groups"]
    dx = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    dweight, dbias = (torch.zeros(C, dtype=torch.float64, device="cuda") for _ in range(2))
    w, b = s["weight"].double(), s["bias"].double()
    for n in range(c["samples"]):
        P = c["positions"] if s["lengths"] is None else int(s["lengths"][n])
        mean, rstd = (s["stats"][n, :, i].double().repeat_interleave(per) for i in (0, 1))
        xh = (s["x"][n, :P].double() - mean) * rstd
        dz = s["dy"][n, :P].double() * _exact_act(xh * w + b, c["act"])[1]
        along, straight = (dz * xh).sum(0), dz.sum(0)
        dweight += along
        dbias += straight
        both = [(v * w).view(-1, per).mean(1).repeat_interleave(per) / P
                for v in (straight, along)]
        dx[n, :P] = rstd * (dz * w - both[0] - xh * both[1])
    return {"dx": dx, "dweight": dweight, "dbias": dbias}


def _bucket_of(c, ahead):
    """The bucket of one key that stands `ahead` places after the query."""
    per, first = c["buckets"], 0
    if c["bidirectional"]:
        per //= 2
        first = per if ahead > 0 else 0
    n = abs(ahead) if c["bidirectional"] else max(0, -ahead)
    half = per // 2
    if n < half:
        return first + n
    parts, j = per - half, 0
    # the largest j with (n / half) ** parts >= (distance / half) ** j, in whole numbers
    while j + 1 < parts and n ** parts * half ** (j + 1) >= c["distance"] ** (j + 1) * half ** parts:
        j += 1
    return first + half + j


def _starts(s):
    """The first query's position in each sequence."""
    return [s["start"]] * s["case"]["batch"] if s["starts"] is None else s["starts"].tolist()


def _exact_relpos(s):
    c = s["case"]
    Q, K = c["q"], c["k"]
    out = torch.zeros((c["batch"], c["heads"], Q, K), dtype=torch.float64, device="cuda")
    starts = _starts(s)
    first = -max(starts) - Q + 1
    by_distance = torch.tensor([_bucket_of(c, d) for d in range(first, K - min(starts))])
    line = s["table"].double()[by_distance.cuda()].t()  # [heads, distances from the first on]
    for b, start in enumerate(starts):
        for i in range(Q if s["q_lengths"] is None else int(s["q_lengths"][b])):
            at = -start - i - first
            out[b, :, i] = line[:, at:at + K]
            if s["scores"] is not None:
                out[b, :, i] += s["scores"][b, :, i].double()
            if c["causal"]:
                out[b, :, i, max(0, i + start + 1):] = -math.inf
            if s["k_lengths"] is not None:
                out[b, :, i, int(s["k_lengths"][b]):] = -math.inf
    return {"out": out}


def _exact_relpos_grad(s):
    c = s["case"]
    Q, K = c["q"], c["k"]
    starts = _starts(s)
    by_start = {}  # sums over the sequences that start at one position
    for b, start in enumerate(starts):
        q = Q if s["q_lengths"] is None else int(s["q_lengths"][b])
        k = K if s["k_lengths"] is None else int(s["k_lengths"][b])
        total = by_start.setdefault(start, torch.zeros((c["heads"], Q, K), dtype=torch.float64,
                                                       device="cuda"))
        total[:, :q, :k] += s["dout"][b, :, :q, :k].double()
    out = torch.zeros((c["buckets"], c["heads"]), dtype=torch.float64, device="cuda")
    bucket = {d: _bucket_of(c, d) for d in range(1 - Q - max(starts), K - min(starts))}
    for start, total in by_start.items():
        for d in range(1 - Q, K):
            if not (c["causal"] and d > start):
                out[bucket[d - start]] += total.diagonal(d, 1, 2).sum(1)
    return {"dtable": out}


# ---------------------------------------------------------------------- work
def _expected(most, ragged):
    """The mean of a length that _lengths draws."""
    return most - most // 2 / 2 if ragged else most


def work(case):
    c, op = case, case["op"]
    if op == "clip":
        n = sum(_sizes(c))
        return {"bytes": n * (_SIZE[c["grad"]] + _SIZE[c["out"]]), "flops": 3 * n}
    if op in ("gn", "gn_grad"):
        n = c["samples"] * _expected(c["positions"], c["ragged"]) * c["channels"]
        par = c["channels"] * _SIZE[c["param"]] * (2 if op == "gn" else 4)
        stats = c["samples"] * c["groups"] * 8
        # x in and y out, or x and dy in and dx out
        return {"bytes": n * _SIZE[c["type"]] * (2 if op == "gn" else 3) + par + stats,
                "flops": n * (10 if op == "gn" else 24)}
    B, H = c["batch"], c["heads"]
    q, k = (_expected(c[x], c["ragged"]) for x in ("q", "k"))
    read = q * k  # places that are read: not the masked ones
    if c["causal"]:
        read = sum(max(0.0, min(k, i + 1 + c["k"] - c["q"])) for i in range(int(q)))
    size, table = _SIZE[c["type"]], c["buckets"] * H * _SIZE[c["table"]]
    if op == "relpos":
        return {"bytes": B * H * size * (q * c["k"] + (read if c["scores"] else 0)) + table,
                "flops": 2 * B * H * q * k}
    return {"bytes": B * H * read * size + table, "flops": B * H * read}
