"""The training operators around the sharded step, as timed cases.

An embedding with its gradient, the norms around a block with its gate and
residual scale, and distillation from a teacher's top logits: what a student
needs besides its matrix products to turn token ids and gathered weights into
the gradients that the sharded optimizer step takes.

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


def _lib():
    import fsdp_sharded_optimizer_gb300 as Z
    return Z


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one new token's embedding: a GPT-2-small table, latency only
        dict(name="embed_one_token", op="embed", tokens=1, vocab=50257, dim=768, table="bf16",
             out="bf16", wide_ids=True, scale=1.0, pad=0.0),
        # a rank's micro-batch of 8 sequences of 2048 at Llama-7B's width, rows scaled by sqrt(dim)
        dict(name="embed_micro_batch", op="embed", tokens=16384, vocab=32000, dim=4096,
             table="bf16", out="bf16", wide_ids=True, scale=64.0, pad=0.0),
        # GPT-2-small's table gradient from 8 sequences of 1024, some of them padded at the end
        dict(name="embed_grad_small", op="embed_grad", tokens=8192, vocab=50257, dim=768,
             dout="bf16", grad="bf16", wide_ids=True, scale=1.0, pad=0.03),
        # Llama-7B's table gradient, 8 sequences of 2048
        dict(name="embed_grad_wide", op="embed_grad", tokens=16384, vocab=32000, dim=4096,
             dout="bf16", grad="bf16", wide_ids=False, scale=64.0, pad=0.0),
        # one token between two blocks of a 7B-wide model: latency only
        dict(name="norm_one_token", op="norm", rows=1, dim=4096, kind="rms", act="bf16",
             res="bf16", gate_span=0, post=True, pre=True, bias=False),
        # the norms between two blocks of a 7B-wide model, 8 sequences of 2048, learned channel gate
        dict(name="norm_wide", op="norm", rows=16384, dim=4096, kind="rms", act="bf16",
             res="bf16", gate_span=0, post=True, pre=True, bias=False),
        # backward at Llama-1.1B's width, fp32 residual stream, one gate row for each sequence of 2048
        dict(name="norm_grad_gated", op="norm_grad", rows=16384, dim=2048, kind="rms", act="bf16",
             res="f32", gate_span=2048, post=True, pre=True, bias=False),
        # backward with LayerNorm and biases at GPT-2-small's width, a ragged number of tokens
        dict(name="norm_grad_layer", op="norm_grad", rows=8191, dim=768, kind="layer", act="bf16",
             res="bf16", gate_span=0, post=True, pre=True, bias=True),
        # validation of a few answers: fp32 logits of the last tokens
        dict(name="distill_eval_few", op="distill", rows=5, vocab=50257, top=16, logits="f32",
             teacher="f32", tau=2.0, labels=True),
        # validation on a batch
        dict(name="distill_eval", op="distill", rows=8192, vocab=32000, top=64, logits="bf16",
             teacher="bf16", tau=1.0, labels=True),
        # training on GPT-2's vocabulary, unpadded logits: every row starts at another alignment
        dict(name="distill_grad_odd", op="distill_grad", rows=8191, vocab=50257, top=64,
             logits="bf16", teacher="bf16", tau=2.0, labels=True),
        # training on a 32,000-token vocabulary with fp32 logits, soft targets only
        dict(name="distill_grad_f32", op="distill_grad", rows=4096, vocab=32000, top=128,
             logits="f32", teacher="f32", tau=1.5, labels=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _dim(rng):
    d = _log_int(rng, 128, 4096)
    return d if rng.random() < 0.2 else max(128, d // 8 * 8)


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "distill", "distill_grad"])
    if op in ("embed", "embed_grad"):
        case = dict(op=op, tokens=_log_int(rng, 1, 16384), vocab=_log_int(rng, 4000, 50257),
                    dim=_dim(rng), wide_ids=rng.random() < 0.5,
                    scale=rng.choice([1.0, 64.0, 0.5]), pad=rng.choice([0.0, 0.03]))
        case["vocab"] = min(case["vocab"], 32000 * 4096 // case["dim"])
        kinds = ("table", "out") if op == "embed" else ("dout", "grad")
        for k in kinds:
            case[k] = rng.choice(["bf16", "bf16", "f32"])
        if "f32" in (case[kinds[0]], case[kinds[1]]):
            case["tokens"] = max(1, case["tokens"] // 2)
            case["vocab"] = min(case["vocab"], 32000 * 4096 // case["dim"] // 2)
        return case
    if op in ("norm", "norm_grad"):
        rows, dim = _log_int(rng, 1, 16384), _dim(rng)
        act, res = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        if res == "f32":
            rows = max(1, rows // 2)
        kind = rng.choice(["rms", "rms", "layer"])
        span = rng.choice([0, 0, 1, max(1, rows // rng.choice([2, 3, 7]))])
        post, pre = rng.choice([(True, True), (True, True), (False, True), (True, False)])
        return dict(op=op, rows=rows, dim=dim, kind=kind, act=act, res=res, gate_span=span,
                    post=post, pre=pre, bias=kind == "layer")
    vocab, top = _log_int(rng, 4000, 50257), _log_int(rng, 1, 256)
    logits = rng.choice(["bf16", "bf16", "f32"])
    rows = _log_int(rng, 1, 8192)
    if logits == "f32":
        rows = max(1, rows // 2)
    return dict(op=op, rows=rows, vocab=vocab, top=top, logits=logits,
                teacher=rng.choice(["bf16", "f32"]), tau=rng.choice([1.0, 1.5, 2.0, 4.0]),
                labels=rng.random() < 0.7)


# -------------------------------------------------------------------- inputs
def _ids(gen, n, vocab, pad, wide):
    """Token ids as text has them: rank-frequency 1/(rank + 2.7), low ids the
    frequent ones; `pad` of the tokens, at the end, are padding (-1)."""
    p = 1.0 / (torch.arange(vocab, device="cuda", dtype=torch.float64) + 2.7)
    cdf = torch.cumsum(p, 0)
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64) * cdf[-1]
    ids = torch.searchsorted(cdf, u).clamp_(max=vocab - 1)
    n_pad = int(n * pad)
    if n_pad:
        ids[n - n_pad:] = -1
    return ids if wide else ids.to(torch.int32)


def _randn(gen, shape, dtype, sigma=1.0, mean=0.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return x.mul_(sigma).add_(mean).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 17)
    s = dict(case=case)
    op = case["op"]
    if op == "embed":
        V, D, T = case["vocab"], case["dim"], case["tokens"]
        s["table"] = _randn(gen, (V, D), _TYPES[case["table"]], 0.02)
        s["ids"] = _ids(gen, T, V, case["pad"], case["wide_ids"])
        if own:
            s["out"] = torch.empty((T, D), dtype=_TYPES[case["out"]], device="cuda")
    elif op == "embed_grad":
        V, D, T = case["vocab"], case["dim"], case["tokens"]
        s["dout"] = _randn(gen, (T, D), _TYPES[case["dout"]], 1e-3)
        s["ids"] = _ids(gen, T, V, case["pad"], case["wide_ids"])
        if own:
            s["dtable"] = torch.empty((V, D), dtype=_TYPES[case["grad"]], device="cuda")
            s["scratch"] = torch.empty(_lib().zero_embed_scratch_bytes(T, V, D),
                                       dtype=torch.uint8, device="cuda")
    elif op in ("norm", "norm_grad"):
        R, D = case["rows"], case["dim"]
        act, res = _TYPES[case["act"]], _TYPES[case["res"]]
        span = case["gate_span"]
        groups = 1 if span == 0 else (R + span - 1) // span
        s["span"] = R if span == 0 else span
        s["branch"] = _randn(gen, (R, D), act, 0.7, 0.05)
        s["gate"] = _randn(gen, (groups, D), torch.bfloat16, 0.3, 0.8)
        for n in ("post", "pre"):
            s[n + "_weight"] = _randn(gen, (D,), torch.bfloat16, 0.1, 1.0) if case[n] else None
            s[n + "_bias"] = (_randn(gen, (D,), torch.bfloat16, 0.05)
                              if case[n] and case["bias"] else None)
        if op == "norm":
            s["x"] = _randn(gen, (R, D), res, 2.0)
            if own:
                s["y"] = torch.empty((R, D), dtype=res, device="cuda")
                s["u"] = torch.empty((R, D), dtype=act, device="cuda") if case["pre"] else None
        else:
            s["y"] = _randn(gen, (R, D), res, 2.0)
            s["dy"] = _randn(gen, (R, D), res, 1e-3)
            s["du"] = _randn(gen, (R, D), act, 1e-3) if case["pre"] else None
            if own:
                s["dx"] = torch.empty((R, D), dtype=res, device="cuda")
                s["dbranch"] = torch.empty((R, D), dtype=act, device="cuda")
                s["dgate"] = torch.empty_like(s["gate"])
                for n in ("post_weight", "post_bias", "pre_weight", "pre_bias"):
                    s["d" + n] = torch.empty_like(s[n]) if s[n] is not None else None
                s["scratch"] = torch.empty(_lib().zero_block_norm_scratch_bytes(R, D, s["span"]),
                                           dtype=torch.uint8, device="cuda")
    else:
        R, V, K = case["rows"], case["vocab"], case["top"]
        logits = torch.empty((R, V), dtype=_TYPES[case["logits"]], device="cuda")
        tl = torch.empty((R, K), dtype=_TYPES[case["teacher"]], device="cuda")
        ti = torch.empty((R, K), dtype=torch.int32, device="cuda")
        labels = torch.empty(R, dtype=torch.int64, device="cuda")
        for a in range(0, R, 1024):
            b = min(R, a + 1024)
            t = torch.randn((b - a, V), generator=gen, device="cuda") * 2.5
            noise = torch.randn((b - a, V), generator=gen, device="cuda")
            top, idx = torch.topk(t, K, dim=1)
            logits[a:b] = 0.8 * t + noise  # a student that has learned part of the teacher
            tl[a:b], ti[a:b] = top, idx.to(torch.int32)
            labels[a:b] = idx[:, min(1, K - 1)]
        short = torch.rand(R, generator=gen, device="cuda") < 0.1  # nucleus lists shorter than K
        ti[:, (K + 1) // 2:] = torch.where(short[:, None], -1, ti[:, (K + 1) // 2:])
        prompt = torch.rand(R, generator=gen, device="cuda") < 0.1  # no label on prompt tokens
        s["labels"] = torch.where(prompt, -100, labels) if case["labels"] else None
        weight = torch.full((R,), 1.0 / R, device="cuda")
        weight[R - R // 32:] = 0.0  # padding tokens
        s.update(logits=logits, teacher_logits=tl, teacher_ids=ti, row_weight=weight)
        if own:
            s["ce"] = torch.empty(R, device="cuda")
            s["kl"] = torch.empty(R, device="cuda")
            if op == "distill_grad":
                s["dlogits"] = torch.empty_like(logits)
    return s


CE_WEIGHT, KL_WEIGHT = 0.4, 0.6
RESIDUAL_SCALE, BRANCH_SCALE, EPS = 0.9, 0.5, 1e-5


# ------------------------------------------------------- the library's calls
def _run_own(s):
    Z, c = _lib(), s["case"]
    op = c["op"]
    if op == "embed":
        Z.zero_embed_forward(s["table"], s["ids"], s["out"], scale=c["scale"])
        return {"out": s["out"]}
    if op == "embed_grad":
        Z.zero_embed_backward(s["dout"], s["ids"], s["dtable"], s["scratch"], scale=c["scale"])
        return {"dtable": s["dtable"]}
    if op in ("norm", "norm_grad"):
        common = dict(branch=s["branch"], gate=s["gate"], rows_per_gate=s["span"],
                      post_norm=c["post"], pre_norm=c["pre"], post_weight=s["post_weight"],
                      post_bias=s["post_bias"], pre_weight=s["pre_weight"], kind=c["kind"],
                      eps=EPS, residual_scale=RESIDUAL_SCALE, branch_scale=BRANCH_SCALE)
        if op == "norm":
            Z.zero_block_norm_forward(s["x"], pre_bias=s["pre_bias"], y=s["y"], u=s["u"],
                                      **common)
            return {k: s[k] for k in ("y", "u") if s[k] is not None}
        grads = {k: s[k] for k in ("dx", "dbranch", "dgate", "dpost_weight", "dpost_bias",
                                   "dpre_weight", "dpre_bias") if s[k] is not None}
        Z.zero_block_norm_backward(s["y"], s["scratch"], dy=s["dy"], du=s["du"], **common,
                                   **grads)
        return grads
    common = dict(labels=s["labels"], row_weight=s["row_weight"], temperature=c["tau"])
    if op == "distill":
        Z.zero_distill_forward(s["logits"], s["teacher_logits"], s["teacher_ids"], s["ce"],
                               s["kl"], **common)
        return {"ce": s["ce"], "kl": s["kl"]}
    Z.zero_distill_forward_backward(s["logits"], s["teacher_logits"], s["teacher_ids"], s["ce"],
                                    s["kl"], s["dlogits"], ce_weight=CE_WEIGHT,
                                    kl_weight=KL_WEIGHT, **common)
    return {"ce": s["ce"], "kl": s["kl"], "dlogits": s["dlogits"]}


# ------------------------------------------------------------ the plain forms
def _norm_plain(v, w, b, kind):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    xh = v * r
    out = xh if w is None else xh * w.float()
    return (out if b is None else out + b.float()), xh, r


def _norm_back_plain(d, w, xh, r, kind):
    dw = d if w is None else d * w.float()
    g = dw - xh * (dw * xh).mean(1, keepdim=True)
    if kind == "layer":
        g = g - dw.mean(1, keepdim=True)
    return g * r


def _gate_rows(s, R):
    gate = s["gate"].float()
    if gate.shape[0] == 1:
        return gate
    return gate[torch.arange(R, device="cuda") // s["span"]]


def _group_sum(x, groups, span):
    """Sums of consecutive runs of `span` rows."""
    if groups == 1:
        return x.sum(0, keepdim=True)
    if span == 1:
        return x
    rest = groups * span - x.shape[0]
    if rest:
        x = torch.cat([x, x.new_zeros((rest, x.shape[1]))])
    return x.view(groups, span, -1).sum(1)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "embed":
        ids = s["ids"].long()
        ok = (ids >= 0) & (ids < c["vocab"])
        rows = s["table"][torch.where(ok, ids, 0)].float() * c["scale"]
        return {"out": torch.where(ok[:, None], rows, 0.0).to(_TYPES[c["out"]])}
    if op == "embed_grad":
        ids = s["ids"].long()
        V = c["vocab"]
        acc = torch.zeros((V + 1, c["dim"]), device="cuda")
        acc.index_add_(0, torch.where((ids >= 0) & (ids < V), ids, V), s["dout"].float())
        return {"dtable": (acc[:V] * c["scale"]).to(_TYPES[c["grad"]])}
    if op == "norm":
        R, act, res = c["rows"], _TYPES[c["act"]], _TYPES[c["res"]]
        n = s["branch"].float()
        if c["post"]:
            n = _norm_plain(n, s["post_weight"], s["post_bias"], c["kind"])[0]
        y = s["x"].float() * RESIDUAL_SCALE + n * _gate_rows(s, R) * BRANCH_SCALE
        out = {"y": y.to(res)}
        if c["pre"]:
            out["u"] = _norm_plain(y, s["pre_weight"], s["pre_bias"], c["kind"])[0].to(act)
        return out
    if op == "norm_grad":
        R, act, res = c["rows"], _TYPES[c["act"]], _TYPES[c["res"]]
        out = {}
        g = s["dy"].float()
        if c["pre"]:
            du = s["du"].float()
            _, xh, r = _norm_plain(s["y"].float(), None, None, c["kind"])
            g = g + _norm_back_plain(du, s["pre_weight"], xh, r, c["kind"])
            out["dpre_weight"] = (du * xh).sum(0).to(torch.bfloat16)
            if c["bias"]:
                out["dpre_bias"] = du.sum(0).to(torch.bfloat16)
        out["dx"] = (g * RESIDUAL_SCALE).to(res)
        g = g * BRANCH_SCALE
        d = g * _gate_rows(s, R)
        h = s["branch"].float()
        if c["post"]:
            n, xh, r = _norm_plain(h, s["post_weight"], s["post_bias"], c["kind"])
            out["dbranch"] = _norm_back_plain(d, s["post_weight"], xh, r, c["kind"]).to(act)
            out["dpost_weight"] = (d * xh).sum(0).to(torch.bfloat16)
            if c["bias"]:
                out["dpost_bias"] = d.sum(0).to(torch.bfloat16)
        else:
            n = h
            out["dbranch"] = d.to(act)
        out["dgate"] = _group_sum(g * n, s["gate"].shape[0], s["span"]).to(torch.bfloat16)
        return {k: out[k] for k in ("dx", "dbranch", "dgate", "dpost_weight", "dpost_bias",
                                    "dpre_weight", "dpre_bias") if k in out}
    return _distill_plain(s, op == "distill_grad")


def _distill_plain(s, grad):
    c = s["case"]
    V, tau = c["vocab"], c["tau"]
    x = s["logits"].float()
    live = s["row_weight"] != 0
    ids = s["teacher_ids"].long()
    valid = (ids >= 0) & (ids < V)
    at = torch.where(valid, ids, 0)
    t = torch.where(valid, s["teacher_logits"].float() / tau, -math.inf)
    tm = t.amax(1, keepdim=True)
    has = (tm > -math.inf) & live[:, None]
    e = torch.exp(t - torch.where(has, tm, 0.0))
    z = torch.where(has, e.sum(1, keepdim=True), 1.0)
    p = torch.where(has, e / z, 0.0)
    m = x.amax(1, keepdim=True)
    e_tau = torch.exp((x - m) / tau)
    z_tau = e_tau.sum(1, keepdim=True)
    logq = (torch.gather(x, 1, at) - m) / tau - torch.log(z_tau)
    logp = t - torch.where(has, tm, 0.0) - torch.log(z)
    kl = torch.where(p > 0, p * (logp - logq), 0.0).sum(1) * (tau * tau)
    ce = torch.zeros_like(kl)
    labelled = None
    if s["labels"] is not None:
        e_one = torch.exp(x - m)
        z_one = e_one.sum(1, keepdim=True)
        labelled = (s["labels"] >= 0) & (s["labels"] < V) & live
        label = torch.where(labelled, s["labels"], 0)[:, None]
        value = (torch.log(z_one) - (torch.gather(x, 1, label) - m))[:, 0]
        ce = torch.where(labelled, value, 0.0)
    out = {"ce": ce, "kl": kl}
    if grad:
        on = has.float() * (KL_WEIGHT * tau)
        g = e_tau * (on / z_tau)
        g.scatter_add_(1, at, -p * on)
        if labelled is not None:
            on = labelled[:, None].float() * CE_WEIGHT
            g += e_one * (on / z_one)
            g.scatter_add_(1, label, -on)
        out["dlogits"] = (g * s["row_weight"][:, None]).to(_TYPES[c["logits"]])
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------- definitions in fp64
def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "embed":
        out = torch.zeros((c["tokens"], c["dim"]), dtype=torch.float64, device="cuda")
        inside = torch.nonzero((s["ids"] >= 0) & (s["ids"] < c["vocab"]))[:, 0]
        out[inside] = c["scale"] * s["table"][s["ids"][inside].long()].double()
        return {"out": out}
    if op == "embed_grad":
        out = torch.zeros((c["vocab"], c["dim"]), dtype=torch.float64, device="cuda")
        inside = torch.nonzero((s["ids"] >= 0) & (s["ids"] < c["vocab"]))[:, 0]
        out.index_put_((s["ids"][inside].long(),), s["dout"][inside].double() * c["scale"],
                       accumulate=True)
        return {"dtable": out}
    if op in ("norm", "norm_grad"):
        return _exact_norm(s, op == "norm_grad")
    return _exact_distill(s, op == "distill_grad")


def _exact_norm(s, grad):
    c = s["case"]
    R, D, layer = c["rows"], c["dim"], c["kind"] == "layer"
    block = 2048
    out = {}

    def wide(name):
        return None if s[name] is None else s[name].double()

    def stats(v):
        mu = v.sum(1, keepdim=True) / D if layer else torch.zeros_like(v[:, :1])
        sd = torch.sqrt(((v - mu) ** 2).sum(1, keepdim=True) / D + EPS)
        return mu, sd

    def affine(v, w, b):
        v = v if w is None else v * w
        return v if b is None else v + b

    def pull(d, v, mu, sd):
        """The transposed Jacobian of (v - mu) / sd applied to d."""
        centred = v - mu
        a = d - d.sum(1, keepdim=True) / D if layer else d
        return a / sd - centred * ((d * centred).sum(1, keepdim=True) / (D * sd ** 3))

    pw, pb, qw, qb = (wide(n) for n in ("post_weight", "post_bias", "pre_weight", "pre_bias"))
    gate = s["gate"].double()
    shape = (R, D)
    if not grad:
        out["y"] = torch.empty(shape, dtype=torch.float64, device="cuda")
        if c["pre"]:
            out["u"] = torch.empty_like(out["y"])
    else:
        out["dx"] = torch.empty(shape, dtype=torch.float64, device="cuda")
        out["dbranch"] = torch.empty_like(out["dx"])
        out["dgate"] = torch.zeros_like(gate)
        for n in ("post_weight", "post_bias", "pre_weight", "pre_bias"):
            if s[n] is not None:
                out["d" + n] = torch.zeros(D, dtype=torch.float64, device="cuda")
    for a in range(0, R, block):
        b = min(R, a + block)
        which = torch.arange(a, b, device="cuda") // s["span"]
        h = s["branch"][a:b].double()
        if c["post"]:
            mu, sd = stats(h)
            hh = (h - mu) / sd
            n = affine(hh, pw, pb)
        else:
            n = h
        if not grad:
            y = RESIDUAL_SCALE * s["x"][a:b].double() + BRANCH_SCALE * gate[which] * n
            out["y"][a:b] = y
            if c["pre"]:
                m2, s2 = stats(y)
                out["u"][a:b] = affine((y - m2) / s2, qw, qb)
            continue
        g = s["dy"][a:b].double()
        if c["pre"]:
            y, du = s["y"][a:b].double(), s["du"][a:b].double()
            m2, s2 = stats(y)
            g = g + pull(affine(du, qw, None), y, m2, s2)
            out["dpre_weight"] += (du * (y - m2) / s2).sum(0)
            if qb is not None:
                out["dpre_bias"] += du.sum(0)
        out["dx"][a:b] = RESIDUAL_SCALE * g
        d = BRANCH_SCALE * gate[which] * g
        out["dgate"].index_put_((which,), BRANCH_SCALE * g * n, accumulate=True)
        if c["post"]:
            out["dbranch"][a:b] = pull(affine(d, pw, None), h, mu, sd)
            out["dpost_weight"] += (d * hh).sum(0)
            if pb is not None:
                out["dpost_bias"] += d.sum(0)
        else:
            out["dbranch"][a:b] = d
    return out


def _exact_distill(s, grad):
    c = s["case"]
    R, V, tau = c["rows"], c["vocab"], c["tau"]
    ce = torch.zeros(R, dtype=torch.float64, device="cuda")
    kl = torch.zeros_like(ce)
    out = {"ce": ce, "kl": kl}
    if grad:
        out["dlogits"] = torch.zeros((R, V), dtype=torch.float64, device="cuda")
    for a in range(0, R, 512):
        b = min(R, a + 512)
        x = s["logits"][a:b].double()
        w = s["row_weight"][a:b].double()
        ids = s["teacher_ids"][a:b].long()
        inside = (ids >= 0) & (ids < V)
        teacher = s["teacher_logits"][a:b].double() / tau
        teacher[~inside] = -math.inf
        logp = torch.log_softmax(teacher, 1)
        p = torch.exp(logp)
        p[~inside] = 0.0  # also where a row has no entry at all
        counted = inside.any(1) & (w != 0)
        logq = torch.log_softmax(x / tau, 1)
        terms = p * (logp - torch.gather(logq, 1, ids.clamp(0, V - 1)))
        terms[~inside] = 0.0
        kl[a:b] = torch.where(counted, tau ** 2 * terms.sum(1), 0.0)
        if grad:
            g = torch.exp(logq)
            g.scatter_add_(1, ids.clamp(0, V - 1), -p)
            g *= (counted * KL_WEIGHT * tau)[:, None]
        if s["labels"] is not None:
            lab = s["labels"][a:b]
            has = (lab >= 0) & (lab < V) & (w != 0)
            logq1 = torch.log_softmax(x, 1)
            pick = torch.gather(logq1, 1, lab.clamp(0, V - 1)[:, None])[:, 0]
            ce[a:b] = torch.where(has, -pick, 0.0)
            if grad:
                one = torch.exp(logq1)
                one[torch.arange(b - a, device="cuda"), lab.clamp(0, V - 1)] -= 1.0
                g += one * (has * CE_WEIGHT)[:, None]
        if grad:
            out["dlogits"][a:b] = g * w[:, None]
    return out


# ---------------------------------------------------------------------- work
def _expected_rows(tokens, vocab):
    """Distinct rows among `tokens` ids of the distribution of _ids."""
    p = 1.0 / (torch.arange(vocab, dtype=torch.float64) + 2.7)
    return float((1.0 - (1.0 - p / p.sum()) ** tokens).sum())


def work(case):
    c, op = case, case["op"]
    if op == "embed":
        rows = _expected_rows(c["tokens"], c["vocab"])
        return {"bytes": rows * c["dim"] * _SIZE[c["table"]]
                + c["tokens"] * (c["dim"] * _SIZE[c["out"]] + (8 if c["wide_ids"] else 4)),
                "flops": c["tokens"] * c["dim"]}
    if op == "embed_grad":
        return {"bytes": c["vocab"] * c["dim"] * _SIZE[c["grad"]]
                + c["tokens"] * (c["dim"] * _SIZE[c["dout"]] + (8 if c["wide_ids"] else 4)),
                "flops": c["tokens"] * c["dim"]}
    if op in ("norm", "norm_grad"):
        n = c["rows"] * c["dim"]
        act, res = _SIZE[c["act"]], _SIZE[c["res"]]
        groups = 1 if c["gate_span"] == 0 else -(-c["rows"] // c["gate_span"])
        vectors = groups + (c["post"] + c["pre"]) * (2 if c["bias"] else 1)
        if op == "norm":
            # x and branch in, y and u out
            total = n * (2 * res + act + (act if c["pre"] else 0)) + 2 * c["dim"] * vectors
            return {"bytes": total, "flops": 10 * n}
        # dy, branch, and du and y for the norm before the next block, in; dx and dbranch out
        total = n * (2 * res + 2 * act + ((res + act) if c["pre"] else 0))
        return {"bytes": total + 4 * c["dim"] * vectors, "flops": 24 * n}
    n = c["rows"] * c["vocab"]
    size = _SIZE[c["logits"]]
    per_row = c["top"] * (4 + _SIZE[c["teacher"]]) + 12 + (8 if c["labels"] else 0)
    passes = 2 if op == "distill_grad" else 1
    return {"bytes": n * size * passes + c["rows"] * per_row,
            "flops": n * (8 if op == "distill_grad" else 4) * (2 if c["labels"] else 1)}
