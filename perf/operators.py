"""Cases of the serving operators: the whole MoE layer for a few tokens
(moe_forward_few) and the per-request low-rank adapters beside a shared
projection (moe_adapter_linear).

A case is a dict of plain values.  `prepare` makes its inputs on the GPU,
`run` is one pass (the plain form in elementary torch operations, or with
`own` the library's kernels), `exact` the definition in float64.
"""
from __future__ import annotations

import math

import torch

own = False

WD = {"bf16": 1, "fp8_e4m3": 2, "int8": 3, "int4": 4}   # moe_dtype of the weights
W_BYTES = {"bf16": 2.0, "fp8_e4m3": 1.0, "int8": 1.0, "int4": 0.5}
MARGIN = 1e-4   # tokens whose routing hangs on less than this are not drawn


def _few(name, T, d, E, k, d_ff, w, shared=False, groups=0, topk_groups=0, cf=0.0,
         overflow="drop", bias=False):
    return dict(name=name, op="few", T=T, d=d, E=E, k=k, d_ff=d_ff, w=w, shared=shared,
                groups=groups, topk_groups=topk_groups, cf=cf, overflow=overflow, bias=bias)


def _adapter(name, T, d_in, d_out, n, rank, w, y, requests, bias=False, base=False, ragged=False):
    return dict(name=name, op="adapter", T=T, d_in=d_in, d_out=d_out, n=n, rank=rank, w=w, y=y,
                requests=requests, bias=bias, base=base, ragged=ragged)


def listed():
    return [
        # one user's next token through the narrow 64-expert layer: latency counts
        _few("few_64experts_t1", 1, 4096, 64, 2, 1408, "bf16", bias=True),
        # one token through the Mixtral-shaped layer: two experts' weights streamed
        _few("few_mixtral_t1", 1, 4096, 8, 2, 14336, "bf16"),
        # a decode batch of eight over the same weights in fp8
        _few("few_mixtral_t8_fp8", 8, 4096, 8, 2, 14336, "fp8_e4m3"),
        # the benchmark's decode batch: every expert touched
        _few("few_mixtral_t64", 64, 4096, 8, 2, 14336, "bf16"),
        # fine-grained layer with its shared expert and device-limited routing, a
        # ragged batch, 4-bit weights
        _few("few_fine_t13_int4", 13, 7168, 256, 8, 2048, "int4", shared=True, groups=8,
             topk_groups=4),
        # a small layer whose capacity drops assignments to the shared expert
        _few("few_small_t37_int8", 37, 768, 32, 8, 256, "int8", shared=True, cf=0.75,
             overflow="shared", bias=True),
        # one request's next token through an attention-output-sized projection
        _adapter("adapter_t1", 1, 4096, 4096, 32, 16, "bf16", "bf16", "scattered"),
        # a decode batch, every row of another request, into a wide fp8 projection
        _adapter("adapter_t64_fp8", 64, 4096, 14336, 128, 16, "fp8_e4m3", "bf16", "scattered",
                 bias=True),
        # a ragged decode batch with adapters of different ranks
        _adapter("adapter_t27_int4", 27, 7168, 2048, 48, 64, "int4", "f32", "scattered",
                 ragged=True),
        # short prompts of several requests together, a width that fills no tile
        _adapter("adapter_t333", 333, 4096, 1416, 16, 32, "bf16", "bf16", "runs", bias=True,
                 ragged=True),
        # whole prompts of a few requests into the wide projection
        _adapter("adapter_t4096", 4096, 4096, 14336, 8, 16, "bf16", "bf16", "runs"),
        # adapters in parallel with the layer, added to its fp32 output
        _adapter("adapter_beside_layer_t2048", 2048, 4096, 4096, 24, 32, "none", "f32", "runs",
                 base=True, ragged=True),
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return max(lo, min(hi, int(v) // step * step))


_CAP = {}


def _largest(op):
    if op not in _CAP:
        ws = [work(c) for c in listed() if c["op"] == op]
        _CAP[op] = (max(w["bytes"] for w in ws), max(w["flops"] for w in ws))
    return _CAP[op]


def draw(rng):
    """One more case: sizes spread over the listed ranges, no costlier than
    the largest listed case of its operator."""
    op = rng.choice(["few", "adapter"])
    while True:
        w = rng.choice(list(WD))
        if op == "few":
            E = _log_int(rng, 1, 256)
            groups = rng.choice([g for g in (0, 0, 2, 4, 8) if g == 0 or E % g == 0])
            tg = rng.randint(1, groups) if groups else 0
            kmax = min(8, E if not groups else tg * (E // groups))
            shared = rng.random() < 0.4
            cf = rng.choice([0.0, 0.0, 0.5, 1.25])
            overflow = rng.choice(["drop", "shared"]) if shared and cf else "drop"
            # quantised matrices hold a scale per 128 rows
            c = _few("", _log_int(rng, 1, 64),
                     _log_int(rng, 256, 7168, 64 if w == "bf16" else 128), E,
                     rng.randint(1, kmax), _log_int(rng, 128, 14336, 128), w, shared, groups, tg,
                     cf, overflow, rng.random() < 0.3)
            if 3.0 * E * c["d"] * c["d_ff"] * W_BYTES[w] > 6e9:   # the stored weights
                continue
        else:
            quant = w != "bf16"
            if rng.random() < 0.15:
                w, quant = "none", False
            c = _adapter("", _log_int(rng, 1, 4096), _log_int(rng, 256, 7168, 64 if quant else 8),
                         _log_int(rng, 256, 14336, 128) if quant else _log_int(rng, 250, 14336),
                         _log_int(rng, 1, 128), _log_int(rng, 8, 64, 8), w,
                         rng.choice(["bf16", "f32"]), rng.choice(["runs", "scattered"]),
                         rng.random() < 0.4, rng.random() < 0.3, rng.random() < 0.5)
        del c["name"]
        cost, cap = work(c), _largest(op)
        if cost["bytes"] <= cap[0] and cost["flops"] <= cap[1]:
            return c


def work(case):
    """Bytes and operations one pass cannot do without.  Which experts and
    adapters a batch touches is random; the expected number of distinct ones
    is counted."""
    c = case
    if c["op"] == "few":
        T, d, E, k, d_ff = c["T"], c["d"], c["E"], c["k"], c["d_ff"]
        A = T * k
        touched = E * (1.0 - (1.0 - k / E) ** T)
        kept = min(A, E * _capacity(c)) if c["cf"] else A
        mats = 3.0 * d * d_ff * W_BYTES[c["w"]]
        by = touched * mats + (mats if c["shared"] else 0.0)
        by += d * E * 4.0 + T * d * (2.0 + 4.0) + A * 8.0 + E * 8.0
        fl = 6.0 * d * d_ff * (kept + (T if c["shared"] else 0)) + 2.0 * T * d * E
        return {"bytes": int(by), "flops": int(fl)}
    T, di, do = c["T"], c["d_in"], c["d_out"]
    yb = 2.0 if c["y"] == "bf16" else 4.0
    r = c["rank"] * (0.625 if c["ragged"] else 1.0)
    adapted = 0.9 * T
    distinct = c["n"] * (1.0 - (1.0 - 1.0 / c["n"]) ** (adapted if c["requests"] == "scattered"
                                                        else _run_count(c)))
    by = T * di * 2.0 + T * do * yb * (2 if c["base"] else 1) + T * 4.0
    by += distinct * r * (di + do) * 2.0 + (do * 4.0 if c["bias"] else 0.0)
    fl = 2.0 * r * (di + do) * adapted
    if c["w"] != "none":
        by += di * do * W_BYTES[c["w"]]
        fl += 2.0 * T * di * do
    return {"bytes": int(by), "flops": int(fl)}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g, dtype=torch.float32)


def _matrix(g, lead, out, inn, w):
    """Random weights [lead, out, in] of std 1/sqrt(in) in format w, and their
    scales [lead, out/128] (None for bf16): made matrix by matrix."""
    std = 1.0 / math.sqrt(inn)
    n = lead if lead else 1
    if w == "bf16":
        q = torch.empty(n, out, inn, dtype=torch.bfloat16, device="cuda")
        for i in range(n):
            q[i] = (_randn(g, out, inn) * std).to(torch.bfloat16)
        return (q if lead else q[0]), None
    width = inn // 2 if w == "int4" else inn
    q = torch.empty(n, out, width, dtype=torch.int8 if w == "int8" else torch.uint8, device="cuda")
    unit = {"fp8_e4m3": 100.0, "int8": 32.0, "int4": 2.25}[w]
    for i in range(n):
        v = _randn(g, out, inn) * unit
        if w == "fp8_e4m3":
            q[i] = v.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        elif w == "int8":
            q[i] = v.round_().clamp_(-127, 127).to(torch.int8)
        else:
            code = (v.round_().clamp_(-7, 7) + 8).to(torch.uint8).view(out, inn // 8, 8)
            q[i] = (code[:, :, :4] | (code[:, :, 4:] << 4)).view(out, width)
    s = (torch.rand(n, out // 128, device="cuda", generator=g) * 0.2 + 0.9) * (std / unit)
    return (q, s) if lead else (q[0], s[0])


def _capacity(c):
    return math.ceil(c["cf"] * float(c["T"] * c["k"]) / float(c["E"]))


def _margin(l, k, groups, topk_groups):
    """Per token: the least gap that its routing hangs on."""
    m = torch.full((l.shape[0],), float("inf"), dtype=l.dtype, device=l.device)
    if groups > 1:
        best = l.view(l.shape[0], groups, -1).amax(2)
        gs = best.sort(1, descending=True).values
        if topk_groups < groups:
            m = gs[:, topk_groups - 1] - gs[:, topk_groups]
        kept = best >= gs[:, topk_groups - 1:topk_groups]
        l = l.view(l.shape[0], groups, -1).masked_fill(~kept[:, :, None], -float("inf"))
        l = l.flatten(1)
    s = l.sort(1, descending=True).values[:, :k + 1]
    if s.shape[1] > 1:
        gaps = (s[:, :-1] - s[:, 1:]).nan_to_num(nan=float("inf"), posinf=float("inf"))
        m = torch.minimum(m, gaps.amin(1))
    return m


def _few_inputs(c, seed):
    g = _gen(seed)
    T, d, E = c["T"], c["d"], c["E"]
    W_g = _randn(g, d, E) / math.sqrt(d)
    b_g = _randn(g, E) * 0.5 if c["bias"] else None
    pool = _randn(g, T + 64, d).to(torch.bfloat16)
    l = pool.double() @ W_g.double()
    if b_g is not None:
        l = l + b_g.double()
    # routing that hangs on a rounding is no case: such rows are passed over
    clear = _margin(l, c["k"], c["groups"], c["topk_groups"]) > MARGIN
    order = torch.argsort((~clear).to(torch.int8), stable=True)[:T]
    x = pool[order].contiguous()
    wt = {}
    for m, out, inn in (("1", c["d_ff"], d), ("3", c["d_ff"], d), ("2", d, c["d_ff"])):
        wt["W" + m], s = _matrix(g, E, out, inn, c["w"])
        if s is not None:
            wt["s" + m] = s
        if c["shared"]:
            wt["W" + m + "s"], s = _matrix(g, 0, out, inn, c["w"])
            if s is not None:
                wt["s" + m + "s"] = s
    return dict(x=x, W_g=W_g, b_g=b_g, wt=wt)


def _run_count(c):
    return max(1, min(2 * c["n"], c["T"] // 16))


def _adapter_inputs(c, seed):
    g = _gen(seed)
    T, di, do, n, R = c["T"], c["d_in"], c["d_out"], c["n"], c["rank"]
    x = _randn(g, T, di).to(torch.bfloat16)
    W = s = None
    if c["w"] != "none":
        W, s = _matrix(g, 0, do, di, c["w"])
    A = (_randn(g, n, R, di) / math.sqrt(di)).to(torch.bfloat16)
    B = (_randn(g, n, do, R) / math.sqrt(R)).to(torch.bfloat16)
    scales = torch.rand(n, device="cuda", generator=g) + 0.5
    ranks = None
    if c["ragged"]:
        ranks = torch.randint(max(1, R // 4), R + 1, (n,), device="cuda", generator=g,
                              dtype=torch.int32)
    if c["requests"] == "scattered":      # every row its own request
        idx = torch.randint(0, n, (T,), device="cuda", generator=g, dtype=torch.int32)
        bare = torch.rand(T, device="cuda", generator=g) < 0.1
    else:                                  # prompts: runs of rows of one request
        m = _run_count(c)
        cuts = torch.randint(0, T, (m - 1,), device="cuda", generator=g).sort().values
        run_of = torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)
        idx = torch.randint(0, n, (m,), device="cuda", generator=g, dtype=torch.int32)[run_of]
        bare = (torch.rand(m, device="cuda", generator=g) < 0.1)[run_of]
    idx = torch.where(bare, torch.full_like(idx, -1), idx).contiguous()
    bias = _randn(g, do) if c["bias"] else None
    ydt = torch.bfloat16 if c["y"] == "bf16" else torch.float32
    base = _randn(g, T, do).to(ydt) if c["base"] else None
    return dict(x=x, W=W, s=s, A=A, B=B, scales=scales, ranks=ranks, idx=idx, bias=bias,
                base=base, ydt=ydt)


def prepare(case, seed):
    """Inputs on the GPU and what a program keeps beside them: the shape, the
    weights' struct, the packed gate, the workspace and the output buffers."""
    c = case
    st = _few_inputs(c, seed) if c["op"] == "few" else _adapter_inputs(c, seed)
    st["case"] = c
    if not own:
        return st
    import mixture_experts_layer_bincount_amd as moe
    st["moe"] = moe
    if c["op"] == "few":
        T, d, E, k = c["T"], c["d"], c["E"], c["k"]
        sh = moe.make_shape(T, d, E, k, c["d_ff"], _capacity(c) if c["cf"] else -1,
                            w_dtype=WD[c["w"]], has_shared=c["shared"], overflow=c["overflow"],
                            n_groups=c["groups"], topk_groups=c["topk_groups"])
        packed = torch.empty(moe.moe_router_packed_bytes(sh), dtype=torch.uint8, device="cuda")
        moe.moe_pack_router(sh, st["W_g"], packed)
        sh.router_packed = 1
        i32 = dict(dtype=torch.int32, device="cuda")
        st.update(shape=sh, packed=packed, weights=moe.make_weights(**st["wt"]),
                  ws=moe.few_workspace(sh), y=torch.empty(T, d, device="cuda"),
                  topk_idx=torch.empty(T, k, **i32), topk_w=torch.empty(T, k, device="cuda"),
                  counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32))
    else:
        sh = moe.make_adapter_shape(c["T"], c["d_in"], c["d_out"], c["n"], c["rank"],
                                    w_dtype=WD.get(c["w"], 1),
                                    y_dtype=moe.DT_BF16 if c["y"] == "bf16" else moe.DT_F32)
        st.update(shape=sh, ws=moe.adapter_workspace(sh),
                  y=torch.empty(c["T"], c["d_out"], dtype=st["ydt"], device="cuda"))
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    st = state
    if st["case"]["op"] == "few":
        return _few_own(st) if own else _few_plain(st)
    return _adapter_own(st) if own else _adapter_plain(st)


def _few_own(st):
    st["moe"].moe_forward_few(st["shape"], st["x"], st["packed"], st["b_g"], st["weights"],
                              st["y"], st["topk_idx"], st["topk_w"], st["counts"],
                              st["offsets"], st["ws"])
    return {n: st[n] for n in ("y", "topk_idx", "topk_w", "counts", "offsets")}


def _adapter_own(st):
    st["moe"].moe_adapter_linear(st["shape"], st["x"], st["W"], st["s"], st["bias"], st["A"],
                                 st["B"], st["ranks"], st["scales"], st["idx"], st["base"],
                                 st["y"], st["ws"])
    return {"y": st["y"]}


def _wide(q, s, w):
    """Weights in format w as fp32 [out, in]."""
    if w == "bf16":
        return q.float()
    if w == "fp8_e4m3":
        v = q.view(torch.float8_e4m3fn).float()
    elif w == "int8":
        v = q.float()
    else:
        b = q.view(q.shape[0], -1, 4)
        v = torch.cat((b & 15, b >> 4), 2).flatten(1).float() - 8.0
    return v * s.repeat_interleave(128)[:, None]


def _swiglu(x, wt, e, w, tag=""):
    def mat(m):
        q, s = wt["W" + m + tag], wt.get("s" + m + tag)
        return _wide(q if e is None else q[e], s if e is None or s is None else s[e], w)
    a = x @ mat("1").t()
    return (a / (1.0 + torch.exp(-a)) * (x @ mat("3").t())) @ mat("2").t()


def _few_plain(st):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = st["x"].float()
    logits = st["x"].double() @ st["W_g"].double()     # choices next to a border: 64 bits
    if st["b_g"] is not None:
        logits = logits + st["b_g"]
    pick = logits
    if c["groups"] > 1:
        best = logits.view(T, c["groups"], -1).amax(2)
        order = best.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, order, True)
        pick = logits.view(T, c["groups"], -1).masked_fill(~kept[:, :, None], -float("inf"))
        pick = pick.flatten(1)
    top, idx = pick.sort(dim=1, descending=True, stable=True)
    top, idx = top[:, :k].float(), idx[:, :k]
    ex = torch.exp(top - top[:, :1])
    wgt = ex / ex.sum(1, keepdim=True)
    hit = torch.zeros(T, E, dtype=torch.int32, device="cuda").scatter_(1, idx, 1)
    counts = hit.sum(0)
    keep = torch.ones_like(wgt, dtype=torch.bool)
    sizes = counts
    if c["cf"]:
        C = _capacity(c)
        keep = (hit.cumsum(0) - 1).gather(1, idx) < C
        sizes = counts.clamp(max=C)
    offsets = torch.cat((torch.zeros_like(sizes[:1]), sizes.cumsum(0)))
    y = torch.zeros(T, c["d"], device="cuda")
    for e in idx[keep].unique().tolist():
        t, j = ((idx == e) & keep).nonzero(as_tuple=True)
        y[t] += wgt[t, j][:, None] * _swiglu(x[t], st["wt"], e, c["w"])
    if c["shared"]:
        ws = torch.ones(T, device="cuda")
        if c["overflow"] == "shared":
            ws = ws + (wgt * ~keep).sum(1)
        y += ws[:, None] * _swiglu(x, st["wt"], None, c["w"], "s")
    return {"y": y, "topk_idx": idx.int(), "topk_w": wgt, "counts": counts.int(),
            "offsets": offsets.int()}


def _adapter_plain(st):
    c = st["case"]
    x = st["x"].float()
    y = torch.zeros(c["T"], c["d_out"], device="cuda")
    if c["w"] != "none":
        y = x @ _wide(st["W"], st["s"], c["w"]).t()
    if st["bias"] is not None:
        y = y + st["bias"]
    if st["base"] is not None:
        y = y + st["base"].float()
    idx = st["idx"]
    ranks = st["ranks"].tolist() if st["ranks"] is not None else None
    for a in idx[idx >= 0].unique().tolist():
        r = ranks[a] if ranks else c["rank"]
        rows = (idx == a).nonzero()[:, 0]
        v = (x[rows] @ st["A"][a, :r].float().t()) * st["scales"][a]
        y[rows] += v @ st["B"][a, :, :r].float().t()
    return {"y": y.to(st["ydt"])}


# ------------------------------------------------------------------ the definition in float64
def _exact_weights(q, s, w):
    """Format w decoded to float64, from the formats' definitions."""
    if w == "bf16":
        return q.double()
    if w == "fp8_e4m3":        # sign, 4 exponent bits (bias 7), 3 fraction bits
        b = q.long()
        ex, fr = (b >> 3) & 15, (b & 7).double()
        v = torch.where(ex == 0, fr / 8.0 * 2.0 ** -6,
                        (1.0 + fr / 8.0) * torch.exp2(ex.double() - 7.0))
        v = torch.where(b >= 128, -v, v)
    elif w == "int8":
        v = q.double()
    else:
        out, half = q.shape
        v = torch.empty(out, 2 * half, dtype=torch.float64, device=q.device)
        for b in range(4):
            v[:, b::8] = (q[:, b::4].int() % 16 - 8).double()
            v[:, b + 4::8] = (q[:, b::4].int() // 16 - 8).double()
    return (v.view(-1, 128, v.shape[1]) * s.double()[:, None, None]).view(v.shape)


def exact(case, seed):
    c = case
    if c["op"] == "adapter":
        return _exact_adapter(c, _adapter_inputs(c, seed))
    return _exact_few(c, _few_inputs(c, seed))


def _exact_few(c, inp):
    T, E, k, wt, w = c["T"], c["E"], c["k"], inp["wt"], c["w"]
    x = inp["x"].double()
    l = torch.empty(T, E, dtype=torch.float64, device="cuda")
    for t in range(T):
        l[t] = (x[t][:, None] * inp["W_g"].double()).sum(0)
    if inp["b_g"] is not None:
        l += inp["b_g"].double()
    lh = l.cpu().tolist()
    gs = E // c["groups"] if c["groups"] > 1 else E
    cap = _capacity(c) if c["cf"] else T * k
    load, kept = [0] * E, [0] * E
    idx, wgt, rows, dropped = [], [], {}, [0.0] * T
    for t in range(T):
        allowed = list(range(E))
        if c["groups"] > 1:
            score = [max(lh[t][g * gs:(g + 1) * gs]) for g in range(c["groups"])]
            ok = sorted(range(c["groups"]), key=lambda g: (-score[g], g))[:c["topk_groups"]]
            allowed = [e for e in allowed if e // gs in ok]
        chosen = sorted(allowed, key=lambda e: (-lh[t][e], e))[:k]
        z = [math.exp(lh[t][e] - lh[t][chosen[0]]) for e in chosen]
        p = [v / math.fsum(z) for v in z]
        idx.append(chosen)
        wgt.append(p)
        for e, pe in zip(chosen, p):
            load[e] += 1
            if kept[e] < cap:
                kept[e] += 1
                rows.setdefault(e, []).append((t, pe))
            else:
                dropped[t] += pe

    def ffn(xs, pick):
        a = torch.matmul(xs, pick("1").t())
        b = torch.matmul(xs, pick("3").t())
        return torch.matmul(a * torch.sigmoid(a) * b, pick("2").t())

    y = torch.zeros(T, c["d"], dtype=torch.float64, device="cuda")
    for e, tp in sorted(rows.items()):
        t = torch.tensor([v[0] for v in tp], device="cuda")
        p = torch.tensor([v[1] for v in tp], dtype=torch.float64, device="cuda")
        out = ffn(x.index_select(0, t), lambda m: _exact_weights(
            wt["W" + m][e], wt["s" + m][e] if w != "bf16" else None, w))
        y.index_add_(0, t, out * p[:, None])
    if c["shared"]:
        p = torch.tensor(dropped, dtype=torch.float64, device="cuda")
        p = 1.0 + (p if c["overflow"] == "shared" else 0.0 * p)
        y += p[:, None] * ffn(x, lambda m: _exact_weights(wt["W" + m + "s"],
                                                          wt.get("s" + m + "s"), w))
    off = [0]
    for e in range(E):
        off.append(off[-1] + kept[e])
    i32 = dict(dtype=torch.int32, device="cuda")
    return {"y": y, "topk_idx": torch.tensor(idx, **i32),
            "topk_w": torch.tensor(wgt, dtype=torch.float64, device="cuda"),
            "counts": torch.tensor(load, **i32), "offsets": torch.tensor(off, **i32)}


def _exact_adapter(c, inp):
    """y = base + bias + x W^T + scale * x A^T B^T, adapter by adapter over all
    rows, the rows of other adapters masked to zero."""
    x = inp["x"].double()
    y = torch.zeros(c["T"], c["d_out"], dtype=torch.float64, device="cuda")
    if inp["base"] is not None:
        y += inp["base"].double()
    if inp["bias"] is not None:
        y += inp["bias"].double()[None, :]
    if c["w"] != "none":
        y += torch.mm(x, _exact_weights(inp["W"], inp["s"], c["w"]).t().contiguous())
    for a in range(c["n"]):
        mine = (inp["idx"] == a).double()[:, None]
        r = int(inp["ranks"][a]) if inp["ranks"] is not None else c["rank"]
        low = torch.mm(x * mine, inp["A"][a, :r].double().t().contiguous())
        y += float(inp["scales"][a]) * torch.mm(low, inp["B"][a, :, :r].double().t().contiguous())
    return {"y": y}
