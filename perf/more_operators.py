"""Cases for the operators of a block whose layers are quantized: what stands between its products.

  gate      norms before and after a block: the branch's norm, its gate and residual scale, the sum kept
            for the residual stream, and that sum's norm with scale and shift for the next layer, as
            16-bit rows or as codes and a scale for each row
  route     routing to experts: from the router's scores to the rows sorted by expert and their weights
  combine   the experts' rows back to their tokens, weighted, gated and added to the residual
  lowrank   low-rank adapters of many requests added to the output of a projection that they share

`run` computes an operator in plain torch operations, or through the package where `own` is true.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token between two blocks: latency
        dict(name="gate_one_token", op="gate", m=1, k=1920, dt="bf16", norm="rms", post="rms", sets=1, even=True, mod32=False, affine=True, branch=True, out=16),
        # every token of a video clip between two blocks, modulation by frame
        dict(name="gate_clip", op="gate", m=17776, k=1920, dt="bf16", norm="layer", post="rms", sets=16, even=True, mod32=True, affine=False, branch=True, out=16),
        # a ragged batch of sequences ahead of a quantized layer
        dict(name="gate_batch_codes", op="gate", m=4113, k=4096, dt="f16", norm="layer", post="none", sets=5, even=False, mod32=False, affine=False, branch=True, out=8),
        # one token over a few experts: latency
        dict(name="route_one_token", op="route", m=1, e=16, top=2, dt="bf16", score="softmax", bias=False, groups=1, keep=1, best=1, renorm=True, masked=0.0),
        # a prompt, balanced by a bias, experts in groups
        dict(name="route_prompt_groups", op="route", m=4124, e=96, top=4, dt="f32", score="sigmoid", bias=True, groups=6, keep=3, best=2, renorm=True, masked=0.1),
        # every token of a clip over many experts
        dict(name="route_clip", op="route", m=17776, e=160, top=6, dt="f32", score="softmax", bias=False, groups=1, keep=1, best=1, renorm=False, masked=0.02),
        # eight new tokens, two experts each
        dict(name="combine_decode", op="combine", m=8, n=1920, top=2, dt="bf16", res=True, sets=8, even=True, mod32=False, dropped=0.0),
        # a padded prompt, four experts each, an odd width
        dict(name="combine_prompt", op="combine", m=4097, n=2047, top=4, dt="f16", res=True, sets=0, even=True, mod32=False, dropped=0.1),
        # every token of a clip, two experts each, a gate by frame
        dict(name="combine_clip", op="combine", m=17776, n=1920, top=2, dt="bf16", res=True, sets=16, even=True, mod32=True, dropped=0.0),
        # one new token of one request: latency
        dict(name="lowrank_one", op="lowrank", m=1, k=1920, n=5760, rank=64, adapters=4, requests=1, none=0.0, dt="bf16"),
        # one new token of each of 48 requests, wide layer
        dict(name="lowrank_decode", op="lowrank", m=48, k=4096, n=12288, rank=16, adapters=12, requests=48, none=0.1, dt="f16"),
        # prompts of seven requests, a clip's length in all
        dict(name="lowrank_prompts", op="lowrank", m=17776, k=1920, n=5760, rank=32, adapters=5, requests=7, none=0.15, dt="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sets(rng, m):
    """Sets of modulation rows over m rows: one, one for each row, an even split or any."""
    kind = rng.choice(["one", "rows", "even", "any"])
    if kind == "one":
        return 1, True
    if kind == "rows":
        return m, True
    most = min(m, 64)
    if kind == "even":
        return rng.choice([s for s in range(1, most + 1) if m % s == 0]), True
    return rng.randint(1, most), False


def draw(rng):
    op = rng.choice(["gate", "route", "combine", "lowrank"])
    dt = rng.choice(["bf16", "f16"])
    if op == "gate":
        out = rng.choice([16, 16, 8, 6, 4])
        k = _log(rng, 64, 12288)
        k = k if out == 16 else max(64, k // 64 * 64)
        m = _log(rng, 1, max(1, min(17776, 34000000 // k)))
        sets, even = _sets(rng, m)
        branch = rng.random() < 0.85
        return dict(op=op, m=m, k=k, dt=dt, norm=rng.choice(["rms", "layer"]), post=rng.choice(["none", "rms", "layer"]) if branch else "none",
                    sets=sets, even=even, mod32=rng.random() < 0.5, affine=rng.random() < 0.5, branch=branch, out=out)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        e = groups * _log(rng, 2, 256 // groups)
        keep = rng.randint(1, groups)
        return dict(op=op, m=_log(rng, 1, 17776), e=e, top=rng.randint(1, min(8, e // groups * keep)), dt=rng.choice(["bf16", "f16", "f32"]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, keep=keep,
                    best=rng.choice([1, 2]) if e // groups > 1 else 1, renorm=rng.random() < 0.6, masked=rng.choice([0.0, 0.05, 0.4]))
    if op == "combine":
        n, top = _log(rng, 64, 8192), rng.randint(1, 8)
        m = _log(rng, 1, max(1, min(17776, 68000000 // (n * top))))
        sets, even = _sets(rng, m) if rng.random() < 0.6 else (0, True)
        return dict(op=op, m=m, n=n, top=top, dt=dt, res=rng.random() < 0.7, sets=sets, even=even, mod32=rng.random() < 0.5, dropped=rng.choice([0.0, 0.2]))
    k, rank = max(256, _log(rng, 256, 12288) // 64 * 64), 8 * _log(rng, 1, 16)
    n = _log(rng, 64, 28672)
    adapters = _log(rng, 1, max(1, min(32, 300000000 // ((n + k) * rank))))
    m = _log(rng, 1, max(1, min(17776, 100000000 // n)))
    return dict(op=op, m=m, k=k, n=n, rank=rank, adapters=adapters, requests=_log(rng, 1, min(m, 64)), none=rng.choice([0.0, 0.3]), dt=dt)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = TYPES[c["dt"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    def index(m, sets):
        """Which set each row uses: sequences of uneven lengths, one after the other."""
        return torch.sort(torch.multinomial(0.2 + rand(sets), m, replacement=True, generator=g)).values.to(torch.int32)

    def modulation(sets, width, mod32):
        """Gate, scale and shift of each set, beside each other in the rows of one tensor."""
        t = torch.cat((0.6 + 0.3 * randn(sets, width), 0.2 * randn(sets, width), 0.3 * randn(sets, width)), 1)
        t = t if mod32 else t.to(dt)
        return t[:, :width], t[:, width:2 * width], t[:, 2 * width:]

    if c["op"] == "gate":
        m, k = c["m"], c["k"]
        h = 2.0 * randn(m, k) + 0.3
        h[:, :: max(1, k // 19)] *= 6.0  # a few loud channels, as residual streams have
        gate, scale, shift = modulation(c["sets"], k, c["mod32"])
        return dict(c=c, h=h.to(dt), y=(3.0 * randn(m, k)).to(dt) if c["branch"] else None, gate=gate if c["branch"] else None, scale=scale,
                    shift=shift, w=(1.0 + 0.2 * randn(k)).to(dt) if c["affine"] else None,
                    pw=1.0 + 0.2 * randn(k) if c["post"] != "none" else None, index=None if c["even"] else index(m, c["sets"]))
    if c["op"] == "route":
        m, e = c["m"], c["e"]
        x = 1.5 * randn(m, e) + 0.5 * randn(e)
        x[rand(m) < c["masked"] / 2] = -math.inf  # padding: rows that no expert sees
        x = torch.where(rand(m, e) < c["masked"], -math.inf, x)  # experts that a token may not use
        return dict(c=c, x=x.to(dt), bias=0.1 * randn(e) if c["bias"] else None)
    if c["op"] == "combine":
        m, n, top = c["m"], c["n"], c["top"]
        place = torch.randperm(m * top, generator=g, device=DEV).to(torch.int32).reshape(m, top)
        gone = rand(m, top) < c["dropped"]
        w = rand(m, top) + 0.1
        w = torch.where(gone, 0.0, w)
        y = torch.empty(m * top, n, dtype=dt, device=DEV)
        y.normal_(generator=g)
        y[place[gone].long()] = math.nan  # rows that no expert wrote
        gate = modulation(c["sets"], n, c["mod32"])[0] if c["sets"] else None
        return dict(c=c, y=y, place=torch.where(gone, -1, place), w=w, res=(2.0 * randn(m, n)).to(dt) if c["res"] else None, gate=gate,
                    index=None if c["even"] else index(m, c["sets"]))
    m, k, n, rank, adapters = c["m"], c["k"], c["n"], c["rank"], c["adapters"]
    request = index(m, c["requests"]).long() if c["requests"] < m else torch.arange(m, device=DEV)
    uses = torch.randint(0, adapters, (c["requests"],), generator=g, device=DEV)
    uses = torch.where(rand(c["requests"]) < c["none"], -1, uses)
    return dict(c=c, base=randn(m, n).to(dt), x=randn(m, k).to(dt), down=(randn(adapters, rank, k) / math.sqrt(k)).to(dt),
                up=(0.5 * randn(adapters, n, rank) / math.sqrt(rank)).to(dt), index=uses[request].to(torch.int32), s=0.5 + rand(adapters))


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _own(state)
    return {"gate": _plain_gate, "route": _plain_route, "combine": _plain_combine, "lowrank": _plain_lowrank}[state["c"]["op"]](state)


def _own(s):
    import bit_quantized_linear_vq_amd as vq

    c = s["c"]
    if c["op"] == "route":
        return vq.vq_route_experts(s["x"], c["top"], score=c["score"], bias=s["bias"], groups=c["groups"], top_groups=c["keep"],
                                   group_best=c["best"], renorm=c["renorm"])
    if c["op"] == "combine":
        return vq.vq_combine_experts(s["y"], s["place"], s["w"], residual=s["res"], gate=s["gate"], index=s["index"])
    if c["op"] == "lowrank":
        return vq.vq_lowrank_add(s["base"], s["x"], s["down"], s["up"], s["index"], scales=s["s"])
    how = dict(weight=s["w"], eps=EPS, norm=c["norm"], gate=s["gate"], branch_scale=0.7, post=c["post"], post_weight=s["pw"],
               mod_scale=s["scale"], mod_shift=s["shift"], index=s["index"])
    if c["out"] == 16:
        return vq.vq_gated_norm(s["y"], s["h"], **how)
    codes, scales, h = vq.vq_gated_norm_quant(s["y"], s["h"], c["out"], **how)
    # the codes leave as the values that they stand for
    return torch.mul(codes, scales[:, None], out=torch.empty_like(s["h"])), scales, h


def _of_rows(t, s, m):
    """The set of each row, [m x width] in float32 (one row where all share it)."""
    t = t.float()
    if s["index"] is not None:
        return t[s["index"].long()]
    return t if t.shape[0] in (1, m) else t.repeat_interleave(m // t.shape[0], 0)


def _norm(x, kind, w):
    """Norm of float32 rows; the moments in 64 bits, where a large mean would cost the variance its digits."""
    d = x.double()
    mean = d.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(d[:, :1])
    r = 1.0 / torch.sqrt((d - mean).square().mean(-1, keepdim=True) + EPS)
    v = (x - mean.float()) * r.float()
    return v if w is None else v * w.float()


def _plain_gate(s):
    c = s["c"]
    h, m = s["h"], c["m"]
    if c["branch"]:
        u = s["y"].float()
        u = u if c["post"] == "none" else _norm(u, c["post"], s["pw"])
        h = (h.float() + u * (_of_rows(s["gate"], s, m) * 0.7)).to(h.dtype)
    v = _norm(h.float(), c["norm"], s["w"])
    v = v * (1.0 + _of_rows(s["scale"], s, m)) + _of_rows(s["shift"], s, m)
    if c["out"] == 16:
        return v.to(h.dtype), h
    big = float(2 ** (c["out"] - 1) - 1)
    top = v.abs().amax(-1, keepdim=True)
    scale = top / big
    codes = (v * torch.where(top > 0, big / top, 0.0)).round().clamp(-big, big)
    return (codes * scale).to(h.dtype), scale[:, 0], h


def _plain_route(s):
    c = s["c"]
    m, e, top = c["m"], c["e"], c["top"]
    x = s["x"].double()  # two scores may differ by less than 32 bits hold
    open_ = x > -math.inf
    if c["score"] == "softmax":
        p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e300)) * open_
        p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
    else:
        p = torch.where(open_, 1.0 / (1.0 + torch.exp(-x)), 0.0)
    pick = x if s["bias"] is None else torch.where(open_, p + s["bias"].double(), -math.inf)
    if c["groups"] > 1:
        size = e // c["groups"]
        by = pick if c["best"] == 1 or s["bias"] is not None else torch.where(open_, p, -math.inf)
        by = torch.sort(by.reshape(m, -1, size), descending=True, stable=True).values
        # a group with fewer open experts than are counted has the sum of those
        mark = by[:, :, 0] if c["best"] == 1 else by[:, :, 0] + torch.where(by[:, :, 1] > -math.inf, by[:, :, 1], 0.0)
        order = torch.sort(mark, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros(m, c["groups"], dtype=torch.bool, device=x.device).scatter_(1, order, True)
        pick = torch.where(kept.repeat_interleave(size, 1), pick, -math.inf)
    best = torch.sort(pick, descending=True, stable=True)
    chosen = best.indices[:, :top]
    none = best.values[:, :top] == -math.inf
    w = torch.where(none, 0.0, torch.gather(p, 1, chosen))
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total.clamp(min=1e-300), 0.0)
    chosen = torch.where(none, e, chosen)
    order = torch.sort(chosen.flatten(), stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(m * top, device=x.device)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=x.device)
    offsets[1:] = (chosen.reshape(-1, 1) == torch.arange(e, device=x.device)).sum(0).cumsum(0)
    rows = torch.where(none.flatten()[order], -1, order // top)
    return (offsets, rows.to(torch.int32), w.float(), torch.where(none, -1, chosen).to(torch.int32),
            torch.where(none, -1, place.reshape(m, top)).to(torch.int32))


def _plain_combine(s):
    c = s["c"]
    there = s["place"] >= 0
    y = torch.where(there[:, :, None], s["y"][s["place"].clamp(min=0).long()].float(), 0.0)
    v = (y * s["w"][:, :, None]).sum(1)
    if s["gate"] is not None:
        v = v * _of_rows(s["gate"], s, c["m"])
    if s["res"] is not None:
        v = v + s["res"].float()
    return v.to(s["y"].dtype)


def _plain_lowrank(s):
    c = s["c"]
    # every row through all adapters, of which its own is kept: no loop, and the host need not see the index
    t = torch.matmul(s["x"].float(), s["down"].float().reshape(-1, c["k"]).t()).reshape(c["m"], -1, c["rank"])
    mine = s["index"][:, None] == torch.arange(c["adapters"], device=t.device)
    t = (t * (mine * s["s"])[:, :, None]).reshape(c["m"], -1)
    up = s["up"].float().permute(0, 2, 1).reshape(-1, c["n"])
    return (s["base"].float() + torch.matmul(t, up)).to(s["base"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "gate":
        m, k, s = c["m"], c["k"], c["sets"] * (4 if c["mod32"] else 2)
        byte = m * k * ((6 if c["branch"] else 2) + (2 if c["out"] == 16 else 1)) + s * k * (3 if c["branch"] else 2)
        byte += k * (2 * c["affine"] + 4 * (c["post"] != "none")) + 4 * m * ((not c["even"]) + (c["out"] != 16))
        return {"bytes": byte, "flops": m * k * (6.0 + (3.0 if c["branch"] else 0.0) + (0.0 if c["post"] == "none" else 4.0))}
    if c["op"] == "route":
        m, e, top = c["m"], c["e"], c["top"]
        return {"bytes": m * e * (4 if c["dt"] == "f32" else 2) + 16 * m * top + 4 * (e + 1) + 4 * e * c["bias"], "flops": 4.0 * m * e}
    if c["op"] == "combine":
        m, n, top = c["m"], c["n"], c["top"]
        kept = 1.0 - c["dropped"]
        return {"bytes": 2 * m * n * (top * kept + c["res"] + 1) + 8 * m * top + c["sets"] * n * (4 if c["mod32"] else 2) + 4 * m * (not c["even"]),
                "flops": 2.0 * m * n * (top * kept + 1)}
    m, k, n, rank = c["m"], c["k"], c["n"], c["rank"]
    asks = c["requests"] * (1.0 - c["none"])  # an adapter that no request uses is not read
    used = c["adapters"] * (1.0 - (1.0 - 1.0 / c["adapters"]) ** asks) if c["adapters"] > 1 else min(1.0, asks)
    return {"bytes": 2 * m * (k + 2 * n) + 2 * used * rank * (k + n) + 4 * m, "flops": 2.0 * m * rank * (k + n) * (1.0 - c["none"])}


# ------------------------------------------------------------------ the definitions in 64 bits

def _set_of(s, sets, m):
    """Which set of the modulation each row uses."""
    if s["index"] is not None:
        return s["index"].long()
    return torch.div(torch.arange(m, device=DEV) * sets, m, rounding_mode="floor")


def _normed(v, kind):
    if kind == "layer":
        v = v - v.sum(1, keepdim=True) / v.shape[1]
    return v / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    m = c["m"]
    if c["op"] == "gate":
        at = _set_of(s, c["sets"], m)
        h = s["h"]
        if c["branch"]:
            u = s["y"].double()
            if c["post"] != "none":
                u = _normed(u, c["post"]) * s["pw"].double()
            # the sum is kept in 16 bits, and the norm is that of the kept sum
            h = (h.double() + 0.7 * s["gate"].double()[at] * u).to(h.dtype)
        v = _normed(h.double(), c["norm"])
        v = v if s["w"] is None else v * s["w"].double()
        v = v + v * s["scale"].double()[at] + s["shift"].double()[at]
        if c["out"] == 16:
            return v, h.double()
        step = torch.max(torch.abs(v), 1).values / (2 ** (c["out"] - 1) - 1)
        return torch.round(torch.nan_to_num(v / step[:, None])) * step[:, None], step, h.double()
    if c["op"] == "combine":
        v = torch.zeros(m, c["n"], dtype=torch.float64, device=DEV)
        for j in range(c["top"]):
            at = s["place"][:, j].long()
            some = torch.nonzero(at >= 0)[:, 0]
            v[some] += s["y"].double()[at[some]] * s["w"][some, j].double()[:, None]
        if s["gate"] is not None:
            v *= s["gate"].double()[_set_of(s, c["sets"], m)]
        return v if s["res"] is None else v + s["res"].double()
    if c["op"] == "lowrank":
        v = s["base"].double()
        for a in range(c["adapters"]):
            at = torch.nonzero(s["index"] == a)[:, 0]
            if len(at):
                t = s["x"][at].double() @ s["down"][a].double().T
                v[at] += s["s"][a].double() * (t @ s["up"][a].double().T)
        return v
    # routing: the weights, from choices made one after the other (the choices themselves are whole numbers)
    e, top, size = c["e"], c["top"], c["e"] // c["groups"]
    x = s["x"].double()
    if c["score"] == "softmax":
        p = torch.nan_to_num(torch.softmax(x, 1))
    else:
        p = torch.sigmoid(x)
    shut = torch.isinf(x)
    order = x if s["bias"] is None else p + s["bias"].double()
    order = order.masked_fill(shut, -math.inf)
    if c["groups"] > 1:
        by = order if s["bias"] is not None or c["best"] == 1 else p.masked_fill(shut, -math.inf)
        left, marks = by.reshape(m, c["groups"], size).clone(), 0.0
        for i in range(c["best"]):
            top1 = left.max(2)
            marks = marks + (top1.values if i == 0 else torch.where(torch.isinf(top1.values), 0.0, top1.values))
            left.scatter_(2, top1.indices[:, :, None], -math.inf)
        far = torch.ones(m, c["groups"], dtype=torch.bool, device=DEV)
        lane = torch.arange(c["groups"], device=DEV)
        done = torch.full_like(marks, False, dtype=torch.bool)
        for _ in range(c["keep"]):
            now = marks.masked_fill(done, -math.inf)
            ok = (now == now.max(1, keepdim=True).values) & ~done
            first = torch.where(ok, lane, c["groups"]).min(1).values
            done[torch.arange(m, device=DEV), first] = True
        far &= ~done
        order = order.masked_fill(far.repeat_interleave(size, 1), -math.inf)
    w = torch.zeros(m, top, dtype=torch.float64, device=DEV)
    lane = torch.arange(e, device=DEV)
    for j in range(top):
        high = order.max(1, keepdim=True).values
        first = torch.where(order == high, lane, e).min(1).values
        got = torch.gather(p, 1, first[:, None])[:, 0]
        w[:, j] = torch.where(torch.isinf(high[:, 0]), 0.0, got)
        order[torch.arange(m, device=DEV), first] = -math.inf
    if c["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    return None, None, w, None, None
