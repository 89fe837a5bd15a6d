"""Cases for the operators around the quantized linear layer: the norm ahead of it, its form for
single tokens, and its form for experts.

  norm     root-mean-square norm of x (+ residual): codes and a scale for each row, or 16-bit rows
  gemv     a few 16-bit rows times 4-bit weights with a scale for each group of inputs
  experts  int8 activation codes times packed 8-bit or 4-bit weights of several experts, dequantized
  dense    16-bit activations times 16-bit weights of several experts

`run` computes an operator in plain torch operations, or through the package where `own` is true.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token between two layers: latency
        dict(name="norm_one_token", op="norm", m=1, k=1920, dt="bf16", res=True, out=8, w32=False),
        # every token of a video clip ahead of its fused-QKV layer
        dict(name="norm_clip_codes", op="norm", m=17776, k=1920, dt="bf16", res=True, out=8, w32=False),
        # a ragged batch ahead of a layer kept at 16 bits, norm weights in float32
        dict(name="norm_batch_16bit", op="norm", m=4113, k=4096, dt="f16", res=True, out=16, w32=True),
        # one token through a small projection: latency
        dict(name="gemv_one_small", op="gemv", m=1, n=1920, k=1920, group=128, dt="bf16"),
        # one token through a feed-forward layer
        dict(name="gemv_one_ffn", op="gemv", m=1, n=12288, k=4096, group=64, dt="bf16"),
        # seven sequences, a large layer with short groups and an odd number of outputs
        dict(name="gemv_seven_large", op="gemv", m=7, n=28671, k=8192, group=32, dt="f16"),
        # eight new tokens, two experts each, 4-bit weights
        dict(name="experts_decode_w4", op="experts", t=16, e=16, n=5760, k=1920, bits=4, kblock=True, top=2, skew=0.0, dt="bf16"),
        # a short prompt over many experts, rows gathered by token
        dict(name="experts_prompt_w8", op="experts", t=4124, e=32, n=2048, k=2048, bits=8, kblock=False, top=4, skew=0.7, dt="bf16"),
        # every token of a clip, few experts, uneven shares
        dict(name="experts_clip_w8", op="experts", t=17776, e=8, n=5760, k=1920, bits=8, kblock=True, top=1, skew=0.5, dt="bf16"),
        # the same way with 4-bit weights and a long input
        dict(name="experts_long_w4", op="experts", t=6001, e=4, n=1920, k=12288, bits=4, kblock=False, top=1, skew=0.3, dt="f16"),
        # twelve new tokens, two experts each, layers kept at 16 bits
        dict(name="dense_decode", op="dense", t=24, e=8, n=1920, k=4096, top=2, skew=0.0, dt="bf16"),
        # a prompt through layers kept at 16 bits, an odd number of outputs
        dict(name="dense_prompt", op="dense", t=8190, e=8, n=5759, k=2048, top=2, skew=0.4, dt="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gemv", "experts", "dense"])
    dt = rng.choice(["bf16", "f16"])
    if op == "norm":
        out = rng.choice([16, 8, 8, 6, 4])
        k = _log(rng, 64, 12288)
        k = k if out == 16 else max(64, k // 64 * 64)
        m = _log(rng, 1, max(1, min(17776, 34000000 // k)))
        return dict(op=op, m=m, k=k, dt=dt, res=rng.random() < 0.7, out=out, w32=rng.random() < 0.3)
    if op == "gemv":
        group = rng.choice([32, 64, 128])
        k = max(group, _log(rng, 256, 16384) // group * group)
        n = _log(rng, 64, max(64, min(32768, 230000000 // k)))
        return dict(op=op, m=_log(rng, 1, 32), n=n, k=k, group=group, dt=dt)
    e = _log(rng, 1, 64)
    k = max(64, _log(rng, 256, 12288) // 64 * 64)
    n = _log(rng, 64, max(64, min(8192, 230000000 // (e * k))))
    top = rng.choice([1, 2, 4])
    t = top * _log(rng, 1, max(1, min(17776, 120000000000 // (n * k)) // top))
    c = dict(op=op, t=t, e=e, n=n, k=k, top=top, skew=round(rng.uniform(0.0, 1.0), 2), dt=dt)
    if op == "experts":
        c.update(bits=rng.choice([8, 4]), kblock=rng.random() < 0.5)
    return c


# ------------------------------------------------------------------ inputs

def _pack_nibbles(c):
    """4-bit codes [rows, k] two to a byte, the even input in the low half."""
    u = (c & 15).to(torch.uint8)
    return u[:, 0::2] | (u[:, 1::2] << 4)


def _pieces(b):
    """Weight codes [rows, bytes] in 64-byte pieces [pieces, rows, 64], the last one padded."""
    rows, row = b.shape
    p = (row + 63) // 64
    full = torch.zeros((rows, p * 64), dtype=b.dtype, device=b.device)
    full[:, :row] = b
    return full.reshape(rows, p, 64).permute(1, 0, 2).contiguous()


def _route(c, g):
    """Rows sorted by expert: offsets [e + 1], and each row's token (None where rows are tokens)."""
    t, e, top = c["t"], c["e"], c["top"]
    share = torch.exp(2.0 * c["skew"] * torch.randn(e, generator=g, device=DEV, dtype=torch.float64))
    pick = torch.multinomial(share, t, replacement=True, generator=g)
    order = torch.argsort(pick, stable=True)
    off = torch.zeros(e + 1, dtype=torch.int32, device=DEV)
    off[1:] = torch.cumsum(torch.bincount(pick, minlength=e), 0).to(torch.int32)
    return off, (order // top).to(torch.int32) if top > 1 else None


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = TYPES[c["dt"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    if c["op"] == "norm":
        m, k = c["m"], c["k"]
        x = randn(m, k)
        x[:, :: max(1, k // 19)] *= 8.0  # a few loud channels, as activations have
        res = (2.0 * randn(m, k)).to(dt) if c["res"] else None
        w = 1.0 + 0.2 * randn(k)
        return dict(c=c, x=x.to(dt), res=res, w=w if c["w32"] else w.to(dt))
    if c["op"] == "gemv":
        m, n, k, group = c["m"], c["n"], c["k"], c["group"]
        codes = (2.5 * randn(n, k)).round_().clamp_(-7, 7).to(torch.int8)
        scales = (0.004 + 0.004 * torch.rand(n, k // group, generator=g, device=DEV)).to(dt)
        return dict(c=c, x=randn(m, k).to(dt), codes=_pack_nibbles(codes), scales=scales)
    t, e, n, k = c["t"], c["e"], c["n"], c["k"]
    off, rows = _route(c, g)
    tokens = t // c["top"]
    if c["op"] == "dense":
        w = torch.empty(e, n, k, dtype=dt, device=DEV)
        for i in range(e):
            w[i] = 0.02 * randn(n, k)
        return dict(c=c, x=randn(tokens, k).to(dt), w=w, off=off, rows=rows)
    a = (36.0 * randn(tokens, k)).round_().clamp_(-127, 127).to(torch.int8)
    sa = 0.02 + 0.01 * torch.rand(tokens, generator=g, device=DEV)
    big, sd = (127, 32.0) if c["bits"] == 8 else (7, 2.0)
    b = torch.empty(e * n, k, dtype=torch.int8, device=DEV)
    for i in range(e):
        b[i * n:(i + 1) * n] = (sd * randn(n, k)).round_().clamp_(-big, big)
    sb = (0.08 + 0.02 * torch.rand(e * n, generator=g, device=DEV)) / big
    b = b if c["bits"] == 8 else _pack_nibbles(b)
    return dict(c=c, a=a, sa=sa, b=_pieces(b) if c["kblock"] else b, sb=sb, off=off, rows=rows)


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "gemv": _plain_gemv, "experts": _plain_experts, "dense": _plain_dense}[state["c"]["op"]](state)


def _own(s):
    import bit_quantized_linear_vq_amd as vq

    c = s["c"]
    dt = TYPES[c["dt"]]
    if c["op"] == "gemv":
        return vq.vq_w4_gemv(s["x"], s["codes"], s["scales"])
    if c["op"] == "experts":
        return vq.vq_qgemm_experts(s["a"], s["sa"], s["b"], s["sb"], c["bits"], s["off"], rows=s["rows"], out_dtype=dt)
    if c["op"] == "dense":
        return vq.vq_gemm_dense_experts(s["x"], s["w"], s["off"], rows=s["rows"])
    if c["out"] == 16:
        return vq.vq_rmsnorm(s["x"], s["w"], EPS, residual=s["res"])
    got = vq.vq_rmsnorm_quant(s["x"], s["w"], c["out"], EPS, residual=s["res"])
    # the codes leave as the values that they stand for
    values = torch.mul(got[0], got[1][:, None], out=torch.empty_like(s["x"]))
    return (values,) + tuple(got[1:])


def _plain_norm(s):
    c = s["c"]
    x, w = s["x"], s["w"]
    h = x if s["res"] is None else (x.float() + s["res"].float()).to(x.dtype)
    h32 = h.float()
    q = h32.double().square().mean(-1, keepdim=True)
    v = h32 * (1.0 / torch.sqrt(q + EPS)).float() * w.float()
    if c["out"] == 16:
        y = v.to(x.dtype)
        return y if s["res"] is None else (y, h)
    big = float(2 ** (c["out"] - 1) - 1)
    top = v.abs().amax(-1, keepdim=True)
    scale = top / big
    codes = (v * torch.where(top > 0, big / top, 0.0)).round().clamp(-big, big)
    values = (codes * scale).to(x.dtype)
    return (values, scale[:, 0]) if s["res"] is None else (values, scale[:, 0], h)


def _nibbles(b):
    """The signed values of 4-bit codes [rows, k / 2] in float32 [rows, k]."""
    lo, hi = b & 15, b >> 4
    u = torch.stack((lo, hi), -1).reshape(b.shape[0], -1)
    return (u ^ 8).float() - 8.0


def _plain_gemv(s):
    c = s["c"]
    w = _nibbles(s["codes"]).reshape(c["n"], -1, c["group"]) * s["scales"].float()[:, :, None]
    return torch.matmul(s["x"].float(), w.reshape(c["n"], c["k"]).t()).to(s["x"].dtype)


def _plain_experts(s):
    c = s["c"]
    n, row = c["n"], c["k"] if c["bits"] == 8 else c["k"] // 2
    y = torch.empty((c["t"], n), dtype=TYPES[c["dt"]], device=s["a"].device)
    off = s["off"].tolist()
    # ragged products have no form without a loop over the experts that does not multiply the work
    for i in range(c["e"]):
        lo, hi = off[i], off[i + 1]
        if lo == hi:
            continue
        pick = slice(lo, hi) if s["rows"] is None else s["rows"][lo:hi]
        b = s["b"][:, i * n:(i + 1) * n].permute(1, 0, 2).reshape(n, -1)[:, :row] if c["kblock"] else s["b"][i * n:(i + 1) * n]
        b = b.float() if c["bits"] == 8 else _nibbles(b)
        acc = torch.matmul(s["a"][pick].float(), b.t())
        y[lo:hi] = acc * (s["sa"][pick][:, None] * s["sb"][i * n:(i + 1) * n])
    return y


def _plain_dense(s):
    c = s["c"]
    y = torch.empty((c["t"], c["n"]), dtype=s["x"].dtype, device=s["x"].device)
    off = s["off"].tolist()
    for i in range(c["e"]):
        lo, hi = off[i], off[i + 1]
        if lo == hi:
            continue
        pick = slice(lo, hi) if s["rows"] is None else s["rows"][lo:hi]
        y[lo:hi] = torch.matmul(s["x"][pick].float(), s["w"][i].float().t())
    return y


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "norm":
        m, k = c["m"], c["k"]
        byte = m * k * ((4 if c["res"] else 2) + (2 if c["res"] else 0) + (2 if c["out"] == 16 else 1))
        return {"bytes": byte + k * (4 if c["w32"] else 2) + (0 if c["out"] == 16 else 4 * m), "flops": 4.0 * m * k}
    if c["op"] == "gemv":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": n * k / 2 + 2 * n * (k // c["group"]) + 2 * m * (k + n), "flops": 2.0 * m * n * k}
    t, e, n, k = c["t"], c["e"], c["n"], c["k"]
    used = e * (1.0 - (1.0 - 1.0 / e) ** t) if e > 1 else 1.0  # experts that have rows, for even shares
    el = 2 if c["op"] == "dense" else c["bits"] / 8
    return {"bytes": used * n * k * el + t // c["top"] * k * (2 if c["op"] == "dense" else 1) + 2 * t * n, "flops": 2.0 * t * n * k}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "norm":
        x = s["x"].double()
        out = []
        if s["res"] is not None:
            x = (x + s["res"].double()).to(s["x"].dtype)  # the sum is kept in 16 bits, and the norm is that of the kept sum
            out = [x.double()]
            x = x.double()
        rms = torch.sqrt((x * x).sum(1) / c["k"] + EPS)
        v = x / rms[:, None] * s["w"].double()[None, :]
        if c["out"] == 16:
            return [v] + out if out else v
        levels = 2 ** (c["out"] - 1) - 1
        step = torch.max(torch.abs(v), 1).values / levels
        ratio = torch.nan_to_num(v / step[:, None])
        return [torch.round(ratio) * step[:, None], step] + out
    if c["op"] == "gemv":
        n, k, group = c["n"], c["k"], c["group"]
        by = s["codes"].to(torch.int16)
        w = torch.empty(n, k, dtype=torch.float64, device=by.device)
        w[:, 0::2] = ((by & 15) + 8) % 16 - 8
        w[:, 1::2] = ((by >> 4) + 8) % 16 - 8
        w *= torch.repeat_interleave(s["scales"].double(), group, dim=1)
        return s["x"].double() @ w.T
    t, e, n, k = c["t"], c["e"], c["n"], c["k"]
    off = s["off"].cpu().numpy()
    token = torch.arange(t, device=DEV) if s["rows"] is None else s["rows"].long()
    y = torch.zeros(t, n, dtype=torch.float64, device=DEV)
    for i in range(e):
        at = token[int(off[i]):int(off[i + 1])]
        if c["op"] == "dense":
            y[int(off[i]):int(off[i + 1])] = s["x"].double()[at] @ s["w"][i].double().T
            continue
        b = s["b"]
        if c["kblock"]:  # byte j of row r lies in piece j // 64
            j = torch.arange(k if c["bits"] == 8 else k // 2, device=DEV)
            b = b[j // 64, :, j % 64].T
        b = b[i * n:(i + 1) * n].to(torch.int16)
        if c["bits"] == 4:
            w = torch.empty(n, k, dtype=torch.float64, device=DEV)
            w[:, 0::2] = ((b & 15) + 8) % 16 - 8
            w[:, 1::2] = ((b >> 4) + 8) % 16 - 8
        else:
            w = b.double()
        part = s["a"].double()[at] @ w.T
        y[int(off[i]):int(off[i + 1])] = part * s["sa"].double()[at][:, None] * s["sb"].double()[i * n:(i + 1) * n][None, :]
    return y
