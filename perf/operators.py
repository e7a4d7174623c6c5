"""Cases of the dense FP8 operators around the routed-expert layer.

Three operators that a transformer block runs next to the expert layer:

- ``norm``: residual addition, root-mean-square norm and 1x128 E4M3
  quantisation of the result in one pass
- ``linear``: y = A W^T with E4M3 codes on both sides, one scale per token and
  128 channels of A and one per 128 x 128 block of W
- ``gated``: h = SiLU(A Wg^T) * (A Wu^T), quantised to 1x128 E4M3 as it is written

Scales are fp32 ("f32") or powers of two held in eight bits ("e8m0").

``run`` computes a case in its plain form (elementary torch operations in
32 bits) or, where ``own`` is true, through the package's public calls.
``exact`` states the same definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
G = 128                      # channels (and weight rows) that share a scale
E4M3_MAX = 448.0
TINY = 2.0 ** -126           # a scale below the normal range is replaced by 1


# ------------------------------------------------------------------ cases

def listed():
    return [
        # decode: one token's hidden state before a block; nothing but latency counts
        dict(name="norm_t1", op="norm", t=1, h=7168, x="bf16", res="bf16", y=False, scale="f32"),
        # a ragged batch of a narrow model: fp32 residual stream, 8.125 scale groups, bf16 copy for the router too
        dict(name="norm_t333_ragged", op="norm", t=333, h=1040, x="bf16", res="f32", y=True, scale="e8m0"),
        # prefill of a long prompt
        dict(name="norm_t8192", op="norm", t=8192, h=7168, x="bf16", res="bf16", y=False, scale="f32"),
        # decode, down projection of a dense block: one token streams the weights
        dict(name="linear_m1", op="linear", m=1, k=2048, n=7168, out="bf16", scale="f32"),
        # a decode batch, wide projection with fp32 results
        dict(name="linear_m16_f32out", op="linear", m=16, k=7168, n=4096, out="f32", scale="e8m0"),
        # a chunk of a prompt through a projection whose sizes end inside tiles and scale blocks
        dict(name="linear_m777_ragged", op="linear", m=777, k=1992, n=1001, out="bf16", scale="f32"),
        # prefill, down projection
        dict(name="linear_m8192", op="linear", m=8192, k=2048, n=7168, out="bf16", scale="f32"),
        # prefill, square projection of a checkpoint with power-of-two scales
        dict(name="linear_m4096_e8m0", op="linear", m=4096, k=7168, n=7168, out="bf16", scale="e8m0"),
        # decode, gate and up projections of a dense block (or of a shared expert)
        dict(name="gated_m1", op="gated", m=1, k=7168, n=2048, scale="f32"),
        # a speculative or batched decode step with ragged sizes
        dict(name="gated_m50_ragged", op="gated", m=50, k=1040, n=1000, scale="e8m0"),
        # prefill, gate and up projections with either kind of scale
        dict(name="gated_m8192", op="gated", m=8192, k=7168, n=2048, scale="f32"),
        dict(name="gated_m8192_e8m0", op="gated", m=8192, k=7168, n=2048, scale="e8m0"),
    ]


MAX_MACS = 4096 * 7168 * 7168


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "linear", "gated"))
    scale = rng.choice(("f32", "e8m0"))
    if op == "norm":
        x = rng.choice(("bf16", "bf16", "f32"))
        res = rng.choice(("none", "f32", "f32" if x == "f32" else "bf16"))
        return dict(op=op, t=_log(rng, 1, 8192), h=_log(rng, 100, 7168), x=x, res=res, y=rng.random() < 0.4, scale=scale)
    m, k, n = _log(rng, 1, 8192), _log(rng, 100, 7168), _log(rng, 64, 7168 if op == "linear" else 2400)
    m = max(1, min(m, MAX_MACS // (k * n * (2 if op == "gated" else 1))))
    if op == "gated":
        return dict(op=op, m=m, k=k, n=n, scale=scale)
    return dict(op=op, m=m, k=k, n=n, out=rng.choice(("bf16", "bf16", "f32")), scale=scale)


def work(case):
    sb = 4 if case["scale"] == "f32" else 1
    if case["op"] == "norm":
        t, h = case["t"], case["h"]
        size = {"bf16": 2, "f32": 4, "none": 0}
        xb, rb = size[case["x"]], size[case["res"]]
        b = t * h * (xb + 2 * rb + 1 + (xb if case["y"] else 0)) + 4 * h + t * _groups(h) * sb
        return {"bytes": b, "flops": 8 * t * h}
    m, k, n = case["m"], case["k"], case["n"]
    w = 2 if case["op"] == "gated" else 1
    b = m * k + m * _groups(k) * sb + w * (n * k + _groups(n) * _groups(k) * sb)
    if case["op"] == "gated":
        b += m * n + m * _groups(n) * sb
    else:
        b += m * n * (4 if case["out"] == "f32" else 2)
    return {"bytes": b, "flops": 2 * m * n * k * w}


# ------------------------------------------------------------------ inputs

def _groups(n):
    return (n + G - 1) // G


def _pad(v, dim, to):
    """v with zeros appended along dim up to a multiple of `to`."""
    short = -v.shape[dim] % to
    if not short:
        return v
    shape = list(v.shape)
    shape[dim] = short
    return torch.cat([v, v.new_zeros(shape)], dim)


def _scale_of(amax, scale):
    """The scale of a group with this largest magnitude: amax / 448, or the
    smallest power of two that is at least that; 1 where there is no normal
    number to divide by."""
    s = amax / E4M3_MAX
    if scale == "e8m0":
        mant, ex = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(mant == 0.5, ex - 1, ex))
    return torch.where(amax / E4M3_MAX < TINY, torch.ones_like(s), s)


def _hold(s, scale):
    """Scales in the type that holds them."""
    if scale == "f32":
        return s.float()
    return (torch.frexp(s)[1] + 126).to(torch.uint8).view(torch.float8_e8m0fnu)


def _quant_rows(v, scale):
    """1x128 quantisation of [rows][cols]: codes [rows][cols], scales [groups][rows] (in v's type)."""
    rows, cols = v.shape
    g = _pad(v, 1, G).view(rows, -1, G)
    s = _scale_of(g.abs().amax(-1), scale)
    q = (g / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.reshape(rows, -1)[:, :cols], s.t()


def _make_weight(n, k, scale, gen):
    """[n][k] weights of a trained layer's spread, in E4M3 with a scale per 128 x 128 block."""
    w = torch.randn(n, k, generator=gen, device="cuda") * 0.02
    b = _pad(_pad(w, 0, G), 1, G).view(_groups(n), G, _groups(k), G)
    s = _scale_of(b.abs().amax((1, 3)), scale)
    q = (b / s[:, None, :, None]).reshape(_groups(n) * G, -1)[:n, :k]
    return q.contiguous().to(torch.float8_e4m3fn), _hold(s, scale)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    st = {"case": dict(case)}
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    if own:
        import moe_expert_ffn_02_gb300 as moe
    if case["op"] == "norm":
        t, h = case["t"], case["h"]
        st["x"] = torch.randn(t, h, generator=gen, device="cuda").to(dt[case["x"]])
        # the residual stream has grown over the layers before this one
        st["res"] = None if case["res"] == "none" else (torch.randn(t, h, generator=gen, device="cuda") * 4).to(dt[case["res"]])
        st["w"] = 1 + 0.2 * torch.randn(h, generator=gen, device="cuda")
        if own:         # the module and the buffers that a serving loop keeps
            st["norm"] = moe.RmsNorm(st["w"], EPS)
            st["out"] = moe.Fp8Tensor(t, h, case["scale"])
            st["res_out"] = None if st["res"] is None else torch.empty_like(st["res"])
            st["y"] = torch.empty_like(st["x"]) if case["y"] else None
        return st
    m, k, n = case["m"], case["k"], case["n"]
    q, s = _quant_rows(torch.randn(m, k, generator=gen, device="cuda"), case["scale"])
    st["aq"], st["as"] = q.to(torch.float8_e4m3fn), _hold(s, case["scale"]).contiguous()
    st["wq"], st["ws"] = _make_weight(n, k, case["scale"], gen)
    if case["op"] == "gated":
        st["uq"], st["us"] = _make_weight(n, k, case["scale"], gen)
    if own:             # the weights' handle, the activations as the norm leaves them, the output's buffer
        st["a"] = moe.Fp8Tensor.from_parts(st["aq"], st["as"])
        if case["op"] == "gated":
            st["lin"] = moe.Fp8GatedLinear(st["wq"], st["ws"], st["uq"], st["us"])
            st["out"] = moe.Fp8Tensor(m, n, case["scale"])
        else:
            st["lin"] = moe.Fp8Linear(st["wq"], st["ws"])
            st["out"] = torch.empty(m, n, dtype=dt[case["out"]], device="cuda")
    return st


# ------------------------------------------------------------------ a pass

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    case = st["case"]
    if case["op"] == "norm":
        st["norm"](st["x"], st["res"], out=st["out"], res_out=st["res_out"], y=st["y"])
        got = {"q": st["out"].q, "s": st["out"].s}
        if st["res"] is not None:
            got["res"] = st["res_out"]
        if case["y"]:
            got["y"] = st["y"]
        return got
    st["lin"](st["a"], st["out"])
    if case["op"] == "gated":
        return {"q": st["out"].q, "s": st["out"].s}
    return {"y": st["out"]}


def _dequant_rows(q, s):
    return q.float() * s.float().t().repeat_interleave(G, 1)[:, :q.shape[1]]


def _dequant_blocks(q, s):
    wide = s.float().repeat_interleave(G, 0)[:q.shape[0]].repeat_interleave(G, 1)[:, :q.shape[1]]
    return q.float() * wide


def _run_plain(st):
    case = st["case"]
    scale = case["scale"]
    if case["op"] == "norm":
        v, got = st["x"].float(), {}
        if st["res"] is not None:
            v = v + st["res"].float()
            got["res"] = v.to(st["res"].dtype)
        n = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * st["w"]
        if case["y"]:
            got["y"] = n.to(st["x"].dtype)
        q, s = _quant_rows(n, scale)
        return {**got, "q": q.to(torch.float8_e4m3fn), "s": _hold(s, scale)}
    a = _dequant_rows(st["aq"], st["as"])
    y = a @ _dequant_blocks(st["wq"], st["ws"]).t()
    if case["op"] == "linear":
        return {"y": y if case["out"] == "f32" else y.to(torch.bfloat16)}
    h = y * torch.sigmoid(y) * (a @ _dequant_blocks(st["uq"], st["us"]).t())
    q, s = _quant_rows(h, scale)
    return {"q": q.to(torch.float8_e4m3fn), "s": _hold(s, scale)}


# ------------------------------------------------------------------ 64 bits

def _exact_codes(v, scale):
    """Scales, and the quotients that the codes stand for before they are rounded to eight bits."""
    rows, cols = v.shape
    groups = _groups(cols)
    q, s = torch.empty_like(v), torch.empty(groups, rows, dtype=v.dtype, device=v.device)
    for g in range(groups):
        part = v[:, g * G:(g + 1) * G]
        top = part.abs().max(dim=1).values / E4M3_MAX
        if scale == "e8m0":
            step = torch.pow(2.0, torch.ceil(torch.log2(top)))
        else:
            step = top
        step = torch.where(top < TINY, torch.ones_like(top), step)
        s[g] = step
        q[:, g * G:(g + 1) * G] = part / step[:, None]
    return {"q": q, "s": s}


def _scaled_product(aq, a_s, wq, w_s):
    """sum over the 128-channel blocks of sa * sw * (codes' products)."""
    m, k, n = aq.shape[0], aq.shape[1], wq.shape[0]
    row_block = torch.arange(n, device=aq.device) // G
    total = torch.zeros(m, n, dtype=torch.float64, device=aq.device)
    for b in range(_groups(k)):
        cut = slice(b * G, min(k, (b + 1) * G))
        part = aq[:, cut].double() @ wq[:, cut].double().T
        total += part * a_s[b].double()[:, None] * w_s[:, b].double()[row_block][None, :]
    return total


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        v, got = st["x"].double(), {}
        if st["res"] is not None:
            v = v + st["res"].double()
            got["res"] = v
        ms = (v * v).sum(dim=1, keepdim=True) / case["h"]
        n = v / torch.sqrt(ms + EPS) * st["w"].double()
        if case["y"]:
            got["y"] = n
        return {**got, **_exact_codes(n, case["scale"])}
    y = _scaled_product(st["aq"], st["as"], st["wq"], st["ws"])
    if case["op"] == "linear":
        return {"y": y}
    h = y / (1 + torch.exp(-y)) * _scaled_product(st["aq"], st["as"], st["uq"], st["us"])
    return _exact_codes(h, case["scale"])
