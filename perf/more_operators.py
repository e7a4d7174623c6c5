"""Cases of the operators that run routed experts outside the fused layer.

Tokens sorted by expert and back, with the weights applied, and the gradients:

- ``dispatch``: expert ids [T][k] -> the stable order by expert (offsets, token of each row, row of each pair) and the
  rows of x in that order; pairs whose expert is held elsewhere get no row
- ``dispatch_grad``: dx[t] = sum over t's rows of the rows' gradients
- ``combine``: y[t] = add[t] + sum over t's rows of w[t][j] * o[row]
- ``combine_grad``: d_o[row] = w[t][j] * dy[t], d_w[t][j] = <o[row], dy[t]>

Products with weights of 4 bits and a scale (and a zero point) per group of input channels:

- ``int4``: y = x W^T, or with gate and up matrices h = SiLU(x Wg^T) * (x Wu^T)
- ``experts4``: the same where each row, or the token that it is of, meets the matrix of its expert

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, where ``own`` is true, through the
package's public calls.  ``exact`` states the same definitions in 64 bits.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases

def listed():
    return [
        # decode: one token's hidden state goes to its experts; nothing but latency counts
        dict(name="dispatch_t1", op="dispatch", t=1, k=8, e=256, first=0, here=256, h=7168, x="bf16"),
        # prefill of a long prompt
        dict(name="dispatch_t8192", op="dispatch", t=8192, k=8, e=256, first=0, here=256, h=7168, x="bf16"),
        # a training step of a narrow model whose rows lie off every vector grid
        dict(name="dispatch_grad_t1500_ragged", op="dispatch_grad", t=1500, k=4, e=60, first=0, here=60, h=1001, x="bf16", y="f32"),
        # a decode batch, back onto the shared expert's output
        dict(name="combine_t16", op="combine", t=16, k=8, e=256, first=0, here=256, h=7168, x="bf16", y="bf16", add=True),
        # prefill
        dict(name="combine_t8192", op="combine", t=8192, k=8, e=256, first=0, here=256, h=7168, x="bf16", y="bf16", add=False),
        # one of four expert-parallel ranks in a training step, fp32
        dict(name="combine_grad_t333_part", op="combine_grad", t=333, k=6, e=64, first=16, here=16, h=1040, x="f32", y="f32"),
        # a training step on long sequences
        dict(name="combine_grad_t8192", op="combine_grad", t=8192, k=8, e=256, first=0, here=256, h=7168, x="bf16", y="bf16"),
        # decode: one token streams a down projection's weights
        dict(name="int4_m1", op="int4", m=1, kin=2048, n=7168, gated=False, group=128, zero=False, s="bf16", y="bf16"),
        # a decode batch through the gate and up projections of a dense block, fine groups with zero points
        dict(name="int4_gated_m16", op="int4", m=16, kin=7168, n=2048, gated=True, group=32, zero=True, s="bf16", y="bf16"),
        # a chunk of a prompt through a projection whose sizes end inside tiles and groups
        dict(name="int4_m777_ragged", op="int4", m=777, kin=1991, n=1001, gated=False, group=64, zero=True, s="f32", y="f32"),
        # a decode batch through the experts' gate and up projections, read from the tokens' own rows
        dict(name="experts4_t16", op="experts4", t=16, k=8, e=256, kin=7168, n=2048, gated=True, group=32, zero=False, s="bf16", y="bf16", gather=True),
        # prefill through the experts' down projections
        dict(name="experts4_t2048", op="experts4", t=2048, k=8, e=256, kin=2048, n=7168, gated=False, group=128, zero=False, s="bf16", y="bf16", gather=False),
    ]


MAX_ROWS = 8192 * 8 * 7168                  # of the routing operators: pairs times width
MAX_MACS = 2048 * 8 * 2048 * 7168           # of the products
MAX_WEIGHTS = 256 * 2048 * 7168


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("dispatch", "dispatch_grad", "combine", "combine_grad", "int4", "int4", "experts4"))
    if op == "int4":
        gated = rng.random() < 0.4
        w = 2 if gated else 1
        m, kin, n = _log(rng, 1, 8192), _log(rng, 64, 7168), _log(rng, 64, 7168 // w)
        m = max(1, min(m, MAX_MACS // (kin * n * w)))
        return dict(op=op, m=m, kin=kin, n=n, gated=gated, group=rng.choice((32, 64, 128)), zero=rng.random() < 0.5,
                    s=rng.choice(("bf16", "f32")), y=rng.choice(("bf16", "bf16", "f32")))
    e = _log(rng, 8, 256)
    k = rng.randint(1, 8)
    if op == "experts4":
        gated = rng.random() < 0.5
        w = 2 if gated else 1
        t, kin, n = _log(rng, 1, 2048), _log(rng, 64, 7168), _log(rng, 64, 2048)
        e = max(k, min(e, MAX_WEIGHTS // (kin * n * w)))
        t = max(1, min(t, MAX_MACS // (k * kin * n * w)))
        return dict(op=op, t=t, k=k, e=e, kin=kin, n=n, gated=gated, group=rng.choice((32, 64, 128)), zero=rng.random() < 0.5,
                    s=rng.choice(("bf16", "f32")), y=rng.choice(("bf16", "bf16", "f32")), gather=rng.random() < 0.5)
    t, h = _log(rng, 1, 8192), _log(rng, 64, 7168)
    here = e if rng.random() < 0.7 else max(1, e // rng.choice((2, 4)))
    case = dict(op=op, t=t, k=k, e=e, first=rng.randint(0, e - here), here=here, h=h, x=rng.choice(("bf16", "bf16", "f32")))
    if case["x"] == "f32":
        case["t"] = max(1, min(t, MAX_ROWS // (2 * k * h)))
    if op != "dispatch":
        case["y"] = rng.choice((case["x"], "f32"))
    if op == "combine":
        case["add"] = rng.random() < 0.5
    return case


SIZE = {"bf16": 2, "f32": 4}


def work(case):
    if case["op"] in ("int4", "experts4"):
        w = 2 if case["gated"] else 1
        kin, n = case["kin"], case["n"]
        groups = -(-kin // case["group"])
        matrix = w * n * (-(-kin // 2) + groups * (SIZE[case["s"]] + (1 if case["zero"] else 0)))
        if case["op"] == "int4":
            rows, read, touched = case["m"], case["m"], 1
        else:
            rows = case["t"] * case["k"]
            read = case["t"] if case["gather"] else rows
            # the router is balanced: each expert is one of a token's k with probability k / e
            touched = case["e"] * (1 - (1 - case["k"] / case["e"]) ** case["t"])
        return {"bytes": touched * matrix + read * kin * 2 + rows * n * SIZE[case["y"]], "flops": 2 * rows * n * kin * w}
    t, k, h = case["t"], case["k"], case["h"]
    pairs = t * k * case["here"] / case["e"]          # as many as have a row here, on average
    xs = SIZE[case["x"]]
    if case["op"] == "dispatch":
        return {"bytes": t * h * xs + pairs * h * xs + 12 * t * k + 4 * case["here"], "flops": 0}
    ys = SIZE[case["y"]]
    b = t * h * ys + pairs * h * xs + 4 * t * k       # y or its gradient, the rows, their places
    if case["op"] == "combine":
        return {"bytes": b + 4 * t * k + (t * h * ys if case["add"] else 0), "flops": 2 * pairs * h}
    if case["op"] == "combine_grad":
        return {"bytes": b + 8 * t * k + pairs * h * xs, "flops": 3 * pairs * h}
    return {"bytes": b, "flops": pairs * h}


# ------------------------------------------------------------------ inputs

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _route(t, k, e, gen, skew):
    """Ids and weights of k of e experts per token: the largest scores, softmax over them; some experts are liked better."""
    score = torch.randn(t, e, generator=gen, device="cuda") + skew * torch.randn(e, generator=gen, device="cuda")
    top, ids = score.topk(k, dim=1)
    return ids.to(torch.int32), torch.softmax(top, dim=1)


def _order(ids, first, here):
    """Stable order of the pairs by expert: offsets [here + 1], pair of each row, row of each pair (-1: none)."""
    flat = ids.reshape(-1).long() - first
    key = torch.where((flat >= 0) & (flat < here), flat, torch.full_like(flat, here))
    pair = torch.argsort(key, stable=True)
    offsets = torch.searchsorted(key[pair], torch.arange(here + 1, device=ids.device))
    place = torch.empty_like(pair)
    place[pair] = torch.arange(pair.numel(), device=ids.device)
    inv = torch.where(key < here, place, torch.full_like(place, -1)).view(ids.shape)
    return offsets.to(torch.int32), pair, inv.to(torch.int32)


def _make_codes(shape, gen):
    """Two codes a byte, spread like a trained matrix's."""
    at = (torch.arange(256, device="cuda", dtype=torch.float64) + 0.5) / 256
    code = torch.clamp(torch.round(torch.erfinv(2 * at - 1) * 2 ** 0.5 * 2.7 + 8), 0, 15).to(torch.uint8)
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat = out.view(-1)
    for lo in range(0, flat.numel(), 1 << 27):
        part = flat[lo:lo + (1 << 27)]
        low, high = (code[torch.randint(0, 256, part.shape, generator=gen, device="cuda", dtype=torch.uint8).int()] for _ in range(2))
        part.copy_(low | (high << 4))
    return out


def _make_matrix(case, gen):
    lead = (case["e"],) if case["op"] == "experts4" else ()
    groups = -(-case["kin"] // case["group"])
    q = _make_codes((*lead, case["n"], -(-case["kin"] // 2)), gen)
    s = (0.006 * (0.6 + 0.8 * torch.rand(*lead, case["n"], groups, generator=gen, device="cuda"))).to(DT[case["s"]])
    z = torch.randint(4, 13, (*lead, case["n"], groups), generator=gen, device="cuda", dtype=torch.uint8) if case["zero"] else None
    return q, s, z


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    st = {"case": dict(case)}
    if own:
        import moe_expert_ffn_02_gb300 as moe

    def randn(*shape, dt):
        return torch.randn(*shape, generator=gen, device="cuda").to(DT[dt])

    if case["op"] in ("int4", "experts4"):
        st["w"] = _make_matrix(case, gen)
        if case["gated"]:
            st["up"] = _make_matrix(case, gen)
        rows = case["m"] if case["op"] == "int4" else case["t"] * case["k"]
        if case["op"] == "experts4":
            ids, _ = _route(case["t"], case["k"], case["e"], gen, 0.0)
            st["offsets"], pair, _ = _order(ids, 0, case["e"])
            st["token"] = (pair // case["k"]).to(torch.int32) if case["gather"] else None
            st["bounds"] = st["offsets"].tolist()     # the plain form's loop goes over the experts that have rows
        st["x"] = randn(case["t"] if case.get("gather") else rows, case["kin"], dt="bf16")
        if own:             # the weights' handle and the buffer that a serving loop keeps
            q, s, z = st["w"]
            more = dict(group=case["group"], in_features=case["kin"])
            if case["gated"]:
                qu, su, zu = st["up"]
                st["lin"] = moe.Int4GatedLinear(q, s, qu, su, z, zu, **more)
            else:
                st["lin"] = moe.Int4Linear(q, s, z, **more)
            st["y"] = torch.zeros(rows, case["n"], dtype=DT[case["y"]], device="cuda")
        return st

    t, k, h = case["t"], case["k"], case["h"]
    st["ids"], st["weight"] = _route(t, k, case["e"], gen, 0.5)
    if own:                 # the plan with its buffers
        st["plan"] = moe.ExpertPlan(t, k, case["here"], case["first"])
    if case["op"] == "dispatch":
        st["x"] = randn(t, h, dt=case["x"])
        if own:
            st["rows"] = torch.zeros(t * k, h, dtype=DT[case["x"]], device="cuda")
        return st
    # the later operators find the order made
    st["offsets"], _, st["inv"] = _order(st["ids"], case["first"], case["here"])
    if own:
        st["plan"].sort(st["ids"])
    st["rows"] = randn(t * k, h, dt=case["x"])
    if case["op"] == "combine_grad":
        st["dy"] = randn(t, h, dt=case["y"])
        if own:
            st["d_rows"] = torch.zeros_like(st["rows"])
            st["d_w"] = torch.empty_like(st["weight"])
        return st
    st["add"] = randn(t, h, dt=case["y"]) if case.get("add") else None
    if own:
        st["y"] = torch.empty(t, h, dtype=DT[case["y"]], device="cuda")
    return st


# ------------------------------------------------------------------ a pass

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    op = st["case"]["op"]
    if op == "int4":
        st["lin"](st["x"], st["y"])
        return {"y": st["y"]}
    if op == "experts4":
        st["lin"](st["x"], st["y"], st["offsets"], st["token"])
        return {"y": st["y"]}
    plan = st["plan"]
    if op == "dispatch":
        plan.dispatch(st["ids"], st["x"], st["rows"])
        return {"rows": st["rows"], "offsets": plan.expert_offsets, "token": plan.sorted_token, "inv": plan.inv_row}
    if op == "dispatch_grad":
        plan.dispatch_grad(st["rows"], st["y"])
        return {"dx": st["y"]}
    if op == "combine":
        plan.combine(st["rows"], st["weight"], st["y"], add=st["add"])
        return {"y": st["y"]}
    plan.combine_grad(st["dy"], st["rows"], st["weight"], st["d_rows"], st["d_w"])
    return {"d_rows": st["d_rows"], "d_w": st["d_w"]}


def _dequant(q, s, z, kin, group):
    """[n][kin] fp32 weights."""
    code = torch.stack((q & 15, q >> 4), -1).flatten(1)[:, :kin].float()
    g = torch.arange(kin, device=q.device) // group
    return (code - (8.0 if z is None else z.float()[:, g])) * s.float()[:, g]


def _product(st, x, at=()):
    case = st["case"]
    parts = [x @ _dequant(*(None if v is None else v[at] for v in w), case["kin"], case["group"]).t()
             for w in ((st["w"], st["up"]) if case["gated"] else (st["w"],))]
    y = parts[0] if len(parts) == 1 else parts[0] * torch.sigmoid(parts[0]) * parts[1]
    return y.to(DT[case["y"]])


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "int4":
        return {"y": _product(st, st["x"].float())}
    if op == "experts4":
        x = (st["x"] if st["token"] is None else st["x"][st["token"]]).float()
        b = st["bounds"]
        return {"y": torch.cat([_product(st, x[b[i]:b[i + 1]], i) for i in range(case["e"]) if b[i + 1] > b[i]])}
    k, h = case["k"], case["h"]
    if op == "dispatch":
        offsets, pair, inv = _order(st["ids"], case["first"], case["here"])
        live = torch.arange(pair.numel(), device=pair.device) < offsets[-1]
        token = torch.where(live, pair // k, torch.full_like(pair, -1))
        rows = torch.where(live[:, None], st["x"][token.clamp(min=0)], torch.zeros((), dtype=st["x"].dtype, device=pair.device))
        return {"rows": rows, "offsets": offsets, "token": token.to(torch.int32), "inv": inv}
    inv = st["inv"].long()
    live = inv >= 0
    if op == "combine_grad":
        dy = st["dy"].float()[:, None]
        got = st["rows"][inv.clamp(min=0)].float()
        d_w = torch.where(live, (got * dy).sum(-1), torch.zeros_like(st["weight"]))
        d_rows = torch.zeros(inv.numel() + 1, h, dtype=DT[case["x"]], device=inv.device)
        d_rows[torch.where(live, inv, inv.numel()).view(-1)] = (st["weight"][..., None] * dy).to(DT[case["x"]]).view(-1, h)
        return {"d_rows": d_rows[:-1], "d_w": d_w}
    w = live.float() * (st["weight"] if op == "combine" else 1.0)
    y = (st["rows"][inv.clamp(min=0)].float() * w[..., None]).sum(1)
    if st["add"] is not None:
        y = y + st["add"].float()
    return {"dx" if op == "dispatch_grad" else "y": y.to(DT[case["y"]])}


# ------------------------------------------------------------------ 64 bits

def _exact_matrix(q, s, z, kin, group):
    n = q.shape[0]
    w = torch.empty(n, 2 * q.shape[1], dtype=torch.float64, device=q.device)
    w[:, 0::2] = torch.remainder(q, 16).double()
    w[:, 1::2] = torch.div(q, 16, rounding_mode="floor").double()
    for g in range(s.shape[1]):
        cut = slice(g * group, min(kin, (g + 1) * group))
        w[:, cut] = (w[:, cut] - (8 if z is None else z[:, g:g + 1].double())) * s[:, g:g + 1].double()
    return w[:, :kin]


def _exact_product(x, mats, kin, group):
    got = [torch.einsum("mk,nk->mn", x.double(), _exact_matrix(*m, kin, group)) for m in mats]
    return got[0] if len(got) == 1 else got[0] / (1 + torch.exp(-got[0])) * got[1]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("int4", "experts4"):
        mats = [st["w"]] + ([st["up"]] if case["gated"] else [])
        if op == "int4":
            return {"y": _exact_product(st["x"], mats, case["kin"], case["group"])}
        y = torch.zeros(case["t"] * case["k"], case["n"], dtype=torch.float64, device="cuda")
        for i in range(case["e"]):
            lo, hi = int(st["offsets"][i]), int(st["offsets"][i + 1])
            if hi > lo:
                x = st["x"][lo:hi] if st["token"] is None else st["x"].index_select(0, st["token"][lo:hi])
                y[lo:hi] = _exact_product(x, [[None if v is None else v[i] for v in m] for m in mats], case["kin"], case["group"])
        return {"y": y}
    ids = st["ids"].cpu()
    t, k = ids.shape
    # row by row: the pairs of expert 0 in order, then those of expert 1, ...
    local = ids.view(-1).long() - case["first"]
    offsets, order = [0], []
    pairs = torch.arange(t * k)
    for i in range(case["here"]):
        order.append(pairs[local == i])
        offsets.append(offsets[-1] + order[-1].numel())
    order = torch.cat(order)
    n = order.numel()
    inv = torch.full((t * k,), -1)
    inv[order] = torch.arange(n)
    order, inv = order.cuda(), inv.view(t, k).cuda()
    token = order // k
    if op == "dispatch":
        rows = torch.zeros(t * k, case["h"], dtype=torch.float64, device="cuda")
        rows[:n] = st["x"].double().index_select(0, token)
        at = torch.full((t * k,), -1, device="cuda")
        at[:n] = token
        return {"rows": rows, "offsets": torch.tensor(offsets, dtype=torch.int32), "token": at.int(), "inv": inv.int()}
    h = case["h"]
    if op == "combine_grad":
        w = st["weight"].double().view(-1)[order]
        dy = st["dy"].double()
        d_rows = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
        d_w = torch.zeros(t * k, dtype=torch.float64, device="cuda")
        for lo in range(0, n, 8192):
            cut = slice(lo, min(n, lo + 8192))
            mine = dy[token[cut]]
            d_rows[cut] = mine * w[cut, None]
            d_w[order[cut]] = torch.einsum("rh,rh->r", st["rows"][cut].double(), mine)
        return {"d_rows": d_rows, "d_w": d_w.view(t, k)}
    y = torch.zeros(t, h, dtype=torch.float64, device="cuda") if st["add"] is None else st["add"].double()
    for j in range(k):
        have = (inv[:, j] >= 0).nonzero()[:, 0]
        part = st["rows"].index_select(0, inv[have, j]).double()
        y[have] += part * (st["weight"][have, j, None].double() if op == "combine" else 1)
    return {"dx" if op == "dispatch_grad" else "y": y}
