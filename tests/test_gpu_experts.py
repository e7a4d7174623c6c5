"""The operators around experts outside the fused layer on the GPU (dispatch,
combine and their gradients) against plain 64-bit forms of their definitions.

Tolerances, derived from the arithmetic (u = 2^-24, half an fp32 ulp):

- the order and the copied rows are exact
- combine: one fused multiply-add per slot, k roundings of partial sums that the
  sum of magnitudes bounds: k u of it; the output adds half a step of its type
- d_rows: one fp32 product (u) and half a step of its type
- d_w: a thread adds up at most 32 terms per 8192 columns (4 per 1024 where rows lie
  off the 16-byte grid), five levels of shuffles, one addition per 8192 (1024)
  columns, eight warps: under 128 roundings for the widths here, 128 u of the
  sum of magnitudes
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import moe_expert_ffn_02_gb300 as m
    m.load()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=gen(seed), device="cuda").to(dtype)


def strided(t, pad):
    """The same values in rows `pad` elements further apart; what lies between them is NaN."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def make_ids(t, k, e, seed, kind):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":                                   # everybody wants the same expert, twice over
        return torch.full((t, k), e - 1, dtype=torch.int32)
    ids = torch.randint(0, e, (t, k), generator=g, dtype=torch.int32)
    if kind == "wild":                                  # dropped pairs and ids of no expert
        bad = torch.tensor([-1, -2 ** 31, 2 ** 31 - 1, e, e + 7], dtype=torch.int32)
        ids = torch.where(torch.rand(t, k, generator=g) < 0.4, bad[torch.randint(0, 5, (t, k), generator=g)], ids)
    return ids


def order(ids, first, here):
    """(offsets, token of each row, inv) by walking the pairs."""
    t, k = ids.shape
    lists = [[] for _ in range(here)]
    for p, i in enumerate(ids.flatten().tolist()):
        if first <= i < first + here:
            lists[i - first].append(p)
    offsets, pairs = [0], []
    for one in lists:
        pairs += one
        offsets.append(len(pairs))
    inv = torch.full((t * k,), -1, dtype=torch.int32)
    inv[pairs] = torch.arange(len(pairs), dtype=torch.int32)
    token = torch.full((t * k,), -1, dtype=torch.int32)
    token[:len(pairs)] = torch.tensor(pairs, dtype=torch.int32) // k
    return torch.tensor(offsets, dtype=torch.int32), token, inv.view(t, k)


def check_order(plan, ids, first, here):
    offsets, token, inv = order(ids, first, here)
    assert torch.equal(plan.expert_offsets.cpu(), offsets)
    assert torch.equal(plan.sorted_token.cpu(), token)
    assert torch.equal(plan.inv_row.cpu(), inv)
    return token, inv


CASES = [  # tokens, top_k, experts in all, first, here, kind
    (1, 1, 1, 0, 1, "plain"), (1, 8, 256, 0, 256, "plain"), (3, 8, 16, 0, 16, "one"), (16, 8, 256, 64, 64, "plain"),
    (128, 8, 256, 0, 256, "wild"), (1024, 1, 1024, 0, 1024, "plain"), (1025, 1, 1024, 0, 1024, "plain"),
    (33, 32, 40, 3, 30, "wild"), (129, 8, 7, 0, 7, "one"), (700, 6, 60, 59, 1, "plain"), (2500, 3, 1000, 500, 500, "wild"),
    (5000, 8, 33, 0, 33, "wild"), (40000, 2, 8, 0, 8, "plain"), (70000, 32, 4, 1, 2, "plain"), (260, 8, 16, 16, 16, "plain"),
]


@pytest.mark.parametrize("t,k,e,first,here,kind", CASES)
def test_sort(moe, t, k, e, first, here, kind):
    ids = make_ids(t, k, e, t + k, kind)
    plan = moe.ExpertPlan(t, k, here, first)
    plan.sort(ids.cuda())
    check_order(plan, ids, first, here)
    assert plan.device_status() == (0, 0)


@pytest.mark.parametrize("t,k,e,first,here,kind", CASES[:8] + CASES[9:11])
@pytest.mark.parametrize("h,pad,dtype", [(1, 0, "bf16"), (7, 1, "bf16"), (1001, 0, "bf16"), (64, 0, "f32"), (257, 0, "f32"), (7168, 8, "bf16"),
                                         (2046, 2, "bf16"), (17000, 0, "bf16")])
def test_dispatch(moe, t, k, e, first, here, kind, h, pad, dtype):
    ids = make_ids(t, k, e, t + k, kind)
    x = strided(randn((t, h), 1, DT[dtype]), pad)
    store = torch.full((t * k, h + pad), 7.0, dtype=DT[dtype], device="cuda")
    rows = store[:, :h]
    plan = moe.ExpertPlan(t + 3, k, here, first)
    assert plan.dispatch(ids.cuda(), x, rows) is rows
    token, _ = check_order(plan, ids, first, here)
    n = int((token >= 0).sum())
    assert torch.equal(rows[:n], x[token[:n].long().cuda()])
    assert (rows[n:] == 7).all() and (store[:, h:] == 7).all()
    # the same order once more, for other rows
    x2 = strided(randn((t, h), 2, DT[dtype]), pad)
    plan.dispatch(None, x2, rows)
    assert torch.equal(rows[:n], x2[token[:n].long().cuda()]) and (rows[n:] == 7).all()
    assert plan.device_status() == (0, 0)


@pytest.mark.parametrize("to", ["bf16", "f32"])
@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("t,k,e,first,here,kind", CASES[:5] + CASES[7:10] + CASES[-1:])
@pytest.mark.parametrize("h,pad", [(1, 0), (8, 8), (1000, 0), (1001, 0), (7168, 0), (9000, 4)])
def test_combine_and_gradients(moe, to, ty, t, k, e, first, here, kind, h, pad):
    ids = make_ids(t, k, e, t + k, kind)
    plan = moe.ExpertPlan(t, k, here, first)
    plan.sort(ids.cuda())
    _, inv = check_order(plan, ids, first, here)
    inv = inv.long().cuda()
    live = inv >= 0
    o = strided(randn((t * k, h), 3, DT[to]), pad)
    n = int(live.sum())
    o[n:] = float("nan")                                # rows that nobody has are not read
    w = torch.randn(t, k, generator=gen(4), device="cuda")
    w[~live] = float("inf")                             # nor is the weight of a pair without a row used
    add = strided(randn((t, h), 5, DT[ty]), pad)
    dy = strided(randn((t, h), 6, DT[ty]), pad)
    od = torch.where(live[..., None], o[inv.clamp(min=0)].double(), 0.0)
    wd = torch.where(live, w.double(), 0.0)

    terms = od * wd[..., None]
    for base in (None, add):
        y = strided(torch.zeros(t, h, dtype=DT[ty], device="cuda"), pad)
        if base is not None and pad:
            y.copy_(base)                               # in place
            base = y
        plan.combine(o, w, y, add=base)
        want = terms.sum(1) + (0 if base is None else add.double())
        mag = terms.abs().sum(1) + (0 if base is None else add.double().abs())
        assert ((y.double() - want).abs() <= want.abs() * HALF[DT[ty]] + mag * (k * U * 1.01)).all()
    dx = torch.empty(t, h, dtype=DT[ty], device="cuda")
    plan.dispatch_grad(o, dx)
    want, mag = od.sum(1), od.abs().sum(1)
    assert ((dx.double() - want).abs() <= want.abs() * HALF[DT[ty]] + mag * (k * U * 1.01)).all()

    store = torch.full((t * k, h + pad), 7.0, dtype=DT[to], device="cuda")
    d_rows, d_w = store[:, :h], torch.full((t, k), 9.0, device="cuda")
    plan.combine_grad(dy, o, w, d_rows, d_w)
    want_rows = (dy.double()[:, None] * wd[..., None])[live]
    got = d_rows[inv[live]].double()
    assert ((got - want_rows).abs() <= want_rows.abs() * (HALF[DT[to]] + U) * 1.01).all()
    assert (d_rows[n:] == 7).all() and (store[:, h:] == 7).all()
    prod = od * dy.double()[:, None]
    assert ((d_w.double() - prod.sum(-1)).abs() <= prod.abs().sum(-1) * (128 * U)).all()
    assert (d_w[~live] == 0).all()
    # either output alone, without weights, and d_rows over rows
    alone = torch.empty_like(d_w)
    plan.combine_grad(dy, o, w, None, alone)
    assert torch.equal(alone, d_w)
    plan.combine_grad(dy, o, w, o, alone)
    assert torch.equal(alone, d_w) and torch.equal(o[:n], d_rows[:n])
    plan.combine_grad(dy, d_rows, None, d_rows)
    assert torch.equal(d_rows[inv[live]], dy[:, None].expand(t, k, h)[live].to(DT[to]))
    assert plan.device_status() == (0, 0)


def test_gradients_by_differences(moe):
    """combine is linear in the rows and in the weights: differences are exact up to rounding, whatever their step."""
    t, k, e, h = 37, 4, 9, 200
    plan = moe.ExpertPlan(t, k, e)
    plan.sort(make_ids(t, k, e, 1, "wild").cuda())
    o, step, dy = (randn((t * k, h), 1), randn((t * k, h), 2), randn((t, h), 3))
    w, w_step = torch.rand(t, k, device="cuda"), torch.rand(t, k, device="cuda")
    d_o, d_w = torch.zeros_like(o), torch.empty_like(w)
    plan.combine_grad(dy, o, w, d_o, d_w)

    def loss(o, w):
        y = torch.empty(t, h, device="cuda")
        plan.combine(o, w, y)
        return (y.double() * dy.double()).sum()

    mag = float((o.double().abs().sum(1).max() + 1) * t * k)
    assert abs(loss(o + step, w) - loss(o, w) - (d_o.double() * step.double()).sum()) <= mag * 64 * U
    assert abs(loss(o, w + w_step) - loss(o, w) - (d_w.double() * w_step.double()).sum()) <= mag * 256 * U
    # and the copy: <dispatch(x), d> = <x, dispatch_grad(d)>
    x, rows, dx = randn((t, h), 4), torch.zeros(t * k, h, device="cuda"), torch.empty(t, h, device="cuda")
    plan.dispatch(None, x, rows)
    plan.dispatch_grad(step, dx)
    assert abs((rows.double() * step.double()).sum() - (x.double() * dx.double()).sum()) <= mag * 64 * U


@pytest.mark.parametrize("cols", [64, 33])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_past_2_to_the_31(moe, cols, dtype):
    """Every operand's last rows start behind 2^31 elements; weights are powers of two and the sums small integers, so
    every result is exact."""
    t, k, e = 60, 2, 8
    far = lambda n: torch.empty((n - 1) * (2 ** 31 // (n - 10) // 8 * 8) + cols, dtype=dtype, device="cuda").as_strided(   # noqa: E731
        (n, cols), (2 ** 31 // (n - 10) // 8 * 8, 1))
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(0, e, (t, k), generator=g, device="cuda", dtype=torch.int32)
    value = torch.randint(-4, 5, (t, cols), generator=g, device="cuda").to(dtype)
    w = 2.0 ** torch.randint(-2, 1, (t, k), generator=g, device="cuda").float()
    plan = moe.ExpertPlan(t, k, e)
    x, rows = far(t), far(t * k)
    x.copy_(value)
    plan.dispatch(ids, x, rows)
    inv = plan.inv_row.long()
    assert torch.equal(rows[inv[:, 1]], value) and torch.equal(rows[plan.inv_row[:, 0].long()], value)
    plan.combine(rows, w, x)
    assert torch.equal(x, (value.float() * w.sum(1, keepdim=True)).to(dtype))
    x.copy_(value)
    d_w = torch.empty(t, k, device="cuda")
    plan.combine_grad(x, rows, w, rows, d_w)
    assert torch.equal(d_w, value.float().square().sum(1, keepdim=True).expand(t, k))
    for j in range(k):
        assert torch.equal(rows[inv[:, j]], (value.float() * w[:, j:j + 1]).to(dtype))
    plan.dispatch_grad(rows, x)
    assert torch.equal(x, (value.float() * w.sum(1, keepdim=True)).to(dtype))
    assert plan.device_status() == (0, 0)


def test_no_tokens_and_fewer_tokens(moe):
    plan = moe.ExpertPlan(3000, 2, 5)
    for t in (3000, 513, 700, 1, 0, 2999):
        ids = make_ids(t, 2, 5, t, "wild")
        x, rows = randn((t, 16), t), torch.zeros(2 * t, 16, device="cuda")
        plan.dispatch(ids.cuda(), x, rows)
        token, _ = check_order(plan, ids, 0, 5)
        live = token >= 0
        assert torch.equal(rows[live.cuda()], x[token[live].long().cuda()])
        y = torch.full((t, 16), 5.0, device="cuda")
        plan.combine(rows, None, y)
        plan.combine_grad(y, rows, None, None, torch.empty(t, 2, device="cuda"))
    assert plan.device_status() == (0, 0)


@pytest.mark.parametrize("t", [5, 700])
def test_rows_that_do_not_fit_are_left_out_and_flagged(moe, t):
    k, e, h = 4, 8, 40
    ids = make_ids(t, k, e, 3, "plain")
    plan = moe.ExpertPlan(t, k, e)
    x = randn((t, h), 1)
    store = torch.full((t * k, h), 7.0, device="cuda")
    short = store[:t * k - 3]
    plan.dispatch(ids.cuda(), x, short)
    token, inv = check_order(plan, ids, 0, e)
    assert torch.equal(short, x[token[:-3].long().cuda()]) and (store[-3:] == 7).all()
    assert plan.device_status() == (5, moe.DEV_BAD_ROW) and plan.device_status() == (0, 0)
    y, want = torch.empty(t, h, device="cuda"), torch.zeros(t, h, dtype=torch.float64, device="cuda")
    plan.combine(short, None, y)
    want.index_add_(0, token[:-3].long().cuda(), short.double())
    assert ((y - want).abs() <= 1e-5).all()
    assert plan.device_status() == (5, moe.DEV_BAD_ROW)
    d_w = torch.full((t, k), 9.0, device="cuda")
    plan.combine_grad(x, short, None, None, d_w)
    assert plan.device_status() == (5, moe.DEV_BAD_ROW)
    lost = inv >= t * k - 3
    assert (d_w.cpu()[lost] == 0).all() and (d_w.cpu()[~lost] != 9).all()


def test_nan_and_infinity_pass_through(moe):
    plan = moe.ExpertPlan(2, 2, 2)
    plan.sort(torch.tensor([[0, 1], [1, 0]], dtype=torch.int32).cuda())
    o = torch.ones(4, 16, device="cuda")
    o[0, 3], o[1, 4] = float("nan"), float("inf")
    y = torch.empty(2, 16, device="cuda")
    plan.combine(o, torch.ones(2, 2, device="cuda"), y)
    assert y[0, 3].isnan() and y[1, 4].isinf() and torch.isfinite(y).sum() == 30


@pytest.mark.parametrize("t", [16, 900])
def test_captured_and_replayed_on_another_stream(moe, t):
    k, e, h = 8, 64, 512
    plan = moe.ExpertPlan(t, k, e)
    ids = make_ids(t, k, e, 1, "plain").cuda()
    x, w = randn((t, h), 1, torch.bfloat16), torch.rand(t, k, device="cuda")
    rows, y = torch.zeros(t * k, h, dtype=torch.bfloat16, device="cuda"), torch.empty(t, h, device="cuda")

    def step():
        plan.dispatch(ids, x, rows)
        plan.combine(rows, w, y, add=None)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (2, 3, 4):
        new = make_ids(t, k, e, seed, "wild")
        ids.copy_(new.cuda())
        x.copy_(randn((t, h), seed, torch.bfloat16))
        rows.zero_()
        graph.replay()
        live = (check_order(plan, new, 0, e)[1] >= 0).cuda()
        want = x.double() * (w.double() * live).sum(1, keepdim=True)
        assert ((y.double() - want).abs() <= (x.double().abs() * w.double().sum(1, keepdim=True)) * (9 * U)).all()


def test_python_refusals(moe):
    plan = moe.ExpertPlan(4, 2, 8)
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    x, rows, y = torch.zeros(4, 16, device="cuda"), torch.zeros(8, 16, device="cuda"), torch.zeros(4, 16, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    plan.dispatch(ids, x, rows)
    for bad in (lambda: plan.sort(ids.long()), lambda: plan.sort(ids.cpu()), lambda: plan.sort(ids[:, :1]), lambda: plan.sort(ids.t().contiguous()),
                lambda: plan.sort(torch.zeros(5, 2, dtype=torch.int32, device="cuda")), lambda: plan.sort(torch.zeros(4, 4, dtype=torch.int32, device="cuda")[:, ::2]),
                lambda: plan.dispatch(ids, x), lambda: plan.dispatch(ids, None, rows), lambda: plan.dispatch(None), lambda: plan.dispatch(ids, x, rows.bfloat16()),
                lambda: plan.dispatch(ids, x, rows[:, :8]), lambda: plan.dispatch(ids, x.cpu(), rows), lambda: plan.dispatch(ids, x.half(), rows.half()),
                lambda: plan.dispatch(ids, x[:3], rows), lambda: plan.dispatch(ids, x.t().contiguous().t(), rows), lambda: plan.dispatch(ids, x[:1].expand(4, 16), rows),
                lambda: plan.combine(rows, w[:3], y), lambda: plan.combine(rows, w.double(), y), lambda: plan.combine(rows, w, y[:3]),
                lambda: plan.combine(rows, w, y, add=y.bfloat16()), lambda: plan.combine(rows, w, y[:, :8]), lambda: plan.combine(rows.cpu(), w, y),
                lambda: plan.combine_grad(y, rows, w), lambda: plan.combine_grad(y, rows, w, rows.bfloat16()), lambda: plan.combine_grad(y, rows, w, rows[:7]),
                lambda: plan.combine_grad(y, rows, w, None, w[:3]),
                lambda: moe.ExpertPlan(4, 33, 8), lambda: moe.ExpertPlan(4, 2, 1025), lambda: moe.ExpertPlan(-1, 2, 8), lambda: moe.ExpertPlan(4, 0, 8),
                lambda: moe.ExpertPlan(4, 2, 8, -1), lambda: moe.ExpertPlan(4, 2, 8, 2 ** 31 - 8), lambda: moe.ExpertPlan(4, 2, 8, device="cpu")):
        with pytest.raises(moe.MoeError):
            bad()
    assert plan.device_status() == (0, 0)


def test_routing_outputs_fit_as_they_are(moe):
    """The order that moe_route makes, used by combine, against the plan's own."""
    import _harness as h
    import synth
    wl = synth.WORKLOADS["tiny"]
    inp = synth.make_inputs(wl, seed=0)
    layer = h.make_layer(wl, inp)
    r = h.route(layer, inp["x"])
    ids = torch.as_tensor(r["topk_ids"])
    plan = moe.ExpertPlan(ids.shape[0], ids.shape[1], wl.n_experts)
    plan.sort(ids.int().cuda())
    assert torch.equal(plan.expert_offsets.cpu(), torch.as_tensor(r["expert_offsets"]).int())
    assert torch.equal(plan.sorted_token.cpu(), torch.as_tensor(r["sorted_token"]).int().flatten())
    assert torch.equal(plan.inv_row.cpu(), torch.as_tensor(r["inv_row"]).int().view(plan.inv_row.shape))
    layer.close()
