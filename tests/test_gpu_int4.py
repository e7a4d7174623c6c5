"""Products with 4-bit weights on the GPU against plain 64-bit forms of their
definition.

Tolerance, derived from the arithmetic (u = 2^-24, half an fp32 ulp): a code less
its zero point is an integer of eight bits and its product with a bf16 value
exact.  The tensor cores add 32 or 64 channels' products with a few fp32 units
lost, each partial sum is scaled and added with one rounding each, and the warps'
(or chunks') sums meet in a tree: (in / 32 + 32) 2^-23 of the sum of the
products' magnitudes, scales included.  SiLU's derivative stays below 1.1, its
exponential, quotient and product add 8 u, and the output half a step of its type.
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


def matrix(lead, n, k, group, zero, s, seed):
    """Codes, scales, zero points and the 64-bit weights."""
    g = gen(seed)
    q = torch.randint(0, 256, (*lead, n, (k + 1) // 2), generator=g, device="cuda", dtype=torch.uint8)
    groups = (k + group - 1) // group
    sc = (0.01 + torch.rand(*lead, n, groups, generator=g, device="cuda") * 0.02).to(DT[s])
    z = torch.randint(0, 128, (*lead, n, groups), generator=g, device="cuda", dtype=torch.uint8) if zero else None
    code = torch.empty(*lead, n, 2 * q.shape[-1], dtype=torch.float64, device="cuda")
    code[..., 0::2], code[..., 1::2] = (q & 15).double(), (q >> 4).double()
    wide = lambda t: t.double().repeat_interleave(group, -1)[..., :k]   # noqa: E731
    return q, sc, z, (code[..., :k] - (8 if z is None else wide(z))) * wide(sc)


def strided(t, pad):
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def expect(x, mats):
    """The exact result and the error that the sums may have, both 64-bit, of rows x and one expert's matrices."""
    k = x.shape[1]
    got = [(x.double() @ w.t(), (x.double().abs() @ w.abs().t()) * ((k / 32 + 32) * 2.0 ** -23)) for w in mats]
    if len(got) == 1:
        return got[0]
    (g, dg), (u, du) = got
    silu = g / (1 + torch.exp(-g))
    h = silu * u
    return h, 1.1 * dg * u.abs() + silu.abs() * du + 1.1 * dg * du + 8 * U * h.abs()


def check(y, want, slack):
    tol = slack + want.abs() * (HALF[y.dtype] * 1.01) + 1e-38
    err = (y.double() - want).abs()
    assert (err <= tol).all(), (float((err / tol).max()), int((err > tol).sum()))


def make(moe, lead, n, k, gated, group, zero, s, seed=0):
    a = matrix(lead, n, k, group, zero, s, seed)
    if not gated:
        return moe.Int4Linear(*a[:3], group=group, in_features=k), [a[3]]
    b = matrix(lead, n, k, group, zero, s, seed + 1)
    return moe.Int4GatedLinear(a[0], a[1], b[0], b[1], a[2], b[2], group=group, in_features=k), [a[3], b[3]]


SHAPES = [(1, 1), (16, 64), (5, 31), (17, 65), (128, 512), (100, 130), (130, 1991), (64, 1000), (1001, 96), (520, 4100)]


@pytest.mark.parametrize("m", [1, 7, 8, 9, 16, 17, 33, 64, 65, 200, 777])
@pytest.mark.parametrize("n,k", SHAPES)
@pytest.mark.parametrize("gated,group,zero,s,yt", [(False, 128, False, "bf16", "bf16"), (False, 32, True, "f32", "f32"), (True, 64, True, "bf16", "f32"),
                                                   (True, 96, False, "f32", "bf16"), (False, 4128, True, "bf16", "f32")])
def test_dense(moe, m, n, k, gated, group, zero, s, yt):
    lin, mats = make(moe, (), n, k, gated, group, zero, s)
    x = torch.randn(m, k, generator=gen(5), device="cuda").bfloat16()
    y = torch.full((m, n), 7.0, dtype=DT[yt], device="cuda")
    assert lin(x, y) is y
    check(y, *expect(x, mats))
    assert lin.device_status() == (0, 0)


@pytest.mark.parametrize("m", [1, 12, 100, 300])
@pytest.mark.parametrize("xpad,ypad", [(8, 0), (1, 3), (2, 2), (7, 16)])
def test_strides(moe, m, xpad, ypad):
    n, k = 200, 320
    lin, mats = make(moe, (), n, k, False, 64, True, "bf16")
    x = strided(torch.randn(m, k, generator=gen(6), device="cuda").bfloat16(), xpad)
    store = torch.full((m, n + ypad), 7.0, device="cuda")
    y = store[:, :n]
    lin(x, y)
    check(y, *expect(x, mats))
    assert (store[:, n:] == 7).all()
    # off the 16-byte grid by its address alone
    x2 = torch.randn(m * k + 1, generator=gen(7), device="cuda").bfloat16()[1:].view(m, k)
    lin(x2, y)
    check(y, *expect(x2, mats))


@pytest.mark.parametrize("m,n,k,group", [(70, 300, 4096, 128), (129, 1000, 2100, 64), (65, 64, 7000, 32), (1000, 4096, 1024, 128), (3000, 520, 640, 32),
                                         (90, 7168, 4096, 128), (250, 2100, 4096, 64), (250, 2100, 4104, 32), (2000, 1000, 520, 64), (400, 2048, 4096, 96)])
@pytest.mark.parametrize("gated", [False, True])
def test_many_rows(moe, m, n, k, group, gated):
    """Tiles that 2, 4 or 8 CTAs share, several tiles per CTA, all three sizes of chunk."""
    lin, mats = make(moe, (), n, k, gated, group, True, "bf16")
    x = (torch.randn(m, k, generator=gen(5), device="cuda") * 0.05).bfloat16()
    for yt in ("bf16", "f32"):
        y = torch.full((m, n), 7.0, dtype=DT[yt], device="cuda")
        lin(x, y)
        check(y, *expect(x, mats))
    assert lin.device_status() == (0, 0)


def offsets_of(counts, start=0):
    return torch.tensor([start, *(start + torch.tensor(counts).cumsum(0)).tolist()], dtype=torch.int32, device="cuda")


COUNTS = [[1], [0, 0, 3], [5, 0, 1, 0, 9, 1, 1, 0], [0] * 30 + [1] + [0] * 9, [40, 1, 0, 17, 8, 64], [300, 0, 129, 1, 128, 77], [1] * 100, [2500, 3]]


@pytest.mark.parametrize("counts", COUNTS, ids=[f"e{len(c)}r{sum(c)}" for c in COUNTS])
@pytest.mark.parametrize("n,k,gated,group,zero,s,yt,gather", [
    (96, 256, False, 128, False, "bf16", "bf16", False), (131, 200, True, 32, True, "bf16", "f32", True),
    (72, 515, False, 64, True, "f32", "f32", True), (256, 1024, True, 64, False, "f32", "bf16", False)])
def test_experts(moe, counts, n, k, gated, group, zero, s, yt, gather):
    e, rows = len(counts), sum(counts)
    lin, mats = make(moe, (e,), n, k, gated, group, zero, s)
    tail, head = 5, 3                       # rows of no expert on both sides stay as they were
    total = head + rows + tail
    g = gen(9)
    x = torch.randn(40 if gather else total, k, generator=g, device="cuda").bfloat16()
    token = torch.randint(0, 40, (total,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    y = torch.full((total, n), 7.0, dtype=DT[yt], device="cuda")
    if gather:
        token[:head] = -5                   # of rows that are not computed nothing is read
    lin(x, y, offsets_of(counts, head), token)
    xr = x[token[head:].clamp(min=0).long()] if gather else x[head:]
    at = 0
    for i, c in enumerate(counts):
        if c:
            check(y[head + at:head + at + c], *expect(xr[at:at + c], [w[i] for w in mats]))
        at += c
    assert (y[:head] == 7).all() and (y[head + rows:] == 7).all()
    assert lin.device_status() == (0, 0)


def test_many_experts_with_long_rows(moe):
    """Images and outputs past 32-bit element counts are covered by their sizes; here the last expert of many."""
    e, n, k = 1024, 64, 128
    lin, mats = make(moe, (e,), n, k, False, 32, False, "bf16")
    offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = 6
    x = torch.randn(6, k, generator=gen(1), device="cuda").bfloat16()
    y = torch.empty(6, n, device="cuda")
    lin(x, y, offsets)
    check(y, *expect(x, [mats[0][-1]]))


def test_image_past_4_gib(moe):
    """Codes of 5 GiB: the last expert's lie behind every 32-bit offset."""
    e, n, k = 320, 4096, 8192
    q = torch.randint(0, 256, (e, n, k // 2), generator=gen(1), device="cuda", dtype=torch.uint8)
    s = torch.full((e, n, k // 128), 0.01, device="cuda").bfloat16()
    lin = moe.Int4Linear(q, s)
    for rows in (2, 200):
        x = torch.randn(rows, k, generator=gen(2), device="cuda").bfloat16()
        y = torch.empty(rows, n, device="cuda")
        offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
        offsets[-1] = rows
        lin(x, y, offsets)
        code = torch.stack((q[-1] & 15, q[-1] >> 4), -1).flatten(1).double()
        check(y, *expect(x, [(code - 8) * float(s[0, 0, 0])]))


def far_rows(rows, cols, dtype, pad=0):
    """Rows so far apart that the last start behind 2^31 elements."""
    ld = 2 ** 31 // (rows - 40) + pad
    ld -= 0 if pad else ld % 8
    return torch.empty(ld * (rows - 1) + cols, dtype=dtype, device="cuda").as_strided((rows, cols), (ld, 1))


@pytest.mark.parametrize("m", [50, 300])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("gather", [False, True])
def test_rows_past_2_to_the_31(moe, m, pad, gather):
    n, k = 72, 200
    lin, mats = make(moe, (), n, k, False, 64, True, "bf16")
    x, y = far_rows(m, k, torch.bfloat16, pad), far_rows(m, n, torch.bfloat16)
    x.copy_(torch.randn(m, k, generator=gen(1), device="cuda"))
    y.fill_(7)
    if gather:
        token = torch.arange(m - 1, -1, -1, dtype=torch.int32, device="cuda")
        lin(x, y, None, token)
        check(y, *expect(x.flip(0), mats))
    else:
        lin(x, y)
        check(y, *expect(x, mats))


@pytest.mark.parametrize("m,n,k,gated,group", [(3, 700, 2048, True, 32), (64, 512, 4096, False, 128), (200, 1000, 1024, True, 64), (1200, 2048, 512, False, 32)])
def test_two_streams_share_the_weights(moe, m, n, k, gated, group):
    lin, mats = make(moe, (), n, k, gated, group, False, "bf16")
    xs = [torch.randn(m, k, generator=gen(i), device="cuda").bfloat16() for i in range(2)]
    want = [torch.empty(m, n, device="cuda") for _ in xs]
    for x, y in zip(xs, want):
        lin(x, y)
        check(y, *expect(x, mats))
    runs = 8
    got = [[torch.empty(m, n, device="cuda") for _ in range(runs)] for _ in xs]
    side = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for i in range(runs):
        for j, st in enumerate(side):
            with torch.cuda.stream(st):
                lin(xs[j], got[j][i])
    torch.cuda.synchronize()
    assert lin.device_status() == (0, 0)
    assert all(torch.equal(y, want[j]) for j in range(2) for y in got[j])


@pytest.mark.parametrize("rows", [4, 300])
def test_bad_offsets_and_tokens_stay_in_bounds_and_are_flagged(moe, rows):
    e, n, k = 4, 64, 128
    lin, mats = make(moe, (e,), n, k, False, 128, False, "bf16")
    x = torch.randn(rows, k, generator=gen(1), device="cuda").bfloat16()
    store = torch.full((rows + 8, n), 7.0, device="cuda")
    y = store[4:4 + rows]
    for off in ([-3, 1, 2, 3, rows], [0, 1, 2, 3, rows + 9], [0, 3, 1, 3, rows]):
        lin(x, y, torch.tensor(off, dtype=torch.int32, device="cuda"))
        assert lin.device_status() == (5, moe.DEV_BAD_ROW)
        assert (store[:4] == 7).all() and (store[-4:] == 7).all()
    token = torch.arange(rows, dtype=torch.int32, device="cuda")
    token[1], token[2] = rows, -1
    lin(x, y, torch.tensor([0, 1, 2, 3, rows], dtype=torch.int32, device="cuda"), token)
    assert lin.device_status() == (5, moe.DEV_BAD_ROW) and lin.device_status() == (0, 0)
    assert (y[1] == 0).all() and (y[2] == 0).all()
    check(y[:1], *expect(x[:1], [mats[0][0]]))


@pytest.mark.parametrize("rows", [4, 300, 3000])
@pytest.mark.parametrize("gather", [False, True])
def test_falling_offsets_give_each_row_one_expert(moe, rows, gather):
    n, k = 64, 128
    r = rows
    for off in ([0, r, 0, r, 1, r, r], [2, 0, 3, 1, r - 1, r, 3], [r, 0, r, 0, r, 0, r], [r + 5, 1, 2, 3, 4, 5, 6], [0, r // 2, r // 4, r, -7, r, 2 * r],
                [0] + [r, 0] * 400):
        e = len(off) - 1
        lin, mats = make(moe, (e,), n, k, False, 128, False, "bf16")
        x = torch.randn(r, k, generator=gen(1), device="cuda").bfloat16()
        token = torch.randperm(r, generator=gen(2), device="cuda").int() if gather else None
        y = torch.full((r, n), 7.0, device="cuda")
        lin(x, y, torch.tensor(off, dtype=torch.int32, device="cuda"), token)
        assert lin.device_status() == (5, moe.DEV_BAD_ROW)
        low, left = min(max(off[0], 0), r), torch.ones(r, dtype=torch.bool)
        for i in range(e):
            high = max(low, min(max(off[i + 1], 0), r))
            if high > low:
                xi = x[low:high] if token is None else x[token[low:high].long()]
                check(y[low:high], *expect(xi, [m[i] for m in mats]))
                left[low:high] = False
            low = high
        assert (y[left.cuda()] == 7).all()


@pytest.mark.parametrize("m", [3, 100])
def test_nan_and_infinity_stay_in_their_row(moe, m):
    n, k = 80, 200
    lin, mats = make(moe, (), n, k, False, 64, False, "bf16")
    x = torch.randn(m, k, generator=gen(1), device="cuda").bfloat16()
    x[1, 7], x[2, 199] = float("nan"), float("inf")
    y = torch.empty(m, n, device="cuda")
    lin(x, y)
    assert y[1].isnan().all() and not torch.isfinite(y[2]).any()
    rest = [i for i in range(m) if i not in (1, 2)]
    check(y[rest], *expect(x[rest], mats))


@pytest.mark.parametrize("m", [4, 150])
def test_same_bits_each_time_and_captured(moe, m):
    n, k = 300, 700
    lin, mats = make(moe, (), n, k, True, 64, True, "bf16")
    x = torch.randn(m, k, generator=gen(1), device="cuda").bfloat16()
    y, again = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    lin(x, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lin(x, again)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin(x, again)
    x.copy_(torch.randn(m, k, generator=gen(2), device="cuda"))
    graph.replay()
    check(again, *expect(x, mats))


@pytest.mark.parametrize("m,n,k", [(600, 2048, 2048), (1500, 7168, 256), (600, 2048, 2047), (600, 7168, 256)])
def test_a_wait_that_expires_leaves_the_output_right_or_as_it_was(moe, m, n, k):
    """Tiles that clusters share, tiles that they do not, rows off the 16-byte grid."""
    lin, mats = make(moe, (), n, k, False, 128, False, "bf16")
    x = torch.randn(m, k, generator=gen(1), device="cuda").bfloat16()
    y = torch.full((m, n), 7.0, device="cuda")
    want, slack = expect(x, mats)
    moe.moe_int4_set_wait_limit(lin.handle, 2000)
    moe.moe_int4_debug_timeout(lin.handle)
    lin(x, y)
    assert lin.device_status() == (6, moe.DEV_WAIT_TIMEOUT)
    kept = y == 7
    assert kept.any() and not kept.all()
    assert (((y.double() - want).abs() <= slack + want.abs() * U * 1.01) | kept).all()
    moe.moe_int4_set_wait_limit(lin.handle, 2_000_000)
    lin(x, y)
    check(y, want, slack)
    assert lin.device_status() == (0, 0)


@pytest.mark.parametrize("m,n,k", [(100, 256, 1024), (100, 256, 1001)])
def test_the_form_without_waits_leaves_the_hook_alone(moe, m, n, k):
    lin, mats = make(moe, (), n, k, False, 128, False, "bf16")
    x = torch.randn(m, k, generator=gen(1), device="cuda").bfloat16()
    y = torch.full((m, n), 7.0, device="cuda")
    moe.moe_int4_debug_timeout(lin.handle)
    lin(x, y)
    check(y, *expect(x, mats))
    assert lin.device_status() == (0, 0)


@pytest.mark.parametrize("m", [2, 40, 300])
@pytest.mark.parametrize("k", [64, 320, 1024])
def test_largest_zero_points_and_scales_of_every_size(moe, m, k):
    """Zero points of 127 and scales from 2^-120 to 2^100: products and scaled sums in fp32's range stay exact to the bound."""
    n, group = 48, 64
    q = torch.randint(0, 256, (n, k // 2), generator=gen(1), device="cuda", dtype=torch.uint8)
    s = torch.exp2(torch.linspace(-120, 100, n, device="cuda").round())[:, None].expand(n, k // group).contiguous()
    z = torch.full((n, k // group), 127, dtype=torch.uint8, device="cuda")
    lin = moe.Int4Linear(q, s, z, group=group)
    code = torch.stack((q & 15, q >> 4), -1).flatten(1).double()
    x = torch.randn(m, k, generator=gen(2), device="cuda").bfloat16()
    y = torch.empty(m, n, device="cuda")
    lin(x, y)
    check(y, *expect(x, [(code - 127) * s[:, :1].double()]))


def test_x_without_rows_is_refused(moe):
    lin, _ = make(moe, (), 64, 128, False, 128, False, "bf16")
    x, y, token = (torch.zeros(64, 128, dtype=t, device="cuda") for t in (torch.bfloat16, torch.float32, torch.int32))
    args = moe.MoeInt4Args(rows=64, x_rows=0, x=x.data_ptr(), ldx=128, token=token.data_ptr(), y=y.data_ptr(), ldy=128, y_type=moe.F32)
    with pytest.raises(moe.MoeError):
        moe.moe_int4_forward(lin.handle, args)


def test_no_rows(moe):
    lin, _ = make(moe, (), 64, 128, False, 64, False, "bf16")
    lin(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 64, device="cuda"))
    ex, _ = make(moe, (3,), 64, 128, False, 64, False, "bf16")
    y = torch.full((4, 64), 7.0, device="cuda")
    ex(torch.ones(4, 128, device="cuda").bfloat16(), y, torch.full((4,), 2, dtype=torch.int32, device="cuda"))
    assert (y == 7).all() and ex.device_status() == (0, 0)


def test_python_refusals(moe):
    q, s, z, _ = matrix((), 32, 128, 64, True, "bf16", 0)
    lin = moe.Int4Linear(q, s, z, group=64)
    x, y = torch.zeros(4, 128, device="cuda").bfloat16(), torch.zeros(4, 32, device="cuda")
    lin(x, y)
    ids = torch.zeros(2, dtype=torch.int32, device="cuda")
    qe, se, _, _ = matrix((3,), 32, 128, 64, False, "bf16", 0)
    ex = moe.Int4Linear(qe, se, group=64)
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: moe.Int4Linear(q.cpu(), s.cpu(), z.cpu(), group=64), lambda: moe.Int4Linear(q.int(), s, z, group=64), lambda: moe.Int4Linear(q, s, z, group=48),
                lambda: moe.Int4Linear(q, s, z, group=128), lambda: moe.Int4Linear(q, s.half(), z, group=64), lambda: moe.Int4Linear(q, s, z.int(), group=64),
                lambda: moe.Int4Linear(q, s, z[:, :1], group=64), lambda: moe.Int4Linear(q, s, z, group=64, in_features=126), lambda: moe.Int4Linear(q[0], s[0], None, group=64),
                lambda: moe.Int4GatedLinear(q, s, q[:16], s[:16], group=64), lambda: moe.Int4GatedLinear(q, s, q, s, z, None, group=64),
                lambda: moe.Int4GatedLinear(q, s, q, s.float(), group=64), lambda: moe.Int4Linear(q, s, z, group=0),
                lambda: lin(x.float(), y), lambda: lin(x, y.half()), lambda: lin(x[:3], y), lambda: lin(x[:, :64], y), lambda: lin(x, y[:, :16]),
                lambda: lin(x.cpu(), y), lambda: lin(x, y, ids.long()), lambda: lin(x, y, ids[:1]), lambda: lin(x, y, None, tok[:3]),
                lambda: lin(x, y, None, tok.cpu()), lambda: lin(x.t().contiguous().t(), y), lambda: ex(x, y), lambda: ex(x, y, ids)):
        with pytest.raises(moe.MoeError):
            bad()
    lin(x, y, torch.tensor([0, 4], dtype=torch.int32, device="cuda"), tok)


# ------------------------------------------------------------------ together

def ffn64(x, ids, w, mats, first):
    """The routed experts in 64 bits, with h and o rounded to bf16 as they are kept, and the error allowed."""
    gate, up, down = mats
    t, k = ids.shape
    y = torch.zeros(t, down.shape[1], dtype=torch.float64, device="cuda")
    slack = torch.zeros_like(y)
    for e in range(gate.shape[0]):
        tok, slot = (ids == e + first).nonzero(as_tuple=True)
        if not len(tok):
            continue
        h, dh = expect(x[tok], [gate[e], up[e]])
        dh = dh + h.abs() * 2.0 ** -8
        o, wide = h @ down[e].t(), dh @ down[e].abs().t()
        wide = wide + (h.abs() @ down[e].abs().t()) * ((h.shape[1] / 32 + 32) * 2.0 ** -23)
        wide = wide + (o.abs() + wide) * 2.0 ** -8
        ww = w[tok, slot].double()[:, None]
        y.index_add_(0, tok, o * ww)
        slack.index_add_(0, tok, wide * ww.abs() + (o * ww).abs() * (k + 1) * U)
    return y, slack


@pytest.mark.parametrize("t,k,e,first,hidden,inter,yt", [(1, 2, 4, 0, 256, 128, "bf16"), (16, 8, 32, 0, 512, 192, "f32"), (7, 4, 8, 8, 200, 96, "bf16"),
                                                         (300, 4, 8, 2, 520, 260, "bf16"), (2000, 2, 6, 0, 256, 320, "f32")])
def test_sorted_multiplied_and_combined(moe, t, k, e, first, hidden, inter, yt):
    gu, (gate, up) = make(moe, (e,), inter, hidden, True, 64, True, "bf16", 1)
    dn, (down,) = make(moe, (e,), hidden, inter, False, 32, False, "f32", 7)
    ffn = moe.Int4ExpertFfn(gu, dn, k, first)
    g = gen(3)
    x = (torch.randn(t, hidden, generator=g, device="cuda") * 0.1).bfloat16()
    ids = torch.randint(0, e + 2 * first, (t, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand(t, k, generator=g, device="cuda")
    add = torch.randn(t, hidden, generator=g, device="cuda").to(DT[yt])
    y = torch.empty(t, hidden, dtype=DT[yt], device="cuda")
    want, slack = ffn64(x, ids, w, (gate, up, down), first)
    ffn(x, ids, w, y)
    check(y, want, slack)
    y.copy_(add)
    ffn(x, ids, w, y, add=y)
    check(y, want + add.double(), slack + add.double().abs() * (k * U))
    assert gu.device_status() == (0, 0) and dn.device_status() == (0, 0)
    # a captured step goes on with its buffers after other sizes were called
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ffn(x, ids, w, y)
    other = torch.empty(2 * t + 1, hidden, dtype=DT[yt], device="cuda")
    ffn(x[:1].repeat(2 * t + 1, 1), ids[:1].repeat(2 * t + 1, 1), w[:1].repeat(2 * t + 1, 1), other)
    y.zero_()
    graph.replay()
    check(y, want, slack)
    # gradients of the weights through the rows that the step left
    plan, _, o = ffn.buffers(t)
    assert plan.tokens == t
    dy = torch.randn(t, hidden, generator=g, device="cuda").to(DT[yt])
    d_o, d_w = torch.zeros_like(o[:t * k]), torch.empty(t, k, device="cuda")
    plan.combine_grad(dy, o[:t * k], w, d_o, d_w)
    inv = plan.inv_row.long()
    rows = torch.where((inv >= 0)[..., None], o[inv.clamp(min=0)].double(), 0.0)
    prod = rows * dy.double()[:, None]
    assert ((d_w.double() - prod.sum(-1)).abs() <= prod.abs().sum(-1) * (128 * U)).all()
