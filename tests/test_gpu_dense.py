"""The dense operators on the GPU (residual RMS norm with E4M3 output, FP8
linear and gated projections) against plain 64-bit forms of their definitions.

Tolerances, derived from the arithmetic (u = 2^-24, half an fp32 ulp):

- norm: x + r rounds once (u).  The sum of squares is a sum of at most 64 terms
  per thread and a tree of 10 levels: its relative error is below 80 u, its
  square root halves that, and the reciprocal, the two products and the square
  root add 5 u: 45 u < 3e-6 relative on n.  Outputs add half a step of their type.
- GEMM: a 128-channel partial is four MMAs whose aligned sums lose at most a few
  fp32 units of the largest term; the scaling and the fp32 sum over kt blocks add
  (kt + 2) u: (kt + 16) 2^-23 of the sum of magnitudes.
- codes: half an E4M3 step of the quotient, 2^-4 relative for normal codes and
  2^-10 absolute below them, plus the quotient's own error.
"""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16_HALF = 2.0 ** -8          # half a step of a type with 8 significant bits, relative to the smallest value of a binade
N_REL = 3e-6


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import moe_expert_ffn_02_gb300 as m
    m.load()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, seed, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * scale).to(dtype)


def pad128(v, dim):
    short = -v.shape[dim] % 128
    if not short:
        return v
    shape = list(v.shape)
    shape[dim] = short
    return torch.cat([v, torch.zeros(shape, dtype=v.dtype, device=v.device)], dim)


def scale64(amax, scale):
    s = amax / 448
    if scale == "e8m0":
        s = torch.exp2(torch.ceil(torch.log2(s)))
    return torch.where(amax / 448 < 2.0 ** -126, torch.ones_like(s), s)


def e8m0(s):
    return (torch.log2(s.double()).round() + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def rows_fp8(v, scale):
    """[rows][cols] -> codes and scales [groups][rows], made in 64 bits."""
    g = pad128(v.double(), 1).view(v.shape[0], -1, 128)
    s = scale64(g.abs().amax(-1), scale)
    if scale == "f32":
        s = s.float().double()
    q = (g / s[..., None]).reshape(v.shape[0], -1)[:, :v.shape[1]].float().clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.contiguous(), (s.float().t().contiguous() if scale == "f32" else e8m0(s.t().contiguous()))


def blocks_fp8(w, scale):
    b = pad128(pad128(w.double(), 0), 1)
    b = b.view(b.shape[0] // 128, 128, -1, 128)
    s = scale64(b.abs().amax((1, 3)), scale)
    if scale == "f32":
        s = s.float().double()
    q = (b / s[:, None, :, None]).reshape(b.shape[0] * 128, -1)[:w.shape[0], :w.shape[1]]
    return q.float().clamp(-448, 448).to(torch.float8_e4m3fn).contiguous(), (s.float() if scale == "f32" else e8m0(s))


def wide_rows(q, s):
    return q.double() * s.double().t().repeat_interleave(128, 1)[:, :q.shape[1]]


def wide_blocks(q, s):
    return q.double() * s.double().repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def check_codes(q, s, want, slack, scale):
    """q * s against the 64-bit values `want`, each known to within `slack`."""
    rows, cols = want.shape
    sd = s.double()
    amax = pad128(want.abs(), 1).view(rows, -1, 128).amax(-1).t()
    loose = pad128(slack.expand(rows, cols), 1).view(rows, -1, 128).amax(-1).t()
    if scale == "f32":
        ref = scale64(amax, scale)
        assert ((sd - ref).abs() <= loose / 448 + ref * 2.0 ** -22).all()
    else:
        lo, hi = scale64((amax - loose).clamp_min(0) * (1 - 2.0 ** -22), scale), scale64((amax + loose) * (1 + 2.0 ** -22), scale)
        assert ((sd == lo) | (sd == hi)).all()
    wide = sd.t().repeat_interleave(128, 1)[:, :cols]
    quot = want / wide
    err = (q.double() - quot).abs()
    tol = torch.maximum(quot.abs() * 2.0 ** -4, torch.full_like(quot, 2.0 ** -10)) + slack / wide + quot.abs() * 2.0 ** -22
    assert (err <= tol).all(), float((err - tol).max())


# ------------------------------------------------------------------ norm

def norm64(x, r, w, eps):
    v = x.double() + (r.double() if r is not None else 0)
    return v, v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps) * w.double()


def check_norm(moe, x, r, w, scale, eps=1e-6, in_place=False):
    rows, cols = x.shape
    norm = moe.RmsNorm(w, eps)
    out = moe.Fp8Tensor(rows, cols, scale)
    y = torch.empty_like(x)
    v, n = norm64(x, r, w, eps)
    ro = None if r is None else (r if in_place else torch.empty_like(r))
    norm(x, r, out=out, res_out=ro, y=y)
    if r is not None:
        half = 0 if r.dtype is torch.float32 else BF16_HALF
        assert ((ro.double() - v).abs() <= v.abs() * (half + 2.0 ** -23)).all()
    half = 0 if x.dtype is torch.float32 else BF16_HALF
    assert ((y.double() - n).abs() <= n.abs() * (half + N_REL) + 1e-38).all()
    check_codes(out.q, out.s, n, n.abs() * N_REL, scale)
    return out, y, ro


@pytest.mark.parametrize("types", ["bf16/bf16", "bf16/f32", "f32/f32", "bf16/-", "f32/-"])
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7168), (3, 127), (2, 128), (5, 129), (17, 1000), (4, 7176), (300, 256),
                                       (2, 16384), (1, 32768), (2, 20001)])
def test_norm_against_64_bits(moe, types, scale, rows, cols):
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    tx, tr = types.split("/")
    x = randn((rows, cols), 1, dtype=dt[tx])
    r = None if tr == "-" else randn((rows, cols), 2, 4.0, dt[tr])
    check_norm(moe, x, r, 1 + randn((cols,), 3, 0.2), scale)


@pytest.mark.parametrize("types", ["bf16/bf16", "bf16/f32", "f32/f32", "bf16/-"])
@pytest.mark.parametrize("rows,cols", [(1300, 264), (2500, 7168), (1217, 8), (1900, 4104), (2500, 7001), (5000, 131), (700, 1000), (1500, 999), (1300, 9001), (1500, 16384), (3000, 1001), (1400, 8192)])
def test_norm_of_many_rows(moe, types, rows, cols):
    """Enough rows for the ring form, and sizes around its limits."""
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    tx, tr = types.split("/")
    x = randn((rows, cols), 1, dtype=dt[tx])
    r = None if tr == "-" else randn((rows, cols), 2, 4.0, dt[tr])
    ref_r = None if r is None else r.clone()
    out, y, ro = check_norm(moe, x, r, 1 + randn((cols,), 3, 0.2), "f32")
    if r is not None:        # the same in place
        norm = moe.RmsNorm(1 + randn((cols,), 3, 0.2))
        norm(x, ref_r, res_out=ref_r)
        assert torch.equal(ref_r, ro)
    assert moe.moe_rmsnorm_device_status(torch.cuda.current_stream().cuda_stream) == (0, 0)


@pytest.mark.parametrize("scale", ["f32", "e8m0"])
def test_norm_strides_and_alignment(moe, scale):
    """Rows inside wider, unaligned storage; only the rows' own elements are written."""
    store = randn((9, 517), 4, dtype=torch.bfloat16)
    x, rs = store[:, 3:503], randn((9, 640), 5, dtype=torch.float32)
    w = 1 + randn((501,), 6, 0.2)[1:]
    before = rs.clone()
    check_norm(moe, x, rs[:, 8:508], w, scale, in_place=True)
    keep = torch.ones(640, dtype=torch.bool, device="cuda")
    keep[8:508] = False
    assert torch.equal(rs[:, keep], before[:, keep])
    out = moe.Fp8Tensor(9, 500, scale)
    guard = out.q.as_strided((9, 512), (512, 1)).view(torch.uint8)
    guard.fill_(0xA5)
    moe.RmsNorm(w)(x, out=out)
    assert (guard[:, 500:] == 0xA5).all()


def test_norm_in_place_equals_out_of_place(moe):
    x, r, w = randn((33, 2048), 7, dtype=torch.bfloat16), randn((33, 2048), 8, 3.0, torch.bfloat16), torch.ones(2048, device="cuda")
    norm = moe.RmsNorm(w)
    ro, y = torch.empty_like(r), torch.empty_like(x)
    norm(x, r, res_out=ro, y=y)
    x2, r2 = x.clone(), r.clone()
    norm(x2, r2, res_out=r2, y=x2)
    assert torch.equal(ro, r2) and torch.equal(y, x2)


@pytest.mark.parametrize("scale", ["f32", "e8m0"])
def test_norm_zeros_tiny_values_and_non_numbers(moe, scale):
    cols = 384
    x = randn((6, cols), 9)
    x[0] = 0
    x[1, 128:256] = 0
    x[2] *= 1e-30
    w = torch.ones(cols, device="cuda")
    x[3, 5] = float("nan")
    x[4, 200] = float("inf")
    out, y = moe.Fp8Tensor(6, cols, scale), torch.empty_like(x)
    moe.RmsNorm(w, 0.0)(x[1:2].expand(6, cols).contiguous(), out=out, y=y)          # a zero group: scale 1, zero codes
    assert (out.s.float()[1] == 1).all() and (out.q.float()[:, 128:256] == 0).all()
    moe.RmsNorm(w, 1e-6)(x, out=out, y=y)
    q, s = out.q.float(), out.s.float()
    assert (q[0] == 0).all() and (s[:, 0] == 1).all()
    assert torch.isnan(y[3]).all() and torch.isnan(s[:, 3]).all() and torch.isnan(q[3]).all()
    assert torch.isnan(s[1, 4]) and torch.isnan(y[4, 200]) and (y[4, :128] == 0).all() and (q[4, :128] == 0).all()
    _, n = norm64(x[5:], None, w, 1e-6)
    assert ((y[5:].double() - n).abs() <= n.abs() * N_REL).all()
    tiny = torch.full((1, cols), 2.0 ** -140, device="cuda")                        # amax / 448 has no normal number
    out1 = moe.Fp8Tensor(1, cols, scale)
    moe.RmsNorm(w, 1.0)(tiny, out=out1)
    assert (out1.s.float() == 1).all() and (out1.q.float() == 0).all()


@pytest.mark.parametrize("rows,cols", [(1, 1032), (2500, 1032), (700, 128), (3, 1033), (2500, 1033), (700, 131)])
def test_norm_weight_written_by_the_kernel_before(moe, rows, cols):
    """The kernel ahead on the stream, which lets the norm start early, writes the norm's weight: every form waits for it."""
    k = 33000
    lin = moe.Fp8Linear(*blocks_fp8(randn((cols, k), 11, 0.02), "f32"))
    a = moe.Fp8Tensor.from_parts(*rows_fp8(randn((1, k), 12), "f32"))
    x, weight = randn((rows, cols), 13), torch.empty(1, cols, device="cuda")
    norm, got, want = moe.RmsNorm(weight[0]), torch.empty_like(x), torch.empty_like(x)
    moe.RmsNorm(lin(a, torch.empty_like(weight))[0])(x, y=want)
    for _ in range(3):
        weight.fill_(float("nan"))
        torch.cuda.synchronize()
        lin(a, weight)
        norm(x, y=got)
        assert torch.equal(got, want)


TIMEOUT = (6, 4)               # MOE_ERR_TIMEOUT, MOE_DEV_WAIT_TIMEOUT


@pytest.mark.parametrize("rows,cols,dtype", [(2500, 7168, torch.bfloat16), (2500, 1032, torch.float32), (2500, 7001, torch.bfloat16),
                                             (3000, 9001, torch.bfloat16)])
def test_norm_wait_that_expires(moe, rows, cols, dtype):
    """The wait for one row expires: the call ends with MOE_ERR_TIMEOUT, each row has all of its outputs or, as the residual was in
    place, is as it was, and the next call is right."""
    stream = torch.cuda.current_stream().cuda_stream
    x, r, norm = randn((rows, cols), 14, dtype=dtype), randn((rows, cols), 15, 3.0, dtype), moe.RmsNorm(1 + randn((cols,), 16, 0.2))

    def call():
        res, y, out = r.clone(), torch.full_like(x, 7.0), moe.Fp8Tensor(rows, cols)
        out.q.view(torch.uint8).fill_(0x7F)
        out.s.fill_(-1)
        norm(x, res, out=out, res_out=res, y=y)
        status = moe.moe_rmsnorm_device_status(stream)
        return status, res, y, out.q.view(torch.uint8), out.s.t()

    def rows_equal(a, b):
        return (a == b).all(1)

    status, *want = call()
    assert status == (0, 0)
    moe.moe_rmsnorm_set_wait_limit(5000)
    try:
        moe.moe_rmsnorm_debug_timeout()
        status, *got = call()
    finally:
        moe.moe_rmsnorm_set_wait_limit(2_000_000)
    assert status == TIMEOUT
    done = rows_equal(got[0], want[0])
    assert 0 < int((~done).sum()) < rows // 50               # the row, and those after it in its thread block
    for g, w, untouched in zip(got, want, (r, torch.full_like(x, 7.0), torch.full_like(want[2], 0x7F), torch.full_like(want[3], -1))):
        assert rows_equal(g, w)[done].all() and rows_equal(g, untouched)[~done].all()
    status, *again = call()                                  # read and cleared; fires once
    assert status == (0, 0)
    assert all(torch.equal(g, w) for g, w in zip(again, want))


def test_norm_offsets_past_32_bits(moe):
    cols, ld = 256, 2 ** 31 + 64
    big = torch.empty(ld + cols, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((2, cols), (ld, 1))
    x.copy_(randn((2, cols), 10, dtype=torch.bfloat16))
    check_norm(moe, x.contiguous(), None, torch.ones(cols, device="cuda"), "f32")
    y = torch.empty(2, cols, dtype=torch.bfloat16, device="cuda")
    z = torch.empty_like(y)
    moe.RmsNorm(torch.ones(cols, device="cuda"))(x, y=y)
    moe.RmsNorm(torch.ones(cols, device="cuda"))(x.contiguous(), y=z)
    assert torch.equal(y, z)


def test_norm_of_as_many_rows_as_a_count_holds(moe):
    rows = 2 ** 31 - 1
    x = torch.full((rows, 1), 2.0, dtype=torch.bfloat16, device="cuda")
    x[-300:] = randn((300, 1), 17, dtype=torch.bfloat16)
    y = torch.zeros_like(x)
    moe.RmsNorm(torch.full((1,), 3.0, device="cuda"))(x, y=y)
    assert (y[:-300] == 3).all()
    _, n = norm64(x[-300:], None, torch.full((1,), 3.0, device="cuda"), 1e-6)
    assert ((y[-300:].double() - n).abs() <= n.abs() * (BF16_HALF + N_REL)).all()


# ------------------------------------------------------------------ projections

def product64(aq, a_s, wq, w_s):
    a, w = wide_rows(aq, a_s), wide_blocks(wq, w_s)
    kt = (aq.shape[1] + 127) // 128
    return a @ w.t(), (a.abs() @ w.abs().t()) * (kt + 16) * 2.0 ** -23


def check_linear(moe, m, k, n, scale, dtype, seed=20):
    aq, a_s = rows_fp8(randn((m, k), seed), scale)
    wq, w_s = blocks_fp8(randn((n, k), seed + 1, 0.02), scale)
    lin = moe.Fp8Linear(wq, w_s)
    y = lin(moe.Fp8Tensor.from_parts(aq, a_s), torch.full((m, n), float("nan"), dtype=dtype, device="cuda"))
    want, tol = product64(aq, a_s, wq, w_s)
    half = 0 if dtype is torch.float32 else BF16_HALF
    err = (y.double() - want).abs()
    assert (err <= tol + want.abs() * half + tol * half).all(), float((err - tol).max())
    assert lin.device_status() == (0, 0)
    return lin, y


ODD = [(1, 1, 1), (1, 128, 16), (2, 100, 17), (7, 127, 127), (8, 129, 128), (9, 256, 129), (31, 1040, 1001), (33, 385, 64),
       (64, 640, 250), (65, 1000, 96), (127, 513, 333), (128, 128, 256), (129, 1153, 257), (300, 1992, 1001), (1, 7168, 2048),
       (16, 2048, 7168), (1000, 256, 2500), (70, 7168, 300), (130, 3000, 128), (200, 2100, 999)]


@pytest.mark.parametrize("m,k,n", ODD)
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_against_64_bits(moe, m, k, n, scale, dtype):
    check_linear(moe, m, k, n, scale, dtype)


@pytest.mark.parametrize("m,k,n", [(3, 70000, 20), (70, 8300, 40), (2, 530000, 16), (40, 33000, 130)])
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
def test_linear_of_long_rows(moe, m, k, n, scale):
    """K past what one chain of scaled MMAs, or one CTA's share of the few-token form, may hold."""
    check_linear(moe, m, k, n, scale, torch.float32)


# few tokens, chains of 64 K blocks in each of eight ranges; many tokens, one chain; ranges of the many-token form
@pytest.mark.parametrize("m,k,n", [(3, 65536, 40), (40, 65300, 130), (2100, 8192, 2100), (1500, 8192, 1500), (100, 8192, 150)])
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("signs", ["one", "cancel"])
def test_linear_sums_of_one_sign_and_sums_that_cancel(moe, m, k, n, scale, signs):
    """Truncation shows where every term has one sign, or a large partial sum is taken back later.

    fp32 scales: rounded sums, (kt + 16) 2^-23 of the magnitudes as above.  e8m0: each of a chain's 4 kt MMAs, at most 256,
    may lose one unit of the last place of its running sum, which the magnitudes bound, and the ranges' sums are rounded."""
    kt = (k + 127) // 128
    half = kt // 2 * 128
    a, w = randn((m, k), 25).abs(), randn((n, k), 26, 0.02).abs()
    if signs == "cancel":
        a[:, half:2 * half] = a[:, :half]
        w[:, half:2 * half] = -w[:, :half] * (1 + randn((n, half), 27, 0.1))
    aq, a_s = rows_fp8(a, scale)
    wq, w_s = blocks_fp8(w, scale)
    y = moe.Fp8Linear(wq, w_s)(moe.Fp8Tensor.from_parts(aq, a_s), torch.empty(m, n, device="cuda"))
    A, W = wide_rows(aq, a_s), wide_blocks(wq, w_s)
    magnitude = A.abs() @ W.abs().t()
    tol = magnitude * 2.0 ** -23 * (kt + 16 + (4 * min(kt, 64) if scale == "e8m0" else 0))
    if signs == "cancel":
        assert ((A @ W.t()).abs() < 0.1 * magnitude).all()
    assert ((y.double() - A @ W.t()).abs() <= tol).all()


def check_gated(moe, m, k, n, scale, seed=30):
    aq, a_s = rows_fp8(randn((m, k), seed), scale)
    g, u = blocks_fp8(randn((n, k), seed + 1, 0.05), scale), blocks_fp8(randn((n, k), seed + 2, 0.05), scale)
    lin = moe.Fp8GatedLinear(*g, *u)
    h = moe.Fp8Tensor(m, n, scale)
    h.q.view(torch.uint8).fill_(0x7F)
    lin(moe.Fp8Tensor.from_parts(aq, a_s), h)
    gv, eg = product64(aq, a_s, *g)
    uv, eu = product64(aq, a_s, *u)
    silu = gv / (1 + torch.exp(-gv))
    want = silu * uv
    # SiLU's slope is at most 1.1; its fast exponential and quotient lose a few ulp, growing with |g|
    slack = 1.1 * eg * (uv.abs() + eu) + silu.abs() * eu + want.abs() * (4 + gv.abs()) * 2.0 ** -22
    check_codes(h.q, h.s, want, slack, scale)
    assert lin.device_status() == (0, 0)
    return lin, h


@pytest.mark.parametrize("m,k,n", [(1, 128, 1), (1, 7168, 2048), (2, 100, 8), (7, 129, 17), (9, 640, 129), (33, 1040, 1000),
                                   (64, 384, 250), (65, 257, 136), (127, 513, 333), (128, 256, 256), (129, 1153, 200),
                                   (300, 1992, 1001), (1000, 256, 2500), (20, 33100, 50), (66, 8300, 136), (70, 7168, 300), (130, 3000, 128), (200, 2100, 999)])
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
def test_gated_against_64_bits(moe, m, k, n, scale):
    check_gated(moe, m, k, n, scale)


@pytest.mark.parametrize("m", [2, 40])
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
def test_gated_of_few_tokens_and_rows_too_long_for_their_form(moe, m, scale):
    """More than 4 x 512 K blocks: the form of many tokens takes the call."""
    check_gated(moe, m, 263000, 24, scale)


@pytest.mark.parametrize("scale", ["f32", "e8m0"])
def test_rows_do_not_depend_on_the_batch(moe, scale):
    """Up to 64 tokens, tile widths follow the batch size but a token's bits do
    not.  (Larger batches may split K by their size.)"""
    m, k, n = 64, 1160, 1400
    aq, a_s = rows_fp8(randn((m, k), 40), scale)
    w, u = blocks_fp8(randn((n, k), 41, 0.05), scale), blocks_fp8(randn((n, k), 42, 0.05), scale)
    lin, gated = moe.Fp8Linear(*w), moe.Fp8GatedLinear(*w, *u)

    def run(lo, hi):
        s = a_s.view(torch.uint8 if scale == "e8m0" else torch.float32)[:, lo:hi].contiguous().view(a_s.dtype)
        part = moe.Fp8Tensor.from_parts(aq[lo:hi].clone(), s)
        h = gated(part, moe.Fp8Tensor(hi - lo, n, scale))
        return (lin(part, torch.empty(hi - lo, n, dtype=torch.float32, device="cuda")), h.q.view(torch.uint8),
                h.s.float().t())

    ref = run(0, m)
    for lo, hi in ((0, 1), (5, 14), (20, 45), (10, 64), (30, 62)):
        for got, want in zip(run(lo, hi), ref):
            assert torch.equal(got, want[lo:hi])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_output_strides(moe, dtype):
    """y inside wider storage, at aligned and odd offsets and strides; nothing beside it is written."""
    m, k, n = 70, 300, 200
    aq, a_s = rows_fp8(randn((m, k), 50), "f32")
    lin = moe.Fp8Linear(*blocks_fp8(randn((n, k), 51, 0.05), "f32"))
    a = moe.Fp8Tensor.from_parts(aq, a_s)
    ref = lin(a, torch.empty(m, n, dtype=dtype, device="cuda"))
    for width, off in ((256, 0), (256, 8), (259, 0), (261, 3), (208, 4)):
        store = torch.full((m, width), 7.0, dtype=dtype, device="cuda")
        y = lin(a, store[:, off:off + n])
        assert torch.equal(y, ref)
        keep = torch.ones(width, dtype=torch.bool, device="cuda")
        keep[off:off + n] = False
        assert (store[:, keep] == 7).all()


@pytest.mark.parametrize("m,k,n", [(2333, 640, 4040), (1921, 1100, 5000)])
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_of_many_rows(moe, m, k, n, scale, dtype):
    """Several tiles per SM, the last ones ending inside the output: against 64 bits, and the same bits in wider storage
    with nothing beside them written."""
    lin, ref = check_linear(moe, m, k, n, scale, dtype, seed=56)
    aq, a_s = rows_fp8(randn((m, k), 56), scale)
    a = moe.Fp8Tensor.from_parts(aq, a_s)
    for width, off in ((n + 24, 8), (n + 3, 1), (n + 6, 1), (n + 6, 2)):
        store = torch.full((m + 2, width), 7.0, dtype=dtype, device="cuda")
        assert torch.equal(lin(a, store[1:m + 1, off:off + n]), ref)
        keep = torch.ones(m + 2, width, dtype=torch.bool, device="cuda")
        keep[1:m + 1, off:off + n] = False
        assert (store[keep] == 7).all()


def test_linear_offsets_past_32_bits(moe):
    m, k, n = 3, 256, 130
    aq, a_s = rows_fp8(randn((m, k), 60), "f32")
    lin = moe.Fp8Linear(*blocks_fp8(randn((n, k), 61, 0.05), "f32"))
    ref = lin(moe.Fp8Tensor.from_parts(aq, a_s), torch.empty(m, n, dtype=torch.bfloat16, device="cuda"))
    ld = 2 ** 31 + 128
    big = torch.empty(2 * ld + k, dtype=torch.uint8, device="cuda")
    wide = big.as_strided((m, k), (ld, 1))
    wide.copy_(aq.view(torch.uint8))
    y = lin(moe.Fp8Tensor.from_parts(wide.view(torch.float8_e4m3fn), a_s), torch.empty(m, n, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(y, ref)
    del big, wide
    out = torch.empty(2 * (2 ** 31 + 3) + n, dtype=torch.bfloat16, device="cuda").as_strided((m, n), (2 ** 31 + 3, 1))
    assert torch.equal(lin(moe.Fp8Tensor.from_parts(aq, a_s), out), ref)


def test_more_rows_than_tiles_can_count_are_refused(moe):
    w = blocks_fp8(randn((16, 16), 62), "f32")
    m = moe.MoeFp8Matrix(0x10000, 0x20000, 16, 2 ** 31, moe.SCALE_F32, 0)
    for call, lin in ((lambda h: moe.moe_linear_forward(h, m, 2 ** 31 - 255, 0x30000, 16, moe.BF16), moe.Fp8Linear(*w)),
                      (lambda h: moe.moe_gated_linear_forward(h, m, 2 ** 31 - 255, m), moe.Fp8GatedLinear(*w, *w))):
        with pytest.raises(moe.MoeError) as e:
            call(lin.handle)
        assert e.value.status == 2


@pytest.mark.parametrize("m", [1, 40, 200])
def test_non_numbers_stay_in_their_row_and_column(moe, m):
    k, n = 300, 260
    aq, a_s = rows_fp8(randn((m, k), 70), "f32")
    wq, w_s = blocks_fp8(randn((n, k), 71, 0.05), "f32")
    aq.view(torch.uint8)[m // 2, 299] = 0x7F
    wq.view(torch.uint8)[77, 3] = 0xFF
    y = moe.Fp8Linear(wq, w_s)(moe.Fp8Tensor.from_parts(aq, a_s), torch.empty(m, n, dtype=torch.float32, device="cuda"))
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[m // 2] = True
    bad[:, 77] = True
    assert torch.equal(torch.isnan(y), bad)
    h = moe.Fp8GatedLinear(wq, w_s, wq, w_s)(moe.Fp8Tensor.from_parts(aq, a_s), moe.Fp8Tensor(m, n))
    s = torch.isnan(h.s)
    assert s[0].all() and s[:, m // 2].all() and int(s.sum()) == m + h.s.shape[0] - 1      # feature 77's group, row m // 2


@pytest.mark.parametrize("m,k,n", [(1, 300, 260), (40, 300, 260), (200, 300, 260), (600, 1000, 1500), (3, 70000, 40), (70, 9000, 300)])
@pytest.mark.parametrize("what", ["code", "weight", "scale", "weight scale"])
def test_non_numbers_with_e8m0_scales(moe, m, k, n, what):
    """A NaN code or scale (255) reaches its row, its column or its scale block's 128 columns, and nothing else."""
    aq, a_s = rows_fp8(randn((m, k), 72), "e8m0")
    wq, w_s = blocks_fp8(randn((n, k), 73, 0.05), "e8m0")
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    if what == "code":
        aq.view(torch.uint8)[m // 2, k - 1] = 0x7F
        bad[m // 2] = True
    elif what == "weight":
        wq.view(torch.uint8)[n - 3, k // 2] = 0xFF
        bad[:, n - 3] = True
    elif what == "scale":
        a_s.view(torch.uint8)[k // 256, m // 2] = 255
        bad[m // 2] = True
    else:
        w_s.view(torch.uint8)[-1, k // 256] = 255
        bad[:, (n - 1) // 128 * 128:] = True
    a = moe.Fp8Tensor.from_parts(aq, a_s)
    y = moe.Fp8Linear(wq, w_s)(a, torch.empty(m, n, dtype=torch.float32, device="cuda"))
    assert torch.equal(torch.isnan(y), bad)
    h = moe.Fp8GatedLinear(wq, w_s, wq, w_s)(a, moe.Fp8Tensor(m, n, "e8m0"))
    groups = pad128(bad, 1).view(m, -1, 128).any(-1)
    assert torch.equal(torch.isnan(h.s.float()).t(), groups)
    assert torch.equal(torch.isnan(h.q.float()), groups.repeat_interleave(128, 1)[:, :n])


@pytest.mark.parametrize("m", [2, 200])
def test_infinite_results_of_the_gated_projection(moe, m):
    """An infinite h: its group's scale is infinite (e8m0: NaN), its own code NaN; finite values beside it become 0 * infinity."""
    k, n = 128, 200
    for scale in ("f32", "e8m0"):
        aq, a_s = rows_fp8(torch.ones(m, k, device="cuda"), scale)
        w, big = torch.full((n, k), 2.0 ** -10, device="cuda"), torch.full((n, k), 2.0 ** 118, device="cuda")
        big[1:] = 2.0 ** 100
        aq = (aq.float() * 0 + 448).to(torch.float8_e4m3fn)
        a = moe.Fp8Tensor.from_parts(aq, (a_s.float() * 0 + 1).to(a_s.dtype) if scale == "f32" else e8m0(torch.ones_like(a_s.float())))
        h = moe.Fp8GatedLinear(*blocks_fp8(w, scale), *blocks_fp8(big, scale))(a, moe.Fp8Tensor(m, n, scale))
        s, q = h.s.float(), h.q.float()
        assert torch.isnan(q[:, 0]).all() and torch.isfinite(s[1]).all() and torch.isfinite(q[:, 128:]).all()
        if scale == "f32":
            assert torch.isinf(s[0]).all() and (q[:, 1:128] == 0).all()
        else:
            assert torch.isnan(s[0]).all() and torch.isnan(q[:, :128]).all()


def test_no_rows_is_a_no_op(moe):
    a, w = moe.Fp8Tensor(0, 256), blocks_fp8(randn((128, 256), 80), "f32")
    assert moe.Fp8Linear(*w)(a, torch.empty(0, 128, device="cuda")).shape == (0, 128)
    moe.Fp8GatedLinear(*w, *w)(a, moe.Fp8Tensor(0, 128))
    moe.RmsNorm(torch.ones(256, device="cuda"))(torch.empty(0, 256, device="cuda"), out=a)


def block(moe, scale="f32", h=512, inner=1024):
    norm = moe.RmsNorm(1 + randn((h,), 90, 0.2))
    g, u = blocks_fp8(randn((inner, h), 91, 0.04), scale), blocks_fp8(randn((inner, h), 92, 0.04), scale)
    d = blocks_fp8(randn((h, inner), 93, 0.04), scale)
    return moe.DenseFfn(norm, moe.Fp8GatedLinear(*g, *u), moe.Fp8Linear(*d)), (g, u, d)


@pytest.mark.parametrize("scale", ["f32", "e8m0"])
@pytest.mark.parametrize("rows", [1, 50, 300])
def test_the_operators_together(moe, scale, rows):
    """Norm, gated and plain projection as one pre-norm FFN, each on what the one before it wrote."""
    ffn, (g, u, d) = block(moe, scale)
    x, r = randn((rows, 512), 94, dtype=torch.bfloat16), randn((rows, 512), 95, 2.0, torch.bfloat16)
    v, n = norm64(x, r, ffn.norm.weight, 1e-6)
    y = ffn(x, r, torch.empty(rows, 512, dtype=torch.float32, device="cuda"))
    a, h = ffn.buffers(rows)
    check_codes(a.q, a.s, n, n.abs() * N_REL, scale)
    want, tol = product64(h.q, h.s, *d)
    assert ((y.double() - want).abs() <= tol).all()
    gv, uv = n @ wide_blocks(*g).t(), n @ wide_blocks(*u).t()
    exact = (gv / (1 + torch.exp(-gv)) * uv) @ wide_blocks(*d).t()
    # two quantisations of relative step 2^-4: errors of about 3 % each, independent over hundreds of terms
    assert torch.linalg.norm(y.double() - exact) <= 0.1 * torch.linalg.norm(exact)


def test_a_graph_outlives_calls_of_other_sizes(moe):
    """A captured call of the dense FFN keeps its buffers when the same object is called with more rows."""
    ffn, _ = block(moe)
    x, res = randn((5, 512), 94, dtype=torch.bfloat16), randn((5, 512), 95, dtype=torch.bfloat16)
    start, y = res.clone(), torch.empty(5, 512, dtype=torch.bfloat16, device="cuda")
    want = ffn(x, res, y).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ffn(x, res, y)
    for rows in (300, 6, 40):
        big = randn((rows, 512), 96, dtype=torch.bfloat16)
        ffn(big, big.clone(), torch.empty_like(big))
        junk = [torch.full((rows, 1024), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(8)]
        res.copy_(start)
        y.zero_()
        g.replay()
        assert torch.equal(y, want)
        del junk


def test_another_stream_and_a_graph(moe):
    """Work goes to the current stream, in order with it, and can be captured."""
    ffn, _ = block(moe)
    x, r = randn((24, 512), 96, dtype=torch.bfloat16), randn((24, 512), 97, 2.0, torch.bfloat16)
    ref_r = r.clone()
    ref = ffn(x, ref_r, torch.empty(24, 512, dtype=torch.bfloat16, device="cuda"))
    side = torch.cuda.Stream()
    xs, rs = torch.zeros_like(x), torch.zeros_like(r)
    y = torch.zeros_like(ref)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        xs.copy_(x)
        rs.copy_(r)
        ffn(xs, rs, y)
    side.synchronize()
    assert torch.equal(y, ref) and torch.equal(rs, ref_r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ffn(xs, rs, y)
    for _ in range(2):
        xs.copy_(x)
        rs.copy_(r)
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and torch.equal(rs, ref_r)


def test_a_dropped_dense_ffn_keeps_its_buffers_for_another_stream(moe):
    """Made on one stream, called on another and dropped while that one still has its kernels queued."""
    first, _ = block(moe)
    ffn = moe.DenseFfn(first.norm, first.gate_up, first.down)       # the weights live on
    x, r = randn((300, 512), 96, dtype=torch.bfloat16), randn((300, 512), 97, 2.0, torch.bfloat16)
    y = torch.zeros(300, 512, dtype=torch.bfloat16, device="cuda")
    want = ffn(x, r.clone(), torch.empty_like(y))
    side, pieces = torch.cuda.Stream(), [t for b in ffn._store[512] for t in (b.q, b.s)]
    held = {t.untyped_storage().data_ptr(): t.untyped_storage().nbytes() for t in pieces}
    del pieces
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        ffn(x, r, y)
    del ffn
    new = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in held.values() for _ in range(8)]
    assert not held.keys() & {t.data_ptr() for t in new}
    assert not side.query()                                         # or the buffers were free by right
    side.synchronize()
    assert torch.equal(y, want)


def test_repeated_calls_give_the_same_bits(moe):
    lin, y = check_linear(moe, 150, 1000, 900, "f32", torch.float32)
    aq, a_s = rows_fp8(randn((150, 1000), 20), "f32")
    a = moe.Fp8Tensor.from_parts(aq, a_s)
    for _ in range(5):
        assert torch.equal(lin(a, torch.empty_like(y)), y)


# ------------------------------------------------------------------ waits that expire

def check_expired(moe, lin, call):
    """call() runs a forward into buffers filled beforehand and returns its outputs, rows first.  With the last products of one
    tile left out it ends with MOE_ERR_TIMEOUT, every element is right or as it was, and the next call is right."""
    want = call()
    assert lin.device_status() == (0, 0)
    moe.moe_linear_set_wait_limit(lin.handle, 20_000)
    try:
        moe.moe_linear_debug_timeout(lin.handle)
        got = call()
        assert lin.device_status() == TIMEOUT
    finally:
        moe.moe_linear_set_wait_limit(lin.handle, 2_000_000)
    again = call()                                           # read and cleared; fires once
    assert lin.device_status() == (0, 0)
    assert all(torch.equal(g, w) for g, w in zip(again, want))
    return got, want


def expired_linear(moe, m, k, n, scale, dtype=torch.float32):
    lin = moe.Fp8Linear(*blocks_fp8(randn((n, k), 111, 0.02), scale))
    a = moe.Fp8Tensor.from_parts(*rows_fp8(randn((m, k), 110), scale))
    (got,), (want,) = check_expired(moe, lin, lambda: [lin(a, torch.full((m, n), 7.0, dtype=dtype, device="cuda"))])
    left = got == 7
    assert torch.equal(torch.where(left, want, got), want)
    return left


# tiles of 256, 80, 48 and 16 weight rows in the fp32-scale form, 256 and 128 in the other
@pytest.mark.parametrize("m,k,n,scale", [(1921, 1100, 5000, "f32"), (700, 1000, 2000, "f32"), (777, 1992, 1001, "f32"),
                                         (65, 1000, 96, "f32"), (1921, 1100, 5000, "e8m0"), (1500, 4000, 1500, "e8m0")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_wait_that_expires(moe, m, k, n, scale, dtype):
    left = expired_linear(moe, m, k, n, scale, dtype)
    assert left.any() and not left.all()


def expired_gated(moe, m, k, n, scale):
    """The rows' groups that were left out, [m][groups]; a group is right or left out as a whole, codes and scale."""
    lin = moe.Fp8GatedLinear(*blocks_fp8(randn((n, k), 121, 0.05), scale), *blocks_fp8(randn((n, k), 122, 0.05), scale))
    a = moe.Fp8Tensor.from_parts(*rows_fp8(randn((m, k), 120), scale))

    def call():
        h = moe.Fp8Tensor(m, n, scale)
        h.q.view(torch.uint8).fill_(0x7F)
        s = h.s.view(torch.uint8 if scale == "e8m0" else torch.float32)
        s.fill_(3)
        lin(a, h)
        return pad128(h.q.view(torch.uint8), 1).view(m, -1, 128), s.t()

    (gq, gs), (wq, ws) = check_expired(moe, lin, call)
    untouched = pad128(torch.full((m, n), 0x7F, dtype=torch.uint8, device="cuda"), 1).view(gq.shape)
    left = (gq == untouched).all(-1) & (gs == 3)
    assert ((gq == wq).all(-1) & (gs == ws))[~left].all()
    return left


# one CTA a tile, four, and eight; few and many K blocks
@pytest.mark.parametrize("m,k,n", [(16, 500, 4000), (40, 7168, 2048), (1, 7168, 300), (64, 33000, 130), (5, 70000, 40)])
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
def test_few_token_linear_wait_that_expires(moe, m, k, n, scale):
    left = expired_linear(moe, m, k, n, scale)
    assert left.any() and not left.all()


@pytest.mark.parametrize("m,k,n", [(5, 1000, 20000), (3, 500, 300), (64, 7168, 2048), (20, 33100, 50)])
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
def test_few_token_gated_wait_that_expires(moe, m, k, n, scale):
    left = expired_gated(moe, m, k, n, scale)
    assert left.any() and not left[:, 1:].any()              # the first unit's features only


# one CTA a unit, two and four, with fp32 scales; one and two with the tensor core's own scaling
@pytest.mark.parametrize("m,k,n,scale", [(3000, 1000, 2048, "f32"), (1000, 1000, 1000, "f32"), (300, 1992, 1001, "f32"),
                                         (3000, 1000, 2048, "e8m0"), (1000, 1000, 1000, "e8m0")])
def test_gated_wait_that_expires(moe, m, k, n, scale):
    left = expired_gated(moe, m, k, n, scale)
    assert left[:128, 0].all() and not left.all()            # the whole first unit


@pytest.mark.parametrize("gated,m,k,n,scale", [(False, 300, 1992, 1001, "f32"), (False, 70, 7168, 300, "f32"), (False, 128, 7168, 7168, "f32"),
                                               (False, 70, 7168, 300, "e8m0"), (False, 1024, 4000, 1024, "e8m0"),
                                               (True, 70, 7168, 300, "f32"), (True, 300, 7168, 1400, "f32"), (True, 70, 7168, 300, "e8m0")])
def test_joined_ranges_wait_that_expires(moe, gated, m, k, n, scale):
    """K split over two, four or eight CTAs: a range that was not finished keeps the whole tile from being joined."""
    left = expired_gated(moe, m, k, n, scale)[:, 0] if gated else expired_linear(moe, m, k, n, scale)[:, 0]
    assert left[:128].all() and not left[128:].any()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m", [3, 200])
@pytest.mark.parametrize("scale", ["f32", "e8m0"])
def test_limit_counts_from_the_end_of_the_kernel_before(moe, gated, m, scale):
    """A call that starts on SMs which a long projection ahead of it (some 250 us) leaves idle, with a limit of 120 us."""
    k = 1 << 20
    ahead = moe.Fp8Linear(*blocks_fp8(randn((16, k), 131, 0.02), "f32"))
    a0, y0 = moe.Fp8Tensor.from_parts(*rows_fp8(randn((1, k), 130), "f32")), torch.empty(1, 16, device="cuda")
    w = blocks_fp8(randn((600, 1000), 132, 0.02), scale)
    lin = moe.Fp8GatedLinear(*w, *w) if gated else moe.Fp8Linear(*w)
    a = moe.Fp8Tensor.from_parts(*rows_fp8(randn((m, 1000), 133), scale))
    y = moe.Fp8Tensor(m, 600, scale) if gated else torch.empty(m, 600, device="cuda")
    moe.moe_linear_set_wait_limit(lin.handle, 120)
    for _ in range(3):
        ahead(a0, y0)
        lin(a, y)
        assert lin.device_status() == (0, 0)


# ------------------------------------------------------------------ refusals

def test_refusals(moe):
    w = blocks_fp8(randn((128, 256), 100), "f32")
    lin, gated = moe.Fp8Linear(*w), moe.Fp8GatedLinear(*w, *w)
    a, y = moe.Fp8Tensor(4, 256), torch.empty(4, 128, device="cuda")
    norm = moe.RmsNorm(torch.ones(256, device="cuda"))
    x = torch.zeros(4, 256, device="cuda")

    def refused(fn, code=1):
        with pytest.raises(moe.MoeError) as e:
            fn()
        assert e.value.status == code
    refused(lambda: lin(moe.Fp8Tensor(4, 256, "e8m0"), y))
    refused(lambda: lin(moe.Fp8Tensor(4, 128), y))
    refused(lambda: lin(a, torch.empty(4, 127, device="cuda")))
    refused(lambda: lin(a, torch.empty(4, 128, dtype=torch.float16, device="cuda")))
    refused(lambda: lin(a, torch.empty(128, 4, device="cuda").t()))
    refused(lambda: lin(a, torch.empty(4, 128)))
    refused(lambda: gated(a, moe.Fp8Tensor(3, 128)))
    refused(lambda: gated(a, moe.Fp8Tensor(4, 128, "e8m0")))
    refused(lambda: norm(x, out=moe.Fp8Tensor(4, 128)))
    refused(lambda: norm(x))
    refused(lambda: norm(x, res_out=x))
    refused(lambda: norm(x, x.bfloat16(), y=x), 2)
    refused(lambda: norm(x.half(), y=x.half()))
    refused(lambda: norm(x, y=torch.empty(4, 256, dtype=torch.bfloat16, device="cuda")))
    refused(lambda: moe.Fp8Linear(w[0], w[1][:, :1]))
    refused(lambda: moe.Fp8Tensor(4, 256, "bf16"))
    refused(lambda: moe.moe_linear_forward(gated.handle, a.matrix, 4, y.data_ptr(), 128, moe.F32))
    refused(lambda: moe.moe_gated_linear_forward(lin.handle, a.matrix, 4, a.matrix))
    refused(lambda: moe.moe_linear_forward(lin.handle, a.matrix, -1, y.data_ptr(), 128, moe.F32))
    refused(lambda: moe.moe_linear_forward(lin.handle, a.matrix, 4, y.data_ptr(), 127, moe.F32))
    refused(lambda: moe.moe_linear_forward(lin.handle, a.matrix, 4, y.data_ptr() + 2, 128, moe.F32))
    odd = moe.MoeFp8Matrix(a.q.data_ptr(), a.s.data_ptr(), 264, 4, 0, 0)
    refused(lambda: moe.moe_linear_forward(lin.handle, odd, 4, y.data_ptr(), 128, moe.F32))
    short = moe.MoeFp8Matrix(a.q.data_ptr(), a.s.data_ptr(), 256, 0, 0, 0)
    ragged = moe.MoeFp8Matrix(a.q.data_ptr(), a.s.data_ptr(), 256, 5, 0, 0)
    refused(lambda: moe.moe_linear_forward(lin.handle, ragged, 4, y.data_ptr(), 128, moe.F32))
    refused(lambda: moe.moe_linear_forward(lin.handle, short, 4, y.data_ptr(), 128, moe.F32))
    assert lin.device_status() == (0, 0) and gated.device_status() == (0, 0)
    lin(a, y)          # a refused call leaves the handle usable


def test_a_refused_dense_ffn_leaves_the_residual(moe):
    ffn, _ = block(moe)
    x, r = randn((4, 512), 94, dtype=torch.bfloat16), randn((4, 512), 95, dtype=torch.bfloat16)
    before, y = r.clone(), torch.empty(4, 512, device="cuda")
    for args in ((x, r, y[:3]), (x, r, y[:, :500]), (x, r, y.half()), (x, r, y.cpu()), (x, r, y[:1].expand(4, 512)), (x, None, y),
                 (x, r[:3], y), (x.half(), r, y), (x[:, :500], r, y), (x.float(), r, y), (x, r, y.t().contiguous().t())):
        with pytest.raises(moe.MoeError):
            ffn(*args)
        torch.cuda.synchronize()
        assert torch.equal(r, before)
    ffn(x, r, y)
    assert not torch.equal(r, before)


@pytest.mark.parametrize("tokens", [8, 100])
def test_the_example_runs(moe, tokens):
    """The dense FFN and the expert layer in one captured step; the script checks its residual stream itself."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "transformer_ffn.py"), "--tokens", str(tokens), "--steps", "3"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "us a step" in r.stdout


def test_a_failed_call_leaves_no_error_behind(moe):
    """Weights that do not fit the device are refused with a CUDA error; the next launches do not inherit it."""
    d, h = moe.MoeLinearDesc(1 << 20, 1 << 20, 1, 0), ctypes.c_void_p()        # 2 TB; refused before the pointers are read
    w = moe.MoeLinearWeights(*[0x10000 * (i + 1) for i in range(4)])
    assert moe.load().moe_linear_create(ctypes.byref(d), ctypes.byref(w), None, ctypes.byref(h)) == 4 and h.value is None
    assert "out of memory" in moe.moe_last_error()
    x = torch.ones(300, device="cuda") + 1                                     # torch checks the last error after its launches
    assert float(x.sum()) == 600
    check_linear(moe, 5, 300, 40, "f32", torch.float32)
