"""Host-only checks of the dense operators' C ABI: argument errors are found
before anything touches CUDA."""
import ctypes

import pytest

import moe_expert_ffn_02_gb300 as moe


@pytest.fixture(scope="module")
def lib():
    return moe.load(build_if_missing=True)


def norm_args(**over):
    a = moe.MoeRmsnormArgs(rows=2, cols=256, x_type=moe.BF16, res_type=moe.BF16, x=0x1000, ldx=256, res=0x2000,
                           ld_res=256, weight=0x3000, res_out=0x4000, ld_res_out=256, y=0x5000, ldy=256, eps=1e-6)
    a.out = moe.MoeFp8Matrix(0x6000, 0x7000, 256, 4, moe.SCALE_F32, 0)
    for k, v in over.items():
        if k.startswith("out_"):
            setattr(a.out, k[4:], v)
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(cols=32769), 2), (dict(x_type=2), 1), (dict(res_type=7), 1),
    (dict(x_type=moe.F32), 2), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(x=None), 1), (dict(weight=None), 1),
    (dict(res=None), 1), (dict(x=0x1001), 1), (dict(ldx=255), 1), (dict(ld_res=255), 1), (dict(ld_res_out=0), 1),
    (dict(ldy=100), 1), (dict(out_q=None), 1), (dict(out_s=None), 1), (dict(out_ldq=250), 1), (dict(out_ldq=240), 1),
    (dict(out_q=0x6008), 1), (dict(out_lds=0), 1), (dict(out_lds=6), 1), (dict(out_scale_type=1), 1), (dict(out_scale_type=2), 1), (dict(out_s=0x7002), 1),
    (dict(y=None, res_out=None, out_q=None, out_s=None), 1),
])
def test_norm_refuses_bad_arguments(lib, over, code):
    assert lib.moe_add_rmsnorm(ctypes.byref(norm_args(**over)), None) == code
    assert moe.moe_last_error()


def test_norm_of_no_rows_and_null(lib):
    assert lib.moe_add_rmsnorm(ctypes.byref(norm_args(rows=0)), None) == 0
    assert lib.moe_add_rmsnorm(None, None) == 1


@pytest.mark.parametrize("desc,ptrs,code", [
    ((0, 128, 0, 0), (1, 1, 1, 1), 2), ((128, 0, 0, 0), (1, 1, 1, 1), 2), ((1 << 21, 128, 0, 0), (1, 1, 1, 1), 2),
    ((128, 128, 2, 0), (1, 1, 1, 1), 1), ((128, 128, 0, 2), (1, 1, 1, 1), 1), ((128, 128, 0, 0), (0, 1, 1, 1), 1),
    ((128, 128, 0, 0), (1, 0, 1, 1), 1), ((128, 128, 1, 0), (1, 1, 0, 1), 1), ((128, 128, 1, 0), (1, 1, 1, 0), 1),
])
def test_create_refuses_bad_descriptors(lib, desc, ptrs, code):
    d, w = moe.MoeLinearDesc(*desc), moe.MoeLinearWeights(*[0x1000 * p or None for p in ptrs])
    h = ctypes.c_void_p()
    assert lib.moe_linear_create(ctypes.byref(d), ctypes.byref(w), None, ctypes.byref(h)) == code
    assert h.value is None and moe.moe_last_error()


def test_null_handles(lib):
    m = moe.MoeFp8Matrix(0x1000, 0x2000, 256, 4, 0, 0)
    assert lib.moe_linear_forward(None, ctypes.byref(m), 1, 0x1000, 128, 0, None) == 1
    assert lib.moe_gated_linear_forward(None, ctypes.byref(m), 1, ctypes.byref(m), None) == 1
    assert lib.moe_linear_destroy(None) == 1
    assert lib.moe_linear_device_status(None, None, None) == 1
    assert lib.moe_linear_create(None, None, None, None) == 1


def test_wait_limit_of_zero_is_refused(lib):
    assert lib.moe_rmsnorm_set_wait_limit(0) == 1
    assert lib.moe_rmsnorm_set_wait_limit(2_000_000) == 0


def test_null_handles_of_the_test_hooks(lib):
    assert lib.moe_linear_set_wait_limit(None, 1000) == 1
    assert lib.moe_linear_debug_timeout(None) == 1
