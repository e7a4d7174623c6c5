"""Host-only checks of the C ABI around experts outside the fused layer:
argument errors are found before anything touches CUDA."""
import ctypes

import pytest

import moe_expert_ffn_02_gb300 as moe


@pytest.fixture(scope="module")
def lib():
    return moe.load(build_if_missing=True)


def with_(cls, base, over):
    return cls(**{**base, **over})


DISPATCH = dict(tokens=4, top_k=2, n_experts=8, first_expert=0, ids=0x1000, expert_offsets=0x2000, sorted_token=0x3000, inv_row=0x4000,
                x=0x5000, ldx=64, rows=0x6000, ld_rows=64, cols=64, n_rows=8, x_type=moe.BF16)
COMBINE = dict(tokens=4, top_k=2, cols=64, n_rows=8, o_type=moe.BF16, y_type=moe.F32, inv_row=0x1000, w=0x2000, o=0x3000, ldo=64,
               add=0x4000, ld_add=64, y=0x5000, ldy=64)
GRAD = dict(tokens=4, top_k=2, cols=64, n_rows=8, o_type=moe.BF16, y_type=moe.F32, inv_row=0x1000, w=0x2000, dy=0x3000, ld_dy=64,
            o=0x4000, ldo=64, d_o=0x5000, ld_d_o=64, d_w=0x6000)
COUNTS = [(dict(tokens=-1), 1), (dict(top_k=0), 1), (dict(top_k=33), 2), (dict(tokens=1 << 27, top_k=32), 2), (dict(cols=0), 1),
          (dict(cols=(1 << 20) + 1), 2), (dict(n_rows=-1), 1)]


@pytest.mark.parametrize("over,code", COUNTS + [
    (dict(n_experts=0), 1), (dict(n_experts=1025), 2), (dict(first_expert=-1), 1), (dict(first_expert=2 ** 31 - 4), 1), (dict(ids=None, x=None), 1),
    (dict(x_type=2), 1), (dict(x=0x5001), 1), (dict(ldx=63), 1), (dict(rows=None), 1), (dict(rows=0x6001), 1), (dict(ld_rows=0), 1),
    (dict(expert_offsets=None), 1), (dict(expert_offsets=0x2002), 1), (dict(ids=0x1001), 1), (dict(sorted_token=None), 1), (dict(inv_row=None), 1),
    (dict(tokens=600), 1),
])
def test_dispatch_refuses(lib, over, code):
    assert lib.moe_dispatch(ctypes.byref(with_(moe.MoeDispatchArgs, DISPATCH, over)), None, 0, None) == code
    assert moe.moe_last_error()


def test_dispatch_workspace(lib):
    assert moe.moe_dispatch_workspace_bytes(512, 2, 8) == 0
    a = with_(moe.MoeDispatchArgs, DISPATCH, dict(tokens=600))
    need = moe.moe_dispatch_workspace_bytes(600, 2, 8)
    assert need > 0
    assert lib.moe_dispatch(ctypes.byref(a), 0x10000, need - 1, None) == 3
    assert lib.moe_dispatch(ctypes.byref(a), 0x10080, need, None) == 1
    last = 0
    for t in [1, 100, 512, 513, 700, 5000, 8192, 8193, 65536, 131072, 131073, 1 << 20, 1 << 28]:
        for k in (2,):
            need = moe.moe_dispatch_workspace_bytes(t, k, 256)
            assert need >= last
            last = need
    assert lib.moe_dispatch_workspace_bytes(4, 2, 8, None) == 1


def test_dispatch_workspace_never_falls(lib):
    for k in (1, 3, 8, 32):
        got = [moe.moe_dispatch_workspace_bytes(t, k, 5) for t in range(0, 40000, 7)]
        assert got == sorted(got)


@pytest.mark.parametrize("over,code", COUNTS + [
    (dict(o_type=2), 1), (dict(y_type=-1), 1), (dict(inv_row=None), 1), (dict(w=0x2002), 1), (dict(o=None), 1), (dict(o=0x3001), 1),
    (dict(ldo=63), 1), (dict(ld_add=0), 1), (dict(add=0x4002), 1), (dict(y=None), 1), (dict(ldy=8), 1),
])
def test_combine_refuses(lib, over, code):
    assert lib.moe_combine(ctypes.byref(with_(moe.MoeCombineArgs, COMBINE, over)), None) == code
    assert moe.moe_last_error()


@pytest.mark.parametrize("over,code", COUNTS + [
    (dict(o_type=2), 1), (dict(y_type=-1), 1), (dict(inv_row=None), 1), (dict(w=0x2002), 1), (dict(dy=None), 1), (dict(ld_dy=63), 1), (dict(o=None), 1),
    (dict(ldo=63), 1), (dict(d_o=0x5001), 1), (dict(ld_d_o=0), 1), (dict(d_o=None, d_w=None), 1), (dict(d_w=0x6002), 1),
])
def test_combine_grad_refuses(lib, over, code):
    assert lib.moe_combine_grad(ctypes.byref(with_(moe.MoeCombineGradArgs, GRAD, over)), None) == code
    assert moe.moe_last_error()


def test_null_and_no_tokens(lib):
    assert lib.moe_dispatch(None, None, 0, None) == 1
    assert lib.moe_combine(None, None) == 1
    assert lib.moe_combine_grad(None, None) == 1
    assert lib.moe_combine(ctypes.byref(with_(moe.MoeCombineArgs, COMBINE, dict(tokens=0, y=None))), None) == 0
    assert lib.moe_combine_grad(ctypes.byref(with_(moe.MoeCombineGradArgs, GRAD, dict(tokens=0, dy=None))), None) == 0
    assert lib.moe_dispatch(ctypes.byref(with_(moe.MoeDispatchArgs, DISPATCH, dict(tokens=0, ids=None))), None, 0, None) == 0


def test_pairs_past_the_largest_grids_are_refused(lib):
    need = ctypes.c_size_t()
    for tokens, k, code in [(2 ** 31 - 65536, 1, 0), (2 ** 31 - 65535, 1, 2), (2 ** 31 - 1, 1, 2), ((2 ** 31 - 65536) // 8, 8, 0), ((2 ** 31 - 65536) // 8 + 1, 8, 2)]:
        assert lib.moe_dispatch_workspace_bytes(tokens, k, 256, ctypes.byref(need)) == code
    for call, cls, base in ((lib.moe_combine, moe.MoeCombineArgs, COMBINE), (lib.moe_combine_grad, moe.MoeCombineGradArgs, GRAD)):
        assert call(ctypes.byref(with_(cls, base, dict(tokens=2 ** 31 - 1, top_k=1))), None) == 2
