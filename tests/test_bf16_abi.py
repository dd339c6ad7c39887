"""Refusals of the bf16 products and SwiGLU calls: invalid arguments come back as status codes
before any CUDA call (no GPU needed)."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from mxfp8_block_scaled_rowwise_gb300 import _build, binding
    _build.build()
    return binding.load()


@pytest.mark.parametrize("name", ["grouped_gemm_bf16_fwd", "grouped_gemm_bf16_dgrad", "grouped_gemm_bf16_wgrad"])
def test_products_refuse(lib, name):
    f = getattr(lib, name)   # (A, B, off, E, R, N, K, out, dev_err, stream)
    ok = dict(A=16, B=16, off=16, E=4, R=10, N=64, K=64, out=16, err=16)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["A"], a["B"], a["off"], a["E"], a["R"], a["N"], a["K"], a["out"], a["err"], None)
    for kw in (dict(A=None), dict(B=None), dict(off=None), dict(out=None), dict(err=None), dict(E=0), dict(E=1025),
               dict(R=-1), dict(N=0), dict(K=0), dict(N=-8)):
        assert call(**kw) == -1, kw
    for kw in (dict(N=12), dict(K=12), dict(R=1 << 31), dict(K=1 << 31), dict(N=1 << 31), dict(N=1 << 20, K=1 << 20)):
        assert call(**kw) == -3, kw
    for kw in (dict(A=8), dict(B=24), dict(out=4)):
        assert call(**kw) == -2, kw


def test_swiglu_refuses(lib):
    fwd, bwd = lib.moe_swiglu_fwd, lib.moe_swiglu_bwd
    assert fwd(None, 4, 16, 16, None) == -1 and fwd(16, 4, 16, None, None) == -1
    assert bwd(None, 16, 4, 16, 16, None) == -1 and bwd(16, None, 4, 16, 16, None) == -1
    for R, I in ((-1, 16), (4, 0), (4, -8)):
        assert fwd(16, R, I, 16, None) == -1 and bwd(16, 16, R, I, 16, None) == -1
    for R, I in ((4, 12), (1 << 31, 8), (4, 1 << 30)):
        assert fwd(16, R, I, 16, None) == -3 and bwd(16, 16, R, I, 16, None) == -3
    assert fwd(8, 4, 16, 16, None) == -2 and fwd(16, 4, 16, 8, None) == -2
    assert bwd(8, 16, 4, 16, 16, None) == -2 and bwd(16, 8, 4, 16, 16, None) == -2


def test_binding_raises_with_the_status_name(lib):
    from mxfp8_block_scaled_rowwise_gb300 import binding as mx
    import torch
    if torch.cuda.is_available():
        pytest.skip("the binding asks torch for the current stream: covered by the raw calls")
    assert lib.mx_status_str(-3) == b"MX_ERR_UNSUPPORTED"
    with pytest.raises(mx.MxError, match="moe_swiglu_fwd failed: MX_ERR_UNSUPPORTED"):
        mx._check(lib.moe_swiglu_fwd(16, 4, 12, 16, None), "moe_swiglu_fwd")


def test_adamw_plan_checks_its_descriptors_and_lays_them_out(lib):
    import ctypes
    from mxfp8_block_scaled_rowwise_gb300 import binding as mx

    def plan(rows, bits=32, image=None, size=0, info=None):
        t = (mx.AdamwTensor * max(1, len(rows)))(*[mx.AdamwTensor(**r) for r in rows])
        info = mx.AdamwInfo() if info is None else info
        return lib.adamw_plan(t, len(rows), bits, image, size, ctypes.byref(info)), info
    ok = dict(param=16, grad=16, moment=16, second=16, n=10, lr_mult=1.0, param_dtype=0, grad_dtype=1)
    assert plan([ok])[0] == 0
    for bad in (dict(param=None), dict(grad=None), dict(moment=None), dict(second=None), dict(n=0), dict(n=-1),
                dict(scale_m=1), dict(param_dtype=2), dict(grad_dtype=-1), dict(copy=16), dict(weight_decay=-0.5),
                dict(weight_decay=float("nan")), dict(lr_mult=float("inf"))):
        assert plan([{**ok, **bad}])[0] == -1, bad
    for bad in (dict(param=8), dict(grad=2), dict(moment=4), dict(second=24)):
        assert plan([{**ok, **bad}])[0] == -2, bad
    assert plan([])[0] == -1 and plan([ok], bits=16)[0] == -1 and plan([ok], bits=8)[0] == -1
    assert plan([{**ok, "scale_m": 1, "scale_r": 3}], bits=8)[0] == 0
    st, info = plan([{**ok, "n": 33}, {**ok, "n": 2048}, {**ok, "n": 1}])
    assert st == 0 and info.positions == 64 + 2048 + 32 and info.tensors == 3 and info.chunks >= 3
    image = (ctypes.c_char * info.bytes)()
    assert plan([{**ok, "n": 33}, {**ok, "n": 2048}, {**ok, "n": 1}], image=image, size=info.bytes - 1)[0] == -1
    assert plan([{**ok, "n": 33}, {**ok, "n": 2048}, {**ok, "n": 1}], image=image, size=info.bytes)[0] == 0


def test_adamw_calls_refuse(lib):
    import ctypes
    from mxfp8_block_scaled_rowwise_gb300 import binding as mx
    info = mx.AdamwInfo(1024, 64, 2, 1, 32)
    i = ctypes.byref(info)
    step = lambda plan=16, inf=i, s=16, lr=0.1, b1=0.9, b2=0.9, eps=1e-8, flags=0: lib.adamw_step(  # noqa: E731
        plan, inf, s, lr, b1, b2, eps, None, None, 0, flags, None)
    for kw in (dict(plan=None), dict(inf=None), dict(s=None), dict(lr=-1.0), dict(lr=float("nan")), dict(b1=1.0),
               dict(b2=1.5), dict(b1=-0.1), dict(eps=0.0), dict(eps=float("nan")), dict(flags=2)):
        assert step(**kw) == -1, kw
    assert step(plan=8) == -2
    assert lib.adamw_grad_norm(16, i, -1.0, 16, None) == -1 and lib.adamw_grad_norm(16, i, 1.0, None, None) == -1
    assert lib.adamw_state_values(16, i, 16, None, None) == -1
    bad = mx.AdamwInfo(1024, 64, 2, 1, 16)
    assert lib.adamw_grad_norm(16, ctypes.byref(bad), 1.0, 16, None) == -1
