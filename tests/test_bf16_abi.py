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
