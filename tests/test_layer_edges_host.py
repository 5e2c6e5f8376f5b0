"""CPU tests of the norm, the base product and the rotated append at the edges of what they take. Nothing is launched."""
import ctypes

import pytest
import torch

import segmented_gather_gemv_amd as sg
from test_layer_host import _append, _base, _norm

E, OK = sg.SGMV_EINVAL, sg.SGMV_OK
# where _norm has its rows
AT = dict(x=0x1000, residual=0x2000, weight=0x3000, residual_out=0x4000, out=0x5000, codes=0x6000, scale=0x7000)
LD = dict(x="x", residual="r", residual_out="s", out="o")


def _call(**kw):
    return sg.library().sgmv_rms_norm(ctypes.byref(_norm(**kw)), None)


@pytest.mark.parametrize("out", ["out", "residual_out"])
@pytest.mark.parametrize("of", ["x", "residual"])
def test_norm_refuses_rows_in_place_with_other_strides(out, of):
    """Rows of an output over other rows of an input, which other workgroups have not read yet."""
    for ld in ("ld%s_token", "ld%s_head"):
        for wider in (out, of):
            kw = {f"ld{a}_{b}": n for a in "xrsoc" for b, n in (("token", 4096), ("head", 64))}
            kw[ld % LD[wider]] *= 2
            assert _call(**kw, **{out: AT[of]}) == E, (ld, wider)


def test_norm_refuses_outputs_in_each_others_or_an_inputs_place():
    for out in ("residual_out", "out", "codes", "scale"):
        others = [n for n in AT if n != out and not (out in ("residual_out", "out") and n in ("x", "residual"))]
        for other in others:
            assert _call(**{out: AT[other]}) == E, (out, other)


def test_append_refuses_queries_over_its_keys_or_values():
    for part in (0x80000, 0x90000):  # k and v
        assert _append(q_out=part) == E


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_that_the_binding_takes_without_a_workspace_need_none(dtype):
    """BaseWeight.few asks the library only past it: as many rows of any weight take none there, one more of a large one does."""
    for kw in (dict(group=128), dict(group=32), dict(group=64, has_zero=0, zero=0), dict(format=sg.BASE_E2M1, group=32, has_zero=0, zero=0)):
        for N, K in ((1, 1), (40, 300), (4194304, 4194304), (4194304, 1), (1, 4194304)):
            desc = _base(N=N, K=K, dtype=sg.SGMV_F32 if dtype is torch.float32 else sg.SGMV_BF16, **kw)
            w = sg.BaseWeight(torch.empty(0, dtype=torch.uint8), torch.empty(0), None, desc, dtype)
            assert all(sg.sgmv_base_product_workspace(T, w) == 0 for T in range(w.few + 1)), (N, K)
            if N == K == 4194304:
                assert sg.sgmv_base_product_workspace(w.few + 1, w) > 0
