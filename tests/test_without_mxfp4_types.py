"""The package under a torch that has no 4-bit types: everything else works, and the calls that need
the types say so.  In child processes, without a GPU."""
import os
import subprocess
import sys
import textwrap

import pytest

import mixture_experts_layer_07_amd as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
    import torch
    for name in {missing}:
        delattr(torch, name)
    import mixture_experts_layer_07_amd as moe
    assert moe.workspace_size(4, 2, 8, 0, 256, 256, torch.bfloat16) > 0
    assert moe.workspace_size(4, 2, 8, 0, 256, 256, torch.float8_e4m3fn) > 0
    assert moe.layer_few_workspace(4, 256, 256, 8, 2, device="cpu").numel() > 256
    moe.MoELayer(4, 256, 256, 8, 2, moe.ROUTE_DEFAULT, device="cpu")
    moe.MoELayer(4, 256, 256, 8, 2, moe.ROUTE_DEFAULT, device="cpu", few=True)
    x, w = torch.zeros(4, 256), torch.zeros(8, 512, 256)
    calls = [lambda: moe.quantize_mxfp4(x), lambda: moe.dequantize_mxfp4(x, x),
             lambda: moe.expert_ffn_mxfp4(x, x, x, x, w, w, x, x, 2, 8),
             lambda: moe.MoELayer(4, 256, 256, 8, 2, moe.ROUTE_DEFAULT, device="cpu", mxfp4=True)]
    for call in calls:
        try:
            call()
        except NotImplementedError as e:
            assert "float4_e2m1fn_x2" in str(e) and "float8_e8m0fnu" in str(e), e
        else:
            raise AssertionError("accepted")
    try:
        moe.layer_few(x, torch.zeros(4, 8), w, w, 2, 0)
    except ValueError as e:
        assert "must be a GPU tensor" in str(e), e
    else:
        raise AssertionError("accepted")
"""


@pytest.mark.parametrize("missing", [["float4_e2m1fn_x2"], ["float8_e8m0fnu"], ["float4_e2m1fn_x2", "float8_e8m0fnu"]])
def test_without(missing):
    if not os.path.exists(moe.binding.LIB_PATH):
        from mixture_experts_layer_07_amd import build
        build.build(verbose=False)
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(CODE.format(missing=missing))], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_with():
    """Here the types are there, and the names are theirs."""
    import torch
    assert moe.binding.dtype_code(torch.float4_e2m1fn_x2) == moe.MXFP4
