"""The tensor types of the binding: calls without a 4-bit form refuse float4 tensors by name as they refuse any other type, and the
package works with a torch that does not know the 4-bit types."""
import os
import subprocess
import sys

import pytest
import torch

import token_dispatch_expert_amd as moe
from token_dispatch_expert_amd import binding as B

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def f4(*shape):
    return torch.zeros(shape, dtype=torch.uint8).view(torch.float4_e2m1fn_x2)


def new(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


def i32(*shape):
    return new(*shape, dtype=I32)


class NoWorkspace:
    ptr, nbytes = None, 0


@pytest.fixture(autouse=True)
def host_tensors(monkeypatch):
    """What is refused for its type is refused before its address is asked for."""
    monkeypatch.setattr(B, "_ptr", lambda t: None)
    monkeypatch.setattr(B, "_stream", lambda s: None)


CALLS = {
    "moe_permute": lambda: moe.moe_permute(f4(4, 64), i32(4, 2), 8, i32(8), i32(9), i32(8), i32(8), f4(8, 64), NoWorkspace),
    "moe_permute_capped": lambda: moe.moe_permute(f4(4, 64), i32(4, 2), 8, i32(8), i32(9), i32(8), i32(8), f4(8, 64), NoWorkspace,
                                                  capacity=3),
    "moe_permute_noalloc": lambda: B.moe_permute_noalloc(f4(4, 64), i32(4, 2), 8, i32(8), i32(9), i32(8), i32(8), f4(8, 64)),
    "moe_route_gemm": lambda: moe.moe_route_gemm(f4(4, 64), f4(8, 64), 2, i32(4, 2), new(4, 2), workspace=NoWorkspace),
    "moe_grouped_ffn": lambda: moe.moe_grouped_ffn(f4(8, 64), i32(9), new(8, 32, 64, dtype=BF), new(8, 32, 64, dtype=BF),
                                                   new(8, 64, 32, dtype=BF), new(8, 64), NoWorkspace),
    "moe_block_weights": lambda: moe.moe_block_weights(f4(2, 64, 64), f4(2, 64, 64)),
    "moe_checkpoint_pack": lambda: moe.moe_checkpoint_pack(f4(8, 128), new(8, 128, dtype=torch.uint8), new(8, 1)),
    "moe_grouped_gemm": lambda: moe.moe_grouped_gemm(f4(8, 64), i32(3), f4(2, 32, 64), new(8, 32)),
}


@pytest.mark.parametrize("name", CALLS)
def test_refused_by_name(name):
    with pytest.raises(TypeError, match="(x|x_sorted|src|w|w_router): .*float4_e2m1fn_x2"):
        CALLS[name]()


def test_sizes():
    """4-bit weights have a workspace; no call's rows in torch's 4-bit type do."""
    assert moe.moe_ffn_workspace_size(64, 4, 256, 128, BF, torch.float4_e2m1fn_x2) == 64 * 128 * 2
    for size in (lambda t: moe.moe_ffn_workspace_size(64, 4, 256, 128, t, BF), lambda t: moe.moe_layer_workspace_size(16, 8, 2, 256, 128, t, BF)):
        with pytest.raises(KeyError):
            size(torch.float4_e2m1fn_x2)


WITHOUT = """
import torch
del torch.float4_e2m1fn_x2, torch.float8_e8m0fnu
import token_dispatch_expert_amd as moe
bf, u8 = torch.bfloat16, torch.uint8
assert moe.moe_layer_workspace_size(16, 8, 2, 256, 128, bf, bf) > 0
codes, scales = moe.mxfp4_buffers((8, 256), device="cpu")
for call, error in ((lambda: moe.moe_mxfp4_quantize(torch.zeros(8, 256, dtype=bf), codes, scales), "expected a device tensor"),
                    (lambda: moe.moe_mxfp4_dequantize(codes.float(), scales, torch.zeros(8, 256)), "expected uint8"),
                    (lambda: moe.moe_mxfp4_dequantize(codes, None, torch.zeros(8, 256)), "codes scales"),
                    (lambda: moe.moe_grouped_ffn(torch.zeros(8, 256, dtype=bf), None, torch.zeros(2, 128, 256, dtype=torch.half),
                                                 torch.zeros(2, 128, 256, dtype=torch.half), torch.zeros(2, 256, 128, dtype=torch.half),
                                                 None, None), "w_gate: unsupported dtype")):
    try:
        call()
    except (TypeError, ValueError) as e:
        assert error in str(e), e
    else:
        raise SystemExit("not refused: " + error)
print("ok")
"""


def test_torch_without_the_types():
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.stdout.strip().endswith("ok"), r.stderr[-2000:]
