"""layer_buffers on the CPU: what it allocates for each kind of layer, and layers
that their call refuses."""
import ctypes as C

import pytest
import torch

from token_routed_expert_amd import _native as N
from token_routed_expert_amd.buffers import layer_buffers
from token_routed_expert_amd.ops import _io


@pytest.mark.parametrize("mode", [1, 2, 3])
@pytest.mark.parametrize("dtype", ["mxfp4", "mxfp4_a8"])
def test_mxfp4_layers_refuse_memory_efficient_modes(dtype, mode):
    sh, b, ws, _ = layer_buffers(4, 128, 8, 2, 128, dtype=dtype, device="cpu", memory_efficient=mode)
    w = N.moe_mx4_weights(16, 16, 16, 16)
    b.update(logits=torch.zeros(4, 8), x=torch.zeros(4, 128, dtype=torch.bfloat16))
    io = _io(b)
    io.wmx4 = C.cast(C.pointer(w), C.c_void_p).value
    status = N.lib().moe_layer_fwd(C.byref(sh), C.byref(io), C.c_void_p(16), 1 << 40, None)
    assert status == N.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3", "mxfp8", "mxfp4", "mxfp4_a8"])
def test_names(dtype):
    for mode in (0, 3):
        _, b, _, _ = layer_buffers(4, 128, 8, 2, 128, dtype=dtype, device="cpu", memory_efficient=mode)
        assert ("ab_q" in b and "ab_s" in b) == (mode == 3)
        assert ("ab" in b) == (mode == 0 and not dtype.startswith("mxfp4"))
        assert ("dW1" in b) == (not dtype.startswith("mxfp4"))
