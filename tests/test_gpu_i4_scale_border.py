"""Packing of a checkpoint's scales at the borders of the format: the rounding to 20
significant bits comes first, and what it gives is kept below 2^124."""
import numpy as np
import pytest
import torch

import oracle
from moe_workloads import to_f64

from gpu_common import announce, need_gpu
from test_gpu_i4 import shaped, tile_buffers

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    announce(request.node.nodeid)
    yield
    torch.cuda.synchronize()


# (scale bits, the stored scale's bits or None for NaN)
BORDER = [(0x7d7fffe0, 0x7d7fffe0), (0x7d7fffe7, 0x7d7fffe0), (0x7d7fffe8, 0x7d7fffe0), (0x7d7fffe9, 0x7d7ffff0),
          (0x7d7fffef, 0x7d7ffff0), (0x7d7ffff0, 0x7d7ffff0), (0x7d7ffff1, 0x7d7ffff0), (0x7d7ffff7, 0x7d7ffff0),
          (0x7d7ffff8, None), (0x7d7ffff9, None), (0x7d7fffff, None), (0x7d800000, None), (0x7d800001, None),
          (0x7f7fffff, None), (0x7f800000, None), (0x7f800001, None), (0x7fffffff, None),
          (0x00000000, 0x00000000), (0x00800008, 0x00800000), (0x00800018, 0x00800020), (0x00000008, 0x00000000),
          (0x00000018, 0x00000020), (0x00000009, 0x00000010), (0x007ffff8, 0x00800000)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_scales_next_to_the_largest(zeros, group):
    import token_routed_expert_amd as tre
    rng = np.random.default_rng(group)
    R, C = 128, 128
    U = R // group
    q = rng.integers(0, 16, (1, R, C)).astype(np.uint8)
    bits = np.array([b | sign for b, _ in BORDER for sign in (0, 1 << 31)], np.uint32)
    want = np.array([0x7fc00000 if w is None else w | sign for _, w in BORDER for sign in (0, 1 << 31)], np.uint32)
    s = np.resize(bits, (1, U, C)).view(np.float32)
    r = np.resize(want, (1, U, C)).view(np.float32)
    z = rng.integers(0, 16, (1, U, C)).astype(np.uint8) if zeros else None
    codes, words = tile_buffers(1, R, C, group, 16)
    tre.moe_pack_weights_i4(*(None if t is None else torch.from_numpy(t).cuda() for t in (q, s, z)), None, group, codes,
                            words)
    z = np.full(s.shape, 8, np.uint8) if z is None else z
    ref = oracle.i4_tiles(q, r.astype(np.float64), z)
    got = shaped(codes, words, 1, R, C, group)
    nan = np.isnan((ref[1] & np.uint32(0xfffffff0)).view(np.float32))
    assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1][~nan], ref[1][~nan])
    assert np.isnan((got[1][nan] & np.uint32(0xfffffff0)).view(np.float32)).all()
    # every number that a stored scale can be gives numbers
    out = torch.empty(1, R, C, dtype=torch.bfloat16, device="cuda")
    tre.moe_dequantize_weights_i4(codes, words, group, out)
    assert np.array_equal(np.isnan(to_f64(out)), np.repeat(np.isnan(r), group, axis=1))
    assert not torch.isinf(out).any()


@pytest.mark.parametrize("asym", [False, True])
def test_the_quantisers_largest_scale_is_kept(asym):
    """Groups whose scale is the largest there is, quantised, and their codes and scales packed again: the same tiles."""
    import token_routed_expert_amd as tre
    top = 2.0 ** 124 * (1 - 2.0 ** -20)
    W = torch.zeros(1, 128, 128)
    W[0, 3] = (15 if asym else 7) * top                     # 4 bits times 20: a number of fp32
    W[0, 9] = top
    codes, words = tile_buffers(1, 128, 128, 128)
    tre.moe_quantize_weights_i4(W.cuda(), None, 128, asym, codes, words)
    got = shaped(codes, words, 1, 128, 128, 128)
    q, s, z = oracle.quant_i4(W.double().numpy(), 128, asym)
    assert (s == top).all()
    assert np.array_equal(got[0], oracle.i4_tiles(q, s, z)[0]) and np.array_equal(got[1], oracle.i4_tiles(q, s, z)[1])
    c2, w2 = tile_buffers(1, 128, 128, 128)
    tre.moe_pack_weights_i4(torch.from_numpy(q).cuda(), torch.from_numpy(s.astype(np.float32)).cuda(),
                            torch.from_numpy(z).cuda(), None, 128, c2, w2)
    assert torch.equal(codes, c2) and torch.equal(words, w2)
