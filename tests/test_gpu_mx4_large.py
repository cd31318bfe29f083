"""The MXFP4 quantiser of rows beyond the threads of one launch."""
import numpy as np
import pytest
import torch

import oracle

from gpu_common import announce, need_gpu

pytestmark = pytest.mark.gpu


def test_rows_of_more_than_one_launch(request):
    import token_routed_expert_amd as tre
    need_gpu()
    announce(request.node.nodeid)
    rows, cols = (1 << 23) + 3, 4096                       # 2^35 values and a little more
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of device memory")
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, (1 << 22) - 1, 1 << 22, (1 << 22) + 1, (1 << 23) - 1, 1 << 23, rows - 1]
    some = torch.from_numpy(np.random.default_rng(1).standard_normal((len(at), cols)).astype(np.float32)).bfloat16()
    x[at] = some.cuda()
    codes = torch.full((rows, cols // 2), 0xA5, dtype=torch.uint8, device="cuda")
    sb = torch.full((rows, cols // 32), 0xA5, dtype=torch.uint8, device="cuda")
    tre.moe_quantize_rows_mx4(x, codes, sb)
    rq, rs = oracle.quant_mx4_rows(some.double().numpy())
    assert np.array_equal(codes[at].cpu().numpy(), rq) and np.array_equal(sb[at].cpu().numpy(), rs)
    codes[at] = 0
    sb[at] = 127
    assert not codes.view(torch.int64).any() and int(sb.min()) == 127 and int(sb.max()) == 127
    del x, codes, sb
    torch.cuda.empty_cache()
