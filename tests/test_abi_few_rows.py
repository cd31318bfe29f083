"""Which kernels a call takes (moe_few_rows), on the CPU: the rules that the GPU
tests choose their sizes by are the library's own, and both kernels are reached by
the cases of those tests."""
import pytest

import test_gpu_ckpt8 as ck
import test_gpu_mx4 as mx4
from token_routed_expert_amd import make_shape, moe_few_rows

SIZES = [(P, E, d, f) for P in (1, 8, 20, 33, 97, 160, 300, 513, 1028, 2048, 4096, 9000, 30000, 65536)
         for E in (1, 4, 8, 24, 64, 128, 256) for d, f in ((128, 128), (384, 2560), (512, 384), (1024, 1024),
                                                         (4096, 1536), (1152, 128), (128, 1152))]


@pytest.mark.parametrize("dtype,rule", [("mxfp4", mx4.few_rows), ("mxfp4_a8", mx4.few_rows), ("bf16", ck.few_rows)])
def test_the_tests_rule_is_the_librarys(dtype, rule):
    seen = [0, 0]
    for P, E, d, f in SIZES:
        got = moe_few_rows(make_shape(P, d, E, 1, f, dtype=dtype))
        assert got == bool(rule(P, E, d, f)), (P, E, d, f)
        seen[got] += 1
    assert min(seen) > 100


def test_both_kernels_are_reached():
    for name, counts in mx4.COUNTS.items():
        d, f = {"edges64": (384, 256), "edges128": (128, 640), "hot": (640, 128), "tail": (256, 384),
                "edges256": (512, 256)}.get(name, (256, 128))
        many = mx4.with_many(counts, d, f)
        assert moe_few_rows(make_shape(sum(counts), d, len(counts), 1, f, dtype="mxfp4")), name
        assert not moe_few_rows(make_shape(sum(many), d, len(many), 1, f, dtype="mxfp4")), name
    took = {n: moe_few_rows(make_shape(sum(c), d, len(c), 1, f)) for n, (c, d, f) in ck.COUNTS.items()}
    assert took == {n: n != "many" for n in ck.COUNTS}


def test_other_shapes():
    assert not moe_few_rows(make_shape(4, 128, 8, 1, 128, dtype="e4m3"))
    assert not moe_few_rows(make_shape(4, 128, 8, 1, 128, dtype="f32"))
    assert not moe_few_rows(make_shape(4, 192, 8, 1, 128, dtype="mxfp4"))   # refused by the call
    assert not moe_few_rows(make_shape(4, 128, 8, 9, 128))
    assert moe_few_rows(make_shape(4, 128, 8, 1, 128))
    # (probability partials that do not fit into dW2)
    assert moe_few_rows(make_shape(8192, 128, 1, 1, 128)) and not moe_few_rows(make_shape(8193, 128, 1, 1, 128))
