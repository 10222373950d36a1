"""Every tile shape nucleus_project chooses among, at sizes on both sides of
its edges, on whole numbers (see test_gpu_project.py): the wide vocabularies,
tall batches and short sums that make each of them the choice."""
import pytest
import torch

from gpu_util import say
from test_gpu_project import DT, _equal, _exact, _whole

pytestmark = pytest.mark.gpu

CASES = [  # M, N, K: around the splits of k, 64 x 32, 64 x 64, 128 x 64, 128 x 128 and 256 x 256 tiles
    (1, 4000, 1000), (16, 257, 512), (17, 4097, 264), (40, 2047, 8), (48, 4096, 520), (49, 1000, 1032), (64, 999, 4096),
    (130, 700, 64), (1, 16400, 72), (31, 20001, 128), (64, 16500, 192), (65, 16383, 64), (128, 16385, 136),
    (250, 4100, 576), (512, 4095, 128), (513, 8200, 64), (1000, 4099, 200), (256, 65600, 64), (255, 70001, 136),
    (2049, 4096, 64), (1025, 16390, 72)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", CASES)
def test_shapes(M, N, K, dtype):
    import nucleus_sampling_amd as ns

    say(f"project shapes {dtype} M={M} N={N} K={K}")
    h, w = _whole(M, K, DT[dtype], M, pad=8), _whole(N, K, DT[dtype], N, pad=16)
    bias = _whole(1, N, torch.float32, 5)[0]
    res = _whole(M, N, DT[dtype], 6)
    wide = torch.full((M, N + 4), 777.0, device="cuda")
    ns.project(h, w, bias, res, out=wide[:, :N])
    want = _exact(h, w, bias, res)
    _equal(wide[:, :N], want, "fp32 out")
    assert (wide[:, N:] == 777.0).all()
    _equal(ns.project(h, w, bias, res), want, "same type out")


def test_a_call_between_others_keeps_its_operands():
    """Products of several shapes queued back to back, then checked."""
    import nucleus_sampling_amd as ns

    say("project back to back")
    cases = [(1, 4096, 512), (300, 5000, 256), (48, 4096, 1024), (1100, 4096, 128), (20, 20000, 64)]
    ops = [(_whole(M, K, torch.bfloat16, M), _whole(N, K, torch.bfloat16, N)) for M, N, K in cases]
    outs = [ns.project(h, w, out_dtype=torch.float32) for _ in range(3) for h, w in ops]
    for i, o in enumerate(outs):
        _equal(o, _exact(*ops[i % len(ops)]), i)
