"""nucleus_project against the same product in 64 bits.

Most inputs are small whole numbers, so every sum is exact in fp32 in
whatever order it is taken (K * 9 < 2^24): without an activation that rounds,
fp32 outputs have to be equal and 16-bit outputs equal to the exact result
rounded once, to nearest even.  That catches any operand in a wrong place."""
import math

import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _whole(rows, cols, dtype, seed, pad=0, offset=0, fill=float("nan")):
    """Whole numbers -3 .. 3 in rows `cols + pad` apart that start `offset`
    elements into their allocation; what lies between rows is `fill`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.full((rows * (cols + pad) + offset + 64,), fill, dtype=dtype, device="cuda")
    t = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    t.copy_(torch.randint(-3, 4, (rows, cols), device="cuda", generator=g))
    return t


def _exact(h, w, bias=None, residual=None, act="none", cap=0.0):
    z = torch.mm(h.contiguous().double().cpu(), w.contiguous().double().cpu().t())
    if bias is not None:
        z = z + bias.double().cpu()
    if act == "relu":
        z = torch.where(z < 0, 0.0, z)
    elif act == "gelu":
        z = 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    elif act == "silu":
        z = z * torch.sigmoid(z)
    elif act == "softcap":
        z = cap * torch.tanh(z / cap)
    if residual is not None:
        z = z + residual.double().cpu()
    return z


def _equal(got, want, what):
    got, want = got.cpu(), want.to(got.dtype)
    bad = (got != want) & ~(got.isnan() & want.isnan())
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(),
                           want[bad][:4].tolist())


# One row to several tiles of rows; sizes below, at and just past every tile edge.
SHAPES = [(1, 1, 1), (1, 16, 8), (3, 5, 7), (1, 200, 64), (16, 64, 64), (17, 65, 72), (33, 100, 40), (48, 1000, 512),
          (63, 129, 200), (64, 4096, 64), (65, 127, 256), (100, 300, 1000), (128, 512, 128), (129, 257, 136),
          (200, 1024, 320), (256, 256, 64), (257, 300, 520), (300, 700, 2048), (512, 768, 448), (1000, 600, 192)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_whole_numbers_are_exact(M, N, K, dtype):
    import nucleus_sampling_amd as ns

    say(f"project {dtype} M={M} N={N} K={K}")
    h, w = _whole(M, K, DT[dtype], 1), _whole(N, K, DT[dtype], 2)
    want = _exact(h, w)
    _equal(ns.project(h, w, out_dtype=torch.float32), want, "fp32 out")
    _equal(ns.project(h, w), want, "same type out")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K,pad,offset", [(5, 40, 64, 8, 0), (5, 40, 64, 3, 0), (70, 90, 128, 8, 8),
                                              (70, 90, 128, 0, 1), (20, 33, 77, 0, 0), (300, 260, 256, 24, 16),
                                              (300, 260, 250, 5, 3), (2, 4, 9, 1, 1), (257, 512, 1024, 8, 0)])
def test_rows_anywhere(M, N, K, pad, offset, dtype):
    """Strided rows, rows that start off 16-byte boundaries, odd K; NaN lies
    between the rows of the inputs and a marker between those of the output."""
    import nucleus_sampling_amd as ns

    say(f"project {dtype} M={M} N={N} K={K} pad={pad} offset={offset}")
    h, w = _whole(M, K, DT[dtype], 3, pad, offset), _whole(N, K, DT[dtype], 4, pad, offset)
    bias = _whole(1, N, DT[dtype], 5)[0]
    res = _whole(M, N, torch.float32, 6, pad, offset)
    wide = torch.full((M, N + 5), 777.0, device="cuda")
    out = wide[:, :N]
    got = ns.project(h, w, bias, res, out=out)
    assert got is out
    _equal(out, _exact(h, w, bias, res), "strided out")
    assert (wide[:, N:] == 777.0).all()


@pytest.mark.parametrize("M", [1, 30, 64, 100, 300])
def test_infinities_and_nan_stay_in_their_place(M):
    """-inf in the residual forbids a token; a NaN in one row of hidden, or an
    infinity in one row of weight, reaches that row or column and no other."""
    import nucleus_sampling_amd as ns

    N, K = 260, 192
    h, w = _whole(M, K, torch.bfloat16, 7), _whole(N, K, torch.bfloat16, 8)
    res = _whole(M, N, torch.float32, 9)
    res[:, 7] = float("-inf")
    res[0] = float("-inf")
    clean = _exact(h, w, None, res)
    _equal(ns.project(h, w, None, res, out_dtype=torch.float32), clean, "mask")
    h[M - 1, 5] = float("nan")
    w[N - 1, 3] = float("inf")
    got = ns.project(h, w, out_dtype=torch.float32).cpu()
    say(f"project NaN/inf M={M}")
    want = _exact(h, w)
    assert got[M - 1].isnan().all() and not got[:M - 1, :N - 1].isnan().any()
    _equal(got[:M - 1, :N - 1], want[:M - 1, :N - 1], "others")
    assert torch.equal(got[:M - 1, N - 1].isfinite(), want[:M - 1, N - 1].isfinite())


# Relative error of the fp32 epilogue on exact sums, in units of 2^-24: silu
# takes exp (2 units of its value), 1 + it, a quotient and the final product,
# each half a unit in the last place = 1 unit; tanh and its argument's
# quotient likewise; gelu's erfc moves by 2 x^2 per unit of its argument
# x = z/sqrt(2) (z^2 in all, twice for the constant's own rounding).  16 units
# cover the fixed parts with the library functions' own few.
@pytest.mark.parametrize("act,cap", [("relu", 0.0), ("gelu", 0.0), ("silu", 0.0), ("softcap", 30.0), ("softcap", 2.5)])
@pytest.mark.parametrize("M,N,K", [(3, 64, 64), (40, 130, 96), (200, 300, 128), (9, 21, 13)])
def test_activations(act, cap, M, N, K):
    import nucleus_sampling_amd as ns

    say(f"project {act} M={M} N={N} K={K}")
    h, w = _whole(M, K, torch.bfloat16, 10), _whole(N, K, torch.bfloat16, 11)
    h[:, :] = h * 0.125  # exact; sums of a few units
    bias = _whole(1, N, torch.float32, 12)[0]
    z = _exact(h, w, bias)
    want = _exact(h, w, bias, None, act, cap)
    got = ns.project(h, w, bias, activation=act, softcap=cap, out_dtype=torch.float32).double().cpu()
    units = 16 + (4 * z * z if act == "gelu" else 0)
    tol = want.abs() * units * 2.0**-24 + 1e-37
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()
    got16 = ns.project(h, w, bias, activation=act, softcap=cap).double().cpu()
    assert ((got16 - want).abs() <= tol + want.abs() * (2.0**-8 + 2.0**-16) + 1e-37).all()


@pytest.mark.parametrize("dtype,M,N,K", [("bf16", 4, 500, 4096), ("f16", 37, 403, 1992), ("f32", 16, 320, 1024),
                                         ("bf16", 300, 512, 4096), ("f32", 150, 260, 2048), ("bf16", 2, 64, 28672)])
def test_real_values(dtype, M, N, K):
    """Normal values: every addition of the sum may be off by one unit 2^-23
    of the running value (a matrix instruction may cut where others round),
    so the error is at most K 2^-23 times the sum of |h w|; the usual error
    is the square root of that many steps.  Held to 8 sqrt(K) 2^-23 of the
    2-norm of the terms, rows and columns alike (a random walk's steps are
    below the running value, itself a few times that norm)."""
    import nucleus_sampling_amd as ns

    say(f"project values {dtype} M={M} N={N} K={K}")
    g = torch.Generator(device="cuda").manual_seed(13)
    h = torch.randn(M, K, device="cuda", generator=g).to(DT[dtype])
    w = (torch.randn(N, K, device="cuda", generator=g) * (2 / math.sqrt(K))).to(DT[dtype])
    want = _exact(h, w)
    got = ns.project(h, w, out_dtype=torch.float32).double().cpu()
    norm = torch.mm(h.double().cpu() ** 2, (w.double().cpu() ** 2).t()).sqrt()
    tol = 8 * math.sqrt(K) * 2.0**-23 * norm
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()


def test_residual_in_place_other_stream_and_repeat():
    """out = residual (x += silu(W x' + b)); a side stream; equal calls give
    equal bits; expanded (stride 0) rows are taken as their values."""
    import nucleus_sampling_amd as ns

    M, N, K = 70, 256, 256
    h, w = _whole(M, K, torch.bfloat16, 14), _whole(N, K, torch.bfloat16, 15)
    x = _whole(M, N, torch.bfloat16, 16)
    say("project in place")
    want = ns.project(h, w, None, x)
    y = x.clone()
    ns.project(h, w, None, y, out=y)
    _equal(y, want.double().cpu(), "in place")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = ns.project(h, w, None, x, stream=side)
    side.synchronize()
    _equal(z, want.double().cpu(), "side stream")
    one = h[:1].expand(M, K)
    _equal(ns.project(one, w, out_dtype=torch.float32), _exact(one, w), "expanded rows")
    with pytest.raises(ValueError):
        ns.project(h, w.t())  # the last dimension is not dense
    with pytest.raises(ns.NucleusError):
        ns.project(h, w, out=h[:, :N])  # the output would overwrite an input


@pytest.mark.parametrize("M", [1, 48, 200])
def test_captured_and_replayed(M):
    import nucleus_sampling_amd as ns

    N, K = 512, 256
    h, w = _whole(M, K, torch.bfloat16, 17), _whole(N, K, torch.bfloat16, 18)
    out = torch.empty(M, N, device="cuda")
    ns.project(h, w, out=out)
    torch.cuda.synchronize()
    say(f"project captured M={M}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ns.project(h, w, out=out)
    for i in range(3):
        h.copy_(_whole(M, K, torch.bfloat16, 20 + i))
        out.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        _equal(out, _exact(h, w), f"replay {i}")
