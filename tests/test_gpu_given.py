"""nucleus_sample_given and nucleus_spec_verify_given against the definition
in 64 bits and more: whole numbers (tokens, keep counts, verdicts) have to be
equal, log-probabilities and probabilities right to a rounding of fp32.

Where a test's rows could put a mass within 1e-11 of its border (where two
correct float64 programs may differ) the row says so itself: the reference
returns the distance, and no test's rows come that close."""
import numpy as np
import pytest
import torch

import workloads
from gpu_util import device_logits, say
from test_gpu_parity import _edge_batch, _random_batch

pytestmark = pytest.mark.gpu


def _reference(x, T, p, k, mp, u):
    """One row after another over its distinct values.  Returns token, count,
    logprob, probs and the least relative distance of any decision."""
    B, V = x.shape
    N = u.shape[1]
    token, count = np.full((B, N), -1, np.int32), np.zeros(B, np.int32)
    logprob, probs = np.full((B, N), np.nan), np.zeros((B, V))
    near = np.inf
    for b in range(B):
        row = x[b].astype(np.float64)
        if np.isnan(row).any() or (row == np.inf).any() or not (row > -np.inf).any() or np.isnan([T[b], p[b], mp[b]]).any():
            continue
        m = row.max()
        if T[b] <= 0:
            i = int(np.argmax(row))
            token[b], count[b], logprob[b] = i, 1, 0.0
            probs[b, i] = 1.0
            continue
        level, inverse, size = np.unique(row, return_inverse=True, return_counts=True)
        with np.errstate(over="ignore", invalid="ignore"):
            weight = np.where(level > -np.inf, 1.0 if np.isinf(T[b]) else np.exp((level - m) / T[b].astype(np.float64)), 0.0)
        alive = level > -np.inf
        if mp[b] > 0:
            alive &= weight >= min(float(mp[b]), 1.0)
        higher = np.cumsum(np.where(alive, size, 0)[::-1])[::-1] - np.where(alive, size, 0)
        if 0 < k[b] < size[alive].sum():
            alive &= higher < k[b]
        mass = np.where(alive, weight * size, 0.0).astype(np.longdouble)
        above = np.concatenate([np.cumsum(mass[::-1])[::-1][1:], [np.longdouble(0)]])
        total = mass.sum()
        kept = alive
        if p[b] < 1:
            kept = alive & (above < np.longdouble(p[b]) * total)
            if p[b] > 0:
                near = min(near, float(np.abs(above[alive] / total - np.longdouble(p[b])).min()))
        kept[-1] = True
        member = kept[inverse]
        where = np.nonzero(member)[0]
        w = weight[inverse[where]].astype(np.longdouble)
        run = np.cumsum(w)
        with_mass = np.nonzero(w > 0)[0]
        count[b] = len(where)
        probs[b, where] = (w / run[-1]).astype(np.float64)
        for n in range(N):
            if np.isnan(u[b, n]):
                continue
            t = np.clip(np.longdouble(u[b, n]), 0, 1)
            i = np.searchsorted(run, t * run[-1], side="right")
            i = min(int(i), int(with_mass[-1]))
            token[b, n] = where[i]
            if np.isinf(T[b]):
                logprob[b, n] = -float(np.log(run[-1]))
            else:
                logprob[b, n] = (row[where[i]] - m) / float(T[b]) - float(np.log(run[-1]))
            if 0 < t < 1:
                near = min(near, float(np.abs(run / run[-1] - t).min()))
    return token, count, logprob, probs, near


def _check(x, T, p, k, mp, u, dtype="f32", what="", strict=True, pad=0, **kw):
    """x: float32 values that `dtype` holds exactly."""
    import nucleus_sampling_amd as ns

    td = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    lg = torch.from_numpy(np.ascontiguousarray(x)).to("cuda:0").to(td)
    if pad:
        wide = torch.full((lg.shape[0], lg.shape[1] + pad), float("nan"), dtype=td, device="cuda:0")
        wide[:, :lg.shape[1]] = lg
        lg = wide[:, :lg.shape[1]]
    B = x.shape[0]
    k = np.zeros(B, np.int32) if k is None else k
    mp = np.zeros(B, np.float32) if mp is None else mp
    say(f"sample_given {what} {dtype} B={B} V={x.shape[1]} N={u.shape[1]}")
    token, count, logprob, probs, near = _reference(x, T, p, k, mp, u)
    if strict:
        assert near > 1e-11, near
    results = []
    for alone in (False, True):  # rows split over workgroups where that is the choice, and one workgroup a row
        got = ns.sample_given(lg, torch.from_numpy(T), torch.from_numpy(p), torch.from_numpy(u), torch.from_numpy(k),
                              torch.from_numpy(mp), want_probs=True, single_workgroup=alone, **kw)
        torch.cuda.synchronize()
        gt, gc = got.token.cpu().numpy(), got.keep_count.cpu().numpy()
        say(what, "one workgroup a row" if alone else "default path")
        assert np.array_equal(gc, count), (what, alone, np.nonzero(gc != count)[0][:5], gc[gc != count][:5],
                                           count[gc != count][:5])
        assert np.array_equal(gt, token), (what, alone, np.argwhere(gt != token)[:5], gt[gt != token][:5],
                                           token[gt != token][:5])
        # logprob: computed in double (errors ~1e-13 relative to the mass), rounded once.
        gl = got.logprob.cpu().numpy().astype(np.float64)
        ok = np.isnan(logprob)
        assert np.array_equal(np.isnan(gl), ok)
        assert (np.abs(gl - logprob)[~ok] <= 2.0**-24 * np.abs(logprob[~ok]) + 1e-11).all()
        gp = got.probs.cpu().numpy().astype(np.float64)
        # 2^-126: the smallest normal fp32; below it, its last place.
        assert (np.abs(gp - probs) <= (2.0**-24 + 1e-11) * probs + 2.0**-149).all()
        results.append(got)
    return results[0]


def _u(rng, B, N, dtype=np.float32):
    return rng.random((B, N)).astype(dtype)


@pytest.mark.parametrize("n", [1, 2])
def test_workloads(n):
    w = workloads.make(n)
    rng = np.random.default_rng(n)
    _check(w["logits"], w["temperature"], w["top_p"], w["top_k"], w["min_p"], _u(rng, w["B"], 3), what=f"workload {n}")


@pytest.mark.parametrize("n,rows,dtype", [(3, 24, "f32"), (4, 24, "bf16"), (5, 12, "f32")])
def test_large_vocabulary_workloads(n, rows, dtype):
    w = workloads.make(n, rows=range(rows))
    x = workloads.bf16_bits_to_f32(w["logits"]) if w["dtype"] == "bf16" else w["logits"]
    rng = np.random.default_rng(n)
    _check(x, w["temperature"], w["top_p"], w["top_k"], w["min_p"], _u(rng, rows, 4), dtype, what=f"workload {n}")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 63, 257, 1000, 4097, 8192, 33001, 49152, 65537, 131073])
def test_ragged_lengths(V, dtype):
    rng = np.random.default_rng(V)
    w = _random_batch(rng, 9, V, "f32")
    x = torch.from_numpy(w["logits"]).to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype])
    k = None if w["top_k"] is None else np.asarray(w["top_k"], np.int32)
    mp = None if w["min_p"] is None else np.asarray(w["min_p"], np.float32)
    _check(x.float().numpy(), np.asarray(w["temperature"], np.float32), np.asarray(w["top_p"], np.float32), k, mp,
           _u(rng, 9, 2), dtype, what="ragged", pad=(0, 5, 8)[V % 3])


def test_edge_rows():
    """NaN, +inf and empty rows, NaN parameters, ties, extreme temperatures."""
    L, T, P, K, MP = _edge_batch()
    rng = np.random.default_rng(3)
    _check(np.asarray(L, np.float32), np.asarray(T, np.float32), np.asarray(P, np.float32),
           None if K is None else np.asarray(K, np.int32), None if MP is None else np.asarray(MP, np.float32),
           _u(rng, len(T), 5), what="edge rows", strict=False)


def test_uniforms_at_and_past_the_ends():
    """u = 0 takes the first kept token, u >= 1 the last, negative the first,
    NaN none; a draw on the border between two equal tokens takes the second."""
    x = np.full((4, 300), -np.inf, np.float32)
    x[0, [7, 90, 200]] = [1.0, 2.0, 0.5]
    x[1, [3, 5]] = 1.25                       # two equal tokens: u = 1/2 is the border
    x[2] = 0.0                                # 300 equal tokens
    x[3, [4, 299]] = [0.0, -800.0]            # the last kept token has weight e^-800: 0 in double
    T, p = np.ones(4, np.float32), np.ones(4, np.float32)
    u = np.tile(np.asarray([0.0, -3.0, 1.0, 7.0, np.nan, 0.5, 0.25, 1.0 - 2.0**-53, np.inf, -np.inf], np.float64), (4, 1))
    got = _check(x, T, p, None, None, u, what="ends", strict=False)
    tok = got.token.cpu().numpy()
    assert tok[0].tolist()[:5] == [7, 7, 200, 200, -1]
    assert tok[1, 5] == 5 and tok[2, 5] == 150 and tok[2, 6] == 75
    assert (tok[3, [0, 2, 3, 5, 7, 8]] == 4).all()


def test_float64_uniforms_and_many_draws():
    rng = np.random.default_rng(4)
    x = rng.normal(0, 2, (3, 5000)).astype(np.float32)
    T, p = np.asarray([0.7, 1.0, 1.3], np.float32), np.asarray([0.9, 0.95, 1.0], np.float32)
    got = _check(x, T, p, None, None, _u(rng, 3, 1500, np.float64), what="many draws")
    # the draws follow the distribution (seeded: 1500 draws, mass of the top 50 tokens)
    probs = got.probs.cpu().numpy().astype(np.float64)
    tok = got.token.cpu().numpy()
    for b in range(3):
        top = np.argsort(-probs[b])[:50]
        mass = probs[b, top].sum()
        assert abs(np.isin(tok[b], top).mean() - mass) < 6 * np.sqrt(mass * (1 - mass) / 1500)


def test_top_k_below_the_window():
    """Low temperatures: the k-th largest token weighs less than 2^-64 of the
    max, where the histogram only counts."""
    rng = np.random.default_rng(5)
    x = (rng.normal(0, 3, (6, 9000))).astype(np.float32)
    x[:, 1000:1100] = x[:, 1000:1001]  # ties there too
    T = np.asarray([0.02, 0.05, 0.1, 1e-30, 3e38, 0.02], np.float32)
    p = np.asarray([1.0, 1.0, 1.0, 1.0, 1.0, 0.9], np.float32)
    k = np.asarray([4000, 8999, 20, 6000, 5000, 4000], np.int32)
    mp = np.asarray([0, 1e-30, 0, 0, 0.5, 0], np.float32)
    _check(x, T, p, k, mp, _u(rng, 6, 4), what="tail", strict=False)


@pytest.mark.parametrize("V", [20000, 70001])
def test_more_undecided_tokens_than_the_list_holds(V):
    """Whole rows tied, or packed into one cell: the undecided tokens are read
    from memory again instead of the list."""
    rng = np.random.default_rng(V)
    x = np.zeros((6, V), np.float32)
    x[1] = np.linspace(0, 0.02, V)[rng.permutation(V)]          # one cell
    x[2] = rng.integers(0, 2, V)                                  # two levels
    x[3] = np.linspace(0, 0.02, V)[rng.permutation(V)]
    x[4] = np.linspace(0, 0.02, V)[rng.permutation(V)]
    x[5] = rng.integers(0, 2, V) * np.float32(1e-3)
    T = np.asarray([1, 1, 1, 0.7, 1.3, 1], np.float32)
    p = np.asarray([0.5, 0.6, 0.3, 0.9, 1.0, 0.7], np.float32)
    k = np.asarray([5, 0, 0, V // 2, 11000, V // 3], np.int32)
    mp = np.asarray([0, 0, 0, 0.99, 0.985, 0], np.float32)
    _check(x, T, p, k, mp, _u(rng, 6, 6), what="overflow")


def test_max_above_the_window():
    """The first tokens of every wave are far below the row's max, or masked:
    the first pass is taken again from the max."""
    rng = np.random.default_rng(6)
    V = 40000
    x = rng.normal(-500, 2, (4, V)).astype(np.float32)
    x[0, 12345] = 300.0
    x[1, 20000:20050] = rng.normal(250, 1, 50)
    x[2] = -np.inf
    x[2, V - 3:] = [1.0, 2.0, 1.5]
    x[3, :39000] = -np.inf
    T = np.asarray([1.0, 0.8, 1.0, 0.5], np.float32)
    p = np.asarray([0.9, 0.9, 0.95, 0.9], np.float32)
    k = np.asarray([0, 10, 0, 500], np.int32)
    _check(x, T, p, k, None, _u(rng, 4, 4), what="max above the window")


@pytest.mark.parametrize("V", [400, 50000])
def test_about_as_many_undecided_tokens_as_a_wave_has_lanes(V):
    """62 to 67 tokens in the cells that the cuts fall into, distinct or in
    ties, cut by top-k, min-p, top-p and pairs of them."""
    rng = np.random.default_rng(V + 1)
    x = rng.normal(-9, 1, (36, V)).astype(np.float32)
    T, p = np.ones(36, np.float32), np.ones(36, np.float32)
    k, mp = np.zeros(36, np.int32), np.zeros(36, np.float32)
    for b in range(36):
        c = 62 + b % 6
        at = rng.choice(V, c, replace=False)
        x[b, at] = (np.linspace(0, 0.01, c) if b % 4 else np.round(np.linspace(0, 0.01, c), 3))[rng.permutation(c)]
        kind = b // 6
        if kind in (0, 3, 5):
            p[b] = 0.5
        if kind in (1, 3):
            k[b] = c // 2 + 3
        if kind in (2, 5):
            mp[b] = 0.996
        if kind == 4:
            k[b], p[b] = 1 + b % 3, 0.01
    _check(x, T, p, k, mp, _u(rng, 36, 3), what="a wave of undecided tokens", strict=False)


@pytest.mark.parametrize("dtype,V", [("f32", 45001), ("bf16", 50000)])
@pytest.mark.parametrize("B", [3, 36])
def test_every_kind_of_row_in_a_split_batch(B, dtype, V):
    """Few and many long rows: planned from parts, or by one workgroup each."""
    rng = np.random.default_rng(B * V)
    x = rng.normal(0, 2, (36, V)).astype(np.float32)
    T, p = rng.uniform(0.5, 1.5, 36).astype(np.float32), rng.uniform(0.3, 1.0, 36).astype(np.float32)
    k, mp = np.zeros(36, np.int32), np.zeros(36, np.float32)
    x[0] = np.linspace(0, 0.02, V)[rng.permutation(V)]   # more undecided tokens than a part lists
    x[1] = rng.normal(-400, 2, V)
    x[1, V - 2] = 300.0                                    # the max above the window
    x[2], k[2], T[2] = rng.normal(0, 3, V), V // 2, 0.02   # the k-th token below the window
    x[3], T[3] = -np.inf, 1.0
    x[3, [5, 44000]] = [1.0, 2.0]                          # two tokens left
    x[4] = np.nan                                          # errors
    x[5, 17] = np.inf
    x[6] = -np.inf
    T[7] = 0.0                                             # greedy
    k[8], k[9], k[10] = 1, 50, V + 7
    p[11], p[12], mp[12] = 1.0, 1.0, 0.1
    x[13] = 1.5                                            # all tied
    x[14, V // 2:] = np.finfo(np.float32).min if dtype == "f32" else -1e38
    x = x[rng.permutation(36)[:B]] if B < 36 else x
    td = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    x = torch.from_numpy(x).to(td).float().numpy()
    _check(x, T[:B], p[:B], k[:B], mp[:B], _u(rng, B, 3), dtype, what="split batch", strict=False)


def test_rows_of_two_million_tokens():
    rng = np.random.default_rng(7)
    x = rng.normal(0, 2, (2, (1 << 21) + 5)).astype(np.float32)
    _check(x, np.asarray([0.8, 1.0], np.float32), np.asarray([0.9, 1.0], np.float32), None, None, _u(rng, 2, 4),
           what="long rows", strict=False)


def test_rows_do_not_depend_on_the_batch_and_repeat():
    import nucleus_sampling_amd as ns

    rng = np.random.default_rng(8)
    lg = torch.from_numpy(rng.normal(0, 2, (40, 6000)).astype(np.float32)).cuda()
    u = torch.from_numpy(rng.random((40, 3)).astype(np.float32)).cuda()
    T, p = torch.full((40,), 0.8), torch.full((40,), 0.9)
    say("sample_given batch independence")
    a = ns.sample_given(lg, T, p, u, want_probs=True)
    c = ns.sample_given(lg, T, p, u, want_probs=True)
    one = ns.sample_given(lg[17:18], T[:1], p[:1], u[17:18], want_probs=True)
    flat = ns.sample_given(lg, T, p, u[:, 0])
    for x, y in zip(a, c):
        assert torch.equal(x, y)
    for x, y in zip(a, one):
        assert torch.equal(x[17:18], y)
    assert flat.token.shape == (40,) and torch.equal(flat.token, a.token[:, 0])


def test_kept_set_is_that_of_sample():
    """Keep counts and kept sets against nucleus_sample's on the same rows
    (its masses are right to 1e-7; rows within that of their border are few
    and none of these)."""
    import nucleus_sampling_amd as ns

    w = workloads.make(2)
    lg = device_logits(w["logits"], "f32")
    say("sample_given against sample")
    a = ns.sample(lg, w["temperature"], w["top_p"], w["top_k"], w["min_p"], want_probs=True)
    g = ns.sample_given(lg, w["temperature"], w["top_p"], torch.rand(w["B"], 1, device="cuda"), w["top_k"], w["min_p"],
                        want_probs=True)
    assert torch.equal(a.keep_count, g.keep_count)
    assert torch.equal(a.probs > 0, g.probs > 0)


def test_captured_replayed_and_side_stream():
    import nucleus_sampling_amd as ns

    rng = np.random.default_rng(9)
    B, V = 12, 20000
    lg = torch.empty(B, V, device="cuda").normal_()
    u = torch.rand(B, 2, device="cuda")
    T, p = torch.full((B,), 0.9, device="cuda"), torch.full((B,), 0.9, device="cuda")
    q = torch.softmax(torch.randn(B, V, device="cuda"), 1)
    ns.sample_given(lg, T, p, u, want_probs=True)
    torch.cuda.synchronize()
    say("sample_given + spec_verify_given captured")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = ns.sample_given(lg, T, p, u, want_probs=True)
        v = ns.spec_verify_given(g.probs, q, g.token[:, 0], u)
    for i in range(4):
        lg.normal_()
        u.uniform_()
        q.copy_(torch.softmax(torch.randn(B, V, device="cuda"), 1))
        graph.replay()
        torch.cuda.synchronize()
        e = ns.sample_given(lg, T, p, u, want_probs=True)
        ev = ns.spec_verify_given(e.probs, q, e.token[:, 0], u)
        for x, y in zip((*g, *v), (*e, *ev)):
            assert torch.equal(x, y), i
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = ns.sample_given(lg, T, p, u, stream=side)
    sv = ns.spec_verify_given(e.probs, q, s.token[:, 0].cpu(), u, stream=side)
    side.synchronize()
    assert torch.equal(s.token, e.token) and torch.equal(sv.token, ev.token)


# ---- verification ---------------------------------------------------------

def _verify_reference(p, q, d, u):
    B, V = p.shape
    tok, acc = np.full(B, -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        if not 0 <= d[b] < V or np.isnan(u[b, 0]):
            continue
        if np.longdouble(u[b, 0]) * np.longdouble(q[b, d[b]]) < np.longdouble(p[b, d[b]]):
            tok[b], acc[b] = d[b], 1
            continue
        r = p[b].astype(np.longdouble) - q[b].astype(np.longdouble)
        where = np.nonzero(r > 0)[0]
        run = np.cumsum(r[where])
        if len(where) == 0 or np.isnan(u[b, 1]) or not np.isfinite(run[-1]):
            continue
        i = np.searchsorted(run, np.clip(np.longdouble(u[b, 1]), 0, 1) * run[-1], side="right")
        tok[b] = where[min(int(i), len(where) - 1)]
    return tok, acc


def _verify(p, q, d, u, what):
    import nucleus_sampling_amd as ns

    say(f"spec_verify_given {what} B={p.shape[0]} V={p.shape[1]}")
    got = ns.spec_verify_given(torch.from_numpy(p).cuda(), torch.from_numpy(q).cuda(), torch.from_numpy(d),
                               torch.from_numpy(u))
    torch.cuda.synchronize()
    tok, acc = _verify_reference(p, q, d, u)
    assert np.array_equal(got.accepted.cpu().numpy(), acc)
    gt = got.token.cpu().numpy()
    assert np.array_equal(gt, tok), (np.nonzero(gt != tok)[0][:5], gt[gt != tok][:5], tok[gt != tok][:5])
    return tok, acc


def _dists(rng, B, V, zero=0.5):
    p = rng.random((B, V)).astype(np.float32) ** 4
    p[rng.random((B, V)) < zero] = 0
    p[:, rng.integers(V)] += 0.01
    q = rng.random((B, V)).astype(np.float32) ** 4 + 1e-6
    return (p / p.sum(1, keepdims=True)).astype(np.float32), (q / q.sum(1, keepdims=True)).astype(np.float32)


@pytest.mark.parametrize("B,V", [(3, 1), (5, 2), (9, 3), (20, 7), (33, 255), (64, 1024), (10, 8191), (10, 8192),
                                 (10, 8193), (7, 40001), (4, 128256), (2, (1 << 20) + 7)])
def test_verify_shapes(B, V):
    rng = np.random.default_rng(V)
    p, q = _dists(rng, B, V)
    d = rng.integers(0, V, B).astype(np.int32)
    u = rng.random((B, 2)).astype(np.float32 if V % 2 else np.float64)
    _verify(p, q, d, u, "shapes")


def test_verify_edges():
    """Draft tokens out of range, a target of zeros (a row error), p = q, NaN
    and infinite entries, uniforms at the ends and NaN, one positive entry."""
    rng = np.random.default_rng(1)
    B, V = 16, 9000
    p, q = _dists(rng, B, V)
    d = rng.integers(0, V, B).astype(np.int32)
    u = rng.random((B, 2))
    d[0], d[1] = -1, V
    p[2] = 0
    q[3] = p[3]
    u[3, 0] = 1.0                   # p = q and nothing to redraw: -1
    p[4, 5], d[4] = np.nan, 5       # not accepted, adds nothing
    p[5, 77], d[5], p[5, 9] = np.inf, 9, 0.0
    u[6] = [np.nan, 0.5]
    p[7, d[7]], u[7] = 0.0, [0.5, np.nan]
    for i, v in ((8, 0.0), (9, 1.0), (10, -2.0), (11, 5.0)):
        p[i, d[i]], u[i] = 0.0, [0.5, v]
    p[12], q[12] = 0.0, 1.0 / V
    p[12, 8999] = 1.0               # one positive entry, at the row's end
    d[12], u[12] = 4, [0.3, 0.999]
    u[13, 0] = 0.0                  # accepted iff p(d) > 0
    q[14, d[14]] = 0.0              # u 0 < p(d)
    q[15, d[15]] = np.nan
    tok, acc = _verify(p, q, d, u, "edges")
    assert (tok[[0, 1, 2, 3, 5, 6, 7]] == -1).all() and tok[12] == 8999


@pytest.mark.parametrize("V", [2047, 2048, 2049, 32767, 32768, 32769])
def test_verify_at_the_sizes_where_its_kernels_change(V):
    rng = np.random.default_rng(V)
    p, q = _dists(rng, 40, V)
    d = rng.integers(0, V, 40).astype(np.int32)
    u = np.stack([rng.random(40) * 2, np.linspace(0, 1, 40)], 1).astype(np.float32)
    d[:20] = p[:20].argmin(1)  # (of weight 0, many: rejected)
    _verify(p, q, d, u, "around a size")


def test_many_draws_of_split_rows():
    rng = np.random.default_rng(31)
    x = rng.normal(0, 2, (2, 60000)).astype(np.float32)
    _check(x, np.asarray([0.7, 1.1], np.float32), np.asarray([0.9, 1.0], np.float32), None, None,
           _u(rng, 2, 300, np.float64), what="many draws of split rows", strict=False)


def test_empty_batches():
    import nucleus_sampling_amd as ns

    say("empty batches")
    none = torch.empty(0, 64, device="cuda")
    e = torch.empty(0, device="cuda")
    got = ns.sample_given(none, e, e, torch.empty(0, 3, device="cuda"), want_probs=True)
    assert got.token.shape == (0, 3) and got.keep_count.shape == (0,) and got.probs.shape == (0, 64)
    v = ns.spec_verify_given(none, none, torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"))
    assert v.token.shape == (0,) and v.accepted.shape == (0,)
    w = torch.zeros(64, 8, device="cuda")
    assert ns.project(torch.empty(0, 8, device="cuda"), w).shape == (0, 64)
    assert ns.sample_hidden(torch.empty(0, 8, device="cuda"), w, e, e, uniforms=e).token.shape == (0,)
    with pytest.raises(ns.NucleusError):
        ns.sample_given(torch.empty(2, 0, device="cuda"), torch.ones(2), torch.ones(2), torch.zeros(2))
