"""The operators around the sampler that are measured, their inputs and their plain forms.

Three operators:

- ``project``: out = act(hidden . weight^T + bias) + residual, the product that makes logits (a vocabulary
  projection) and the block of a draft head (x + silu(W x + b));
- ``sample``: temperature -> min-p -> top-k -> top-p -> renormalise, drawn by inverse CDF from uniforms that the
  caller brings, several draws a row from one distribution;
- ``verify``: speculative acceptance and the residual draw from given uniforms.

With ``own`` false, ``run`` computes the plain form: elementary torch operations in 32 bits, or in 64 where a
probability mass is compared with a border.  With ``own`` true it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # One sequence being decoded: a hidden state against the whole vocabulary matrix (weights read once).
        dict(name="head_one", op="project", M=1, K=4096, N=128256, dtype="bf16", out="f32", act="none", cap=0.0,
             bias=False, residual="none", pad=0),
        # A decode step of the benchmark's batch of 256 rows, with the logits' soft cap in the epilogue.
        dict(name="head_batch", op="project", M=256, K=4096, N=128256, dtype="bf16", out="f32", act="softcap", cap=30.0,
             bias=False, residual="none", pad=0),
        # A ragged batch, an odd vocabulary and a per-request additive mask (-inf forbids a token) as the residual.
        dict(name="head_ragged", op="project", M=37, K=1992, N=32003, dtype="f16", out="f32", act="none", cap=0.0,
             bias=True, residual="mask", pad=0),
        # A projection kept in 32 bits throughout.
        dict(name="head_f32", op="project", M=16, K=1024, N=32000, dtype="f32", out="f32", act="none", cap=0.0,
             bias=True, residual="none", pad=0),
        # A draft head's block on a decode batch: few weights, latency counts.
        dict(name="draft_block", op="project", M=48, K=4096, N=4096, dtype="bf16", out="same", act="silu", cap=0.0,
             bias=True, residual="hidden", pad=0),
        # The same block over the tokens of whole prompts: bound by the matrix cores.
        dict(name="draft_block_prompt", op="project", M=4096, K=4096, N=4096, dtype="bf16", out="same", act="silu",
             cap=0.0, bias=True, residual="hidden", pad=0),
        # The smallest batch of the repository's workloads: pure latency.
        dict(name="sample_small", op="sample", B=15, V=1024, N=1, dtype="f32", shape="normal", sigma=2.0, probs=True,
             topk=0, minp=0.0, pad=0),
        # The benchmark's batch: Zipf-shaped logits, every row its own temperature and p.
        dict(name="sample_zipf", op="sample", B=256, V=128256, N=1, dtype="f32", shape="zipf", sigma=0.5, probs=False,
             topk=0, minp=0.0, pad=0),
        # The whole chain on 16-bit logits with masked tokens and greedy rows, four draws a row.
        dict(name="sample_chain", op="sample", B=256, V=128256, N=4, dtype="bf16", shape="masked", sigma=3.0,
             probs=False, topk=50, minp=0.05, pad=0),
        # One prompt's first token drawn for sixteen continuations, with the distribution written out.
        dict(name="sample_one_row", op="sample", B=1, V=128256, N=16, dtype="f32", shape="normal", sigma=3.0, probs=True,
             topk=0, minp=0.0, pad=0),
        # Verification of a few draft tokens of a small batch.
        dict(name="verify_small", op="verify", B=5, V=32000, keep=0.9),
        # Verification of the benchmark's batch.
        dict(name="verify_batch", op="verify", B=256, V=128256, keep=0.95),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["project", "project", "sample", "sample", "verify"])
    if op == "project":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        K = _log_int(rng, 64, 8192)
        K = K - K % 64 if rng.random() < 0.6 else (K - K % 8 if rng.random() < 0.6 else K)
        square = rng.random() < 0.3
        N = K if square else _log_int(rng, 64, 128256)
        M = _log_int(rng, 1, 4096)
        cap = 6e9 if dtype == "f32" else 1.3e11
        M = max(1, min(M, int(cap / (N * K))))
        act = rng.choice(["none", "relu", "gelu", "silu", "softcap"])
        # the largest listed weight matrix has 525 million elements
        N = max(1, min(N, 525_000_000 // K)) if not square else N
        return dict(op=op, M=M, K=K, N=N, dtype=dtype, out=rng.choice(["f32", "same"]), act=act,
                    cap=round(rng.uniform(5.0, 50.0), 2) if act == "softcap" else 0.0, bias=rng.random() < 0.5,
                    residual="hidden" if square and rng.random() < 0.7 else rng.choice(["none", "mask"]),
                    pad=rng.choice([0, 0, 0, 8, 24, 5]))
    if op == "sample":
        V = _log_int(rng, 50, 152064)
        B = max(1, min(_log_int(rng, 1, 300), 32_000_000 // V))
        return dict(op=op, B=B, V=V, N=rng.choice([1, 1, 2, 5, 16]), dtype=rng.choice(["f32", "f32", "bf16", "f16"]),
                    shape=rng.choice(["normal", "zipf", "masked", "flat", "ties"]), sigma=round(rng.uniform(0.3, 4.0), 3),
                    probs=rng.random() < 0.3, topk=rng.choice([0, 0, 1, 20, 50, 1000, 40000]),
                    minp=rng.choice([0.0, 0.0, 0.02, 0.1]), pad=rng.choice([0, 0, 0, 8, 3]))
    V = _log_int(rng, 50, 152064)
    B = max(1, min(_log_int(rng, 1, 300), 32_000_000 // V))
    return dict(op=op, B=B, V=V, keep=round(rng.uniform(0.5, 1.0), 4))


def work(case):
    if case["op"] == "project":
        M, K, N, b = case["M"], case["K"], case["N"], BYTES[case["dtype"]]
        ob = 4 if case["out"] == "f32" else b
        nbytes = (M * K + N * K) * b + M * N * ob + (N * b if case["bias"] else 0)
        nbytes += M * N * 4 if case["residual"] == "mask" else 0  # the draft block's residual is `hidden`, read already
        return {"bytes": nbytes, "flops": 2 * M * N * K}
    if case["op"] == "sample":
        B, V, N = case["B"], case["V"], case["N"]
        return {"bytes": B * V * BYTES[case["dtype"]] + (B * V * 4 if case["probs"] else 0) + B * (16 + 12 * N) + 4 * B,
                "flops": 4 * B * V}
    B, V = case["B"], case["V"]
    return {"bytes": 2 * B * V * 4 + B * 20, "flops": 2 * B * V}


def _padded(t, pad):
    """`t` as a view whose rows are `pad` elements further apart."""
    if pad == 0:
        return t
    wide = torch.empty(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    wide[:, t.shape[1]:] = float("nan")  # what lies between rows is not the operator's to read
    view = wide[:, :t.shape[1]]
    view.copy_(t)
    return view


def _logits(case, g):
    B, V, sigma = case["B"], case["V"], case["sigma"]
    kind = case["shape"]
    n = torch.randn(B, V, device="cuda", generator=g)
    if kind == "zipf":  # token ranks in random order, weights like a power law
        rank = torch.rand(B, V, device="cuda", generator=g).argsort(1).argsort(1) + 1
        x = -1.1 * rank.float().log() + sigma * n
    elif kind == "flat":  # nearly equal logits: most tokens stay
        x = torch.rand(B, V, device="cuda", generator=g) + 0.01 * n
    elif kind == "ties":  # few distinct values: whole levels tie at the cut
        x = (sigma * n).round().clamp(-4, 4)
    else:
        x = sigma * n
    if kind == "masked":  # a grammar forbids tokens, here and there all but one, or all (a row error)
        x = torch.where(torch.rand(B, V, device="cuda", generator=g) < 0.05, float("-inf"), x)
        rare = torch.rand(B, 1, device="cuda", generator=g)
        x = torch.where((rare < 0.02) & (torch.arange(V, device="cuda")[None] != V // 2), float("-inf"), x)
        x = torch.where(rare > 0.99, float("-inf"), x)
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "project":
        M, K, N = case["M"], case["K"], case["N"]
        dt = DTYPES[case["dtype"]]
        hidden = torch.randn(M, K, device="cuda", generator=g).to(dt)
        weight = torch.empty(N, K, device="cuda", dtype=dt).normal_(0, 2.0 / math.sqrt(K), generator=g)
        s = dict(case=case, hidden=_padded(hidden, case["pad"]), weight=_padded(weight, case["pad"]), bias=None,
                 residual=None)
        if case["bias"]:
            s["bias"] = torch.randn(N, device="cuda", generator=g).mul_(0.5).to(dt)
        if case["residual"] == "hidden":
            s["residual"] = s["hidden"]
        elif case["residual"] == "mask":
            r = torch.randn(M, N, device="cuda", generator=g)
            u = torch.rand(M, N, device="cuda", generator=g)
            s["residual"] = torch.where(u < 0.1, float("-inf"), torch.where(u < 0.15, r, 0.0))
        s["out_dtype"] = torch.float32 if case["out"] == "f32" else dt
        return s
    B, V = case["B"], case["V"]
    if case["op"] == "sample":
        x = _logits(case, g).to(DTYPES[case["dtype"]])
        T = torch.rand(B, device="cuda", generator=g) * 1.2 + 0.3
        p = torch.rand(B, device="cuda", generator=g) * 0.49 + 0.5
        kind = torch.rand(B, device="cuda", generator=g)
        if case["shape"] in ("normal", "masked", "flat", "ties"):
            T = torch.where(kind < 0.12, 0.0, T)                       # greedy requests
            p = torch.where((kind > 0.88) & (kind < 0.96), 1.0, p)     # no nucleus cut
            p = torch.where(kind >= 0.96, 1e-4, p)                     # the top level only
        s = dict(case=case, logits=_padded(x, case["pad"]), temperature=T, top_p=p, top_k=None, min_p=None,
                 uniforms=torch.rand(B, case["N"], device="cuda", generator=g))
        if case["topk"] > 0:  # every other request asks for it
            s["top_k"] = torch.where(torch.rand(B, device="cuda", generator=g) < 0.5, case["topk"], 0).to(torch.int32)
        if case["minp"] > 0:
            s["min_p"] = torch.where(torch.rand(B, device="cuda", generator=g) < 0.7, case["minp"], 0.0)
        return s
    z = 3.0 * torch.randn(B, V, device="cuda", generator=g)
    zd = z + 0.7 * torch.randn(B, V, device="cuda", generator=g)
    p, q = torch.softmax(z, 1), torch.softmax(zd, 1)
    # the target is truncated to roughly its most probable share `keep`
    v, _ = p.sort(1, descending=True)
    n = (v.cumsum(1) < case["keep"]).sum(1, keepdim=True).clamp(max=V - 1)
    p = torch.where(p >= v.gather(1, n), p, 0.0)
    p = p / p.sum(1, keepdim=True)
    noise = torch.empty(B, V, device="cuda").exponential_(generator=g)
    d = (q / noise).argmax(1).to(torch.int32)
    return dict(case=case, target=p, draft=q, token=d, uniforms=torch.rand(B, 2, device="cuda", generator=g))


def _project_plain(s):
    case = s["case"]
    z = s["hidden"].float() @ s["weight"].float().T
    if s["bias"] is not None:
        z = z + s["bias"].float()
    act = case["act"]
    if act == "relu":
        z = z.clamp(min=0)
    elif act == "gelu":
        z = z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    elif act == "silu":
        z = z / (1 + torch.exp(-z))
    elif act == "softcap":
        z = case["cap"] * torch.tanh(z / case["cap"])
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return {"out": z.to(s["out_dtype"])}


def _inverse_cdf(w, u):
    """The lowest index whose running sum of `w` [B, V] exceeds u times the whole, for u [B, N]; at the end the last
    index with a weight."""
    c = w.cumsum(1)
    t = u.double().clamp(0, 1) * c[:, -1:]
    i = torch.searchsorted(c, t, right=True)
    idx = torch.arange(w.shape[1], device=w.device)
    last = torch.where(w > 0, idx, 0).amax(1, keepdim=True)
    return torch.minimum(i, last)


def _sample_plain(s):
    case = s["case"]
    x32 = s["logits"].float()
    B, V = x32.shape
    T, p = s["temperature"].double()[:, None], s["top_p"].double()[:, None]
    idx = torch.arange(V, device=x32.device)
    m = x32.amax(1, keepdim=True)
    greedy = T <= 0
    Ts = torch.where(greedy, 1.0, T)
    bad = m == float("-inf")  # nothing left to draw: token -1
    weigh = lambda v: torch.where(v > float("-inf"), torch.exp((v.double() - m.double()) / Ts), 0.0)  # noqa: E731
    v, _ = x32.sort(1, descending=True)
    e = weigh(v)
    n = (v > float("-inf")).sum(1, keepdim=True)
    if s["min_p"] is not None:
        mp = s["min_p"].double()[:, None].clamp(max=1.0)
        n = torch.where(mp > 0, torch.minimum(n, (e >= mp).sum(1, keepdim=True)), n)
    rank = idx[None]
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        kth = v.gather(1, (torch.minimum(torch.where(k > 0, k, V), n) - 1).clamp(min=0))
        n = torch.where((k > 0) & (k < n), (v >= kth).sum(1, keepdim=True), n)
    e = torch.where(rank < n, e, 0.0)
    c = e.cumsum(1)
    total = c[:, -1:]
    first = torch.searchsorted(-v, -v)  # where each value's level begins
    above = (c - e).gather(1, first)
    keep = (rank < n) & ((above < p * total) | (p >= 1) | (v == m))
    count = keep.sum(1, keepdim=True)
    low = v.gather(1, (count - 1).clamp(min=0))
    lone = torch.where(x32 == m, idx, V).amin(1, keepdim=True)
    kept = torch.where(greedy, idx == lone, x32 >= low) & (x32 > float("-inf"))
    count = torch.where(bad, 0, torch.where(greedy, 1, count))
    w = torch.where(kept, weigh(x32), 0.0)
    mass = w.sum(1, keepdim=True)
    token = _inverse_cdf(w, s["uniforms"])
    logprob = torch.where(greedy, 0.0, (x32.gather(1, token).double() - m.double()) / Ts - mass.log())
    return {"token": torch.where(bad, -1, token).int(), "keep_count": count[:, 0].int(),
            "logprob": torch.where(bad, float("nan"), logprob).float(),
            "probs": torch.where(bad, 0.0, w / mass).float() if case["probs"] else None}


def _verify_plain(s):
    p, q, u = s["target"].double(), s["draft"].double(), s["uniforms"].double()
    d = s["token"].long()[:, None]
    accepted = u[:, :1] * q.gather(1, d) < p.gather(1, d)
    r = (p - q).clamp(min=0)
    token = torch.where(accepted, d, _inverse_cdf(r, u[:, 1:]))
    return {"token": token[:, 0].int(), "accepted": accepted[:, 0].int()}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"project": _project_plain, "sample": _sample_plain, "verify": _verify_plain}[op](s)
    import nucleus_sampling_amd as ns

    if op == "project":
        case = s["case"]
        return {"out": ns.project(s["hidden"], s["weight"], s["bias"], s["residual"], activation=case["act"],
                                  softcap=case["cap"], out_dtype=s["out_dtype"])}
    if op == "sample":
        r = ns.sample_given(s["logits"], s["temperature"], s["top_p"], s["uniforms"], s["top_k"], s["min_p"],
                            want_probs=s["case"]["probs"])
        return {"token": r.token, "keep_count": r.keep_count, "logprob": r.logprob, "probs": r.probs}
    r = ns.spec_verify_given(s["target"], s["draft"], s["token"], s["uniforms"])
    return {"token": r.token, "accepted": r.accepted}


def _exact_rows(x, T, p, k, mp, u, want_probs):
    """The chain of one row at a time over its distinct values, in 64 bits and more."""
    B, V = x.shape
    N = u.shape[1]
    token, logprob = np.empty((B, N), np.int32), np.empty((B, N))
    count = np.empty(B, np.int32)
    probs = np.zeros((B, V)) if want_probs else None
    for b in range(B):
        row = x[b].astype(np.float64)
        m = row.max()
        if m == -np.inf:
            token[b], logprob[b], count[b] = -1, np.nan, 0
            continue
        if T[b] <= 0:
            i = int(np.argmax(row))
            token[b], logprob[b], count[b] = i, 0.0, 1
            if want_probs:
                probs[b, i] = 1.0
            continue
        level, inverse, size = np.unique(row, return_inverse=True, return_counts=True)
        weight = np.exp((level - m) / T[b])          # of one token of each level, ascending
        alive = level > -np.inf
        if mp[b] > 0:
            alive &= weight >= min(mp[b], 1.0)
        if 0 < k[b] < int(size[alive].sum()):
            higher = np.cumsum(np.where(alive, size, 0)[::-1])[::-1] - size  # tokens strictly above a level
            alive &= higher < k[b]
        mass = np.where(alive, weight * size, 0.0).astype(np.longdouble)
        above = np.concatenate([np.cumsum(mass[::-1])[::-1][1:], [np.longdouble(0)]])
        kept = alive if p[b] >= 1 else alive & (above < np.longdouble(p[b]) * mass.sum())
        kept[-1] = True
        member = kept[inverse]
        where = np.nonzero(member)[0]
        w = np.exp((row[where] - m) / T[b]).astype(np.longdouble)
        run_sum = np.cumsum(w)
        at = np.searchsorted(run_sum, u[b].astype(np.longdouble) * run_sum[-1], side="right")
        at = np.minimum(at, len(where) - 1)
        token[b], count[b] = where[at], len(where)
        logprob[b] = (row[where[at]] - m) / T[b] - float(np.log(run_sum[-1]))
        if want_probs:
            probs[b, where] = (w / run_sum[-1]).astype(np.float64)
    return {"token": token, "keep_count": count, "logprob": logprob, "probs": probs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "project":
        z = torch.mm(s["hidden"].contiguous().double(), s["weight"].contiguous().double().t())
        if s["bias"] is not None:
            z += s["bias"].double()
        if case["act"] == "relu":
            z = torch.where(z > 0, z, 0.0)
        elif case["act"] == "gelu":
            z = 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
        elif case["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif case["act"] == "softcap":
            z = torch.tanh(z / case["cap"]) * case["cap"]
        if s["residual"] is not None:
            z += s["residual"].double()
        return {"out": z}
    if case["op"] == "sample":
        host = lambda t: t.cpu().double().numpy()  # noqa: E731
        B = case["B"]
        zero = np.zeros(B)
        return _exact_rows(s["logits"].float().cpu().numpy(), host(s["temperature"]), host(s["top_p"]),
                           zero if s["top_k"] is None else host(s["top_k"]),
                           zero if s["min_p"] is None else host(s["min_p"]), host(s["uniforms"]), case["probs"])
    p, q = s["target"].cpu().numpy(), s["draft"].cpu().numpy()
    d, u = s["token"].cpu().numpy(), s["uniforms"].cpu().numpy()
    token, accepted = d.copy(), np.ones(len(d), np.int32)
    for b in range(len(d)):
        if np.longdouble(u[b, 0]) * np.longdouble(q[b, d[b]]) < np.longdouble(p[b, d[b]]):
            continue
        accepted[b] = 0
        gain = p[b].astype(np.longdouble) - q[b].astype(np.longdouble)
        where = np.nonzero(gain > 0)[0]
        run_sum = np.cumsum(gain[where])
        at = np.searchsorted(run_sum, np.longdouble(u[b, 1]) * run_sum[-1], side="right")
        token[b] = where[min(at, len(where) - 1)]
    return {"token": token, "accepted": accepted}
