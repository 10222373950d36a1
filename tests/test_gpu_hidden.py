"""sample_hidden, and a round of speculative decoding with the projection, the
draws and the verification together: every stage against 64 bits on what the
stage before it really gave, then captured and replayed."""
import math

import numpy as np
import pytest
import torch

from gpu_util import say
from test_gpu_given import _reference, _verify_reference

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _product(h, w):
    """The exact product, and the bound of what fp32 sums of normal values may
    be off: a walk of sqrt(K) steps of 2^-23 of the terms' 2-norm, 8 of them."""
    hd, wd = h.double().cpu(), w.double().cpu().t().contiguous()
    return torch.mm(hd, wd), 8 * math.sqrt(h.shape[1]) * 2.0**-23 * torch.mm(hd**2, wd**2).sqrt()


def _drawn(got, logits, T, p, u, k=None, mp=None):
    B = logits.shape[0]
    zero = lambda v, t: np.zeros(B, t) if v is None else v.cpu().numpy()
    token, count, logprob, probs, _ = _reference(logits.float().cpu().numpy(), T.cpu().numpy(), p.cpu().numpy(),
                                                 zero(k, np.int32), zero(mp, np.float32),
                                                 u.cpu().numpy().reshape(B, -1))
    assert np.array_equal(got.token.cpu().numpy().reshape(B, -1), token)
    assert np.array_equal(got.keep_count.cpu().numpy(), count)
    if got.probs is not None:
        assert (np.abs(got.probs.cpu().numpy() - probs) <= (2.0**-24 + 1e-11) * probs + 2.0**-149).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,K,V,cap", [(1, 64, 33001, 0.0), (5, 200, 1000, 30.0), (70, 256, 4096, 0.0)])
def test_sample_hidden(B, K, V, cap, dtype):
    import nucleus_sampling_amd as ns

    say(f"sample_hidden {dtype} B={B} K={K} V={V} cap={cap}")
    g = torch.Generator(device="cuda").manual_seed(B + V)
    h = torch.randn(B, K, device="cuda", generator=g).to(DT[dtype])
    w = (torch.randn(V, K, device="cuda", generator=g) * (3 / math.sqrt(K))).to(DT[dtype])
    T, p = torch.full((B,), 0.9, device="cuda"), torch.full((B,), 0.95, device="cuda")
    k = torch.full((B,), 300, dtype=torch.int32, device="cuda")
    u = torch.rand(B, 3, device="cuda", generator=g)
    logits = torch.empty(B, V, device="cuda")
    got = ns.sample_hidden(h, w, T, p, k, uniforms=u, softcap=cap, logits=logits, want_probs=True)
    z, tol = _product(h, w)
    if cap:  # (tanh's slope is at most 1; 16 units cover its own and the divide's)
        z = cap * torch.tanh(z / cap)
        tol = tol + z.abs() * 16 * 2.0**-24
    assert ((logits.double().cpu() - z).abs() <= tol).all()
    _drawn(got, logits, T, p, u, k)
    # without uniforms, and on another stream: what sample makes of the same logits
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = ns.sample_hidden(h, w, T, p, k, softcap=cap, seed=7, step=3, stream=side)
    side.synchronize()
    b = ns.sample(logits, T, p, k, seed=7, step=3)
    assert torch.equal(a.token, b.token) and torch.equal(a.keep_count, b.keep_count)


class _Round:
    """A draft block over the last hidden states, the draft's token from its
    head, the target's distribution from the target's head, the verification."""

    def __init__(self, B, K, V, dtype, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(*s, device="cuda", generator=g)
        self.h = n(B, K).to(dtype)
        self.block = (n(K, K) / math.sqrt(K)).to(dtype)
        self.bias = n(K) * 0.1
        self.head = (n(V, K) * (2 / math.sqrt(K))).to(dtype)
        self.T, self.p = torch.full((B,), 0.8, device="cuda"), torch.full((B,), 0.9, device="cuda")
        self.u = torch.rand(B, 4, device="cuda", generator=g, dtype=torch.float64)
        self.draft_logits, self.target_logits = torch.empty(B, V, device="cuda"), torch.empty(B, V, device="cuda")

    def run(self):
        import nucleus_sampling_amd as ns

        drafted = ns.project(self.h, self.block, self.bias, self.h, activation="silu")
        draft = ns.sample_hidden(drafted, self.head, self.T, self.p, uniforms=self.u[:, 0], logits=self.draft_logits,
                                 want_probs=True)
        target = ns.sample_hidden(self.h, self.head, self.T, self.p, uniforms=self.u[:, 1], logits=self.target_logits,
                                  want_probs=True)
        return drafted, draft, target, ns.spec_verify_given(target.probs, draft.probs, draft.token, self.u[:, 2:])


@pytest.mark.parametrize("dtype,B,K,V", [("bf16", 6, 256, 32000), ("f16", 33, 128, 1001), ("f32", 2, 64, 50000)])
def test_a_round_of_speculative_decoding(dtype, B, K, V):
    say(f"speculative round {dtype} B={B} K={K} V={V}")
    r = _Round(B, K, V, DT[dtype], 1)
    drafted, draft, target, verdict = r.run()
    z, tol = _product(r.h, r.block)
    z = z + r.bias.double().cpu()
    want = z * torch.sigmoid(z) + r.h.double().cpu()
    # silu's slope is below 1.1; then 16 units of the activation's value for its
    # own steps and the sum, and half a step of the output's type.
    tol = 1.1 * tol + (z * torch.sigmoid(z)).abs() * 16 * 2.0**-24 + want.abs() * (
        torch.finfo(DT[dtype]).eps / 2 * 1.01 + 2.0**-23) + 1e-7
    assert ((drafted.double().cpu() - want).abs() <= tol).all()
    for hidden, logits, drawn, u in ((drafted, r.draft_logits, draft, r.u[:, 0]), (r.h, r.target_logits, target, r.u[:, 1])):
        z, tol = _product(hidden, r.head)
        assert ((logits.double().cpu() - z).abs() <= tol).all()
        _drawn(drawn, logits, r.T, r.p, u)
    token, accepted = _verify_reference(target.probs.cpu().numpy(), draft.probs.cpu().numpy(), draft.token.cpu().numpy(),
                                        r.u[:, 2:].cpu().numpy())
    assert np.array_equal(verdict.token.cpu().numpy(), token)
    assert np.array_equal(verdict.accepted.cpu().numpy(), accepted)


def test_two_captured_rounds_replayed_in_turn():
    """Two graphs of different sizes, replayed in turn with eager rounds between:
    neither's workspaces are the other's."""
    say("speculative rounds captured")
    rounds = [_Round(6, 256, 32000, torch.bfloat16, 2), _Round(40, 128, 45000, torch.bfloat16, 3)]
    flat = lambda out: [out[0], *(t for part in out[1:] for t in part if t is not None)]
    graphs = []
    for r in rounds:
        r.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = r.run()
        graphs.append((graph, flat(out)))
    for turn in range(3):
        for r in rounds:
            r.h.normal_()
            r.u.uniform_()
        torch.cuda.synchronize()
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        kept = [[t.clone() for t in out] for _, out in graphs]
        for r, out in zip(rounds, kept):
            for a, b in zip(out, flat(r.run())):
                assert torch.equal(a, b), turn
