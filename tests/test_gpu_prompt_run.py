"""The prompt operators together, as a target's pass over packed prompts uses them: norm
with the residual, e4m3 projection, cache write, attention, then the final norm, the
vocabulary's projection and verification; the same on another stream and in a replayed
graph."""

import numpy as np
import pytest
import torch

import draft_token_verification_04_amd as sv
from gpu_helpers import dev, ints_to_dev, note

pytestmark = pytest.mark.gpu
H, HKV, D, PAGE, V = 8, 2, 64, 16, 1000
HIDDEN = H * D


def _weights(g, n, k):
    w = torch.randn(n, k, generator=g, device=dev()) / k ** 0.5
    nb, kb = -(-n // 128), -(-k // 128)
    full = torch.nn.functional.pad(w, (0, kb * 128 - k, 0, nb * 128 - n))
    s = full.view(nb, 128, kb, 128).abs().amax((1, 3)) / 448
    q = (full / s.repeat_interleave(128, 0).repeat_interleave(128, 1)).to(torch.float8_e4m3fn)[:n, :k].contiguous()
    return q, s.contiguous()


def _values(w, s):
    return w.double() * s.double().repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :w.shape[1]]


class Layer:
    def __init__(self, seed, lengths, base, kind):
        g = torch.Generator(device=dev())
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        B = len(lengths)
        self.starts_ = np.concatenate([[0], np.cumsum(lengths)])
        self.base_, self.lengths = np.array(base), lengths
        T = int(self.starts_[-1])
        P = -(-int(np.max(self.base_ + lengths)) // PAGE)
        self.table_ = rng.permutation(B * P).reshape(B, P)
        self.starts, self.base, self.table = (ints_to_dev(x) for x in (self.starts_, self.base_, self.table_))
        self.positions = ints_to_dev(np.concatenate([b + np.arange(n) for b, n in zip(base, lengths)]))
        self.x = torch.randn(T, HIDDEN, generator=g, device=dev()).bfloat16()
        self.residual = torch.randn(T, HIDDEN, generator=g, device=dev()).bfloat16()
        self.norms = [(1 + 0.1 * torch.randn(HIDDEN, generator=g, device=dev())).bfloat16() for _ in range(2)]
        self.head_norms = [(1 + 0.1 * torch.randn(D, generator=g, device=dev())).bfloat16() for _ in range(2)]
        self.qkv, self.head = _weights(g, (H + 2 * HKV) * D, HIDDEN), _weights(g, V, HIDDEN)
        angle = torch.arange(400, device=dev())[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device=dev()) / D)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float()
        dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
        # what lies in the cache before: small random values
        self.k = (torch.randn(B * P, HKV, PAGE, D, generator=g, device=dev())).to(dt)
        self.v = (torch.randn(B * P, HKV, PAGE, D, generator=g, device=dev())).to(dt)
        self.scales = [None if kind == "bf16" else torch.full((B * P, HKV, PAGE), 0.5, device=dev()) for _ in range(2)]
        self.cache = sv.PagedKV(self.k, self.v, *self.scales)

    def run(self, stream=None):
        kw = dict(stream=stream)
        a = sv.spec_rms_norm(self.x, self.norms[0], residual=self.residual, e4m3=True, **kw)
        qkv = sv.spec_linear_e4m3(a["out"], a["scales"], *self.qkv, **kw)
        heads = qkv.unflatten(-1, (H + 2 * HKV, D))
        p = sv.spec_append_kv_packed(heads[:, :H], heads[:, H:H + HKV], heads[:, H + HKV:], self.cache, self.table,
                                     self.starts, self.base, self.positions, q_weight=self.head_norms[0],
                                     k_weight=self.head_norms[1], rope=self.rope, **kw)
        o = sv.spec_attend_packed(p["q"], self.cache, self.table, self.starts, self.base, lse=True, **kw)
        f = sv.spec_rms_norm(o["out"].flatten(1), self.norms[1], residual=a["residual"], e4m3=True, **kw)
        logits = sv.spec_linear_e4m3(f["out"], f["scales"], *self.head, out_dtype=torch.float32, **kw)
        return dict(a=a, qkv=qkv, p=p, o=o, f=f, logits=logits)


def _read(pages, scales, table, n):
    slots = torch.arange(n, device=dev())
    pg, row = torch.as_tensor(table, device=dev()).long()[slots // PAGE], slots % PAGE
    x = pages.view(torch.uint8)[pg, :, row].view(pages.dtype).double() if scales is not None else pages[pg, :, row].double()
    return x if scales is None else x * scales[pg, :, row].double()[..., None]


def _check(c, r):
    """Each step against 64 bits of its own inputs."""
    h = c.x.double() + c.residual.double()
    assert ((r["a"]["residual"].double() - h).abs() <= 2.0 ** -8 * h.abs() * 1.001).all()
    x = r["a"]["out"].double() * r["a"]["scales"].double().t().repeat_interleave(128, 1)[:, :HIDDEN]
    y = h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * c.norms[0].double()
    s = r["a"]["scales"].double().t().repeat_interleave(128, 1)[:, :HIDDEN]
    assert ((x - y).abs() <= (2.0 ** -4 + 2.0 ** -14) * y.abs() + 2.0 ** -9 * s).all()
    want = x @ _values(*c.qkv).t()
    assert ((r["qkv"].double() - want).norm() <= 2.0 ** -8 * want.norm())
    assert (r["p"]["status"] == 0).all() and (r["o"]["status"] == 0).all()
    for b, n in enumerate(c.lengths):
        if n == 0:
            continue
        at = slice(int(c.starts_[b]), int(c.starts_[b]) + n)
        total = int(c.base_[b]) + n
        k, v = (_read(p, s, c.table_[b], total) for p, s in ((c.k, c.scales[0]), (c.v, c.scales[1])))
        k, v = (t.repeat_interleave(H // HKV, 1).transpose(0, 1) for t in (k, v))
        w = torch.matmul(r["p"]["q"][at].double().transpose(0, 1), k.transpose(1, 2).contiguous()) * D ** -0.5
        unseen = torch.arange(total, device=dev())[None, :] > int(c.base_[b]) + torch.arange(n, device=dev())[:, None]
        w = w.masked_fill(unseen, -float("inf"))
        want = torch.matmul(torch.softmax(w, -1), v).transpose(0, 1)
        assert (r["o"]["out"][at].double() - want).norm() <= 2.0 ** -7 * want.norm()
        assert (r["o"]["lse"][at].double() - torch.logsumexp(w, -1).t()).abs().max() <= 1e-4
    x = r["f"]["out"].double() * r["f"]["scales"].double().t().repeat_interleave(128, 1)[:, :HIDDEN]
    want = x @ _values(*c.head).t()
    assert ((r["logits"].double() - want).norm() <= 2.0 ** -19 * want.norm())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_layer_and_the_logits_of_packed_prompts(kind):
    note(f"prompt run {kind}")
    c = Layer(3, [70, 0, 33, 130, 1], [0, 0, 20, 7, 150], kind)
    r = c.run()
    _check(c, r)
    # the logits of the last tokens go to greedy verification of one draft each
    rows = torch.tensor([68, 69, 101, 102, 231, 232], device=dev())
    target = r["logits"][rows].view(3, 2, V).contiguous()
    drafts = target[:, 0].argmax(1, keepdim=True).to(torch.int32)
    g = sv.spec_verify_greedy(target, drafts)
    assert (g["accept_len"] == 1).all() and torch.equal(g["tokens"][:, 1], target[:, 1].argmax(1).to(torch.int32))


def test_on_another_stream():
    note("prompt run side stream")
    c = Layer(4, [40, 90], [0, 30], "bf16")
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=s)
    junk = [torch.full((133, 2000), float("nan"), device=dev()) for _ in range(8)]  # blocks freed too early would be hit
    s.synchronize()
    assert torch.equal(got["logits"], want["logits"]) and torch.equal(got["o"]["out"], want["o"]["out"]) and junk


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_captured_and_replayed_with_other_lengths(kind):
    note(f"prompt run graph {kind}")
    c = Layer(5, [64, 50, 30], [0, 40, 3], kind)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = c.run()
    for lengths, base in (([64, 50, 30], [0, 40, 3]), ([20, 60, 64], [44, 4, 0]), ([0, 90, 54], [9, 0, 36])):
        c.lengths, c.base_ = lengths, np.array(base)
        c.starts_ = np.concatenate([[0], np.cumsum(lengths)])
        c.starts.copy_(ints_to_dev(c.starts_))
        c.base.copy_(ints_to_dev(base))
        c.positions.copy_(ints_to_dev(np.concatenate([b + np.arange(n) for b, n in zip(base, lengths)])))
        graph.replay()
        torch.cuda.synchronize()
        _check(c, r)
        eager = c.run()
        torch.cuda.synchronize()
        assert torch.equal(eager["logits"], r["logits"]) and torch.equal(eager["o"]["out"], r["o"]["out"])
