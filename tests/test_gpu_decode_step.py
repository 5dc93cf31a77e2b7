"""The example's decode step -- deltas, cache, attention, sampling together --
against the same step in 64 bits.

The step rounds to bf16 after each projection and each delta, the rotation, o
and h; the reference rounds its 64-bit values there too, since a rounded score
between two strong keys moves o by several per cent.  What is left is a value
now and then that rounds the other way, and the weights' rounding: 2^-4 of the
logits' rms bounds them, and 2^-8 of a logit its own rounding.  The mistakes
that the step could make (adapters, rotation or prompt left out) move logits of
some request by more than 2^-2 of the rms, which the test shows on the
reference, early, while the prompt outweighs the requests' own tokens.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def built():
    from tenant_composite_lora_gb300 import build
    build.build()


def rotate(x, positions, rope):
    """x [T, heads, d]; pairs are half of d apart."""
    h = x.shape[-1] // 2
    c, s = rope[positions][:, None, :h], rope[positions][:, None, h:]
    return torch.cat([x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s], -1)


class Reference:
    @staticmethod
    def r(t):
        return t.to(torch.bfloat16).double()

    def __init__(self, m, adapters=True, rotation=True, prompt=True):
        self.m, self.adapters, self.prompt = m, adapters, prompt
        f = lambda t: t.double().cpu()
        self.emb, self.head, self.w = f(m.emb), f(m.head), {n: f(w) for n, w in m.w.items()}
        self.rope = f(m.rope)
        if not rotation:
            self.rope[:, :m.d // 2], self.rope[:, m.d // 2:] = 1.0, 0.0
        x = self.emb[m.prompt.cpu()]
        n = x.shape[0]
        self.pk = self.r(rotate(self.r(x @ self.w["k"]).view(n, m.hkv, m.d), torch.arange(n), self.rope))
        self.pv = self.r(x @ self.w["v"]).view(n, m.hkv, m.d)
        self.k, self.v, self.at = [], [], n

    def project(self, n, x, add=0.0):
        y = self.r(add + x @ self.w[n])
        if self.adapters:
            for b in range(self.m.B):
                for i, alpha in zip(self.m.ids[b].tolist(), self.m.alpha[b].tolist()):
                    A, B = (t.double() for t in self.m.factors[n][i])
                    r = int(self.m.ranks[i])
                    y[b] += alpha * (x[b] @ A[:, :r]) @ B[:r]
        return self.r(y)

    def step(self, tokens):
        m = self.m
        x = self.emb[tokens.long()]
        at = torch.full((m.B,), self.at)
        q = self.r(rotate(self.project("q", x).view(m.B, m.hq, m.d), at, self.rope))
        self.k.append(self.r(rotate(self.project("k", x).view(m.B, m.hkv, m.d), at, self.rope)))
        self.v.append(self.project("v", x).view(m.B, m.hkv, m.d))
        self.at += 1
        o = torch.zeros(m.B, m.hq, m.d, dtype=torch.float64)
        for b in range(m.B):
            keys, values = torch.stack([k[b] for k in self.k]), torch.stack([v[b] for v in self.v])
            if self.prompt:
                keys, values = torch.cat([self.pk, keys]), torch.cat([self.pv, values])
            for h in range(m.hq):
                g = h * m.hkv // m.hq
                o[b, h] = torch.softmax(keys[:, g] @ q[b, h] * m.d ** -0.5, 0) @ values[:, g]
        o = self.r(o.view(m.B, -1))
        return self.project("o", o, x) @ self.head


def interval(l, tau, k, p, token):
    """The token's part of the kept mass, by the definition in 64 bits."""
    order = np.argsort(-l, kind="stable")[:k or None]
    e = np.exp((l[order] - l[order[0]]) / tau)
    kept = np.cumsum(e) - e < p * e.sum()
    order, e = order[kept], e[kept]
    by = np.argsort(order)
    order, c = order[by], np.cumsum(e[by]) / e.sum()
    at = int(np.flatnonzero(order == token)[0])
    return (c[at - 1] if at else 0.0), c[at]


@pytest.mark.parametrize("requests,prompt,heads", [(1, 5, dict(hq=2, hkv=2, d=128)), (5, 37, {}),
                                                   (33, 200, dict(hq=8, hkv=1, page=32))])
def test_steps_match_the_reference(requests, prompt, heads):
    from examples.decode_step import DecodeStep
    m = DecodeStep(requests, prompt, 20, vocab=1003, hidden=256, **heads)
    ref, draw = Reference(m), torch.Generator().manual_seed(requests)
    wrong = [Reference(m, **{x: False}) for x in ("adapters", "rotation", "prompt")]
    for step in range(18):  # over the end of a page
        tokens = m.tokens.cpu()
        logits = m.step().double().cpu()
        m.check()
        want = ref.step(tokens)
        rms = float(want.square().mean().sqrt())
        assert float(((logits - want).abs() - 2 ** -8 * want.abs()).max()) < 2 ** -4 * rms
        if step == 3 and requests > 1:
            for w in wrong:
                w.k, w.v, w.at = list(ref.k[:-1]), list(ref.v[:-1]), ref.at - 1
                assert float((w.step(tokens) - want).abs().max()) > 2 ** -2 * rms
        for b, token in enumerate(m.tokens.tolist()):
            lo, hi = interval(logits[b].numpy(), *(float(x[b]) for x in (m.temperature,)), int(m.top_k[b]),
                              float(m.top_p[b]), token)
            assert lo - 1e-5 <= float(m.u[b]) <= hi + 1e-5
        m.u.copy_(torch.rand(requests, generator=draw))


def test_a_captured_step_gives_the_same_tokens():
    from examples.decode_step import DecodeStep
    a, b = (DecodeStep(9, 50, 12, vocab=1003, hidden=256) for _ in range(2))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b.step()
    torch.cuda.synchronize()
    a.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    for _ in range(8):
        a.step()
        graph.replay()
        assert torch.equal(a.tokens, b.tokens)
    a.check()
    b.check()
