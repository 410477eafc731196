"""A step of adapters beside a frozen 4-bit projection, as they are used together: rows by token,
the shared 4-bit logits with every request's adapter added, log probabilities and entropies, and
the gradients back to the adapters and the token table, against 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import spmv_storage_formats_amd as spmv  # noqa: E402

U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spmv.load_library()
    return torch.device("cuda:0")


class Model:
    """A token table, a 4-bit projection to logits and adapters of it, all of whole numbers
    times powers of two, so that rows, logits and both inner numbers are exact in fp32."""

    def __init__(self, dev, n, seed, V=700, C=96, L=5, rank=6):
        rng = np.random.default_rng(seed)
        whole = lambda lo, hi, *s: rng.integers(lo, hi, s).astype(np.float64)
        self.table, self.w = whole(-2, 3, V, C), whole(-3, 4, V, C) / 8
        self.down, self.up = whole(-1, 2, L, rank, C) / 8, whole(-1, 2, L, V, rank) / 8
        self.scales = 2.0 ** rng.integers(-2, 1, L)
        self.tokens, self.given = rng.integers(0, V, n), rng.integers(0, V, n)
        self.given[rng.random(n) < 0.2] = -1
        self.of = rng.integers(-1, L, n)
        self.gl, self.gh = rng.normal(0, 1, n), rng.normal(0, 0.1, n)
        t = lambda a, k=torch.float32: torch.from_numpy(a).to(k).to(dev)
        codes = (self.w * 8 + 8).astype(np.uint8)
        self.q = spmv.build_quant_packed(
            torch.from_numpy(codes[:, 0::2] | (codes[:, 1::2] << 4)).to(dev),
            torch.full((V, C // 32), 0.125, device=dev), C, group_size=32)
        self.d = dict(table=t(self.table), down=t(self.down), up=t(self.up), scales=t(self.scales),
                      tokens=t(self.tokens, torch.int64), given=t(self.given, torch.int64),
                      of=t(self.of, torch.int32), gl=t(self.gl), gh=t(self.gh))
        self.V, self.C, self.L = V, C, L

    def step(self, stream=None):
        d = self.d
        x = spmv.lookup(d["table"], d["tokens"], stream=stream)
        y = torch.empty(len(self.tokens), self.V, device=x.device)
        self.q.run(x, y, accumulate=False, stream=stream)
        spmv.adapt(x, d["down"], d["up"], d["of"], y, y, scales=d["scales"], stream=stream)
        r = spmv.token_logprobs(y, d["given"], top=3, stream=stream)
        dy = spmv.token_logprobs_grad(d["gl"], y, d["given"], r.stats, entropy=r.entropy,
                                      grad_entropy=d["gh"], stream=stream)
        dx, ddown, dup = spmv.adapt_grad(dy, x, d["down"], d["up"], d["of"],
                                         scales=d["scales"], stream=stream)
        table = spmv.lookup_grad(dx, d["tokens"], self.V, stream=stream)
        return [y, *r, dy, dx, ddown, dup, table]

    def check(self, got):
        y, lp, h, stats, top_ids, top_lp, dy, dx, ddown, dup, table = (
            g.double().cpu().numpy() for g in got)
        n = len(self.tokens)
        x = self.table[self.tokens]
        want = x @ self.w.T
        hidden = np.zeros((n, self.down.shape[1]))
        for t, a in enumerate(self.of):
            if a >= 0:
                hidden[t] = self.scales[a] * (self.down[a] @ x[t])
                want[t] += self.up[a] @ hidden[t]
        assert np.array_equal(y, want)
        m = want.max(1, keepdims=True)
        e = np.exp(want - m)
        total = np.log(e.sum(1, keepdims=True))
        lpv = want - m - total
        p = np.exp(lpv)
        ent = -(p * lpv).sum(1)
        there = self.given >= 0
        at = np.where(there, self.given, 0)
        # sums of 700 terms below 1 and exponents below 2^9: see the bounds of the operator's
        # own tests, which this exceeds by far
        tol = 1e-4
        assert np.abs(lp - np.where(there, lpv[np.arange(n), at], 0)).max() < tol
        assert np.abs(h - ent).max() < tol
        order = np.lexsort((np.broadcast_to(np.arange(self.V), want.shape), -want))[:, :3]
        assert np.array_equal(top_ids, order)
        assert np.abs(top_lp - np.take_along_axis(lpv, order, 1)).max() < tol
        gl = np.where(there, self.gl.astype(np.float32), 0)
        d = -(gl[:, None] * p) - self.gh.astype(np.float32)[:, None] * p * (lpv + ent[:, None])
        d[np.arange(n), at] += gl
        assert np.abs(dy - d).max() < tol
        # from the gradient that the operator handed on: fp32 sums of at most 700 and n terms
        back, dd, du = np.zeros((n, self.C)), np.zeros(ddown.shape), np.zeros(dup.shape)
        mag = 0.0
        for t, a in enumerate(self.of):
            if a < 0:
                continue
            g = self.scales[a] * (self.up[a].T @ dy[t])
            back[t] = self.down[a].T @ g
            dd[a] += np.outer(g, x[t])
            du[a] += np.outer(dy[t], hidden[t])
            mag = max(mag, np.abs(dy[t]).sum() * 2)
        bound = 2 * (self.V + 200) * U * mag * 100 * n
        for a, b in ((dx, back), (ddown, dd), (dup, du)):
            assert np.abs(a - b).max() <= bound
        want = np.zeros_like(table)
        np.add.at(want, self.tokens, dx)
        assert np.abs(table - want).max() <= 2 * n * U * np.abs(dx).sum()


@pytest.mark.parametrize("n", [1, 9, 40, 300])
def test_step(dev, n):
    model = Model(dev, n, n)
    got = model.step()
    model.check(got)
    assert all(torch.equal(a, b) for a, b in zip(got, model.step()))


def test_loss_falls_as_its_gradient_says(dev):
    """The step's weighted log probabilities and entropies, differentiated along a direction of
    the adapters' matrices by central differences in 64 bits of the definition: with a step of
    2^-10 they agree with the gradients' product with the direction to its square."""
    model = Model(dev, 12, 5)
    *_, ddown, dup, _ = model.step()
    rng = np.random.default_rng(1)
    vd, vu = rng.normal(0, 1, model.down.shape), rng.normal(0, 1, model.up.shape)

    def loss(down, up):
        x = model.table[model.tokens]
        y = x @ model.w.T
        for t, a in enumerate(model.of):
            if a >= 0:
                y[t] += model.scales[a] * (up[a] @ (down[a] @ x[t]))
        z = y - y.max(1, keepdims=True)
        lp = z - np.log(np.exp(z).sum(1, keepdims=True))
        there = model.given >= 0
        own = np.where(there, lp[np.arange(12), np.where(there, model.given, 0)], 0)
        return (model.gl * own).sum() - (model.gh * (np.exp(lp) * lp).sum(1)).sum()

    s = 2.0 ** -12
    diff = (loss(model.down + s * vd, model.up + s * vu)
            - loss(model.down - s * vd, model.up - s * vu)) / (2 * s)
    want = (ddown.double().cpu().numpy() * vd).sum() + (dup.double().cpu().numpy() * vu).sum()
    scale = (np.abs(ddown.double().cpu().numpy()) * np.abs(vd)).sum() + (
        np.abs(dup.double().cpu().numpy()) * np.abs(vu)).sum()
    assert abs(diff - want) <= 1e-3 * scale


def test_step_captured_and_replayed(dev):
    """Two captured steps replayed in turn on other tokens, requests and weights, with eager
    steps between; every replay equals the eager result."""
    models = [Model(dev, 300, 2), Model(dev, 7, 3)]
    graphs = []
    for m in models:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            m.step()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = m.step()
        graphs.append((g, m, out))
    for turn in range(3):
        for g, m, out in graphs:
            other = Model(dev, len(m.tokens), 10 + turn)
            for k in ("tokens", "given", "of", "gl", "down", "up"):
                m.d[k].copy_(other.d[k])
            for t in out:
                t.fill_(3)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, m.step()))


def test_step_on_another_stream(dev):
    model = Model(dev, 60, 4)
    want = model.step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = model.step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
