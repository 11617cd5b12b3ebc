"""The layer calls together, as a training program over M workers uses them: one
pass over the joined batch (lookup, layer norm, tied output product,
distillation loss, and back) leaves every worker's gradient in its G[m], and
signmuon_step takes them.  Held against M separate float64 passes; captured
into a CUDA graph; on streams of their own."""
import numpy as np
import pytest

from oracle import signmuon_ref as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import sign_muon_optimizer_b200 as smo  # noqa: E402

V, E, K, ROWS = 97, 48, 4, [13, 0, 29, 7]
M, N = len(ROWS), sum(ROWS)
SHAPES = [(V, E), (1, E), (1, E)]
SCALE, T, EPS = 2.0, 2.0, 1e-5
BOUNDS = [slice(sum(ROWS[:m]), sum(ROWS[:m + 1])) for m in range(M)]


class Pass:
    """The buffers of one pass and its calls, on the handle's stream."""

    def __init__(self, stream=None, flags=0):
        self.opt = smo.SignMuon(SHAPES, M, beta=0.9, lam=0.0, K=0, eps=1e-7, scale="fro",
                                flags=smo.SIGNMUON_TERNARY | flags, stream=stream)
        self.opt.layers_reserve(N, E)
        z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
        self.W = z((self.opt.d + 3) // 4 * 4)
        self.G = [z((self.opt.d + 3) // 4 * 4) for _ in range(M)]
        self.ids, self.idx = z(N, dtype=torch.int64), z(N, K, dtype=torch.int32)
        self.t = z(N, K)
        self.X, self.Y, self.dY, self.Z = z(N, E), z(N, E), z(N, E), z(N, V)
        self.mean, self.rstd, self.loss = z(N), z(N), z(M)

    def fill(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = torch.randn(self.opt.d, generator=g, device="cuda") * 0.5
        w[V * E:V * E + E] += 1
        self.W[:self.opt.d] = w
        self.ids.copy_(torch.randint(0, V // 2, (N,), generator=g, device="cuda"))
        self.idx.copy_(torch.randint(0, V, (N, K), generator=g, device="cuda"))
        self.idx[3] = -1
        self.t.copy_(torch.randn(N, K, generator=g, device="cuda"))
        return self

    def gradients(self):
        opt, W = self.opt, self.W
        table = W[:V * E].view(V, E)
        opt.embed(W, 0, self.ids, self.X, scale=SCALE)
        opt.layernorm(W, 1, 2, self.X, self.Y, self.mean, self.rstd, eps=EPS)
        torch.mm(self.Y, table.t(), out=self.Z)
        opt.distill(self.Z, self.idx, self.t, self.loss, ROWS, dZ=self.Z, temperature=T)      # in place
        torch.mm(self.Z, table, out=self.dY)
        for m, s in enumerate(BOUNDS):                # the output product's share of the table's gradient
            torch.mm(self.Z[s].t(), self.Y[s], out=self.G[m][:V * E].view(V, E))
        opt.layernorm_grad(W, 1, 2, self.X, self.dY, self.mean, self.rstd, self.dY, self.G, ROWS)
        opt.embed_grad(0, self.ids, self.dY, self.G, ROWS, scale=SCALE, accumulate=True)

    def step(self, eta=0.01):
        self.gradients()
        self.opt.step(self.W, self.G, eta)


def exact(p):
    """Every worker's loss and gradient by autograd in float64, a pass each."""
    losses, grads = [], []
    for s in BOUNDS:
        w = p.W[:p.opt.d].cpu().double().requires_grad_(True)
        table, gamma, beta = w[:V * E].view(V, E), w[V * E:V * E + E], w[V * E + E:V * E + 2 * E]
        x = table[p.ids[s].cpu()] * SCALE
        y = torch.nn.functional.layer_norm(x, (E,), gamma, beta, EPS)
        lp = torch.log_softmax(y @ table.t() / T, 1)
        idx, t = p.idx[s].cpu().long(), p.t[s].cpu().double()
        some = (idx >= 0).all(1)
        q = torch.softmax(t / T, 1)
        rows = (q * (q.log() - lp.gather(1, idx.clamp(min=0)))).sum(1) * T * T
        loss = (rows * some).sum() / max(1, int(some.sum()))
        if s.stop > s.start:
            loss.backward()
        losses.append(float(loss.detach()))
        grads.append(np.zeros(p.opt.d) if w.grad is None else w.grad.numpy())
    return losses, grads


# Each of the six float32 calls and three products is off by at most about
# (terms / 32 + 60) roundings of its terms' absolute sum, below 70 for the
# 97-term sums here; the parts of dX cancel to no less than a tenth.  Nine such
# stages, each of gain near 1 on the scale of the block's largest gradient:
# 9 * 70 * 10 * 2^-24 = 3.8e-4 of it.
TOL = 3.8e-4


def test_gradients_of_every_worker_from_one_pass():
    p = Pass().fill(1)
    p.gradients()
    p.opt.layers_sync()
    losses, grads = exact(p)
    for m in range(M):
        assert abs(float(p.loss[m]) - losses[m]) <= TOL * (1 + abs(losses[m]))
        got = p.G[m][:p.opt.d].cpu().double().numpy()
        off = 0
        for r, c in SHAPES:
            a, b = got[off:off + r * c], grads[m][off:off + r * c]
            assert np.abs(a - b).max() <= TOL * np.abs(b).max(), f"worker {m}, matrix at {off}"
            off += r * c


def test_step_on_the_gradients():
    """The vote and the update from them: where every worker's gradient is
    clearly off zero, or exactly zero, W moves as the oracle says."""
    p = Pass().fill(2)
    w0 = p.W[:p.opt.d].cpu().numpy().copy()
    p.step()
    p.opt.sync()
    q = Pass().fill(2)
    _, grads = exact(q)
    want = oracle.step(w0, [g.astype(np.float32) for g in grads], [np.zeros(p.opt.d, np.float32)] * M, SHAPES, beta=0.9,
                       lam=0.0, eta=0.01, K=0, eps=1e-7, scale="fro", signs="ternary")
    clear = np.ones(p.opt.d, bool)
    for g in grads:
        off = 0
        for r, c in SHAPES:
            b = np.abs(g[off:off + r * c])
            clear[off:off + r * c] &= (b > TOL * b.max()) | (b == 0)
            off += r * c
    # (of the exact gradients alone: the rows that no entry points to get only the
    # small p of the output product, below TOL of the largest in some worker)
    assert clear.sum() > 500
    got = p.W[:p.opt.d].cpu().numpy()
    assert np.array_equal(got[clear], want["W"].astype(np.float32)[clear])


def test_the_pass_and_step_replay_from_a_cuda_graph():
    eager, seeds = Pass(flags=smo.SIGNMUON_ASYNC), (5, 6, 7)
    want = []
    for s in seeds:
        eager.fill(s)
        eager.step()
        eager.opt.sync()
        want.append([x.clone() for x in (eager.W, eager.loss, *eager.G)])
    stream = torch.cuda.Stream()
    p = Pass(stream=stream.cuda_stream, flags=smo.SIGNMUON_ASYNC).fill(4)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        p.gradients()                                  # cuBLAS and the kernels are loaded before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        p.step()
    for s, w in zip(seeds, want):
        with torch.cuda.stream(stream):
            p.fill(s)
            g.replay()
        stream.synchronize()
        p.opt.sync()
        p.opt.layers_sync()
        for a, b in zip((p.W, p.loss, *p.G), w):
            assert torch.equal(a, b)


def test_two_handles_on_two_streams_at_once():
    alone = Pass().fill(9)
    alone.gradients()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ps = [Pass(stream=s.cuda_stream).fill(9) for s in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s in zip(ps, streams):
            with torch.cuda.stream(s):
                p.gradients()
    torch.cuda.synchronize()
    for p in ps:
        p.opt.layers_sync()
        for a, b in zip((p.loss, *p.G), (alone.loss, *alone.G)):
            assert torch.equal(a, b)


def test_calls_follow_one_another_at_once():
    """A call's kernels may start while the one before still ends: a chain in
    which each call reads what the one before wrote, over the same buffers, run
    many times, gives the same bits as with a wait after every call."""
    p = Pass().fill(11)
    opt, W = p.opt, p.W
    out = []
    for wait in (True, False):
        p.fill(11)
        for k in range(30):
            for call in (lambda: opt.embed(W, 0, p.ids, p.X, scale=SCALE + k),
                         lambda: opt.layernorm(W, 1, 2, p.X, p.Y, p.mean, p.rstd),
                         lambda: opt.layernorm_grad(W, 1, 2, p.X, p.Y, p.mean, p.rstd, p.dY, p.G, ROWS),
                         lambda: opt.embed_grad(0, p.ids, p.dY, p.G, ROWS),
                         lambda: opt.apply_update(W, p.G[0], opt.d, 1e-3),
                         lambda: opt.layernorm(W, 2, 1, p.dY, p.X),
                         lambda: opt.distill(p.X, p.idx, p.t, p.loss, ROWS, dZ=p.X)):
                call()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        out.append([x.clone() for x in (p.W, p.X, p.Y, p.dY, p.loss, p.mean, p.rstd, *p.G)])
    with pytest.raises(smo.SignMuonError):             # entries at 48 ... 96 point beyond the 48 columns of X
        opt.layers_sync()
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_reserve_and_refusals_of_a_handle():
    opt = smo.SignMuon([(10, 8), (1, 8), (2, 4), (1, 9)], 2, flags=smo.SIGNMUON_VOTE_ONLY)
    W = torch.zeros(opt.d, device="cuda")
    X = torch.zeros(6, 8, device="cuda")
    ids = torch.zeros(6, dtype=torch.int64, device="cuda")
    G = [torch.zeros(opt.d + 3, device="cuda") for _ in range(2)]
    mean = torch.zeros(6, device="cuda")

    def refused(status, call, *a, **k):
        with pytest.raises(smo.SignMuonError) as e:
            call(*a, **k)
        assert e.value.status == status, e.value

    U, I = smo.SIGNMUON_E_UNSUPPORTED, smo.SIGNMUON_E_INVALID  # noqa: E741
    refused(U, opt.embed, W, 0, ids, X)                        # nothing reserved
    refused(U, opt.layers_sync)
    for bad in ((0, 8), (4, 0), (1 << 31, 8), (4, 1 << 31)):
        refused(I, opt.layers_reserve, *bad)
    before = opt.info["device_bytes"]
    opt.layers_reserve(4, 8)
    assert smo.signmuon_info(opt.h)["device_bytes"] > before
    bytes4 = smo.signmuon_info(opt.h)["device_bytes"]
    opt.layers_reserve(3, 5)                                   # smaller: nothing to do
    assert smo.signmuon_info(opt.h)["device_bytes"] == bytes4
    refused(I, opt.embed_grad, 0, ids, X, G)                   # 6 rows
    refused(I, opt.layernorm_grad, W, 1, None, X, X.clone(), mean, mean, X.clone(), G)
    opt.layers_reserve(6, 8)
    opt.embed_grad(0, ids, X, G)
    opt.embed(W, 0, ids, X)
    # gamma and beta of other sizes, the same matrix twice, a row too wide
    Y = torch.zeros(6, 8, device="cuda")
    opt.layernorm(W, 1, 2, X, Y)                               # 1 x 8 and 2 x 4: the same size
    refused(I, opt.layernorm, W, 1, 3, X, Y)
    refused(I, opt.layernorm, W, 1, 1, X, Y)
    refused(I, opt.layernorm, W, 1, 2, X, Y, eps=0.0)
    refused(I, opt.layernorm, W, 1, 2, X, Y, mean=mean)        # rstd missing
    refused(I, opt.embed, W[1:1 + opt.d] if W.numel() > opt.d else torch.zeros(opt.d + 1, device="cuda")[1:], 0, ids, X)
    refused(I, opt.embed_grad, 0, ids, X, [g[1:] for g in G])  # misaligned vectors
    refused(I, opt.embed_grad, 0, ids, X, G, rows=[7, -1])
    both = torch.zeros(2 * opt.d, device="cuda")
    refused(I, opt.embed_grad, 0, ids, X, [G[0], G[0]])        # two workers' gradients in the same place
    refused(I, opt.embed_grad, 0, ids, X, [both, both[opt.d // 4 * 4 - 4:][:opt.d]])
    loss, t, idx = torch.zeros(2, device="cuda"), torch.zeros(6, 2, device="cuda"), torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-45, 1e-19, 1e19):
        refused(I, opt.distill, X, idx, t, loss, temperature=bad)
    refused(U, opt.distill, X, torch.zeros(6, 1025, dtype=torch.int32, device="cuda"), torch.zeros(6, 1025, device="cuda"), loss)
    big = torch.zeros(12, 8, device="cuda")
    refused(I, opt.distill, big[::2], idx, t, loss, dZ=big.view(-1)[:48].view(6, 8))   # the same memory, another stride
    refused(I, opt.layernorm_grad, W, 1, None, X, big[::2], mean, mean, big.view(-1)[:48].view(6, 8), G)
    # outputs per worker are written for no rows too
    none = torch.zeros(0, 8, device="cuda"), torch.zeros(0, 2, dtype=torch.int32, device="cuda"), torch.zeros(0, 2, device="cuda")
    ints = torch.zeros(4, dtype=torch.int32, device="cuda")
    for where in (1, 2, 3):
        with pytest.raises(smo.SignMuonError):
            smo.signmuon_distill(opt.h, none[0].data_ptr(), 0, 8, 8, none[1].data_ptr(), 0, none[2].data_ptr(), 0, 2, 2,
                                 [0, 0], 1.0, 1.0, loss, ints.data_ptr() + where, None, None, 8)
    wide = smo.SignMuon([(1, smo.SIGNMUON_LAYERNORM_MAX_COLS + 1)], 1, flags=smo.SIGNMUON_VOTE_ONLY)
    wide.layers_reserve(1, 8)
    x = torch.zeros(1, wide.d, device="cuda")
    refused(U, wide.layernorm, torch.zeros(wide.d, device="cuda"), 0, None, x, x.clone())
    opt.layers_sync()


def test_a_graph_keeps_its_workspace_when_more_is_reserved():
    stream = torch.cuda.Stream()
    p = Pass(stream=stream.cuda_stream).fill(5)
    torch.cuda.synchronize()

    def check():
        stream.synchronize()
        for a, b in zip(p.G, want):
            assert torch.equal(a[:p.opt.d], b[:p.opt.d])
            a.fill_(float("nan"))
        torch.cuda.synchronize()

    with torch.cuda.stream(stream):
        p.gradients()
        want = [g.clone() for g in p.G]
        check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        p.gradients()
    p.opt.layers_reserve(40 * N, 3 * E)
    for _ in range(2):
        with torch.cuda.stream(stream):
            graph.replay()
            check()
            p.gradients()                          # the same handle's calls, in the new workspace
            check()
    p.opt.layers_sync()


@pytest.mark.parametrize("shift", [0, 1])
def test_offsets_beyond_32_bits(shift):
    """Three rows 2^30 elements apart, at byte offsets up to 2^32: the same bits
    as the rows next to each other."""
    n, v, e, ld, ld_near = 3, 90, 64, (1 << 30) + 8 + shift, 128 + shift
    opt = smo.SignMuon([(v, e), (1, e), (1, e)], 1, flags=smo.SIGNMUON_VOTE_ONLY)
    opt.layers_reserve(n, e)
    g = torch.Generator(device="cuda").manual_seed(3)
    W = torch.randn(opt.d, generator=g, device="cuda")
    ids = torch.tensor([4, 89, 4], device="cuda")
    idx, t = torch.tensor([[1, 2], [80, 3], [5, -1]], device="cuda"), torch.randn(n, 2, generator=g, device="cuda")
    logits = torch.randn(n, v, generator=g, device="cuda").bfloat16()
    store = [torch.empty(2 * ld + 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    results = []
    for stride in (ld_near, ld):
        def make(i, cols):
            return store[i].as_strided((n, cols), (stride, 1))

        a, b = make(0, e), make(1, e)
        G = [torch.full((opt.d,), float("nan"), device="cuda")]
        mean, rstd, loss = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(1, device="cuda")
        opt.embed(W, 0, ids, a)
        got = [a.clone()]
        opt.layernorm(W, 1, 2, a, b, mean, rstd)
        got += [b.clone(), mean, rstd]
        opt.layernorm_grad(W, 1, 2, a, b, mean, rstd, b, G)
        got += [b.clone()]
        opt.embed_grad(0, ids, b, G)
        got += [G[0]]
        z, dz = make(0, v), make(1, v)
        z.copy_(logits)
        opt.distill(z, idx, t, loss, dZ=dz)
        results.append(got + [dz.clone(), loss])
        opt.layers_sync()
    for x, y in zip(*results):
        assert torch.equal(x, y)
