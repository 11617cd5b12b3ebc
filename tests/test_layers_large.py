"""The forms of the layer calls that only larger batches reach: the table
gradient's units of 32 tokens a warp, layer norm with several rows a block,
its gradient with a reduction of its own, and the distillation of more rows than
few with 256 and 512 threads a row.  Held against float64 forms; the bounds are
those of layers_ref, and every call made twice gives the same bits."""
import numpy as np
import pytest

import layers_ref as ref
from layers_ref import DT, U

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import sign_muon_optimizer_b200 as smo  # noqa: E402


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def handle(shapes, M, rows, cols):
    opt = smo.SignMuon(shapes, M, flags=smo.SIGNMUON_VOTE_ONLY)
    opt.layers_reserve(rows, cols)
    return opt


def worker_of(rows):
    return torch.repeat_interleave(torch.arange(len(rows), device="cuda"), torch.tensor(rows, device="cuda"))


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: got {float(got[i])!r}, "
                             f"wanted {float(want[i])!r} within {float(tol[i]):.3g}")


def vectors(opt):
    n = (opt.d + 3) // 4 * 4
    buf = torch.full((opt.M, n), float("nan"), device="cuda")
    return buf, [buf[m] for m in range(opt.M)]


# ---- embedding -------------------------------------------------------------------

@pytest.mark.parametrize("dt,E", [("f32", 768), ("bf16", 768), ("f16", 1001)])
def test_embed_of_more_tokens_than_go_at_once(dt, E):
    n, V = 30011, 501
    opt = handle([(V, E)], 1, 1, E)
    W = torch.randn(opt.d, generator=gen(1), device="cuda")
    ids = torch.randint(-3, V, (n,), generator=gen(2), device="cuda")
    out = torch.full((n, E), float("nan"), dtype=DT[dt], device="cuda")
    opt.embed(W, 0, ids, out, scale=1.7)
    opt.layers_sync()
    want = torch.where((ids >= 0)[:, None], W[:V * E].view(V, E)[ids.clamp(min=0)] * 1.7, 0.0).to(DT[dt])
    assert torch.equal(out, want)


def token_ids(kind, n, V, g):
    if kind == "same":
        return torch.full((n,), V // 2, device="cuda")
    if kind == "lengths":            # runs that end before, at and behind the borders of 32 and 256 tokens
        c = torch.tensor([1, 31, 32, 33, 64, 1, 95, 255, 256, 257, 2, 512, 30, 770], device="cuda")
        ids = torch.repeat_interleave(torch.arange(len(c), device="cuda"), c)
        ids = ids.repeat(n // len(ids) + 1)[:n]
        return ids[torch.randperm(n, generator=g, device="cuda")]
    if kind == "zipf":
        return ((V + 1.0) ** torch.rand(n, generator=g, device="cuda", dtype=torch.float64)).long().clamp(1, V) - 1
    return torch.randint(0, V, (n,), generator=g, device="cuda")


# A warp takes 32 tokens where (rows / 256) strips of 512 bytes are more than 400,
# else 8: 102655 rows of one strip are the last ones with 8, 102656 the first with 32.
@pytest.mark.parametrize("dt,rows,V,E,kind,accumulate", [
    ("bf16", [20000, 0, 15001, 255], 900, 768, "zipf", False),
    ("f16", [30001, 9], 77, 1001, "random", False),
    ("f32", [18001, 0, 257], 300, 772, "zipf", True),
    ("f32", [102655], 40, 4, "random", False),
    ("f32", [102656], 40, 4, "random", False),
    ("f32", [60000, 43001], 1200, 3, "zipf", True),
    ("bf16", [35072, 33], 20, 768, "lengths", False),
    ("bf16", [35001], 5, 776, "same", False),
    ("bf16", [52000, 52000], 2, 24, "same", False),
    ("f16", [2000] * 60, 1001, 33, "random", False),
])
def test_table_gradient_with_32_tokens_a_warp(dt, rows, V, E, kind, accumulate):
    n, M = sum(rows), len(rows)
    opt = handle([(1, 6), (V, E), (1, 3)], M, n, E)
    g = gen(n + V)
    ids = token_ids(kind, n, V, g)
    ids[3::701] = -5
    dY = torch.randn(n, E, generator=g, device="cuda").to(DT[dt])
    scale = float(np.float32(0.37))
    got = []
    for _ in range(2):
        G, Gm = vectors(opt)
        old = torch.randn(M, V * E, generator=gen(7), device="cuda")
        if accumulate:
            G[:, 6:6 + V * E] = old
        opt.embed_grad(1, ids, dY, Gm, rows, scale=scale, accumulate=accumulate)
        opt.layers_sync()
        assert bool(G[:, :6].isnan().all()) and bool(G[:, 6 + V * E:].isnan().all())
        got.append(G[:, 6:6 + V * E])
    assert torch.equal(*got)
    keep = ids >= 0
    at = (worker_of(rows) * V + ids)[keep]
    d = dY[keep].double()
    want = torch.zeros(M * V, E, dtype=torch.float64, device="cuda").index_add_(0, at, d) * scale
    tol = torch.zeros_like(want).index_add_(0, at, d.abs()) * scale
    tol *= (torch.bincount(at, minlength=M * V)[:, None] + 2) * U
    if accumulate:
        want += old.view(M * V, E)
        tol = torch.where(tol > 0, tol + U * want.abs(), 0)
    close(got[0].reshape(M * V, E), want, tol, "G")


# ---- layer norm --------------------------------------------------------------------

def norm_inputs(n, E, dt, g):
    X = torch.randn(n, E, generator=g, device="cuda") * 2 + 3
    X[1] = 1.5
    X[2] *= 30
    return X.to(DT[dt])


@pytest.mark.parametrize("dt,n,E", [
    ("f32", 20011, 768), ("bf16", 20011, 768), ("f16", 30011, 96), ("bf16", 20011, 1001), ("bf16", 9001, 1536),
    ("f32", 6001, 4096), ("bf16", 6001, 5000), ("f16", 3001, 8192), ("f32", 2001, 16384), ("bf16", 3001, 16384),
    ("bf16", 2001, 16383)])
def test_layernorm_of_more_rows_than_go_at_once(dt, n, E):
    opt = handle([(1, E), (1, E)], 1, 1, 1)
    W = torch.randn(opt.d, generator=gen(5), device="cuda")
    X = norm_inputs(n, E, dt, gen(E))
    Y = torch.full_like(X, float("nan"))
    mean, rstd = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    opt.layernorm(W, 0, 1, X, Y, mean, rstd, eps=1e-5)
    opt.layers_sync()
    x, gamma, beta = X.double(), W[:E].double(), W[E:2 * E].double()
    k = ref.depth(E)
    mu = x.mean(1)
    var = (x - mu[:, None]).square().mean(1)
    rs = 1 / (var + 1e-5).sqrt()
    t_mean = (k + 3) * U * x.abs().mean(1)
    r_rstd = ((k + 5) / 2 + 3) * U + t_mean ** 2 / (2 * (var + 1e-5))
    close(mean, mu, t_mean, "mean")
    close(rstd, rs, r_rstd * rs, "rstd")
    xh = (x - mu[:, None]) * rs[:, None]
    want = xh * gamma + beta
    tol = gamma.abs() * (rs[:, None] * t_mean[:, None] + xh.abs() * (r_rstd[:, None] + 2 * U)) * 1.001
    tol += 2 * U * ((xh * gamma).abs() + beta.abs())
    tol += ref.half(DT[dt]) * (want.abs() + tol) + ref.tiny(DT[dt])
    close(Y, want, tol, "Y")


@pytest.mark.parametrize("dt,rows,E,accumulate", [
    ("f32", [700, 0, 900], 1028, False), ("bf16", [1501, 129], 1536, True), ("f16", [900, 0, 640], 2048, False),
    ("bf16", [3000, 1000, 0, 7], 4096, False), ("f32", [700, 131], 4096, False), ("f32", [500, 333], 4097, True),
    ("bf16", [900, 1, 500], 5000, False), ("f32", [600, 150], 8192, False), ("bf16", [700, 0, 130], 8200, False),
    ("f32", [300, 401], 9000, True), ("f16", [500, 3, 140], 16383, False), ("bf16", [900, 250], 16384, False),
    ("f32", [129], 16384, False), ("bf16", [900, 700], 2001, False), ("f16", [20000, 0, 15000], 64, False)])
def test_layernorm_gradient_of_many_rows(dt, rows, E, accumulate):
    n, M = sum(rows), len(rows)
    opt = handle([(2, 2), (1, E), (1, 5), (1, E)], M, n, E)
    W = torch.randn(opt.d, generator=gen(11), device="cuda")
    g = gen(E + 1)
    X = norm_inputs(n, E, dt, g)
    dY = (torch.randn(n, E, generator=g, device="cuda") * 0.1).to(DT[dt])
    x, dy = X.double(), dY.double()
    mean = x.mean(1).float()
    rstd = (1 / (x.var(1, correction=0) + 1e-5).sqrt()).float()
    at_gamma, at_beta = 4, 9 + E
    old = torch.randn(M, opt.d, generator=gen(7), device="cuda")
    got = []
    for _ in range(2):
        G, Gm = vectors(opt)
        if accumulate:
            G[:, :opt.d] = old
        dX = torch.full_like(X, float("nan"))
        opt.layernorm_grad(W, 1, 3, X, dY, mean, rstd, dX, Gm, rows, accumulate=accumulate)
        opt.layers_sync()
        if not accumulate:
            assert bool(G[:, :4].isnan().all()) and bool(G[:, 4 + E:at_beta].isnan().all())
        got.append((dX, G[:, at_gamma:at_gamma + E].clone(), G[:, at_beta:at_beta + E].clone()))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    dX, dgamma, dbeta = got[0]
    k = ref.depth(E)
    rs = rstd.double()[:, None]
    xh = (x - mean.double()[:, None]) * rs
    gr = dy * W[4:4 + E].double()
    a, b = gr.mean(1, keepdim=True), (gr * xh).mean(1, keepdim=True)
    want = rs * (gr - a - xh * b)
    t_a = (k + 4) * U * gr.abs().mean(1, keepdim=True)
    t_b = (k + 7) * U * (gr * xh).abs().mean(1, keepdim=True)
    tol = rs * (t_a + xh.abs() * t_b + U * (5 * gr.abs() + 4 * a.abs() + 7 * (xh * b).abs()))
    tol += ref.half(DT[dt]) * (want.abs() + tol) + ref.tiny(DT[dt])
    close(dX, want, tol, "dX")
    m = worker_of(rows)
    r = torch.tensor(rows, device="cuda")[:, None]

    def per_worker(v):
        return torch.zeros(M, E, dtype=torch.float64, device="cuda").index_add_(0, m, v)

    for name, out, v, more, base in (("dgamma", dgamma, dy * xh, 3, at_gamma), ("dbeta", dbeta, dy, 0, at_beta)):
        want, tol = per_worker(v), (r + more) * U * per_worker(v.abs())
        if accumulate:
            want += old[:, base:base + E]
            tol += U * want.abs()
        close(out, want, tol, name)


# ---- distillation -------------------------------------------------------------------

@pytest.mark.parametrize("dt,V", [("bf16", 30000), ("f16", 40001), ("f32", 17001),        # 256 threads
                                  ("bf16", 50304), ("f16", 50257), ("f32", 40001), ("bf16", 128256)])   # 512
@pytest.mark.parametrize("K", [1, 33])
def test_distill_of_many_long_rows(dt, V, K):
    rows = [1003, 0, 90, 7]
    n, M, T, gscale = sum(rows), len(rows), 2.0, 1.5
    opt = handle([(1, 4)], M, n, 4)
    g = gen(V + K)
    Z = (torch.randn(n, V, generator=g, device="cuda") * 3).to(DT[dt])
    idx = torch.randint(0, V, (n, K), generator=g, device="cuda")
    t = torch.randn(n, K, generator=g, device="cuda") * 2
    idx[torch.rand(n, K, generator=g, device="cuda") < 0.2] = -1
    idx[::3, K // 2:] = idx[::3, :K - K // 2].clone()    # the same index twice
    got = []
    logits = Z.clone()
    for dZ in (torch.full_like(Z, float("nan")), logits, None):
        loss, row_loss = torch.full((M,), float("nan"), device="cuda"), torch.full((n,), float("nan"), device="cuda")
        count = torch.full((M,), -7, dtype=torch.int32, device="cuda")
        opt.distill(logits if dZ is logits else Z, idx, t, loss, rows, count=count, row_loss=row_loss, dZ=dZ, temperature=T,
                    gscale=gscale)
        opt.layers_sync()
        got.append((loss, count, row_loss, dZ))
    assert torch.equal(got[0][1], got[1][1]) and torch.equal(got[0][1], got[2][1])
    for k in (0, 2, 3):
        assert torch.equal(got[0][k], got[1][k])
    # float64, with the bounds of layers_ref.distill_bounds (A, the largest
    # argument, over the whole row), blocks of rows at a time
    m = worker_of(rows)
    here = idx >= 0
    some = here.any(1)
    count = torch.zeros(M, dtype=torch.int64, device="cuda").index_add_(0, m, some.long())
    assert torch.equal(got[0][1].long(), count)
    at = idx.clamp(min=0)
    x = torch.where(here, t.double() / T, -torch.inf)
    top = torch.where(some, x.amax(1), 0.0)[:, None]
    b = torch.where(here, top - x, torch.inf)
    sq = torch.exp(-b).sum(1, keepdim=True).clamp(min=1e-300)
    q = torch.exp(-b) / sq
    bb = torch.where(here, b, 0.0)
    rel_sq = U * (ref.depth(K) + 10 + 4 * bb.amax(1, keepdim=True))
    rel_q = rel_sq + U * (6 + 4 * bb)
    lq = -bb - sq.log()
    row, t_row = torch.zeros(n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
    for i in range(0, n, 256):
        s = slice(i, min(n, i + 256))
        z = Z[s].double() / T
        a = z.amax(1, keepdim=True) - z
        ssum = torch.exp(-a).sum(1, keepdim=True)
        p, log_s = torch.exp(-a) / ssum, ssum.log()
        rel_s = U * (5 * ref.depth(V) + 12 + 5 * a.amax(1, keepdim=True))
        ak = a.gather(1, at[s])
        lp = -ak - log_s
        e_l = rel_sq[s] + rel_s + U * (6 + 5 * bb[s] + 5 * ak + 4 * log_s.abs())
        row[s] = T * T * (q[s] * (lq[s] - lp)).sum(1)
        t_row[s] = T * T * (q[s] * (e_l + (rel_q[s] + U * (ref.depth(K) + 6)) * (lq[s] - lp).abs())).sum(1) * 1.001
        w = (abs(gscale) * T / count[m[s]].clamp(min=1) * some[s])[:, None]
        want = p.scatter_add(1, at[s], -q[s])
        tol = (p * (rel_s + U * (12 + 5 * a))).scatter_add_(1, at[s], q[s] * (rel_q[s] + (K + 4) * U))
        tol = w * (tol + 2 * U * want.abs()) * 1.001
        want *= w
        tol += ref.half(DT[dt]) * (want.abs() + tol) + ref.tiny(DT[dt])
        close(got[0][3][s], want, tol, f"dZ from row {i}")
    t_row += U * row.abs()
    n_m = count.clamp(min=1).double()

    def mean(v):
        return torch.zeros(M, dtype=torch.float64, device="cuda").index_add_(0, m, v) / n_m

    for form, (loss, _, row_loss, _) in zip(("gradient", "in place", "loss only"), got):
        close(row_loss, row, t_row, f"row_loss, {form}")
        close(loss, mean(row), mean(t_row) + 3 * U * mean(row.abs()), f"loss, {form}")
