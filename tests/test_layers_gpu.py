"""The layer calls (include/signmuon_layers.h) against plain float64 forms, at
the sizes, types, strides and masks where they can go wrong."""
import numpy as np
import pytest

import layers_ref as ref
from layers_ref import DT, U, f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import sign_muon_optimizer_b200 as smo  # noqa: E402

MARK = -7.5  # what buffers hold where a call must not write


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def handle(shapes, M, rows, cols):
    opt = smo.SignMuon(shapes, M, flags=smo.SIGNMUON_VOTE_ONLY)
    opt.layers_reserve(max(1, rows), cols)
    return opt


def flat(opt, seed):
    return torch.randn(opt.d, generator=gen(seed), device="cuda")


def grads(opt):
    n = (opt.d + 3) // 4 * 4
    buf = torch.full((opt.M, n + 4), MARK, device="cuda")
    return buf, [buf[m] for m in range(opt.M)]


def strided(n, cols, dt, gap, shift=0):
    """An n x cols matrix inside a larger buffer, and the buffer."""
    buf = torch.full((shift + (n + 1) * (cols + gap),), MARK, dtype=dt, device="cuda")
    return buf[shift:].as_strided((n, cols), (cols + gap, 1)), buf


def untouched(buf, mat):
    """Everything of buf outside mat still holds the mark."""
    seen = torch.ones_like(buf, dtype=torch.bool)
    seen[mat.storage_offset():].as_strided(mat.shape, mat.stride()).fill_(False)
    return bool((buf[seen] == MARK).all())


# ---- embedding lookup ---------------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,V,E,gap,shift,idt", [
    (1, 1, 1, 0, 0, torch.int64), (8, 100, 768, 0, 0, torch.int64), (5, 7, 1001, 0, 0, torch.int32),
    (37, 50, 64, 8, 0, torch.int32), (37, 50, 64, 3, 1, torch.int64), (3, 9, 2056, 0, 0, torch.int64),
    (300, 1000, 36, 4, 0, torch.int64)])
def test_embed_is_one_rounding(dt, n, V, E, gap, shift, idt):
    opt = handle([(3, 5), (V, E), (2, 2)], 2, n, E)
    W = flat(opt, 1)
    g = gen(2)
    ids = torch.randint(0, V, (n,), generator=g, device="cuda").to(idt)
    ids[::4] = -1 - ids[::4]
    out, buf = strided(n, E, DT[dt], gap, shift)
    opt.embed(W, 1, ids, out, scale=1.7)
    opt.layers_sync()
    table = W[15:15 + V * E].view(V, E)
    want = torch.where((ids >= 0)[:, None], table[ids.clamp(min=0).long()] * 1.7, 0.0).to(DT[dt])
    assert torch.equal(out, want)
    assert untouched(buf, out)


def test_embed_reports_an_id_beyond_the_table():
    opt = handle([(10, 8)], 1, 4, 8)
    W = flat(opt, 3)
    ids = torch.tensor([9, 10, -1, 2 ** 40], device="cuda")
    out = torch.full((4, 8), MARK, device="cuda")
    opt.embed(W, 0, ids, out)
    with pytest.raises(smo.SignMuonError) as e:
        opt.layers_sync()
    assert e.value.status == smo.SIGNMUON_E_INVALID
    assert torch.equal(out[0], W[72:80]) and not out[1:].any()
    opt.layers_sync()  # reported once
    opt.embed(W, 0, ids[:0], out[:0])
    opt.layers_sync()


# ---- embedding gradient --------------------------------------------------------

def ids_of(kind, n, V, g):
    if kind == "random":
        return torch.randint(0, V, (n,), generator=g, device="cuda")
    if kind == "zipf":
        return ((V + 1.0) ** torch.rand(n, generator=g, device="cuda", dtype=torch.float64)).long().clamp(1, V) - 1
    if kind == "same":
        return torch.full((n,), V // 2, device="cuda")
    if kind == "lengths":            # runs that end before, at and behind every border of 32 and 256 tokens
        c = torch.tensor([1, 31, 32, 33, 64, 1, 95, 255, 256, 257, 2, 512, 30, 770], device="cuda")
        ids = torch.repeat_interleave(torch.arange(len(c), device="cuda"), c)
        ids = ids.repeat(n // len(ids) + 1)[:n]
        return ids[torch.randperm(n, generator=g, device="cuda")]
    if kind == "absent":
        return torch.full((n,), -1, device="cuda")
    return torch.arange(n, device="cuda").flip(0) % V   # "falling"


@pytest.mark.parametrize("dt,rows,V,E,kind,gap,accumulate", [
    ("f32", [1], 1, 1, "random", 0, False),
    ("f32", [33, 0, 31], 10, 8, "random", 0, False),
    ("bf16", [64, 65, 1], 300, 768, "zipf", 0, False),
    ("f16", [100, 0, 0, 200], 77, 1001, "zipf", 0, False),
    ("bf16", [2047, 2049], 50, 24, "zipf", 8, False),
    ("bf16", [300, 40], 50, 24, "same", 0, False),
    ("f32", [0, 0], 50, 24, "random", 0, False),
    ("f32", [0, 0], 50, 24, "random", 0, True),
    ("f16", [70, 5], 50, 40, "absent", 0, False),
    ("f32", [500, 3], 1000, 12, "falling", 1, False),
    ("bf16", [257, 3], 60, 264, "zipf", 0, True),
    ("f32", [129, 63], 5, 7, "same", 0, True),
    ("f32", [40000, 5, 2048], 700, 4, "zipf", 0, False),
    ("f32", [33000], 20000, 8, "random", 0, False),
    ("bf16", [4096, 4097], 3, 16, "same", 0, False),         # one run over many units
    ("f32", [12000], 20, 16, "same", 0, False),              # ... over more than 32
    ("bf16", [2339, 2340, 2338], 14, 40, "lengths", 0, False),
    ("f32", [4678], 20, 3, "lengths", 0, False),
    ("f16", [256, 512, 255, 257], 2, 300, "random", 0, False),
    ("f32", [1, 2] * 128, 9, 5, "random", 0, False),         # 256 workers
    ("f32", [70000], 300, 4, "zipf", 0, False),
    ("f32", [1500, 3, 2048], (1 << 21) - 1, 1, "random", 0, False),   # the largest table of 32-bit sort keys
    ("f32", [1500, 3, 2048], 1 << 21, 1, "random", 0, False),   # ... and one row more
    ("bf16", [700, 9], 3, 9000, "random", 0, False),         # rows zeroed by a whole block
    ("f32", [16639], 300, 4, "zipf", 0, False),              # the last size of small units
    ("f32", [16640], 300, 4, "zipf", 0, False),
    ("bf16", [40, 0, 3], 700, 77, "random", 0, False),        # tables of several chunks of zeros at odd addresses,
    ("f32", [3000, 0], 901, 77, "random", 0, False),          # in each form of the sort
    ("f16", [9000, 0], 1100, 61, "random", 0, False),
    ("f16", [4097, 0, 4096], 500, 6, "random", 0, True),      # borders of the sort's forms
    ("bf16", [4096, 17], 70, 9, "zipf", 1, True),
])
def test_embed_grad(dt, rows, V, E, kind, gap, accumulate):
    n, M = sum(rows), len(rows)
    opt = handle([(1, 6), (V, E), (1, 3)], M, n, E)
    g = gen(n + V)
    ids = ids_of(kind, n, V, g)
    ids[3::7] = -5
    dY, _ = strided(n, E, DT[dt], gap)
    dY.copy_(torch.randn(n, E, generator=g, device="cuda"))
    dY[3::7] = float("nan")          # padding rows are not read
    G, Gm = grads(opt)
    old = torch.randn(M, V * E, generator=g, device="cuda")
    if accumulate:
        G[:, 6:6 + V * E] = old
    opt.embed_grad(1, ids, dY, Gm, rows, scale=0.37, accumulate=accumulate)
    opt.layers_sync()
    want, tol = ref.embed_grad(ids.cpu().numpy(), f64(dY), rows, V, np.float32(0.37).astype(float))
    got = G[:, 6:6 + V * E].reshape(M, V, E)
    if accumulate:
        o = f64(old).reshape(M, V, E)
        want = want + o
        tol = np.where(tol > 0, tol + U * np.abs(want), 0)
    ref.assert_within(got, want, tol, "G")
    assert bool((G[:, :6] == MARK).all()) and bool((G[:, 6 + V * E:] == MARK).all())
    again, Am = grads(opt)
    if accumulate:
        again[:, 6:6 + V * E] = old
    opt.embed_grad(1, ids.int(), dY, Am, rows, scale=0.37, accumulate=accumulate)
    assert torch.equal(G, again)     # a fixed order of every sum


@pytest.mark.parametrize("V", [400, (1 << 18) - 1, 1 << 18, (1 << 27) + 5])
@pytest.mark.parametrize("n", [2500, 8192, 8193])      # (by a block, and by several)
def test_embed_grad_with_one_to_four_sort_digits(V, n):
    """The sort takes the bits of 0 ... V in digits of at most 9; the ids differ
    in every one of them."""
    opt = handle([(V, 1)], 1, n, 1)
    g = gen(V)
    ids = torch.randint(0, V, (n,), generator=g, device="cuda")
    ids[:1500] = ids[1000:2500].clone()   # several tokens a row
    ids[::11] = -1
    ids[5], ids[6] = 0, V - 1
    dY = torch.randn(n, 1, generator=g, device="cuda")
    G, Gm = grads(opt)
    opt.embed_grad(0, ids, dY, Gm)
    opt.layers_sync()
    keep = ids >= 0
    want = torch.zeros(V, dtype=torch.float64, device="cuda").index_add_(0, ids[keep], dY[keep, 0].double())
    size = torch.zeros(V, dtype=torch.float64, device="cuda").index_add_(0, ids[keep], dY[keep, 0].double().abs())
    count = torch.bincount(ids[keep], minlength=V)
    assert bool(((G[0, :V] - want).abs() <= size * (count + 2) * U).all())
    assert bool((G[0, V:] == MARK).all())


def test_embed_grad_skips_and_reports_ids_beyond_the_table():
    opt = handle([(6, 8)], 1, 64, 8)
    ids = torch.tensor([5, 6, 7, 5] * 16, device="cuda")
    dY = torch.ones(64, 8, device="cuda")
    G, Gm = grads(opt)
    opt.embed_grad(0, ids, dY, Gm)
    with pytest.raises(smo.SignMuonError) as e:
        opt.layers_sync()
    assert e.value.status == smo.SIGNMUON_E_INVALID
    assert bool((G[0, 40:48] == 32).all()) and not G[0, :40].any() and bool((G[0, 48:] == MARK).all())


# ---- layer norm --------------------------------------------------------------------

NORMS = [(1, 1), (1, 768), (9, 7), (8, 768), (33, 1001), (5, 1024), (6, 1028), (3, 2047), (4, 4096), (3, 5000), (2, 8192),
         (3, 16383), (2, 16384)]


def norm_inputs(n, E, dt, gap, seed, shift=0):
    g = gen(seed)
    X, bx = strided(n, E, DT[dt], gap, shift)
    X.copy_(torch.randn(n, E, generator=g, device="cuda") * 2 + 3)
    if n > 2:
        X[1] = 1.5                    # a constant row: variance 0
        X[2] *= 30
    return X, bx, g


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,E", NORMS)
@pytest.mark.parametrize("gap,with_beta", [(0, True), (8, False), (3, True)])
def test_layernorm(dt, n, E, gap, with_beta):
    opt = handle([(1, E), (1, E)], 1, n, E)
    W = flat(opt, 5)
    X, bx, _ = norm_inputs(n, E, dt, gap, E)
    Y, by = strided(n, E, DT[dt], gap)
    mean, rstd = (torch.full((n + 4,), MARK, device="cuda") for _ in range(2))
    opt.layernorm(W, 0, 1 if with_beta else None, X, Y, mean, rstd, eps=1e-5)
    w = f64(W)
    want = ref.layernorm(f64(X), w[:E], w[E:] if with_beta else None, 1e-5, DT[dt])
    ref.assert_within(mean[:n], want[1], want[4], "mean")
    ref.assert_within(rstd[:n], want[2], want[5], "rstd")
    ref.assert_within(Y, want[0], want[3], "Y")
    assert untouched(by, Y) and bool((mean[n:] == MARK).all()) and bool((rstd[n:] == MARK).all())
    Y2 = torch.empty_like(Y)
    opt.layernorm(W, 0, 1 if with_beta else None, X, Y2)
    assert torch.equal(Y, Y2)


def test_layernorm_variance_survives_a_large_mean():
    E = 768
    opt = handle([(1, E)], 1, 4, E)
    W = torch.ones(E, device="cuda")
    x = 1000 + torch.randn(4, E, generator=gen(7), device="cuda")
    Y = torch.empty_like(x)
    opt.layernorm(W, 0, None, x, Y)
    want = ref.layernorm(f64(x), np.ones(E), None, 1e-5, torch.float32)
    ref.assert_within(Y, want[0], want[3], "Y")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,E,gap,in_place,accumulate", [
    ([1], 1, 0, False, False), ([1], 768, 0, False, False), ([5, 0, 9], 7, 0, False, False),
    ([70, 0, 33], 512, 0, True, False), ([200, 31], 768, 0, False, False), ([40], 1001, 0, False, True),
    ([9, 9], 1028, 8, True, False), ([17, 1], 2047, 3, False, False), ([3, 30, 0, 2], 4096, 0, False, False),
    ([7, 2], 5000, 0, True, True), ([5], 8192, 0, False, False), ([3, 2], 16383, 0, True, False),
    ([4, 1], 16384, 0, True, False), ([3000] * 3, 64, 0, False, False), ([0, 0], 64, 0, False, False),
    ([0, 2], 64, 0, False, True)])
def test_layernorm_grad(dt, rows, E, gap, in_place, accumulate):
    n, M = sum(rows), len(rows)
    opt = handle([(2, 2), (1, E), (1, 5), (1, E)], M, n, E)
    W = flat(opt, 11)
    X, _, g = norm_inputs(n, E, dt, gap, E + 1)
    dY, bd = strided(n, E, DT[dt], gap)
    dY.copy_(torch.randn(n, E, generator=g, device="cuda") * 0.1)
    dy = f64(dY)
    x = f64(X)
    mean = torch.from_numpy(x.mean(1)).float().cuda() if n else torch.empty(1, device="cuda")
    rstd = (torch.from_numpy(1 / np.sqrt(x.var(1) + 1e-5)).float().cuda() if n else torch.empty(1, device="cuda"))
    dX, bX = (dY, bd) if in_place else strided(n, E, DT[dt], gap)
    G, Gm = grads(opt)
    o = 0.0
    if accumulate:
        old = torch.randn(M, opt.d, generator=g, device="cuda")
        G[:, :opt.d] = old
        o = f64(old)
    opt.layernorm_grad(W, 1, 3, X, dY, mean, rstd, dX, Gm, rows, accumulate=accumulate)
    opt.layers_sync()
    w = f64(W)
    want = ref.layernorm_grad(x, dy, f64(mean)[:n], f64(rstd)[:n], w[4:4 + E], rows, DT[dt])
    ref.assert_within(dX, want[0], want[3], "dX")
    assert untouched(bX, dX)
    b = 9 + E
    for name, at, k in (("dgamma", 4, 1), ("dbeta", b, 2)):
        base = o[:, at:at + E] if accumulate else 0.0
        ref.assert_within(G[:, at:at + E], want[k] + base, want[k + 3] + (U * np.abs(want[k] + base) if accumulate else 0),
                          name)
    if not accumulate:
        assert bool((G[:, :4] == MARK).all()) and bool((G[:, 4 + E:b] == MARK).all()) and bool((G[:, b + E:] == MARK).all())
    else:
        assert torch.equal(G[:, :4], old[:, :4]) and torch.equal(G[:, 4 + E:b], old[:, 4 + E:b])


def test_layernorm_grad_without_beta_leaves_its_place():
    E = 48
    opt = handle([(1, E), (1, E)], 2, 8, E)
    W = flat(opt, 13)
    X, _, g = norm_inputs(8, E, "f32", 0, 3)
    dY = torch.randn(8, E, generator=g, device="cuda")
    Y, mean, rstd = torch.empty_like(X), torch.empty(8, device="cuda"), torch.empty(8, device="cuda")
    opt.layernorm(W, 0, None, X, Y, mean, rstd)
    G, Gm = grads(opt)
    opt.layernorm_grad(W, 0, None, X, dY, mean, rstd, torch.empty_like(X), Gm)
    assert bool((G[:, E:] == MARK).all()) and not bool((G[:, :E] == MARK).any())


def test_layernorm_grad_against_differences():
    """<dX, v> and <dgamma, v>, <dbeta, v> against central differences of the
    float64 forward form with step h: the difference is off by h^2/6 of the
    third derivative (below 1e-6 here), the call by its own bounds."""
    E, rows = 40, [3, 2]
    n = sum(rows)
    opt = handle([(1, E), (1, E)], 2, n, E)
    W = flat(opt, 17)
    g = gen(19)
    X = torch.randn(n, E, generator=g, device="cuda")
    dY = torch.randn(n, E, generator=g, device="cuda")
    Y, mean, rstd = torch.empty_like(X), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    opt.layernorm(W, 0, 1, X, Y, mean, rstd, eps=1e-5)
    dX = torch.empty_like(X)
    G, Gm = grads(opt)
    opt.layernorm_grad(W, 0, 1, X, dY, mean, rstd, dX, Gm, rows)
    w, x, dy = f64(W), f64(X), f64(dY)

    def value(x, w, s):
        return float((ref.layernorm(x, w[:E], w[E:], 1e-5, torch.float32)[0] * dy)[s].sum())

    h = 1e-5
    rng = np.random.default_rng(0)
    v = rng.standard_normal(x.shape)
    num = (value(x + h * v, w, slice(None)) - value(x - h * v, w, slice(None))) / (2 * h)
    want = float((f64(dX) * v).sum())
    scale = float((np.abs(f64(dX)) * np.abs(v)).sum())
    assert abs(num - want) <= 1e-5 * scale
    for m, s in enumerate(ref.bounds(rows)):
        v = rng.standard_normal(2 * E)
        num = (value(x, w + h * v, s) - value(x, w - h * v, s)) / (2 * h)
        got = f64(G[m, :2 * E])
        assert abs(num - float(got @ v)) <= 1e-5 * float(np.abs(got) @ np.abs(v))


# ---- distillation -------------------------------------------------------------------

def teacher(n, V, K, g, idt, absent=0.2):
    idx = torch.randint(0, V, (n, K), generator=g, device="cuda")
    t = torch.randn(n, K, generator=g, device="cuda") * 2
    gone = torch.rand(n, K, generator=g, device="cuda") < absent
    idx[gone] = -1
    return idx.to(idt), t


def run_distill(opt, Z, idx, t, rows, T, gscale, grad=True, in_place=False, gap=0):
    n, V = Z.shape
    loss = torch.full((opt.M + 1,), MARK, device="cuda")
    count = torch.full((opt.M + 1,), -7, dtype=torch.int32, device="cuda")
    row_loss = torch.full((n + 1,), MARK, device="cuda")
    dZ = bz = None
    if grad:
        dZ, bz = (Z, None) if in_place else strided(n, V, Z.dtype, gap)
    opt.distill(Z, idx, t, loss, rows, count=count, row_loss=row_loss, dZ=dZ, temperature=T, gscale=gscale)
    opt.layers_sync()
    assert float(loss[opt.M]) == MARK and int(count[opt.M]) == -7 and float(row_loss[n]) == MARK
    assert bz is None or untouched(bz, dZ)
    return loss[:opt.M], count[:opt.M], row_loss[:n], dZ


def check_distill(got, Zf, idx, t, rows, T, gscale, dt):
    loss, count, row_loss, dZ = got
    i, tt = idx.cpu().numpy(), f64(t)
    want = ref.distill(Zf, i, tt, rows, T, gscale)
    t_row, t_dZ = ref.distill_bounds(Zf, i, tt, rows, T, gscale, dt)
    assert np.array_equal(count.cpu().numpy(), want[1])
    ref.assert_within(row_loss, want[2], t_row + U * np.abs(want[2]), "row_loss")
    t_loss = np.array([t_row[s].sum() / max(1, c) for s, c in zip(ref.bounds(rows), want[1])])
    mean_abs = np.array([np.abs(want[2][s]).sum() / max(1, c) for s, c in zip(ref.bounds(rows), want[1])])
    ref.assert_within(loss, want[0], t_loss + 3 * U * mean_abs, "loss")
    if dZ is not None:
        ref.assert_within(dZ, want[3], t_dZ, "dZ")


@pytest.mark.parametrize("dt,tdt,idt,rows,V,K,T,gap,grad,in_place", [
    ("f32", "f32", torch.int32, [1], 1, 1, 1.0, 0, True, False),
    ("f32", "f32", torch.int64, [2, 0, 3], 10, 4, 2.0, 0, True, False),
    ("bf16", "bf16", torch.int32, [5, 6], 1000, 8, 1.0, 0, True, False),
    ("f16", "f32", torch.int64, [4, 3], 1003, 16, 3.0, 0, True, False),
    ("bf16", "f32", torch.int32, [3, 2], 4099, 33, 2.0, 5, True, False),
    ("bf16", "f16", torch.int32, [3], 50257, 64, 2.0, 0, True, True),
    ("f32", "bf16", torch.int32, [2], 33000, 3, 0.5, 0, True, True),
    ("f32", "f32", torch.int64, [2, 1], 513, 1024, 2.0, 0, True, False),
    ("f16", "f16", torch.int32, [70, 0, 7], 64, 2, 1.0, 0, False, False),
    ("f32", "f32", torch.int32, [0, 0], 64, 2, 1.0, 0, True, False),
    ("f32", "f32", torch.int32, [300, 1, 0, 299], 31, 1, 1.0, 1, True, False),
    ("bf16", "f32", torch.int32, [2, 2], 128000, 20, 2.0, 0, True, False),
    ("f32", "f32", torch.int32, [2], 70001, 5, 2.0, 0, True, False)])
def test_distill(dt, tdt, idt, rows, V, K, T, gap, grad, in_place):
    n, M = sum(rows), len(rows)
    opt = handle([(1, 4)], M, n, 4)
    g = gen(V + K)
    Z, _ = strided(n, V, DT[dt], gap)
    Z.copy_(torch.randn(n, V, generator=g, device="cuda") * 3)
    if n > 1:
        Z[1] += 40
    idx, t = teacher(n, V, K, g, idt)
    t = t.to(DT[tdt])
    if n > 2:
        idx[2] = -1                   # a row without entries; its logits are not read
        Z[2] = float("nan")
    Zf = np.where(np.isnan(f64(Z)), 0, f64(Z))
    got = run_distill(opt, Z, idx, t, rows, T, 1.5, grad, in_place, gap)
    check_distill(got, Zf, idx, t, rows, T, 1.5, DT[dt])


def test_distill_same_index_twice_and_masked_entries():
    opt = handle([(1, 4)], 2, 4, 4)
    V = 50
    g = gen(23)
    Z = torch.randn(4, V, generator=g, device="cuda")
    Z[:, 30:] = float("-inf")         # masked vocabulary
    Z[1, :10] = torch.finfo(torch.float32).min
    idx = torch.tensor([[3, 3, 3, 9], [12, 12, 9, -1], [4, 5, 4, 5], [7, 7, 7, 7]], device="cuda")
    t = torch.randn(4, 4, generator=g, device="cuda")
    t[0, 1] = float("-inf")           # an entry that does not count
    t[3] = float("-inf")              # ... a row of them
    idx[1, 2] = 15
    rows = [2, 2]
    got = run_distill(opt, Z, idx, t, rows, 2.0, 1.0)
    Zf = f64(Z)
    Zf[1, :10] = -1e6                 # as good as masked at any precision
    check_distill(got, Zf, idx, t, rows, 2.0, 1.0, torch.float32)
    assert not got[3][:, 30:].any() and not got[3][3].any() and got[1].tolist() == [2, 1]


def test_distill_entry_on_a_masked_logit_and_nonfinite_rows():
    opt = handle([(1, 4)], 1, 5, 4)
    V = 600
    Z = torch.randn(5, V, generator=gen(29), device="cuda")
    idx = torch.tensor([[3, 4]] * 5, dtype=torch.int32, device="cuda")
    t = torch.zeros(5, 2, device="cuda")
    Z[0, 3] = float("-inf")           # half the teacher's weight where p = 0
    Z[1, 77] = float("nan")
    Z[2, 78] = float("inf")
    Z[3] = float("-inf")
    loss, count, row_loss, dZ = run_distill(opt, Z, idx, t, [5], 1.0, 1.0)
    assert row_loss[0] == float("inf") and torch.isfinite(dZ[0]).all()
    assert abs(float(dZ[0, 3]) + 0.5 / 5) <= 0.5 / 5 * 8 * U
    assert torch.isnan(row_loss[1:4]).all() and torch.isnan(dZ[1]).all()
    assert torch.isnan(dZ[2, 78]) and torch.isnan(dZ[3]).all()
    assert torch.isfinite(row_loss[4]) and torch.isfinite(dZ[4]).all() and int(count[0]) == 5


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [40, 3000, 20003, 140001])
def test_distill_rows_of_the_types_extreme_values(dt, V):
    """Rows masked with the type's lowest value, wholly and all but a few, rows
    at its largest value, and rows far from zero."""
    opt = handle([(1, 4)], 1, 6, 4)
    f = torch.finfo(DT[dt])
    Z = torch.randn(6, V, generator=gen(V), device="cuda").to(DT[dt])
    Z[0] = f.min                      # all masked: p = 1 / V
    Z[1] = f.min
    Z[1, 5:9] = 1.5                   # p = 1 / 4 there
    Z[2] = f.max
    Z[3] = f.min
    Z[3, 7] = f.max                   # p = 1 there
    Z[4] += 900
    Z[5] -= 900
    idx = torch.tensor([[7, 5]] * 6, dtype=torch.int32, device="cuda")
    t = torch.zeros(6, 2, device="cuda")
    _, count, row_loss, dZ = run_distill(opt, Z, idx, t, [6], 1.0, 1.0)
    z = Z.double()
    p = torch.softmax(z - z.amax(1, keepdim=True), 1)
    want = p.clone()
    want[:, 7] -= 0.5
    want[:, 5] -= 0.5
    a = (z.amax(1, keepdim=True) - z).clamp(max=200)
    tol = (p * U * (5 * ref.depth(V) + 20 + 10 * a) + 4 * U * want.abs()) / 6
    ref.assert_within(dZ, f64(want / 6), f64(tol + ref.half(DT[dt]) * (want.abs() / 6 + tol)) + ref.tiny(DT[dt]), "dZ")
    lp = torch.log_softmax(z - z.amax(1, keepdim=True), 1)
    loss = -0.5 * (lp[:, 7] + lp[:, 5]) - np.log(2.0)
    fine = [0, 1, 2, 4, 5]
    ref.assert_within(row_loss[fine], f64(loss)[fine], f64(U * (5 * ref.depth(V) + 40 + 10 * loss.abs()))[fine], "row_loss")
    # the teacher's second entry sits where p = 0: as far below as the type goes
    gap = 0.5 * (float(f.max) - float(f.min))
    assert float(row_loss[3]) > 0.49 * min(gap * 2, 3e38)


def test_distill_reports_an_index_beyond_the_row():
    opt = handle([(1, 4)], 1, 2, 4)
    Z = torch.randn(2, 9, generator=gen(31), device="cuda")
    idx = torch.tensor([[1, 9], [3, 2]], device="cuda")
    t = torch.zeros(2, 2, device="cuda")
    loss = torch.empty(1, device="cuda")
    row = torch.empty(2, device="cuda")
    opt.distill(Z, idx, t, loss, row_loss=row)
    with pytest.raises(smo.SignMuonError) as e:
        opt.layers_sync()
    assert e.value.status == smo.SIGNMUON_E_INVALID
    lp = torch.log_softmax(Z.double(), 1)
    # the entry counts as absent: row 0 is a cross-entropy with label 1
    assert abs(float(row[0]) + float(lp[0, 1])) <= 200 * U * (1 + abs(float(lp[0, 1])))


def test_distill_gradient_against_differences():
    rows, V, K, T = [3, 2], 37, 5, 2.0
    n = sum(rows)
    opt = handle([(1, 4)], 2, n, 4)
    g = gen(37)
    Z = torch.randn(n, V, generator=g, device="cuda")
    idx, t = teacher(n, V, K, g, torch.int64)
    _, _, _, dZ = run_distill(opt, Z, idx, t, rows, T, 1.0)
    i, tt, z = idx.cpu().numpy(), f64(t), f64(Z)
    v = np.random.default_rng(1).standard_normal(z.shape)
    h = 1e-5
    num = (ref.distill(z + h * v, i, tt, rows, T, 1.0)[0].sum() - ref.distill(z - h * v, i, tt, rows, T, 1.0)[0].sum()) / (2 * h)
    d = f64(dZ)
    # the difference is off by h^2 of the third derivative and 1e-16 / h of the loss
    assert abs(num - float((d * v).sum())) <= 1e-5 * float((np.abs(d) * np.abs(v)).sum()) + 1e-9


@pytest.mark.parametrize("V", [300, 3000, 12000])
@pytest.mark.parametrize("K", [1, 100, 300])
@pytest.mark.parametrize("grad,in_place", [(True, False), (True, True), (False, False)])
def test_distill_many_rows_with_gaps_and_repeats(V, K, grad, in_place):
    """More rows than blocks, half of them without entries in runs of every
    length, repeated indices in some."""
    rows = [301, 0, 1500, 7]
    n = sum(rows)
    opt = handle([(1, 4)], len(rows), n, 4)
    g = gen(V + K)
    Z = (torch.randn(n, V, generator=g, device="cuda") * 2).to(torch.bfloat16)
    idx, t = teacher(n, V, K, g, torch.int32, absent=0.3)
    idx[::3, K // 2:] = idx[::3, :K - K // 2]          # the same index twice
    gone = torch.rand(n // 4 + 1, generator=g, device="cuda").repeat_interleave(4)[:n] < 0.4
    idx[gone] = -1
    Zf, want = Z.double(), Z.clone()
    got = run_distill(opt, Z, idx, t, rows, 2.0, 1.0, grad, in_place)
    check_distill(got, f64(Zf), idx, t, rows, 2.0, 1.0, torch.bfloat16)
    again = run_distill(opt, want, idx, t, rows, 2.0, 1.0, grad, in_place)
    for a, b in zip(got, again):
        assert (a is None and b is None) or torch.equal(a, b)


def test_distill_loss_of_many_long_rows():
    """Loss only, rows at every alignment, more of them than go at once."""
    rows = [3000, 1, 199]
    n, V = sum(rows), 26003
    opt = handle([(1, 4)], len(rows), n, 4)
    g = gen(V)
    Z = (torch.randn(n, V, generator=g, device="cuda") * 2).to(torch.bfloat16)
    Z[5, 100:] = -float("inf")
    idx, t = teacher(n, V, 12, g, torch.int64, absent=0.1)
    idx[5] = torch.arange(12, device="cuda")
    got = run_distill(opt, Z, idx, t, rows, 1.0, 1.0, False)
    check_distill(got, f64(Z), idx, t, rows, 1.0, 1.0, torch.bfloat16)


def test_distill_loss_only_equals_loss_with_gradient():
    opt = handle([(1, 4)], 3, 40, 4)
    g = gen(41)
    Z = torch.randn(40, 777, generator=g, device="cuda")
    idx, t = teacher(40, 777, 6, g, torch.int32, absent=0.8)
    rows = [11, 20, 9]
    a = run_distill(opt, Z, idx, t, rows, 2.0, 1.0, True)
    b = run_distill(opt, Z, idx, t, rows, 2.0, 1.0, False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
