"""The distillation where logits / temperature are far from zero: finite masks of
every size, over parts of a row and over all of it, logits far above zero, and
temperatures over the whole accepted range, in each of the row kernel's forms
(32, 128, 256 and 512 threads a row, few rows and many).  Held against the
float64 form."""
import numpy as np
import pytest

import layers_ref as ref
from layers_ref import DT, U

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import sign_muon_optimizer_b200 as smo  # noqa: E402

K = 4


def exact(Z, idx, t, T, gscale):
    """Loss, row losses and dZ of one worker whose rows all count, in float64, and
    their bounds.

    Arguments of exponentials are differences to a maximum, a and b in natural
    units, off by 5 (4) roundings each; an exponential is off by 4u besides.  A
    term's own error weighs in the row's sum with its share p, so that the sum is
    off by 5u sum p a, besides its additions and the rescalings with new maxima
    (5u each, and at most as many as terms in a row).  2^x is zero below 2^-126,
    and a row's sum is at least 1/2: p is off by 2^-125 besides."""
    n, V = Z.shape
    z = Z.double() / T
    a = z.amax(1, keepdim=True) - z
    e = torch.exp(-a)
    s = e.sum(1, keepdim=True)
    p, log_s = e / s, s.log()
    rel_s = U * (5 * ref.depth(V) + 12 + 5 * (p * a).sum(1, keepdim=True))
    x = t.double() / T
    b = x.amax(1, keepdim=True) - x
    q = torch.softmax(-b, 1)
    lq = -b - torch.exp(-b).sum(1, keepdim=True).log()
    ak = a.gather(1, idx)
    lp = -ak - log_s
    rel_sq = U * (ref.depth(K) + 10 + 4 * (q * b).sum(1, keepdim=True))
    rel_q = rel_sq + U * (6 + 4 * b)
    e_l = rel_sq + rel_s + U * (6 + 5 * b + 5 * ak + 4 * log_s.abs())
    none = q == 0
    row = T * T * torch.where(none, 0, q * (lq - lp)).sum(1)
    t_row = T * T * torch.where(none, 0, q * (e_l + (rel_q + U * (ref.depth(K) + 6)) * (lq - lp).abs())).sum(1) * 1.001
    t_row += U * row.abs()
    w = gscale * T / n
    want = p.scatter_add(1, idx, -q)
    tol = p * (rel_s + U * (12 + 5 * a)) + 2.0 ** -125
    tol.scatter_add_(1, idx, q * (rel_q + (K + 4) * U))
    tol = w * 1.001 * (tol + 6 * U * want.abs())
    want *= w
    tol += ref.half(Z.dtype) * (want.abs() + tol) + ref.tiny(Z.dtype)
    return row, t_row, want, tol


def close(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)      # (a NaN is bad)
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off in rows "
                             f"{sorted(set(bad.nonzero()[:, 0].tolist()))[:20]}; first at {i}: got {float(got[i])!r}, "
                             f"wanted {float(want[i])!r} within {float(tol[i]):.3g}")


def check(Z, idx, t, T, gscale):
    """The call with a gradient of its own, in place, and for the loss alone."""
    n, V = Z.shape
    opt = smo.SignMuon([(1, 4)], 1, flags=smo.SIGNMUON_VOTE_ONLY)
    opt.layers_reserve(n, 4)
    T, gscale = float(np.float32(T)), float(np.float32(gscale))
    row, t_row, want, tol = exact(Z, idx, t, T, gscale)
    logits = Z.clone()
    for form in ("own", "in place", "loss"):
        dZ = {"own": torch.full_like(Z, float("nan")), "in place": logits, "loss": None}[form]
        loss = torch.full((1,), float("nan"), device="cuda")
        rows = torch.full((n,), float("nan"), device="cuda")
        count = torch.zeros(1, dtype=torch.int32, device="cuda")
        opt.distill(logits if form == "in place" else Z, idx, t, loss, count=count, row_loss=rows, dZ=dZ, temperature=T,
                    gscale=gscale)
        opt.layers_sync()
        assert int(count[0]) == n
        close(rows, row, t_row, f"row_loss, {form}")
        close(loss, row.mean()[None], (t_row.mean() + 3 * U * row.abs().mean())[None], f"loss, {form}")
        if dZ is not None:
            close(dZ, want, tol, f"dZ, {form}")


MASKS = [-5e9, -1e10, -1e15, -1e20, -1e30, -1e36]


def masked_rows(n, V, dt, g):
    """Ordinary logits, with a mask over a part that changes from row to row; and
    the K entries' places, in what the mask leaves."""
    Z = torch.randn(n, V, generator=g, device="cuda") * 3
    col = torch.arange(V, device="cuda")
    idx = torch.empty(n, K, dtype=torch.int64, device="cuda")
    for r in range(n):
        v, kind = MASKS[r % 6], r // 6 % 8
        free = torch.tensor([V // 2, V // 2 + 1, V // 2 + 5, V // 2 + 9], device="cuda")
        if kind == 0:
            part = col < V // 2
        elif kind == 1:
            part = col > V // 2 + 9
        elif kind == 2:
            part = (col < V // 4) | (col > V // 2 + 9)
        elif kind == 3:
            part = (col // 64 % 2 == 0) & ~torch.isin(col, free)
        elif kind == 4:
            part = ~torch.isin(col, free)
        elif kind == 5:
            part = col >= 0                       # all of it
        elif kind == 6:
            Z[r, :V // 4] = MASKS[(r + 1) % 6]    # two masks
            part = (col >= V // 4) & (col < V // 2)
        else:
            part = col == V // 2 + 1              # far above zero
            v = -v
        Z[r, part] = v
        idx[r] = free
    idx[3, 0] = 2                                 # an entry on a masked logit
    return Z.to(DT[dt]), idx


# row bytes up to 16, 48 and 80 KB and beyond: 32, 128, 256 and 512 threads (the loss alone: 32, 128, 256)
FORMS = [("f32", 1000), ("f32", 9001), ("f32", 17000), ("f32", 40001),
         ("bf16", 1000), ("bf16", 12001), ("bf16", 30000), ("bf16", 60007)]


@pytest.mark.parametrize("dt,V", FORMS)
@pytest.mark.parametrize("T", [0.5, 1.0, 2.0, 3.0])
def test_distill_finite_masks(dt, V, T):
    g = torch.Generator(device="cuda").manual_seed(V)
    Z, idx = masked_rows(48, V, dt, g)
    check(Z, idx, torch.randn(48, K, generator=g, device="cuda"), T, 1.0)


@pytest.mark.parametrize("dt,V", FORMS)
def test_distill_finite_masks_in_many_rows(dt, V):
    g = torch.Generator(device="cuda").manual_seed(V + 1)
    Z, idx = masked_rows(1104, V, dt, g)
    check(Z, idx, torch.randn(1104, K, generator=g, device="cuda"), 1.0, 1.0)


@pytest.mark.parametrize("dt,V", FORMS + [("f16", 1000), ("f16", 50000)])
@pytest.mark.parametrize("T", [1e-6, 3e-8, 1e-9, 1e-12, 1e-18, 1e18])
def test_distill_over_the_accepted_temperatures(dt, V, T):
    n = 40
    g = torch.Generator(device="cuda").manual_seed(V + 2)
    Z = (torch.randn(n, V, generator=g, device="cuda") * 2).to(DT[dt])
    eps = torch.finfo(DT[dt]).eps
    Z[1] = 0
    Z[2] = 1.5                                                        # p = 1 / V
    Z[3, ::7] = 20                                                    # equal largest logits
    Z[4, 11:13] = -Z[4].abs().amax() - 30
    Z[5] = (1 + eps * torch.randint(0, 9, (V,), generator=g, device="cuda")).to(DT[dt])   # neighbours of 1
    Z[6] = -Z[5]
    Z[7] = Z[5].float() * 2.0 ** -20                                  # small and close together
    idx = (torch.randint(0, V, (n, 1), generator=g, device="cuda") + torch.arange(K, device="cuda") * 17) % V
    t = torch.randn(n, K, generator=g, device="cuda")
    t[5:9] = 1
    check(Z, idx, t, T, 1 / T)
