"""Plain float64 forms of the layer calls on the CPU (numpy), and the bounds
that their float32 results are held to.

u = 2^-24 is half a step of float32 relative to the value, half(type) the same
of an output type (bf16 2^-8, fp16 2^-11, fp32 2^-24).  Every bound counts the
roundings of the formula as written beside it, to first order, with a sum of n
terms over at least one warp per row taken as n/32 additions in a row and at
most 40 more to join the parts (for n < 32 this covers any order)."""
import numpy as np
import torch

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    """Half the spacing of the type's subnormals (fp16's are reached here)."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def depth(n):
    return n / 32 + 40


def f64(t):
    return t.detach().cpu().double().numpy()


def bounds(rows):
    b = np.concatenate([[0], np.cumsum(rows)]).astype(int)
    return [slice(b[m], b[m + 1]) for m in range(len(rows))]


def assert_within(got, want, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - want) <= tol)
    assert got.shape == want.shape
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        t = np.broadcast_to(tol, want.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off; first at {i}: got {got[i]!r}, "
                             f"wanted {want[i]!r} within {t[i]:.3g}")


# ---- embedding ---------------------------------------------------------------

def embed_grad(ids, dY, rows, V, scale):
    """(G, bound): c terms of a sum add at most c roundings of the terms'
    absolute sum, whatever the order; the scale and the store add two."""
    M, E = len(rows), dY.shape[1]
    G, tol = np.zeros((M, V, E)), np.zeros((M, V, E))
    for m, s in enumerate(bounds(rows)):
        keep = (ids[s] >= 0) & (ids[s] < V)
        i, d = ids[s][keep], dY[s][keep]
        np.add.at(G[m], i, d)
        np.add.at(tol[m], i, np.abs(d))
        c = np.bincount(i, minlength=V)[:, None]
        tol[m] *= (c + 2) * U * abs(scale)
    return G * scale, tol


# ---- layer norm ----------------------------------------------------------------

def layernorm(X, gamma, beta, eps, dt):
    """Y, mean, rstd and their bounds."""
    E = X.shape[1]
    n = depth(E)
    mean = X.mean(1)
    var = ((X - mean[:, None]) ** 2).mean(1)
    rstd = 1 / np.sqrt(var + eps)
    # mean: the sum's additions and the product with 1/E (itself rounded)
    t_mean = (n + 3) * U * np.abs(X).mean(1)
    # var around a mean that is off by t_mean is larger by t_mean^2; a term
    # carries 3 roundings, the sum n, the product with 1/E 2; rstd = 1/sqrt
    # halves that and adds the sum with eps, the root and the quotient
    r_rstd = ((n + 5) / 2 + 3) * U + t_mean ** 2 / (2 * (var + eps))
    xh = (X - mean[:, None]) * rstd[:, None]
    Y = xh * gamma + (0 if beta is None else beta)
    t_xh = rstd[:, None] * t_mean[:, None] + np.abs(xh) * (r_rstd[:, None] + 2 * U)
    t_Y = np.abs(gamma) * t_xh * 1.001 + 2 * U * (np.abs(xh * gamma) + (0 if beta is None else np.abs(beta)))
    t_Y += half(dt) * (np.abs(Y) + t_Y) + tiny(dt)
    return Y, mean, rstd, t_Y, t_mean, r_rstd * rstd


def layernorm_grad(X, dY, mean, rstd, gamma, rows, dt):
    """dX, dgamma, dbeta per worker, and their bounds; mean and rstd as given."""
    E = X.shape[1]
    n = depth(E)
    rs = rstd[:, None]
    xh = (X - mean[:, None]) * rs                      # 2 roundings
    g = dY * gamma                                     # 1
    a = g.mean(1, keepdims=True)
    b = (g * xh).mean(1, keepdims=True)
    dX = rs * (g - a - xh * b)
    t_a = (n + 4) * U * np.abs(g).mean(1, keepdims=True)
    t_b = (n + 7) * U * np.abs(g * xh).mean(1, keepdims=True)
    t = rs * (t_a + np.abs(xh) * t_b + U * (5 * np.abs(g) + 4 * np.abs(a) + 7 * np.abs(xh * b)))
    t += half(dt) * (np.abs(dX) + t) + tiny(dt)
    M = len(rows)
    out = [np.zeros((M, E)) for _ in range(4)]
    for m, s in enumerate(bounds(rows)):
        r = rows[m]
        out[0][m], out[1][m] = (dY[s] * xh[s]).sum(0), dY[s].sum(0)
        out[2][m] = (r + 3) * U * np.abs(dY[s] * xh[s]).sum(0)
        out[3][m] = r * U * np.abs(dY[s]).sum(0)
    return dX, out[0], out[1], t, out[2], out[3]


# ---- distillation ----------------------------------------------------------------

def distill(Z, idx, t, rows, T, gscale):
    """loss, count, row_loss, dZ as the formulas say."""
    N, V = Z.shape
    M = len(rows)
    row_loss, dZ = np.zeros(N), np.zeros((N, V))
    loss, count = np.zeros(M), np.zeros(M, int)
    for m, s in enumerate(bounds(rows)):
        some = []
        for r in range(s.start, s.stop):
            k = (idx[r] >= 0) & (idx[r] < V) & ~(t[r] == -np.inf)
            if not k.any():
                continue
            some.append(r)
            x = t[r][k] / T
            lq = x - x.max()
            lq = lq - np.log(np.exp(lq).sum())
            z = Z[r] / T
            with np.errstate(invalid="ignore"):
                lp = z - z.max()
                lp = lp - np.log(np.exp(lp).sum())
            q = np.exp(lq)
            with np.errstate(invalid="ignore"):
                row_loss[r] = T * T * np.where(q > 0, q * (lq - lp[idx[r][k]]), 0).sum()
            dZ[r] = np.exp(lp)
            np.subtract.at(dZ[r], idx[r][k], q)
        count[m] = len(some)
        if some:
            loss[m] = row_loss[some].sum() / len(some)
            dZ[some] *= gscale * T / len(some)
    return loss, count, row_loss, dZ


def distill_bounds(Z, idx, t, rows, T, gscale, dt):
    """Bounds of row_loss and dZ (loss: the mean of the rows' bounds and one
    rounding).  All arguments of exponentials are differences to a maximum:
    A, B (natural units, after 1/T) are the largest of the student's and the
    teacher's, off by 4 roundings each; an exponential is off by 4u besides."""
    N, V = Z.shape
    K = idx.shape[1]
    t_row, t_dZ = np.zeros(N), np.zeros((N, V))
    for m, s in enumerate(bounds(rows)):
        n = 0
        for r in range(s.start, s.stop):
            k = (idx[r] >= 0) & (idx[r] < V) & ~(t[r] == -np.inf)
            n += k.any()
        for r in range(s.start, s.stop):
            k = (idx[r] >= 0) & (idx[r] < V) & ~(t[r] == -np.inf)
            if not k.any():
                continue
            z = Z[r] / T
            fin = np.isfinite(z)
            a = np.where(fin, z.max() - z, 0)
            A = a.max()
            x = t[r][k] / T
            b = x.max() - x
            # the sum of exponentials: its additions, a rescaling (4u and its
            # argument) with every new maximum, of which there are at most as
            # many as terms in a row; the terms weigh their own errors
            rel_s = U * (5 * depth(V) + 12 + 5 * A)
            rel_p = rel_s + U * (8 + 5 * a)
            rel_sq = U * (depth(K) + 10 + 4 * b.max())
            q = np.exp(-b)
            q /= q.sum()
            rel_q = rel_sq + U * (6 + 4 * b)
            p = np.where(fin, np.exp(-a), 0)
            p /= p.sum()
            log_s = np.log(np.where(fin, np.exp(-a), 0).sum())
            lq = np.log(q)
            lp = -a[idx[r][k]] - log_s
            e_l = rel_sq + rel_s + U * (6 + 5 * b + 5 * a[idx[r][k]] + 4 * abs(log_s))
            t_row[r] = T * T * ((q * (e_l + (rel_q + U * (depth(K) + 6)) * np.abs(lq - lp))).sum()) * 1.001
            e = p * (rel_p + 4 * U)
            qq, eq = np.zeros(V), np.zeros(V)
            np.add.at(qq, idx[r][k], q)
            np.add.at(eq, idx[r][k], q * (rel_q + (K + 4) * U))
            w = abs(gscale) * T / n
            e = w * (e + eq + 2 * U * np.abs(p - qq)) * 1.001
            t_dZ[r] = e + half(dt) * (w * np.abs(p - qq) + e) + tiny(dt)
    return t_row, t_dZ
