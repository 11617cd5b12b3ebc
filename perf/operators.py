"""Cases, plain forms and exact results of the layer operators.

The operators are the parts of a training pass over M workers' rows that are
not weight products: the embedding lookup and its gradient, layer norm forward
and backward, and the distillation loss with its gradient.  What belongs to a
worker (the gradients of the parameters, the loss) comes out per worker.
Rows are joined in worker order; ``_rows`` says how many each worker has.
"""
import torch

own = False

F32, BF16, F16 = "float32", "bfloat16", "float16"
LN_EPS = 1e-5


def listed():
    return [
        # one token per worker: the lookup of a sampling step between training steps, where latency counts
        dict(name="lookup_8_tokens", op="embed", M=8, N=8, V=50304, E=768, dtype=BF16, ragged=False),
        # 8 workers x 16 sequences x 1024 tokens
        dict(name="lookup_131072_tokens", op="embed", M=8, N=131072, V=50304, E=768, dtype=BF16, ragged=False),
        # a small model's table, float32 throughout: the smallest gradient
        dict(name="embed_grad_small", op="embed_grad", M=3, N=120, V=1000, E=256, dtype=F32, ragged=False),
        # the largest: every worker's dense table gradient from its own 16,384 tokens on average, one worker without any
        dict(name="embed_grad_131072_ragged", op="embed_grad", M=8, N=131072, V=50304, E=768, dtype=BF16, ragged=True),
        # odd table and odd width: no row starts on a 16-byte boundary
        dict(name="embed_grad_odd", op="embed_grad", M=4, N=9001, V=8191, E=1001, dtype=F16, ragged=True),
        # one token per worker through a norm
        dict(name="layernorm_8_rows", op="layernorm", M=8, N=8, V=0, E=768, dtype=BF16, ragged=False),
        # a training batch through one norm
        dict(name="layernorm_131072_rows", op="layernorm", M=8, N=131072, V=0, E=768, dtype=BF16, ragged=False),
        # odd width in float32, few rows
        dict(name="layernorm_grad_odd", op="layernorm_grad", M=3, N=1023, V=0, E=1001, dtype=F32, ragged=True),
        # 16 workers, wide rows: a larger model's norm
        dict(name="layernorm_grad_32768_wide", op="layernorm_grad", M=16, N=32768, V=0, E=4096, dtype=BF16, ragged=True),
        # a classifier's 1000 outputs, small batch
        dict(name="distill_small", op="distill", M=3, N=48, V=1000, K=8, dtype=F32, grad=True, ragged=False),
        # 8 workers x 1024 tokens over a whole vocabulary, 64 teacher logits a token
        dict(name="distill_8192_rows", op="distill", M=8, N=8192, V=50304, K=64, dtype=BF16, grad=True, ragged=False),
        # evaluation, loss only, odd vocabulary: rows start at every alignment
        dict(name="distill_loss_odd", op="distill", M=5, N=3001, V=32003, K=33, dtype=F16, grad=False, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "layernorm", "layernorm_grad", "distill"])
    c = dict(op=op, M=rng.randint(1, 16), dtype=rng.choice([F32, BF16, F16]), ragged=rng.random() < 0.5)
    if op == "distill":
        c["V"] = _log_int(rng, 500, 60000)
        c["K"] = _log_int(rng, 1, 128)
        c["N"] = _log_int(rng, 1, min(16384, 200_000_000 // c["V"]))
        c["grad"] = rng.random() < 0.7
        return c
    c["E"] = _log_int(rng, 64, 5000)
    if rng.random() < 0.5:
        c["E"] = max(64, c["E"] // 64 * 64)
    c["V"] = _log_int(rng, 100, 60000) if op.startswith("embed") else 0
    if op == "embed_grad":
        c["M"] = max(1, min(c["M"], 300_000_000 // (c["V"] * c["E"])))
    c["N"] = _log_int(rng, 1, min(131072, 100_000_000 // c["E"]))
    return c


def _rows(case):
    """Rows of each worker: equal shares, or uneven ones with every fifth worker empty."""
    M, N = case["M"], case["N"]
    w = [(3 * m + 1) % 5 if case["ragged"] else 1 for m in range(M)]
    rows = [N * x // sum(w) for x in w]
    rows[0] += N - sum(rows)
    return rows


def _pad4(n):
    return (n + 3) // 4 * 4


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    dev = dict(device="cuda")
    dt = getattr(torch, case["dtype"])
    M, N, op = case["M"], case["N"], case["op"]
    s = dict(case=case, rows=_rows(case), own=None)
    s["worker"] = torch.repeat_interleave(torch.arange(M, **dev), torch.tensor(s["rows"], **dev), output_size=N)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, dtype=dtype, **dev)

    def rand(*shape):
        return torch.rand(*shape, generator=g, **dev)

    if op == "distill":
        V, K = case["V"], case["K"]
        s["T"], s["gscale"] = 2.0, 1.0
        # the teacher's top logits, falling with the rank, at distinct places; one entry in ten of the later ones absent,
        # one row in fifty (padding of a batch) without any
        step = 1 + (rand(N, 1) * max(1, V // K - 1)).long()
        idx = ((rand(N, 1) * V).long() + step * torch.arange(K, **dev)) % V
        t = 8 - 2 * torch.log1p(torch.arange(K, **dev).float()) + 0.3 * randn(N, K)
        gone = (rand(N, K) < 0.1) & (torch.arange(K, **dev) > 0)
        gone |= rand(N, 1) < 0.02
        s["idx"] = torch.where(gone, -1, idx).to(torch.int32)
        s["t"] = t
        z = randn(N, V, dtype=dt).mul_(2)
        z.scatter_add_(1, idx[:, :1], torch.full((N, 1), 4.0, dtype=dt, **dev))
        s["Z"] = z
        s["loss"] = torch.empty(M, **dev)
        s["count"] = torch.empty(M, dtype=torch.int32, **dev)
        s["row_loss"] = torch.empty(N, **dev)
        s["dZ"] = torch.empty_like(z) if case["grad"] else None
        shapes, width = [(1, 4)], 4
    else:
        V, E = case["V"], case["E"]
        if op.startswith("embed"):
            # ids fall off like 1 / rank, as words do; one row in a hundred is padding
            ids = (float(V + 1) ** rand(N).double()).long().clamp_(1, V) - 1
            s["ids"] = torch.where(rand(N) < 0.01, -1, ids)
            s["scale"] = float(E) ** 0.5
            shapes = [(V, E)]
        else:
            shapes = [(1, E), (1, E)]
        d = sum(r * c for r, c in shapes)
        if op == "embed":
            s["W"] = randn(_pad4(d)).mul_(0.02)
            s["out"] = torch.empty(N, E, dtype=dt, **dev)
        elif op == "embed_grad":
            s["dY"] = randn(N, E, dtype=dt)
            s["G"] = torch.empty(M, _pad4(d), **dev)
        else:
            s["W"] = torch.cat([1 + 0.1 * randn(E), 0.1 * randn(E), torch.zeros(_pad4(d) - d, **dev)])
            # channels have their own offsets, a few of them large
            s["X"] = (randn(N, E) * 1.5 + randn(E) * (1 + 10 * (rand(E) < 0.01))).to(dt)
            if op == "layernorm":
                s["Y"] = torch.empty_like(s["X"])
                s["mean"], s["rstd"] = torch.empty(N, **dev), torch.empty(N, **dev)
            else:
                x = s["X"].float()
                mu = x.mean(1, keepdim=True)
                s["mean"] = mu[:, 0].contiguous()
                s["rstd"] = ((x - mu).square().mean(1) + LN_EPS).rsqrt()
                s["dY"] = randn(N, E, dtype=dt)
                s["dX"] = torch.empty_like(s["X"])
                s["G"] = torch.empty(M, _pad4(d), **dev)
        width = E
    if own:
        # the handle that a training program keeps
        import sign_muon_optimizer_b200 as smo
        opt = smo.SignMuon(shapes, M, flags=smo.SIGNMUON_VOTE_ONLY)
        opt.layers_reserve(N, width)
        s["own"] = opt
        if "G" in s:
            s["Gm"] = [s["G"][m] for m in range(M)]
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    c, opt = s["case"], s["own"]
    op = c["op"]
    if op == "embed":
        opt.embed(s["W"], 0, s["ids"], s["out"], scale=s["scale"])
        return s["out"]
    if op == "embed_grad":
        opt.embed_grad(0, s["ids"], s["dY"], s["Gm"], s["rows"], scale=s["scale"])
        return s["G"][:, :c["V"] * c["E"]].unflatten(1, (c["V"], c["E"]))
    if op == "layernorm":
        opt.layernorm(s["W"], 0, 1, s["X"], s["Y"], s["mean"], s["rstd"], eps=LN_EPS)
        return dict(Y=s["Y"], mean=s["mean"], rstd=s["rstd"])
    if op == "layernorm_grad":
        opt.layernorm_grad(s["W"], 0, 1, s["X"], s["dY"], s["mean"], s["rstd"], s["dX"], s["Gm"], s["rows"])
        E = c["E"]
        return dict(dX=s["dX"], dgamma=s["G"][:, :E], dbeta=s["G"][:, E:2 * E])
    opt.distill(s["Z"], s["idx"], s["t"], s["loss"], s["rows"], count=s["count"], row_loss=s["row_loss"], dZ=s["dZ"],
                temperature=s["T"], gscale=s["gscale"])
    out = dict(loss=s["loss"], count=s["count"], row_loss=s["row_loss"])
    return dict(out, dZ=s["dZ"]) if c["grad"] else out


def _run_plain(s):
    c = s["case"]
    op, M = c["op"], c["M"]
    dt = getattr(torch, c["dtype"])
    dev = s["worker"].device
    if op == "embed":
        V, E = c["V"], c["E"]
        ids = s["ids"]
        rows = s["W"][:V * E].view(V, E).index_select(0, ids.clamp(min=0)) * s["scale"]
        return torch.where((ids >= 0)[:, None], rows, 0.0).to(dt)
    if op == "embed_grad":
        V, E = c["V"], c["E"]
        ids = s["ids"]
        keep = ids >= 0
        dY = torch.where(keep[:, None], s["dY"].float(), 0.0)
        G = torch.zeros(M * V, E, device=dev)
        G.index_add_(0, s["worker"] * V + ids.clamp(min=0), dY)
        return G.mul_(s["scale"]).view(M, V, E)
    if op == "layernorm":
        E = c["E"]
        x = s["X"].float()
        mu = x.mean(1, keepdim=True)
        xc = x - mu
        rstd = (xc.square().mean(1, keepdim=True) + LN_EPS).rsqrt()
        y = xc * rstd * s["W"][:E] + s["W"][E:2 * E]
        return dict(Y=y.to(dt), mean=mu[:, 0], rstd=rstd[:, 0])
    if op == "layernorm_grad":
        E = c["E"]
        xh = (s["X"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dy = s["dY"].float()
        g = dy * s["W"][:E]
        dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
        dgamma = torch.zeros(M, E, device=dev).index_add_(0, s["worker"], dy * xh)
        dbeta = torch.zeros(M, E, device=dev).index_add_(0, s["worker"], dy)
        return dict(dX=dx.to(dt), dgamma=dgamma, dbeta=dbeta)
    T = s["T"]
    V = c["V"]
    idx = s["idx"].long()
    here = idx >= 0
    at = idx.clamp(min=0)
    some = here.any(1)
    t = torch.where(here, s["t"].float() / T, float("-inf"))
    e = torch.exp(t - torch.where(some, t.amax(1), 0.0)[:, None])
    q = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    logq = torch.where(q > 0, q, 1.0).log()
    z = s["Z"].float() / T
    zmax = z.amax(1, keepdim=True)
    ez = torch.exp(z - zmax)
    total = ez.sum(1, keepdim=True)
    logp = z.gather(1, at) - zmax - total.log()
    row = torch.where(q > 0, q * (logq - logp), 0.0).sum(1) * (T * T)
    count = torch.zeros(M, dtype=torch.int32, device=dev).index_add_(0, s["worker"], some.int())
    n = count.clamp(min=1).float()
    loss = torch.zeros(M, device=dev, dtype=torch.float64).index_add_(0, s["worker"], row.double()) / n
    out = dict(loss=loss.float(), count=count, row_loss=row)
    if c["grad"]:
        p = ez / total
        p.scatter_add_(1, at, -q)
        w = torch.where(some, s["gscale"] * T / n[s["worker"]], 0.0)
        out["dZ"] = (p * w[:, None]).to(dt)
    return out


def work(case):
    es = 4 if case["dtype"] == F32 else 2
    M, N, op = case["M"], case["N"], case["op"]
    if op == "distill":
        V, K = case["V"], case["K"]
        return dict(bytes=N * V * es * (2 if case["grad"] else 1) + N * K * 8 + 4 * N + 8 * M, flops=N * V * (6 if case["grad"] else 4))
    V, E = case["V"], case["E"]
    if op == "embed":
        return dict(bytes=N * 8 + min(N, V) * E * 4 + N * E * es, flops=N * E)
    if op == "embed_grad":
        return dict(bytes=N * 8 + N * E * es + M * V * E * 4, flops=N * E)
    if op == "layernorm":
        return dict(bytes=2 * N * E * es + 8 * N + 8 * E, flops=8 * N * E)
    return dict(bytes=3 * N * E * es + 8 * N + 4 * E + 8 * M * E, flops=14 * N * E)


def exact(case, seed):
    """The definitions in 64 bits, worker by worker and in blocks of rows."""
    s = prepare(case, seed)
    op, M, N = case["op"], case["M"], case["N"]
    bounds = [sum(s["rows"][:m]) for m in range(M + 1)]
    f64 = dict(dtype=torch.float64, device="cuda")
    if op == "embed":
        table = s["W"][:case["V"] * case["E"]].double().reshape(case["V"], case["E"])
        out = torch.zeros(N, case["E"], **f64)
        real = (s["ids"] >= 0).nonzero()[:, 0]
        out[real] = table[s["ids"][real]] * s["scale"]
        return out
    if op == "embed_grad":
        G = torch.zeros(M, case["V"], case["E"], **f64)
        for m in range(M):
            ids, dY = s["ids"][bounds[m]:bounds[m + 1]], s["dY"][bounds[m]:bounds[m + 1]].double()
            real = (ids >= 0).nonzero()[:, 0]
            G[m].index_put_((ids[real],), dY[real] * s["scale"], accumulate=True)
        return G
    if op == "layernorm":
        E = case["E"]
        X, gamma, beta = s["X"].double(), s["W"][:E].double(), s["W"][E:2 * E].double()
        var, mean = torch.var_mean(X, dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + LN_EPS)
        return dict(Y=(X - mean[:, None]) * (rstd[:, None] * gamma) + beta, mean=mean, rstd=rstd)
    if op == "layernorm_grad":
        E = case["E"]
        gamma = s["W"][:E].double()
        dX = torch.empty(N, E, **f64)
        dgamma, dbeta = torch.zeros(M, E, **f64), torch.zeros(M, E, **f64)
        for m in range(M):
            r = slice(bounds[m], bounds[m + 1])
            rstd = s["rstd"][r].double()[:, None]
            xh = (s["X"][r].double() - s["mean"][r].double()[:, None]) * rstd
            dY = s["dY"][r].double()
            dgamma[m], dbeta[m] = (dY * xh).sum(0), dY.sum(0)
            a = (dY @ gamma / E)[:, None]
            b = ((dY * xh) @ gamma / E)[:, None]
            dX[r] = rstd * (dY * gamma - a - xh * b)
        return dict(dX=dX, dgamma=dgamma, dbeta=dbeta)
    V, T = case["V"], s["T"]
    loss = torch.zeros(M, **f64)
    row_loss = torch.zeros(N, **f64)
    dZ = torch.empty(N, V, **f64) if case["grad"] else None
    for m in range(M):
        lo, hi = bounds[m], bounds[m + 1]
        counted = (s["idx"][lo:hi] >= 0).any(1)
        n = int(counted.sum())
        for a in range(lo, hi, 2048):
            b = min(hi, a + 2048)
            keep = counted[a - lo:b - lo, None]
            # the teacher's probabilities laid out over the vocabulary
            w = torch.where(s["idx"][a:b] >= 0, s["t"][a:b].double() / T, float("-inf"))
            w = torch.where(keep, w, 0.0)
            q = torch.softmax(w, 1) * keep
            full = torch.zeros(b - a, V, **f64).scatter_add_(1, s["idx"][a:b].clamp(min=0).long(), q)
            logp = torch.log_softmax(s["Z"][a:b].double() / T, 1)
            row_loss[a:b] = (torch.special.xlogy(full, full) - full * logp).sum(1) * T * T
            if dZ is not None:
                dZ[a:b] = (logp.exp() - full) * keep * (s["gscale"] * T / max(n, 1))
        loss[m] = row_loss[lo:hi].sum() / max(n, 1)
    return dict(loss=loss, count=None, row_loss=row_loss, dZ=dZ) if case["grad"] else dict(loss=loss, count=None, row_loss=row_loss)
