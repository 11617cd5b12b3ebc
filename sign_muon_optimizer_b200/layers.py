"""Python binding of include/signmuon_layers.h: the embedding lookup, layer
norm and distillation loss of a training pass over M workers' rows, with the
gradients per worker, as signmuon_step reads them.

The functions keep the C names and only marshal; the methods of SignMuon
(``opt.layers_reserve``, ``opt.embed``, ...) also check shapes, types, strides
and devices of the tensors and take sizes from them.  Nothing here computes.
"""
from __future__ import annotations

import ctypes

SIGNMUON_F32 = 0
SIGNMUON_BF16 = 1
SIGNMUON_F16 = 2
SIGNMUON_I32 = 0
SIGNMUON_I64 = 1
SIGNMUON_LAYERNORM_MAX_COLS = 16384
SIGNMUON_DISTILL_MAX_K = 1024

EXPORTED_LAYERS = [
    "signmuon_layers_reserve", "signmuon_layers_sync", "signmuon_embed", "signmuon_embed_grad",
    "signmuon_layernorm", "signmuon_layernorm_grad", "signmuon_distill",
]

__all__ = EXPORTED_LAYERS + [
    "EXPORTED_LAYERS", "SIGNMUON_F32", "SIGNMUON_BF16", "SIGNMUON_F16", "SIGNMUON_I32", "SIGNMUON_I64",
    "SIGNMUON_LAYERNORM_MAX_COLS", "SIGNMUON_DISTILL_MAX_K",
]

# by the dtype's name: the package itself does not import torch
_TYPES = {"torch.float32": SIGNMUON_F32, "torch.bfloat16": SIGNMUON_BF16, "torch.float16": SIGNMUON_F16}
_ID_TYPES = {"torch.int32": SIGNMUON_I32, "torch.int64": SIGNMUON_I64}


def _declare(lib):
    P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    PP, PI64 = ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_int64)
    sig = {
        "signmuon_layers_reserve": [P, I64, I64],
        "signmuon_layers_sync": [P],
        "signmuon_embed": [P, P, I, P, I, I64, F, P, I, I64],
        "signmuon_embed_grad": [P, I, P, I, PI64, F, P, I, I64, PP, I],
        "signmuon_layernorm": [P, P, I, I, I64, P, I64, P, I64, I, F, P, P],
        "signmuon_layernorm_grad": [P, P, I, I, PI64, P, I64, P, I64, P, P, P, I64, I, PP, I],
        "signmuon_distill": [P, P, I, I64, I64, P, I, P, I, I64, I, PI64, F, F, P, P, P, P, I64],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.restype = I
        fn.argtypes = args


from . import _check, _lib, _ptr, _ptr_array  # noqa: E402  (the package imports this module when they exist)

_declare(_lib)


def _rows_arr(rows):
    return (ctypes.c_int64 * max(1, len(rows)))(*rows)


# ---- functions with the C names -------------------------------------------

def signmuon_layers_reserve(h, max_rows, max_cols):
    _check(h, _lib.signmuon_layers_reserve(h, int(max_rows), int(max_cols)))


def signmuon_layers_sync(h):
    _check(h, _lib.signmuon_layers_sync(h))


def signmuon_embed(h, W, mat, ids, id_type, n, scale, out, type, ld):
    _check(h, _lib.signmuon_embed(h, _ptr(W), mat, _ptr(ids), id_type, n, scale, _ptr(out), type, ld))


def signmuon_embed_grad(h, mat, ids, id_type, rows, scale, dY, type, ld, G, accumulate):
    _check(h, _lib.signmuon_embed_grad(h, mat, _ptr(ids), id_type, _rows_arr(rows), scale, _ptr(dY), type, ld,
                                       _ptr_array(G), accumulate))


def signmuon_layernorm(h, W, gamma, beta, n, X, ldx, Y, ldy, type, eps, mean, rstd):
    _check(h, _lib.signmuon_layernorm(h, _ptr(W), gamma, beta, n, _ptr(X), ldx, _ptr(Y), ldy, type, eps, _ptr(mean),
                                      _ptr(rstd)))


def signmuon_layernorm_grad(h, W, gamma, beta, rows, X, ldx, dY, ldy, mean, rstd, dX, ldd, type, G, accumulate):
    _check(h, _lib.signmuon_layernorm_grad(h, _ptr(W), gamma, beta, _rows_arr(rows), _ptr(X), ldx, _ptr(dY), ldy,
                                           _ptr(mean), _ptr(rstd), _ptr(dX), ldd, type, _ptr_array(G), accumulate))


def signmuon_distill(h, Z, type, ldz, V, idx, id_type, t, t_type, ldt, K, rows, temperature, gscale, loss, count,
                     row_loss, dZ, ldd):
    _check(h, _lib.signmuon_distill(h, _ptr(Z), type, ldz, V, _ptr(idx), id_type, _ptr(t), t_type, ldt, K,
                                    _rows_arr(rows), temperature, gscale, _ptr(loss), _ptr(count), _ptr(row_loss),
                                    _ptr(dZ), ldd))


# ---- checks of the methods --------------------------------------------------

def _on(opt, name, x):
    if not hasattr(x, "is_cuda"):
        raise TypeError(f"{name}: a torch tensor is wanted, got {type(x).__name__}")
    if not x.is_cuda or x.device.index != opt.device:
        raise ValueError(f"{name} is on {x.device}, the handle on cuda:{opt.device}")


def _matrix(opt, name, x, n=None, cols=None, dtype=None):
    """Type code and row stride of a 2-D activation with unit column stride."""
    _on(opt, name, x)
    code = _TYPES.get(str(x.dtype))
    if code is None or (dtype is not None and x.dtype != dtype):
        raise TypeError(f"{name} is {x.dtype}, wanted {dtype or 'float32, bfloat16 or float16'}")
    if x.dim() != 2 or (n is not None and x.shape[0] != n) or (cols is not None and x.shape[1] != cols):
        raise ValueError(f"{name} has shape {tuple(x.shape)}, wanted ({'rows' if n is None else n}, "
                         f"{'columns' if cols is None else cols})")
    ld, one = x.stride()
    if x.shape[1] > 1 and one != 1:
        raise ValueError(f"{name}: the elements of a row must be adjacent")
    if x.shape[0] > 1 and ld < x.shape[1]:
        raise ValueError(f"{name}: rows overlap (row stride {ld})")
    return code, max(ld, x.shape[1])


def _vector(opt, name, x, n, dtype="torch.float32"):
    _on(opt, name, x)
    if str(x.dtype) != dtype:
        raise TypeError(f"{name} is {x.dtype}, wanted {dtype}")
    if x.numel() < n or not x.is_contiguous():
        raise ValueError(f"{name}: {n} adjacent elements are wanted, got shape {tuple(x.shape)}, strides {x.stride()}")


def _id_type(opt, name, x):
    _on(opt, name, x)
    code = _ID_TYPES.get(str(x.dtype))
    if code is None:
        raise TypeError(f"{name} is {x.dtype}, wanted int32 or int64")
    return code


def _ids(opt, name, x):
    code = _id_type(opt, name, x)
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return code, x.numel()


def _share(opt, rows, n):
    """Row counts of the workers: as given, or n split evenly."""
    if rows is None:
        if n % opt.M:
            raise ValueError(f"{n} rows do not split evenly over {opt.M} workers: give rows")
        return [n // opt.M] * opt.M
    if len(rows) != opt.M or sum(rows) != n:
        raise ValueError(f"rows must be {opt.M} counts that add up to {n}, got {list(rows)}")
    return rows


def _grads(opt, G):
    if len(G) != opt.M:
        raise ValueError(f"G has {len(G)} vectors, wanted one for each of {opt.M} workers")
    for m, g in enumerate(G):
        _vector(opt, "G[%d]" % m, g, opt.d)


def _mat(opt, name, mat):
    if not 0 <= mat < len(opt.shapes):
        raise ValueError(f"{name} = {mat}: the handle has {len(opt.shapes)} matrices")
    return opt.shapes[mat]


class LayerCalls:
    """The layer calls as methods of SignMuon (see include/signmuon_layers.h
    for what each computes).  Tensors are on the handle's device and are used on
    the handle's stream; W and every G[m] are flat float32 vectors of d
    elements."""

    def layers_reserve(self, max_rows, max_cols):
        signmuon_layers_reserve(self.h, max_rows, max_cols)

    def layers_sync(self):
        signmuon_layers_sync(self.h)

    def embed(self, W, mat, ids, out, scale=1.0):
        """out[r] = scale * W[mat][ids[r]]; a negative id gives a row of zeros."""
        cols = _mat(self, "mat", mat)[1]
        _vector(self, "W", W, self.d)
        id_type, n = _ids(self, "ids", ids)
        code, ld = _matrix(self, "out", out, n, cols)
        signmuon_embed(self.h, W, mat, ids, id_type, n, scale, out, code, ld)

    def embed_grad(self, mat, ids, dY, G, rows=None, scale=1.0, accumulate=False):
        """G[m][mat][v] = scale * sum of dY[r] over worker m's rows with ids[r] = v."""
        cols = _mat(self, "mat", mat)[1]
        id_type, n = _ids(self, "ids", ids)
        code, ld = _matrix(self, "dY", dY, n, cols)
        _grads(self, G)
        signmuon_embed_grad(self.h, mat, ids, id_type, _share(self, rows, n), scale, dY, code, ld, G, bool(accumulate))

    def _norm_cols(self, gamma, beta):
        r, c = _mat(self, "gamma", gamma)
        if beta is not None:
            _mat(self, "beta", beta)
        return r * c

    def layernorm(self, W, gamma, beta, X, Y, mean=None, rstd=None, eps=1e-5):
        """Y = (X - mean) * rstd * W[gamma] + W[beta]; beta may be None."""
        cols = self._norm_cols(gamma, beta)
        _vector(self, "W", W, self.d)
        code, ldx = _matrix(self, "X", X, None, cols)
        n = X.shape[0]
        _, ldy = _matrix(self, "Y", Y, n, cols, X.dtype)
        if mean is not None:
            _vector(self, "mean", mean, n)
        if rstd is not None:
            _vector(self, "rstd", rstd, n)
        signmuon_layernorm(self.h, W, gamma, -1 if beta is None else beta, n, X, ldx, Y, ldy, code, eps, mean, rstd)

    def layernorm_grad(self, W, gamma, beta, X, dY, mean, rstd, dX, G, rows=None, accumulate=False):
        """dX, and per worker the gradients of W[gamma] and W[beta] in G[m]."""
        cols = self._norm_cols(gamma, beta)
        _vector(self, "W", W, self.d)
        code, ldx = _matrix(self, "X", X, None, cols)
        n = X.shape[0]
        _, ldy = _matrix(self, "dY", dY, n, cols, X.dtype)
        _, ldd = _matrix(self, "dX", dX, n, cols, X.dtype)
        _vector(self, "mean", mean, n)
        _vector(self, "rstd", rstd, n)
        _grads(self, G)
        signmuon_layernorm_grad(self.h, W, gamma, -1 if beta is None else beta, _share(self, rows, n), X, ldx, dY, ldy,
                                mean, rstd, dX, ldd, code, G, bool(accumulate))

    def distill(self, Z, idx, t, loss, rows=None, count=None, row_loss=None, dZ=None, temperature=1.0, gscale=1.0):
        """Distillation loss per worker from the teacher's entries (idx, t) and,
        with dZ, its gradient with respect to the logits Z."""
        code, ldz = _matrix(self, "Z", Z)
        n, V = Z.shape
        t_code, ldt = _matrix(self, "t", t, n)
        K = t.shape[1]
        id_type = _id_type(self, "idx", idx)
        if idx.shape != t.shape or (n > 1 and idx.stride(0) != t.stride(0)) or (K > 1 and idx.stride(1) != 1):
            raise ValueError(f"idx (shape {tuple(idx.shape)}, strides {idx.stride()}) must be laid out like t "
                             f"(shape {tuple(t.shape)}, strides {t.stride()})")
        _vector(self, "loss", loss, self.M)
        if count is not None:
            _vector(self, "count", count, self.M, "torch.int32")
        if row_loss is not None:
            _vector(self, "row_loss", row_loss, n)
        ldd = V
        if dZ is not None:
            _, ldd = _matrix(self, "dZ", dZ, n, V, Z.dtype)
        signmuon_distill(self.h, Z, code, ldz, V, idx, id_type, t, t_code, ldt, K, _share(self, rows, n), temperature,
                         gscale, loss, count, row_loss, dZ, ldd)
