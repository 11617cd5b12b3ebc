"""Python binding of include/signmuon_layers.h: the embedding lookup, layer
norm and distillation loss of a training pass over M workers' rows, with the
gradients per worker, as signmuon_step reads them.

The functions keep the C names and only marshal; the methods of SignMuon
(``opt.layers_reserve``, ``opt.embed``, ...) also check shapes, types, strides
and devices of the tensors and take sizes from them.  Nothing here computes.
"""
from __future__ import annotations

import ctypes
from array import array
from operator import attrgetter

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

_types = {}     # torch dtype -> type code, filled with the first tensor: the package itself does not import torch
_id_types = {}
_dtype_of = attrgetter("dtype")


def _fill_types():
    import torch
    _types.update({torch.float32: SIGNMUON_F32, torch.bfloat16: SIGNMUON_BF16, torch.float16: SIGNMUON_F16,
                   "Tensor": torch.Tensor, "float32": {torch.float32}})
    _id_types.update({torch.int32: SIGNMUON_I32, torch.int64: SIGNMUON_I64})


def _declare(lib):
    P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    PP = PI64 = P    # addresses of arrays: array.array is several times quicker to make than a ctypes array
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
    """Row counts as an array; its address is arr.buffer_info()[0]."""
    return array("q", rows)


# ---- functions with the C names -------------------------------------------

def signmuon_layers_reserve(h, max_rows, max_cols):
    _check(h, _lib.signmuon_layers_reserve(h, int(max_rows), int(max_cols)))


def signmuon_layers_sync(h):
    _check(h, _lib.signmuon_layers_sync(h))


def signmuon_embed(h, W, mat, ids, id_type, n, scale, out, type, ld):
    _check(h, _lib.signmuon_embed(h, _ptr(W), mat, _ptr(ids), id_type, n, scale, _ptr(out), type, ld))


def signmuon_embed_grad(h, mat, ids, id_type, rows, scale, dY, type, ld, G, accumulate):
    r = _rows_arr(rows)
    _check(h, _lib.signmuon_embed_grad(h, mat, _ptr(ids), id_type, r.buffer_info()[0], scale, _ptr(dY), type, ld,
                                       _ptr_array(G), accumulate))


def signmuon_layernorm(h, W, gamma, beta, n, X, ldx, Y, ldy, type, eps, mean, rstd):
    _check(h, _lib.signmuon_layernorm(h, _ptr(W), gamma, beta, n, _ptr(X), ldx, _ptr(Y), ldy, type, eps, _ptr(mean),
                                      _ptr(rstd)))


def signmuon_layernorm_grad(h, W, gamma, beta, rows, X, ldx, dY, ldy, mean, rstd, dX, ldd, type, G, accumulate):
    r = _rows_arr(rows)
    _check(h, _lib.signmuon_layernorm_grad(h, _ptr(W), gamma, beta, r.buffer_info()[0], _ptr(X), ldx, _ptr(dY), ldy,
                                           _ptr(mean), _ptr(rstd), _ptr(dX), ldd, type, _ptr_array(G), accumulate))


def signmuon_distill(h, Z, type, ldz, V, idx, id_type, t, t_type, ldt, K, rows, temperature, gscale, loss, count,
                     row_loss, dZ, ldd):
    r = _rows_arr(rows)
    _check(h, _lib.signmuon_distill(h, _ptr(Z), type, ldz, V, _ptr(idx), id_type, _ptr(t), t_type, ldt, K,
                                    r.buffer_info()[0], temperature, gscale, _ptr(loss), _ptr(count), _ptr(row_loss),
                                    _ptr(dZ), ldd))


# ---- checks of the methods --------------------------------------------------
# (they run before every launch, so they look at each tensor with few calls)

def _wrong_device(opt, name, x):
    if not hasattr(x, "get_device"):
        return TypeError(f"{name}: a torch tensor is wanted, got {type(x).__name__}")
    return ValueError(f"{name} is on {x.device}, the handle on cuda:{opt.device}")


def _device_of(x):
    try:
        return x.get_device()
    except AttributeError:
        return None


def _matrix(opt, name, x, n=None, cols=None, code=None):
    """Type code and row stride of a 2-D activation with unit column stride."""
    if _device_of(x) != opt.device:
        raise _wrong_device(opt, name, x)
    if not _types:
        _fill_types()
    got = _types.get(x.dtype)
    if got is None or (code is not None and got != code):
        raise TypeError(f"{name} is {x.dtype}, wanted float32, bfloat16 or float16, one type for all activations")
    shape = x.shape
    if len(shape) != 2 or (n is not None and shape[0] != n) or (cols is not None and shape[1] != cols):
        raise ValueError(f"{name} has shape {tuple(shape)}, wanted ({'rows' if n is None else n}, "
                         f"{'columns' if cols is None else cols})")
    ld, one = x.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the elements of a row must be adjacent")
    if ld < shape[1]:
        if shape[0] > 1:
            raise ValueError(f"{name}: rows overlap (row stride {ld})")
        ld = shape[1]
    return got, ld


def _vector(opt, name, x, n, integer=False):
    """The address of n adjacent float32 (or int32) elements."""
    if _device_of(x) != opt.device:
        raise _wrong_device(opt, name, x)
    if not _types:
        _fill_types()
    if (_id_types if integer else _types).get(x.dtype) != 0:
        raise TypeError(f"{name} is {x.dtype}, wanted {'int32' if integer else 'float32'}")
    if x.numel() < n or not x.is_contiguous():
        raise ValueError(f"{name}: {n} adjacent elements are wanted, got shape {tuple(x.shape)}, strides {x.stride()}")
    return x.data_ptr()


def _id_type(opt, name, x):
    if _device_of(x) != opt.device:
        raise _wrong_device(opt, name, x)
    if not _types:
        _fill_types()
    code = _id_types.get(x.dtype)
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
        rows = [n // opt.M] * opt.M
    elif len(rows) != opt.M or sum(rows) != n:
        raise ValueError(f"rows must be {opt.M} counts that add up to {n}, got {list(rows)}")
    return array("q", rows)


def _grads(opt, G):
    """Addresses of the M gradient vectors."""
    if len(G) != opt.M:
        raise ValueError(f"G has {len(G)} vectors, wanted one for each of {opt.M} workers")
    if not _types:
        _fill_types()
    T = _types["Tensor"]
    try:
        if (set(map(T.get_device, G)) == {opt.device} and set(map(_dtype_of, G)) == _types["float32"]
                and min(map(T.numel, G)) >= opt.d and all(map(T.is_contiguous, G))):
            return array("Q", map(T.data_ptr, G))
    except TypeError:                    # not a tensor
        pass
    return array("Q", [_vector(opt, "G[m]", g, opt.d) for g in G])   # says which, and what is wrong


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
        w = _vector(self, "W", W, self.d)
        id_type, n = _ids(self, "ids", ids)
        code, ld = _matrix(self, "out", out, n, cols)
        rc = _lib.signmuon_embed(self.h, w, mat, ids.data_ptr(), id_type, n, scale, out.data_ptr(), code, ld)
        if rc:
            _check(self.h, rc)

    def embed_grad(self, mat, ids, dY, G, rows=None, scale=1.0, accumulate=False):
        """G[m][mat][v] = scale * sum of dY[r] over worker m's rows with ids[r] = v."""
        cols = _mat(self, "mat", mat)[1]
        id_type, n = _ids(self, "ids", ids)
        code, ld = _matrix(self, "dY", dY, n, cols)
        r, g = _share(self, rows, n), _grads(self, G)
        rc = _lib.signmuon_embed_grad(self.h, mat, ids.data_ptr(), id_type, r.buffer_info()[0], scale, dY.data_ptr(),
                                      code, ld, g.buffer_info()[0], bool(accumulate))
        if rc:
            _check(self.h, rc)

    def _norm_cols(self, gamma, beta):
        r, c = _mat(self, "gamma", gamma)
        if beta is not None:
            _mat(self, "beta", beta)
        return r * c

    def layernorm(self, W, gamma, beta, X, Y, mean=None, rstd=None, eps=1e-5):
        """Y = (X - mean) * rstd * W[gamma] + W[beta]; beta may be None."""
        cols = self._norm_cols(gamma, beta)
        w = _vector(self, "W", W, self.d)
        code, ldx = _matrix(self, "X", X, None, cols)
        n = X.shape[0]
        _, ldy = _matrix(self, "Y", Y, n, cols, code)
        mean = None if mean is None else _vector(self, "mean", mean, n)
        rstd = None if rstd is None else _vector(self, "rstd", rstd, n)
        rc = _lib.signmuon_layernorm(self.h, w, gamma, -1 if beta is None else beta, n, X.data_ptr(), ldx, Y.data_ptr(),
                                     ldy, code, eps, mean, rstd)
        if rc:
            _check(self.h, rc)

    def layernorm_grad(self, W, gamma, beta, X, dY, mean, rstd, dX, G, rows=None, accumulate=False):
        """dX, and per worker the gradients of W[gamma] and W[beta] in G[m]."""
        cols = self._norm_cols(gamma, beta)
        w = _vector(self, "W", W, self.d)
        code, ldx = _matrix(self, "X", X, None, cols)
        n = X.shape[0]
        _, ldy = _matrix(self, "dY", dY, n, cols, code)
        _, ldd = _matrix(self, "dX", dX, n, cols, code)
        r, g = _share(self, rows, n), _grads(self, G)
        rc = _lib.signmuon_layernorm_grad(self.h, w, gamma, -1 if beta is None else beta, r.buffer_info()[0],
                                          X.data_ptr(), ldx, dY.data_ptr(), ldy, _vector(self, "mean", mean, n),
                                          _vector(self, "rstd", rstd, n), dX.data_ptr(), ldd, code, g.buffer_info()[0],
                                          bool(accumulate))
        if rc:
            _check(self.h, rc)

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
        to = _vector(self, "loss", loss, self.M)
        count = None if count is None else _vector(self, "count", count, self.M, True)
        row_loss = None if row_loss is None else _vector(self, "row_loss", row_loss, n)
        grad, ldd = None, V
        if dZ is not None:
            ldd = _matrix(self, "dZ", dZ, n, V, code)[1]
            grad = dZ.data_ptr()
        r = _share(self, rows, n)
        rc = _lib.signmuon_distill(self.h, Z.data_ptr(), code, ldz, V, idx.data_ptr(), id_type, t.data_ptr(), t_code, ldt,
                                   K, r.buffer_info()[0], temperature, gscale, to, count, row_loss, grad, ldd)
        if rc:
            _check(self.h, rc)
