"""CPU-side checks of the layer calls: declared and exported symbols, null
handles, and the refusals of the tensor methods (no kernel is launched)."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import sign_muon_optimizer_b200 as smo
from sign_muon_optimizer_b200 import layers

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "signmuon_layers.h")


def test_library_exports_every_declared_layer_call():
    names = sorted(set(re.findall(r"^int (signmuon_[a-z_0-9]+)\s*\(", open(HEADER).read(), re.M)))
    lib = ctypes.CDLL(smo.LIB_PATH)
    for n in names:
        assert hasattr(lib, n)
        assert callable(getattr(smo, n))
    assert sorted(smo.EXPORTED_LAYERS) == names


def test_header_constants():
    text = open(HEADER).read()
    for name in ("SIGNMUON_F32", "SIGNMUON_BF16", "SIGNMUON_F16", "SIGNMUON_I32", "SIGNMUON_I64",
                 "SIGNMUON_LAYERNORM_MAX_COLS", "SIGNMUON_DISTILL_MAX_K"):
        assert int(re.search(r"#define %s\s+(\d+)" % name, text).group(1)) == getattr(smo, name)


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "c.c"
    src.write_text('#include "signmuon_layers.h"\nint main(void) { return signmuon_layers_sync(0) == SIGNMUON_E_INVALID ? 0 : 1; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", str(src), "-o",
                    str(tmp_path / "c.o")], check=True)


_NULL = """
import sys
sys.path.insert(0, {root!r})
import sign_muon_optimizer_b200 as smo
L = smo._lib
n = None
calls = {{
    "signmuon_layers_reserve": (n, 1, 1), "signmuon_layers_sync": (n,),
    "signmuon_embed": (n, n, 0, n, 0, 1, 1.0, n, 0, 1),
    "signmuon_embed_grad": (n, 0, n, 0, n, 1.0, n, 0, 1, n, 0),
    "signmuon_layernorm": (n, n, 0, 0, 1, n, 1, n, 1, 0, 1.0, n, n),
    "signmuon_layernorm_grad": (n, n, 0, 0, n, n, 1, n, 1, n, n, n, 1, 0, n, 0),
    "signmuon_distill": (n, n, 0, 1, 1, n, 0, n, 0, 1, 1, n, 1.0, 1.0, n, n, n, n, 1),
}}
assert sorted(calls) == sorted(smo.EXPORTED_LAYERS)
bad = [k for k, a in calls.items() if getattr(L, k)(*a) != smo.SIGNMUON_E_INVALID or not L.signmuon_last_error(None)]
print("BAD" if bad else "ALL", bad)
"""


def test_every_layer_call_rejects_a_null_handle():
    res = subprocess.run([sys.executable, "-c", _NULL.format(root=ROOT)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stderr[-2000:]
    assert res.stdout.startswith("ALL"), res.stdout


class OnCpu(layers.LayerCalls):
    """The methods on a handle that does not exist: a call that gets past the
    checks ends at the library's null handle."""

    def __init__(self, shapes, M):
        self.shapes, self.M, self.h, self.device = shapes, M, None, 0
        self.d = sum(r * c for r, c in shapes)


class Dev:
    """A CPU tensor that says it is on a GPU: what the checks look at."""

    def __init__(self, t, index=0):
        self.t, self.device = t, torch.device("cuda", index)

    def get_device(self):
        return self.device.index

    def __getattr__(self, name):
        return getattr(self.t, name)


V, E, N, M = 10, 8, 6, 2


def opt():
    return OnCpu([(V, E), (1, E), (1, E), (1, 3)], M)


def dev(*shape, dtype=torch.float32, index=0):
    return Dev(torch.zeros(*shape, dtype=dtype), index)


def calls():
    """For each method its good arguments by name, and bad ones."""
    d = V * E + 2 * E + 3
    W, ids = dev(d), dev(N, dtype=torch.int64)
    G = [dev(d) for _ in range(M)]
    X = lambda: dev(N, E)  # noqa: E731
    vec = dev(N)
    bad_matrix = [dev(N, E, dtype=torch.float64), dev(N, E + 1), dev(N + 1, E), dev(N, E, index=1), torch.zeros(N, E),
                  Dev(torch.zeros(E, N).t()), Dev(torch.zeros(1, E).expand(N, E)), None]
    bad_ids = [dev(N, dtype=torch.int16), dev(N), Dev(torch.zeros(2 * N, dtype=torch.int64)[::2]), None]
    bad_W = [dev(d - 1), dev(d, dtype=torch.float64), Dev(torch.zeros(2 * d)[::2]), None]
    bad_G = [G[:1], [G[0], dev(d - 1)], [G[0], None]]
    bad_rows = [[3], [3, 4], [1, 2, 3]]
    yield "embed", dict(W=W, mat=0, ids=ids, out=X()), dict(W=bad_W, mat=[-1, 4], ids=bad_ids, out=bad_matrix)
    yield "embed_grad", dict(mat=0, ids=ids, dY=X(), G=G, rows=[2, 4]), dict(mat=[-1, 4], ids=bad_ids, dY=bad_matrix,
                                                                            G=bad_G, rows=bad_rows)
    yield "layernorm", dict(W=W, gamma=1, beta=2, X=X(), Y=X(), mean=vec, rstd=vec), dict(
        W=bad_W, gamma=[-1, 4], beta=[-1, 4], Y=bad_matrix + [dev(N, E, dtype=torch.bfloat16)], mean=[dev(N - 1)],
        rstd=[dev(N, dtype=torch.float64)], X=[dev(N, E + 1), dev(N)])
    yield "layernorm_grad", dict(W=W, gamma=1, beta=2, X=X(), dY=X(), mean=vec, rstd=vec, dX=X(), G=G, rows=None), dict(
        W=bad_W, dY=bad_matrix, dX=bad_matrix, mean=[None, dev(N - 1)], rstd=[None, dev(N - 1)], G=bad_G, rows=bad_rows)
    yield "distill", dict(Z=dev(N, V), idx=dev(N, 3, dtype=torch.int32), t=dev(N, 3), loss=dev(M), rows=[6, 0],
                          count=dev(M, dtype=torch.int32), row_loss=vec, dZ=dev(N, V)), dict(
        Z=[dev(N), dev(N, V, dtype=torch.int32)], idx=[dev(N, 4, dtype=torch.int32), dev(N, 3), None,
                                                      Dev(torch.zeros(N, 6, dtype=torch.int32)[:, :3])],
        t=[dev(N + 1, 3), dev(N, 3, dtype=torch.float64)], loss=[dev(M - 1), None], rows=bad_rows,
        count=[dev(M)], row_loss=[dev(N - 1)], dZ=[dev(N, V + 1), dev(N, V, dtype=torch.float16)])


@pytest.mark.parametrize("name", ["embed", "embed_grad", "layernorm", "layernorm_grad", "distill"])
def test_methods_refuse_bad_tensors(name):
    good, bad = next((g, b) for n, g, b in calls() if n == name)
    o = opt()
    with pytest.raises(smo.SignMuonError) as e:   # past the checks: the null handle
        getattr(o, name)(**good)
    assert e.value.status == smo.SIGNMUON_E_INVALID
    for arg, values in bad.items():
        for v in values:
            with pytest.raises((TypeError, ValueError)):
                getattr(o, name)(**dict(good, **{arg: v}))


def test_rows_default_to_equal_shares():
    with pytest.raises(ValueError):
        layers._share(opt(), None, 7)
    assert list(layers._share(opt(), None, 8)) == [4, 4]


def test_no_layer_kernel_spills_or_keeps_a_stack_frame(tmp_path):
    from concurrent.futures import ThreadPoolExecutor

    import test_build_resources as resources
    nvcc = resources._nvcc()
    if nvcc is None:
        pytest.skip("no nvcc")
    sources = sorted(f for f in os.listdir(resources.CSRC) if f.startswith("layers_") and f != "layers_api.cu" and f.endswith(".cu"))
    assert len(sources) == 4
    with ThreadPoolExecutor(max_workers=4) as ex:
        reports = list(ex.map(lambda s: resources._ptxas_report(nvcc, s, str(tmp_path)), sources))
    found = {name: frame for rep in reports for name, (frame, _) in rep.items()}
    assert len(found) >= 60
    # the 512-thread distillation kernels may keep a few bytes: 40 registers let
    # a third block onto an SM, which is worth 324 against 376 us
    assert not {name: frame for name, frame in found.items()
                if frame != (0, 0, 0) and not ("k_distill_rows" in name and "Li512ELb1ELb0E" in name and frame[0] <= 16)}
