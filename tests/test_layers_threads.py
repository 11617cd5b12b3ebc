"""Layer calls of two handles from two host threads at once, with sizes that ask
for different amounts of shared memory of the same kernel: every call succeeds
and gives what it gives alone."""
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import sign_muon_optimizer_b200 as smo  # noqa: E402

ROUNDS = 4000


def together(jobs, rounds=ROUNDS):
    """Every job's calls in a thread of its own; what they raised."""
    errors, start = [], threading.Barrier(len(jobs))

    def loop(job):
        try:
            start.wait(60)
            for _ in range(rounds):
                job()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


def handle(shapes, rows, cols):
    stream = torch.cuda.Stream()
    opt = smo.SignMuon(shapes, 1, flags=smo.SIGNMUON_VOTE_ONLY, stream=stream.cuda_stream)
    opt.layers_reserve(rows, cols)
    opt.keep = stream
    return opt


def test_distill_of_two_row_lengths_from_two_threads():
    """bf16 rows of 128256 and 64000 logits: one kernel, which holds more of the
    longer rows in shared memory."""
    jobs, checks = [], []
    for V in (128256, 64000):
        opt = handle([(1, 4)], 2, 4)
        g = torch.Generator(device="cuda").manual_seed(V)
        Z = torch.randn(2, V, generator=g, device="cuda").bfloat16()
        idx = torch.randint(0, V, (2, 4), generator=g, device="cuda")
        t, loss, dZ = torch.randn(2, 4, generator=g, device="cuda"), torch.zeros(1, device="cuda"), torch.empty_like(Z)
        call = lambda o=opt, z=Z, i=idx, t=t, s=loss, d=dZ: o.distill(z, i, t, s, dZ=d)  # noqa: E731
        torch.cuda.synchronize()
        call()
        opt.layers_sync()
        checks.append((opt, loss, loss.clone(), dZ, dZ.clone()))
        jobs.append(call)
    torch.cuda.synchronize()
    assert together(jobs) == []
    for opt, loss, want, dZ, grad in checks:
        opt.layers_sync()
        assert torch.equal(loss, want) and torch.equal(dZ, grad)


def test_table_gradients_of_two_sizes_from_two_threads():
    """Tables of 400 and 600 rows: the sort of 2500 tokens in one block, with
    digits of 9 and of 5 bits."""
    jobs, checks = [], []
    for V in (400, 600):
        opt = handle([(V, 8)], 2500, 8)
        g = torch.Generator(device="cuda").manual_seed(V)
        ids = torch.randint(0, V, (2500,), generator=g, device="cuda")
        dY, G = torch.randn(2500, 8, generator=g, device="cuda"), torch.zeros(V * 8, device="cuda")
        call = lambda o=opt, i=ids, d=dY, G=G: o.embed_grad(0, i, d, [G])  # noqa: E731
        torch.cuda.synchronize()
        call()
        opt.layers_sync()
        checks.append((opt, G, G.clone()))
        jobs.append(call)
    torch.cuda.synchronize()
    assert together(jobs) == []
    for opt, G, want in checks:
        opt.layers_sync()
        assert torch.equal(G, want)
