"""Norms around a block on a B200 at widths whose rings take between 48 KB less the kernels' static shared memory and 48 KB of dynamic
shared memory, where a launch depends on the kernel's limit having been raised: each width in a process in which it is the first
call of its kernel. And two host threads that call one kernel with different widths.

Tolerances as in test_gpu_block_norm.py: 1e-5 of the magnitudes that enter a value, and half a step of the stored type.
"""
import os
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

N = pytest.importorskip("mixture_experts_ffn_11_b200._native")

T = 300  # more than two rows per SM: rows come through the ring
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    N.get_device_error()
    yield
    torch.cuda.synchronize()
    assert N.get_device_error() == 0


def near(got, ref, size, what):
    h = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    err = (got.double() - ref).abs()
    assert (err <= 1e-5 * size + h * ref.abs() * (1 + 2e-5)).all(), what


def norm64(v):
    return (v.square().mean(1, keepdim=True) + EPS).rsqrt()


def inputs(d, res):
    g = torch.Generator(device="cuda").manual_seed(d)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return n(T, d).to(res), n(T, d).bfloat16(), 1 + 0.3 * n(d), n(1, d).bfloat16()


def norm_in(d, res):
    x, _, w, _ = inputs(d, res)
    xn, rstd = torch.empty(T, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, device="cuda")
    N.block_norm_in(x, w, EPS, xn, rstd)
    ref = x.double() * norm64(x.double()) * w.double()
    near(xn, ref, ref.abs(), ("norm_in", d, res))


def norm_out(d, res, gated, next_norm):
    r, y, w, gate = inputs(d, res)
    new = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    out, rstd, xn, rstd_next = torch.empty_like(r), new(T), new(T, d, t=torch.bfloat16), new(T)
    N.block_norm_out(y, r, w, gate if gated else None, T if gated else 0, 0.5, w if next_norm else None, EPS, out, rstd, xn, rstd_next)
    n = y.double() * norm64(y.double()) * w.double() * (gate.double() if gated else 1.0)
    near(out, 0.5 * r.double() + n, 0.5 * r.double().abs() + n.abs(), ("norm_out", d, res, gated, next_norm))
    if next_norm:
        ref = out.double() * norm64(out.double()) * w.double()
        near(xn, ref, ref.abs(), ("norm_out, next", d, res, gated))


def norm_in_grad(d, res):
    x, dxn, w, _ = inputs(d, res)
    dres, rstd = torch.randn(T, d, device="cuda").to(res), norm64(x.double())[:, 0].float()
    dx, dw = torch.empty_like(x), torch.empty(d, device="cuda")
    ws = torch.empty(N.block_norm_backward_workspace_size(T, d), dtype=torch.uint8, device="cuda")
    N.block_norm_in_backward(dxn, dres, x, w, rstd, dx, dw, ws)
    rs = rstd.double()[:, None]
    hat, dn = x.double() * rs, dxn.double() * w.double()
    ref = dres.double() + rs * (dn - hat * (dn * hat).mean(1, keepdim=True))
    near(dx, ref, dres.double().abs() + rs * (dn.abs() + hat.abs() * (dn * hat).abs().mean(1, keepdim=True)), ("norm_in_grad", d, res))
    near(dw, (dxn.double() * hat).sum(0), (dxn.double() * hat).abs().sum(0), ("norm_in_grad, dw", d, res))


BF, F32 = torch.bfloat16, torch.float32
# one process each, in which every call is the first of its kernel (in the order: stream type, vectors per thread, next norm or not)
FIRST = [
    [(norm_in, 3064, BF), (norm_in, 2040, F32), (norm_in, 12240, BF), (norm_out, 2040, BF, False, True), (norm_out, 1632, F32, False, True),
     (norm_in_grad, 816, F32), (norm_out, 1632, BF, True, False), (norm_out, 2040, F32, True, False)],
    [(norm_in, 3496, BF), (norm_in, 2448, F32), (norm_in, 12232, BF), (norm_out, 1632, BF, True, True), (norm_out, 2040, F32, False, True),
     (norm_out, 2040, BF, True, False), (norm_out, 1632, F32, False, False)],
    [(norm_in, 4080, BF), (norm_in, 3064, F32), (norm_in, 12248, BF), (norm_out, 2040, BF, True, True), (norm_out, 2040, F32, True, True),
     (norm_out, 2040, BF, False, False), (norm_out, 2040, F32, False, False)],
    [(norm_in, 4896, BF), (norm_in, 4080, F32), (norm_in, 12256, BF)],
    [(norm_in, 6120, BF), (norm_in, 6120, F32)],
    [(norm_in, 6128, BF), (norm_in, 6128, F32)],
]


@pytest.mark.parametrize("group", range(len(FIRST)))
def test_width_as_the_first_call_of_its_kernel(group):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, __file__, str(group)], capture_output=True, text=True, timeout=120, cwd=root,
                       env={**os.environ, "PYTHONPATH": root})
    assert p.returncode == 0, p.stdout[-2000:] + p.stderr[-2000:]


def test_threads_with_different_widths():
    """One kernel (bf16 rows of 129 to 1024 vectors), rings of 49 KB in two threads and 57 KB in two: 20000 calls each."""
    failed, go = [], threading.Barrier(4)

    def work(d):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                x, w = torch.randn(T, d, device="cuda").bfloat16(), torch.ones(d, device="cuda")
                xn, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
                args = (x.data_ptr(), 0, w.data_ptr(), T, d, EPS, xn.data_ptr(), rstd.data_ptr(), stream.cuda_stream)
                call = N.lib().moe_block_norm_in
                go.wait(60)
                bad = sum(call(*args) != N.MOE_OK for _ in range(20000))
                stream.synchronize()
                ref = x.double() * norm64(x.double())
                near(xn, ref, ref.abs(), d)
                if bad:
                    failed.append((d, bad))
        except Exception as e:  # noqa: BLE001 - reported by the test
            failed.append((d, repr(e)))

    threads = [threading.Thread(target=work, args=(d,)) for d in (4096, 7168, 4096, 7168)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not failed and not any(t.is_alive() for t in threads), failed


if __name__ == "__main__":
    wrong = []
    for fn, *args in FIRST[int(sys.argv[1])]:
        try:
            fn(*args)
        except Exception as e:  # noqa: BLE001 - the others are tried as well
            wrong.append(f"{fn.__name__} {args}: {e!r}")
    print("\n".join(wrong))
    sys.exit(1 if wrong else 0)
