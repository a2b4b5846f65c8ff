"""Calls of one operator from two host threads at once, on streams and with workspaces of their own: each gives what it gives alone.  The
two calls take the same kernel with different needs of shared memory.  The threads call the C entry in a loop of compiled code, where no
lock of the interpreter comes between (a limit that each call set to its own need made 3% of such calls fail, 1 of 20,000 from Python)."""
import ctypes
import subprocess
import threading

import pytest
import torch

from clebsch_gordan_tensor_receiver_gb300 import uvu

pytestmark = pytest.mark.gpu

C_TYPE = {ctypes.c_int: "int", ctypes.c_int64: "long long", ctypes.c_uint64: "unsigned long long", ctypes.c_double: "double",
          ctypes.c_size_t: "size_t"}


@pytest.fixture(scope="module")
def looped(tmp_path_factory):
    """looped(entry): a function of a count and the entry's arguments, which calls it so often and returns how often it failed."""
    made, folder = {}, tmp_path_factory.mktemp("threads")

    def of(entry):
        if entry not in made:
            types = getattr(uvu.lib, entry).argtypes
            names = [C_TYPE.get(t, "void*") for t in types]
            head = ", ".join(f"{t} a{i}" for i, t in enumerate(names))
            (folder / f"{entry}.c").write_text(
                f"#include <stddef.h>\nint loop(int (*f)({', '.join(names)}), int n, {head}) {{\n  int bad = 0;\n"
                f"  for (int i = 0; i < n; ++i) bad += f({', '.join(f'a{i}' for i in range(len(names)))}) != 0;\n  return bad;\n}}\n")
            out = folder / f"{entry}.so"
            subprocess.run(["gcc", "-O1", "-shared", "-fPIC", str(folder / f"{entry}.c"), "-o", str(out)], check=True)
            loop = ctypes.CDLL(str(out)).loop
            loop.argtypes = [ctypes.c_void_p, ctypes.c_int, *types]
            f = ctypes.cast(getattr(uvu.lib, entry), ctypes.c_void_p)
            made[entry] = lambda n, *args: loop(f, n, *args)
        return made[entry]

    return of


def arguments(monkeypatch, entry, call):
    """What `call` hands to the entry, which it also runs."""
    got, real = [], getattr(uvu, entry)
    with monkeypatch.context() as m:
        m.setattr(uvu, entry, lambda *args: (got.append(args), real(*args)))
        call()
    assert len(got) == 1
    return got[0]


def both(monkeypatch, looped, entry, made, times=3000):
    """made: for each thread a function of a stream that calls the entry once, and the tensors that it writes."""
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    args = [arguments(monkeypatch, entry, lambda c=call, s=stream: c(s)) for (call, _), stream in zip(made, streams)]
    torch.cuda.synchronize()
    want = [[t.clone() for t in out] for _, out in made]
    loop, failed, begin = looped(entry), [None] * len(made), threading.Barrier(len(made))

    def work(i):
        begin.wait()
        failed[i] = loop(times, *args[i])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(made))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * len(made), f"failed calls of {times}: {failed}"
    assert all(torch.equal(a, b) for (_, out), kept in zip(made, want) for a, b in zip(out, kept))


def rand(*shape, dtype=torch.float32):
    return torch.randn(*shape, device="cuda").to(dtype)


def rms(rows, width, dtype, form):
    x, residual, gamma = rand(rows, width, dtype=dtype), rand(rows, width, dtype=dtype), torch.ones(width, device="cuda")
    y, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
    if form == "fwd":
        return lambda s: uvu.rms_norm_fwd(x, gamma, y, rstd, residual=residual, h=h, stream=s), [y, h, rstd]
    if form == "quant":
        q, scales = torch.empty(rows, width, dtype=torch.uint8, device="cuda"), torch.empty(rows, -(-width // 40), device="cuda")
        return lambda s: uvu.rms_norm_quant(x, gamma, q, scales, group=40, residual=residual, h=h, stream=s), [q, scales, h]
    uvu.rms_norm_fwd(x, gamma, y, rstd)
    dx, dgamma = torch.empty_like(x), torch.empty_like(gamma)
    ws = torch.empty(uvu.rms_norm_workspace_bytes(x), dtype=torch.uint8, device="cuda")
    return lambda s: uvu.rms_norm_bwd(residual, x, gamma, rstd, dx, dgamma, workspace=ws, stream=s), [dx, dgamma]


@pytest.mark.parametrize("form", ["fwd", "quant", "bwd"])
@pytest.mark.parametrize("shapes, dtype", [(((4000, 512), (5000, 512)), torch.float32), (((40, 5000), (60, 7000)), torch.float32),
                                           (((4000, 512), (9000, 512)), torch.bfloat16)], ids=["rows", "width", "bf16"])
def test_rms_norm(monkeypatch, looped, shapes, dtype, form):
    both(monkeypatch, looped, f"uvu_rms_norm_{form}", [rms(*s, dtype, form) for s in shapes])
