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


# ------------------------------------------------------------------------ the operators of other files

def i32(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def space(need):
    return torch.empty(max(16, need), dtype=torch.uint8, device="cuda")


def norm(rows, graphs, form, channels=64, groups=4):
    x, gamma, beta = rand(rows * graphs, channels), rand(channels), rand(channels)
    offsets = i32(*range(0, rows * graphs + 1, rows))
    y, mean, rstd = torch.empty_like(x), torch.empty(graphs, groups, device="cuda"), torch.empty(graphs, groups, device="cuda")
    f, b = uvu.group_norm_workspace_bytes(x, graphs, groups, rows)
    if form == "fwd":
        ws = space(f)
        return lambda s: uvu.group_norm_fwd(x, gamma, beta, offsets, groups, y, mean, rstd, max_rows=rows, workspace=ws, stream=s), [y, mean, rstd]
    uvu.group_norm_fwd(x, gamma, beta, offsets, groups, y, mean, rstd, max_rows=rows)
    dy, dx, dgamma, dbeta, ws = rand(*x.shape), torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta), space(b)
    return (lambda s: uvu.group_norm_bwd(dy, x, gamma, beta, offsets, groups, mean, rstd, dx, dgamma, dbeta, max_rows=rows, workspace=ws, stream=s),
            [dx, dgamma, dbeta])


@pytest.mark.parametrize("form, rows", [("fwd", (390, 410)), ("bwd", (200, 260))], ids=["fwd", "bwd"])  # 50 to 70 KB a block
def test_group_norm(monkeypatch, looped, form, rows):
    both(monkeypatch, looped, f"uvu_group_norm_{form}", [norm(n, 100, form) for n in rows])


@pytest.mark.parametrize("heads", [2, 24], ids=["one", "two"])  # row tiles of a block
def test_attention(monkeypatch, looped, heads):
    def one(mask):
        rows, states = 1000, 1000
        at = uvu.Attention(heads, heads, 64, i32(0, rows), i32(0, states))
        q, k, v = (rand(n, heads, 64, dtype=torch.bfloat16) for n in (rows, states, states))
        keep = (torch.arange(states, device="cuda") % 3 > 0).to(torch.uint8) if mask else None
        out, lse = torch.empty_like(q), torch.empty(rows, heads, device="cuda")
        ws = space(at.workspace_bytes(q, k)[0])
        return lambda s: at.fwd(q, k, v, out, lse, keep=keep, workspace=ws, stream=s), [out, lse]

    both(monkeypatch, looped, "uvu_attn_fwd", [one(False), one(True)])


def test_radial_network(monkeypatch, looped):
    def one(widths):
        plan = uvu.Plan("16x0e+16x1o", "1x0e+1x1o", 1)
        weights = rand(sum(a * b for a, b in zip(widths, widths[1:]))) * 0.2
        r, h = torch.rand(500, device="cuda") * 4 + 0.5, torch.empty(500, widths[-1], device="cuda")
        return lambda s: plan.radial_hidden(r, 5.0, 5, widths, weights, h, stream=s), [h, plan]

    made = [one([8, 32, 32]), one([8, 64, 64, 64])]
    both(monkeypatch, looped, "uvu_radial_hidden", [(call, out[:1]) for call, out in made])


@pytest.mark.parametrize("dtype", ["float32", "float64"])
def test_mixing(monkeypatch, looped, dtype):
    def one(irreps, sh, lmax, u, w, nodes=20):
        plan = uvu.Plan(irreps, sh, lmax, dtype)
        t = torch.float32 if dtype == "float32" else torch.float64
        inp, m = rand(nodes, u, plan.info.dim_out, dtype=t), rand(plan.info.n_paths, u, w, dtype=t)
        out, ws = torch.empty(nodes, w, plan.info.dim_out, dtype=t, device="cuda"), space(plan.mix_workspace_bytes(nodes, w)[0])
        return lambda s: plan.mix_fwd(nodes, w, inp, m, out, workspace=ws, stream=s), [out, plan]

    made = [one("32x0e+32x1o", "1x0e+1x1o", 1, 32, 32), one("64x0e+64x1o+64x2e", "1x0e+1x1o+1x2e+1x3o", 3, 64, 512)]
    both(monkeypatch, looped, "uvu_mix_fwd", [(call, out[:1]) for call, out in made])
