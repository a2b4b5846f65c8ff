"""Measured cases of the operators around a layer's convolution in training: the nodes' first features from a table of
species, RMS norm with the residual's addition (and 8-bit output for serving), and updates of weight matrices made
orthogonal by Newton-Schulz products.

Each operator has a plain form (elementary torch operations in 32 bits, rounded once at the end) and a call of this
repository's kernels; `own` chooses between them.  The sizes of a case follow from the case alone, its values from the seed.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
MUON = (3.4445, -4.7750, 2.0315)  # the optimiser's coefficients, five steps
STEPS = 5
EPS = 1e-5
TOP = 448.0  # the largest e4m3 value


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the first features 128x0e+128x1o of one molecule: latency
        dict(name="embed-molecule", op="embed", type="f32", train=False, tokens=61, rows=10, channels=128, inner=4, pad=False),
        # the same of a batch of 50,000 atoms of 89 species, padded, in training: every species sums hundreds of atoms
        dict(name="embed-atoms", op="embed", type="f32", train=True, tokens=50000, rows=89, channels=128, inner=4, pad=True),
        # scalar features of a large training batch: memory, and long sums of a few rows
        dict(name="embed-batch", op="embed", type="f16", train=True, tokens=300007, rows=119, channels=512, inner=1, pad=False),
        # the context states' tokens from a large vocabulary: most rows of the gradient have no token or one
        dict(name="embed-vocab", op="embed", type="bf16", train=True, tokens=16384, rows=65536, channels=1024, inner=1, pad=True),
        # the smallest graph of the framework's own workloads, 100 nodes of 16x0e+16x1o: latency
        dict(name="rms-tiny", op="rms", type="f32", train=False, rows=100, channels=16, inner=4, residual=True, group=-1),
        # 5000 nodes of 128x0e+128x1o in training, one norm over the components of all channels
        dict(name="rms-train-f32", op="rms", type="f32", train=True, rows=5000, channels=128, inner=4, residual=True, group=-1),
        # scalar features of a large training batch in 16 bits: memory
        dict(name="rms-train-bf16", op="rms", type="bf16", train=True, rows=262144, channels=512, inner=1, residual=True, group=-1),
        # context states on their way to an 8-bit product, one scale for 128 values: memory
        dict(name="rms-8bit", op="rms", type="bf16", train=False, rows=65537, channels=1024, inner=1, residual=True, group=128),
        # the 13 mixing matrices of a convolution of 128 channels: latency of a chain of small products
        dict(name="ortho-mixing", op="ortho", type="f32", matrices=13, rows=128, cols=128),
        # the radial network's last layer, 64 x 13 paths of 128 channels
        dict(name="ortho-radial", op="ortho", type="f32", matrices=1, rows=64, cols=1664),
        # 25 mixing matrices of 256 channels, in 16 bits
        dict(name="ortho-wide", op="ortho", type="bf16", matrices=25, rows=256, cols=256),
        # two dense layers of the encoder: arithmetic
        dict(name="ortho-large", op="ortho", type="f32", matrices=2, rows=4096, cols=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "rms", "ortho"])
    kind = rng.choice(["f32", "bf16", "f16"])
    train = rng.random() < 0.6
    if op == "embed":
        inner = rng.choice([1, 1, 4, 9])
        tokens, channels = _log(rng, 1, 300007), _log(rng, 8, 1024)
        rows = _log(rng, 2, 65536)
        while float(tokens) * channels * inner > 1.5e8:
            tokens = max(1, tokens * 3 // 4)
        return dict(op=op, type=kind, train=train, tokens=tokens, rows=rows, channels=channels, inner=inner, pad=rng.random() < 0.5)
    if op == "rms":
        inner = rng.choice([1, 1, 4, 9])
        channels, rows = _log(rng, 8, 1024), _log(rng, 1, 262144)
        while float(rows) * channels * inner > 1.3e8:
            rows = max(1, rows * 3 // 4)
        group = -1 if train or rng.random() < 0.4 else rng.choice([0, 32, 64, 128])
        return dict(op=op, type=kind, train=train, rows=rows, channels=channels, inner=inner, residual=rng.random() < 0.7, group=group)
    rows, cols, matrices = _log(rng, 8, 4096), _log(rng, 8, 4096), _log(rng, 1, 32)
    while matrices * _ortho_flops(rows, cols) > 4e11:
        rows, cols, matrices = max(8, rows * 3 // 4), max(8, cols * 3 // 4), max(1, matrices * 3 // 4)
    return dict(op=op, type=kind, matrices=matrices, rows=rows, cols=cols)


def _ortho_flops(rows, cols):
    """Of one matrix: X X^T and its square (symmetric: half of each), and the product with X."""
    m, n = min(rows, cols), max(rows, cols)
    return STEPS * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n)


def work(case):
    c, s = case, SIZE[case["type"]]
    if c["op"] == "embed":
        values = c["tokens"] * c["channels"]
        size = 4 * c["tokens"] + min(c["tokens"], c["rows"]) * c["channels"] * s + values * c["inner"] * s
        if c["train"]:  # the gradient reads one component of each channel
            size += 4 * c["tokens"] + values * s + c["rows"] * c["channels"] * s
        return {"bytes": size, "flops": values * (2 if c["train"] else 1)}
    if c["op"] == "rms":
        n = c["rows"] * c["channels"] * c["inner"]
        if c["train"]:  # x, residual, h, y; then dy, dh, h, dx
            return {"bytes": n * s * ((4 if c["residual"] else 2) + 4), "flops": n * 16}
        out = n * s if c["group"] < 0 else n + 4 * c["rows"] * _groups(c)
        return {"bytes": n * s * (3 if c["residual"] else 1) + out, "flops": n * (6 if c["group"] < 0 else 9)}
    return {"bytes": 2 * c["matrices"] * c["rows"] * c["cols"] * s, "flops": c["matrices"] * _ortho_flops(c["rows"], c["cols"])}


def _groups(c):
    """Scales of a row in the 8-bit output: `group` values share one, all of the row where it is 0."""
    n = c["channels"] * c["inner"]
    return -(-n // c["group"]) if c["group"] else 1


# ------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    c, kind = case, TYPES[case["type"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6007 + 29)

    def normal(*shape, dtype=kind):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    st = {"case": case}
    if c["op"] == "embed":
        # a few species or tokens are much more frequent than the others; padding is -1
        u = torch.rand(c["tokens"], generator=g, device="cuda", dtype=torch.float64)
        index = (u.pow(3) * c["rows"]).long().clamp(max=c["rows"] - 1).to(torch.int32)
        if c["pad"]:
            index[torch.rand(c["tokens"], generator=g, device="cuda") < 0.05] = -1
        st.update(index=index, table=normal(c["rows"], c["channels"]), scale=math.sqrt(c["channels"]),
                  out=torch.empty(c["tokens"], c["channels"], c["inner"], dtype=kind, device="cuda"))
        if c["train"]:
            st.update(d_out=normal(c["tokens"], c["channels"], c["inner"]), d_table=torch.empty_like(st["table"]))
    elif c["op"] == "rms":
        shape = (c["rows"], c["channels"], c["inner"])
        x = normal(*shape)
        st.update(x=x, residual=2 * normal(*shape) if c["residual"] else None, h=torch.empty_like(x) if c["residual"] else None,
                  gamma=1 + 0.2 * normal(c["channels"], dtype=torch.float32))
        if c["group"] >= 0:
            st.update(y=torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda"),
                      scales=torch.empty(c["rows"], _groups(c), dtype=torch.float32, device="cuda"))
        else:
            st.update(y=torch.empty_like(x), rstd=torch.empty(c["rows"], dtype=torch.float32, device="cuda"))
        if c["train"]:
            st.update(d_y=normal(*shape), d_h=normal(*shape), d_x=torch.empty_like(x), d_gamma=torch.empty_like(st["gamma"]))
    else:
        # a gradient: a few strong directions above noise, of small size
        few = max(1, min(c["rows"], c["cols"]) // 8)
        a, b = (normal(c["matrices"], n, few, dtype=torch.float32) for n in (c["rows"], c["cols"]))
        noise = normal(c["matrices"], c["rows"], c["cols"], dtype=torch.float32)
        st["g"] = ((torch.matmul(a, b.transpose(1, 2)) / math.sqrt(few) + 0.3 * noise) * 1e-3).to(kind)
        st["out"] = torch.empty_like(st["g"])
    return st


# ------------------------------------------------------------------------------------------ passes

def run(state):
    op = state["case"]["op"]
    if own:
        return {"embed": _own_embed, "rms": _own_rms, "ortho": _own_ortho}[op](state)
    return {"embed": _plain_embed, "rms": _plain_rms, "ortho": _plain_ortho}[op](state)


def _kept_workspace(st, need):
    """The workspace that a program keeps from step to step."""
    if "workspace" not in st:
        st["workspace"] = torch.empty(max(16, need()), dtype=torch.uint8, device="cuda")
    return st["workspace"]


def _own_embed(st):
    from clebsch_gordan_tensor_receiver_gb300 import uvu
    uvu.embed_fwd(st["index"], st["table"], st["out"], scale=st["scale"])
    r = {"out": st["out"]}
    if st["case"]["train"]:
        ws = _kept_workspace(st, lambda: uvu.embed_workspace_bytes(st["d_out"], st["d_table"]))
        uvu.embed_bwd(st["index"], st["d_out"], st["d_table"], scale=st["scale"], workspace=ws)
        r["d_table"] = st["d_table"]
    return r


def _own_rms(st):
    from clebsch_gordan_tensor_receiver_gb300 import uvu
    c = st["case"]
    r = {} if st["h"] is None else {"h": st["h"]}
    if c["group"] >= 0:
        uvu.rms_norm_quant(st["x"], st["gamma"], st["y"], st["scales"], group=c["group"], residual=st["residual"], h=st["h"], eps=EPS)
        return r | {"y": st["y"], "scales": st["scales"]}
    uvu.rms_norm_fwd(st["x"], st["gamma"], st["y"], st["rstd"], residual=st["residual"], h=st["h"], eps=EPS)
    r.update(y=st["y"], rstd=st["rstd"])
    if c["train"]:
        h = st["x"] if st["h"] is None else st["h"]
        ws = _kept_workspace(st, lambda: uvu.rms_norm_workspace_bytes(h))
        uvu.rms_norm_bwd(st["d_y"], h, st["gamma"], st["rstd"], st["d_x"], st["d_gamma"], dh=st["d_h"], workspace=ws)
        r.update(d_x=st["d_x"], d_gamma=st["d_gamma"])
    return r


def _own_ortho(st):
    from clebsch_gordan_tensor_receiver_gb300 import uvu
    ws = _kept_workspace(st, lambda: uvu.orthogonalize_workspace_bytes(st["g"]))
    uvu.orthogonalize(st["g"], st["out"], workspace=ws)
    return {"out": st["out"]}


def _plain_embed(st):
    c = st["case"]
    kind = TYPES[c["type"]]
    index = st["index"].long()
    own_row = (index >= 0) & (index < c["rows"])
    row = torch.where(own_row, index, torch.zeros_like(index))
    picked = torch.where(own_row[:, None], st["table"].float()[row] * st["scale"], torch.zeros((), device=row.device))
    out = torch.zeros(c["tokens"], c["channels"], c["inner"], dtype=kind, device=row.device)
    out[:, :, 0] = picked.to(kind)
    r = {"out": out}
    if c["train"]:  # sums of many values: in 64 bits
        d = torch.where(own_row[:, None], st["d_out"][:, :, 0].double(), torch.zeros((), dtype=torch.float64, device=row.device))
        total = torch.zeros(c["rows"], c["channels"], dtype=torch.float64, device=row.device).index_add(0, row, d)
        r["d_table"] = (total * st["scale"]).to(kind)
    return r


def _plain_rms(st):
    c = st["case"]
    kind = TYPES[c["type"]]
    gamma = st["gamma"][:, None]
    if st["residual"] is None:
        r, stored = {}, st["x"]
    else:
        stored = (st["x"].float() + st["residual"].float()).to(kind)  # the stream as it is stored is what the norm is of
        r = {"h": stored}
    h = stored.float()
    rstd = 1.0 / torch.sqrt((h * h).mean((1, 2), keepdim=True) + EPS)
    unit = h * rstd
    y = unit * gamma
    if c["group"] >= 0:
        n, each = c["channels"] * c["inner"], _groups(c)
        wide = torch.nn.functional.pad(y.reshape(c["rows"], n), (0, (each * c["group"] if c["group"] else n) - n))
        wide = wide.view(c["rows"], each, -1)
        scales = wide.abs().amax(2) / TOP
        q = torch.where(scales[:, :, None] > 0, wide / scales[:, :, None], torch.zeros_like(wide)).clamp(-TOP, TOP)
        return r | {"y": q.view(c["rows"], -1)[:, :n].reshape(y.shape).to(torch.float8_e4m3fn), "scales": scales}
    r.update(y=y.to(kind), rstd=rstd.view(-1))
    if c["train"]:
        dy = st["d_y"].float()
        t = dy * gamma
        d_x = rstd * (t - unit * (t * unit).mean((1, 2), keepdim=True)) + st["d_h"].float()
        r.update(d_x=d_x.to(kind), d_gamma=(dy * unit).double().sum((0, 2)).float())
    return r


def _plain_ortho(st):
    a, b, c = MUON
    g = st["g"].float()
    turned = g.shape[1] > g.shape[2]
    x = g.transpose(1, 2) if turned else g
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + 1e-7)
    for _ in range(STEPS):  # each step takes the last one's result
        p = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * p + c * torch.matmul(p, p), x)
    return {"out": (x.transpose(1, 2) if turned else x).to(st["g"].dtype).contiguous()}


# ------------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"embed": _exact_embed, "rms": _exact_rms, "ortho": _exact_ortho}[case["op"]](st, case)


def _exact_embed(st, c):
    # by the sorted tokens: runs of one row between two cuts of a running sum would lose bits, so a product with 0 and 1
    keep = (st["index"] >= 0).nonzero()[:, 0]
    row = st["index"][keep].long()
    out = torch.zeros(c["tokens"], c["channels"], c["inner"], dtype=torch.float64, device="cuda")
    out[keep, :, 0] = st["table"].double()[row] * st["scale"]
    r = {"out": out}
    if c["train"]:
        ones = torch.sparse_coo_tensor(torch.stack((row, keep)), torch.ones(len(keep), dtype=torch.float64, device="cuda"),
                                       (c["rows"], c["tokens"]))
        r["d_table"] = torch.sparse.mm(ones, st["d_out"][:, :, 0].double().contiguous()) * st["scale"]
    return r


def _exact_rms(st, c):
    x = st["x"].double()
    r = {}
    if st["residual"] is not None:
        r["h"] = x + st["residual"].double()
        x = r["h"].to(TYPES[c["type"]]).double()  # the operator's definition: the norm of the stream as stored
    n = c["channels"] * c["inner"]
    flat = x.view(c["rows"], n)
    gamma = st["gamma"].double().repeat_interleave(c["inner"])
    rstd = (torch.linalg.vector_norm(flat, dim=1).square() / n + EPS) ** -0.5
    y = flat * rstd[:, None] * gamma
    if c["group"] >= 0:
        size = c["group"] or n
        which = torch.arange(n, device="cuda") // size
        top = torch.zeros(c["rows"], _groups(c), dtype=torch.float64, device="cuda")
        top.scatter_reduce_(1, which.expand(c["rows"], n), y.abs(), "amax")
        scales = top / TOP
        each = scales[:, which]
        return r | {"y": torch.where(each > 0, y / each.clamp(min=1e-300), 0.0).view(x.shape), "scales": scales}
    r.update(y=y.view(x.shape), rstd=rstd)
    if c["train"]:
        dy = st["d_y"].double().view(c["rows"], n)
        t = dy * gamma
        inner = torch.einsum("ij,ij->i", t, flat) / n
        d_x = rstd[:, None] * t - flat * (rstd ** 3 * inner)[:, None] + st["d_h"].double().view(c["rows"], n)
        d_gamma = torch.einsum("ij,ij,i->j", dy, flat, rstd).view(c["channels"], c["inner"]).sum(1)
        r.update(d_x=d_x.view(x.shape), d_gamma=d_gamma)
    return r


def _exact_ortho(st, c):
    if c["matrices"] * _ortho_flops(c["rows"], c["cols"]) > 2e12:
        return None
    out = []
    for g in st["g"].double():
        tall = g.shape[0] >= g.shape[1]
        x = (g if tall else g.T) / (torch.linalg.matrix_norm(g) + 1e-7)
        for _ in range(STEPS):  # on the side of the small Gram matrix, by Horner's rule
            p = x.T @ x
            q = MUON[2] * p
            q.diagonal().add_(MUON[1])
            q = q @ p
            q.diagonal().add_(MUON[0])
            x = x @ q
        out.append(x if tall else x.T)
    return {"out": torch.stack(out)}
