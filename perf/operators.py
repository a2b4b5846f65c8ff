"""Measured cases of the node-update operators that follow a convolution: group norm with an activation, attention of a
graph's nodes to another set of states, and dropout with a residual.

Each operator has a plain form (elementary torch operations in 32 bits, rounded once at the end) and a call of this
repository's kernels; `own` chooses between them.  A batch of graphs is packed: the rows of its graphs lie back to back and
`offsets` [B+1] says where each begins.  The lengths of a case follow from the case alone, its values from the seed.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one new token for each of 16 sequences over short encodings, a few kept back by the mask: latency
        dict(name="attend-token", op="attend", type="bf16", train=False, graphs=16, q=1, k=512, heads=8, kv_heads=2, dim=64,
             ragged=True, mask=True),
        # one new token each over long encodings: K and V are read once, nothing else is large
        dict(name="attend-token-long", op="attend", type="f16", train=False, graphs=8, q=1, k=16384, heads=32, kv_heads=8,
             dim=128, ragged=True, mask=False),
        # small molecules, 128 channels in 8 heads, each attending to the atoms around its own site; one has none
        dict(name="attend-molecules", op="attend", type="f32", train=False, graphs=64, q=61, k=333, heads=8, kv_heads=8, dim=16,
             ragged=True, mask=True),
        # four large structures against long encodings: arithmetic
        dict(name="attend-large", op="attend", type="bf16", train=False, graphs=4, q=4096, k=8192, heads=16, kv_heads=16,
             dim=128, ragged=False, mask=False),
        # a training batch in 32 bits, 128 channels in 4 heads
        dict(name="attend-train-f32", op="attend", type="f32", train=True, graphs=32, q=200, k=500, heads=4, kv_heads=4, dim=32,
             ragged=True, mask=True),
        # a training batch in 16 bits with shared key and value heads
        dict(name="attend-train-bf16", op="attend", type="bf16", train=True, graphs=8, q=4096, k=4096, heads=16, kv_heads=4,
             dim=64, ragged=True, mask=True),
        # the smallest graph of the framework's own workloads: 100 nodes, 16 channels: latency
        dict(name="norm-tiny", op="norm", type="f32", train=False, graphs=1, rows=100, channels=16, groups=4, act="silu",
             ragged=False),
        # the scalar channels of a batch of 64 molecules, 5000 atoms in all, in training
        dict(name="norm-train-f32", op="norm", type="f32", train=True, graphs=64, rows=127, channels=128, groups=8, act="silu",
             ragged=True),
        # a large training batch in 16 bits: memory
        dict(name="norm-train-bf16", op="norm", type="bf16", train=True, graphs=256, rows=1531, channels=512, groups=32,
             act="silu", ragged=True),
        # one structure of 200,001 atoms: the sums of a group go over the whole card
        dict(name="norm-one-graph", op="norm", type="f16", train=False, graphs=1, rows=200001, channels=256, groups=16,
             act="none", ragged=False),
        # equivariant features 128x0e+128x1o of 1000 nodes: one draw for the four components of a channel pair, with a residual
        dict(name="dropout-irreps", op="dropout", type="f32", train=False, rows=1000, channels=128, inner=4, p=0.1, residual=True),
        # scalar features of a large training batch: memory
        dict(name="dropout-train", op="dropout", type="bf16", train=True, rows=262144, channels=512, inner=1, p=0.1,
             residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "norm", "dropout"])
    kind = rng.choice(["f32", "bf16", "f16"])
    train = rng.random() < 0.5
    if op == "attend":
        token = not train and rng.random() < 0.4
        dim = rng.choice([16, 24, 32, 40, 64, 80, 96, 128])
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 1, 2, 4, 7])
        graphs = _log(rng, 1, 64)
        q, k = 1 if token else _log(rng, 2, 4096), _log(rng, 1, 16384)
        most = 2e11 if kind == "f32" else 6e11
        while 4.0 * graphs * q * k * heads * dim * (3.5 if train else 1) > most or graphs * k * kv * dim > 2e8:
            q, k, graphs = max(1, q * 3 // 4), max(1, k * 3 // 4), max(1, graphs * 3 // 4)
        return dict(op=op, type=kind, train=train, graphs=graphs, q=q, k=k, heads=heads, kv_heads=kv, dim=dim,
                    ragged=rng.random() < 0.7, mask=rng.random() < 0.5)
    if op == "norm":
        per = rng.choice([1, 2, 4, 8, 16, 32, 40])
        groups = rng.choice([1, 2, 4, 8, 16, 32])
        graphs = _log(rng, 1, 256)
        rows = _log(rng, 1, 200000)
        while float(graphs) * rows * per * groups > 1.3e8:
            rows, graphs = max(1, rows * 3 // 4), max(1, graphs * 3 // 4)
        return dict(op=op, type=kind, train=train, graphs=graphs, rows=rows, channels=per * groups, groups=groups,
                    act=rng.choice(["silu", "silu", "none"]), ragged=rng.random() < 0.7)
    inner = rng.choice([1, 1, 4, 9, 16])
    rows, channels = _log(rng, 1, 262144), _log(rng, 8, 512)
    while float(rows) * channels * inner > 1.3e8:
        rows = max(1, rows * 3 // 4)
    return dict(op=op, type=kind, train=train, rows=rows, channels=channels, inner=inner,
                p=rng.choice([0.05, 0.1, 0.25, 0.5]), residual=rng.random() < 0.7)


def _lengths(graphs, most, ragged, empty=False):
    """Lengths of the graphs of a batch: the first the longest, the others spread evenly over [1, most]; with `empty` the last
    of several has none."""
    n = [most] * graphs
    if ragged:
        n = [most] + [1 + int((most - 1) * ((b * 0.6180339887498949 + 0.35) % 1.0)) for b in range(1, graphs)]
        if empty and graphs > 2:
            n[-1] = 0
    return n


def _offsets(lengths):
    return np.concatenate([[0], np.cumsum(np.asarray(lengths, dtype=np.int64))]).astype(np.int32)


def _attend_lengths(c):
    # the two lengths of a graph are spread differently, so that short ones meet long ones
    return _lengths(c["graphs"], c["q"], c["ragged"]), _lengths(c["graphs"], c["k"], c["ragged"], True)[::-1]


def work(case):
    c, s = case, SIZE[case["type"]]
    if c["op"] == "attend":
        nq, nk = _attend_lengths(c)
        pairs, tq, tk = sum(a * b for a, b in zip(nq, nk)), sum(nq), sum(nk)
        hd, kd = c["heads"] * c["dim"], c["kv_heads"] * c["dim"]
        size = 2 * tq * hd * s + 2 * tk * kd * s + 4 * tq * c["heads"] + (tk if c["mask"] else 0)
        flops = 4 * pairs * hd
        if c["train"]:  # d_out read, three gradients written
            size += 2 * tq * hd * s + 2 * tk * kd * s
            flops += 10 * pairs * hd
        return {"bytes": size, "flops": flops}
    if c["op"] == "norm":
        n = sum(_lengths(c["graphs"], c["rows"], c["ragged"])) * c["channels"]
        return {"bytes": n * s * (5 if c["train"] else 2), "flops": n * (30 if c["train"] else 10)}
    n = c["rows"] * c["channels"] * c["inner"]
    return {"bytes": n * s * (2 + (1 if c["residual"] else 0) + (2 if c["train"] else 0)), "flops": n * (4 if c["train"] else 2)}


# ------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    c, kind = case, TYPES[case["type"]]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)

    def normal(*shape, dtype=kind):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    def device(a):
        return torch.from_numpy(a).cuda()

    st = {"case": case}
    if c["op"] == "attend":
        nq, nk = _attend_lengths(c)
        tq, tk = sum(nq), sum(nk)
        st.update(q=normal(tq, c["heads"], c["dim"]), k=normal(tk, c["kv_heads"], c["dim"]),
                  v=normal(tk, c["kv_heads"], c["dim"]) + 0.25, q_offsets=device(_offsets(nq)), k_offsets=device(_offsets(nk)),
                  keep=None)
        st["v"] = st["v"].to(kind)
        if c["mask"]:  # padding of the encodings: a tenth of the states says nothing
            st["keep"] = (torch.rand(tk, generator=g, device="cuda") < 0.9).to(torch.uint8)
        if c["train"]:
            st["d_out"] = normal(tq, c["heads"], c["dim"])
    elif c["op"] == "norm":
        n = _lengths(c["graphs"], c["rows"], c["ragged"])
        st.update(x=(normal(sum(n), c["channels"], dtype=torch.float32) * 1.7 + 0.3).to(kind), offsets=device(_offsets(n)),
                  gamma=1 + 0.2 * normal(c["channels"], dtype=torch.float32), beta=0.2 * normal(c["channels"], dtype=torch.float32))
        if c["train"]:
            st["d_y"] = normal(sum(n), c["channels"])
    else:
        shape = (c["rows"], c["channels"], c["inner"])
        st.update(x=normal(*shape), residual=normal(*shape) if c["residual"] else None, seed=int(seed) * 1000003 + 12345,
                  offset=int(seed) % 1000)
        if c["train"]:
            st["d_y"] = normal(*shape)
    _output_buffers(st)
    return st


def _output_buffers(st):
    """The output tensors that a program keeps from step to step."""
    c = st["case"]
    empty = torch.empty_like
    if c["op"] == "attend":
        st.update(out=empty(st["q"]), lse=torch.empty(st["q"].shape[0], c["heads"], dtype=torch.float32, device="cuda"))
        if c["train"]:
            st.update(d_q=empty(st["q"]), d_k=empty(st["k"]), d_v=empty(st["v"]))
    elif c["op"] == "norm":
        st.update(y=empty(st["x"]), mean=torch.empty(c["graphs"], c["groups"], dtype=torch.float32, device="cuda"),
                  rstd=torch.empty(c["graphs"], c["groups"], dtype=torch.float32, device="cuda"))
        if c["train"]:
            st.update(d_x=empty(st["x"]), d_gamma=empty(st["gamma"]), d_beta=empty(st["beta"]))
    else:
        st["y"] = empty(st["x"])
        if c["train"]:
            st["d_x"] = empty(st["x"])


# ------------------------------------------------------------------------------------------ passes

def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _own_attend, "norm": _own_norm, "dropout": _own_dropout}[op](state)
    return {"attend": _plain_attend, "norm": _plain_norm, "dropout": _plain_dropout}[op](state)


def _workspace(need):
    return torch.empty(max(16, *need), dtype=torch.uint8, device="cuda")


def _own_attend(st):
    from clebsch_gordan_tensor_receiver_gb300 import uvu
    c = st["case"]
    if "attention" not in st:  # the descriptor and the workspace that a program keeps
        st["attention"] = uvu.Attention(c["heads"], c["kv_heads"], c["dim"], st["q_offsets"], st["k_offsets"], c["q"], c["k"])
        need = st["attention"].workspace_bytes(st["q"], st["k"])
        st["workspace"] = _workspace(need if c["train"] else need[:1])
    at = st["attention"]
    at.fwd(st["q"], st["k"], st["v"], st["out"], st["lse"], keep=st["keep"], workspace=st["workspace"])
    r = {"out": st["out"], "lse": st["lse"]}
    if c["train"]:
        at.bwd(st["q"], st["k"], st["v"], st["out"], st["lse"], st["d_out"], st["d_q"], st["d_k"], st["d_v"], keep=st["keep"],
               workspace=st["workspace"])
        r.update(d_q=st["d_q"], d_k=st["d_k"], d_v=st["d_v"])
    return r


def _own_norm(st):
    from clebsch_gordan_tensor_receiver_gb300 import uvu
    c = st["case"]
    act = uvu.UVU_ACT_SILU if c["act"] == "silu" else uvu.UVU_ACT_NONE
    if "workspace" not in st:
        need = uvu.group_norm_workspace_bytes(st["x"], c["graphs"], c["groups"], c["rows"])
        st["workspace"] = _workspace(need if c["train"] else need[:1])
    uvu.group_norm_fwd(st["x"], st["gamma"], st["beta"], st["offsets"], c["groups"], st["y"], st["mean"], st["rstd"], act=act,
                       max_rows=c["rows"], workspace=st["workspace"])
    r = {"y": st["y"], "mean": st["mean"], "rstd": st["rstd"]}
    if c["train"]:
        uvu.group_norm_bwd(st["d_y"], st["x"], st["gamma"], st["beta"], st["offsets"], c["groups"], st["mean"], st["rstd"],
                           st["d_x"], st["d_gamma"], st["d_beta"], act=act, max_rows=c["rows"], workspace=st["workspace"])
        r.update(d_x=st["d_x"], d_gamma=st["d_gamma"], d_beta=st["d_beta"])
    return r


def _own_dropout(st):
    from clebsch_gordan_tensor_receiver_gb300 import uvu
    c = st["case"]
    uvu.dropout_fwd(st["x"], c["p"], st["seed"], st["y"], offset=st["offset"], inner=c["inner"], residual=st["residual"])
    r = {"y": st["y"]}
    if c["train"]:
        uvu.dropout_bwd(st["d_y"], c["p"], st["seed"], st["d_x"], offset=st["offset"], inner=c["inner"])
        r["d_x"] = st["d_x"]
    return r


def _pad(offsets, most):
    """Row numbers [B, most] of a packed batch, those past a graph's end clamped to a row that exists, and which are its own."""
    first, end = offsets[:-1, None].long(), offsets[1:, None].long()
    rows = first + torch.arange(most, device=offsets.device)
    return torch.minimum(rows, (offsets[-1].long() - 1).clamp(min=0)), rows < end


def _plain_attend(st):
    c = st["case"]
    kind, dim, group = TYPES[c["type"]], c["dim"], c["heads"] // c["kv_heads"]
    qi, qv = _pad(st["q_offsets"], c["q"])
    ki, kv = _pad(st["k_offsets"], c["k"])
    b, mq = qi.shape

    def queries(t):  # [T, H, D] -> [B, Hkv, group * q, D]
        t = t.float()[qi].view(b, mq, c["kv_heads"], group, dim)
        return t.permute(0, 2, 3, 1, 4).reshape(b, c["kv_heads"], group * mq, dim)

    def packed_q(t):  # and back, the rows of each graph alone
        last = t.shape[-1]
        t = t.view(b, c["kv_heads"], group, mq, last).permute(0, 3, 1, 2, 4).reshape(b, mq, c["heads"], last)
        return t[qv]

    scale = 1.0 / math.sqrt(dim)
    q = queries(st["q"])
    k = st["k"].float()[ki].transpose(1, 2)
    v = st["v"].float()[ki].transpose(1, 2)
    kept = kv if st["keep"] is None else kv & (st["keep"][ki] != 0)
    s = torch.matmul(q, k.transpose(-1, -2)) * scale
    s = torch.where(kept[:, None, None, :], s, torch.full((), -math.inf, device=s.device))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(total, -math.inf))
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    out = torch.matmul(p, v)
    r = {"out": packed_q(out).to(kind), "lse": packed_q(lse)[..., 0].contiguous()}
    if c["train"]:
        do = torch.where(qv[:, None, None, :, None], st["d_out"].float()[qi].view(b, mq, c["kv_heads"], group, dim)
                         .permute(0, 2, 3, 1, 4), torch.zeros((), device=q.device)).reshape(b, c["kv_heads"], group * mq, dim)
        dv = torch.matmul(p.transpose(-1, -2), do)
        dp = torch.matmul(do, v.transpose(-1, -2))
        ds = p * (dp - (do * out).sum(-1, keepdim=True)) * scale
        dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(-1, -2), q)
        r.update(d_q=packed_q(dq).to(kind), d_k=dk.transpose(1, 2)[kv].to(kind), d_v=dv.transpose(1, 2)[kv].to(kind))
    return r


def _plain_norm(st):
    c = st["case"]
    kind, per = TYPES[c["type"]], c["channels"] // c["groups"]
    rows, valid = _pad(st["offsets"], c["rows"])
    b, m = rows.shape
    own_row = valid[:, :, None, None]
    zero = torch.zeros((), device=rows.device)
    count = (valid.sum(1).float() * per).clamp(min=1)[:, None, None, None]

    def mean_of(t):
        return t.sum((1, 3), keepdim=True) / count

    x = torch.where(own_row, st["x"].float()[rows].view(b, m, c["groups"], per), zero)
    gamma, beta = st["gamma"].view(c["groups"], per), st["beta"].view(c["groups"], per)
    mean = mean_of(x)
    centred = torch.where(own_row, x - mean, zero)
    rstd = 1.0 / torch.sqrt(mean_of(centred * centred) + 1e-5)
    xh = centred * rstd
    z = xh * gamma + beta
    sig = 1.0 / (1.0 + torch.exp(-z))
    silu = c["act"] == "silu"
    y = z * sig if silu else z
    r = {"y": y.view(b, m, -1)[valid].to(kind), "mean": mean.view(b, -1), "rstd": rstd.view(b, -1)}
    if c["train"]:
        dz = torch.where(own_row, st["d_y"].float()[rows].view(b, m, c["groups"], per), zero)
        if silu:
            dz = dz * sig * (1.0 + z * (1.0 - sig))
        t = dz * gamma
        dx = rstd * (t - mean_of(t) - xh * mean_of(t * xh))
        r.update(d_x=dx.view(b, m, -1)[valid].to(kind), d_gamma=(dz * xh).sum((0, 1)).view(-1), d_beta=dz.sum((0, 1)).view(-1))
    return r


def _philox(seed, first, count, device):
    """Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3") of the counters first .. first + count - 1
    under the key `seed`, as 16-bit draws [count * 8]: the low half of each word before its high half."""
    low = 0xFFFFFFFF
    at = torch.arange(count, device=device, dtype=torch.int64) + first
    a, b, x, y = at & low, (at >> 32) & low, torch.zeros_like(at), torch.zeros_like(at)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        p, q = a * 0xD2511F53, x * 0xCD9E8D57  # modulo 2^64; the shifts below take the high halves
        a, b, x, y = ((q >> 32) & low) ^ b ^ k0, q & low, ((p >> 32) & low) ^ y ^ k1, p & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((a, b, x, y), 1)
    return torch.stack((words & 0xFFFF, words >> 16), 2).view(-1)


def _plain_dropout(st):
    c = st["case"]
    kind, draws = TYPES[c["type"]], c["rows"] * c["channels"]
    limit = int(math.floor(c["p"] * 65536 + 0.5))
    keep = (_philox(st["seed"], st["offset"], -(-draws // 8), "cuda")[:draws] >= limit).view(c["rows"], c["channels"], 1)
    scale = torch.where(keep, torch.full((), 65536.0 / (65536 - limit), device="cuda"), torch.zeros((), device="cuda"))
    y = st["x"].float() * scale
    if st["residual"] is not None:
        y = st["residual"].float() + y
    r = {"y": y.to(kind)}
    if c["train"]:
        r["d_x"] = (st["d_y"].float() * scale).to(kind)
    return r


# ------------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"attend": _exact_attend, "norm": _exact_norm, "dropout": _exact_dropout}[case["op"]](st, case)


def _exact_attend(st, c):
    nq, nk = st["q_offsets"].tolist(), st["k_offsets"].tolist()
    f = torch.float64
    group = c["heads"] // c["kv_heads"]
    tq, tk = nq[-1], nk[-1]
    out = torch.zeros(tq, c["heads"], c["dim"], dtype=f, device="cuda")
    lse = torch.full((tq, c["heads"]), -math.inf, dtype=f, device="cuda")
    dq, dk, dv = torch.zeros_like(out), torch.zeros(tk, c["kv_heads"], c["dim"], dtype=f, device="cuda"), None
    dv = torch.zeros_like(dk)
    for b in range(c["graphs"]):
        i = slice(nq[b], nq[b + 1])
        at = torch.arange(nk[b], nk[b + 1], device="cuda")
        if st["keep"] is not None:
            at = at[st["keep"][at] != 0]
        if not len(at) or nq[b] == nq[b + 1]:
            continue
        for h in range(c["heads"]):
            q, k, v = st["q"][i, h].to(f), st["k"][at, h // group].to(f), st["v"][at, h // group].to(f)
            s = (q @ k.T) / math.sqrt(c["dim"])
            lse[i, h] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            out[i, h] = p @ v
            if c["train"]:
                do = st["d_out"][i, h].to(f)
                dp = do @ v.T
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(c["dim"])
                dq[i, h] = ds @ k
                dk[at, h // group] += ds.T @ q
                dv[at, h // group] += p.T @ do
    r = {"out": out, "lse": lse}
    if c["train"]:
        r.update(d_q=dq, d_k=dk, d_v=dv)
    return r


def _exact_norm(st, c):
    offsets, f = st["offsets"].tolist(), torch.float64
    per = c["channels"] // c["groups"]
    x = st["x"].to(f)
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    mean = torch.zeros(c["graphs"], c["groups"], dtype=f, device="cuda")
    rstd = torch.full_like(mean, 1e-5 ** -0.5)
    gamma, beta = st["gamma"].to(f), st["beta"].to(f)
    dg, db = torch.zeros_like(gamma), torch.zeros_like(beta)
    for b in range(c["graphs"]):
        i = slice(offsets[b], offsets[b + 1])
        if offsets[b] == offsets[b + 1]:
            continue
        var, mu = torch.var_mean(x[i].view(-1, c["groups"], per), dim=(0, 2), unbiased=False)
        mean[b], rstd[b] = mu, (var + 1e-5) ** -0.5
        xh = (x[i] - mu.repeat_interleave(per)) * rstd[b].repeat_interleave(per)
        z = xh * gamma + beta
        y[i] = torch.nn.functional.silu(z) if c["act"] == "silu" else z
        if c["train"]:
            dz = st["d_y"][i].to(f)
            if c["act"] == "silu":
                sig = torch.sigmoid(z)
                dz = dz * (sig + y[i] * (1 - sig))
            dg += (dz * xh).sum(0)
            db += dz.sum(0)
            t = (dz * gamma).view(-1, c["groups"], per)
            u = xh.view(-1, c["groups"], per)
            dx[i] = (rstd[b][:, None] * (t - t.mean((0, 2))[:, None] - u * (t * u).mean((0, 2))[:, None])).view(-1, c["channels"])
    r = {"y": y, "mean": mean, "rstd": rstd}
    if c["train"]:
        r.update(d_x=dx, d_gamma=dg, d_beta=db)
    return r


def _exact_dropout(st, c):
    draws = c["rows"] * c["channels"]
    blocks = -(-draws // 8)
    at = np.arange(blocks, dtype=np.uint64) + np.uint64(st["offset"])
    half, low = np.uint64(32), np.uint64(0xFFFFFFFF)
    ctr = [at & low, at >> half, np.zeros_like(at), np.zeros_like(at)]
    key = [st["seed"] & 0xFFFFFFFF, st["seed"] >> 32]
    for r in range(10):
        p0, p1 = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        k0 = np.uint64((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF)
        k1 = np.uint64((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF)
        ctr = [(p1 >> half) ^ ctr[1] ^ k0, p1 & low, (p0 >> half) ^ ctr[3] ^ k1, p0 & low]
    lanes = np.stack([w.astype(np.uint32) for w in ctr], 1).astype("<u4").view("<u2").reshape(-1)[:draws]
    limit = round(c["p"] * 65536)
    keep = torch.from_numpy(lanes >= limit).cuda().view(c["rows"], c["channels"], 1).double()
    scale = 1.0 / (1.0 - limit / 65536)
    y = st["x"].double() * keep * scale
    if st["residual"] is not None:
        y = y + st["residual"].double()
    r = {"y": y}
    if c["train"]:
        r["d_x"] = st["d_y"].double() * keep * scale
    return r
