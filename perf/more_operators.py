"""Measured cases of the gated delta rule and of the norms around its block.

``run`` computes a case in plain torch operations (``own`` false) or through
the package's entry points (``own`` true) on the inputs that ``prepare`` made.

Operators, by the case's ``op``:

* ``delta``        gated_delta over prompts
* ``delta_train``  gated_delta with its checkpoints, then gated_delta_bwd
* ``delta_step``   gated_delta_step, one token per sequence
* ``gated``        gated_norm: the norm after the recurrence, with its gate
* ``gated_train``  gated_norm, then gated_norm_bwd
* ``residual``     residual_norm: the block's output added to the stream, and the next block's norm
* ``residual_train``  residual_norm, then residual_norm_bwd
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
CHUNK = 64  # tokens that the plain form takes together
EPS = 1e-6


def listed():
    return [
        # the first token's latency of a short chat prompt
        dict(name="delta_prompt_short", op="delta", dtype="bf16", batch=1, length=37, kheads=16, heads=16, dk=128,
             dv=128, ragged=False, start=False),
        # the prefill of one long document by a layer with two value heads to a key head
        dict(name="delta_prompt_long", op="delta", dtype="bf16", batch=1, length=32768, kheads=16, heads=32, dk=128,
             dv=128, ragged=False, start=True),
        # a right-padded batch of prompts that continue earlier states, evaluated in fp32, odd head sizes
        dict(name="delta_prompt_fp32", op="delta", dtype="f32", batch=3, length=1000, kheads=4, heads=8, dk=96,
             dv=72, ragged=True, start=True),
        # a layer's share of a training step
        dict(name="delta_train", op="delta_train", dtype="bf16", batch=4, length=2048, kheads=16, heads=16, dk=128,
             dv=128, ragged=False, start=False),
        # fine-tuning of a small fp32 layer on a padded batch of odd lengths
        dict(name="delta_train_fp32", op="delta_train", dtype="f32", batch=2, length=301, kheads=2, heads=4, dk=64,
             dv=80, ragged=True, start=True),
        # one sequence being decoded: launch latency
        dict(name="delta_step_one", op="delta_step", dtype="bf16", batch=1, kheads=16, heads=32, dk=128, dv=128),
        # a server's decode batch
        dict(name="delta_step_batch", op="delta_step", dtype="bf16", batch=128, kheads=16, heads=32, dk=128, dv=128),
        # the norm and gate of each head's output in a training step
        dict(name="gated_train", op="gated_train", dtype="bf16", rows=8192, heads=16, dim=128, gate_first=False),
        # the same behind an SSD layer, whose gate comes before a norm over all heads; a prompt of odd length
        dict(name="gated_prompt", op="gated", dtype="bf16", rows=1021, heads=1, dim=5120, gate_first=True),
        # a decode step's
        dict(name="gated_step", op="gated", dtype="bf16", rows=64, heads=32, dim=128, gate_first=False),
        # the residual stream in fp32 in a training step, each channel of the block's output with a learned scale
        dict(name="residual_train", op="residual_train", dtype="bf16", rows=8192, dim=2048, stream="f32", scaled=True),
        # the residual stream of a prompt
        dict(name="residual_prompt", op="residual", dtype="bf16", rows=16384, dim=4096, stream="bf16", scaled=False),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["delta", "delta", "delta_train", "delta_train", "delta_step", "gated", "gated_train", "residual",
                     "residual_train"])
    dtype = rng.choice(["bf16", "bf16", "f32", "f16"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op.startswith("delta"):
        kheads = rng.choice([1, 2, 4, 8, 16])
        heads = kheads * rng.choice([1, 1, 2, 4])
        dk = rng.choice([64, 128, 128, 256, log(8, 256)])
        dv = rng.choice([64, 128, 128, 256, log(8, 256)])
        if op == "delta_step":
            most = 128 * 32 * 128 * 128 // (heads * dk * dv)
            return dict(op=op, dtype=dtype, batch=log(1, max(1, min(256, most))), kheads=kheads, heads=heads, dk=dk,
                        dv=dv)
        batch = log(1, 16)
        size = heads * dk * dv * (8 if dtype == "f32" else 1)
        tokens = int((1.7e10 if op == "delta" else 2.1e9) / (batch * size))
        return dict(op=op, dtype=dtype, batch=batch, length=log(1, max(1, min(32768 if op == "delta" else 4096, tokens))),
                    kheads=kheads, heads=heads, dk=dk, dv=dv, ragged=flag(), start=flag())
    if op.startswith("gated"):
        dim = rng.choice([64, 128, 128, 256, log(8, 8192)])
        heads = rng.choice([1, 4, 16, 32]) if dim <= 512 else 1
        return dict(op=op, dtype=dtype, rows=log(1, max(1, min(16384, 3 * 10 ** 7 // (heads * dim)))), heads=heads, dim=dim,
                    gate_first=flag())
    dim = rng.choice([1024, 2048, 4096, log(64, 8192)])
    return dict(op=op, dtype=dtype, rows=log(1, max(1, min(16384, 3 * 10 ** 7 // dim))), dim=dim,
                stream=rng.choice(["f32", dtype]), scaled=flag())


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    s, op, dt = dict(case), case["op"], DTYPES[case["dtype"]]
    if op.startswith("gated"):
        n, H, dim = case["rows"], case["heads"], case["dim"]
        # the gate is a column range of the layer's first projection
        s["z"] = randn(n, (H + 1) * dim).to(dt)[:, dim:].unflatten(-1, (H, dim))
        s["x"] = (randn(n, H, dim) * torch.exp(0.5 * randn(n, H, 1))).to(dt)
        s["weight"] = 1 + 0.1 * randn(dim)
        s["dy"] = randn(n, H, dim).to(dt) if op == "gated_train" else None
        return s
    if op.startswith("residual"):
        n, dim, st = case["rows"], case["dim"], DTYPES[case["stream"]]
        s["x"] = randn(n, dim).to(dt)
        s["residual"] = (2 * randn(n, dim)).to(st)
        s["weight"] = 1 + 0.1 * randn(dim)
        s["scale"] = 0.5 + 0.1 * randn(dim) if case["scaled"] else None
        s["dy"] = randn(n, dim).to(dt) if op == "residual_train" else None
        s["dr"] = randn(n, dim).to(st) if op == "residual_train" else None
        return s
    n, Hk, H, dk, dv = (case[k] for k in ("batch", "kheads", "heads", "dk", "dv"))
    step = op == "delta_step"
    lead = (n,) if step else (n, case["length"])
    s["seqlens"] = None
    if case.get("ragged"):
        s["seqlens"] = (rand(n) * (case["length"] + 1)).to(torch.int32).clamp(max=case["length"])
    silu = lambda x: x * torch.sigmoid(x)  # noqa: E731
    # queries and keys have length one, after an activation that makes them alike in part
    s["q"] = _unit(silu(randn(*lead, Hk, dk))).to(dt)
    s["k"] = _unit(silu(randn(*lead, Hk, dk))).to(dt)
    # values are a column range of the convolution's output
    s["v"] = silu(randn(*lead, 8 + H * dv)).to(dt)[..., 8:].unflatten(-1, (H, dv))
    first = torch.exp(rand(H) * math.log(100.0)) * 0.001  # time steps spread over 0.001 to 0.1
    rate = 1 + 15 * rand(H)
    s["g"] = -rate * torch.nn.functional.softplus(randn(*lead, H) + torch.log(torch.expm1(first)))
    s["beta"] = torch.sigmoid(randn(*lead, H))
    s["h0"] = 0.3 * randn(n, H, dv, dk) if step or case["start"] else None
    s["dy"] = randn(*lead, H, dv).to(dt) if op == "delta_train" else None
    return s


def run(state):
    s, op = state, state["op"]
    if own:
        import chunked_linear_scan_amd as cls
        if op.startswith("gated"):
            args = (s["x"], s["weight"], s["z"])
            more = dict(eps=EPS, gate_first=s["gate_first"])
            if op == "gated":
                return {"y": cls.gated_norm(*args, **more)}
            y, kept = cls.gated_norm(*args, **more, want_rstd=True)
            return {"y": y, **cls.gated_norm_bwd(s["dy"], *args, rstd=kept, gate_first=s["gate_first"])}
        if op.startswith("residual"):
            args = (s["x"], s["residual"], s["weight"])
            if op == "residual":
                y, r = cls.residual_norm(*args, scale=s["scale"], eps=EPS)
                return {"y": y, "r": r}
            y, r, kept = cls.residual_norm(*args, scale=s["scale"], eps=EPS, want_rstd=True)
            return {"y": y, "r": r, **cls.residual_norm_bwd(s["dy"], r, s["weight"], kept, dr=s["dr"], x=s["x"],
                                                            scale=s["scale"])}
        args = tuple(s[k] for k in ("q", "k", "v", "g", "beta"))
        if op == "delta_step":
            return {"y": cls.gated_delta_step(s["h0"], *args), "h": s["h0"]}
        more = dict(h0=s["h0"], seqlens=s["seqlens"])
        if op == "delta":
            y, h = cls.gated_delta(*args, **more)
            return {"y": y, "h": h}
        y, _, kept = cls.gated_delta(*args, **more, want_final_state=False, want_checkpoints=True)
        return {"y": y, **cls.gated_delta_bwd(s["dy"], *args, **more, checkpoints=kept)}
    if op.startswith("gated"):
        return _plain_gated(s)
    if op.startswith("residual"):
        return _plain_residual(s)
    return {"delta": _plain_delta, "delta_train": _plain_delta_train, "delta_step": _plain_delta_step}[op](s)


# ---------------------------------------------------------------------------
# the plain forms: torch operations over whole tensors, in 32 bits
# ---------------------------------------------------------------------------
def _plain_gated(s):
    kind, w = s["x"].dtype, s["weight"]
    x, z = s["x"].float(), s["z"].float()
    sig = torch.sigmoid(z)
    gate = z * sig
    first = s["gate_first"]
    u = x * gate if first else x
    rstd = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
    unit = u * rstd
    y = unit * w if first else unit * w * gate
    if s["op"] == "gated":
        return {"y": y.to(kind)}
    dy = s["dy"].float()
    dgate = sig * (1 + z * (1 - sig))
    dn = dy if first else dy * gate  # the gradient of the norm's result
    dunit = dn * w
    du = rstd * (dunit - unit * (dunit * unit).mean(-1, keepdim=True))
    dx = du * gate if first else du
    dz = (du * x if first else dy * unit * w) * dgate
    return {"y": y.to(kind), "dx": dx.to(kind), "dweight": (dn * unit).sum((0, 1)), "dz": dz.to(kind)}


def _plain_residual(s):
    kind, w = s["x"].dtype, s["weight"]
    x = s["x"].float()
    r = s["residual"].float() + (x if s["scale"] is None else x * s["scale"])
    r = r.to(s["residual"].dtype)  # the stream as it goes on: what the norm sees
    u = r.float()
    rstd = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
    unit = u * rstd
    got = {"y": (unit * w).to(kind), "r": r}
    if s["op"] == "residual":
        return got
    dy = s["dy"].float()
    dunit = dy * w
    du = s["dr"].float() + rstd * (dunit - unit * (dunit * unit).mean(-1, keepdim=True))
    got |= {"dresidual": du.to(r.dtype), "dweight": (dy * unit).sum(0)}
    got["dx"] = (du if s["scale"] is None else du * s["scale"]).to(kind)
    if s["scale"] is not None:
        got["dscale"] = (du * x).sum(0)
    return got


def _inverse(A):
    """(I + A)^-1 of strictly lower triangular matrices, by halves."""
    n = A.shape[-1]
    T = A.new_ones(*A.shape[:-2], n, 1, 1)  # the diagonal blocks' inverses
    size = 1
    while size < n:
        parts = n // (2 * size)
        pair = T.unflatten(-3, (parts, 2))
        T1, T2 = pair[..., 0, :, :], pair[..., 1, :, :]
        low = torch.stack([A[..., (2 * i + 1) * size:(2 * i + 2) * size, 2 * i * size:(2 * i + 1) * size]
                           for i in range(parts)], -3)
        low = -(T2 @ (low @ T1))
        T = torch.cat([torch.cat([T1, torch.zeros_like(T1)], -1), torch.cat([low, T2], -1)], -2)
        size *= 2
    return T[..., 0, :, :]


def _chunks(s, q, k, v, g, beta, h0):
    """y [n, L, H, dv] and the last state [n, H, dv, dk] in 32 bits, a chunk of tokens at a time."""
    n, L, H, dv = v.shape
    dk, rep, pad = q.shape[-1], H // q.shape[2], -v.shape[1] % CHUNK
    if s["seqlens"] is not None:
        on = torch.arange(L, device="cuda") < s["seqlens"][:, None]
        g, beta = torch.where(on[..., None], g, 0.0), torch.where(on[..., None], beta, 0.0)
        q, k, v = (torch.where(on[..., None, None], x, 0.0) for x in (q, k, v))
    q, k = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    # [n, H, chunks, CHUNK, ..]
    cut = lambda x: torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, pad)).unflatten(1, (-1, CHUNK)).movedim(  # noqa: E731
        3, 1).contiguous()
    q, k, v, g, beta = (cut(x) for x in (q, k, v, g, beta))
    sums = torch.cumsum(g.double(), -1)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    span = (sums[..., :, None] - sums[..., None, :]).masked_fill(~lower, -math.inf)
    decay = torch.exp(span).float()
    start, end = torch.exp(sums).float(), torch.exp(sums[..., -1:] - sums).float()
    kT = k.transpose(-1, -2).contiguous()
    T = _inverse((beta[..., None] * decay * (k @ kT)).tril(-1)) * beta[..., None, :]
    P = decay * (q @ kT) * dk ** -0.5
    qs, ks, kend = q * (start * dk ** -0.5)[..., None], k * start[..., None], (k * end[..., None]).transpose(-1, -2).contiguous()
    h = torch.zeros(n, H, dk, dv, device="cuda") if h0 is None else h0.transpose(-1, -2).contiguous()
    ys = []
    for c in range(q.shape[2]):
        new = T[:, :, c] @ (v[:, :, c] - ks[:, :, c] @ h)
        ys.append(qs[:, :, c] @ h + P[:, :, c] @ new)
        h = h * start[:, :, c, -1, None, None] + kend[:, :, c] @ new
    y = torch.stack(ys, 2).flatten(2, 3)[:, :, :L].transpose(1, 2)
    return y, h.transpose(-1, -2)


def _plain_delta(s):
    y, h = _chunks(s, s["q"].float(), s["k"].float(), s["v"].float(), s["g"], s["beta"], s["h0"])
    return {"y": y.to(s["v"].dtype).contiguous(), "h": h.contiguous()}


def _plain_delta_train(s):
    names = ["q", "k", "v", "g", "beta"] + ([] if s["h0"] is None else ["h0"])
    with torch.enable_grad():
        leaf = {k: s[k].detach().float().clone().requires_grad_() for k in names}
        y, _ = _chunks(s, *(leaf.get(k) for k in ("q", "k", "v", "g", "beta", "h0")))
        grads = torch.autograd.grad(y, [leaf[k] for k in names], s["dy"].float())
    got = {"y": y.detach().to(s["v"].dtype).contiguous()}
    for k, d in zip(names, grads):
        got["d" + k] = d.to(s[k].dtype).contiguous()
    return got


def _plain_delta_step(s):
    h, rep, dk = s["h0"], s["v"].shape[1] // s["q"].shape[1], s["q"].shape[-1]
    q, k = (s[x].float().repeat_interleave(rep, 1)[:, :, None, :] for x in "qk")
    h.mul_(torch.exp(s["g"])[..., None, None])
    new = s["beta"][..., None] * (s["v"].float() - (h * k).sum(-1))
    h.addcmul_(new[..., None], k)
    return {"y": ((h * q).sum(-1) * dk ** -0.5).to(s["v"].dtype), "h": h}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, size = case["op"], SIZE[case["dtype"]]
    if op.startswith("gated"):
        values = case["rows"] * case["heads"] * case["dim"]
        params = case["dim"] * 4
        if op == "gated":  # x, z in; y out
            return {"bytes": 3 * values * size + params, "flops": 10 * values}
        return {"bytes": 6 * values * size + 2 * params, "flops": 35 * values}  # and dy in, dx, dz out
    if op.startswith("residual"):
        values, wide = case["rows"] * case["dim"], SIZE[case["stream"]]
        params = case["dim"] * (8 if case["scaled"] else 4)
        if op == "residual":  # x, residual in; y, r out
            return {"bytes": 2 * values * (size + wide) + params, "flops": 7 * values}
        return {"bytes": values * (4 * size + 4 * wide) + 2 * params, "flops": 20 * values}
    n, Hk, H, dk, dv = (case[k] for k in ("batch", "kheads", "heads", "dk", "dv"))
    tokens, state = n * case.get("length", 1), n * H * dk * dv * 4
    io = tokens * ((2 * Hk * dk + 2 * H * dv) * size + 2 * H * 4)
    # a chunk of 64 tokens: keys with keys and queries, the two products with the state, the state's update, the
    # triangle's inverse and its products with the values
    per = 2 * dk * dv * 3 + 64 * (2 * dk + 2 * dv) + 64 * 64 // 3
    if op == "delta_train":  # the gradients of all that came in, too, and dy
        io += tokens * ((2 * Hk * dk + 2 * H * dv) * size + 2 * H * 4)
        return {"bytes": io + (2 * state if case["start"] else 0), "flops": 3 * tokens * H * per}
    if op == "delta_step":
        return {"bytes": io + 2 * state, "flops": tokens * H * 8 * dk * dv}
    return {"bytes": io + (2 * state if case["start"] else state), "flops": tokens * H * per}


# ---------------------------------------------------------------------------
# the definitions in 64 bits: token by token, row by row
# ---------------------------------------------------------------------------
def _wide(v):
    return None if v is None else v.double()


def _exact_gated(s):
    x, z, w = _wide(s["x"]), _wide(s["z"]), _wide(s["weight"])
    dim, first = x.shape[-1], s["gate_first"]
    sig = 1 / (1 + torch.exp(-z))
    u = x * z * sig if first else x
    length = torch.sqrt((u ** 2).sum(-1, keepdim=True) / dim + EPS)
    y = u / length * w
    y = y if first else y * (z * sig)
    if s["op"] == "gated":
        return {"y": y}
    dy = _wide(s["dy"])
    slope = sig + z * sig * (1 - sig)
    into = dy * w if first else dy * w * z * sig  # of u / length
    du = into / length - u * (into * u).sum(-1, keepdim=True) / (dim * length ** 3)
    if first:
        dx, dz, dw = du * z * sig, du * x * slope, dy * u / length
    else:
        dx, dz, dw = du, dy * w * u / length * slope, dy * z * sig * u / length
    return {"y": y, "dx": dx, "dweight": dw.sum((0, 1)), "dz": dz}


def _exact_residual(s):
    x, w, res = _wide(s["x"]), _wide(s["weight"]), _wide(s["residual"])
    scale = torch.ones_like(w) if s["scale"] is None else _wide(s["scale"])
    exact_r = res + scale * x
    r = _wide(exact_r.to(s["residual"].dtype))  # the stream's values are of its type by definition
    dim = r.shape[-1]
    length = torch.sqrt((r ** 2).sum(-1, keepdim=True) / dim + EPS)
    got = {"y": r / length * w, "r": exact_r}
    if s["op"] == "residual":
        return got
    dy = _wide(s["dy"])
    into = dy * w
    du = _wide(s["dr"]) + into / length - r * (into * r).sum(-1, keepdim=True) / (dim * length ** 3)
    got |= {"dresidual": du, "dweight": (dy * r / length).sum(0), "dx": du * scale}
    if s["scale"] is not None:
        got["dscale"] = (du * x).sum(0)
    return got


def _exact_delta(s, train):
    one = s["op"] == "delta_step"
    q, k, v, g, beta = (_wide(s[x])[:, None] if one else _wide(s[x]) for x in ("q", "k", "v", "g", "beta"))
    n, L, H, dv = v.shape
    dk = q.shape[-1]
    of = torch.arange(H, device="cuda") // (H // q.shape[2])  # a head's key head
    ends = torch.full((n,), L, device="cuda") if s.get("seqlens") is None else s["seqlens"].long()
    h = torch.zeros(n, H, dv, dk, dtype=torch.float64, device="cuda") if s["h0"] is None else _wide(s["h0"])
    c = 1 / math.sqrt(dk)
    y, kept = torch.zeros_like(v), []
    for t in range(L):
        on = (t < ends)[:, None, None]
        kt, qt = k[:, t, of], q[:, t, of]
        faded = torch.exp(g[:, t])[..., None, None] * h
        miss = v[:, t] - torch.einsum("nhvk,nhk->nhv", faded, kt)
        new = faded + torch.einsum("nhv,nhk->nhvk", beta[:, t, :, None] * miss, kt)
        if train:
            kept.append((h, miss))
        h = torch.where(on[..., None], new, h)
        y[:, t] = torch.where(on, c * torch.einsum("nhvk,nhk->nhv", new, qt), 0.0)
    if not train:
        return {"y": y[:, 0] if one else y, "h": h}
    dq, dk_, dv_, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
    back = torch.zeros_like(h)  # the gradient of the state after the token
    for t in reversed(range(L)):
        on = (t < ends)[:, None, None]
        kt, qt, (before, miss) = k[:, t, of], q[:, t, of], kept[t]
        kept[t] = None
        a, b = torch.exp(g[:, t])[..., None, None], beta[:, t, :, None]
        dy = torch.where(on, _wide(s["dy"][:, t]), 0.0)
        new = a * before + torch.einsum("nhv,nhk->nhvk", b * miss, kt)
        dq[:, t].index_add_(1, of, c * torch.einsum("nhvk,nhv->nhk", new, dy))
        d = torch.where(on[..., None], back + c * torch.einsum("nhv,nhk->nhvk", dy, qt), 0.0)
        dk_b = torch.einsum("nhvk,nhk->nhv", d, kt)  # the gradient of beta times the miss
        dmiss = b * dk_b
        db[:, t] = (dk_b * miss).sum(-1)
        dv_[:, t] = dmiss
        dkt = torch.einsum("nhvk,nhv->nhk", d, b * miss) - torch.einsum("nhvk,nhv->nhk", a * before, dmiss)
        dk_[:, t].index_add_(1, of, dkt)
        dfaded = d - torch.einsum("nhv,nhk->nhvk", dmiss, kt)
        dg[:, t] = (dfaded * a * before).sum((-1, -2))
        back = torch.where(on[..., None], dfaded * a, back)
    got = {"y": y, "dq": dq, "dk": dk_, "dv": dv_, "dg": dg, "dbeta": db}
    if s["h0"] is not None:
        got["dh0"] = back
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("gated"):
        return _exact_gated(s)
    if case["op"].startswith("residual"):
        return _exact_residual(s)
    return _exact_delta(s, case["op"].endswith("_train"))
