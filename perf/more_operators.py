"""Workloads of the norm, gate and delta-rule operators: what is measured of
them, in plain torch (`own` false) and through the framework's calls (`own`
true).

  norm   layer norm over rows or padded sequences: forward, or forward and backward
         with the gradients of weight and bias
  gate   a router's choices, weights, counts and losses from its logits, and the
         logits' gradient
  delta  the gated delta rule over [batch, time, heads, dim]: forward, forward and
         backward, or one token per session on state rows
"""
import torch

own = False

DTYPE = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZE = {"float32": 4, "bfloat16": 2, "float16": 2}
EPS = 1e-5
CHUNK = 64           # positions that the plain form of the delta rule takes at once


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # serving: one new event for each of 192 sessions
        dict(name="norm_serve", op="norm", mode="forward", rows=192, dim=256, dtype="bfloat16"),
        # odd sizes: training a narrow layer
        dict(name="norm_odd", op="norm", mode="train", rows=5003, dim=99, dtype="float16"),
        # training over the padded sequences of the benchmark's sequence workload (batch 1024, lengths 200..1000 of
        # 1000)
        dict(name="norm_sequences", op="norm", mode="train", batch=1024, time=1000, min_len=200, dim=64,
             dtype="float32"),
        # training a wide layer
        dict(name="norm_wide", op="norm", mode="train", rows=131072, dim=1024, dtype="bfloat16"),
        # serving: eight tokens choose among sixteen experts
        dict(name="gate_decode", op="gate", mode="forward", tokens=8, top_k=2, experts=16, dead=0.0, normalize=True,
             dtype="bfloat16"),
        # odd sizes, padded tokens, weights that are not normalised
        dict(name="gate_odd", op="gate", mode="train", tokens=5003, top_k=3, experts=37, dead=0.1, normalize=False,
             dtype="float16"),
        # training a wide layer of many experts
        dict(name="gate_wide", op="gate", mode="train", tokens=131072, top_k=4, experts=128, dead=0.0, normalize=True,
             dtype="float32"),
        # serving: one new event for each of 192 sessions, their states among 5000
        dict(name="delta_step", op="delta", mode="step", batch=192, rows=5000, heads=4, key_heads=4, key_dim=64,
             value_dim=64, dtype="bfloat16"),
        # serving: the first pass over a handful of new sessions, odd widths
        dict(name="delta_prefill_odd", op="delta", mode="forward", batch=5, time=333, min_len=1, heads=3, key_heads=1,
             key_dim=50, value_dim=42, dtype="float16"),
        # training over the padded sequences of the benchmark's sequence workload, two heads of 32
        dict(name="delta_sequences", op="delta", mode="train", batch=1024, time=1000, min_len=200, heads=2, key_heads=2,
             key_dim=32, value_dim=32, dtype="float32"),
        # training over one long history, a few wide heads
        dict(name="delta_long", op="delta", mode="train", batch=1, time=32768, min_len=32768, heads=4, key_heads=4,
             key_dim=128, value_dim=128, dtype="bfloat16"),
        # training a wide layer, two value heads to a key head
        dict(name="delta_wide", op="delta", mode="train", batch=32, time=2048, min_len=1024, heads=8, key_heads=4,
             key_dim=128, value_dim=128, dtype="bfloat16"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "gate", "delta", "delta"])
    dtype = rng.choice(["float32", "bfloat16", "float16"])
    if op == "norm":
        mode = rng.choice(["forward", "train", "train"])
        dim = _log(rng, 8, 8192)
        if rng.random() < 0.6:
            dim = max(8, dim // 8 * 8)
        rows = max(1, _log(rng, 2_000, 60_000_000) // dim)
        if rng.random() < 0.5:
            return dict(op=op, mode=mode, rows=rows, dim=dim, dtype=dtype)
        time = _log(rng, 1, min(rows, 5000))
        return dict(op=op, mode=mode, batch=max(1, rows // time), time=time,
                    min_len=rng.choice([0, (time + 1) // 2, time]), dim=dim, dtype=dtype)
    if op == "gate":
        experts = _log(rng, 4, 1024)
        top_k = min(rng.choice([1, 2, 3, 4, 6, 8]), experts)
        return dict(op=op, mode=rng.choice(["forward", "train", "train"]),
                    tokens=_log(rng, 1, min(200_000, 16_000_000 // experts)), top_k=top_k, experts=experts,
                    dead=rng.choice([0.0, 0.0, 0.2]), normalize=rng.random() < 0.7, dtype=dtype)
    mode = rng.choice(["step", "forward", "train", "train"])
    key_dim, value_dim = (rng.choice([16, 32, 64, 128, _log(rng, 8, 128)]) for _ in range(2))
    key_heads = rng.choice([1, 2, 3, 4])
    heads = key_heads * rng.choice([1, 1, 2])
    if mode == "step":
        batch = _log(rng, 1, 4096)
        return dict(op=op, mode=mode, batch=batch, rows=batch + _log(rng, 1, 5000), heads=heads, key_heads=key_heads,
                    key_dim=key_dim, value_dim=value_dim, dtype=dtype)
    budget = _log(rng, 200, 250_000) // heads      # positions
    time = _log(rng, 1, min(16384, max(2, budget)))
    batch = max(1, budget // time)
    return dict(op=op, mode=mode, batch=batch, time=time, min_len=rng.choice([0, (time + 1) // 2, time]), heads=heads,
                key_heads=key_heads, key_dim=key_dim, value_dim=value_dim, dtype=dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(gen, *shape, scale=1.0, shift=0.0, dtype=torch.float32):
    x = torch.empty(shape, dtype=torch.float32, device="cuda")
    return x.normal_(shift, scale, generator=gen).to(dtype)


def _offsets(case, gen):
    lens = torch.randint(case["min_len"], case["time"] + 1, (case["batch"],), generator=gen, device="cuda")
    return torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"norm": _prepare_norm, "gate": _prepare_gate, "delta": _prepare_delta}[case["op"]](case, gen)


def _prepare_norm(case, gen):
    s = dict(case=case, plan=None, offsets=None)
    D, dt = case["dim"], DTYPE[case["dtype"]]
    padded = "batch" in case
    shape = (case["batch"], case["time"], D) if padded else (case["rows"], D)
    # channels of different means and sizes, as a residual stream has them
    size, mean = torch.exp(_randn(gen, D, scale=0.5)), _randn(gen, D, scale=0.3)
    s["x"] = (_randn(gen, *shape) * size + mean).to(dt)
    s["weight"], s["bias"] = _randn(gen, D, scale=0.2, shift=1.0), _randn(gen, D, scale=0.2)
    if padded:
        s["offsets"] = _offsets(case, gen)
    if case["mode"] == "train":
        s["grad_y"] = _randn(gen, *shape, dtype=dt)
    if own:     # the handle a program keeps between calls
        import sparse_lookup_gb300 as sl
        s["plan"] = sl.LayerNorm(D, eps=EPS)
    return s


def _prepare_gate(case, gen):
    s = dict(case=case, plan=None, live=None)
    T, K, E, dt = case["tokens"], case["top_k"], case["experts"], DTYPE[case["dtype"]]
    # logits with a tilt, so that experts get unequal shares
    s["logits"] = (_randn(gen, T, E) + _randn(gen, E, scale=0.7)).to(dt)
    if case["dead"]:
        s["live"] = torch.rand(T, generator=gen, device="cuda") >= case["dead"]
    if case["mode"] == "train":
        # of a mean over the tokens, under a loss scale of T that keeps 16-bit gradients in range
        s["grad_weights"] = _randn(gen, T, K)
        s["grad_losses"] = torch.tensor([0.01 * T, 0.001 * T], device="cuda")
    if own:     # the handle a program keeps between calls
        import sparse_lookup_gb300 as sl
        s["plan"] = sl.ExpertRouter(E, K, max_tokens=T)
    return s


def _prepare_delta(case, gen):
    s = dict(case=case, plan=None)
    B, H, J, N, V, dt = (case[k] for k in ("batch", "heads", "key_heads", "key_dim", "value_dim", "dtype"))
    dt = DTYPE[dt]
    step = case["mode"] == "step"
    lead = (B,) if step else (B, case["time"])

    def unit(x):
        return x / x.square().sum(-1, keepdim=True).sqrt()
    k = unit(_randn(gen, *lead, J, N))
    if not step:        # now and then an item comes twice in a row
        again = torch.rand(*lead, 1, 1, generator=gen, device="cuda") < 0.2
        k = torch.where(again, k.roll(1, 1), k)
    s["q"], s["k"] = unit(_randn(gen, *lead, J, N)).to(dt), k.to(dt)
    s["v"] = _randn(gen, *lead, H, V, dtype=dt)
    # logarithms of the decays: mostly some per cent a position, now and then nearly all
    s["decay"] = -torch.exp(_randn(gen, *lead, H, scale=1.2, shift=-3.0))
    s["beta"] = torch.sigmoid(_randn(gen, *lead, H))
    if step:
        # one more row than the calls are told of: the plain form writes there what has no row
        s["pool"] = _randn(gen, case["rows"] + 1, H, N, V, scale=0.3)
        s["states"] = s["pool"][:-1]
        s["rows"] = torch.randperm(case["rows"], generator=gen, device="cuda")[:B].contiguous()
        if B > 8:
            s["rows"][5] = -1               # a session whose key has no row yet
    else:
        s["offsets"] = _offsets(case, gen)
        s["state"] = _randn(gen, B, H, N, V, scale=0.3)
        if case["mode"] == "train":
            s["grad_y"] = _randn(gen, *lead, H, V, dtype=dt)
            s["grad_last"] = _randn(gen, B, H, N, V, scale=0.1)
    if own:     # the handle a program keeps between calls
        import sparse_lookup_gb300 as sl
        s["plan"] = sl.DeltaScan(N, V, H, key_heads=J, max_batch=B, max_len=case.get("time", 1),
                                 training=case["mode"] == "train")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return {"norm": _run_norm, "gate": _run_gate, "delta": _run_delta}[state["case"]["op"]](state)


def _live(s, shape):
    """Which positions of [batch, time] are not past their entry's end."""
    lens = s["offsets"].diff().clamp(max=shape[1])
    return torch.arange(shape[1], device="cuda")[None] < lens[:, None]


def _run_norm(s):
    train = s["case"]["mode"] == "train"
    if own:
        y, stats = s["plan"].forward(s["x"], s["weight"], s["bias"], offsets=s["offsets"])
        if not train:
            return dict(y=y)
        gx, gw, gb = s["plan"].backward(s["x"], s["grad_y"], stats, s["weight"], offsets=s["offsets"])
        return dict(y=y, grad_x=gx, grad_weight=gw, grad_bias=gb)
    dt, D = s["x"].dtype, s["x"].shape[-1]
    live = None if s["offsets"] is None else _live(s, s["x"].shape)[..., None]
    x = s["x"].float()
    if live is not None:
        x = torch.where(live, x, 0.0)
    c = x - x.mean(-1, keepdim=True)
    rstd = (c.square().mean(-1, keepdim=True) + EPS).rsqrt()
    xh = c * rstd
    y = xh * s["weight"] + s["bias"]
    out = dict(y=(y if live is None else y * live).to(dt))
    if train:
        dy = s["grad_y"].float()
        if live is not None:
            dy = torch.where(live, dy, 0.0)
        dxh = dy * s["weight"]
        gx = rstd * (dxh - dxh.mean(-1, keepdim=True) - xh * (dxh * xh).mean(-1, keepdim=True))
        out["grad_x"] = gx.to(dt)
        out["grad_weight"], out["grad_bias"] = (dy * xh).view(-1, D).sum(0), dy.view(-1, D).sum(0)
    return out


def _run_gate(s):
    c = s["case"]
    train = c["mode"] == "train"
    if own:
        g = s["plan"].gate(s["logits"], live=s["live"], normalize=c["normalize"])
        out = dict(experts=g.experts, weights=g.weights, counts=g.counts, losses=g.losses)
        if train:
            out["grad_logits"] = s["plan"].gate_backward(s["logits"], g, s["grad_weights"], s["grad_losses"])
        return out
    T, K, E, dt = c["tokens"], c["top_k"], c["experts"], s["logits"].dtype
    x = s["logits"].float()
    live = torch.ones(T, 1, dtype=torch.bool, device="cuda") if s["live"] is None else s["live"][:, None]
    x = torch.where(live, x, 0.0)
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)      # ties go to the lowest expert
    ids = ids[:, :K]
    e = torch.exp(x - top[:, :1])
    total = e.sum(1, keepdim=True)
    p, lse = e / total * live, (top[:, :1] + torch.log(total)) * live
    n = live.sum().clamp(min=1)
    chosen = torch.zeros_like(x).scatter_(1, ids, 1.0) * live
    counts = torch.zeros(E, dtype=torch.int32, device="cuda").index_add_(
        0, ids.reshape(-1), live.expand(T, K).reshape(-1).to(torch.int32))
    w = p.gather(1, ids)
    if c["normalize"]:
        w = torch.where(live, e.gather(1, ids), 0.0)
        w = w / torch.where(live, w.sum(1, keepdim=True), 1.0)
    share = counts.float() / (n * K)
    balance = E * (share * (p.double().sum(0) / n).float()).sum()
    z = (lse.double().square().sum() / n).float()
    out = dict(experts=torch.where(live, ids, -1).to(torch.int32), weights=w, counts=counts,
               losses=torch.stack([balance, z]))
    if train:
        gw = torch.where(live, s["grad_weights"], 0.0)
        gb, gz = s["grad_losses"][0], s["grad_losses"][1]
        each = gb * E * share / n
        grad = p * (each - (p * each).sum(1, keepdim=True)) + 2 * gz / n * lse * p
        mean = (w * gw).sum(1, keepdim=True)
        if c["normalize"]:
            grad = grad.scatter_add(1, ids, w * (gw - mean))
        else:
            grad = grad.scatter_add(1, ids, w * gw) - p * mean
        out["grad_logits"] = (grad * live).to(dt)
    return out


def _run_delta(s):
    c = s["case"]
    H, J, N = c["heads"], c["key_heads"], c["key_dim"]
    scale, share = N ** -0.5, H // J
    if c["mode"] == "step":
        if own:
            y = s["plan"].step(s["q"], s["k"], s["v"], s["decay"], s["beta"], s["rows"], s["states"])
            return dict(y=y, states=s["states"])
        live = (s["rows"] >= 0)[:, None, None]
        rows = s["rows"].clamp(min=0)
        q, k = (s[x].float().repeat_interleave(share, 1)[..., None] for x in "qk")
        old = s["states"][rows] * torch.exp(s["decay"])[..., None, None]
        error = s["v"].float() - (old * k).sum(2)
        new = old + (s["beta"][..., None] * error)[:, :, None] * k
        s["pool"][torch.where(live[:, 0, 0], rows, s["states"].shape[0])] = new
        return dict(y=((new * q).sum(2) * scale * live).to(s["v"].dtype), states=s["states"])
    train = c["mode"] == "train"
    if own:
        args = (s["q"], s["k"], s["v"], s["decay"], s["beta"])
        y, last = s["plan"].forward(*args, offsets=s["offsets"], state=s["state"])
        if not train:
            return dict(y=y, last=last)
        gq, gk, gv, gd, gb, gs = s["plan"].backward(*args, s["grad_y"], offsets=s["offsets"], state=s["state"],
                                                    grad_last=s["grad_last"])
        return dict(y=y, last=last, grad_q=gq, grad_k=gk, grad_v=gv, grad_decay=gd, grad_beta=gb, grad_state=gs)
    B, T, dt = c["batch"], c["time"], s["v"].dtype
    live = _live(s, (B, T))
    chunks = (T + CHUNK - 1) // CHUNK

    def split(x, repeat=1):     # [B, T, h, d] -> [B, h, chunks, CHUNK, d], nothing past an entry's end
        x = torch.where(live[:, :, None, None], x.float(), 0.0).repeat_interleave(repeat, 2)
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, chunks * CHUNK - T))
        return x.view(B, chunks, CHUNK, H, -1).permute(0, 3, 1, 2, 4)

    def join(x):
        return x.permute(0, 2, 3, 1, 4).reshape(B, chunks * CHUNK, H, -1)[:, :T]
    q, k, v = split(s["q"], share) * scale, split(s["k"], share), split(s["v"])
    beta = split(s["beta"][..., None])
    G = split(s["decay"][..., None])[..., 0].double().cumsum(-1)       # logarithms of the decays since the chunk began
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    D = torch.exp(torch.where(lower, G[..., :, None] - G[..., None, :], -torch.inf)).float()
    since, until = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    whole = since[..., -1:, :]
    M = (k @ k.mT) * D.tril(-1)
    inv = _unit_lower_inverse(M * beta.mT)
    A = (q @ k.mT) * D
    W, U0 = inv @ (k * since), inv @ v
    kb = k * (until * beta)
    step = whole * torch.eye(N, device="cuda") - kb.mT @ W
    S1 = _states(step, kb.mT @ U0, s["state"].float())
    S0 = torch.cat([s["state"].float()[:, :, None], S1[:, :, :-1]], 2)
    E = U0 - W @ S0
    U = beta * E
    y = since * (q @ S0) + A @ U
    out = dict(y=join(y).to(dt), last=S1[:, :, -1])
    if not train:
        return out
    dy = split(s["grad_y"])
    dU = A.mT @ dy
    # what the state before a chunk gets from the chunk itself, and through the state after it
    own_part = (q * since).mT @ dy - W.mT @ (beta * dU)
    d0 = _states(step.flip(2).mT, own_part.flip(2), s["grad_last"]).flip(2)
    d1 = torch.cat([d0[:, :, 1:], s["grad_last"][:, :, None]], 2)
    dU = dU + until * (k @ d1)
    dZ = inv.mT @ (beta * dU)
    dA = (dy @ U.mT) * D
    X = -(dZ @ U.mT) * D.tril(-1)
    gq = since * (dy @ S0.mT) + dA @ k
    gk = until * (U @ d1.mT) - since * (dZ @ S0.mT) + dA.mT @ q + X @ k + X.mT @ k
    gb = (E * (dU - M.mT @ dZ)).sum(-1)
    e = dA * (q @ k.mT) + X * (k @ k.mT)
    after = (until * U * (k @ d1)).sum(-1)
    dG = e.sum(-1) - e.sum(-2) + since[..., 0] * ((dy * (q @ S0)).sum(-1) - (dZ * (k @ S0)).sum(-1)) - after
    dG[..., -1] += after.sum(-1) + (whole * d1 * S0).sum((-1, -2))
    gd = dG.double().flip(-1).cumsum(-1).flip(-1).float()

    def shared(x):      # a key head's gradient is the sum over its value heads
        x = join(x)
        return x.view(B, T, J, share, N).sum(3) if share > 1 else x
    out.update(grad_q=(shared(gq) * scale).to(dt), grad_k=shared(gk).to(dt), grad_v=join(dZ).to(dt),
               grad_decay=join(gd[..., None])[..., 0], grad_beta=join(gb[..., None])[..., 0], grad_state=d0[:, :, 0])
    for name in ("grad_decay", "grad_beta"):
        out[name] = torch.where(live[:, :, None], out[name], 0.0)
    return out


def _unit_lower_inverse(M):
    """(I + M)^-1 for strictly lower M: the two halves' inverses together, then the block below them."""
    n = M.shape[-1]
    if n == 4:
        return torch.eye(4, device="cuda") - M + M @ M - M @ M @ M
    h = n // 2
    both = _unit_lower_inverse(torch.stack([M[..., :h, :h], M[..., h:, h:]], -3))
    a, b = both[..., 0, :, :], both[..., 1, :, :]
    out = torch.zeros_like(M)
    out[..., :h, :h], out[..., h:, h:] = a, b
    out[..., h:, :h] = -(b @ M[..., h:, :h] @ a)
    return out


def _states(M, N, S):
    """S_n = M_n S_{n-1} + N_n along axis 2 from S, in log depth: neighbours are joined to pairs, the pairs' states
    found first, the odd ones out filled in."""
    return _joined(M, torch.cat([N[:, :, :1] + M[:, :, :1] @ S[:, :, None], N[:, :, 1:]], 2))


def _joined(M, N):
    n = M.shape[2]
    if n == 1:
        return N
    m = n // 2
    Me, Mo, Ne, No = M[:, :, 0:2 * m:2], M[:, :, 1::2], N[:, :, 0:2 * m:2], N[:, :, 1::2]
    odd = _joined(Mo @ Me, Mo @ Ne + No)
    S = torch.empty_like(N)
    S[:, :, 1::2] = odd
    S[:, :, 0] = N[:, :, 0]
    S[:, :, 2::2] = M[:, :, 2::2] @ odd[:, :, :(n - 1) // 2] + N[:, :, 2::2]
    return S


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    e, train = SIZE[case["dtype"]], case["mode"] == "train"
    if case["op"] == "norm":
        D = case["dim"]
        if "batch" in case:
            whole = case["batch"] * case["time"]
            rows = case["batch"] * (case["min_len"] + case["time"]) / 2
        else:
            whole = rows = case["rows"]
        bytes_ = rows * D * e + whole * D * e + 8 * D            # x; y; weight and bias
        flops = 8 * rows * D
        if train:       # x and grad_y again; the gradients; the rows' mean and deviation there and back
            bytes_ += 2 * rows * D * e + whole * D * e + 12 * D + 16 * rows
            flops += 15 * rows * D
        return {"bytes": bytes_, "flops": flops}
    if case["op"] == "gate":
        T, K, E = case["tokens"], case["top_k"], case["experts"]
        rows = T * (1 - case["dead"])
        bytes_ = rows * E * e + 8 * T * K + 4 * E
        flops = (6 + K) * rows * E
        if train:       # logits again and the choices, their weights and gradients; the logits' gradient
            bytes_ += rows * E * e + T * E * e + 12 * T * K
            flops += 10 * rows * E
        return {"bytes": bytes_, "flops": flops}
    B, H, J, N, V = (case[k] for k in ("batch", "heads", "key_heads", "key_dim", "value_dim"))
    if case["mode"] == "step":
        return {"bytes": B * (H * N * V * 8 + (2 * J * N + 2 * H * V) * e + 8 * H + 8), "flops": 7 * B * H * N * V}
    whole = B * case["time"]
    rows = B * (case["min_len"] + case["time"]) / 2
    bytes_ = rows * ((2 * J * N + H * V) * e + 8 * H) + whole * H * V * e + 8 * B * H * N * V
    flops = 7 * rows * H * N * V
    if train:       # the inputs again with grad_y; their gradients
        bytes_ += rows * ((2 * J * N + 2 * H * V) * e + 8 * H) + whole * ((2 * J * N + H * V) * e + 8 * H)
        bytes_ += 12 * B * H * N * V
        flops += 18 * rows * H * N * V
    return {"bytes": bytes_, "flops": flops}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "gate": _exact_gate, "delta": _exact_delta}[case["op"]](s)


def _exact_norm(s):
    c = s["case"]
    D = c["dim"]
    x = s["x"].double().reshape(-1, D)
    on = torch.ones(x.shape[0], 1, dtype=torch.float64, device="cuda")
    if "batch" in c:
        lens = (s["offsets"][1:] - s["offsets"][:-1]).clamp(max=c["time"])
        on = (torch.arange(c["time"], device="cuda").expand(c["batch"], -1) < lens[:, None]).reshape(-1, 1).double()
    w, b = s["weight"].double(), s["bias"].double()
    mean = torch.einsum("nd->n", x)[:, None] / D
    var = torch.einsum("nd,nd->n", x - mean, x - mean)[:, None] / D
    hat = (x - mean) / torch.sqrt(var + EPS)
    out = dict(y=((hat * w + b) * on).view(s["x"].shape))
    if c["mode"] == "train":
        dy = s["grad_y"].double().reshape(-1, D) * on
        g = dy * w
        along = torch.einsum("nd,nd->n", g, hat)[:, None] / D
        gx = (g - torch.einsum("nd->n", g)[:, None] / D - hat * along) / torch.sqrt(var + EPS)
        out.update(grad_x=(gx * on).view(s["x"].shape), grad_weight=torch.einsum("nd,nd->d", dy, hat),
                   grad_bias=torch.einsum("nd->d", dy))
    return out


def _exact_gate(s):
    c = s["case"]
    T, K, E = c["tokens"], c["top_k"], c["experts"]
    held = torch.arange(T, device="cuda") if s["live"] is None else torch.nonzero(s["live"])[:, 0]
    x = s["logits"][held].double()
    n = held.numel()
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    left, picks = x.clone(), []
    for _ in range(K):          # the largest that is left, the lowest expert of equals
        best = left.amax(1, keepdim=True)
        place = torch.where(left == best, torch.arange(E, device="cuda"), E).amin(1, keepdim=True)
        picks.append(place)
        left.scatter_(1, place, -torch.inf)
    ids = torch.cat(picks, 1)
    counts = torch.bincount(ids.reshape(-1), minlength=E).double()
    w = p.gather(1, ids)
    if c["normalize"]:
        w = torch.softmax(x.gather(1, ids), 1)
    f = counts / max(n * K, 1)
    losses = torch.stack([E * (f * p.sum(0) / max(n, 1)).sum(), lse.square().sum() / max(n, 1)])
    weights = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    weights[held] = w
    out = dict(experts=None, weights=weights, counts=None, losses=losses)
    if c["mode"] == "train":
        gw = s["grad_weights"][held].double()
        gb, gz = s["grad_losses"].double()
        dp = (gb * E * f / max(n, 1)).expand(n, E).clone()
        dx = 2 * gz * lse[:, None] * p / max(n, 1)
        if c["normalize"]:
            dx.scatter_add_(1, ids, w * gw - w * torch.einsum("nk,nk->n", w, gw)[:, None])
        else:
            dp.scatter_add_(1, ids, gw)
        dx = dx + p * (dp - torch.einsum("ne,ne->n", p, dp)[:, None])
        out["grad_logits"] = torch.zeros(T, E, dtype=torch.float64, device="cuda")
        out["grad_logits"][held] = dx
    return out


def _exact_delta(s):
    """The recurrence position by position, and its adjoint from the last position to the first; the states are kept
    at every 64th position and found again between them."""
    c = s["case"]
    H, J, N = c["heads"], c["key_heads"], c["key_dim"]
    of = torch.arange(H, device="cuda") // (H // J)       # the key head of each head
    q, k = s["q"].double() * N ** -0.5, s["k"].double()
    v, a, b = s["v"].double(), torch.exp(s["decay"].double())[..., None], s["beta"].double()[..., None]
    if c["mode"] == "step":
        states, y = s["states"].double(), torch.zeros_like(v)
        held = torch.nonzero(s["rows"] >= 0)[:, 0]
        rows = s["rows"][held]
        S, kh = states[rows] * a[held, ..., None], k[held][:, of]
        S = S + torch.einsum("bhn,bhv->bhnv", kh, b[held] * (v[held] - torch.einsum("bhnv,bhn->bhv", S, kh)))
        y[held] = torch.einsum("bhnv,bhn->bhv", S, q[held][:, of])
        states[rows] = S
        return dict(y=y, states=states)
    B, T = c["batch"], c["time"]
    lens = (s["offsets"][1:] - s["offsets"][:-1]).clamp(max=T)
    on = (torch.arange(T, device="cuda").expand(B, T) < lens[:, None])[..., None, None]
    if T * B * H * N * c["value_dim"] > 3 << 32:
        return None
    on64 = on.double()
    a = torch.where(on, a, 1.0)
    b, k, q, v = b * on64, k * on64, q * on64, v * on64

    def step(S, t):
        kt = k[:, t, of]
        S = S * a[:, t, :, :, None]
        e = v[:, t] - torch.einsum("bhnv,bhn->bhv", S, kt)
        return S, kt, e, S + kt[..., None] * (b[:, t] * e)[:, :, None]
    S, kept, y = s["state"].double(), [], torch.zeros_like(v)
    for t in range(T):
        if t % 64 == 0:
            kept.append(S)
        S = step(S, t)[3]
        y[:, t] = torch.einsum("bhnv,bhn->bhv", S, q[:, t, of])
    out = dict(y=y, last=S)
    if c["mode"] == "forward":
        return out
    dy, dS = s["grad_y"].double() * on64, s["grad_last"].double()
    gq, gk, gv, ga, gb = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(a), torch.zeros_like(b)
    for first in range((T - 1) // 64 * 64, -1, -64):
        S, found = kept[first // 64], []
        for t in range(first, min(first + 64, T)):
            found.append((S,) + step(S, t))
            S = found[-1][4]
        for t in range(min(first + 64, T) - 1, first - 1, -1):
            before, faded, kt, e, S = found.pop()
            dS = dS + q[:, t, of][..., None] * dy[:, t][:, :, None]
            dk = torch.einsum("bhnv,bhv->bhn", dS, b[:, t] * e)
            along = torch.einsum("bhnv,bhn->bhv", dS, kt)
            gb[:, t] = (along * e).sum(-1, keepdim=True)
            de = b[:, t] * along
            gv[:, t] = de
            dk = dk - torch.einsum("bhnv,bhv->bhn", faded, de)
            gq[:, t].index_add_(1, of, torch.einsum("bhnv,bhv->bhn", S, dy[:, t]))
            gk[:, t].index_add_(1, of, dk)
            dS = dS - kt[..., None] * de[:, :, None]
            ga[:, t] = (dS * faded).sum((-1, -2))[..., None]
            dS = dS * a[:, t, :, :, None]
    out.update(grad_q=gq * N ** -0.5 * on64, grad_k=gk * on64, grad_v=gv, grad_decay=(ga * on64)[..., 0],
               grad_beta=(gb * on64)[..., 0], grad_state=dS)
    return out
