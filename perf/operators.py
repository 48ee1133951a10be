"""Workloads of the sequence, expert and optimizer operators: what is measured of
them, in plain torch (`own` false) and through the framework's calls (`own`
true).

  scan   gated linear recurrence over [batch, time, dim]: forward, forward and
         backward, or one token per session on state rows
  moe    tokens sorted by expert and back, weights applied, with the gradients
  adamw  one AdamW step over a list of tensors, states in 32 or 8 bits
"""
import math

import torch

own = False

DTYPE = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZE = {"float32": 4, "bfloat16": 2, "float16": 2}
BLOCK = 256          # elements that share one largest value in an 8-bit state
LR, BETA1, BETA2, EPS = 1e-4, 0.9, 0.999, 1e-8


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # serving: one new event for each of 192 sessions, their states among 5000
        dict(name="scan_step", op="scan", mode="step", batch=192, rows=5000, dim=256, dtype="bfloat16"),
        # serving: the first pass over a handful of new sessions, an odd width
        dict(name="scan_prefill_odd", op="scan", mode="forward", batch=5, time=333, min_len=1, dim=50,
             dtype="float16"),
        # training over the padded sequences of the benchmark's sequence workload
        # (batch 1024, lengths 200..1000 of 1000)
        dict(name="scan_sequences", op="scan", mode="train", batch=1024, time=1000, min_len=200, dim=64,
             dtype="float32"),
        # training over one very long history
        dict(name="scan_long", op="scan", mode="train", batch=1, time=131072, min_len=131072, dim=512,
             dtype="bfloat16"),
        # serving: eight tokens through sixteen experts
        dict(name="moe_decode", op="moe", mode="forward", tokens=8, top_k=2, experts=16, dim=256, align=1, drop=0.0,
             dtype="bfloat16"),
        # odd sizes: dropped choices, segments rounded up to 8 rows
        dict(name="moe_odd", op="moe", mode="train", tokens=5003, top_k=3, experts=37, dim=99, align=8, drop=0.05,
             dtype="float16"),
        # training a small tower in fp32
        dict(name="moe_tower", op="moe", mode="train", tokens=16384, top_k=2, experts=32, dim=512, align=1, drop=0.0,
             dtype="float32"),
        # training a wide layer, segments rounded up to the matrix tile
        dict(name="moe_large", op="moe", mode="train", tokens=131072, top_k=4, experts=128, dim=1024, align=128,
             drop=0.0, dtype="bfloat16"),
        # the dense weights of a small tower
        dict(name="adamw_small", op="adamw", tensors=18, elements=150_000, bits=32, dtype="float32", master=False),
        # a large tower in fp32
        dict(name="adamw_large", op="adamw", tensors=60, elements=128_000_000, bits=32, dtype="float32",
             master=False),
        # very many small tensors, bf16 weights, 8-bit states
        dict(name="adamw8_many", op="adamw", tensors=1500, elements=20_000_000, bits=8, dtype="bfloat16",
             master=False),
        # a large tower, bf16 weights with fp32 masters, 8-bit states
        dict(name="adamw8_large", op="adamw", tensors=60, elements=128_000_000, bits=8, dtype="bfloat16",
             master=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["scan", "moe", "adamw"])
    dtype = rng.choice(["float32", "bfloat16", "float16"])
    if op == "scan":
        mode = rng.choice(["step", "forward", "train", "train"])
        dim = _log(rng, 16, 1024)
        if rng.random() < 0.6:
            dim = max(16, dim // 8 * 8)
        if mode == "step":
            batch = _log(rng, 1, 16384)
            return dict(op=op, mode=mode, batch=batch, rows=batch + _log(rng, 1, 50000), dim=dim, dtype=dtype)
        budget = _log(rng, 20_000, 60_000_000)      # elements
        time = _log(rng, 1, min(131072, max(2, budget // dim)))
        batch = max(1, budget // dim // time)
        return dict(op=op, mode=mode, batch=batch, time=time, min_len=rng.choice([0, (time + 1) // 2, time]), dim=dim,
                    dtype=dtype)
    if op == "moe":
        mode = rng.choice(["forward", "train", "train"])
        dim = _log(rng, 16, 2048)
        if rng.random() < 0.6:
            dim = max(16, dim // 8 * 8)
        experts = _log(rng, 4, 512)
        top_k = rng.choice([1, 2, 4, 6, 8])
        top_k = min(top_k, experts)
        tokens = _log(rng, 1, max(2, min(200_000, 800_000_000 // (dim * top_k * SIZE[dtype]))))
        return dict(op=op, mode=mode, tokens=tokens, top_k=top_k, experts=experts, dim=dim,
                    align=rng.choice([1, 1, 8, 64]), drop=rng.choice([0.0, 0.0, 0.1]), dtype=dtype)
    elements = _log(rng, 20_000, 100_000_000)
    return dict(op=op, tensors=_log(rng, 1, min(1000, elements // 1000)), elements=elements, bits=rng.choice([8, 32]),
                dtype=dtype, master=dtype != "float32" and rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(gen, *shape, scale=1.0, shift=0.0, dtype=torch.float32):
    x = torch.empty(shape, dtype=torch.float32, device="cuda")
    return x.normal_(shift, scale, generator=gen).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"scan": _prepare_scan, "moe": _prepare_moe, "adamw": _prepare_adamw}[case["op"]](case, gen)


def _prepare_scan(case, gen):
    s = dict(case=case, plan=None)
    B, D, dt = case["batch"], case["dim"], DTYPE[case["dtype"]]
    if case["mode"] == "step":
        s["x"] = _randn(gen, B, D, dtype=dt)
        s["gate"] = _randn(gen, B, D, scale=1.5, shift=1.0, dtype=dt)
        # one more row than the calls are told of: the plain form writes there what has no row
        s["pool"] = _randn(gen, case["rows"] + 1, D)
        s["states"] = s["pool"][:-1]
        s["rows"] = torch.randperm(case["rows"], generator=gen, device="cuda")[:B].contiguous()
        if B > 8:
            s["rows"][5] = -1               # a session whose key has no row yet
    else:
        T = case["time"]
        s["x"] = _randn(gen, B, T, D, dtype=dt)
        s["gate"] = _randn(gen, B, T, D, scale=1.5, shift=1.0, dtype=dt)
        lens = torch.randint(case["min_len"], T + 1, (B,), generator=gen, device="cuda")
        s["offsets"] = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)
        s["state"] = _randn(gen, B, D)
        if case["mode"] == "train":
            s["grad_y"] = _randn(gen, B, T, D, dtype=dt)
            s["grad_last"] = _randn(gen, B, D)
    if own:     # the handle a program keeps between calls
        import sparse_lookup_gb300 as sl
        s["plan"] = sl.GatedScan(D, max_batch=B, max_len=case.get("time", 1))
    return s


def _moe_rows(case):
    """Rows of the expert-ordered arrays: every choice, and room to round each expert's segment up."""
    a = case["align"]
    return (case["tokens"] * case["top_k"] + case["experts"] * (a - 1) + a - 1) // a * a


def _prepare_moe(case, gen):
    s = dict(case=case, plan=None)
    T, K, E, D, dt = case["tokens"], case["top_k"], case["experts"], case["dim"], DTYPE[case["dtype"]]
    s["x"] = _randn(gen, T, D, dtype=dt)
    # router logits with a tilt, so that experts get unequal shares
    logits = _randn(gen, T, E) + _randn(gen, E, scale=0.7)
    top, ids = logits.topk(K, dim=1)
    s["weights"] = torch.softmax(top, 1)
    s["experts"] = ids.to(torch.int32)
    if case["drop"]:
        s["experts"][torch.rand(T, K, generator=gen, device="cuda") < case["drop"]] = -1
    s["ys"] = _randn(gen, _moe_rows(case), D, dtype=dt)           # what the experts answered
    if case["mode"] == "train":
        s["grad_y"] = _randn(gen, T, D, dtype=dt)
        s["grad_xs"] = _randn(gen, _moe_rows(case), D, dtype=dt)  # what came back through the experts
    if own:     # the handle a program keeps between calls
        import sparse_lookup_gb300 as sl
        s["plan"] = sl.ExpertRouter(E, K, max_tokens=T, align=case["align"])
    return s


def _tensor_sizes(case):
    """Elements of each tensor: a few wide matrices, vectors and odd sizes, the same for every seed."""
    n, total = case["tensors"], case["elements"]
    weight = [(1 + (i * 7919) % 97) ** 2 if i % 3 else 3 + i % 5 for i in range(n)]
    unit = total / sum(weight)
    return [max(1, int(w * unit) - i % 4) for i, w in enumerate(weight)]


def _prepare_adamw(case, gen):
    """Parameters, gradients and states as views of flat arrays in which every tensor starts at a multiple of BLOCK."""
    sizes, dt = _tensor_sizes(case), DTYPE[case["dtype"]]
    starts, n = [], 0
    for k in sizes:
        starts.append(n)
        n += (k + BLOCK - 1) // BLOCK * BLOCK
    sizes_d = torch.tensor(sizes, device="cuda")
    blocks = (sizes_d + BLOCK - 1) // BLOCK
    tensor_of = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), blocks)
    first = torch.repeat_interleave(torch.cumsum(blocks, 0) - blocks, blocks)
    left = sizes_d[tensor_of] - (torch.arange(n // BLOCK, device="cuda") - first) * BLOCK
    live = (torch.arange(BLOCK, device="cuda")[None] < left[:, None]).reshape(-1)

    def flat(scale, dtype=torch.float32):
        return (_randn(gen, n, scale=scale) * live).to(dtype)

    s = dict(case=case, plan=None, step=100)
    decay = [0.0 if i % 3 == 0 else 0.01 for i in range(len(sizes))]       # vectors do not decay
    s["decay"] = torch.tensor(decay, device="cuda")[tensor_of]             # one per block
    master = flat(0.05)
    s["p"] = master.to(dt) if dt != torch.float32 else master
    s["master"] = master if case["master"] else None
    # gradients of very different sizes from tensor to tensor
    size = torch.exp(_randn(gen, len(sizes), scale=2.0, shift=-5.0))[tensor_of].repeat_interleave(BLOCK)
    g = flat(1.0) * size
    s["g"] = g.to(dt)
    m, v = 0.3 * size * flat(1.0), size * size * flat(1.0).square() * 0.7
    if case["bits"] == 8:
        s["seed"] = int(torch.randint(1, 1 << 30, (1,), generator=gen, device="cuda"))
        zero = torch.zeros(n, dtype=torch.int32, device="cuda")
        s["m"], s["m_top"] = _encode(m, zero, True)
        s["v"], s["v_top"] = _encode(v, zero, False)
    else:
        s["m"], s["v"] = m, v
    if own:     # the handle a program keeps between calls
        import sparse_lookup_gb300 as sl

        def views(x):
            return None if x is None else [x[a:a + k] for a, k in zip(starts, sizes)]

        def block_views(x):
            return [x[a // BLOCK:(a + k + BLOCK - 1) // BLOCK] for a, k in zip(starts, sizes)]
        tops = dict(m_top=block_views(s["m_top"]), v_top=block_views(s["v_top"])) if case["bits"] == 8 else {}
        s["plan"] = sl.AdamW(views(s["p"]), views(s["g"]), masters=views(s["master"]), weight_decay=decay,
                             betas=(BETA1, BETA2), eps=EPS, state_bits=case["bits"], m=views(s["m"]),
                             v=views(s["v"]), seed=s.get("seed", 0), step=s["step"], **tops)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return {"scan": _run_scan, "moe": _run_moe, "adamw": _run_adamw}[state["case"]["op"]](state)


def _run_scan(s):
    mode = s["case"]["mode"]
    if mode == "step":
        if own:
            return dict(y=s["plan"].step(s["x"], s["gate"], s["rows"], s["states"]), states=s["states"])
        live = (s["rows"] >= 0)[:, None]
        rows = s["rows"].clamp(min=0)
        old = s["states"][rows]
        a = torch.sigmoid(s["gate"].float())
        new = a * old + torch.sigmoid(-s["gate"].float()) * s["x"].float()
        s["pool"][torch.where(live[:, 0], rows, s["states"].shape[0])] = new
        return dict(y=(new * live).to(s["x"].dtype), states=s["states"])
    if own:
        y, last = s["plan"].forward(s["x"], s["gate"], offsets=s["offsets"], state=s["state"])
        if mode == "forward":
            return dict(y=y, last=last)
        gx, gg, gs = s["plan"].backward(s["x"], s["gate"], y, s["grad_y"], offsets=s["offsets"], state=s["state"],
                                        grad_last=s["grad_last"])
        return dict(y=y, last=last, grad_x=gx, grad_gate=gg, grad_state=gs)
    T = s["x"].shape[1]
    lens = s["offsets"].diff().clamp(max=T)
    live = torch.arange(T, device="cuda")[None, :, None] < lens[:, None, None]
    x, f = s["x"].float(), s["gate"].float()
    # a position past the end keeps the state: a = 1, b = 0
    a = torch.where(live, torch.sigmoid(f), 1.0)
    na = torch.where(live, torch.sigmoid(-f), 0.0)
    h = _scan(a, torch.cat([na[:, :1] * x[:, :1] + a[:, :1] * s["state"][:, None], na[:, 1:] * x[:, 1:]], 1))
    last = h[:, -1]
    out = dict(y=(h * live).to(s["x"].dtype), last=last)
    if mode == "forward":
        return out
    dy = torch.where(live, s["grad_y"].float(), 0.0)
    dy[:, -1] += s["grad_last"]
    # G_t = dy_t + a_{t+1} G_{t+1}, as a scan over reversed time
    G = _scan(torch.cat([torch.ones_like(a[:, :1]), a[:, 1:].flip(1)], 1), dy.flip(1)).flip(1)
    before = torch.cat([s["state"][:, None], h[:, :-1]], 1)
    out["grad_x"] = (na * G).to(s["x"].dtype)
    out["grad_gate"] = (a * na * (before - x) * G).to(s["x"].dtype)
    out["grad_state"] = a[:, 0] * G[:, 0]
    return out


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1 (h_{-1} = 0), in log depth: neighbours are joined to pairs, the pairs'
    states found first, the odd ones out filled in."""
    n = a.shape[1]
    if n == 1:
        return b
    m = n // 2
    ae, ao, be, bo = a[:, 0:2 * m:2], a[:, 1::2], b[:, 0:2 * m:2], b[:, 1::2]
    odd = _scan(ae * ao, ao * be + bo)
    h = torch.empty_like(b)
    h[:, 1::2] = odd
    h[:, 0] = b[:, 0]
    h[:, 2::2] = a[:, 2::2] * odd[:, :(n - 1) // 2] + b[:, 2::2]
    return h


def _run_moe(s):
    c = s["case"]
    train = c["mode"] == "train"
    if own:
        r = s["plan"].route(s["experts"])
        out = dict(offsets=r.offsets, counts=r.counts, pos=r.pos, src=r.src)
        out["xs"] = s["plan"].dispatch(s["x"], r)
        out["y"] = s["plan"].combine(s["ys"], s["weights"], r)
        if train:
            out["grad_ys"], out["grad_weights"] = s["plan"].combine_backward(s["grad_y"], s["ys"], s["weights"], r)
            out["grad_x"] = s["plan"].dispatch_backward(s["grad_xs"], r)
        return out
    T, K, E, align, cap = c["tokens"], c["top_k"], c["experts"], c["align"], _moe_rows(c)
    dt = s["x"].dtype
    ids = s["experts"].reshape(-1).long()
    ids = torch.where((ids >= 0) & (ids < E), ids, E)
    order = torch.argsort(ids, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda").index_add_(0, ids, torch.ones_like(ids))
    padded = (counts[:E] + align - 1) // align * align
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    by = ids[order]
    row = offsets[by] + torch.arange(T * K, device="cuda") - (counts.cumsum(0) - counts)[by]
    live = by < E
    pos = torch.empty_like(ids)
    pos[order] = torch.where(live, row, -1)
    src = torch.full((cap + 1,), -1, dtype=torch.int64, device="cuda")
    src[torch.where(live, row, cap)] = torch.where(live, order, -1)
    src = src[:cap]
    pos = pos.view(T, K)
    out = dict(offsets=offsets.int(), counts=counts[:E].int(), pos=pos.int(), src=src.int())
    token, used = src.clamp(min=0) // K, (src >= 0)[:, None]
    out["xs"] = torch.where(used, s["x"][token], 0.0)
    kept, at = (pos >= 0)[..., None], pos.clamp(min=0)
    w = s["weights"]
    ys = torch.where(kept, s["ys"][at], 0.0).float()                   # [T, K, D]
    out["y"] = (ys * w[..., None]).sum(1).to(dt)
    if train:
        dy = s["grad_y"].float()
        ws = torch.where(used[:, 0], w.reshape(-1)[src.clamp(min=0)], 0.0)
        out["grad_ys"] = (dy[token] * ws[:, None]).to(dt)
        out["grad_weights"] = (ys * dy[:, None]).sum(2)
        out["grad_x"] = torch.where(kept, s["grad_xs"][at], 0.0).float().sum(1).to(dt)
    return out


def _run_adamw(s):
    c = s["case"]
    if own:
        s["plan"].step(LR)
        m, v = s["plan"].states() if c["bits"] == 8 else (s["m"], s["v"])
    else:
        s["step"] += 1
        t = s["step"]
        eight = c["bits"] == 8
        g = s["g"].float()
        m = _decode(s["m"], s["m_top"], True) if eight else s["m"]
        v = _decode(s["v"], s["v_top"], False) if eight else s["v"]
        m = m * BETA1 + g * (1 - BETA1)
        v = v * BETA2 + (g * g) * (1 - BETA2)
        p = s["p"].float() if s["master"] is None else s["master"]
        decay = s["decay"].repeat_interleave(BLOCK)
        update = (m * (1 / (1 - BETA1 ** t))) / ((v * (1 / (1 - BETA2 ** t))).sqrt() + EPS)
        p = p - (p * decay) * LR - update * LR
        if s["master"] is not None:
            s["master"].copy_(p)
        s["p"].copy_(p)
        if eight:
            noise = _noise(m.numel(), s["seed"], t)
            code, top = _encode(m, noise, True)
            s["m"].copy_(code), s["m_top"].copy_(top)
            m = _decode(code, top, True).bfloat16()
            code, top = _encode(v, noise, False)
            s["v"].copy_(code), s["v_top"].copy_(top)
            v = _decode(code, top, False).bfloat16()
        else:
            s["m"].copy_(m), s["v"].copy_(v)
            m, v = s["m"], s["v"]
    out = dict(p=s["p"], m=m, v=v)
    if s["master"] is not None:
        out["master"] = s["master"]
    return out


# The 8-bit states.  A value's place on the grid is its fp32 pattern without the sign, shifted right by 20: exponent and
# three bits of the fraction.  A block of 256 holds `top`, the place of its largest magnitude rounded up; a code counts
# places up from top - 127 (m: 7 bits and the sign) or top - 255 (v: 8 bits); code 0 is zero.  Places are rounded up
# or down by 16 bits of noise, so that a state's small steps are kept on average.  Every value that a code stands for has
# three bits of fraction: bf16 holds it exactly.

def _encode(x, noise, signed):
    bits = x.view(torch.int32)
    mag = bits & 0x7FFFFFFF
    mag = torch.where(mag < 0x7F800000, mag, 0)
    top = (mag.view(-1, BLOCK).amax(1) + 0xFFFFF) >> 20
    levels = 127 if signed else 255
    base = (top - levels).clamp(min=0).repeat_interleave(BLOCK)
    code = (((mag + (noise << 4)) >> 20) - base).clamp(min=0)
    if signed:
        code = code | ((bits >> 24) & 0x80)
    return code.to(torch.uint8), top.to(torch.int16)


def _decode(code, top, signed):
    levels = 127 if signed else 255
    base = (top.int() - levels).clamp(min=0).repeat_interleave(BLOCK)
    c = code.int()
    mag = c & levels
    bits = torch.where(mag > 0, (mag + base) << 20, 0)
    if signed:
        bits = bits | ((c & 0x80) << 24)
    return bits.view(torch.float32)


def _wrap(x):
    x &= (1 << 64) - 1
    return x - (1 << 64) if x >> 63 else x


def _mix(z):
    """One SplitMix64 output for each state in z (int64, wrapping)."""
    z = z + _wrap(0x9E3779B97F4A7C15)
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * _wrap(0xBF58476D1CE4E5B9)
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * _wrap(0x94D049BB133111EB)
    return z ^ ((z >> 31) & ((1 << 33) - 1))


def _noise(n, seed, step):
    """16 bits for each of n elements: four from each SplitMix64 output of the group of four's number, offset by the
    output for seed and step."""
    key = _mix(torch.tensor([(seed << 32) + step], device="cuda"))
    z = _mix(torch.arange(n // 4, device="cuda") + key)
    return ((z[:, None] >> torch.tensor([0, 16, 32, 48], device="cuda")) & 0xFFFF).reshape(-1).to(torch.int32)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "scan":
        e, B, D = SIZE[case["dtype"]], case["batch"], case["dim"]
        if case["mode"] == "step":      # x, gate, y; the state read and written
            return {"bytes": B * D * (3 * e + 8) + 8 * B, "flops": 6 * B * D}
        whole = B * case["time"] * D
        live = B * (case["min_len"] + case["time"]) / 2 * D
        bytes_, flops = live * 2 * e + whole * e + 8 * B * D, 6 * live
        if case["mode"] == "train":     # x, gate and grad_y of the live positions; both gradients of all
            bytes_ += live * 3 * e + whole * 2 * e + 12 * B * D
            flops += 14 * live
        return {"bytes": bytes_, "flops": flops}
    if case["op"] == "moe":
        e, T, K, D, R = SIZE[case["dtype"]], case["tokens"], case["top_k"], case["dim"], _moe_rows(case)
        rows = T * K * (1 - case["drop"])
        index = 8 * T * K + 4 * R + 8 * case["experts"]
        bytes_ = index + (T * D + R * D) * e                # route; dispatch
        bytes_ += (rows * D + T * D) * e + 8 * T * K        # combine
        flops = 2 * rows * D
        if case["mode"] == "train":
            bytes_ += (T * D + rows * D + R * D) * e + 12 * T * K      # combine, backward
            bytes_ += (rows * D + T * D) * e + 4 * T * K               # dispatch, backward
            flops += 4 * rows * D
        return {"bytes": bytes_, "flops": flops}
    n = sum(_tensor_sizes(case))
    e = SIZE[case["dtype"]]
    each = e + (8 + e if case["master"] else 2 * e)          # gradient; weights read and written, or masters
    if case["bits"] == 8:
        each += 4 + 6 + 16 / BLOCK      # both states read and written; what they stand for written out in bf16
    else:
        each += 16
    return {"bytes": n * each, "flops": 14 * n}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"scan": _exact_scan, "moe": _exact_moe, "adamw": _exact_adamw}[case["op"]](s)


def _exact_scan(s):
    c = s["case"]
    x, f = s["x"].double(), s["gate"].double()
    a, na = 1 / (1 + torch.exp(-f)), 1 / (1 + torch.exp(f))
    if c["mode"] == "step":
        states, y = s["states"].double(), torch.zeros_like(x)
        held = torch.nonzero(s["rows"] >= 0)[:, 0]
        rows = s["rows"][held]
        y[held] = a[held] * states[rows] + na[held] * x[held]
        states[rows] = y[held]
        return dict(y=y, states=states)
    T = c["time"]
    lens = (s["offsets"][1:] - s["offsets"][:-1]).clamp(max=T)
    on = torch.arange(T, device="cuda").expand(c["batch"], T) < lens[:, None]
    on = on[..., None].double()
    a, na = a * on + (1 - on), na * on
    start = s["state"].double()
    h = _one_by_one(a, na * x, start)
    out = dict(y=h * on, last=h[:, -1])
    if c["mode"] == "forward":
        return out
    # e_t = a_t (dy_t + e_{t+1}): what position t passes on to the one before
    dy = s["grad_y"].double() * on
    e = _one_by_one(a.flip(1), (a * dy).flip(1), s["grad_last"].double()).flip(1)
    grad = dy + torch.cat([e[:, 1:], s["grad_last"].double()[:, None]], 1)
    before = torch.cat([start[:, None], h[:, :-1]], 1)
    out.update(grad_x=grad * na, grad_gate=grad * (before - x) * a * na, grad_state=e[:, 0])
    return out


def _one_by_one(a, b, state):
    """h_t = a_t h_{t-1} + b_t from `state`, position by position: in about sqrt(T) stretches at once from zero, then
    from stretch to stretch."""
    B, T, D = a.shape
    L = math.isqrt(T - 1) + 1
    N = (T + L - 1) // L
    pad = N * L - T
    a = torch.cat([a, a.new_ones(B, pad, D)], 1).view(B, N, L, D)
    b = torch.cat([b, b.new_zeros(B, pad, D)], 1).view(B, N, L, D)
    h, p = torch.empty_like(b), torch.empty_like(a)
    h[:, :, 0], p[:, :, 0] = b[:, :, 0], a[:, :, 0]
    for t in range(1, L):
        h[:, :, t] = a[:, :, t] * h[:, :, t - 1] + b[:, :, t]
        p[:, :, t] = a[:, :, t] * p[:, :, t - 1]
    for n in range(N):
        h[:, n] += p[:, n] * state[:, None]
        state = h[:, n, -1]
    return h.view(B, N * L, D)[:, :T]


def _exact_moe(s):
    c = s["case"]
    T, K, E, align, cap = c["tokens"], c["top_k"], c["experts"], c["align"], _moe_rows(c)
    flat = s["experts"].reshape(-1)
    pos = torch.full((T * K,), -1, dtype=torch.int64, device="cuda")
    start = 0
    for e in range(E):          # one expert after another, its choices in order
        mine = torch.nonzero(flat == e)[:, 0]
        pos[mine] = start + torch.arange(mine.numel(), device="cuda")
        start += (mine.numel() + align - 1) // align * align
    pos = pos.view(T, K)
    x, ys, w = s["x"].double(), s["ys"], s["weights"].double()
    out = dict(offsets=None, counts=None, pos=None, src=None)
    out["xs"], out["y"] = x.new_zeros(cap, x.shape[1]), torch.zeros_like(x)
    train = c["mode"] == "train"
    if train:
        dy = s["grad_y"].double()
        out.update(grad_ys=torch.zeros_like(out["xs"]), grad_weights=torch.zeros_like(w), grad_x=torch.zeros_like(x))
    for k in range(K):
        held = torch.nonzero(pos[:, k] >= 0)[:, 0]
        at = pos[held, k]
        out["xs"][at] = x[held]
        out["y"][held] += w[held, k, None] * ys[at].double()
        if train:
            out["grad_ys"][at] = w[held, k, None] * dy[held]
            out["grad_weights"][held, k] = torch.einsum("nd,nd->n", dy[held], ys[at].double())
            out["grad_x"][held] += s["grad_xs"][at].double()
    return out


def _exact_adamw(s):
    c = s["case"]
    t = s["step"] + 1
    eight = c["bits"] == 8
    levels = dict(m=127, v=255)

    def stands_for(code, top, k):
        place = (code.long() & k) + (top.long() - k).clamp(min=0).repeat_interleave(BLOCK)
        value = torch.ldexp(1 + (place % 8).double() / 8, place // 8 - 127)
        value = torch.where((code.long() & k) > 0, value, 0.0)
        return torch.where(code >= 128, -value, value) if k == 127 else value

    def held(value, noise, k):
        frac, exponent = torch.frexp(value.abs())                # |value| = frac 2^exponent, frac in [1/2, 1)
        place = (exponent + 126).double() * 8 + (2 * frac - 1) * 8
        place = torch.where(value == 0, 0.0, place)
        top = torch.ceil(place.view(-1, BLOCK).amax(1))
        base = (top - k).clamp(min=0).repeat_interleave(BLOCK)
        place = torch.floor(place + noise.double() / 65536)
        out = torch.ldexp(1 + (place % 8) / 8, (place // 8 - 127).long())
        return torch.where(place > base, out, 0.0) * torch.sign(value)

    g = s["g"].double()
    m = stands_for(s["m"], s["m_top"], levels["m"]) if eight else s["m"].double()
    v = stands_for(s["v"], s["v_top"], levels["v"]) if eight else s["v"].double()
    m.lerp_(g, 1 - BETA1)
    v.lerp_(g * g, 1 - BETA2)
    p = (s["p"] if s["master"] is None else s["master"]).double()
    decay = s["decay"].double().repeat_interleave(BLOCK)
    p = p * (1 - LR * decay) - LR * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    out = dict(p=p, m=m, v=v)
    if eight:
        i = torch.arange(m.numel() // 4, device="cuda")
        z = _mix(i + int(_mix(torch.tensor([(s["seed"] << 32) + t]))[0]))
        noise = torch.stack([(z >> k) & 0xFFFF for k in (0, 16, 32, 48)], 1).reshape(-1)
        out["m"], out["v"] = held(m, noise, levels["m"]), held(v, noise, levels["v"])
    if s["master"] is not None:
        out["master"] = p
    return out
