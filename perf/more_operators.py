"""Cases, plain forms and exact values of two sets of operators: the gated linear recurrence (forward,
training step, single-token decode) and the norm of queries and keys with the rotation of their
positions (forward, training step).

Gated linear recurrence, per channel of x [B, T, D] or of packed sequences, with an fp32 state h:

    gates given:   h_t = exp(g_t) h_{t-1} + x_t,
    fused gates:   log a_t = -c softplus(lam) sigmoid(r_t),
                   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t.

Norm and rotation of each head of q [B, T, Hq, K] and k [B, T, Hk, K]: n = x / sqrt(mean(x^2) + eps) * w
(or x / sqrt(sum(x^2) + eps)), then the pairs j < R / 2 of the first R dims turn by the angle
pos[axis(j)] * inv_freq[j]; a pair is (j, j + R / 2), or (2 j, 2 j + 1) interleaved.
"""
import math

import torch

own = False

BLOCK = 256      # tokens of a block in the plain scan
EPS = 1e-6
C_GATE = 8.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a short prompt in fp32 (a test, a small model): the call's latency
        dict(name="lr_fwd_tiny_fp32", op="lr_fwd", B=1, T=256, D=256, gates="given", dtype="fp32",
             state="given"),
        # one long prompt: the sequence axis is what there is to split
        dict(name="lr_fwd_one_32768_bf16", op="lr_fwd", B=1, T=32768, D=2048, gates="given",
             dtype="bf16", state="given"),
        # prefill of 32 packed prompts of 100 to 4096 tokens, states in a 64-slot cache
        dict(name="lr_fwd_packed32_fused_bf16", op="lr_fwd", num_seqs=32, min_len=100, max_len=4096,
             D=4096, gates="fused", dtype="bf16", state="slots", num_slots=64),
        # a long-context training batch's forward
        dict(name="lr_fwd_4x32768_fused_bf16", op="lr_fwd", B=4, T=32768, D=4096, gates="fused",
             dtype="bf16", state="none"),
        # a training step on a few odd packed sequences in fp32, an odd width
        dict(name="lr_train_packed5_fp32", op="lr_train", num_seqs=5, min_len=1, max_len=1777, D=333,
             gates="given", dtype="fp32", state="given"),
        # a training step of a layer
        dict(name="lr_train_2x8192_fused_bf16", op="lr_train", B=2, T=8192, D=4096, gates="fused",
             dtype="bf16", state="none"),
        # a serving batch's next tokens, a tenth of it padding, on a 512-slot cache
        dict(name="lr_decode_256_fused_bf16", op="lr_decode", n=256, num_slots=512, pad=0.1, D=4096,
             gates="fused", dtype="bf16"),
        # a decode step of 256 requests, q and k slices of one projection
        dict(name="qk_fwd_256_bf16", op="qk_fwd", B=256, T=1, Hq=16, Hk=2, K=128, R=128, axes=1,
             norm="rms", pairs="halves", sliced=True, max_pos=131072, dtype="bf16"),
        # a long-context batch in front of linear attention
        dict(name="qk_fwd_4x32768_bf16", op="qk_fwd", B=4, T=32768, Hq=16, Hk=16, K=128, R=128, axes=1,
             norm="l2", pairs="halves", sliced=False, max_pos=32768, dtype="bf16"),
        # tokens of a video, three axes, pairs next to each other, odd count
        dict(name="qk_fwd_video_2x9731_bf16", op="qk_fwd", B=2, T=9731, Hq=12, Hk=12, K=128, R=128,
             axes=3, norm="rms", pairs="interleaved", sliced=True, max_pos=4096, dtype="bf16"),
        # a training step of a layer with grouped heads, q and k slices of one projection
        dict(name="qk_train_2x8192_bf16", op="qk_train", B=2, T=8192, Hq=32, Hk=8, K=128, R=128, axes=1,
             norm="rms", pairs="halves", sliced=True, max_pos=8192, dtype="bf16"),
        # a training step in fp32 on heads of 80 of which half turn
        dict(name="qk_train_3x1213_fp32", op="qk_train", B=3, T=1213, Hq=6, Hk=2, K=80, R=40, axes=2,
             norm="rms", pairs="halves", sliced=False, max_pos=1 << 20, dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lr_fwd", "lr_fwd", "lr_train", "lr_decode", "qk_fwd", "qk_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    # elements: fp32 up to 1/4, a training step up to 1/4 of the largest listed forward
    most = (1 << 29) // (4 if dtype == "fp32" else 1) // (4 if op.endswith("train") else 1)
    if op.startswith("lr_"):
        D = 16 * _log_int(rng, 1, 512) if rng.random() < 0.7 else _log_int(rng, 1, 6000)
        c = dict(op=op, D=D, gates=rng.choice(["given", "fused"]), dtype=dtype)
        if op == "lr_decode":
            n = _log_int(rng, 1, 2048)
            return dict(c, n=n, num_slots=n + rng.randint(0, n), pad=rng.choice([0.0, 0.1, 0.3]))
        if rng.random() < 0.5:
            num = _log_int(rng, 1, 300)
            hi = _log_int(rng, 2, max(2, min(32768, most // (D * num))))
            return dict(c, num_seqs=num, min_len=rng.randint(0, hi // 2), max_len=hi,
                        state=rng.choice(["none", "given"] + (["slots"] if op == "lr_fwd" else [])),
                        num_slots=num + rng.randint(0, 16))
        B = rng.choice([1, 1, 2, 3, 4, 16])
        T = _log_int(rng, 1, max(1, min(65536, most // (D * B))))
        return dict(c, B=B, T=T, state=rng.choice(["none", "given"]))
    K = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
    R = rng.choice([K, K, K // 2, 0 if K < 64 else K // 4])
    Hk = rng.choice([1, 2, 3, 4, 8, 16])
    Hq = Hk * rng.choice([1, 2, 4, 5])
    B = rng.choice([1, 2, 3, 8])
    T = _log_int(rng, 1, max(1, min(65536, most // (B * (Hq + Hk) * K))))
    return dict(op=op, B=B, T=T, Hq=Hq, Hk=Hk, K=K, R=R, axes=rng.choice([1, 1, 2, 3]) if R >= 6 else 1,
                norm=rng.choice(["rms", "rms", "l2", "none"]), pairs=rng.choice(["halves", "interleaved"]),
                sliced=rng.random() < 0.5, max_pos=_log_int(rng, max(64, T), 1 << 20), dtype=dtype)


# ---------------------------------------------------------------- inputs

def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case, seed):
    """The same lengths for every seed (the packed token count is the case's), in another order.
    Empty sequences are among them where min_len is 0; an empty batch is not."""
    g = torch.Generator().manual_seed(7919 * case["num_seqs"] + case["max_len"])
    n = torch.randint(case["min_len"], case["max_len"] + 1, (case["num_seqs"],), generator=g)
    n[0] = max(1, int(n[0]))
    order = torch.randperm(case["num_seqs"], generator=torch.Generator().manual_seed(int(seed)))
    return n[order].tolist()


def _sections(case):
    """How the R / 2 pairs are shared out over the axes, the first axis the smallest share."""
    pairs, A = case["R"] // 2, case["axes"]
    if A == 1:
        return None
    first = pairs // 4 if A == 3 else pairs // 2
    rest = pairs - first
    return (first, rest) if A == 2 else (first, rest // 2, rest - rest // 2)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = _dt(case)

    def rn(*shape, std=1.0, mean=0.0, dtype=dt):
        x = torch.randn(*shape, generator=gen, device=dev)
        return (x * std + mean).to(dtype)

    s = dict(case=case)
    if case["op"].startswith("lr_"):
        D = case["D"]
        if case["op"] == "lr_decode":
            lead, tokens = (case["n"],), case["n"]
            slots = case["num_slots"]
            s["cache"] = rn(slots, D, dtype=torch.float32)
            idx = torch.randperm(slots, generator=gen, device=dev)[:tokens].to(torch.int32)
            idx[torch.randperm(tokens, generator=gen, device=dev)[: int(round(case["pad"] * tokens))]] = -1
            s["idx"] = idx
        else:
            if "num_seqs" in case:
                s["lens"] = _lengths(case, seed)
                lead = (1, sum(s["lens"]))
            else:
                s["lens"] = [case["T"]] * case["B"]
                lead = (case["B"], case["T"])
            cu = [0]
            for n in s["lens"]:
                cu.append(cu[-1] + n)
            cu = torch.tensor(cu, dtype=torch.int32, device=dev)
            s["cu"] = cu if "num_seqs" in case else None
            # where sequences that have tokens start and end, and which they are
            alive = [n for n, m in enumerate(s["lens"]) if m > 0]
            s["alive"] = torch.tensor(alive, dtype=torch.int64, device=dev)
            s["first"] = cu[:-1].long()[s["alive"]]
            s["last"] = cu[1:].long()[s["alive"]] - 1
            N = len(s["lens"])
            s["h0"] = s["idx"] = None
            if case["state"] == "given":
                s["h0"] = rn(N, D, dtype=torch.float32)
            elif case["state"] == "slots":
                s["h0"] = rn(case["num_slots"], D, dtype=torch.float32)
                s["idx"] = torch.randperm(case["num_slots"], generator=gen, device=dev)[:N].to(torch.int32)
            if case["op"] == "lr_train":
                s["dh"] = rn(*lead, D)
                s["dfin"] = rn(N, D, dtype=torch.float32) if s["h0"] is not None else None
        s["x"] = rn(*lead, D)
        if case["gates"] == "given":       # decays from a few tokens to a few thousand
            s["g"] = (-torch.exp(rn(*lead, D, std=1.5, mean=-4.0, dtype=torch.float32))).to(dt)
        else:                              # a between 0.9 and 0.999 for a fully open gate
            s["r"], s["i"] = rn(*lead, D), rn(*lead, D)
            u = torch.rand(D, generator=gen, device=dev) * 0.099 + 0.9
            s["lam"] = torch.log(torch.expm1(-torch.log(u) / C_GATE))
        return s
    B, T, Hq, Hk, K = case["B"], case["T"], case["Hq"], case["Hk"], case["K"]
    if case["sliced"]:      # q, k, v from one projection
        both = rn(B, T, Hq + 2 * Hk, K, std=1.3)
        s["q"], s["k"] = both[:, :, :Hq], both[:, :, Hq:Hq + Hk]
    else:
        s["q"], s["k"] = rn(B, T, Hq, K, std=1.3), rn(B, T, Hk, K, std=1.3)
    s["wq"] = s["wk"] = None
    if case["norm"] == "rms":
        s["wq"] = rn(K, std=0.2, mean=1.0, dtype=torch.float32)
        s["wk"] = rn(K, std=0.2, mean=1.0, dtype=torch.float32)
    j = torch.arange(case["R"] // 2, device=dev, dtype=torch.float64)
    s["inv_freq"] = (10000.0 ** (-2 * j / max(case["R"], 1))).float()
    A = case["axes"]
    if A == 1:              # rows that start somewhere in a long context
        start = torch.randint(0, max(1, case["max_pos"] - T + 1), (B, 1), generator=gen, device=dev)
        pos = start + torch.arange(T, device=dev)
    else:                   # time, height, width of each token
        pos = torch.randint(0, case["max_pos"], (A, B, T), generator=gen, device=dev)
    s["pos"] = pos.to(torch.int32)
    if case["op"] == "qk_train":
        s["dq"], s["dk"] = rn(B, T, Hq, K), rn(B, T, Hk, K)
    return s


# ---------------------------------------------------------------- plain forms (fp32)

def _scan(a, b):
    """y_t = a_t y_{t-1} + b_t along dim 1 of [N, T, D], from zero: doubling inside blocks, the blocks'
    ends likewise, then every block from the one before it."""
    N, T, D = a.shape
    if T > BLOCK:
        pad = -T % BLOCK
        if pad:
            a, b = (torch.nn.functional.pad(t, (0, 0, 0, pad)) for t in (a, b))
        nb = (T + pad) // BLOCK
        a, b = (t.reshape(N * nb, BLOCK, D) for t in (a, b))
    a, b = a.clone(), b.clone()
    step = 1
    while step < a.shape[1]:
        b[:, step:] += a[:, step:] * b[:, :-step].clone()
        a[:, step:] *= a[:, :-step].clone()
        step *= 2
    if T <= BLOCK:
        return b
    ends = _scan(a[:, -1].reshape(N, nb, D), b[:, -1].reshape(N, nb, D))
    a, b = a.view(N, nb, BLOCK, D), b.view(N, nb, BLOCK, D)
    b[:, 1:] += a[:, 1:] * ends[:, :-1, None]
    return b.view(N, nb * BLOCK, D)[:, :T]


def _gates(s):
    """a_t and what is added to the state, both fp32, and what the gradients need of the way there."""
    x = s["x"].float()
    if s["case"]["gates"] == "given":
        return torch.exp(s["g"].float()), x, None
    sr, si = torch.sigmoid(s["r"].float()), torch.sigmoid(s["i"].float())
    la = (-C_GATE * torch.nn.functional.softplus(s["lam"])) * sr
    sq = torch.sqrt(-torch.expm1(2 * la))
    return torch.exp(la), sq * si * x, (x, sr, si, la, sq)


def _plain_lr(s, train):
    c = s["case"]
    dt, D, shape = _dt(c), c["D"], s["x"].shape
    flat = lambda t: t.reshape(1, -1, D)
    a, b, way = _gates(s)
    a, b = flat(a), flat(b)
    first, last, alive = s["first"], s["last"], s["alive"]
    start, kept, bb = None, a.clone(), b.clone()
    if s["h0"] is not None:
        start = s["h0"] if s["idx"] is None else s["h0"][s["idx"].long()]
        bb[0, first] += a[0, first] * start[alive]
    kept[0, first] = 0.0
    h = _scan(kept, bb)
    fin = torch.zeros(len(s["lens"]), D, device=h.device) if start is None else start.clone()
    fin[alive] = h[0, last]
    y = h.view(shape).to(dt)
    if not train:
        if s["idx"] is not None:
            fin = s["h0"].index_copy_(0, s["idx"].long(), fin)
        return {"y": y, "state": fin}
    d = flat(s["dh"].float()).clone()
    if start is not None:
        d[0, last] += s["dfin"][alive]
    nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    nxt[0, last] = 0.0
    delta = _scan(nxt.flip(1), d.flip(1)).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    before[0, first] = 0.0 if start is None else start[alive]
    out = {"y": y}
    if start is not None:
        out["state"] = fin
        dh0 = s["dfin"].clone()
        dh0[alive] = a[0, first] * delta[0, first]
        out["dh0"] = dh0
    if way is None:
        out["dx"] = delta.view(shape).to(dt)
        out["dg"] = (delta * a * before).view(shape).to(dt)
        return out
    x, sr, si, la, sq = (flat(t) for t in way)
    dla = delta * a * (before - si * x * a / sq)
    out["dx"] = (delta * sq * si).view(shape).to(dt)
    out["di"] = (delta * sq * x * si * (1 - si)).view(shape).to(dt)
    out["dr"] = (dla * la * (1 - sr)).view(shape).to(dt)
    out["dlam"] = (dla * sr).sum((0, 1), dtype=torch.float64).float() * (-C_GATE * torch.sigmoid(s["lam"]))
    return out


def _plain_lr_decode(s):
    a, b, _ = _gates(s)
    on = (s["idx"] >= 0)[:, None]
    at = s["idx"].clamp(min=0).long()
    old = s["cache"][at]
    new = a * old + b
    s["cache"].index_add_(0, at, torch.where(on, new - old, 0.0))
    return {"y": torch.where(on, new, 0.0).to(_dt(s["case"])), "state": s["cache"]}


def _angles(s):
    """cos and sin [B, T, 1, R / 2] (angles of far positions need 64 bits)."""
    pos = s["pos"].double()
    if s["case"]["axes"] > 1:
        axis = torch.repeat_interleave(torch.arange(s["case"]["axes"], device=pos.device),
                                       torch.tensor(_sections(s["case"]), device=pos.device))
        phi = pos[axis].permute(1, 2, 0) * s["inv_freq"].double()
    else:
        phi = pos[..., None] * s["inv_freq"].double()
    phi = torch.remainder(phi, 2 * math.pi)[:, :, None]
    return torch.cos(phi).float(), torch.sin(phi).float()


def _turn(x, cos, sin, case):
    """The pairs of the first R dims by the angle, the rest as it is."""
    R = case["R"]
    if R == 0:
        return x
    if case["pairs"] == "halves":
        u, v = x[..., : R // 2], x[..., R // 2:R]
        return torch.cat([u * cos - v * sin, v * cos + u * sin, x[..., R:]], -1)
    u, v = x[..., 0:R:2], x[..., 1:R:2]
    return torch.cat([torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2), x[..., R:]], -1)


def _plain_qk(s, train):
    c = s["case"]
    dt, K = _dt(c), c["K"]
    cos, sin = _angles(s)
    out = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s["w" + n]
        inv = None
        if c["norm"] != "none":
            inv = torch.rsqrt(x.square().sum(-1, keepdim=True) / (K if c["norm"] == "rms" else 1) + EPS)
            xh = x * inv
        else:
            xh = x
        out[n] = _turn(xh if w is None else xh * w, cos, sin, c).to(dt)
        if train:
            d = _turn(s["d" + n].float(), cos, -sin, c)
            if w is not None:
                out["dw" + n] = (d * xh).sum((0, 1, 2))
                d = d * w
            if inv is not None:
                part = (d * xh).sum(-1, keepdim=True) / (K if c["norm"] == "rms" else 1)
                d = inv * (d - xh * part)
            out["d" + n] = d.to(dt)
    return out


# ---------------------------------------------------------------- the framework's calls

def _own_lr(s, gdn):
    c = s["case"]
    fused = c["gates"] == "fused"
    if c["op"] == "lr_fwd":
        kw = dict(initial_state=s["h0"], output_final_state=True, cu_seqlens=s["cu"], state_indices=s["idx"])
        if fused:
            y, fin = gdn.gated_linear_recurrence_fused_gates(s["x"], s["r"], s["i"], s["lam"], C_GATE, **kw)
        else:
            y, fin = gdn.gated_linear_recurrence(s["x"], s["g"], **kw)
        return {"y": y, "state": fin}
    if c["op"] == "lr_decode":
        if fused:
            y = gdn.gated_linear_recurrence_decode_fused_gates(s["x"], s["r"], s["i"], s["lam"], s["cache"],
                                                               s["idx"], C_GATE)
        else:
            y = gdn.gated_linear_recurrence_decode(s["x"], s["g"], s["cache"], s["idx"])
        return {"y": y, "state": s["cache"]}
    names = ["x", "r", "i", "lam"] if fused else ["x", "g"]
    leaves = [s[n].detach().requires_grad_() for n in names]
    given = s["h0"] is not None
    h0 = s["h0"].detach().requires_grad_() if given else None
    if fused:
        y, fin = gdn.gated_linear_recurrence_fused_gates_trainable(
            *leaves, C_GATE, initial_state=h0, output_final_state=given, cu_seqlens=s["cu"])
    else:
        y, fin = gdn.gated_linear_recurrence_trainable(
            *leaves, initial_state=h0, output_final_state=given, cu_seqlens=s["cu"])
    if given:
        got = torch.autograd.grad((y, fin), leaves + [h0], (s["dh"], s["dfin"]))
    else:
        got = torch.autograd.grad(y, leaves, s["dh"])
    out = {"y": y.detach()}
    out.update(("d" + n, t) for n, t in zip(names, got))
    if given:
        out.update(state=fin.detach(), dh0=got[-1])
    return out


def _own_qk(s, gdn):
    c = s["case"]
    kw = dict(norm=None if c["norm"] == "none" else c["norm"], eps=EPS, sections=_sections(c),
              interleaved=c["pairs"] == "interleaved")
    if c["op"] == "qk_fwd":
        q, k = gdn.qk_norm_rotate(s["q"], s["k"], s["inv_freq"], s["pos"], s["wq"], s["wk"], **kw)
        return {"q": q, "k": k}
    names = ["q", "k"] + (["wq", "wk"] if s["wq"] is not None else [])
    leaf = {n: s[n].detach().requires_grad_() for n in names}
    q, k = gdn.qk_norm_rotate_trainable(leaf["q"], leaf["k"], s["inv_freq"], s["pos"], leaf.get("wq"),
                                        leaf.get("wk"), **kw)
    got = torch.autograd.grad((q, k), [leaf[n] for n in names], (s["dq"], s["dk"]))
    out = {"q": q.detach(), "k": k.detach()}
    out.update(("d" + n, t) for n, t in zip(names, got))
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        import chunked_gated_delta_gdn_gb300 as gdn
        return _own_lr(state, gdn) if op.startswith("lr_") else _own_qk(state, gdn)
    if op == "lr_decode":
        return _plain_lr_decode(state)
    if op.startswith("lr_"):
        return _plain_lr(state, op == "lr_train")
    return _plain_qk(state, op == "qk_train")


# ---------------------------------------------------------------- work

def work(case):
    eb = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("lr_"):
        D, fused = case["D"], case["gates"] == "fused"
        tensors = 4 if fused else 3
        per = 24 if fused else 3          # operations of an element, an exponential as one
        if case["op"] == "lr_decode":
            n = case["n"]
            real = n - int(round(case["pad"] * n))
            return {"bytes": n * D * tensors * eb + real * D * 8 + 4 * n + 4 * D, "flops": n * D * per}
        if "num_seqs" in case:
            tokens, N = sum(_lengths(case, 0)), case["num_seqs"]
        else:
            tokens, N = case["B"] * case["T"], case["B"]
        states = 4 * N * D * (2 if case["state"] != "none" else 1)
        if case["op"] == "lr_train":
            tensors += 7 if fused else 5
            per *= 3
            states = 16 * N * D if case["state"] != "none" else 0
        return {"bytes": tokens * D * tensors * eb + states + (8 * D if fused else 0),
                "flops": tokens * D * per}
    tokens = case["B"] * case["T"]
    n = tokens * (case["Hq"] + case["Hk"]) * case["K"]
    train = case["op"] == "qk_train"
    weights = (16 if train else 8) * case["K"] if case["norm"] == "rms" else 0
    return {"bytes": n * (5 if train else 2) * eb + tokens * case["axes"] * 4 + 2 * case["R"] + weights,
            "flops": n * (24 if train else 8)}


# ---------------------------------------------------------------- exact values (64 bits)

def _sigmoid64(t):
    return 1.0 / (1.0 + torch.exp(-t))


def _exact_inputs(s):
    """The inputs that a_t and what is added to the state are made of, in 64 bits, [tokens, D]."""
    d = torch.float64
    names = ["x", "g"] if s["case"]["gates"] == "given" else ["x", "r", "i", "lam"]
    return {n: s[n].to(d).reshape(-1, s["case"]["D"]) if n != "lam" else s[n].to(d) for n in names}


def _exact_ab(leaf):
    """a_t and what is added to the state, differentiable."""
    if "g" in leaf:
        return torch.exp(leaf["g"]), leaf["x"]
    la = -C_GATE * torch.log1p(torch.exp(leaf["lam"])) * _sigmoid64(leaf["r"])
    return torch.exp(la), torch.sqrt(-torch.expm1(2 * la)) * _sigmoid64(leaf["i"]) * leaf["x"]


def _exact_lr(case, s):
    """Token after token, the sequences that still have one side by side (longest first); backwards the
    same from the end, then through the gates by differentiation of their formulas."""
    d = torch.float64
    dev = s["x"].device
    D, N = case["D"], len(s["lens"])
    train = case["op"] == "lr_train"
    leaf = _exact_inputs(s)
    with torch.no_grad():
        a, b = _exact_ab(leaf)
    order = sorted(range(N), key=lambda n: -s["lens"][n])
    begin = [0]
    for n in s["lens"]:
        begin.append(begin[-1] + n)
    at = torch.tensor([begin[n] for n in order], device=dev)
    lens = [s["lens"][n] for n in order]
    pick = torch.tensor(order, device=dev)
    start = None
    if s["h0"] is not None:
        start = s["h0"].to(d)
        start = start if s["idx"] is None else start[s["idx"].long()]
    h = torch.zeros(N, D, dtype=d, device=dev) if start is None else start[pick]
    y = torch.empty_like(a)
    before = torch.empty_like(a) if train else None
    count, counts = N, []
    for t in range(lens[0]):
        while lens[count - 1] <= t:
            count -= 1
        counts.append(count)
        rows = at[:count] + t
        if train:
            before[rows] = h[:count]
        h[:count] = a[rows] * h[:count] + b[rows]
        y[rows] = h[:count]
    fin = torch.empty_like(h)
    fin[pick] = h
    out = {"y": y.view(s["x"].shape)}
    if not train:
        out["state"] = fin
        if s["idx"] is not None:
            out["state"] = s["h0"].to(d).index_copy(0, s["idx"].long(), fin)
        return out
    e = torch.zeros(N, D, dtype=d, device=dev) if start is None else s["dfin"].to(d)[pick]
    dy = s["dh"].to(d).reshape(-1, D)
    da, db = torch.empty_like(a), torch.empty_like(a)
    for t in range(lens[0] - 1, -1, -1):
        rows = at[:counts[t]] + t
        delta = e[:counts[t]] + dy[rows]
        db[rows] = delta
        da[rows] = delta * before[rows]
        e[:counts[t]] = delta * a[rows]
    del before, y, dy
    if start is not None:
        out["state"] = fin
        out["dh0"] = torch.empty_like(e)
        out["dh0"][pick] = e
    leaf = {n: t.requires_grad_() for n, t in leaf.items()}
    with torch.enable_grad():
        a, b = _exact_ab(leaf)
        got = torch.autograd.grad((a, b), list(leaf.values()), (da, db))
    for n, t in zip(leaf, got):
        out["d" + n] = t.view(s[n].shape)
    return out


def _exact_qk(case, s):
    d = torch.float64
    R, K = case["R"], case["K"]
    axis = [0] * (R // 2)
    if case["axes"] > 1:
        axis = [i for i, n in enumerate(_sections(case)) for _ in range(n)]
    pos = s["pos"].to(d)
    pos = pos[None] if case["axes"] == 1 else pos
    phi = torch.stack([pos[axis[j]] * s["inv_freq"][j].to(d) for j in range(R // 2)], -1) if R else None
    train = case["op"] == "qk_train"
    out = {}
    for n in ("q", "k"):
        x = s[n].to(d).contiguous().requires_grad_(train)
        w = None if s["w" + n] is None else s["w" + n].to(d).requires_grad_(train)
        with torch.set_grad_enabled(train):
            u = x
            if case["norm"] == "rms":
                u = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
            elif case["norm"] == "l2":
                u = x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)
            y = u
            if R:
                j = torch.arange(R // 2, device=x.device)
                lo, hi = (j, j + R // 2) if case["pairs"] == "halves" else (2 * j, 2 * j + 1)
                z = torch.complex(u[..., lo], u[..., hi]) * torch.exp(torch.complex(
                    torch.zeros_like(phi), phi))[:, :, None]
                y = u.index_copy(-1, lo, z.real).index_copy(-1, hi, z.imag)
            out[n] = y.detach()
            if train:
                leaves = [x] if w is None else [x, w]
                got = torch.autograd.grad(y, leaves, s["d" + n].to(d))
                out["d" + n] = got[0]
                if w is not None:
                    out["dw" + n] = got[1]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("qk_"):
        return _exact_qk(case, s)
    if case["op"] != "lr_decode":
        return _exact_lr(case, s)
    a, b = _exact_ab(_exact_inputs(s))
    cache = s["cache"].to(torch.float64)
    y = torch.zeros_like(a)
    for n, slot in enumerate(s["idx"].tolist()):
        if slot >= 0:
            y[n] = cache[slot] = a[n] * cache[slot] + b[n]
    return {"y": y, "state": cache}
