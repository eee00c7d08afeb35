"""Cases, plain forms and exact values of two sets of operators: linear attention with a decay for
each head (chunked forward, training step, single-token decode) and group norm with an activation,
channels last (forward, training step).

Linear attention, value head h with gamma = exp(log_decay[h]) and a K x V state S:

    S_t = gamma S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t,

value head h reading query/key head h // (Hv / Hqk).  Group norm over x [N, L, C]: mean and variance
of each (row n, group of C / G channels) over L and the group's channels, y = silu(n) of the
normalised, scaled and shifted value n, or n * silu(z) with a gate z.
"""
import math

import torch

own = False

CHUNK = 128      # tokens of a chunk in the plain form of linear attention
BLOCK = 256      # tokens of a block in exact()


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a short prompt in fp32 (a test, a small model): the call's latency
        dict(name="la_fwd_tiny_fp32", op="la_fwd", B=1, T=256, Hqk=2, Hv=2, K=64, V=64,
             dtype="fp32", state="given"),
        # one long prompt, few chains: the sequence axis is what there is to split
        dict(name="la_fwd_one_8192_bf16", op="la_fwd", B=1, T=8192, Hqk=16, Hv=32, K=128, V=128,
             dtype="bf16", state="given"),
        # prefill of 32 packed prompts of 100 to 4096 tokens, states in a 64-slot cache
        dict(name="la_fwd_packed32_bf16", op="la_fwd", num_seqs=32, min_len=100, max_len=4096,
             Hqk=16, Hv=32, K=128, V=128, dtype="bf16", state="slots", num_slots=64),
        # a long-context training batch's forward
        dict(name="la_fwd_4x32768_bf16", op="la_fwd", B=4, T=32768, Hqk=16, Hv=32, K=128, V=128,
             dtype="bf16", state="none"),
        # a training step on a few odd packed sequences in fp32, key and value dims that differ
        dict(name="la_train_packed5_fp32", op="la_train", num_seqs=5, min_len=1, max_len=777,
             Hqk=2, Hv=4, K=64, V=96, dtype="fp32", state="given"),
        # a training step of a layer
        dict(name="la_train_2x8192_bf16", op="la_train", B=2, T=8192, Hqk=16, Hv=32, K=128, V=128,
             dtype="bf16", state="none"),
        # one request's next token: latency
        dict(name="la_decode_1_bf16", op="la_decode", n=1, num_slots=8, pad=0.0, Hqk=16, Hv=32,
             K=128, V=128, dtype="bf16"),
        # a serving batch, a tenth of it padding, on a 512-slot cache
        dict(name="la_decode_256_bf16", op="la_decode", n=256, num_slots=512, pad=0.1, Hqk=16,
             Hv=32, K=128, V=128, dtype="bf16"),
        # the norm and gate behind a decode step of 256 requests
        dict(name="gn_fwd_256x4096_gate_bf16", op="gn_fwd", N=256, L=1, C=4096, G=32, gate=True,
             dtype="bf16"),
        # feature maps, channels last
        dict(name="gn_fwd_8x128x128x256_bf16", op="gn_fwd", N=8, L=16384, C=256, G=32, gate=False,
             dtype="bf16"),
        # a training step of the norm and gate behind 2 x 8192 tokens
        dict(name="gn_train_16384x4096_gate_bf16", op="gn_train", N=16384, L=1, C=4096, G=32,
             gate=True, dtype="bf16"),
        # a training step on odd feature maps in fp32, groups of 10 channels
        dict(name="gn_train_3x57x61x320_fp32", op="gn_train", N=3, L=57 * 61, C=320, G=32,
             gate=False, dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["la_fwd", "la_fwd", "la_train", "la_decode", "gn_fwd", "gn_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("la_fwd", "la_train", "la_decode"):
        K, V = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (96, 96), (128, 32)])
        Hqk = rng.choice([1, 2, 3, 4, 8, 16])
        Hv = Hqk * rng.choice([1, 1, 2, 4])
        c = dict(op=op, Hqk=Hqk, Hv=Hv, K=K, V=V, dtype=dtype)
        if op == "la_decode":
            n = _log_int(rng, 1, 320)
            slots = n + rng.randint(0, n)
            return dict(c, n=n, num_slots=slots, pad=rng.choice([0.0, 0.1, 0.3]))
        # tokens x value heads: fp32 up to 1/16, a training step up to 1/8 of the largest listed
        most = (4 * 32768 * 32) // (16 if dtype == "fp32" else 8 if op == "la_train" else 1)
        if rng.random() < 0.5:
            num = _log_int(rng, 1, 48)
            most_len = max(2, min(16384, most // (Hv * num)))
            hi = _log_int(rng, 2, most_len)
            return dict(c, num_seqs=num, min_len=rng.randint(0, hi // 2), max_len=hi,
                        state=rng.choice(["none", "given"] + (["slots"] if op == "la_fwd" else [])),
                        num_slots=num + rng.randint(0, 16))
        B = rng.choice([1, 1, 2, 3, 4])
        T = _log_int(rng, 1, max(1, min(32768, most // (Hv * B))))
        return dict(c, B=B, T=T, state=rng.choice(["none", "given"]))
    G = rng.choice([1, 2, 4, 8, 16, 32])
    gate = rng.random() < 0.5
    cg = rng.choice([1, 2, 3, 5, 8, 10, 16, 32, 64, 96, 128]) if G > 2 else \
        rng.choice([16, 40, 100, 128, 500, 1024])
    C = G * cg
    most = (1 << 26) // (2 if op == "gn_train" else 1)   # elements
    if rng.random() < 0.5:
        L = 1
        N = _log_int(rng, 1, max(1, min(65536, most // C)))
    else:
        N = rng.randint(1, 16)
        L = _log_int(rng, 2, max(2, min(65536, most // (C * N))))
    # a group of two or three elements leaves dx next to nothing but its own rounding
    if L * cg < 8:
        L = -(-8 // cg)
    return dict(op=op, N=N, L=L, C=C, G=G, gate=gate, dtype=dtype)


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


def _decays(Hv):
    """log gamma per head, gamma = 1 - 2^(-5 .. -12) evenly over the heads (layers with a fixed
    decay per head span short to long memory like this)."""
    e = torch.linspace(5.0, 12.0, Hv) if Hv > 1 else torch.tensor([7.0])
    return torch.log1p(-torch.exp2(-e.double())).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = _dt(case)

    def rn(*shape, std=1.0, mean=0.0, dtype=dt):
        x = torch.randn(*shape, generator=gen, device=dev)
        return (x * std + mean).to(dtype)

    s = dict(case=case)
    if case["op"].startswith("la_"):
        Hqk, Hv, K, V = case["Hqk"], case["Hv"], case["K"], case["V"]
        s["log_decay"] = _decays(Hv).to(dev)
        if case["op"] == "la_decode":
            n, slots = case["n"], case["num_slots"]
            s["q"], s["k"], s["v"] = rn(n, Hqk, K), rn(n, Hqk, K), rn(n, Hv, V)
            s["cache"] = rn(slots, Hv, K, V, dtype=torch.float32)
            idx = torch.randperm(slots, generator=gen, device=dev)[:n].to(torch.int32)
            pad = torch.randperm(n, generator=gen, device=dev)[: int(round(case["pad"] * n))]
            idx[pad] = -1
            s["idx"] = idx
            return s
        if "num_seqs" in case:
            lens = _lengths(case, seed)
            cu = [0]
            for x in lens:
                cu.append(cu[-1] + x)
            s["lens"] = torch.tensor(lens, dtype=torch.int64, device=dev)
            s["max_len"] = max(lens)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
            B, T, N = 1, cu[-1], len(lens)
        else:
            B, T = case["B"], case["T"]
            s["cu"], N = None, B
        s["N"] = N
        s["q"], s["k"], s["v"] = rn(B, T, Hqk, K), rn(B, T, Hqk, K), rn(B, T, Hv, V)
        s["h0"] = s["idx"] = None
        if case["state"] == "given":
            s["h0"] = rn(N, Hv, K, V, dtype=torch.float32)
        elif case["state"] == "slots":
            s["h0"] = rn(case["num_slots"], Hv, K, V, dtype=torch.float32)
            s["idx"] = torch.randperm(case["num_slots"], generator=gen, device=dev)[:N].to(torch.int32)
        if case["op"] == "la_train":
            s["do"] = rn(B, T, Hv, V)
            s["dh"] = rn(N, Hv, K, V, dtype=torch.float32) if s["h0"] is not None else None
        return s
    N, L, C = case["N"], case["L"], case["C"]
    s["x"] = rn(N, L, C, std=1.5, mean=0.4) if L > 1 else rn(N, C, std=1.5)
    s["w"] = rn(C, std=0.2, mean=1.0, dtype=torch.float32)
    s["b"] = rn(C, std=0.2, dtype=torch.float32)
    s["z"] = rn(*s["x"].shape) if case["gate"] else None
    if case["op"] == "gn_train":
        s["dy"] = rn(*s["x"].shape)
    return s


# ---------------------------------------------------------------- plain forms (fp32)

def _scan(q, k, v, ld, h0, steps):
    """Dense linear attention without scale, heads expanded: q, k [N, T, H, K], v [N, T, H, V] fp32,
    left-padded so that every sequence ends at T; steps [N, T]: a token's index in its sequence
    (padding: negative, its k is zero).  Returns (o, final state)."""
    N, T, H, K = q.shape
    V = v.shape[-1]
    pad = -T % CHUNK
    if pad:
        q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, 0, pad, 0)) for x in (q, k, v))
    nc = (T + pad) // CHUNK
    q, k, v = (x.view(N, nc, CHUNK, H, x.shape[-1]).permute(0, 3, 1, 2, 4) for x in (q, k, v))
    ar = torch.arange(CHUNK, device=q.device)
    d = (ar[:, None] - ar[None, :])
    mask = torch.where(d >= 0, torch.exp(ld[:, None, None] * d.clamp(min=0)), 0.0)       # [H, C, C]
    o = ((q @ k.transpose(-1, -2)) * mask[None, :, None]) @ v
    w = torch.exp(ld[:, None] * (CHUNK - 1 - ar))                                        # [H, C]
    u = (k * w[None, :, None, :, None]).transpose(-1, -2) @ v                            # [N, H, nc, K, V]
    m = torch.arange(nc + 1, device=q.device)
    e = (m[:, None] - 1 - m[None, :nc])
    carry = torch.where(e >= 0, torch.exp(ld[:, None, None] * (e.clamp(min=0) * CHUNK)), 0.0)  # [H, nc+1, nc]
    s = (carry[None] @ u.reshape(N, H, nc, K * V)).view(N, H, nc + 1, K, V)
    o = o + torch.exp(ld[:, None] * (ar + 1))[None, :, None, :, None] * (q @ s[:, :, :nc])
    o = o.permute(0, 2, 3, 1, 4).reshape(N, T + pad, H, V)[:, pad:]
    fin = s[:, :, nc]
    if h0 is not None:
        qf = q.permute(0, 2, 3, 1, 4).reshape(N, T + pad, H, K)[:, pad:]
        g = torch.exp(ld * (steps + 1).clamp(min=0)[..., None])                          # [N, T, H]
        o = o + g[..., None] * torch.einsum("nthk,nhkv->nthv", qf, h0)
        count = steps[:, -1] + 1 if T else torch.zeros(N, device=q.device)
        fin = fin + torch.exp(ld * count[:, None])[..., None, None] * h0
    return o, fin


def _rows(s, B, T):
    """Where each token of the left-padded [N, max_len] layout stands in the packed one, and its
    index in its sequence (negative: padding)."""
    dev = s["q"].device
    if s["cu"] is None:
        return None, torch.arange(T, device=dev).expand(B, T)
    M = max(1, s["max_len"])
    steps = torch.arange(M, device=dev)[None] - (M - s["lens"])[:, None]
    at = s["cu"][:-1, None].long() + steps.clamp(min=0)
    return at.clamp(max=max(T - 1, 0)), steps


def _padded(x, at, steps, rep):
    x = x.float()
    if at is not None:
        x = torch.where((steps >= 0)[..., None, None], x[0][at], 0.0)
    return x.repeat_interleave(rep, dim=2) if rep > 1 else x


def _packed(x, at, steps, T):
    if at is None:
        return x
    dst = torch.where(steps >= 0, at, T).reshape(-1)
    out = x.new_zeros((T + 1,) + tuple(x.shape[2:]))
    return out.index_copy_(0, dst, x.reshape((-1,) + tuple(x.shape[2:])))[None, :T]


def _plain_la(s, train):
    c = s["case"]
    dt, rep = _dt(c), c["Hv"] // c["Hqk"]
    B, T = s["q"].shape[:2]
    sc = 1.0 / math.sqrt(c["K"])
    ld = s["log_decay"]
    at, steps = _rows(s, B, T)
    q, k = (_padded(s[n], at, steps, rep) for n in ("q", "k"))
    v = _padded(s["v"], at, steps, 1)
    h0 = s["h0"] if s["idx"] is None else s["h0"][s["idx"].long()]
    o, fin = _scan(q, k, v, ld, h0, steps)
    o = _packed(o * sc, at, steps, T).to(dt)
    if not train:
        if s["idx"] is not None:
            fin = s["h0"].index_copy_(0, s["idx"].long(), fin)
        return {"o": o, "state": fin}
    do = _padded(s["do"], at, steps, 1) * sc
    tr = None if h0 is None else h0.transpose(-1, -2)
    dq, _ = _scan(do, v, k, ld, tr, steps)
    # backwards in time: o'_t reads the state before its own decay, so the given state enters with
    # one decay fewer and leaves with one more
    un = torch.exp(-ld)[:, None, None]
    dh = None if s["dh"] is None else s["dh"] * un
    f = lambda x: x.flip(1)
    count = (steps[:, -1] + 1)
    if at is not None:      # reversed sequences end at T as well: turn each inside its own length
        M = steps.shape[1]
        turn = torch.where(steps >= 0, (M - 1 - steps), torch.arange(M, device=ld.device)[None])
        f = lambda x: torch.gather(x, 1, turn[..., None, None].expand_as(x))
    dv, dh0 = _scan(f(k), f(q), f(do), ld, dh, steps)
    dk, _ = _scan(f(v), f(do), f(q), ld, None if dh is None else dh.transpose(-1, -2), steps)
    dv, dk = f(dv), f(dk)
    fold = lambda x: x.unflatten(2, (c["Hqk"], rep)).sum(3)
    back = lambda x: _packed(x, at, steps, T).to(dt)
    out = {"o": o, "dq": back(fold(dq)), "dk": back(fold(dk)), "dv": back(dv)}
    if h0 is not None:      # a step with states carried from batch to batch
        out["state"] = fin
        out["dh0"] = dh0 * torch.exp(ld)[:, None, None]
    return out


def _plain_decode(s):
    c = s["case"]
    rep = c["Hv"] // c["Hqk"]
    q, k = (s[n].float().repeat_interleave(rep, dim=1) for n in ("q", "k"))
    v = s["v"].float()
    on = (s["idx"] >= 0)
    at = s["idx"].clamp(min=0).long()
    old = s["cache"][at]
    new = old * torch.exp(s["log_decay"])[:, None, None] + k[..., :, None] * v[..., None, :]
    o = (q[..., None, :] @ new)[..., 0, :] / math.sqrt(c["K"])
    o = torch.where(on[:, None, None], o, 0.0).to(s["q"].dtype)
    s["cache"].index_add_(0, at, torch.where(on[:, None, None, None], new - old, 0.0))
    return {"o": o, "state": s["cache"]}


def _plain_gn(s, train):
    c = s["case"]
    N, L, C, G = c["N"], c["L"], c["C"], c["G"]
    dt = _dt(c)
    x = s["x"].float().view(N, L, G, C // G)
    w, b = s["w"].view(G, -1), s["b"].view(G, -1)
    mean = x.mean((1, 3), keepdim=True)
    d = x - mean
    rstd = torch.rsqrt(d.square().mean((1, 3), keepdim=True) + 1e-5)
    xh = d * rstd
    n = xh * w + b
    a = n if s["z"] is None else s["z"].float().view_as(n)
    sig = torch.sigmoid(a)
    y = a * sig if s["z"] is None else n * (a * sig)
    out = {"y": y.to(dt).view(s["x"].shape)}
    if train:
        dy = s["dy"].float().view_as(n)
        slope = sig * (1 + a * (1 - sig))
        if s["z"] is None:
            dn = dy * slope
        else:
            dn = dy * (a * sig)
            out["dz"] = (dy * n * slope).to(dt).view(s["x"].shape)
        out["dw"] = (dn * xh).sum((0, 1)).view(C)
        out["db"] = dn.sum((0, 1)).view(C)
        g = dn * w
        dx = rstd * (g - g.mean((1, 3), keepdim=True) - xh * (g * xh).mean((1, 3), keepdim=True))
        out["dx"] = dx.to(dt).view(s["x"].shape)
    return out


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    import chunked_gated_delta_gdn_gb300 as gdn
    c = s["case"]
    if c["op"] == "la_fwd":
        o, fin = gdn.chunk_linear_attn(s["q"], s["k"], s["v"], s["log_decay"],
                                       initial_state=s["h0"], output_final_state=True,
                                       cu_seqlens=s["cu"], state_indices=s["idx"])
        return {"o": o, "state": fin}
    if c["op"] == "la_train":
        given = s["h0"] is not None
        q, k, v = (s[n].detach().requires_grad_() for n in ("q", "k", "v"))
        h0 = s["h0"].detach().requires_grad_() if given else None
        o, fin = gdn.chunk_linear_attn_trainable(q, k, v, s["log_decay"], initial_state=h0,
                                                 output_final_state=given, cu_seqlens=s["cu"])
        if given:
            dq, dk, dv, dh0 = torch.autograd.grad((o, fin), (q, k, v, h0), (s["do"], s["dh"]))
        else:
            dq, dk, dv = torch.autograd.grad(o, (q, k, v), s["do"])
        out = {"o": o.detach(), "dq": dq, "dk": dk, "dv": dv}
        if given:
            out.update(state=fin.detach(), dh0=dh0)
        return out
    if c["op"] == "la_decode":
        o = gdn.linear_attn_decode(s["q"], s["k"], s["v"], s["log_decay"], s["cache"], s["idx"])
        return {"o": o, "state": s["cache"]}
    if c["op"] == "gn_fwd":
        return {"y": gdn.group_norm_act(s["x"], c["G"], s["w"], s["b"], eps=1e-5,
                                        activation="silu", gate=s["z"])}
    leaf = lambda t: None if t is None else t.detach().requires_grad_()
    x, w, b, z = leaf(s["x"]), leaf(s["w"]), leaf(s["b"]), leaf(s["z"])
    y = gdn.group_norm_act_trainable(x, c["G"], w, b, eps=1e-5, activation="silu", gate=z)
    got = torch.autograd.grad(y, (x, w, b) if z is None else (x, w, b, z), s["dy"])
    out = {"y": y.detach(), "dx": got[0], "dw": got[1], "db": got[2]}
    if z is not None:
        out["dz"] = got[3]
    return out


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "la_decode":
        return _plain_decode(state)
    if op.startswith("la_"):
        return _plain_la(state, op == "la_train")
    return _plain_gn(state, op == "gn_train")


# ---------------------------------------------------------------- work

def work(case):
    eb = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("la_"):
        Hqk, Hv, K, V = case["Hqk"], case["Hv"], case["K"], case["V"]
        if case["op"] == "la_decode":
            real = case["n"] - int(round(case["pad"] * case["n"]))
            io = case["n"] * (2 * Hqk * K + 2 * Hv * V) * eb
            return {"bytes": io + real * Hv * K * V * 8 + 4 * Hv, "flops": real * Hv * 5 * K * V}
        if "num_seqs" in case:
            tokens, N = sum(_lengths(case, 0)), case["num_seqs"]
        else:
            tokens, N = case["B"] * case["T"], case["B"]
        states = N * Hv * K * V * 4 * (2 if case["state"] != "none" else 1)
        if case["op"] == "la_train" and case["state"] == "none":
            states = 0
        io = tokens * (2 * Hqk * K + 2 * Hv * V) * eb
        # one token's products at chunks of 64: half of the causal square, and the state's two
        fl = tokens * Hv * (64 * (K + V) + 4 * K * V)
        if case["op"] == "la_train":
            io += tokens * (4 * Hqk * K + 3 * Hv * V) * eb
            if case["state"] != "none":
                states *= 2
            fl += tokens * Hv * (64 * (3 * K + 2 * V) + 8 * K * V)
        return {"bytes": max(1, io + states), "flops": fl}
    n = case["N"] * case["L"] * case["C"]
    g = 1 if case["gate"] else 0
    passes = 2 + g
    fl = 12 * n
    if case["op"] == "gn_train":
        passes += 3 + 2 * g
        fl += 24 * n
    return {"bytes": n * passes * eb + 8 * case["C"], "flops": fl}


# ---------------------------------------------------------------- exact values (64 bits)

def _exact_seq(q, k, v, ld, h0):
    """The recurrence in 64 bits over one batch of equal sequences, BLOCK tokens at a time: q, k
    [B, T, H, K], v [B, T, H, V] (heads expanded, scale applied to q), h0 [B, H, K, V]."""
    outs, S = [], h0
    for t0 in range(0, q.shape[1], BLOCK):
        qc, kc, vc = (x[:, t0:t0 + BLOCK] for x in (q, k, v))
        n = qc.shape[1]
        t = torch.arange(n, device=q.device, dtype=torch.float64)
        dist = t[:, None] - t[None, :]
        dec = torch.exp(ld[:, None, None] * dist.clamp(min=0)) * (dist >= 0)
        att = torch.einsum("bihk,bjhk->bhij", qc, kc) * dec
        o = torch.einsum("bhij,bjhv->bihv", att, vc)
        into = torch.exp((t[:, None] + 1) * ld)
        o = o + torch.einsum("bihk,bhkv->bihv", qc * into[None, :, :, None], S)
        left = torch.exp((n - 1 - t)[:, None] * ld)
        S = S * torch.exp(n * ld)[:, None, None] + torch.einsum("bjhk,bjhv->bhkv",
                                                                kc * left[None, :, :, None], vc)
        outs.append(o)
    return (torch.cat(outs, 1) if outs else v[:, :0]), S


def _exact_la(case, s):
    d = torch.float64
    Hqk, Hv, K, V = case["Hqk"], case["Hv"], case["K"], case["V"]
    rep, train = Hv // Hqk, case["op"] == "la_train"
    ld = s["log_decay"].to(d)
    N = s["N"]
    slot = list(range(N)) if s["idx"] is None else s["idx"].tolist()
    q, k, v = (s[n].to(d) for n in ("q", "k", "v"))
    state = None if s["h0"] is None else s["h0"].to(d)
    if s["cu"] is None:
        parts = [(slice(0, N), slice(None), None)]
    else:
        cu = s["cu"].tolist()
        parts = [(slice(0, 1), slice(cu[n], cu[n + 1]), n) for n in range(N)]
    keep = {n: [] for n in ("o", "dq", "dk", "dv", "dh0", "state")}
    for rows, span, n in parts:
        xs = [x[rows, span].detach().requires_grad_(train) for x in (q, k, v)]
        B = xs[0].shape[0]
        if state is None:
            h0 = torch.zeros(B, Hv, K, V, dtype=d, device=q.device)
        else:
            h0 = state if n is None else state[slot[n]:slot[n] + 1]
        h0 = h0.detach().requires_grad_(train)
        with torch.set_grad_enabled(train):
            qe, ke = (x.repeat_interleave(rep, dim=2) for x in xs[:2])
            o, fin = _exact_seq(qe / math.sqrt(K), ke, xs[2], ld, h0)
            if train:
                loss = (o * s["do"][rows, span].to(d)).sum()
                if s["dh"] is not None:
                    loss = loss + (fin * (s["dh"] if n is None else s["dh"][n:n + 1]).to(d)).sum()
                got = torch.autograd.grad(loss, xs + [h0], allow_unused=True)
                got = [torch.zeros_like(x) if g is None else g for g, x in zip(got, xs + [h0])]
                for name, g in zip(("dq", "dk", "dv", "dh0"), got):
                    keep[name].append(g)
        keep["o"].append(o.detach())
        keep["state"].append(fin.detach())
    axis = 0 if s["cu"] is None else 1
    out = {"o": torch.cat(keep["o"], axis)}
    if not train or state is not None:
        out["state"] = torch.cat(keep["state"], 0)
    if s["idx"] is not None:
        out["state"] = state.index_copy(0, s["idx"].long(), out["state"])
    if train:
        out.update({n: torch.cat(keep[n], axis) for n in ("dq", "dk", "dv")})
        if state is not None:
            out["dh0"] = torch.cat(keep["dh0"], 0)
    return out


def _exact_gn(case, s):
    d = torch.float64
    N, L, C, G = case["N"], case["L"], case["C"], case["G"]
    train = case["op"] == "gn_train"
    leaf = lambda t: None if t is None else t.to(d).requires_grad_(train)
    x, w, b, z = leaf(s["x"]), leaf(s["w"]), leaf(s["b"]), leaf(s["z"])
    with torch.set_grad_enabled(train):
        xr = x.reshape(N, L, G, C // G).transpose(1, 2).reshape(N, G, -1)
        var, mean = torch.var_mean(xr, dim=2, unbiased=False, keepdim=True)
        n = ((xr - mean) / torch.sqrt(var + 1e-5)).view(N, G, L, C // G).transpose(1, 2).reshape(N, L, C)
        n = (n * w + b).view(x.shape)
        y = n / (1 + torch.exp(-n)) if z is None else n * z / (1 + torch.exp(-z))
        out = {"y": y.detach()}
        if train:
            got = torch.autograd.grad(y, (x, w, b) if z is None else (x, w, b, z), s["dy"].to(d))
            out.update(dict(zip(("dx", "dw", "db", "dz"), got)))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("gn_"):
        return _exact_gn(case, s)
    if case["op"] != "la_decode":
        return _exact_la(case, s)
    d = torch.float64
    rep = case["Hv"] // case["Hqk"]
    cache = s["cache"].to(d)
    o = torch.zeros(s["v"].shape, dtype=d, device=cache.device)
    gamma = torch.exp(s["log_decay"].to(d))[:, None, None]
    for i, slot in enumerate(s["idx"].tolist()):
        if slot < 0:
            continue
        k, q = (s[n][i].to(d).repeat_interleave(rep, dim=0) for n in ("k", "q"))
        cache[slot] = gamma * cache[slot] + torch.einsum("hk,hv->hkv", k, s["v"][i].to(d))
        o[i] = torch.einsum("hk,hkv->hv", q, cache[slot]) / math.sqrt(case["K"])
    return {"o": o, "state": cache}
