"""Linear attention with a decay for each head on the GPU against the 64-bit recurrence.

Tolerances (relative 2-norm), from the number formats:
* fp32 values (fp32 I/O, every state): products and sums of 24-bit values; a sum of n terms of
  random sign errs by about sqrt(n) 2^-24 of its terms' norm and the longest chains here have a
  few hundred terms, so 24 * 2^-24 = 1.4e-6 typically; 5e-6 leaves a factor of 3.5.
* bf16 outputs: rounding to 8 bits errs by 2^-9 at most, 1.7e-3 in the 2-norm; one operand of
  each matrix product may be rounded likewise, which adds the same in quadrature: 2.4e-3, and
  4e-3 for every case.
"""
import math

import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn
from chunked_gated_delta_gdn_gb300 import _lib
from tests import linear_attn_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 5e-6, BF16: 4e-3}


def decays(Hv, kind="span"):
    if kind == "span":      # memories of 4 to 4096 tokens
        return torch.log1p(-torch.exp2(-torch.linspace(2, 12, Hv).double())).float()
    if kind == "edge":      # no decay, none kept, nearly none kept, strong, slow
        x = [0.0, float("-inf"), -30.0, -1.5, -1e-6, -200.0]
        return torch.tensor([x[i % len(x)] for i in range(Hv)])
    raise ValueError(kind)


def make(B=1, T=64, Hqk=2, Hv=2, K=128, V=128, dtype=BF16, lens=None, h0=True, seed=0, decay="span",
         tail=0):
    g = torch.Generator().manual_seed(seed)
    cu = None
    N = B
    if lens is not None:
        cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(lens).cumsum(0)
        B, T, N = 1, int(cu[-1]) + tail, len(lens)
    r = lambda *s: torch.randn(*s, generator=g)
    x = dict(q=r(B, T, Hqk, K).to(dtype), k=r(B, T, Hqk, K).to(dtype), v=r(B, T, Hv, V).to(dtype),
             log_decay=decays(Hv, decay), cu=cu)
    x["h0"] = r(N, Hv, K, V) if h0 else None
    return x


def on_gpu(x):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in x.items()}


def check_forward(x, **kw):
    c = on_gpu(x)
    B, T, _, _ = x["q"].shape
    out = torch.full(x["v"].shape, float("nan"), dtype=x["v"].dtype, device="cuda")
    o, fin = gdn.chunk_linear_attn(c["q"], c["k"], c["v"], c["log_decay"], initial_state=c["h0"],
                                   output_final_state=True, cu_seqlens=c["cu"], out=out, check=True, **kw)
    o_ref, fin_ref = ref.forward(c["q"], c["k"], c["v"], c["log_decay"], h0=c["h0"], cu=x["cu"], **kw)
    e_o, e_s = ref.rel(o, o_ref), ref.rel(fin, fin_ref)
    print("o %.2e state %.2e" % (e_o, e_s))
    assert e_o <= TOL[x["q"].dtype] and e_s <= TOL[F32]
    return o, fin


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 200])
def test_forward_lengths(T, dtype):
    check_forward(make(B=2, T=T, dtype=dtype, seed=T))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dims", [(1, 1, 128, 128), (2, 6, 64, 64), (3, 3, 64, 128), (1, 4, 128, 32),
                                  (2, 2, 96, 96), (1, 2, 8, 16), (5, 5, 128, 8), (1, 1, 24, 104)])
def test_forward_dims_and_heads(dims, dtype):
    Hqk, Hv, K, V = dims
    check_forward(make(B=1, T=150, Hqk=Hqk, Hv=Hv, K=K, V=V, dtype=dtype, seed=K + V))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("KV", [(128, 128), (64, 96)])
def test_forward_packed(KV, dtype):
    x = make(lens=[0, 1, 64, 129, 0, 63, 300, 2, 0], tail=37, Hqk=1, Hv=2, K=KV[0], V=KV[1],
             dtype=dtype, seed=5)
    o, fin = check_forward(x)
    assert torch.count_nonzero(o[0, -37:]).item() == 0          # rows of no sequence
    for n in (0, 4, 8):                                         # empty: the state passes through
        assert torch.equal(fin[n].cpu(), x["h0"][n])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward_edge_decays(dtype):
    check_forward(make(B=1, T=190, Hqk=6, Hv=6, dtype=dtype, decay="edge", seed=9))


def test_forward_long_memory_state():
    """The state's error must not add up over thousands of chunks (one head, almost no decay)."""
    x = make(B=1, T=20000, Hqk=1, Hv=1, K=64, V=64, dtype=F32, seed=3)
    x["log_decay"] = torch.tensor([-2.0 ** -12])
    check_forward(x)
    y = make(B=1, T=20000, Hqk=1, Hv=1, dtype=BF16, seed=4)
    y["log_decay"] = torch.tensor([-2.0 ** -12])
    check_forward(y)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,Hv", [(1500, 1), (4097, 2)])
def test_forward_few_long_chains(T, Hv, dtype):
    check_forward(make(B=1, T=T, Hqk=1, Hv=Hv, dtype=dtype, seed=T))


def test_forward_options():
    x = make(B=2, T=70, h0=False)
    check_forward(x, scale=0.37)
    c = on_gpu(x)
    o, fin = gdn.chunk_linear_attn(c["q"], c["k"], c["v"], c["log_decay"])
    assert fin is None
    o2, _ = gdn.chunk_linear_attn(c["q"], c["k"], c["v"], c["log_decay"], output_final_state=True,
                                  initial_state=torch.zeros(2, 2, 128, 128, device="cuda"))
    assert ref.rel(o, o2.double()) <= 4e-3


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward_slot_cache(dtype):
    lens = [70, 0, 130, 65, 20]
    x = make(lens=lens, Hqk=2, Hv=4, dtype=dtype, h0=False, seed=11)
    g = torch.Generator().manual_seed(12)
    cache = torch.randn(9, 4, 128, 128, generator=g)
    slots = [7, 2, -1, 0, 100]          # padding, and one out of range
    c = on_gpu(x)
    dcache = cache.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(x["v"].shape, float("nan"), dtype=dtype, device="cuda")
    o, fin = gdn.chunk_linear_attn(c["q"], c["k"], c["v"], c["log_decay"], initial_state=dcache,
                                   output_final_state=True, cu_seqlens=c["cu"], out=out,
                                   state_indices=torch.tensor(slots, dtype=torch.int32, device="cuda"),
                                   dev_status=status)
    assert fin is dcache and int(status.item()) == _lib.GDN_DEV_BAD_SLOT
    h0 = torch.stack([cache[s if 0 <= s < 9 else 0] for s in slots])
    o_ref, fin_ref = ref.forward(c["q"], c["k"], c["v"], c["log_decay"], h0=h0.cuda(), cu=x["cu"])
    cu = x["cu"].tolist()
    for n, s in enumerate(slots):
        rows = o[0, cu[n]:cu[n + 1]]
        if 0 <= s < 9:
            assert ref.rel(rows, o_ref[0, cu[n]:cu[n + 1]]) <= TOL[dtype]
            assert ref.rel(dcache[s], fin_ref[n]) <= TOL[F32]
        else:
            assert torch.count_nonzero(rows).item() == 0
    for s in set(range(9)) - {7, 2, 0}:
        assert torch.equal(dcache[s].cpu(), cache[s])


@pytest.mark.parametrize("T,dtype", [(1100, BF16), (2049, BF16), (190, F32), (2049, F32)])
def test_one_long_slot_in_place(T, dtype):
    """Few chains: the sequence is worked on in segments, the slot's state read and written in place."""
    x = make(lens=[T, 70], Hqk=1, Hv=2, dtype=dtype, h0=False, seed=T)
    c = on_gpu(x)
    for _ in range(3):
        cache = torch.randn(4, 2, 128, 128, generator=torch.Generator().manual_seed(13))
        dcache = cache.cuda()
        idx = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
        o, fin = gdn.chunk_linear_attn(c["q"], c["k"], c["v"], c["log_decay"], initial_state=dcache,
                                       output_final_state=True, cu_seqlens=c["cu"], state_indices=idx,
                                       check=True)
        o_ref, fin_ref = ref.forward(c["q"], c["k"], c["v"], c["log_decay"], h0=dcache.new_tensor(
            cache[[2, 1]].numpy()), cu=x["cu"])
        assert ref.rel(o, o_ref) <= TOL[dtype]
        assert ref.rel(dcache[[2, 1]], fin_ref) <= TOL[F32]
        assert torch.equal(dcache[[0, 3]].cpu(), cache[[0, 3]])


def test_non_finite_rows_stay_in_their_sequence():
    """Neighbouring sequences and the tail hold NaN and infinities; the sequence between them, of a
    length that ends inside a chunk, must not see them."""
    for dtype in (F32, BF16):
        for bad in (float("nan"), float("inf")):
            x = make(lens=[30, 75, 40], tail=20, dtype=dtype, seed=2)
            clean = {n: (t.clone() if isinstance(t, torch.Tensor) else t) for n, t in x.items()}
            for n in ("q", "k", "v"):
                x[n][0, :30] = bad
                x[n][0, 105:] = bad
            c = on_gpu(x)
            o, fin = gdn.chunk_linear_attn(c["q"], c["k"], c["v"], c["log_decay"], initial_state=c["h0"],
                                           output_final_state=True, cu_seqlens=c["cu"])
            d = on_gpu(clean)
            o_ref, fin_ref = ref.forward(d["q"], d["k"], d["v"], d["log_decay"], h0=d["h0"], cu=x["cu"])
            assert ref.rel(o[0, 30:105], o_ref[0, 30:105]) <= TOL[dtype]
            assert ref.rel(fin[1], fin_ref[1]) <= TOL[F32]
            do = torch.zeros_like(c["v"])
            do[0, 30:105] = 1
            do[0, :30] = bad
            do[0, 105:] = bad
            dq, dk, dv, _ = gdn.chunk_linear_attn_bwd(c["q"], c["k"], c["v"], c["log_decay"], do,
                                                      cu_seqlens=c["cu"])
            for g in (dq, dk, dv):
                assert torch.isfinite(g[0, 30:105].float()).all()


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [5, 50, 100], [0, 50, 130], [0, -3, 100]])
def test_bad_cu_seqlens_are_reported(cu):
    for dtype in (F32, BF16):
        x = on_gpu(make(B=1, T=100, dtype=dtype, h0=False))
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        with pytest.raises(gdn.GdnDeviceError):
            gdn.chunk_linear_attn(x["q"], x["k"], x["v"], x["log_decay"], cu_seqlens=c, check=True)
        with pytest.raises(gdn.GdnDeviceError):
            gdn.chunk_linear_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["v"], cu_seqlens=c,
                                      check=True)


def grads_ref(x, do, dh, scale=None):
    leaves = [x[n].double().requires_grad_() for n in ("q", "k", "v")]
    h0 = None if x["h0"] is None else x["h0"].double().requires_grad_()
    o, fin = ref.forward(*leaves, x["log_decay"], h0=h0, cu=x["cu"], scale=scale)
    loss = (o * do.double()).sum() + (0 if dh is None else (fin * dh.double()).sum())
    return torch.autograd.grad(loss, leaves + ([] if h0 is None else [h0]))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", [dict(B=2, T=130, Hqk=2, Hv=2), dict(B=1, T=1, Hqk=1, Hv=2),
                                  dict(lens=[0, 1, 64, 97, 0, 130], tail=11, Hqk=1, Hv=3),
                                  dict(B=1, T=100, Hqk=2, Hv=4, K=64, V=96),
                                  dict(B=1, T=100, Hqk=1, Hv=1, K=96, V=32),
                                  dict(B=1, T=190, Hqk=6, Hv=6, decay="edge"),
                                  dict(B=1, T=1000, Hqk=1, Hv=2)])
def test_backward(case, dtype):
    for state in (True, False):
        x = on_gpu(make(dtype=dtype, h0=state, seed=21, **case))
        g = torch.Generator().manual_seed(22)
        do = torch.randn(x["v"].shape, generator=g).to(dtype).cuda()
        dh = torch.randn(x["h0"].shape, generator=g).cuda() if state else None
        got = gdn.chunk_linear_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], do, dh,
                                        initial_state=x["h0"], cu_seqlens=x["cu"], check=True)
        want = grads_ref(x, do, dh)
        errs = [ref.rel(a, b) for a, b in zip(got, want)]
        print(["%.2e" % e for e in errs])
        assert all(e <= TOL[dtype] for e in errs[:3])
        if state:
            assert errs[3] <= TOL[F32]
        if "tail" in case:
            for a in got[:3]:
                assert torch.count_nonzero(a[0, -11:]).item() == 0


def test_backward_matches_differences():
    """The loss is linear in each of q, k, v and h0 alone, so loss(x + d) - loss(x) = <grad, d>
    for a direction of any length.  fp32: the losses' own rounding is about 1e-6 of their size."""
    x = on_gpu(make(B=1, T=140, Hqk=2, Hv=4, dtype=F32, seed=31))
    g = torch.Generator().manual_seed(32)
    do, dh = torch.randn(x["v"].shape, generator=g).cuda(), torch.randn(x["h0"].shape, generator=g).cuda()

    def loss(**kw):
        y = {**x, **kw}
        o, fin = gdn.chunk_linear_attn(y["q"], y["k"], y["v"], y["log_decay"], initial_state=y["h0"],
                                       output_final_state=True)
        return (o.double() * do).sum() + (fin.double() * dh).sum()

    got = gdn.chunk_linear_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], do, dh, initial_state=x["h0"])
    for name, grad in zip(("q", "k", "v", "h0"), got):
        d = torch.randn(x[name].shape, generator=g).cuda()
        a, b = loss(**{name: x[name] + d}), loss()
        want = (grad.double() * d).sum()
        size = grad.double().norm() * d.double().norm()
        assert abs((a - b) - want) <= 1e-5 * size


def test_autograd_op():
    x = on_gpu(make(B=2, T=100, Hqk=1, Hv=2, dtype=BF16, seed=41))
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "h0")]
    o, fin = gdn.chunk_linear_attn_trainable(*leaves[:3], x["log_decay"], initial_state=leaves[3],
                                             output_final_state=True)
    do, dh = torch.randn_like(o), torch.randn_like(fin)
    got = torch.autograd.grad((o, fin), leaves, (do, dh))
    want = gdn.chunk_linear_attn_bwd(x["q"].detach(), x["k"].detach(), x["v"].detach(), x["log_decay"],
                                     do, dh, initial_state=x["h0"].detach())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    o, fin = gdn.chunk_linear_attn_trainable(*leaves[:3], x["log_decay"], initial_state=leaves[3],
                                             output_final_state=True)
    only = torch.autograd.grad(fin, leaves[:2], dh, allow_unused=True)   # the state alone
    assert torch.count_nonzero(only[0]).item() == 0 and torch.isfinite(only[1].float()).all()
    with pytest.raises(ValueError, match="constant"):
        gdn.chunk_linear_attn_trainable(*leaves[:3], x["log_decay"].requires_grad_())


def test_runs_are_bitwise_equal_and_on_any_stream():
    x = on_gpu(make(B=2, T=333, Hqk=2, Hv=4, dtype=BF16, seed=51))

    def call():
        o, fin = gdn.chunk_linear_attn(x["q"], x["k"], x["v"], x["log_decay"], initial_state=x["h0"],
                                       output_final_state=True)
        return (o, fin) + gdn.chunk_linear_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], o, fin,
                                                    initial_state=x["h0"])

    a = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = call()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_first_call_of_a_thread():
    """A thread that has made no CUDA call yet (as autograd's) has no current context."""
    import threading
    x = on_gpu(make(B=1, T=100, Hqk=1, Hv=1, dtype=BF16, seed=55, h0=False))
    want = gdn.chunk_linear_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["v"])
    spare = [torch.empty_like(t) for t in want if t is not None]
    torch.cuda.synchronize()
    del spare       # blocks for the thread's outputs, so that it allocates nothing on the device
    got = []
    t = threading.Thread(target=lambda: got.append(
        gdn.chunk_linear_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["v"])))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert len(got) == 1 and all(torch.equal(a, b) for a, b in zip(got[0], want))


def test_graph_capture():
    x = on_gpu(make(lens=[100, 0, 37], Hqk=2, Hv=2, dtype=BF16, seed=61))
    o = torch.empty_like(x["v"])
    fin = torch.empty_like(x["h0"])

    def call():
        gdn.chunk_linear_attn(x["q"], x["k"], x["v"], x["log_decay"], initial_state=x["h0"],
                              output_final_state=True, cu_seqlens=x["cu"], out=o, final_state=fin)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    y = make(lens=[37, 50, 50], Hqk=2, Hv=2, dtype=BF16, seed=62)
    for n in ("q", "k", "v", "h0", "cu"):
        x[n].copy_(y[n])
    g.replay()
    o_ref, fin_ref = ref.forward(x["q"], x["k"], x["v"], x["log_decay"], h0=x["h0"], cu=y["cu"])
    assert ref.rel(o, o_ref) <= TOL[BF16] and ref.rel(fin, fin_ref) <= TOL[F32]


# ------------------------------------------------------------------ decode

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dims", [(2, 4, 128, 128), (1, 1, 64, 64), (3, 3, 8, 16), (1, 2, 128, 32),
                                  (2, 2, 96, 96), (1, 1, 24, 104)])
def test_decode(dims, dtype):
    Hqk, Hv, K, V = dims
    g = torch.Generator().manual_seed(71)
    n, slots = 13, 20
    r = lambda *s: torch.randn(*s, generator=g)
    q, k, v = r(n, Hqk, K).to(dtype), r(n, Hqk, K).to(dtype), r(n, Hv, V).to(dtype)
    cache = r(slots, Hv, K, V)
    idx = torch.randperm(slots, generator=g)[:n].to(torch.int32)
    idx[3] = idx[7] = -1
    ld = decays(Hv, "edge" if Hv > 2 else "span")
    dc = cache.cuda()
    out = torch.full((n, Hv, V), float("nan"), dtype=dtype, device="cuda")
    o = gdn.linear_attn_decode(q.cuda(), k.cuda(), v.cuda(), ld.cuda(), dc, idx.cuda(), out=out, check=True)
    used = []
    for i in range(n):
        if idx[i] < 0:
            assert torch.count_nonzero(o[i]).item() == 0
            continue
        s = int(idx[i])
        used.append(s)
        o_ref, fin = ref.forward(q[None, i:i + 1], k[None, i:i + 1], v[None, i:i + 1], ld,
                                 h0=cache[s:s + 1])
        assert ref.rel(o[i], o_ref[0, 0]) <= TOL[dtype] and ref.rel(dc[s], fin[0]) <= TOL[F32]
    for s in set(range(slots)) - set(used):
        assert torch.equal(dc[s].cpu(), cache[s])


def test_decode_continues_a_prompt():
    x = make(B=1, T=90, Hqk=2, Hv=4, dtype=F32, seed=81, h0=False)
    c = on_gpu(x)
    o, fin = gdn.chunk_linear_attn(c["q"], c["k"], c["v"], c["log_decay"], output_final_state=True)
    part = [c[n][:, :70].contiguous() for n in ("q", "k", "v")]
    _, cache = gdn.chunk_linear_attn(*part, c["log_decay"], output_final_state=True)
    for t in range(70, 90):
        y = gdn.linear_attn_decode(*(c[n][:, t].contiguous() for n in ("q", "k", "v")), c["log_decay"], cache)
        assert ref.rel(y, o[:, t].double()) <= 2e-5
    assert ref.rel(cache, fin.double()) <= 1e-5


def test_decode_slots_past_32_bit_offsets():
    """A cache of more than 2^31 floats: the slots at its end."""
    slots = 4200
    cache = torch.empty(slots, 32, 128, 128, device="cuda")
    g = torch.Generator().manual_seed(91)
    idx = torch.tensor([slots - 1, 4097, 0], dtype=torch.int32)
    h = torch.randn(3, 32, 128, 128, generator=g)
    for i, s in enumerate(idx.tolist()):
        cache[s] = h[i].cuda()
    q, k, v = (torch.randn(3, 32, 128, generator=g) for _ in range(3))
    ld = decays(32)
    o = gdn.linear_attn_decode(q.cuda(), k.cuda(), v.cuda(), ld.cuda(), cache, idx.cuda())
    for i, s in enumerate(idx.tolist()):
        o_ref, fin = ref.forward(q[None, i:i + 1], k[None, i:i + 1], v[None, i:i + 1], ld, h0=h[i:i + 1])
        assert ref.rel(o[i], o_ref[0, 0]) <= TOL[F32] and ref.rel(cache[s], fin[0]) <= TOL[F32]
    out, _ = gdn.chunk_linear_attn(*(x[:1, None].cuda().contiguous() for x in (q, k, v)), ld.cuda(),
                                   initial_state=cache, output_final_state=True,
                                   state_indices=idx[:1].cuda())
    assert torch.isfinite(out).all()


def test_decode_status_and_identity_slots():
    q = torch.randn(3, 1, 16, device="cuda")
    v = torch.randn(3, 1, 16, device="cuda")
    ld = torch.zeros(1, device="cuda")
    cache = torch.zeros(3, 1, 16, 16, device="cuda")
    o = gdn.linear_attn_decode(q, q, v, ld, cache)
    want = (q * q).sum(-1, keepdim=True) * v / 4
    assert ref.rel(o, want.double()) <= 1e-5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = torch.tensor([0, 3, -2], dtype=torch.int32, device="cuda")
    o = gdn.linear_attn_decode(q, q, v, ld, cache, bad, dev_status=status)
    assert int(status.item()) == _lib.GDN_DEV_BAD_SLOT and torch.count_nonzero(o[1:]).item() == 0


def test_refusals():
    x = on_gpu(make(B=1, T=8, Hqk=2, Hv=4))
    q, k, v, ld = x["q"], x["k"], x["v"], x["log_decay"]
    with pytest.raises(ValueError):
        gdn.chunk_linear_attn(q, k[:, :4].contiguous(), v, ld)
    with pytest.raises(TypeError):
        gdn.chunk_linear_attn(q, k.float(), v, ld)
    with pytest.raises(TypeError):
        gdn.chunk_linear_attn(q.half(), k.half(), v.half(), ld)
    with pytest.raises(ValueError):
        gdn.chunk_linear_attn(q, k, v, ld[:3].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        gdn.chunk_linear_attn(q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), ld)
    with pytest.raises(ValueError):
        gdn.chunk_linear_attn(q, k, v, ld, initial_state=torch.zeros(1, 4, 128, 64, device="cuda"))
    with pytest.raises(ValueError, match="B == 1"):
        y = on_gpu(make(B=2, T=8))
        gdn.chunk_linear_attn(y["q"], y["k"], y["v"], y["log_decay"],
                              cu_seqlens=torch.tensor([0, 8], dtype=torch.int32, device="cuda"))
    with pytest.raises((ValueError, _lib.GdnError)):
        z = torch.zeros(1, 8, 3, 128, device="cuda", dtype=BF16)
        gdn.chunk_linear_attn(q, k, z, torch.zeros(3, device="cuda"))
    with pytest.raises((ValueError, _lib.GdnError)):
        z = torch.zeros(1, 8, 1, 144, device="cuda", dtype=BF16)
        gdn.chunk_linear_attn(z, z, z, torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError):
        gdn.linear_attn_decode(q[0], k[0], v[0], ld, torch.zeros(9, 4, 128, 64, device="cuda"))
    with pytest.raises((ValueError, _lib.GdnError)):
        gdn.linear_attn_decode(q[0], k[0], v[0], ld, torch.zeros(3, 4, 128, 128, device="cuda"))


def test_nothing_to_do():
    q = torch.zeros(0, 5, 1, 16, device="cuda")
    o, fin = gdn.chunk_linear_attn(q, q, q, torch.zeros(1, device="cuda"), output_final_state=True)
    assert o.shape == q.shape and fin.shape[0] == 0
    q = torch.zeros(2, 0, 1, 16, device="cuda")
    h = torch.randn(2, 1, 16, 16, device="cuda")
    o, fin = gdn.chunk_linear_attn(q, q, q, torch.zeros(1, device="cuda"), initial_state=h,
                                   output_final_state=True)
    assert torch.equal(fin, h)
    dq, dk, dv, dh = gdn.chunk_linear_attn_bwd(q, q, q, torch.zeros(1, device="cuda"), q, h)
    assert torch.equal(dh, h) and dq.numel() == 0
    q = torch.ones(1, 6, 1, 16, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")   # no sequence at all
    o, _ = gdn.chunk_linear_attn(q, q, q, torch.zeros(1, device="cuda"), cu_seqlens=cu)
    assert torch.count_nonzero(o).item() == 0
    assert gdn.linear_attn_decode(q[0, :0], q[0, :0], q[0, :0], torch.zeros(1, device="cuda"), h).shape[0] == 0
