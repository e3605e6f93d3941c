"""moe_balance_loss, its backward and moe_router_backward against plain 64-bit
implementations, and with the layer's own routing and backward pass."""
import numpy as np
import pytest
import torch

import workloads
from layer_cases import announce, make_shape, to_device
from operator_cases import U32, as64, balance64

pytestmark = pytest.mark.gpu


def inputs(T, n, k, seed, S=None, mask=False, empty=False):
    rng = np.random.default_rng(seed)
    s = 1 / (1 + np.exp(-rng.standard_normal((T, n)) - 0.5 * rng.standard_normal(n)))
    s = s.astype(np.float32)
    idx = np.argsort(-s, axis=1, kind="stable")[:, :k].astype(np.int32)
    off = None
    if S is not None:
        cuts = np.sort(rng.integers(0, T + 1, S + 1))
        if not empty:
            cuts[0], cuts[-1] = 0, T
        off = cuts.astype(np.int32)
    m = (rng.random(T) < 0.8) if mask else None
    return s, np.ascontiguousarray(idx), off, m


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rounds(T, n):
    """fp32 roundings on the way to q_t and 1/S_t: 16 products and sums in a
    lane, 6 across the wave, the division; the wave's own sum over its tokens."""
    return 2 * (16 + 6) + 4, -(-T // 4096) + 2


def check(out, ref, T, n):
    loss, counts, tokens, grad, size = ref
    row, chain = rounds(T, n)
    assert np.array_equal(out["counts"].cpu().numpy(), counts)
    assert np.array_equal(out["tokens"].cpu().numpy(), tokens)
    got = as64(out["loss"])
    assert (np.abs(got - loss) <= (row + chain + 2) * U32 * loss).all(), (got, loss)
    if "dscores" in out:
        d = np.abs(as64(out["dscores"]) - grad)
        assert (d <= (row + 8) * U32 * size + 1e-44).all(), d.max()


CASES = [  # T, n, k, sequences, mask, tokens outside the sequences
    (1, 1, 1, None, False, False), (1, 8, 2, None, False, False), (64, 32, 4, None, False, False),
    (37, 40, 6, 3, True, False), (200, 64, 4, 7, False, True), (300, 129, 5, 5, True, True),
    (500, 255, 8, 1, True, False), (257, 256, 16, 40, False, False), (129, 260, 3, 9, True, True),
    (96, 512, 2, 4, False, False), (150, 513, 7, 6, True, True), (640, 896, 16, 11, True, True),
    (9000, 36, 4, 13, True, True), (50, 1024, 16, 60, False, True), (77, 1023, 9, 2, True, False),
]


@pytest.mark.parametrize("T,n,k,S,mask,empty", CASES)
def test_balance_loss_and_gradient(T, n, k, S, mask, empty):
    import sparse_moe_ffn_sigmoid_amd as moe
    announce(f"balance T={T} n={n} k={k} S={S} mask={mask} empty={empty}")
    s, idx, off, m = inputs(T, n, k, 7 * T + n, S, mask, empty)
    dloss = np.linspace(-1.0, 2.0, 1 if S is None else S).astype(np.float32)
    ref = balance64(s, idx, off, m, dloss)
    kw = dict(seq_offsets=cuda(off), token_mask=cuda(m))
    r = moe.balance_loss(cuda(s), cuda(idx), dloss=cuda(dloss), want_grad=True, **kw)
    check(r, ref, T, n)
    # the loss alone, and the backward as its own call: the same bits
    f = moe.balance_loss(cuda(s), cuda(idx), **kw)
    assert torch.equal(f["counts"], r["counts"]) and torch.equal(f["loss"], r["loss"])
    g = moe.balance_loss_backward(cuda(s), f["counts"], f["tokens"], k, dloss=cuda(dloss), **kw)
    assert torch.equal(g, r["dscores"])
    # without dloss: ones
    ones = balance64(s, idx, off, m)
    check(moe.balance_loss(cuda(s), cuda(idx), want_grad=True, **kw), ones, T, n)


def test_balance_gradient_is_the_losss():
    """dscores against differences of the 64-bit loss (choices held fixed)."""
    import sparse_moe_ffn_sigmoid_amd as moe
    s, idx, off, m = inputs(23, 12, 3, 5, 2, True)
    announce("balance gradient by differences")
    g = as64(moe.balance_loss(cuda(s), cuda(idx), seq_offsets=cuda(off), token_mask=cuda(m),
                              want_grad=True)["dscores"])
    base = s.astype(np.float64)
    size = balance64(s, idx, off, m)[4]
    h = 1e-5
    for t, e in [(0, 0), (3, 7), (10, 11), (22, 5), (15, 2)]:
        up, down = base.copy(), base.copy()
        up[t, e] += h
        down[t, e] -= h
        d = (balance64(up, idx, off, m)[0].sum() - balance64(down, idx, off, m)[0].sum()) / (2 * h)
        # the gradient's own roundings; a third-derivative term h^2 f / 6 and 1e-16 / h
        assert abs(g[t, e] - d) <= 60 * U32 * size[t, e] + 1e-9


def test_balance_even_routing_has_loss_one():
    import sparse_moe_ffn_sigmoid_amd as moe
    T, n, k = 64, 32, 2
    idx = (np.arange(T)[:, None] * k + np.arange(k)) % n
    announce("balance even counts")
    s = np.random.default_rng(0).random((T, n)).astype(np.float32)
    r = moe.balance_loss(cuda(s), cuda(idx.astype(np.int32)), want_grad=True)
    assert abs(r["loss"].item() - 1) < 60 * U32
    assert r["dscores"].abs().max().item() < 200 * U32 / (s.sum(1).min() * T)


def test_balance_masked_rows_are_not_read_and_odd_indices_not_counted():
    import sparse_moe_ffn_sigmoid_amd as moe
    T, n, k = 90, 100, 4
    s, idx, off, m = inputs(T, n, k, 3, 4, True, True)
    out = ~m
    out[:off[0]] = True
    out[off[-1]:] = True
    s[out] = np.nan
    s[np.nonzero(out)[0][::2]] = np.inf
    live = np.nonzero(~out)[0]
    s[live[0]] = 0.0                       # no shares: no gradient
    idx[live[1], 0] = -1
    idx[live[2]] = n
    idx[live[3]] = 2 ** 31 - 1
    idx[live[4], 1] = idx[live[4], 0]      # the same expert twice counts twice
    announce("balance masked NaN rows")
    ref = balance64(s, idx, off, m)
    r = moe.balance_loss(cuda(s), cuda(idx), seq_offsets=cuda(off), token_mask=cuda(m),
                         want_grad=True)
    check(r, ref, T, n)
    assert (as64(r["dscores"])[out] == 0).all() and (as64(r["dscores"])[live[0]] == 0).all()


def test_balance_strided_rows_nothing_to_do_and_all_masked():
    import sparse_moe_ffn_sigmoid_amd as moe
    s, idx, off, m = inputs(60, 44, 3, 9)
    for lead, width in ((0, 45), (4, 52), (1, 48)):
        announce(f"balance strided {lead} {width}")
        wide = torch.full((60, width + lead), float("nan"), device="cuda")
        view = wide[:, lead:lead + 44]
        view.copy_(cuda(s))
        r = moe.balance_loss(view, cuda(idx), want_grad=True)
        check(r, balance64(s, idx), 60, 44)
        assert torch.equal(moe.balance_loss_backward(view, r["counts"], r["tokens"], 3), r["dscores"])
    announce("balance T=0 and all masked")
    r = moe.balance_loss(torch.empty((0, 16), device="cuda"),
                         torch.empty((0, 2), dtype=torch.int32, device="cuda"), want_grad=True)
    assert r["loss"].item() == 0 and r["tokens"].item() == 0 and not r["counts"].any()
    assert r["dscores"].shape == (0, 16)
    r = moe.balance_loss(cuda(s), cuda(idx), token_mask=torch.zeros(60, dtype=torch.bool,
                                                                    device="cuda"), want_grad=True)
    assert r["loss"].item() == 0 and not r["counts"].any() and not r["dscores"].any()


def test_balance_large_batch():
    """The routing-only batch: counts against torch's, loss and gradient in
    float64 on the device."""
    import sparse_moe_ffn_sigmoid_amd as moe
    T, n, k = 57344, 896, 16
    announce("balance 57344 x 896")
    s = torch.sigmoid(torch.randn((T, n), generator=torch.Generator("cuda").manual_seed(1),
                                  device="cuda"))
    idx = torch.topk(s, k, dim=1)[1].to(torch.int32)
    off = torch.tensor([0, 5, 5, 20000, 57344], dtype=torch.int32, device="cuda")
    r = moe.balance_loss(s, idx, seq_offsets=off, want_grad=True)
    row, chain = rounds(T, n)
    for q in range(4):
        b, e = int(off[q]), int(off[q + 1])
        c = torch.bincount(idx[b:e].flatten().long(), minlength=n).double()
        assert torch.equal(r["counts"][q].double(), c)
        if e == b:
            assert r["loss"][q].item() == 0
            continue
        S = s[b:e].double().sum(1)
        inner = (s[b:e].double() @ c) / S
        w = n / (k * (e - b) ** 2)
        loss = (w * inner.sum()).item()
        assert abs(r["loss"][q].item() - loss) <= (row + chain + 2) * U32 * loss
        g = w / S[:, None] * (c - inner[:, None])
        size = w / S[:, None] * (c + inner[:, None])
        assert ((r["dscores"][b:e].double() - g).abs() <= (row + 8) * U32 * size).all()


def test_balance_graph_replays_and_streams():
    import sparse_moe_ffn_sigmoid_amd as moe
    T, n, k = 700, 96, 4
    s1, i1, off, m = inputs(T, n, k, 21, 5, True, True)
    s2, i2, _, _ = inputs(T, n, k, 22)
    announce("balance graph")
    a = [cuda(s1), cuda(i1)]
    kw = dict(seq_offsets=cuda(off), token_mask=cuda(m), want_grad=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = moe.balance_loss(*a, **kw)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    check(warm, balance64(s1, i1, off, m), T, n)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = moe.balance_loss(*a, **kw)
    for rep in range(4):
        s, i = ((s2, i2), (s1, i1))[rep % 2]
        a[0].copy_(cuda(s))
        a[1].copy_(cuda(i))
        g.replay()
        torch.cuda.synchronize()
        got = {key: v.clone() for key, v in r.items()}
        eager = moe.balance_loss(*a, **kw)
        for key in r:
            assert torch.equal(got[key], eager[key]), key


# --- router backward --------------------------------------------------------
def router64(x, w, s, ds):
    g = ds * s * (1 - s)
    return g, g @ w, g.T @ x, g.sum(0)


@pytest.mark.parametrize("T,d,n", [(1, 64, 1), (5, 64, 7), (64, 128, 64), (200, 512, 40),
                                   (333, 192, 129), (130, 1024, 896), (700, 64, 1024), (200, 512, 80), (1, 64, 1024),
                                   (1024, 64, 5)])
def test_router_backward(T, d, n):
    import sparse_moe_ffn_sigmoid_amd as moe
    rng = np.random.default_rng(T + d + n)
    announce(f"router backward T={T} d={d} n={n}")
    x = torch.from_numpy(rng.standard_normal((T, d))).to(torch.bfloat16).cuda()
    w = cuda((rng.standard_normal((n, d)) * d ** -0.5).astype(np.float32))
    s = cuda((1 / (1 + np.exp(-rng.standard_normal((T, n))))).astype(np.float32))
    ds = cuda((rng.standard_normal((T, n)) * 1e-3).astype(np.float32))
    g, dx, dw, doff = router64(as64(x), as64(w), as64(s), as64(ds))
    # g: a difference and two products in fp32 (the difference is exact to 2^-24
    # of 1, the products to 2^-24 each)
    s64 = as64(s)
    ge = np.abs(as64(ds)) * s64 * U32 + 3 * U32 * np.abs(g)
    ax, aw = np.abs(as64(x)), np.abs(as64(w))
    # sums of up to 3 (T + 64) exact products, each addition to 2^-23 of the sum
    bw = ge.T @ ax + 3 * (T + 64) * 2.0 ** -23 * (np.abs(g).T @ ax) + 1e-40
    # two bf16 parts leave 2^-16 of a value; the product of the low parts is left out
    size = np.abs(g) @ aw
    bx = ge @ aw + (3 * 2.0 ** -16 + 3 * (n + 64) * 2.0 ** -23) * size
    bx = bx + 2.0 ** -8 * (np.abs(dx) + bx) + 1e-38
    boff = ge.sum(0) + 70 * U32 * np.abs(g).sum(0) + 1e-40
    r = moe.router_backward(x, w, s, ds)
    assert (np.abs(as64(r["d_w_router"]) - dw) <= bw).all()
    assert (np.abs(as64(r["dx"]) - dx) <= bx).all()
    assert (np.abs(as64(r["d_router_logit_offset"]) - doff) <= boff).all()
    # added to gradients that are there; what is None is left out
    into = dict(dx=torch.ones_like(x), d_w_router=torch.full_like(w, 2.0),
                d_router_logit_offset=None, other=None)
    assert moe.router_backward(x, w, s, ds, into=into) is into
    assert (np.abs(as64(into["d_w_router"]) - (dw + 2)) <= bw + U32 * (np.abs(dw) + 2)).all()
    b1 = bx + 2.0 ** -8 * (np.abs(dx) + 1)
    assert (np.abs(as64(into["dx"]) - (dx + 1)) <= b1).all()


def test_router_backward_no_tokens():
    import sparse_moe_ffn_sigmoid_amd as moe
    announce("router backward T=0")
    z = lambda *sh, dt=torch.float32: torch.empty(sh, dtype=dt, device="cuda")
    w = torch.ones((8, 64), device="cuda")
    r = moe.router_backward(z(0, 64, dt=torch.bfloat16), w, z(0, 8), z(0, 8))
    assert not r["d_w_router"].any() and not r["d_router_logit_offset"].any()
    into = dict(dx=None, d_w_router=w.clone(), d_router_logit_offset=None)
    moe.router_backward(z(0, 64, dt=torch.bfloat16), w, z(0, 8), z(0, 8), into=into)
    assert torch.equal(into["d_w_router"], w)


def test_balance_loss_in_a_training_step():
    """Forward, balance loss, backward with the loss's gradient: the layer's
    gradients plus the loss's own, by a route of its own in 64 bits."""
    import sparse_moe_ffn_sigmoid_amd as moe
    shape = workloads.small_shape(T=160, n=24, k=4)
    announce("balance loss in a training step")
    inp = workloads.layer_inputs(shape, "cpu", seed=5)
    x, w = to_device(inp)
    w["router_logit_offset"] = w.pop("logit_offset")
    sh = make_shape(moe, shape, qb_mode=0)
    f = moe.latent_forward(sh, w, x, want_scores=True)
    dout = torch.randn((shape.T, shape.d), generator=torch.Generator("cuda").manual_seed(2),
                       device="cuda").to(torch.bfloat16)
    off = torch.tensor([0, 70, 160], dtype=torch.int32, device="cuda")
    dl = torch.full((2,), 5.0, device="cuda")
    b = moe.balance_loss(f["scores"], f["idx"], seq_offsets=off, dloss=dl, want_grad=True)
    assert torch.equal(b["counts"].sum(0).int(), f["loads"])
    plain = moe.latent_backward(sh, w, x, f["scores"], f["idx"], f["w"], dout)
    both = moe.latent_backward(sh, w, x, f["scores"], f["idx"], f["w"], dout,
                               dscores=b["dscores"])
    s, ds = as64(f["scores"]), as64(b["dscores"])
    g, dx, dw, doff = router64(as64(x), as64(w["w_router"]), s, ds)
    for name, add, half in (("d_w_router", dw, 1e-5), ("d_router_logit_offset", doff, 1e-5)):
        want = as64(plain[name]) + add
        assert np.linalg.norm(as64(both[name]) - want) <= half * np.linalg.norm(want) + 1e-9
    want = as64(plain["dx"]) + dx
    assert (np.abs(as64(both["dx"]) - want) <=
            2.0 ** -8 * np.abs(want) + 4 * 2.0 ** -16 * (np.abs(g) @ np.abs(as64(w["w_router"])))
            ).all()
    for name in plain:
        if name not in ("dx", "d_w_router", "d_router_logit_offset"):
            assert torch.equal(plain[name], both[name]), name
    # the training forward's saved activations take the same path
    saved = torch.empty(moe.saved_activations_bytes(sh), dtype=torch.uint8, device="cuda")
    f2 = moe.latent_forward(sh, w, x, want_scores=True, saved=saved)
    tr = moe.latent_backward_train(sh, w, x, f2["scores"], f2["idx"], f2["w"], dout, saved,
                                   dscores=b["dscores"])
    want = as64(both["d_w_router"])
    assert np.linalg.norm(as64(tr["d_w_router"]) - want) <= 1e-2 * np.linalg.norm(want)
    for bad in (b["dscores"].double(), b["dscores"][:, :-1], b["dscores"].cpu()):
        with pytest.raises(ValueError):
            moe.latent_backward(sh, w, x, f["scores"], f["idx"], f["w"], dout, dscores=bad)
    with pytest.raises(ValueError):
        moe.latent_backward_train(sh, w, x, f2["scores"], f2["idx"], f2["w"], dout, saved, lr=0.1,
                                  dscores=b["dscores"])


def test_balance_rows_beyond_4_gib():
    import sparse_moe_ffn_sigmoid_amd as moe
    T, n, k = 1 << 20, 1024, 2                              # 4.3 GB of scores
    announce("balance 2^20 x 1024")
    s = torch.zeros((T, n), device="cuda")
    s[:, :7] = 0.25
    s[-3:] = torch.rand((3, n), generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    idx = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    idx[:, 1] = torch.arange(T, device="cuda") % n
    off = torch.tensor([0, T - 3, T], dtype=torch.int32, device="cuda")
    r = moe.balance_loss(s, idx, seq_offsets=off, want_grad=True)
    loss, counts, tokens, grad, size = balance64(s[-3:].cpu().numpy(), idx[-3:].cpu().numpy())
    assert np.array_equal(r["counts"][1].cpu().numpy(), counts[0]) and r["tokens"].tolist() == [T - 3, 3]
    assert r["counts"][0].sum().item() == (T - 3) * k
    row, chain = rounds(T, n)
    assert abs(r["loss"][1].item() - loss[0]) <= (row + chain) * U32 * loss[0]
    assert (np.abs(as64(r["dscores"][-3:]) - grad) <= (row + 8) * U32 * size + 1e-44).all()
    with pytest.raises(moe.MoeError):
        moe.balance_loss(s, idx, seq_offsets=off, workspace=torch.empty(256, dtype=torch.uint8,
                                                                        device="cuda"))


@pytest.mark.parametrize("T", [64, 600])
def test_balance_scores_near_the_smallest(T):
    """Rows whose sum's reciprocal overflows fp32 still have shares and gradients."""
    import sparse_moe_ffn_sigmoid_amd as moe
    n, k = 32, 4
    announce(f"balance of tiny scores T={T}")
    s, idx, off, m = inputs(T, n, k, T)
    s = np.ldexp(np.round(s * 512) / 512 + 2.0 ** -9, -138).astype(np.float32)  # exact, sums too
    ref = balance64(s, idx)
    r = moe.balance_loss(cuda(s), cuda(idx), want_grad=True)
    # dot = sum c s rounds to whole denormals, 2^-149, at most n times a row
    extra = n * 2.0 ** -149 / s.sum(1, dtype=np.float64).min()
    loss, counts, tokens, grad, size = ref
    row, chain = rounds(T, n)
    w = n / (k * T * T)
    assert abs(as64(r["loss"])[0] - loss[0]) <= (row + chain + 2) * U32 * loss[0] + w * T * extra
    bound = (row + 8) * U32 * size + w / s.sum(1, dtype=np.float64)[:, None] * extra
    got = as64(r["dscores"])
    # 1 / S_t is about 2^134 here: a gradient past fp32's largest value is an
    # infinity of its sign, every other one is that value
    most = float(torch.finfo(torch.float32).max)
    sure = np.abs(grad) > most + bound
    assert (got[sure] == np.sign(grad[sure]) * np.inf).all()
    fits = np.abs(grad) + bound < most
    assert fits.any() and (np.abs(got - grad)[fits] <= bound[fits]).all()
    assert not np.isnan(got).any()


def test_router_backward_beyond_4_gib():
    import sparse_moe_ffn_sigmoid_amd as moe
    T, d, n = 300032, 7168, 36                              # 4.3 GB of x
    announce("router backward 300032 x 7168")
    gen = torch.Generator("cuda").manual_seed(3)
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    x[-500:] = torch.randn((500, d), generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.randn((n, d), generator=gen, device="cuda") * d ** -0.5
    s = torch.rand((T, n), generator=gen, device="cuda")
    ds = torch.randn((T, n), generator=gen, device="cuda") * 1e-3
    r = moe.router_backward(x, w, s, ds)
    xe, we, se, de = as64(x[-500:]), as64(w), as64(s[-500:]), as64(ds[-500:])
    g, dx, dw, _ = router64(xe, we, se, de)
    # the terms of every bound as in test_router_backward
    ge = np.abs(de) * se * U32 + 3 * U32 * np.abs(g)
    size = np.abs(g) @ np.abs(we)
    bx = ge @ np.abs(we) + (3 * 2.0 ** -16 + 3 * (n + 64) * 2.0 ** -23) * size
    bx = bx + 2.0 ** -8 * (np.abs(dx) + bx) + 1e-38
    assert (np.abs(as64(r["dx"][-500:]) - dx) <= bx).all()
    # rows of zeros add nothing: the sum has the last 500 rows' terms, rounded
    # once more for each part it is split into, at most one per 64 rows
    bw = ge.T @ np.abs(xe) + 3 * (500 + T // 64) * 2.0 ** -23 * (np.abs(g).T @ np.abs(xe)) + 1e-40
    assert (np.abs(as64(r["d_w_router"]) - dw) <= bw).all()
    g = ds.double() * s.double() * (1 - s.double())
    off = (r["d_router_logit_offset"].double() - g.sum(0)).abs()
    assert (off <= (3 + 64 + 2) * U32 * ((ds.double() * s.double()).abs().sum(0))).all()


def test_balance_refusals_on_the_device():
    import sparse_moe_ffn_sigmoid_amd as moe
    announce("balance refusals")
    s = torch.rand((8, 16), device="cuda")
    i = torch.zeros((8, 2), dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    for bad in (lambda: moe.balance_loss(s.double(), i), lambda: moe.balance_loss(s[0], i),
                lambda: moe.balance_loss(s[:, ::2], i), lambda: moe.balance_loss(s, i.long()),
                lambda: moe.balance_loss(s, i[:4]), lambda: moe.balance_loss(s, i.cpu()),
                lambda: moe.balance_loss(s, i, seq_offsets=off.long()),
                lambda: moe.balance_loss(s, i, token_mask=torch.ones(7, dtype=torch.bool,
                                                                     device="cuda")),
                lambda: moe.balance_loss(s, i, seq_offsets=off, dloss=torch.ones(2, device="cuda")),
                lambda: moe.balance_loss_backward(s, i, off, 2),
                lambda: moe.router_backward(s, s, s, s),
                lambda: moe.router_backward(s.bfloat16(), s, s, s)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: moe.balance_loss(torch.rand((4, 1025), device="cuda"), i[:4]),
                lambda: moe.balance_loss(s[:, :1], i)):       # more choices than experts
        with pytest.raises(moe.MoeError):
            bad()
