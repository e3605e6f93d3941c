"""Workloads of the router's balance loss and of the MXFP4 products.

Each case is one pass through an operator as a program that trains or serves
the layer calls it: the sequence-wise balance loss of the router with its
per-expert counts and gradient, the gradient of the router's scores taken to
its weights and tokens, MXFP4 packing along rows and columns, and products of
MXFP4 operands (one matrix, a matrix per expert, and the experts' weight
gradients).  With ``own`` false a pass runs in elementary torch operations,
with ``own`` true through the package's entry points; ``exact`` gives the
results in 64 bits from the operators' definitions.
"""
from __future__ import annotations

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def listed():
    return [
        # the 64-token test layer's router, loss and gradient in one call: latency
        dict(name="balance_small", kind="balance", mode="train", T=64, n=32, k=4, S=1, mask=False),
        # a packed training batch of ragged sequences with padding tokens, the
        # loss and its backward as two calls of a training loop
        dict(name="balance_ragged", kind="balance", mode="two", T=16384, n=896, k=16, S=11,
             mask=True),
        # the routing-only batch: loss, counts and gradient in one call
        dict(name="balance_57344", kind="balance", mode="train", T=57344, n=896, k=16, S=14,
             mask=False),
        # the small parity layer: the scores' gradient to weights and tokens
        dict(name="router_grad_small", kind="router", T=200, d=512, n=40),
        # the prefill layer's router at training
        dict(name="router_grad_4096", kind="router", T=4096, d=7168, n=896),
        # fp32 master rows of an odd width out of a wider matrix
        dict(name="pack_f32_odd", kind="pack", dtype="f32", rows=997, K=2043, extra=5, cols=False),
        # a long batch's tokens, packed for the forward and for the weight gradient
        dict(name="pack_16384", kind="pack", dtype="bf16", rows=16384, K=7168, extra=0, cols=True),
        # one token through the latent down-projection
        dict(name="linear_1", kind="linear", dtype="bf16", T=1, K=7168, N=3584),
        # a training step of that projection: output, dx and dW
        dict(name="linear_train", kind="train", T=4096, K=7168, N=3584),
        # decode: 64 tokens on 16 of 896 experts each
        dict(name="experts_64", kind="experts", T=64, E=896, k=16, K=3584, N=2048, balanced=False),
        # the 16,384-token batch, balanced
        dict(name="experts_16384", kind="experts", T=16384, E=896, k=16, K=3584, N=2048,
             balanced=True),
        # a training step of some experts with ragged loads, one of them unused
        dict(name="experts_train", kind="experts_train", R=4681, E=24, K=3584, N=2048),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["balance", "balance", "router", "pack", "linear", "train", "experts",
                       "experts_train"])
    if kind == "balance":
        n = _log(rng, 8, 1024)
        T = _log(rng, 1, 57344)
        return dict(kind=kind, mode=rng.choice(["train", "two"]), T=T, n=n,
                    k=rng.randint(1, min(16, n)), S=rng.randint(1, 16), mask=rng.random() < 0.5)
    if kind == "router":
        return dict(kind=kind, T=_log(rng, 16, 4096), d=64 * _log(rng, 4, 112),
                    n=_log(rng, 8, 896))
    if kind == "pack":
        return dict(kind=kind, dtype=rng.choice(sorted(DTYPES)), rows=_log(rng, 1, 16384),
                    K=_log(rng, 1, 7168), extra=rng.choice([0, 0, 3, 8]), cols=rng.random() < 0.5)
    if kind == "linear":
        return dict(kind=kind, dtype=rng.choice(sorted(DTYPES)), T=_log(rng, 1, 700),
                    K=32 * _log(rng, 1, 224), N=_log(rng, 16, 7168))
    if kind == "train":
        return dict(kind=kind, T=_log(rng, 32, 4096), K=_log(rng, 64, 7168), N=_log(rng, 64, 3584))
    if kind == "experts":
        E = _log(rng, 4, 256)
        return dict(kind=kind, T=_log(rng, 1, 8192), E=E, k=rng.randint(1, min(8, E)),
                    K=32 * _log(rng, 2, 112), N=_log(rng, 32, 2048), balanced=rng.random() < 0.5)
    return dict(kind=kind, R=_log(rng, 40, 4681), E=_log(rng, 2, 24), K=_log(rng, 64, 2048),
                N=_log(rng, 64, 2048))


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 131 + salt)
    return g


def _normal(shape, seed, salt, std=1.0, dtype=torch.float32):
    t = torch.randn(shape, generator=_gen(seed, salt), device="cuda")
    return t.mul_(std).to(dtype)


def _scores(T, n, seed):
    """Sigmoid scores of logits N(0, 1) plus a per-expert offset N(0, 0.5^2)."""
    return torch.sigmoid(_normal((T, n), seed, 1) + _normal((n,), seed, 2, 0.5))


def _sequences(T, S, seed):
    """Offsets [S + 1]: random cuts, the last sequence ending before the batch
    does where there are several (the rest is padding)."""
    if S == 1:
        return np.array([0, T], np.int32)
    rng = np.random.default_rng([seed, 3])
    return np.concatenate([[0], np.sort(rng.integers(0, T + 1, S))]).astype(np.int32)


def _loads(R, E, balanced, seed):
    """Rows per expert: equal, or from random popularities, one expert unused."""
    rng = np.random.default_rng([seed, 4])
    if balanced:
        return np.full(E, R // E) + (np.arange(E) < R % E)
    pop = np.exp(0.5 * rng.standard_normal(E))
    pop[rng.integers(E)] = 0.0 if E > 1 else 1.0
    return rng.multinomial(R, pop / pop.sum())


def _offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _mx_codes(w):
    """Rows [.., K] (K % 32 == 0) to MXFP4 codes [.., K/2] and scales [.., K/32]."""
    v, e = _mx_grid(w.float())
    mag = v.abs()
    code = torch.where(mag < 2, mag * 2, torch.where(mag < 4, mag + 2, mag * 0.5 + 4))
    code = code.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), (e + 127).to(torch.uint8)


def _packed_weights(E, N, K, seed):
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, N, K // 32), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, E, step):
        c = min(E, e + step)
        codes[e:c], scales[e:c] = _mx_codes(_normal((c - e, N, K), seed, 100 + e, K ** -0.5))
    return codes, scales


def prepare(case, seed):
    kind = case["kind"]
    st = dict(case)
    if kind == "balance":
        T, n, k, S = case["T"], case["n"], case["k"], case["S"]
        st["scores"] = _scores(T, n, seed)
        bias = _normal((n,), seed, 5, 0.05)
        st["idx"] = torch.topk(st["scores"] + bias, k, dim=1)[1].to(torch.int32)
        st["offsets"] = torch.from_numpy(_sequences(T, S, seed)).cuda()
        st["mask"] = None
        if case["mask"]:
            st["mask"] = (torch.rand(T, generator=_gen(seed, 6), device="cuda") < 0.9)
        # the coefficient of the loss over the number of sequences, as a
        # training program weighs it
        st["dloss"] = torch.full((S,), 1e-4 / S, device="cuda")
    elif kind == "router":
        T, d, n = case["T"], case["d"], case["n"]
        st["x"] = _normal((T, d), seed, 1, 1.0, torch.bfloat16)
        st["w"] = _normal((n, d), seed, 2, d ** -0.5)
        st["scores"] = torch.sigmoid(st["x"].float() @ st["w"].T + _normal((n,), seed, 3, 0.5))
        st["dscores"] = _normal((T, n), seed, 4, 1e-3)
    elif kind == "pack":
        rows, K, extra = case["rows"], case["K"], case["extra"]
        wide = _normal((rows, K + extra), seed, 1)
        wide *= torch.exp(_normal((K + extra,), seed, 2))     # channels of unlike sizes
        st["x"] = wide.to(DTYPES[case["dtype"]])[:, :K]
    elif kind == "linear":
        st["x"] = _normal((case["T"], case["K"]), seed, 1, 1.0, DTYPES[case["dtype"]])
        c, s = _packed_weights(1, case["N"], case["K"], seed)
        st["codes"], st["scales"] = c[0], s[0]
    elif kind == "train":
        T, K, N = case["T"], case["K"], case["N"]
        st["x"] = _normal((T, K), seed, 1, 1.0, torch.bfloat16)
        st["w"] = _normal((N, K), seed, 2, K ** -0.5, torch.bfloat16)
        st["dy"] = _normal((T, N), seed, 3, 1e-3, torch.bfloat16)
    elif kind == "experts":
        T, E, k = case["T"], case["E"], case["k"]
        lens = _loads(T * k, E, case["balanced"], seed)
        st["offsets"], st["most"] = _offsets(lens), int(lens.max())
        # every token k times, ascending within each expert
        token = torch.randperm(T * k, generator=_gen(seed, 2), device="cuda") % T
        expert = torch.repeat_interleave(torch.arange(E, device="cuda"),
                                         torch.from_numpy(lens).cuda())
        st["rows"] = torch.sort(expert * T + token)[0].remainder(T).to(torch.int32)
        st["x"] = _normal((T, case["K"]), seed, 1, 1.0, torch.bfloat16)
        st["codes"], st["scales"] = _packed_weights(E, case["N"], case["K"], seed)
    else:
        R, E, K, N = case["R"], case["E"], case["K"], case["N"]
        lens = _loads(R, E, False, seed)
        st["offsets"], st["most"] = _offsets(lens), int(lens.max())
        st["x"] = _normal((R, K), seed, 1, 1.0, torch.bfloat16)
        st["w"] = _normal((E, N, K), seed, 2, K ** -0.5, torch.bfloat16)
        st["dy"] = _normal((R, N), seed, 3, 1e-3, torch.bfloat16)
    return st


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------
def _pow2(e):
    """2^e for whole e in [-1022, 1023], exactly (pow() and ldexp() may round)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _mx_grid(x):
    """Blocks of 32 along the last axis (zeros behind its end) on the E2M1 grid:
    (elements [.., blocks, 32] over the block's scale, scale exponents)."""
    K = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, -K % 32)).unflatten(-1, (-1, 32))
    amax = x.abs().amax(-1)
    e = torch.frexp(amax)[1] - 3                        # floor(log2 amax) - 2
    e = torch.where(amax > 0, e, -127).clamp(-127, 127)
    a = x * _pow2(-e).float()[..., None]
    m = a.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    r = (torch.round(m / step) * step).clamp(max=6.0)   # round() takes ties to even
    return torch.copysign(r, a), e


def _mx_round(x):
    """The values of x [.., K] after MXFP4 rounding along the last axis, fp32."""
    v, e = _mx_grid(x.float())
    return (v * _pow2(e).float()[..., None]).flatten(-2)[..., :x.shape[-1]]


def _mx_round_cols(x):
    return _mx_round(x.transpose(-1, -2).contiguous())


def _mx_decode(codes, scales):
    """MXFP4 codes [.., K/2] and scales [.., K/32] to fp32 values [.., K]."""
    mag = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    one = torch.cat([mag, -mag])
    byte = torch.arange(256, device=codes.device)
    pair = torch.stack([one[byte & 15], one[byte >> 4]], dim=1)
    v = pair[codes.int()].flatten(-2).unflatten(-1, (-1, 32))
    v *= _pow2(scales.int() - 127).float()[..., None]
    return v.flatten(-2)


def _members(st):
    """[S, T] one where a counted token belongs to a sequence."""
    t = torch.arange(st["T"], device="cuda")
    off = st["offsets"].long()
    m = (t >= off[:-1, None]) & (t < off[1:, None])
    return m if st["mask"] is None else m & st["mask"]


def _balance_plain(st):
    T, n, k, S = st["T"], st["n"], st["k"], st["S"]
    scores = st["scores"].float()
    member = _members(st)
    tokens = member.sum(1, dtype=torch.int32)
    seq = torch.where(member.any(0), member.int().argmax(0), S)      # S: not counted
    counts = torch.zeros((S + 1) * n, dtype=torch.int32, device="cuda")
    where = (seq[:, None] * n + st["idx"]).flatten()
    counts = counts.scatter_add_(0, where, torch.ones_like(where, dtype=torch.int32))
    counts = counts.view(S + 1, n)[:S]
    share = scores / scores.sum(1, keepdim=True)
    many = tokens.clamp(min=1).float()
    f = counts.float() * (n / k) / many[:, None]
    loss = (f * (member.float() @ share)).sum(1) / many
    # gradient
    weight = torch.cat([st["dloss"] / many, torch.zeros(1, device="cuda")])[seq]
    fs = torch.cat([f, torch.zeros((1, n), device="cuda")])[seq]
    grad = (fs - (fs * share).sum(1, keepdim=True)) * (weight / scores.sum(1))[:, None]
    return dict(loss=loss, counts=counts, tokens=tokens, dscores=grad)


def _router_plain(st):
    s = st["scores"].float()
    g = st["dscores"].float() * s * (1 - s)
    return dict(dx=(g @ st["w"].float()).to(torch.bfloat16), d_w_router=g.T @ st["x"].float(),
                d_offset=g.sum(0))


def _pad_groups(st, x):
    """Rows [R, K] to [E, most, K], zeros behind each expert's rows."""
    off = st["offsets"].long()
    at = off[:-1, None] + torch.arange(st["most"], device="cuda")
    return x[at.clamp(max=x.shape[0] - 1)] * (at < off[1:, None])[..., None]


def _unpad_groups(st, y, R):
    off = st["offsets"].long()
    r = torch.arange(R, device="cuda")
    e = torch.bucketize(r, off[1:], right=True)
    return y[e, r - off[e]]


def _plain(st):
    kind = st["kind"]
    if kind == "balance":
        return _balance_plain(st)
    if kind == "router":
        return _router_plain(st)
    if kind == "pack":
        r = dict(values=_mx_round(st["x"]))
        if st["cols"]:
            r["values_t"] = _mx_round_cols(st["x"])
        return {key: v.to(torch.bfloat16) for key, v in r.items()}
    if kind == "linear":
        w = _mx_decode(st["codes"], st["scales"])
        return (_mx_round(st["x"]) @ w.T).to(st["x"].dtype)
    if kind == "train":
        x, w, dy = st["x"], st["w"], st["dy"]
        return dict(y=(_mx_round(x) @ _mx_round(w).T).to(torch.bfloat16),
                    dx=(_mx_round(dy) @ _mx_round_cols(w).T).to(torch.bfloat16),
                    dw=_mx_round_cols(dy) @ _mx_round_cols(x).T)
    if kind == "experts":
        w = _mx_decode(st["codes"], st["scales"])
        x = _mx_round(st["x"])[st["rows"].long()]
        y = torch.bmm(_pad_groups(st, x), w.transpose(1, 2))
        return _unpad_groups(st, y, x.shape[0]).to(torch.bfloat16)
    x, w, dy, R = st["x"].float(), st["w"], st["dy"].float(), st["R"]
    y = torch.bmm(_mx_round(_pad_groups(st, x)), _mx_round(w).transpose(1, 2))
    dx = torch.bmm(_mx_round(_pad_groups(st, dy)), _mx_round_cols(w).transpose(1, 2))
    dw = torch.bmm(_mx_round_cols(_pad_groups(st, dy)),
                   _mx_round_cols(_pad_groups(st, x)).transpose(1, 2))
    return dict(y=_unpad_groups(st, y, R).to(torch.bfloat16),
                dx=_unpad_groups(st, dx, R).to(torch.bfloat16), dw=dw)


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def _own(st):
    import sparse_moe_ffn_sigmoid_amd as moe
    kind = st["kind"]
    if kind == "balance":
        if st["mode"] == "train":
            r = moe.balance_loss(st["scores"], st["idx"], seq_offsets=st["offsets"],
                                 token_mask=st["mask"], dloss=st["dloss"], want_grad=True)
            return {key: r[key] for key in ("loss", "counts", "tokens", "dscores")}
        r = moe.balance_loss(st["scores"], st["idx"], seq_offsets=st["offsets"],
                             token_mask=st["mask"])
        g = moe.balance_loss_backward(st["scores"], r["counts"], r["tokens"], st["k"],
                                      seq_offsets=st["offsets"], token_mask=st["mask"],
                                      dloss=st["dloss"])
        return dict(loss=r["loss"], counts=r["counts"], tokens=r["tokens"], dscores=g)
    if kind == "router":
        r = moe.router_backward(st["x"], st["w"], st["scores"], st["dscores"])
        return dict(dx=r["dx"], d_w_router=r["d_w_router"],
                    d_offset=r["d_router_logit_offset"])
    if kind == "pack":
        p = moe.mxfp4_pack(st["x"], cols=st["cols"])
        r = dict(values=moe.mxfp4_unpack(p["codes"], p["scales"], st["K"], torch.bfloat16))
        if st["cols"]:
            r["values_t"] = moe.mxfp4_unpack(p["codes_t"], p["scales_t"], st["rows"],
                                             torch.bfloat16)
        return r
    if kind == "linear":
        return moe.mxfp4_linear(st["x"], st["codes"], st["scales"])
    if kind == "experts":
        return moe.mxfp4_linear(st["x"], st["codes"], st["scales"], offsets=st["offsets"],
                                rows=st["rows"])
    off = st.get("offsets")
    x = moe.mxfp4_pack(st["x"], cols=True, offsets=off)
    w = moe.mxfp4_pack(st["w"], cols=True)
    dy = moe.mxfp4_pack(st["dy"], cols=True, offsets=off)
    dw = moe.mxfp4_matmul_kgroup(dy["codes_t"], dy["scales_t"], x["codes_t"], x["scales_t"],
                                 offsets=dy["offsets_t"] if off is not None else None)
    return dict(y=moe.mxfp4_matmul(x["codes"], x["scales"], w["codes"], w["scales"], offsets=off),
                dx=moe.mxfp4_matmul(dy["codes"], dy["scales"], w["codes_t"], w["scales_t"],
                                    offsets=off),
                dw=dw)


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# Bytes and operations of a pass
# --------------------------------------------------------------------------
def work(case):
    c, kind = case, case["kind"]
    if kind == "balance":
        reads = 4 * c["T"] * (c["n"] + c["k"]) + (c["T"] if c["mask"] else 0)
        writes = 4 * c["T"] * c["n"] + 4 * c["S"] * (c["n"] + 2)
        if c["mode"] == "two":       # two calls: the backward reads the scores again
            reads += 4 * c["T"] * c["n"] + 4 * c["S"] * c["n"]
        return dict(bytes=reads + writes, flops=8 * c["T"] * c["n"])
    if kind == "router":
        T, d, n = c["T"], c["d"], c["n"]
        return dict(bytes=2 * 2 * T * d + 2 * 4 * n * d + 2 * 4 * T * n + 4 * n,
                    flops=2 * 2 * T * n * d)
    if kind == "pack":
        # the rows in, and each direction's rounded values out
        n = c["rows"] * c["K"]
        size = 4 if c["dtype"] == "f32" else 2
        sides = 2 if c["cols"] else 1
        return dict(bytes=n * (size + 2 * sides), flops=4 * n * sides)
    if kind == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        size = 4 if c["dtype"] == "f32" else 2
        return dict(bytes=size * T * (K + N) + N * K // 2 + N * K // 32, flops=2 * T * N * K)
    if kind == "train":
        T, K, N = c["T"], c["K"], c["N"]
        return dict(bytes=2 * (T * K + N * K + T * N) + 2 * (T * N + T * K) + 4 * N * K,
                    flops=3 * 2 * T * N * K)
    if kind == "experts":
        T, E, K, N, R = c["T"], c["E"], c["K"], c["N"], c["T"] * c["k"]
        used = E if R >= E else R
        return dict(bytes=2 * T * K + 4 * R + used * N * (K // 2 + K // 32) + 2 * R * N,
                    flops=2 * R * N * K)
    R, E, K, N = c["R"], c["E"], c["K"], c["N"]
    return dict(bytes=2 * (R * K + E * N * K + R * N) + 2 * (R * N + R * K) + 4 * E * N * K,
                flops=3 * 2 * R * N * K)


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------
def _round64(x):
    """MXFP4 rounding of float64 x along its last axis, by comparison with the
    points halfway between neighbours (a tie goes to the even code)."""
    K = x.shape[-1]
    full = torch.zeros(x.shape[:-1] + (-(-K // 32) * 32,), dtype=torch.float64, device=x.device)
    full[..., :K] = x
    b = full.reshape(x.shape[:-1] + (-1, 32))
    top = b.abs().max(-1, keepdim=True)[0]
    # floor(log2 top), put right where the logarithm rounds across a power of two
    low = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    low = torch.where(_pow2(low) > top, low - 1, low)
    low = torch.where(_pow2(low + 1) <= top, low + 1, low)
    unit = _pow2((low - 2).clamp(min=-127, max=127))
    q = b.abs() / unit
    mags = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    out = torch.zeros_like(q)
    for code in range(1, 8):
        half = (mags[code - 1] + mags[code]) / 2
        up = (q >= half) if code % 2 == 0 else (q > half)
        out = torch.where(up, mags[code], out)
    out = torch.where(top > 0, out * unit * torch.sign(b), 0.0)
    return out.reshape(full.shape)[..., :K]


def _decode64(codes, scales):
    mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64,
                        device=codes.device)
    out = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64,
                      device=codes.device)
    for half in range(2):
        nib = (codes >> (4 * half)) & 15
        out[..., half::2] = mags[(nib & 7).long()] * (1 - 2 * (nib >> 3).double())
    return out * _pow2(scales.int() - 127).repeat_interleave(32, dim=-1)


def exact(case, seed):
    st, kind = prepare(case, seed), case["kind"]
    if kind == "balance":
        return _balance64(case, st)
    if kind == "router":
        s = st["scores"].double()
        g = st["dscores"].double() * (s - s * s)
        return dict(dx=g.matmul(st["w"].double()), d_w_router=g.t().matmul(st["x"].double()),
                    d_offset=g.sum(dim=0))
    if kind == "pack":
        x = st["x"].double()
        r = dict(values=_round64(x))
        if case["cols"]:
            r["values_t"] = _round64(x.t())
        return r
    if kind == "linear":
        return _round64(st["x"].double()).matmul(_decode64(st["codes"], st["scales"]).t())
    if kind == "train":
        x, w, dy = st["x"].double(), st["w"].double(), st["dy"].double()
        return dict(y=_round64(x).matmul(_round64(w).t()),
                    dx=_round64(dy).matmul(_round64(w.t()).t()),
                    dw=_round64(dy.t()).matmul(_round64(x.t()).t()))
    off = st["offsets"].tolist()
    if kind == "experts":
        x = _round64(st["x"].double())
        y = torch.zeros((case["T"] * case["k"], case["N"]), dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            b, c = off[e], off[e + 1]
            if c > b:
                y[b:c] = x[st["rows"][b:c].long()].matmul(
                    _decode64(st["codes"][e], st["scales"][e]).t())
        return y
    x, w, dy = st["x"].double(), st["w"].double(), st["dy"].double()
    y = torch.zeros((case["R"], case["N"]), dtype=torch.float64, device="cuda")
    dx = torch.zeros((case["R"], case["K"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros(w.shape, dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        b, c = off[e], off[e + 1]
        if c > b:
            y[b:c] = _round64(x[b:c]).matmul(_round64(w[e]).t())
            dx[b:c] = _round64(dy[b:c]).matmul(_round64(w[e].t()).t())
            dw[e] = _round64(dy[b:c].t()).matmul(_round64(x[b:c].t()).t())
    return dict(y=y, dx=dx, dw=dw)


def _balance64(case, st):
    T, n, k, S = case["T"], case["n"], case["k"], case["S"]
    off = st["offsets"].tolist()
    loss = torch.zeros(S, dtype=torch.float64, device="cuda")
    grad = torch.zeros((T, n), dtype=torch.float64, device="cuda")
    for q in range(S):
        rows = torch.arange(off[q], off[q + 1], device="cuda")
        if st["mask"] is not None:
            rows = rows[st["mask"][rows]]
        N = len(rows)
        if N == 0:
            continue
        s = st["scores"][rows].double()
        c = torch.bincount(st["idx"][rows].flatten().long(), minlength=n).double()
        total = s.sum(1, keepdim=True)
        loss[q] = (s / total).mean(0).dot(c) * n / (k * N)
        inner = (s.matmul(c) / total[:, 0])[:, None]
        grad[rows] = st["dloss"][q].double() * n / (k * N * N) * (c - inner) / total
    return dict(loss=loss, counts=None, tokens=None, dscores=grad)
