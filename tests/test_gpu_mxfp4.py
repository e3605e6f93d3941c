"""MXFP4 packing, unpacking and products against plain 64-bit
implementations: codes and scales bit for bit, products within the bound of an
fp32 sum of exact products."""
import numpy as np
import pytest
import torch

import workloads
from layer_cases import announce
from operator_cases import (as64, edge_rows, mx_decode64, mx_encode64, mx_round64, nibbles,
                            product_bound)

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def same_codes(codes, scales, want):
    wc, ws = want
    gs = scales.cpu().numpy()
    assert gs.shape == ws.shape
    bad = np.argwhere(gs != ws)
    assert bad.size == 0, f"scales differ at {bad[:4].tolist()}: {gs[tuple(bad[0])]} {ws[tuple(bad[0])]}"
    gc = nibbles(codes)
    bad = np.argwhere(gc != wc)
    assert bad.size == 0, f"codes differ at {bad[:4].tolist()}: {gc[tuple(bad[0])]} {wc[tuple(bad[0])]}"


# --- packing ----------------------------------------------------------------
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 32), (3, 31), (40, 33), (130, 64), (257, 100),
                                    (64, 127), (100, 512), (33, 545), (129, 129), (16, 2043)])
def test_pack_bit_exact(dtype, rows, K):
    import sparse_moe_ffn_sigmoid_amd as moe
    announce(f"pack {dtype} {rows}x{K}")
    x = edge_rows(rows, K, dtype, rows * 1000 + K)
    v = as64(x)
    p = moe.mxfp4_pack(x.cuda())
    same_codes(p["codes"], p["scales"], mx_encode64(v))
    both = moe.mxfp4_pack(x.cuda(), cols=True)
    assert torch.equal(both["codes"], p["codes"]) and torch.equal(both["scales"], p["scales"])
    same_codes(both["codes_t"], both["scales_t"], mx_encode64(v.T))
    only = moe.mxfp4_pack(x.cuda(), rows=False, cols=True)
    assert "codes" not in only and torch.equal(only["codes_t"], both["codes_t"])
    assert torch.equal(only["scales_t"], both["scales_t"])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_pack_columns_reach_the_edges(dtype):
    """The edge blocks along columns (whole rows of the transposed input)."""
    import sparse_moe_ffn_sigmoid_amd as moe
    announce(f"pack columns {dtype}")
    x = edge_rows(200, 160, dtype, 77).T.contiguous()          # blocks run down the columns
    p = moe.mxfp4_pack(x.cuda(), rows=False, cols=True)
    same_codes(p["codes_t"], p["scales_t"], mx_encode64(as64(x).T))


def test_pack_as_the_layer_quantises():
    import sparse_moe_ffn_sigmoid_amd as moe
    announce("pack = mxfp4_quantize on bf16 rows")
    x = torch.randn((70, 256), generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    p = moe.mxfp4_pack(x)
    c, s = moe.mxfp4_quantize(x)
    assert torch.equal(p["codes"], c) and torch.equal(p["scales"], s)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("lead,extra", [(0, 1), (1, 0), (8, 8), (3, 13)])
def test_pack_strided_rows_and_batches(dtype, lead, extra):
    import sparse_moe_ffn_sigmoid_amd as moe
    announce(f"pack strided {dtype} lead={lead} extra={extra}")
    B, R, K = 3, 50, 70
    wide = torch.full((B, R, K + lead + extra), float("nan"), dtype=dtype)
    x = wide[:, :, lead:lead + K]
    for b in range(B):
        x[b] = edge_rows(R, K, dtype, 10 * b + lead)
    p = moe.mxfp4_pack(wide.cuda()[:, :, lead:lead + K], cols=True)
    for b in range(B):
        same_codes(p["codes"][b], p["scales"][b], mx_encode64(as64(x[b])))
        same_codes(p["codes_t"][b], p["scales_t"][b], mx_encode64(as64(x[b]).T))
    every = moe.mxfp4_pack(wide.cuda()[:, ::2, lead:lead + K])      # every other row
    for b in range(B):
        same_codes(every["codes"][b], every["scales"][b], mx_encode64(as64(x[b, ::2])))


def test_pack_row_groups():
    import sparse_moe_ffn_sigmoid_amd as moe
    R, K = 300, 90
    for dtype in (F32, BF16, F16):
        for off in ([0, 300], [0, 0, 33, 33, 64, 200, 290], [7, 8, 40, 300], [5, 5, 5],
                    [0] + sorted(np.random.default_rng(3).integers(0, 301, 60).tolist()) + [300]):
            announce(f"pack groups {dtype} {off[:8]}")
            x = edge_rows(R, K, dtype, len(off))
            G = len(off) - 1
            p = moe.mxfp4_pack(x.cuda(), cols=True, offsets=dev(np.array(off, np.int32)))
            pof = p["offsets_t"].tolist()
            assert pof == np.concatenate([[0], np.cumsum([-(-(off[g + 1] - off[g]) // 32) * 32
                                                          for g in range(G)])]).tolist()
            v = as64(x)
            for g in range(G):
                b, e = off[g], off[g + 1]
                if e == b:
                    continue
                same_codes(p["codes"][b:e], p["scales"][b:e], mx_encode64(v[b:e]))
                same_codes(p["codes_t"][:, pof[g] // 2:pof[g + 1] // 2],
                           p["scales_t"][:, pof[g] // 32:pof[g + 1] // 32], mx_encode64(v[b:e].T))


def test_pack_leaves_rows_outside_groups():
    """Through the C ABI, so that the outputs' bytes before the call are known."""
    import ctypes
    import sparse_moe_ffn_sigmoid_amd as moe
    announce("pack rows outside groups")
    R, K, off = 100, 64, np.array([10, 20, 75], np.int32)
    x = edge_rows(R, K, BF16, 4).cuda()
    codes = torch.full((R, 32), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, 2), 0x5A, dtype=torch.uint8, device="cuda")
    rp = moe.lib().moe_mxfp4_padded_rows(R, 2)
    ct = torch.full((K, rp // 2), 0xA5, dtype=torch.uint8, device="cuda")
    st = torch.full((K, rp // 32), 0x5A, dtype=torch.uint8, device="cuda")
    po, o = torch.zeros(3, dtype=torch.int32, device="cuda"), dev(off)
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())
    assert moe.lib().moe_mxfp4_pack(ptr(x), moe.MOE_BF16, 1, R, K, K, R * K, ptr(codes),
                                    ptr(scales), ptr(ct), ptr(st), ptr(o), 2, ptr(po), None) == 0
    torch.cuda.synchronize()
    assert po.tolist() == [0, 32, 96]
    for t, v in ((codes, 0xA5), (scales, 0x5A)):
        assert (t[:10] == v).all() and (t[75:] == v).all()
    assert (ct[:, 48:] == 0xA5).all() and (st[:, 3:] == 0x5A).all()
    same_codes(codes[10:75], scales[10:75], mx_encode64(as64(x[10:75])))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_unpack_every_code_and_scale(dtype):
    import sparse_moe_ffn_sigmoid_amd as moe
    announce(f"unpack {dtype}")
    codes = np.arange(16, dtype=np.uint8)[None, :].repeat(256, 0)
    codes = np.concatenate([codes, codes[:, ::-1]], axis=1)            # [256, 32]
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    sb = np.arange(256, dtype=np.uint8)[:, None]
    want = mx_decode64(codes, sb)
    for K in (32, 17, 8):
        got = moe.mxfp4_unpack(dev(packed), dev(sb), K, dtype)
        ref = torch.from_numpy(want[:, :K]).to(dtype)                  # exact but in fp16
        assert got.dtype == dtype and torch.equal(torch.isnan(got.cpu()), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(got.cpu(), 0.0), torch.nan_to_num(ref, 0.0))
    x = edge_rows(90, 1000, F32, 5)
    p = moe.mxfp4_pack(x.cuda())
    got = as64(moe.mxfp4_unpack(p["codes"], p["scales"], 1000, F32))
    assert np.array_equal(got, mx_round64(as64(x)), equal_nan=True)


# --- products ---------------------------------------------------------------
def operand(rows, K, seed, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, K), generator=g) * torch.exp(torch.randn((rows, 1), generator=g))
    return x.to(dtype)


def check_product(got, a, b, out_dtype):
    ref, bound = product_bound(a, b, out_dtype, a.shape[1])
    d = np.abs(as64(got) - ref)
    assert got.dtype == out_dtype and (d <= bound).all(), (d / bound).max()


SHAPES = [(1, 1, 32), (1, 3584, 7168), (2, 17, 64), (5, 300, 96), (16, 48, 160), (17, 33, 288),
          (31, 1000, 512), (33, 64, 224), (64, 257, 2080), (65, 31, 32), (128, 256, 256),
          (129, 255, 1056), (200, 300, 768), (256, 256, 512), (300, 520, 3584), (513, 129, 992)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul(M, N, K):
    import sparse_moe_ffn_sigmoid_amd as moe
    xa, xb = operand(M, K, M + N), operand(N, K, M * N)
    a, b = mx_round64(as64(xa)), mx_round64(as64(xb))
    pa, pb = moe.mxfp4_pack(xa.cuda()), moe.mxfp4_pack(xb.cuda())
    args = (pa["codes"], pa["scales"], pb["codes"], pb["scales"])
    for dt in (BF16, F32, F16):
        announce(f"matmul {M}x{N}x{K} {dt}")
        check_product(moe.mxfp4_matmul(*args, out_dtype=dt), a, b, dt)
    wide = torch.full((M, N + 3), 7.0, device="cuda")
    announce(f"matmul strided out {M}x{N}x{K}")
    moe.mxfp4_matmul(*args, out_dtype=F32, out=wide[:, :N])
    check_product(wide[:, :N], a, b, F32)
    assert (wide[:, N:] == 7.0).all()
    announce(f"kgroup without offsets {M}x{N}x{K}")
    check_product(moe.mxfp4_matmul_kgroup(*args), a, b, F32)


@pytest.mark.parametrize("M", [1, 2, 9, 16, 17, 40, 200])
@pytest.mark.parametrize("dtype", [BF16, F32, F16])
def test_linear(M, dtype):
    import sparse_moe_ffn_sigmoid_amd as moe
    for N, K in ((100, 64), (3, 32), (500, 1184), (64, 4096), (20, 7168), (33, 8224)):
        announce(f"linear {dtype} {M}x{N}x{K}")
        x, w = operand(M, K, M + N, dtype), operand(N, K, N, F32)
        p = moe.mxfp4_pack(w.cuda())
        b = mx_round64(as64(w))
        y = moe.mxfp4_linear(x.cuda(), p["codes"], p["scales"])
        check_product(y, mx_round64(as64(x)), b, dtype)
        y = moe.mxfp4_linear(x.cuda(), p["codes"], p["scales"], out_dtype=F32)
        check_product(y, mx_round64(as64(x)), b, F32)
        # rows out of a wider matrix, at any alignment, gathered with repeats
        announce(f"linear strided, gathered {dtype} {M}x{N}x{K}")
        wide = torch.full((M, K + 5), float("nan"), dtype=dtype)
        wide[:, 3:3 + K] = x
        rows = torch.from_numpy(np.random.default_rng(M).integers(0, M, 2 * M + 1).astype(np.int32))
        y = moe.mxfp4_linear(wide.cuda()[:, 3:3 + K], p["codes"], p["scales"], rows=rows.cuda(),
                             out_dtype=F32)
        check_product(y, mx_round64(as64(x))[rows.numpy()], b, F32)


def group_offsets(lens, lead=0):
    return np.concatenate([[lead], lead + np.cumsum(lens)]).astype(np.int32)


GROUPS = [  # rows per group, rows before the first and behind the last group
    ([1], 0, 0), ([0, 3, 0, 1, 0], 2, 3), ([5, 16, 17, 1, 2, 33], 0, 0), ([40, 0, 70, 64], 1, 5),
    ([200, 1, 0, 300, 129], 0, 7), ([0, 0, 0], 4, 4), ([293, 292, 293], 0, 0), ([600], 3, 0),
    ([2] * 70, 0, 1), ([31, 32, 33, 255, 256, 257, 0, 1], 0, 0),
]


@pytest.mark.parametrize("lens,lead,tail", GROUPS)
def test_matmul_groups(lens, lead, tail):
    import sparse_moe_ffn_sigmoid_amd as moe
    G, N, K = len(lens), 90, 288
    off = group_offsets(lens, lead)
    M = int(off[-1]) + tail
    xa, xb = operand(M, K, 1), operand(G * N, K, 2)
    pa, pb = moe.mxfp4_pack(xa.cuda()), moe.mxfp4_pack(xb.view(G, N, K).cuda())
    a, b = mx_round64(as64(xa)), mx_round64(as64(xb)).reshape(G, N, K)
    for dt in (F32, BF16):
        announce(f"groups {lens[:8]} lead={lead} tail={tail} {dt}")
        out = torch.full((M, N), -3.0, dtype=dt, device="cuda")
        got = moe.mxfp4_matmul(pa["codes"], pa["scales"], pb["codes"], pb["scales"],
                               offsets=dev(off), out_dtype=dt, out=out)
        assert got is out
        for g in range(G):
            if lens[g]:
                check_product(out[off[g]:off[g + 1]], a[off[g]:off[g + 1]], b[g], dt)
        assert (out[:lead] == -3).all() and (out[M - tail:] == -3).all()
    # rows gathered from few tokens, some of them from nowhere
    announce(f"groups gathered {lens[:8]}")
    T = 11
    rows = np.random.default_rng(M).integers(0, T, M).astype(np.int32)
    rows[::7] = -1
    rows[3::11] = T
    xt = operand(T, K, 3)
    y = moe.mxfp4_linear(xt.cuda(), pb["codes"], pb["scales"], offsets=dev(off), rows=dev(rows),
                         out_dtype=F32)
    at = np.concatenate([mx_round64(as64(xt)), np.zeros((1, K))])
    at = at[np.where((rows >= 0) & (rows < T), rows, T)]
    for g in range(G):
        if lens[g]:
            check_product(y[off[g]:off[g + 1]], at[off[g]:off[g + 1]], b[g], F32)


@pytest.mark.parametrize("lens", [[64], [0, 5, 0, 33, 100, 0], [293, 17, 1, 600], [3] * 40])
def test_experts_forward_and_gradients(lens):
    """Grouped forward, dx and dW of packed operands, ragged groups."""
    import sparse_moe_ffn_sigmoid_amd as moe
    G, N, K = len(lens), 70, 130
    off = group_offsets(lens)
    R = int(off[-1])
    announce(f"experts training {lens[:6]}")
    x, dy, w = operand(R, K, 4), operand(R, N, 5), operand(G * N, K, 6).view(G, N, K)
    o = dev(off)
    px = moe.mxfp4_pack(x.cuda(), cols=True, offsets=o)
    pd = moe.mxfp4_pack(dy.cuda(), cols=True, offsets=o)
    pw = moe.mxfp4_pack(w.cuda(), cols=True)
    assert torch.equal(px["offsets_t"], pd["offsets_t"])
    y = moe.mxfp4_matmul(px["codes"], px["scales"], pw["codes"], pw["scales"], offsets=o)
    dx = moe.mxfp4_matmul(pd["codes"], pd["scales"], pw["codes_t"], pw["scales_t"], offsets=o,
                          out_dtype=F32)
    dw = moe.mxfp4_matmul_kgroup(pd["codes_t"], pd["scales_t"], px["codes_t"], px["scales_t"],
                                 offsets=px["offsets_t"])
    assert dw.shape == (G, N, K)
    xv, dv, wv = as64(x), as64(dy), as64(w)
    for g in range(G):
        b, e = off[g], off[g + 1]
        if e == b:
            assert not dw[g].any()
            continue
        check_product(y[b:e], mx_round64(xv[b:e]), mx_round64(wv[g]), BF16)
        check_product(dx[b:e], mx_round64(dv[b:e]), mx_round64(wv[g].T), F32)
        check_product(dw[g], mx_round64(dv[b:e].T), mx_round64(xv[b:e].T), F32)


def test_gradients_are_the_formulas_on_exact_operands():
    """With operands that E2M1 holds exactly, packing rounds nothing: the
    products are the gradients of sum(dy * (x W^T)), checked by differences."""
    import sparse_moe_ffn_sigmoid_amd as moe
    announce("gradients by differences")
    rng = np.random.default_rng(8)
    grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6.0])
    pick = lambda *s: rng.choice(grid, s) * rng.choice([-1.0, 1.0], s)
    T, K, N = 64, 96, 32
    x, w, dy = pick(T, K), pick(N, K), pick(T, N)
    for v in (x, w, dy):
        v[::32] = np.sign(v[::32] + 0.1) * 6      # every block of a column has scale 1 ...
        v[:, ::32] = 4                            # ... and every block of a row
    px, pw, pd = (moe.mxfp4_pack(dev(v, F32), cols=True) for v in (x, w, dy))
    dx = as64(moe.mxfp4_matmul(pd["codes"], pd["scales"], pw["codes_t"], pw["scales_t"], out_dtype=F32))
    dw = as64(moe.mxfp4_matmul_kgroup(pd["codes_t"], pd["scales_t"], px["codes_t"], px["scales_t"]))
    f = lambda x, w: (dy * (x @ w.T)).sum()
    for t, c in ((0, 0), (13, 95), (63, 40)):
        e = np.zeros_like(x)
        e[t, c] = 1.0
        assert abs((f(x + e, w) - f(x - e, w)) / 2 - dx[t, c]) <= 1e-9   # f is linear in x
    for n, c in ((0, 0), (31, 95), (7, 33)):
        e = np.zeros_like(w)
        e[n, c] = 1.0
        assert abs((f(x, w + e) - f(x, w - e)) / 2 - dw[n, c]) <= 1e-9


def test_matmul_nan_blocks_stay_in_their_rows():
    import sparse_moe_ffn_sigmoid_amd as moe
    for M, N, K in ((3, 40, 96), (200, 300, 320)):
        announce(f"NaN blocks {M}x{N}x{K}")
        xa, xb = operand(M, K, 1), operand(N, K, 2)
        xa[1, 40] = float("inf")
        xb[5, 95] = float("nan")
        pa, pb = moe.mxfp4_pack(xa.cuda()), moe.mxfp4_pack(xb.cuda())
        y = as64(moe.mxfp4_matmul(pa["codes"], pa["scales"], pb["codes"], pb["scales"], out_dtype=F32))
        bad = np.zeros((M, N), bool)
        bad[1], bad[:, 5] = True, True
        assert np.array_equal(np.isnan(y), bad)
        a, b = mx_round64(as64(xa)), mx_round64(as64(xb))
        ref, bound = product_bound(np.nan_to_num(a), np.nan_to_num(b), F32, K)
        assert (np.abs(y - ref) <= bound)[~bad].all()
        # zeros times a NaN block are NaN too, as in floating point
        z = moe.mxfp4_linear(torch.zeros((M, K), device="cuda"), pb["codes"], pb["scales"])
        assert torch.isnan(z[:, 5]).all() and not z[:, :5].any()


def test_matmul_layer_weights_and_wide_scales():
    """Weights as the layer holds them (workloads' quantiser), scales across the
    exponent range."""
    import sparse_moe_ffn_sigmoid_amd as moe
    announce("layer weights")
    G, N, K = 3, 64, 256
    w = torch.randn((G * N, K), generator=torch.Generator().manual_seed(3)) * 2.0 ** -40
    c, s = workloads.mxfp4_quantize(w)
    x = operand(50, K, 9) * 2.0 ** 60
    off = np.array([0, 20, 20, 50], np.int32)
    y = moe.mxfp4_linear(x.cuda(), c.view(G, N, -1).cuda(), s.view(G, N, -1).cuda(),
                         offsets=dev(off), out_dtype=F32)
    b = mx_decode64(nibbles(c), s.numpy()).reshape(G, N, K)
    for g in range(G):
        if off[g + 1] > off[g]:
            check_product(y[off[g]:off[g + 1]], mx_round64(as64(x[off[g]:off[g + 1]])), b[g], F32)


def test_products_empty():
    import sparse_moe_ffn_sigmoid_amd as moe
    announce("empty products")
    e = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")
    y = moe.mxfp4_matmul(e(0, 32), e(0, 2), e(8, 32), e(8, 2))
    assert y.shape == (0, 8)
    x = torch.empty((0, 64), dtype=BF16, device="cuda")
    assert moe.mxfp4_linear(x, e(8, 32), e(8, 2)).shape == (0, 8)
    p = moe.mxfp4_pack(x, cols=True)
    assert p["codes"].shape == (0, 32) and p["codes_t"].shape == (64, 0)


@pytest.mark.parametrize("M,G", [(1, 0), (24, 0), (300, 0), (90, 5)])
def test_linear_graph_replays(M, G):
    import sparse_moe_ffn_sigmoid_amd as moe
    N, K = 160, 256
    announce(f"linear graph M={M} G={G}")
    w = operand(max(G, 1) * N, K, 1)
    p = moe.mxfp4_pack((w.view(G, N, K) if G else w).cuda())
    off = dev(group_offsets([M // G] * G)) if G else None
    x = operand(M, K, 2).cuda()
    other = operand(M, K, 3).cuda()

    def call():
        q = moe.mxfp4_pack(x, cols=True)
        return moe.mxfp4_linear(x, p["codes"], p["scales"], offsets=off), q["codes_t"]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = call()
    for _ in range(4):
        keep = x.clone()
        x.copy_(other)
        other = keep
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in r]
        for g, e in zip(got, call()):
            assert torch.equal(g, e)


def test_experts_run_of_the_operators():
    """Routing, balance loss and one expert layer in MXFP4 as a program runs
    them: the routing's counts are the groups of the product."""
    import sparse_moe_ffn_sigmoid_amd as moe
    T, n, k, K, N = 120, 16, 4, 128, 96
    announce("route, balance, experts")
    g = torch.Generator().manual_seed(4)
    s = torch.sigmoid(torch.randn((T, n), generator=g)).cuda()
    r = moe.route_qb(s, k)
    b = moe.balance_loss(s, r["idx"], want_grad=True)
    assert torch.equal(b["counts"][0], r["loads"])
    assert abs(b["loss"].item() - 1) < 1e-5          # balanced routing: even counts
    off = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.cumsum(r["loads"], 0)
    order = torch.argsort(r["idx"].flatten().long(), stable=True)
    rows = (order // k).to(torch.int32)
    x, w = operand(T, K, 5), operand(n * N, K, 6)
    p = moe.mxfp4_pack(w.view(n, N, K).cuda())
    y = moe.mxfp4_linear(x.cuda(), p["codes"], p["scales"], offsets=off, rows=rows, out_dtype=F32)
    a, wv = mx_round64(as64(x)), mx_round64(as64(w)).reshape(n, N, K)
    o, at = off.tolist(), rows.cpu().numpy()
    for e in range(n):
        check_product(y[o[e]:o[e + 1]], a[at[o[e]:o[e + 1]]], wv[e], F32)


def random_codes(*shape):
    g = torch.Generator("cuda").manual_seed(sum(shape))
    return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)


def test_weights_beyond_4_gib():
    import sparse_moe_ffn_sigmoid_amd as moe
    G, N, K = 1024, 2080, 4096                     # 4.4 GB of codes
    announce("weights beyond 4 GiB")
    codes = torch.zeros((G, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((G, N, K // 32), 120, dtype=torch.uint8, device="cuda")
    for g in (5, G - 1):
        codes[g] = random_codes(N, K // 2)
    for few, many in ((3, 40), (300, 20000)):      # a few rows per group, and many
        off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
        off[6:] = few
        off[G] = few + many
        x = operand(few + many, K, few)
        y = moe.mxfp4_linear(x.cuda(), codes, scales, offsets=off, out_dtype=F32)
        for g, rows in ((5, slice(0, few)), (G - 1, slice(few + many - 33, few + many))):
            b = mx_decode64(nibbles(codes[g]), scales[g].cpu().numpy())
            check_product(y[rows], mx_round64(as64(x[rows])), b, F32)


def test_gathered_rows_beyond_4_gib():
    import sparse_moe_ffn_sigmoid_amd as moe
    R, K, N, M = 2_200_000, 4096, 70, 200          # 4.5 GB of codes
    announce("gathered rows beyond 4 GiB")
    codes = torch.zeros((R, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((R, K // 32), 125, dtype=torch.uint8, device="cuda")
    codes[R - 50:] = random_codes(50, K // 2)
    rows = torch.from_numpy(np.random.default_rng(0).integers(R - 50, R, M).astype(np.int32))
    rows[7], rows[150] = R, -5
    w = operand(N, K, 2)
    p = moe.mxfp4_pack(w.cuda())
    y = moe.mxfp4_matmul(codes, scales, p["codes"], p["scales"], rows=rows.cuda(), out_dtype=F32)
    last = mx_decode64(nibbles(codes[R - 50:]), scales[R - 50:].cpu().numpy())
    a = np.concatenate([last, np.zeros((1, K))])
    at = rows.numpy() - (R - 50)
    at[[7, 150]] = 50
    check_product(y, a[at], mx_round64(as64(w)), F32)


def test_output_beyond_32_bits():
    import sparse_moe_ffn_sigmoid_amd as moe
    M, N, K = 70001, 32768, 64                     # 2.3e9 outputs
    announce("outputs beyond 2^31")
    x, w = operand(M, K, 1), operand(N, K, 2)
    p = moe.mxfp4_pack(w.cuda())
    y = moe.mxfp4_linear(x.cuda(), p["codes"], p["scales"])
    rows = [0, 65535, 65536, 69999, 70000]
    check_product(y[rows][:, -300:], mx_round64(as64(x[rows])), mx_round64(as64(w[-300:])), BF16)


def test_linear_of_very_many_columns():
    """More columns than one launch has threads for at 32 a column."""
    import sparse_moe_ffn_sigmoid_amd as moe
    N, K = (1 << 27) + 48, 32                      # 2.1 GB of codes
    announce("2^27 columns")
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((N, 1), 127, dtype=torch.uint8, device="cuda")
    codes[-100:] = random_codes(100, K // 2)
    x = operand(2, K, 1)
    y = moe.mxfp4_linear(x.cuda(), codes, scales, out_dtype=F32)
    b = mx_decode64(nibbles(codes[-100:]), scales[-100:].cpu().numpy())
    check_product(y[:, -100:], mx_round64(as64(x)), b, F32)
    assert not y[:, :1000].any()


def test_products_on_two_streams_and_given_buffers():
    import sparse_moe_ffn_sigmoid_amd as moe
    N, K = 300, 512
    announce("two streams")
    w = operand(N, K, 1)
    p = moe.mxfp4_pack(w.cuda())
    b = mx_round64(as64(w))
    xs = [operand(M, K, M).cuda() for M in (1, 100, 400, 9)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    ys = []
    for x, s in zip(xs, streams):
        with torch.cuda.stream(s):
            ys.append([moe.mxfp4_linear(x, p["codes"], p["scales"], out_dtype=F32)
                       for _ in range(5)])
    torch.cuda.synchronize()
    for x, many in zip(xs, ys):
        for y in many:
            check_product(y, mx_round64(as64(x)), b, F32)
    ws = torch.empty(moe.lib().moe_mxfp4_linear_workspace_bytes(400, K), dtype=torch.uint8,
                     device="cuda")
    y = moe.mxfp4_linear(xs[2], p["codes"], p["scales"], out_dtype=F32, workspace=ws)
    assert torch.equal(y, ys[2][0])
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.mxfp4_linear(xs[2], p["codes"], p["scales"], workspace=ws[:1024])


def test_python_refusals_on_the_device():
    import sparse_moe_ffn_sigmoid_amd as moe
    announce("refusals")
    x = operand(8, 64, 1).cuda()
    p = moe.mxfp4_pack(x)
    c, s = p["codes"], p["scales"]
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    for bad in (lambda: moe.mxfp4_pack(x.double()), lambda: moe.mxfp4_pack(x[:, ::2]),
                lambda: moe.mxfp4_pack(x[0]), lambda: moe.mxfp4_pack(x, rows=False),
                lambda: moe.mxfp4_pack(x, offsets=off),
                lambda: moe.mxfp4_pack(x, cols=True, offsets=off.long()),
                lambda: moe.mxfp4_pack(x.expand(2, 8, 64), cols=True, offsets=off),
                lambda: moe.mxfp4_unpack(c, s, 32), lambda: moe.mxfp4_unpack(c, s, 65),
                lambda: moe.mxfp4_unpack(c, s[:4], 64),
                lambda: moe.mxfp4_unpack(c, s, 64, torch.float64),
                lambda: moe.mxfp4_matmul(c, s, c[:, :16].contiguous(), s[:, :1].contiguous()),
                lambda: moe.mxfp4_matmul(c, s, c, s, offsets=off),
                lambda: moe.mxfp4_matmul(c, s, c[None], s[None]),
                lambda: moe.mxfp4_matmul(c, s, c, s, out_dtype=torch.int32),
                lambda: moe.mxfp4_matmul(c, s, c, s, out=torch.empty((8, 7), device="cuda")),
                lambda: moe.mxfp4_matmul(c, s, c, s, rows=off.long()),
                lambda: moe.mxfp4_matmul_kgroup(c, s, c[:, :16].contiguous(), s[:, :1].contiguous()),
                lambda: moe.mxfp4_linear(x[:, :48], c, s), lambda: moe.mxfp4_linear(x[0], c, s)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.MoeError):                       # nothing to gather from
        moe.mxfp4_linear(x[:0], c, s, rows=off)
    with pytest.raises(moe.MoeError):
        moe.mxfp4_pack(x, cols=True, offsets=torch.zeros(1026, dtype=torch.int32, device="cuda"))


def sampled_rows(M, edges, seed):
    """Row numbers at and around multiples of the tile heights, and others."""
    near = {r + d for e in edges for r in range(0, M + 1, e) for d in (-1, 0, 1, 31, 32)}
    other = np.random.default_rng(seed).integers(0, M, 40).tolist()
    return sorted(r for r in near | set(other) | {M - 1} if 0 <= r < M)


# columns enough that each tile height is the cheapest for some number of rows:
# 64, 128, 192, 256, 320, the last ones with short last tiles
@pytest.mark.parametrize("M", [200, 1000, 1500, 2000, 2300, 2500])
@pytest.mark.parametrize("N,K", [(8190, 96), (8192, 1312)])
def test_matmul_tile_heights(M, N, K):
    import sparse_moe_ffn_sigmoid_amd as moe
    announce(f"tile heights {M}x{N}x{K}")
    xa, xb = operand(M, K, M), operand(N, K, N)
    pa, pb = moe.mxfp4_pack(xa.cuda()), moe.mxfp4_pack(xb.cuda())
    rows = sampled_rows(M, (64, 128, 192, 256, 320), M)
    a, b = mx_round64(as64(xa[rows])), mx_round64(as64(xb))
    for dt in (F32, BF16, F16):
        y = moe.mxfp4_matmul(pa["codes"], pa["scales"], pb["codes"], pb["scales"], out_dtype=dt)
        check_product(y[rows], a, b, dt)
    index = torch.from_numpy(np.random.default_rng(1).permutation(M).astype(np.int32))
    index[M // 2] = -1
    y = moe.mxfp4_matmul(pa["codes"], pa["scales"], pb["codes"], pb["scales"], rows=index.cuda(),
                         out_dtype=F32)
    take = index[rows].numpy()
    a = mx_round64(as64(xa[np.maximum(take, 0)])) * (take >= 0)[:, None]
    check_product(y[rows], a, b, F32)
    assert not y[M // 2].any()


@pytest.mark.parametrize("lens", [[320, 1, 0, 64, 65, 257, 400, 1293], [300] * 8,
                                  [0, 0, 1500, 0, 20, 0, 0, 3], [100, 130, 90, 128, 127, 129, 64, 1]])
def test_groups_tile_heights(lens):
    import sparse_moe_ffn_sigmoid_amd as moe
    G, N, K, T = len(lens), 8192, 800, 77
    announce(f"groups, tile heights {lens}")
    off = group_offsets(lens, 2)
    M = int(off[-1]) + 5
    xt, xb = operand(T, K, 1), operand(G * N, K, 2)
    pb = moe.mxfp4_pack(xb.view(G, N, K).cuda())
    index = np.random.default_rng(M).integers(0, T, M).astype(np.int32)
    out = torch.full((M, N), 9.0, device="cuda")
    moe.mxfp4_linear(xt.cuda(), pb["codes"], pb["scales"], offsets=dev(off), rows=dev(index),
                     out_dtype=F32, out=out)
    a = mx_round64(as64(xt))
    for g in range(G):
        rows = [int(off[g]) + r for r in sampled_rows(lens[g], (64, 256, 320), g)] if lens[g] else []
        if rows:
            check_product(out[rows], a[index[rows]], mx_round64(as64(xb[g * N:(g + 1) * N])), F32)
    assert (out[:2] == 9).all() and (out[M - 5:] == 9).all()


@pytest.mark.parametrize("M", [700, 1000, 2300])
def test_kgroup_tile_heights(M):
    import sparse_moe_ffn_sigmoid_amd as moe
    N, lens = 4096, [300, 0, 33, 1, 700]
    off = group_offsets(lens)
    R = int(off[-1])
    announce(f"kgroup tile heights {M}")
    dy, x = operand(R, M, 1), operand(R, N, 2)
    pd = moe.mxfp4_pack(dy.cuda(), rows=False, cols=True, offsets=dev(off))
    px = moe.mxfp4_pack(x.cuda(), rows=False, cols=True, offsets=dev(off))
    for dt in (F32, BF16):
        dw = moe.mxfp4_matmul_kgroup(pd["codes_t"], pd["scales_t"], px["codes_t"], px["scales_t"],
                                     offsets=pd["offsets_t"], out_dtype=dt)
        rows = sampled_rows(M, (64, 128, 192, 256, 320), M)
        dv, xv = as64(dy)[:, rows], as64(x)
        for g in range(len(lens)):
            b, e = off[g], off[g + 1]
            if e == b:
                assert not dw[g].any()
            else:
                check_product(dw[g][rows], mx_round64(dv[b:e].T), mx_round64(xv[b:e].T), dt)
