"""Arguments of the balance loss, the dense router gradient and the MXFP4
calls are refused on the host, before anything is launched (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from operator_cases import balance64, mx_encode64, mx_round64

FAKE = ctypes.c_void_p(1 << 20)            # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def moe():
    import sparse_moe_ffn_sigmoid_amd
    return sparse_moe_ffn_sigmoid_amd


def test_balance_loss_refusals(moe):
    lib = moe.lib()
    need = lib.moe_balance_loss_workspace_bytes(2000, 3)
    assert need >= 4 * 2003 and need % 256 == 0
    assert lib.moe_balance_loss_workspace_bytes(0, 1) > 0
    assert lib.moe_balance_loss_workspace_bytes(-1, 1) == 0
    assert lib.moe_balance_loss_workspace_bytes(10, 0) == 0
    assert lib.moe_balance_loss_workspace_bytes((1 << 20) + 1, 1) == 0

    def call(T=2000, n=64, k=4, ld=64, S=3, scores=FAKE, idx=FAKE, off=FAKE, loss=FAKE, counts=FAKE,
             tokens=FAKE, ws=FAKE, nb=need):
        return lib.moe_balance_loss(scores, ld, T, n, k, idx, off, S, None, None, loss, counts,
                                    tokens, None, ws, nb, None)

    for bad in (dict(T=-1), dict(n=0), dict(k=0), dict(k=65), dict(ld=63), dict(S=0),
                dict(off=None), dict(scores=None), dict(idx=None), dict(loss=None),
                dict(counts=None), dict(tokens=None), dict(ws=ODD)):
        assert call(**bad) == -1, bad
    assert call(n=1025, ld=1025) == -2
    assert call(T=(1 << 20) + 1) == -2
    assert call(nb=need - 256) == -3 and call(ws=None, nb=0) == -3

    def back(T=100, n=64, k=4, ld=64, S=3, scores=FAKE, counts=FAKE, tokens=FAKE, off=FAKE,
             d=FAKE):
        return lib.moe_balance_loss_backward(scores, ld, T, n, k, counts, tokens, off, S, None,
                                             None, d, None)

    for bad in (dict(T=-1), dict(k=65), dict(ld=1), dict(S=2, off=None), dict(scores=None),
                dict(counts=None), dict(tokens=None), dict(d=None)):
        assert back(**bad) == -1, bad
    assert back(T=0) == 0


def test_router_backward_refusals(moe):
    lib = moe.lib()
    need = lib.moe_router_backward_workspace_bytes(3000, 128, 40)
    assert need > 0 and lib.moe_router_backward_workspace_bytes(0, 128, 40) > 0
    for bad in ((-1, 128, 40), (100, 96, 40), (100, 0, 40), (100, 128, 0), (100, 128, 1025),
                ((1 << 20) + 1, 128, 40)):
        assert lib.moe_router_backward_workspace_bytes(*bad) == 0, bad

    def call(T=3000, d=128, n=40, x=FAKE, w=FAKE, s=FAKE, ds=FAKE, dx=FAKE, dw=FAKE, ws=FAKE,
             nb=need):
        return lib.moe_router_backward(x, w, s, ds, T, d, n, 0, dx, dw, FAKE, ws, nb, None)

    for bad in (dict(T=-1), dict(d=100), dict(n=0), dict(x=None), dict(w=None), dict(s=None),
                dict(ds=None), dict(ws=ODD), dict(dx=ODD), dict(dw=ODD)):
        assert call(**bad) == -1, bad
    assert call(n=2000) == -2
    assert call(nb=need - 1) == -3 and call(ws=None, nb=0) == -3


def test_pack_refusals(moe):
    lib = moe.lib()
    assert lib.moe_mxfp4_padded_rows(33, 0) == 64 and lib.moe_mxfp4_padded_rows(0, 0) == 0
    assert lib.moe_mxfp4_padded_rows(100, 3) == 192     # 100 + 3 * 31 = 193, whole blocks
    assert lib.moe_mxfp4_padded_rows(-1, 0) == -1 and lib.moe_mxfp4_padded_rows(5, 1025) == -1

    def call(x=FAKE, dt=moe.MOE_BF16, B=1, R=8, C=64, rs=64, bs=512, c=FAKE, s=FAKE, ct=FAKE,
             st=FAKE, off=None, G=0, po=None):
        return lib.moe_mxfp4_pack(x, dt, B, R, C, rs, bs, c, s, ct, st, off, G, po, None)

    for bad in (dict(B=-1), dict(R=-1), dict(C=0), dict(rs=63), dict(bs=-1), dict(s=None),
                dict(c=None), dict(st=None), dict(ct=None), dict(G=2), dict(x=None),
                dict(c=None, s=None, ct=None, st=None), dict(c=ODD), dict(ct=ODD),
                dict(x=ctypes.c_void_p((1 << 20) + 1)), dict(off=FAKE, G=0, po=FAKE),
                dict(off=FAKE, G=2), dict(off=FAKE, G=2, po=FAKE, B=2),
                dict(off=FAKE, G=2, po=FAKE, ct=None, st=None), dict(rs=1 << 55)):
        assert call(**bad) == -1, bad
    for bad in (dict(dt=moe.MOE_MXFP4), dict(dt=77), dict(B=65536), dict(R=1 << 31),
                dict(off=FAKE, G=1025, po=FAKE), dict(R=1 << 25)):
        assert call(**bad) == -2, bad
    assert call(R=0) == 0 and call(B=0) == 0

    def un(c=FAKE, s=FAKE, R=8, K=64, dt=moe.MOE_F32, out=FAKE, rs=64):
        return lib.moe_mxfp4_unpack(c, s, R, K, dt, out, rs, None)

    for bad in (dict(R=-1), dict(K=0), dict(rs=63), dict(c=None), dict(s=None), dict(out=None),
                dict(c=ctypes.c_void_p((1 << 20) + 2)), dict(out=ctypes.c_void_p((1 << 20) + 2))):
        assert un(**bad) == -1, bad
    assert un(dt=3) == -2 and un(R=0) == 0


def test_product_refusals(moe):
    lib = moe.lib()

    def mm(ac=FAKE, as_=FAKE, R=8, bc=FAKE, bs=FAKE, M=8, N=16, K=64, off=None, G=1, rows=None,
           out=FAKE, dt=moe.MOE_F32, ldo=16):
        return lib.moe_mxfp4_matmul(ac, as_, R, bc, bs, M, N, K, off, G, rows, out, dt, ldo, None)

    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(K=48), dict(R=-1), dict(R=7), dict(G=2),
                dict(off=FAKE, G=0), dict(ac=None), dict(as_=None), dict(bc=None), dict(bs=None),
                dict(out=None), dict(ldo=15), dict(ac=ODD), dict(bc=ODD),
                dict(out=ctypes.c_void_p((1 << 20) + 2))):
        assert mm(**bad) == -1, bad
    for bad in (dict(dt=moe.MOE_MXFP4), dict(off=FAKE, G=1025), dict(N=(1 << 30) + 1, ldo=1 << 31)):
        assert mm(**bad) == -2, bad
    assert mm(M=0, R=0) == 0 and mm(M=0, R=0, rows=FAKE) == 0
    assert mm(R=0, rows=FAKE) == -1                     # nothing to gather from
    assert mm(M=(1 << 24) + 1, R=1, rows=FAKE, off=FAKE, G=8) == -2

    def kg(ac=FAKE, as_=FAKE, bc=FAKE, bs=FAKE, M=8, N=16, K=64, off=None, G=1, out=FAKE,
           dt=moe.MOE_F32):
        return lib.moe_mxfp4_matmul_kgroup(ac, as_, bc, bs, M, N, K, off, G, out, dt, None)

    for bad in (dict(M=0), dict(N=0), dict(K=-32), dict(K=40), dict(G=3), dict(off=FAKE, G=0),
                dict(ac=None), dict(bs=None), dict(out=None), dict(ac=ODD), dict(bc=ODD)):
        assert kg(**bad) == -1, bad
    assert kg(dt=9) == -2 and kg(off=FAKE, G=1025) == -2

    need = lib.moe_mxfp4_linear_workspace_bytes(80, 64)
    assert need >= 80 * 34 and lib.moe_mxfp4_linear_workspace_bytes(8, 40) == 0

    def lin(x=FAKE, xt=moe.MOE_BF16, R=80, rs=64, wc=FAKE, ws=FAKE, M=80, N=16, K=64, off=None, G=1,
            rows=None, out=FAKE, dt=moe.MOE_BF16, ldo=16, wk=FAKE, nb=need):
        return lib.moe_mxfp4_linear(x, xt, R, rs, wc, ws, M, N, K, off, G, rows, out, dt, ldo, wk,
                                    nb, None)

    for bad in (dict(x=None), dict(rs=63), dict(wc=None), dict(ws=None), dict(K=33), dict(M=81),
                dict(out=None), dict(ldo=8), dict(wk=ODD), dict(wc=ODD),
                dict(off=FAKE, G=0), dict(x=ctypes.c_void_p((1 << 20) + 1)),
                dict(R=0, rows=FAKE)):
        assert lin(**bad) == -1, bad
    assert lin(xt=moe.MOE_MXFP4_A8) == -2 and lin(dt=4) == -2
    assert lin(nb=need - 1) == -3 and lin(wk=None, nb=0) == -3 and lin(M=0) == 0


def test_python_refusals(moe):
    """Host tensors, wrong types and wrong shapes raise before the library is called."""
    s, i = torch.rand(4, 8), torch.zeros((4, 2), dtype=torch.int32)
    for fn in (lambda: moe.balance_loss(s, i), lambda: moe.mxfp4_pack(s),
               lambda: moe.balance_loss_backward(s, i, i, 2),
               lambda: moe.router_backward(s, s, s, s),
               lambda: moe.mxfp4_unpack(i, i, 2), lambda: moe.mxfp4_matmul(i, i, i, i),
               lambda: moe.mxfp4_matmul_kgroup(i, i, i, i), lambda: moe.mxfp4_linear(s, i, i)):
        with pytest.raises(ValueError, match="must be on a GPU"):
            fn()
    with pytest.raises(TypeError):
        moe.balance_loss(None, i)


def test_plain_balance_is_the_closed_form():
    """The tests' own 64-bit form: even counts give 1, one expert for all gives
    n times its share, and the gradient is its difference quotient."""
    rng = np.random.default_rng(0)
    s = rng.random((16, 8))
    idx = (np.arange(16)[:, None] * 2 + np.arange(2)) % 8
    assert abs(balance64(s, idx)[0][0] - 1) < 1e-12
    one = np.full((16, 1), 3)
    share = (s[:, 3] / s.sum(1)).mean()
    assert abs(balance64(s, one)[0][0] - 8 * share) < 1e-12
    grad = balance64(s, one)[3]
    up, down = s.copy(), s.copy()
    up[5, 3] += 1e-6
    down[5, 3] -= 1e-6
    d = (balance64(up, one)[0][0] - balance64(down, one)[0][0]) / 2e-6
    assert abs(d - grad[5, 3]) < 1e-8


def test_plain_rounding_is_nearest():
    """The tests' own MXFP4 rounding: no grid value is nearer, scales as stated."""
    rng = np.random.default_rng(1)
    v = rng.standard_normal((20, 70)) * np.exp2(rng.integers(-20, 20, (20, 1)).astype(float))
    r = mx_round64(v)
    codes, sb = mx_encode64(v)
    grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6.0])
    scale = np.repeat(np.ldexp(1.0, sb.astype(int) - 127), 32, axis=1)[:, :70]
    near = np.abs(np.abs(v)[..., None] - grid * scale[..., None]).min(-1)
    assert np.allclose(np.abs(v - r), near)
    v[0, 3], v[1, 40] = np.inf, np.nan
    bad = np.isnan(mx_round64(v))
    assert bad[0, :32].all() and bad[1, 32:64].all() and bad.sum() == 64
