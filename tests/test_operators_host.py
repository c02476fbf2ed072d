"""Rotary positions, the vocabulary loss and the 4-bit product through the C ABI without a GPU: frequencies
against their closed forms, workspace plans, and every refusal before any CUDA call."""
import ctypes

import numpy as np
import pytest

from oracle import decoder_ops as R64

V = ctypes.c_void_p
F = ctypes.c_float


@pytest.fixture(scope="module")
def q():
    from bit_nf4_quantized_14_b200 import build
    build.build()
    import bit_nf4_quantized_14_b200 as mod
    return mod


@pytest.mark.parametrize("R", [2, 4, 36, 64, 128, 512])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "banded", "yarn"])
def test_rope_frequencies(q, R, scaling):
    if scaling == "ntk" and R == 2:
        with pytest.raises(q.QLoRAError):
            q.RotaryConfig(R, scaling=scaling, factor=2.0).frequencies()
        return
    for kw in (dict(factor=1.0), dict(factor=4.0), dict(factor=8.0, base=500000.0)):
        kw = {**kw, "original_length": 8192.0} if scaling in ("banded", "yarn") else kw
        th, m = q.RotaryConfig(R, scaling=scaling, **kw).frequencies()
        ref, mr = R64.rope_frequencies(R, scaling=scaling, **kw)
        # a power of a rounded exponent: a few ulps of |ln| <= 14
        assert np.allclose(th, ref.numpy(), rtol=2.0 ** -47, atol=0) and abs(m - mr) < 1e-15, (kw, th / ref.numpy())


def test_rope_refusals(q):
    th = (ctypes.c_double * 64)(*([0.5] * 64))
    m = ctypes.c_double()
    fr = q.lib.qlora_rope_frequencies
    ok = (128, 1e4, 4, 4.0, 4096.0, 1.0, 32.0)
    assert fr(*ok, th, ctypes.byref(m)) == 0
    for i, bad, rc in [(0, 0, -2), (0, 3, -2), (0, 514, -2), (1, 1.0, -1), (1, float("nan"), -1), (2, 5, -1), (2, -1, -1),
                       (3, 0.5, -1), (3, float("inf"), -1), (4, 0.0, -1), (5, 0.0, -1), (5, 32.0, -1)]:
        a = list(ok)
        a[i] = bad
        assert fr(*a, th, ctypes.byref(m)) == rc, (i, bad)
    assert fr(*ok, None, ctypes.byref(m)) == -1

    def call(nx=1, dtype=1, B=1, T=4, D=128, R=128, layout=0, theta=th, mscale=1.0, pos=None, pd=1, ptr=0x100000,
             heads=2, tensors=True):
        s = (q._RopeTensor * 2)(*[(ptr, 0x200000, heads, 1024, 256, 128, 1024, 256, 128)] * 2)
        return q.lib.qlora_rope(ctypes.cast(s, V) if tensors else None, nx, dtype, B, T, D, R, layout, theta, mscale, pos, pd, 0, 0, 0,
                                None)

    assert call(tensors=False) == -1 and call(nx=0) == -1 and call(nx=3) == -1 and call(dtype=2) == -1
    assert call(layout=2) == -1 and call(theta=None) == -1 and call(mscale=float("nan")) == -1
    assert call(pos=V(0x300000), pd=7) == -1 and call(ptr=0) == -1
    for kw in (dict(B=0), dict(T=0), dict(T=1 << 31), dict(D=64), dict(D=1026), dict(R=0), dict(R=127), dict(heads=0),
               dict(heads=1 << 20), dict(B=1 << 40, T=1 << 40)):
        assert call(**kw) == -2, kw
    assert call(ptr=0x100002) == -3
    bad = (ctypes.c_double * 64)(*([float("inf")] * 64))
    assert call(theta=bad) == -1


def test_vocab_loss_refusals_and_workspace(q):
    X, W, Y, L, D, ws = V(0x300000), V(0x310000), V(0x320000), V(0x330000), V(0x340000), V(0x400000)
    big = 1 << 40

    def call(X=X, T=8, W=W, Vn=100, K=64, y=Y, td=1, red=2, dl=None, loss=None, total=L, dX=D, ws=ws, nb=big):
        return q.lib.qlora_vocab_loss(X, T, W, Vn, K, y, td, -100, red, dl, loss, total, dX, ws, nb, None)

    assert call(X=None) == -1 and call(W=None) == -1 and call(y=None) == -1 and call(td=2) == -1
    assert call(red=3) == -1 and call(red=-1) == -1 and call(total=None) == -1
    assert call(red=0, total=None) == -1 and call(red=0, loss=L) == -1      # per token: loss, and no total
    assert call(dl=D) == -1                                                 # token gradients only per token
    for kw in (dict(T=0), dict(Vn=0), dict(K=0), dict(K=4), dict(K=68), dict(Vn=1 << 30), dict(T=1 << 40), dict(K=1 << 21)):
        assert call(**kw) == -2, kw
    for kw in (dict(X=V(0x300008)), dict(W=V(0x310002)), dict(y=V(0x320008)), dict(total=V(0x330004)), dict(dX=V(0x340008)),
               dict(ws=V(0x400008))):
        assert call(**kw) == -3, kw
    need = q.vocab_loss_workspace_bytes(8, 100, 64, True)
    assert call(nb=need - 1) == -4 and call(ws=None) == -4
    assert q.vocab_loss_workspace_bytes(8, 100, 64, False) < need
    # the buffer for the weights is bounded whatever the number of tokens
    at = [q.vocab_loss_workspace_bytes(t, 32000, 4096, True) for t in (8192, 65536)]
    # 2^26 bf16 weights, 3 fp32 tiles of 128 x 256 per SM, 2048 packed rows, 125 tiles' statistics twice, 16 B a token
    most = (1 << 27) + 3 * 148 * 128 * 256 * 4 + 2048 * 4096 * 2 + 2 * 125 * 2048 * 8 + (1 << 20)
    assert at[0] < most and at[1] - at[0] <= 57344 * 16 + (1 << 20)
    for bad in [(0, 100, 64), (8, 0, 64), (8, 100, 12)]:
        with pytest.raises(q.QLoRAError) as e:
            q.vocab_loss_workspace_bytes(*bad, True)
        assert e.value.code == -2


def test_codebook_linear_refusals(q):
    X, C, A, Y = V(0x300000), V(0x310000), V(0x320000), V(0x330000)
    lv = (F * 15)(*(np.arange(-7, 8, dtype=np.float32) / np.float32(7)).tolist())

    def call(X=X, T=1, C=C, A=A, N=16, K=128, levels=lv, nl=15, Y=Y):
        return q.lib.qlora_codebook_linear(X, T, C, A, N, K, levels, nl, Y, None)

    assert call(X=None) == -1 and call(C=None) == -1 and call(A=None) == -1 and call(Y=None) == -1
    for kw in (dict(T=0), dict(T=65), dict(N=0), dict(K=0), dict(K=96), dict(N=1 << 31), dict(K=1 << 31)):
        assert call(**kw) == -2, kw
    assert call(nl=1) == -10 and call(levels=None) == -10 and call(nl=17) == -10
    for kw in (dict(X=V(0x300008)), dict(C=V(0x310001)), dict(A=V(0x320004)), dict(Y=V(0x330002))):
        assert call(**kw) == -3, kw


def test_new_status_has_its_message(q):
    assert b"vocabulary" in q.lib.qlora_error_string(-11)


@pytest.mark.parametrize("gradient", [False, True])
@pytest.mark.parametrize("T", [1, 128, 8192, 16384, 65536, 1 << 20])
@pytest.mark.parametrize("V,K", [(32000, 4096), (131072, 8192), (1000000, 8192), (500, 1 << 20), (1 << 21, 64)])
def test_vocab_loss_workspace_is_bounded(q, gradient, T, V, K):
    """As documented: 12 bytes a token; a piece's rows of X, its tiles' sums (16 bytes per row and tile of 128 words at
    least) and its weights, each 128 MB or what 128 rows need; 59 MB of partial sums; 256 bytes of rounding a part."""
    most = lambda per_row: max(1 << 27, 128 * per_row)  # noqa: E731
    limit = 12 * T + most(2 * K) + most(16 * -(-V // 128)) + 12 * 16384 + (1 << 13)
    if gradient:
        limit += most(2 * (V + 15)) + 3 * 148 * 128 * 256 * 4
    assert q.vocab_loss_workspace_bytes(T, V, K, gradient) <= limit
