"""Rotary positions on the GPU against the 64-bit form, element by element.

Tolerance, counted in roundings: the fraction of a turn is rounded to fp32 (2^-26 turns at most, 2 pi 2^-26 of
angle) and sine and cosine are good to a few units in 2^-24, so each is within 2^-22; two products and a sum
add 3 x 2^-24 relative to m (|a| + |b|); a bf16 result adds half a step, 2^-8 of its value.
"""
import pytest
import torch

from oracle import decoder_ops as R64

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def bound(x, ref, R, layout, m):
    """Elementwise: m (|a| + |b|) (2^-22 + 3 2^-24) + half a step of the result (and of what that is off by)."""
    a = x.double().abs()
    pair = torch.zeros_like(a)
    lo, hi = (slice(0, R // 2), slice(R // 2, R)) if layout == "half" else (slice(0, R, 2), slice(1, R, 2))
    pair[..., lo] = pair[..., hi] = a[..., lo] + a[..., hi]
    t = m * pair * (2.0 ** -22 + 3 * 2.0 ** -24)
    return t + (ref.abs() + t) * HALF_STEP[x.dtype] * (pair > 0)


def check(q, qx, kx, cfg, positions=None, offset=0, inverse=False, out=None, kw64=None):
    B, T = qx.shape[:2]
    pos = (torch.arange(T, device="cuda").expand(B, T) if positions is None else positions.expand(B, T)) + offset
    theta, m = R64.rope_frequencies(cfg.rotary_dim, **(kw64 or {}))
    refs = [None if x is None else R64.rope(x, pos, theta, m, cfg.layout, inverse) for x in (qx, kx)]
    tols = [None if x is None else bound(x, r, cfg.rotary_dim, cfg.layout, m) for x, r in zip((qx, kx), refs)]
    got = q.rotary(qx, kx, cfg, positions, offset, inverse, out)
    for g, r, t in zip(got, refs, tols):
        if r is not None:
            assert bool(((g.double() - r).abs() <= t).all()), float(((g.double() - r).abs() - t).max())
    return got


def rand(shape, dtype, seed=0):
    return torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (80, 36), (64, 62), (33, 2), (96, 24), (576, 512), (2, 2)])
def test_sizes_types_layouts(lib, layout, dtype, D, R):
    """Every access width, odd head sizes, rotated parts; one token, several, more than one CTA's worth."""
    for B, T, Hq, Hk in ((1, 1, 1, 1), (2, 7, 5, 1), (1, 2500, 3, 2)):
        check(lib, rand((B, T, Hq, D), dtype, 1), rand((B, T, Hk, D), dtype, 2), lib.RotaryConfig(R, layout=layout),
              offset=5)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "banded", "yarn"])
def test_scalings_far_positions_and_inverse(lib, scaling):
    kw = dict(base=500000.0, scaling=scaling, factor=8.0, original_length=8192.0)
    pos = torch.randint(0, 1 << 24, (3, 65), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    pos[0, 0], pos[0, 1] = (1 << 31) - 1, -17
    cfg = lib.RotaryConfig(64, **kw)
    x, k = rand((3, 65, 4, 128), torch.float32), rand((3, 65, 2, 128), torch.float32, 4)
    for inverse in (False, True):
        check(lib, x, k, cfg, pos, inverse=inverse, kw64=kw)
    check(lib, x, None, cfg, pos.clamp(max=1 << 30).to(torch.int32), offset=1 << 20, kw64=kw)
    check(lib, x, k, cfg, pos[1], kw64=kw)                     # one row of positions for every batch row


def test_strides(lib):
    """Views of a fused projection, heads before tokens, odd strides, expanded rows; outputs of other strides."""
    cfg = lib.RotaryConfig(32, layout="interleaved")
    qkv = rand((2, 9, 3 * 4, 48), torch.bfloat16)
    check(lib, qkv[:, :, :4], qkv[:, :, 4:8], cfg)
    h = rand((2, 4, 9, 48), torch.bfloat16).transpose(1, 2)
    got, _ = check(lib, h, None, cfg, out=(torch.empty(2, 9, 4, 48, device="cuda", dtype=torch.bfloat16), None))
    assert got.is_contiguous()
    for layout in ("half", "interleaved"):
        odd = rand((2, 9, 3, 51), torch.bfloat16)[..., :48]     # rows 51 apart: no wide access fits
        check(lib, odd, odd, lib.RotaryConfig(32, layout=layout), offset=3)
    one = rand((1, 9, 4, 48), torch.float32).expand(3, 9, 4, 48)
    out = torch.empty(3, 9, 4, 48, device="cuda")
    check(lib, one, None, cfg, out=(out, None))
    assert lib.rotary(one[0], None, cfg)[0].equal(out[0])       # (T, heads, dim)
    assert lib.rotary(one, None, cfg)[0].equal(out)             # an expanded input gets an output of its own


def test_more_batch_rows_than_a_grid_takes(lib):
    x = rand((65535 + 300, 1, 1, 4), torch.float32)
    pos = torch.randint(0, 1000, (65835, 1), device="cuda", dtype=torch.int32)
    check(lib, x, None, lib.RotaryConfig(4, layout="interleaved"), pos)


def test_in_place_touches_nothing_else(lib):
    buf = rand((1, 70, 6, 64), torch.bfloat16)
    keep = buf.clone()
    q, k = buf[:, :64, :3], buf[:, :64, 3:5]
    cfg = lib.RotaryConfig(48)
    ref = lib.rotary(q, k, cfg, offset=9)
    lib.rotary(q, k, cfg, offset=9, out=(q, k))
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1])
    assert torch.equal(buf[:, 64:], keep[:, 64:]) and torch.equal(buf[:, :, 5], keep[:, :, 5])


def test_gradients(lib):
    from bit_nf4_quantized_14_b200.autograd import rotary
    cfg = lib.RotaryConfig(16, layout="half")
    pos = torch.tensor([3, 50, 7], device="cuda")
    q, k = rand((3, 4, 24), torch.float32).requires_grad_(), rand((3, 2, 24), torch.float32, 1).requires_grad_()
    qo, ko = rotary(q, k, cfg, pos)
    dq, dk = rand((3, 4, 24), torch.float32, 2), rand((3, 2, 24), torch.float32, 3)
    (qo * dq).sum().add((ko * dk).sum()).backward()
    theta, m = R64.rope_frequencies(16)
    for x, d in ((q, dq), (k, dk)):
        ref = R64.rope(d[None], pos[None], theta, m, "half", True)[0]
        assert bool(((x.grad.double() - ref).abs() <= bound(d[None], ref[None], 16, "half", m)[0]).all())
        # against differences of the forward, in one direction: the operator is linear
        e = torch.zeros_like(x)
        e[1, 1, 2] = 1.0
        y = lib.rotary(e, None, cfg, pos)[0]
        assert abs(float((y * d).sum() - x.grad[1, 1, 2])) < 1e-6
    only, none = rotary(q, None, cfg, pos)
    only.sum().backward()
    assert none is None


def test_capture_and_streams(lib):
    """A captured call replays on new contents; a call on another stream than the tensors' own."""
    cfg = lib.RotaryConfig(64)
    x, pos = rand((1, 1, 8, 64), torch.bfloat16), torch.zeros(1, dtype=torch.int64, device="cuda")
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lib.rotary(x, None, cfg, pos, out=(out, None))
    for p in (0, 12345):
        x.copy_(rand(x.shape, x.dtype, p))
        pos.fill_(p)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, lib.rotary(x, None, cfg, pos)[0])
    with torch.cuda.stream(side):
        got = lib.rotary(x, None, cfg, pos)[0]
    side.synchronize()
    assert torch.equal(got, out)


def test_refusals(lib):
    x = rand((2, 3, 4, 32), torch.bfloat16)
    cfg = lib.RotaryConfig(32)
    for bad in (x.cpu(), x.half(), x[..., ::2], x[0, 0]):
        with pytest.raises(ValueError):
            lib.rotary(bad, None, lib.RotaryConfig(16))
    with pytest.raises(ValueError):
        lib.rotary(x, x[:, :2], cfg)
    with pytest.raises(ValueError):
        lib.rotary(x, x.float(), cfg)
    with pytest.raises(ValueError):
        lib.rotary(x, None, cfg, torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        lib.rotary(x, None, cfg, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        lib.rotary(x, None, lib.RotaryConfig(32, layout="pairs"))
    with pytest.raises(ValueError):
        lib.rotary(x, x, cfg, out=(x, x))
    for R in (48, 31):
        with pytest.raises(lib.QLoRAError):
            lib.rotary(x, None, lib.RotaryConfig(R))
    with pytest.raises(lib.QLoRAError) as e:
        lib.rotary(x[:, :0], None, cfg)
    assert e.value.code == -2
    with pytest.raises(lib.QLoRAError) as e:
        lib.rotary(rand((1, 1, 1, 40), torch.bfloat16)[..., 1:33], None, cfg)
    assert e.value.code == -3


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("prefix", [1, 4, 7, 36])
def test_gradients_that_begin_anywhere(lib, dtype, prefix):
    """A rotated part joined behind other features of its head, for one token (whose gradient is a contiguous view
    `prefix` features in) and for several, and behind other heads; heads that are such a part themselves. Copies give
    the reference, bit for bit."""
    from bit_nf4_quantized_14_b200.autograd import rotary
    cfg = lib.RotaryConfig(16)
    for T, H in ((1, 1), (5, 3)):
        whole = rand((T, H, prefix + 24), dtype).requires_grad_()
        w = rand((T, H, prefix + 24), dtype, 1)
        turned, none = rotary(whole[..., prefix:], None, cfg, offset=3)
        assert none is None and torch.equal(turned, lib.rotary(whole[..., prefix:].detach().clone(), None, cfg, offset=3)[0])
        torch.cat([whole[..., :prefix], turned], -1).backward(w)
        ref = lib.rotary(w[..., prefix:].clone(), None, cfg, offset=3, inverse=True)[0]
        assert torch.equal(whole.grad[..., prefix:], ref) and torch.equal(whole.grad[..., :prefix], w[..., :prefix])
    q, k = rand((4, 3, 17), dtype).requires_grad_(), rand((4, prefix, 17), dtype, 1).requires_grad_()
    qo, ko = rotary(q, k, cfg)
    w = rand((4, prefix + 3, 17), dtype, 2)
    torch.cat([ko, qo], 1).backward(w)
    assert torch.equal(q.grad, lib.rotary(w[:, prefix:].clone(), None, cfg, inverse=True)[0])
    assert torch.equal(k.grad, lib.rotary(w[:, :prefix].clone(), None, cfg, inverse=True)[0])
