"""The vocabulary loss and its gradient on the GPU against the 64-bit form, element by element.

Tolerances, counted in roundings. A logit: K/16 tensor-core steps, each a truncation of at most 2^-23 of what it
holds (at most S = sum |x w|), and 16 more for the additions inside a step: e = (K/16 + 16) 2^-23 S. The loss is
a mean of logits against the target's, so it is off by at most e (largest over the words) plus the target's own
(32 additions after K/32 in a lane: less than e), plus a few steps of the exponentials (2^-21 (1 + |d|)) and of
itself. The gradient: each weight p_v is off by that relatively and by half a bf16 step (2^-8), the sum over the
words by (V/16 + 16) 2^-23 of sum p |W|, the result by half a bf16 step. fp32 and bf16 end at 2^-126: a weight
below it may be lost whole, so V words can lose V 2^-126 of the loss and V 2^-126 max |W| of a gradient.
"""
import math

import pytest
import torch

from oracle import decoder_ops as R64

pytestmark = pytest.mark.gpu


def case(T, V, K, seed=0, lean=0.3, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    W = (torch.randn(V, K, device="cuda", generator=g) * 0.1).bfloat16()
    y = torch.randint(0, V, (T,), device="cuda", generator=g)
    X = (scale * (torch.randn(T, K, device="cuda", generator=g) + lean * W[y].float() / 0.1)).bfloat16()
    return X, W, y


def tolerances(X, W, y, g, ignore=-100):
    X64, W64 = X.double(), W.double()
    V, K = W.shape
    at = torch.where(y != ignore, y, 0).long()
    l = X64 @ W64.t()
    S = X64.abs() @ W64.abs().t()
    d = (l - l.gather(1, at[:, None])).abs()
    e = ((K / 16 + 16) * 2.0 ** -23 * S + 2.0 ** -21 * (1 + d)).amax(1) * 2 + 2.0 ** -20
    loss, _ = R64.vocab_loss(X, W, y, ignore=ignore)
    # d loss = sum p (d l_v - d l_y): nothing of it where the target has all of the probability
    rest = -torch.expm1(-loss)
    tl = e * (rest + e).clamp(max=1.0) + 2.0 ** -22 * loss + V * 2.0 ** -126
    p = torch.softmax(l, 1)
    p.scatter_(1, at[:, None], rest[:, None])
    mass = p @ W64.abs()
    tx = mass * ((2.0 ** -8 + 2 * e) * 1.01 + (V / 16 + 16) * 2.0 ** -23)[:, None] + V * 2.0 ** -126 * W64.abs().max()
    return tl, tx * g.double().abs()[:, None] + 2.0 ** -126


def check(lib, X, W, y, g=None, ignore=-100, **kw):
    ones = torch.ones(X.shape[0], device="cuda") if g is None else g
    with torch.no_grad():
        ref, dref = R64.vocab_loss(X, W, y, g, ignore)
        used = y != ignore
        X0 = torch.where(used[:, None], X, 0)
        tl, tx = tolerances(X0, W, y, ones, ignore)
        loss, dX = lib.vocab_loss(X, W, y, ignore_index=ignore, reduction="none", dloss=g, **kw)
        assert lib.get_status() == 0
        off = (loss.double() - ref).abs()
        assert bool((off <= tl).all()), (float((off - tl).max()), int((off - tl).argmax()))
        off = (dX.double() - dref).abs()
        lim = tx + (dref.abs() + tx) * 2.0 ** -8
        assert bool((off <= lim).all()), (float((off - lim).max()), float((off / lim.clamp_min(1e-300)).max()))
        # the loss alone is the same loss, bit for bit
        alone, none = lib.vocab_loss(X, W, y, ignore_index=ignore, reduction="none", need_dx=False)
        assert none is None and torch.equal(alone, loss)
    return loss, dX


@pytest.mark.parametrize("T,V,K", [(1, 1, 8), (1, 2, 64), (3, 17, 72), (5, 255, 8), (127, 256, 136), (128, 257, 64),
                                   (129, 1000, 264), (300, 511, 520), (1, 32000, 256), (257, 5003, 64)])
def test_sizes(lib, T, V, K):
    check(lib, *case(T, V, K))


def test_token_gradients_and_ignored_tokens(lib):
    X, W, y = case(200, 700, 96, seed=1)
    y[::3] = -100
    X[3] = float("nan")                                   # what stands in an ignored token does not matter
    g = torch.randn(200, device="cuda", generator=torch.Generator("cuda").manual_seed(9))
    loss, dX = check(lib, X, W, y, g)
    assert bool((loss[::3] == 0).all()) and bool((dX[::3] == 0).all())
    check(lib, X, W, torch.where(y < 0, 5, y).int(), ignore=5)    # int32 targets, another index left out


def test_all_tokens_ignored(lib):
    X, W, _ = case(70, 300, 64)
    y = torch.full((70,), -100, device="cuda")
    loss, dX = lib.vocab_loss(X, W, y)
    assert torch.isnan(loss) and bool((dX == 0).all())
    loss, dX = lib.vocab_loss(X, W, y, reduction="sum")
    assert float(loss) == 0.0 and bool((dX == 0).all()) and lib.get_status() == 0


def test_far_apart_logits(lib):
    """Targets hundreds below the best word (every tile has a shift, and different ones), hundreds above it, and
    rows of both kinds in one tile; equal logits."""
    X, W, y = case(140, 1500, 64, seed=2, lean=0.0, scale=60.0)
    X[::2] = case(140, 1500, 64, seed=2, lean=3.0, scale=40.0)[0][::2]
    loss, dX = check(lib, X, W, y)
    assert float(loss[1::2].max()) > 88 and float(loss[::2].min()) == 0.0
    assert bool(torch.isfinite(dX.float()).all())
    X.zero_()
    loss, _ = check(lib, X, W, y)


def test_reductions_and_pieces(lib):
    """More tokens than one piece of the workspace takes (a large vocabulary), reduced in the call."""
    X, W, y = case(1100, 131072, 64, seed=3)
    y[::7] = -100
    ref, _ = R64.vocab_loss(X, W, y)
    n = int((y != -100).sum())
    g = (y != -100).float() / n
    each, dX = check(lib, X, W, y, g)
    mean, dmean = lib.vocab_loss(X, W, y)
    total, dsum = lib.vocab_loss(X, W, y, reduction="sum")
    # the sum of the tokens' fp32 losses in fp64, rounded once
    assert abs(float(mean) - float(each.double().sum()) / n) <= 2.0 ** -23 * float(mean)
    assert abs(float(total) - float(each.double().sum())) <= 2.0 ** -23 * float(total)
    assert abs(float(mean) - float(ref.sum()) / n) <= 1e-4 * float(mean)
    _, dones = lib.vocab_loss(X, W, y, reduction="none")
    assert torch.equal(dsum, dones)
    d = (dmean.double() - dX.double()).abs()              # g = 1 / n formed in one division either way
    assert bool((d <= 2.0 ** -7 * dX.double().abs()).all())


def test_split_vocabulary_is_deterministic(lib):
    """A few tokens and features: the gradient's vocabulary is split over the SMs."""
    X, W, y = case(4, 9000, 128, seed=4)
    a = check(lib, X, W, y)
    b = lib.vocab_loss(X, W, y, reduction="none")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_targets_outside_the_vocabulary(lib):
    X, W, y = case(130, 300, 64, seed=5)
    bad = y.clone()
    bad[7], bad[9], bad[128] = 300, -1, 1 << 40
    loss, dX = lib.vocab_loss(X, W, bad, reduction="none")
    assert lib.get_status() == lib.STATUS_TARGET and lib.get_status() == 0
    rows = [7, 9, 128]
    assert bool((loss[rows] == 0).all()) and bool((dX[rows] == 0).all())
    keep = torch.ones(130, dtype=torch.bool, device="cuda")
    keep[rows] = False
    ok, dok = lib.vocab_loss(X, W, y, reduction="none")
    assert torch.equal(loss[keep], ok[keep]) and torch.equal(dX[keep], dok[keep])


def test_guards_around_every_output_and_the_workspace(lib):
    T, V, K = 131, 777, 72
    X, W, y = case(T, V, K, seed=6)
    need = lib.vocab_loss_workspace_bytes(T, V, K, True)
    ws = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    buf = torch.full((T * K + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    dX = buf[2048:2048 + T * K].view(T, K)
    loss, _ = lib.vocab_loss(X, W, y, reduction="none", dX=dX, workspace=ws[4096:4096 + need])
    ref, dref = lib.vocab_loss(X, W, y, reduction="none")
    assert torch.equal(loss, ref) and torch.equal(dX, dref)
    assert bool((ws[:4096] == 0xA5).all()) and bool((ws[4096 + need:] == 0xA5).all())
    assert bool((buf[:2048] == 7).all()) and bool((buf[2048 + T * K:] == 7).all())


def test_autograd(lib):
    from bit_nf4_quantized_14_b200.autograd import vocab_loss
    X, W, y = case(150, 600, 64, seed=7)
    y[5] = -100
    for red in ("mean", "sum"):
        x = X.view(3, 50, 64).clone().requires_grad_()
        loss = vocab_loss(x, W, y.view(3, 50), reduction=red)
        (3.0 * loss).backward()
        ref, dref = lib.vocab_loss(X, W, y, reduction=red)
        assert torch.equal(loss.detach(), ref)
        lim = 2.0 ** -8 * (3 * dref.double()).abs()       # one more rounding to bf16
        assert bool(((x.grad.view(150, 64).double() - 3 * dref.double()).abs() <= lim).all())
    x = X.clone().requires_grad_()
    g = torch.rand(150, device="cuda")
    vocab_loss(x, W, y, reduction="none").backward(g)
    assert torch.equal(x.grad, lib.vocab_loss(X, W, y, reduction="none", dloss=g)[1])
    with torch.no_grad():
        assert vocab_loss(X, W, y).requires_grad is False
    with pytest.raises(ValueError):
        vocab_loss(X, W.clone().requires_grad_(), y)          # the head is frozen
    x = X.clone().requires_grad_()
    (dx,) = torch.autograd.grad(vocab_loss(x, W, y), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()                                   # once differentiable


def test_gradient_against_differences(lib):
    """Along one direction, a step of the fp32 loss itself (64-bit logits of the moved input are not needed: the
    sum of 20 tokens' losses moves by 1e-1 and is good to 1e-4)."""
    X, W, y = case(20, 400, 64, seed=8)
    g = torch.Generator("cuda").manual_seed(1)
    d = torch.randn(20, 64, device="cuda", generator=g)
    up, dn = ((X.float() + s * 0.0625 * d).bfloat16() for s in (1, -1))
    moved = up.double() - dn.double()
    _, dX = lib.vocab_loss(X, W, y, reduction="sum")
    diff = lib.vocab_loss(up, W, y, reduction="sum", need_dx=False)[0] - lib.vocab_loss(dn, W, y, reduction="sum", need_dx=False)[0]
    ref = R64.vocab_loss(up, W, y)[0].sum() - R64.vocab_loss(dn, W, y)[0].sum()
    lin = (R64.vocab_loss(X, W, y)[1] * moved).sum()
    assert abs(float(diff) - float(ref)) < 1e-3
    # the gradient predicts the step as well as the exact one does, up to its bf16 roundings
    assert abs(float((dX.double() * moved).sum()) - float(lin)) <= 2.0 ** -6 * float((dX.double() * moved).abs().sum())
    assert abs(float(lin) - float(ref)) <= 0.05 * abs(float(ref)) + 0.05


def test_capture_streams_and_two_calls_at_once(lib):
    X, W, y = case(160, 900, 128, seed=9)
    X2, _, y2 = case(160, 900, 128, seed=10)
    ref, dref = lib.vocab_loss(X, W, y)
    ref2, dref2 = lib.vocab_loss(X2, W, y2)
    need = lib.vocab_loss_workspace_bytes(160, 900, 128, True)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    x, t, dX = X.clone(), y.clone(), torch.empty_like(X)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        loss, _ = lib.vocab_loss(x, W, t, dX=dX, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, ref) and torch.equal(dX, dref)
    x.copy_(X2)
    t.copy_(y2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, ref2) and torch.equal(dX, dref2)
    # two streams, workspaces of their own
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for st, (a, b) in zip(s, ((X, y), (X2, y2))):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append(lib.vocab_loss(a, W, b))
    torch.cuda.synchronize()
    assert torch.equal(got[0][1], dref) and torch.equal(got[1][1], dref2) and lib.get_status() == 0


def test_backward_captured_beside_an_eager_graph(lib):
    """A training step captured while an eager loss of the same leaf is still alive, replayed on new inputs. (The
    eager one is built on the capturing stream too: torch ties a leaf's gradient to the stream of its first live
    graph, and refuses to capture, for any operator, where that is the default stream.)"""
    from bit_nf4_quantized_14_b200.autograd import vocab_loss
    X, W, y = case(150, 900, 64, seed=11)
    x = X.clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        alive = vocab_loss(x, W, y)
        (warm,) = torch.autograd.grad(vocab_loss(x, W, y), x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loss = vocab_loss(x, W, y)
        (dx,) = torch.autograd.grad(loss, x)
    X2, _, y2 = case(150, 900, 64, seed=12)
    with torch.no_grad():
        x.copy_(X2)
        y.copy_(y2)
    graph.replay()
    torch.cuda.synchronize()
    ref, dref = lib.vocab_loss(X2, W, y2)
    assert torch.equal(loss, ref) and torch.equal(dx, dref)
    (da,) = torch.autograd.grad(alive, x)
    assert torch.equal(da, warm)


def test_refusals(lib):
    X, W, y = case(8, 64, 64)
    for bad in (dict(X=X.float()), dict(X=X[:, :32]), dict(W=W.half()), dict(targets=y.float()), dict(targets=y[:4]),
                dict(reduction="max"), dict(dloss=torch.ones(8, device="cuda")),
                dict(reduction="none", dloss=torch.ones(7, device="cuda")), dict(targets=y.cpu()), dict(X=X.cpu()),
                dict(dX=torch.empty(8, 32, device="cuda", dtype=torch.bfloat16))):
        a = dict(X=X, W=W, targets=y)
        a.update(bad)
        with pytest.raises(ValueError):
            lib.vocab_loss(**a)
    with pytest.raises(lib.QLoRAError) as e:
        lib.vocab_loss(X, W, y, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -4
    with pytest.raises(lib.QLoRAError) as e:
        lib.vocab_loss(X[:, :60].contiguous(), W[:, :60].contiguous(), y)
    assert e.value.code == -2


def test_broadcast_workspace_is_refused(lib):
    """Its numel is that of a real workspace, its memory one byte (refused on the host, before any launch)."""
    X = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(10, 64, dtype=torch.bfloat16, device="cuda")
    need = lib.vocab_loss_workspace_bytes(4, 10, 64, True)
    one = torch.empty(1, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        lib.vocab_loss(X, W, torch.zeros(4, dtype=torch.int64, device="cuda"), workspace=one.expand(need))


def test_memory_of_a_call_on_a_given_stream_is_the_streams(lib, monkeypatch):
    """Every tensor that the operators make for themselves is allocated with the stream of the call current."""
    side = torch.cuda.Stream()
    X, W, tg, codes, absmax = (torch.zeros(*s, dtype=t, device="cuda") for s, t in (
        ((4, 64), torch.bfloat16), ((10, 64), torch.bfloat16), ((4,), torch.int64), ((320,), torch.uint8),
        ((10,), torch.float32)))
    torch.cuda.synchronize()
    seen = []
    for name in ("empty", "empty_like"):
        make = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, make=make, **k: (
            seen.append(torch.cuda.current_stream().cuda_stream), make(*a, **k))[1])
    loss, dX = lib.vocab_loss(X, W, tg, stream=side)
    q, _ = lib.rotary(X.view(4, 1, 64), None, lib.RotaryConfig(64), stream=side)
    Y = lib.codebook_linear(X, codes, absmax, 10, lib.codebook()[0], stream=side)
    monkeypatch.undo()
    side.synchronize()
    assert len(seen) == 5 and set(seen) == {side.cuda_stream}        # dX, workspace, loss; q'; Y
    assert abs(float(loss) - math.log(10.0)) < 1e-5                  # ten equal logits; fp32: 2.3 * 2^-24 a rounding
    assert not dX.any() and not q.any() and not Y.any()


@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
@pytest.mark.parametrize("first", [1, 2, 3, 5])
def test_targets_and_token_gradients_that_begin_anywhere(lib, dtype, first):
    """The next-token shift of one sequence: ids[first:] begins 4 to 40 bytes into its memory. Its copy gives the
    reference, bit for bit."""
    from bit_nf4_quantized_14_b200.autograd import vocab_loss
    X, W, y = case(60, 300, 64, seed=13)
    ids = torch.cat([torch.zeros(first, dtype=torch.int64, device="cuda"), y]).to(dtype)
    ids[first + 3] = -100
    view, copy = ids[first:], ids[first:].clone()
    g = torch.rand(60 + first, device="cuda")
    for red, d, d0 in (("mean", None, None), ("none", g[first:], g[first:].clone())):
        got, ref = (lib.vocab_loss(X, W, t, reduction=red, dloss=w) for t, w in ((view, d), (copy, d0)))
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]) and lib.get_status() == 0
    x, x0 = (X.clone().requires_grad_() for _ in range(2))
    for red in ("mean", "none"):
        for a, t in ((x, view), (x0, copy)):
            vocab_loss(a.view(1, 60, 64), W, t.view(1, 60), reduction=red).sum().backward()
        assert torch.equal(x.grad, x0.grad)


def test_token_losses_of_joined_parts(lib):
    """Per-token losses joined by torch.cat: the second part's gradient is a view that begins 7 floats in."""
    from bit_nf4_quantized_14_b200.autograd import vocab_loss
    X, W, y = case(18, 300, 64, seed=14)
    w = torch.rand(18, device="cuda")
    x = X.clone().requires_grad_()
    parts = [vocab_loss(x[a:b], W, y[a:b], reduction="none") for a, b in ((0, 7), (7, 18))]
    (torch.cat(parts) * w).sum().backward()
    for a, b in ((0, 7), (7, 18)):
        ref = lib.vocab_loss(X[a:b].clone(), W, y[a:b].clone(), reduction="none", dloss=w[a:b].clone())[1]
        assert torch.equal(x.grad[a:b], ref)


@pytest.mark.parametrize("T,V,K", [(3, 40, 1032), (130, 257, 2056), (300, 511, 4104), (70, 1000, 8200), (257, 130, 16384)])
def test_long_contractions(lib, T, V, K):
    """More than one run of 1024 features, whole and near-equal ones, single CTAs and pairs."""
    check(lib, *case(T, V, K, seed=15, lean=0.05))


@pytest.mark.parametrize("T", [40, 200])
@pytest.mark.parametrize("K", [1024, 1032, 8192, 131072])
@pytest.mark.parametrize("kind", ["mixed", "one sign", "first 128", "last 128", "large first", "large last"])
def test_sums_do_not_drift(lib, kind, K, T):
    """A logit of about 12 against a target's of exactly 0, so the loss is log(1 + exp l): the error of l itself, for
    features that grow the sum in different ways.

    Bound: runs of at most 1024 features are summed in fp32. Inside a run each tensor-core step that adds something
    truncates by at most 2^-23 of what it holds, and the additions inside a step count as 16 more: (steps + 16) 2^-23 S,
    S = sum |x w|, steps = the most nonzero steps of one run. Adding the runs: 2^-24 S each. The loss: 2^-21 (1 + l).
    The kernel puts back 1.65e-8 of a run per step, which may not be missing: 1.06e-6 of each run of 64 steps more.
    The mean over the rows: half of 2^-23 of what each step holds is lost on average, at most a whole one: the sum over
    the steps of the 64-bit partial sums, times 2^-23; the roundings inside steps, of the runs and of the loss are of
    both signs, and the exponential's and the logarithm's own at most 2^-22 (1 + l)."""
    g = torch.Generator("cuda").manual_seed(K + T)
    x, w = torch.randn(T, K, device="cuda", generator=g), torch.randn(K, device="cuda", generator=g)
    if kind == "mixed":
        x, w = x + 12 / K ** 0.5 * w, w / K ** 0.5
    elif kind == "one sign":
        x, w = x.abs(), w.abs() * 12 * math.pi / 2 / K
    elif kind in ("first 128", "last 128"):
        keep = torch.arange(K, device="cuda") < 128 if kind == "first 128" else torch.arange(K, device="cuda") >= K - 128
        x, w = torch.where(keep, x.abs(), 0.0), torch.full_like(w, 15 / 128)
    else:
        at = 0 if kind == "large first" else K - 1
        w = w * 0.5 / K ** 0.5
        x[:, at], w[at] = 6.0, 2.0
    X, W = x.bfloat16(), torch.zeros(2, K, device="cuda", dtype=torch.bfloat16)
    W[0] = w.bfloat16()
    products = X.double() * W[0].double()
    l, S = products.sum(1), products.abs().sum(1)
    loss, _ = lib.vocab_loss(X, W, torch.ones(T, dtype=torch.int64, device="cuda"), reduction="none", need_dx=False)
    off = loss.double() - torch.nn.functional.softplus(l)
    steps = 8 if kind.endswith("128") else 64
    blocks = math.ceil(K / 64)
    runs = math.ceil(blocks / 16)
    parts = [products[:, 64 * (blocks * r // runs):64 * (blocks * (r + 1) // runs)] for r in range(runs)]
    back = 64 * 1.65e-8 * sum(p.sum(1).abs() for p in parts)
    lim = (steps + 16) * 2.0 ** -23 * S + back + math.ceil(K / 1024) * 2.0 ** -24 * S + 2.0 ** -21 * (1 + l.abs())
    assert bool((off.abs() <= lim).all()), float((off.abs() / lim).max())
    held = torch.zeros((), dtype=torch.float64, device="cuda")
    for part in parts:
        part = torch.nn.functional.pad(part, (0, -part.shape[1] % 16)).unflatten(1, (-1, 16)).sum(2).cumsum(1)
        held += part.abs().sum()
    lim = 2.0 ** -23 * held / T + back.mean() + 2.0 ** -22 * (1 + l.mean())
    assert abs(float(off.mean())) <= float(lim), (float(off.mean()), float(lim))


def test_pieces_of_long_rows(lib):
    """512 rows of 2^17 features are what a piece's copy of X takes: three pieces, with the gradient and without, tokens
    left out and none."""
    X, W, y = case(1100, 40, 1 << 17, seed=16, lean=0.0, scale=0.03)
    check(lib, X, W, y)
    y[::5] = -100
    check(lib, X, W, y)


def test_hidden_state_that_begins_anywhere(lib):
    """One token's features behind 9 others of its row: a contiguous view 18 bytes in."""
    from bit_nf4_quantized_14_b200.autograd import vocab_loss
    X, W, y = case(1, 300, 64, seed=17)
    row = torch.cat([torch.zeros(1, 9, dtype=torch.bfloat16, device="cuda"), X], -1).requires_grad_()
    for red in ("mean", "none"):
        row.grad = None
        loss = vocab_loss(row[:, 9:], W, y, reduction=red)
        loss.sum().backward()
        ref, dref = lib.vocab_loss(X, W, y, reduction=red)
        assert torch.equal(loss.detach(), ref) and torch.equal(row.grad[:, 9:], dref) and not row.grad[:, :9].any()
