"""Rotary positions, the vocabulary loss and the 4-bit product together, as a decoder around the quantized linears
uses them: one training step, single-token generation, and the calls captured into graphs. Each operator is held
to its own 64-bit form on the tensors that it gets there (the tolerances of test_gpu_rope.py, test_gpu_vocab_loss.py
and test_gpu_codebook_linear.py)."""
import pytest
import torch

from oracle import decoder_ops as R64
from test_gpu_codebook_linear import check as check_linear
from test_gpu_rope import bound as rope_bound
from test_gpu_vocab_loss import tolerances as loss_tolerances

pytestmark = pytest.mark.gpu
D, HEADS, VOCAB, T = 256, 4, 1000, 70


def decoder(lib, **kw):
    import bench
    gen = torch.Generator("cuda").manual_seed(5)
    cfg = lib.RotaryConfig(D // HEADS, scaling="linear", factor=2.0)
    m = bench.build_decoder(layers=2, d=D, ffn=512, heads=HEADS, vocab=VOCAB, r=8, gen=gen, device="cuda", positions=cfg,
                            fused_loss=True, **kw)
    for p in m.parameters():                       # adapters that do something
        with torch.no_grad():
            p.add_(torch.randn(p.shape, device="cuda", generator=gen), alpha=0.02)
    ids = torch.randint(0, VOCAB, (T,), device="cuda", generator=gen)
    targets = torch.randint(0, VOCAB, (T,), device="cuda", generator=gen)
    targets[::9] = -100
    return m, cfg, ids, targets


def within(got, ref, tol):
    off = (got.double() - ref).abs()
    assert bool((off <= tol).all()), float((off - tol).max())


def test_training_step(lib, monkeypatch):
    from bit_nf4_quantized_14_b200 import autograd
    m, cfg, ids, targets = decoder(lib)
    seen = {"rope": [], "loss": []}
    rotary, vocab_loss = autograd.rotary, autograd.vocab_loss

    def watch(kind, inputs, outputs):
        for t in inputs + outputs:
            t.retain_grad()
        seen[kind].append((inputs, outputs))

    def rotary_seen(q, k, *a):
        q, k = (t if t.requires_grad else t.clone().requires_grad_() for t in (q, k))
        out = rotary(q, k, *a)
        watch("rope", [q, k], list(out))
        return out

    def loss_seen(x, *a):
        out = vocab_loss(x, *a)
        watch("loss", [x], [out])
        return out

    monkeypatch.setattr(autograd, "rotary", rotary_seen)
    monkeypatch.setattr(autograd, "vocab_loss", loss_seen)
    loss = m(ids, targets)
    loss.backward()
    assert lib.get_status() == 0 and len(seen["rope"]) == 2
    assert all(p.grad is not None and bool(torch.isfinite(p.grad).all()) and float(p.grad.norm()) > 0 for p in m.parameters())
    theta, ms = R64.rope_frequencies(D // HEADS, scaling="linear", factor=2.0)
    pos = torch.arange(T, device="cuda")[None]
    for ins, outs in seen["rope"]:
        for x, y in zip(ins, outs):
            for a, b, inv in ((x, y, False), (y.grad, x.grad, True)):
                ref = R64.rope(a[None], pos, theta, ms, "half", inv)
                within(b[None], ref, rope_bound(a[None], ref, D // HEADS, "half", ms))
    (x,), (l,) = seen["loss"][0]
    n = (targets != -100).sum()
    g = (targets != -100).float() / n
    each, dx = R64.vocab_loss(x.detach(), m.head, targets, g)
    tl, tx = loss_tolerances(x.detach(), m.head, targets, g)
    within(l.detach(), each.sum() / n, tl[targets != -100].sum() / n + 2.0 ** -23 * l.detach())
    # the gradient is rounded once by the operator and once by the scale of the loss's own gradient (1 here: exact)
    within(x.grad, dx, tx + (dx.abs() + tx) * 2.0 ** -8)


def test_generation_step(lib):
    """One token at a time: its positions as in the whole text, and its logits from a head in 4 bits."""
    m, cfg, ids, _ = decoder(lib)
    layer = m.layers[0]
    with torch.no_grad():
        h = m.emb[ids]
        q, k = layer.q(h).view(T, HEADS, -1), layer.k(h).view(T, HEADS, -1)
        qa, ka = lib.rotary(q, k, cfg)
        for t in (0, 1, T - 1):
            q1, k1 = lib.rotary(q[t:t + 1], k[t:t + 1], cfg, offset=t)
            assert torch.equal(q1[0], qa[t]) and torch.equal(k1[0], ka[t])
            at = torch.full((1,), t, dtype=torch.int32, device="cuda")
            assert torch.equal(lib.rotary(q[t:t + 1], None, cfg, at)[0][0], qa[t])
        lv = [v / 8 for v in range(-8, 8)]
        codes, absmax = lib.codebook_quantize(m.head, lv)
        logits = check_linear(lib, h[-1:].contiguous(), codes, absmax, VOCAB, lv)
        word = logits.argmax(-1)
        for b in (2, 16):                      # a batch of sequences gives the same token the same logits
            many = lib.codebook_linear(h[-1:].repeat(b, 1), codes, absmax, VOCAB, lv)
            assert torch.equal(many.argmax(-1), word.expand(b)) and torch.equal(many, many[:1].expand(b, -1))


def test_two_graphs_share_a_workspace(lib):
    """Two captured losses with one workspace, replayed in turn and interleaved with rotary calls; then eager again."""
    gen = torch.Generator("cuda").manual_seed(3)
    W = (torch.randn(VOCAB, D, device="cuda", generator=gen) * 0.1).bfloat16()
    xs = [torch.randn(n, D, device="cuda", generator=gen).bfloat16() for n in (300, 40)]
    ys = [torch.randint(0, VOCAB, (n,), device="cuda", generator=gen) for n in (300, 40)]
    need = max(lib.vocab_loss_workspace_bytes(n, VOCAB, D, True) for n in (300, 40))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    ref = [lib.vocab_loss(x, W, y) for x, y in zip(xs, ys)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    for x, y in zip(xs, ys):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(lib.vocab_loss(x, W, y, workspace=ws))
        graphs.append(g)
    for order in ((0, 1), (1, 0, 1, 0)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for (l, d), (lr, dr) in zip(outs, ref):
            assert torch.equal(l, lr) and torch.equal(d, dr)
    again = lib.vocab_loss(xs[0], W, ys[0], workspace=ws)
    assert torch.equal(again[1], ref[0][1]) and lib.get_status() == 0
