"""The product of a few tokens with a codebook-quantized weight against the 64-bit form, element by element.

Tolerance: each level is rounded to bf16 (2^-8 of it), the fp32 accumulation is off by at most a truncation
(2^-23) of what it holds in each of its K/16 tensor-core steps and by as much again for the blocks' sums:
sum |x w| (2^-8 + (K/8 + 64) 2^-23), and the result is rounded to bf16 (2^-8 of it). X is drawn with signs
independent of the weights, so the levels' roundings add up as a random walk: by Hoeffding's inequality their sum
passes 6 x 2^-8 sqrt(sum x^2 w^2) with a probability below 2 e^-18, whatever the weights.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import decoder_ops as R64

pytestmark = pytest.mark.gpu
INT4 = [k / 7 for k in range(-7, 8)]
GRID = [k / 8 for k in range(-8, 8)]


def check(lib, X, codes, absmax, N, levels, **kw):
    K = X.shape[1]
    W = R64.codebook_weight(codes, absmax, N, K, levels)
    ref = X.double() @ W.t()
    mass = X.double().abs() @ W.abs().t()
    t = mass * (2.0 ** -8 + (K / 8 + 64) * 2.0 ** -23)
    Y = lib.codebook_linear(X, codes, absmax, N, levels, **kw)
    off = (Y.double() - ref).abs()
    lim = t + (ref.abs() + t) * 2.0 ** -8
    assert bool((off <= lim).all()), float((off - lim).max())
    quad = (X.double().square() @ W.square().t()).sqrt()
    t = mass * (K / 8 + 64) * 2.0 ** -23 + 6 * 2.0 ** -8 * quad
    assert bool((off <= t + (ref.abs() + t) * 2.0 ** -8).all()), float((off - t).max())
    return Y


def weight(lib, N, K, levels, seed=0):
    w = torch.from_numpy(synth.weight_f32(N, K, seed=seed, tensor_id=91)).cuda()
    return lib.codebook_quantize(w, levels)


def tokens(T, K, seed=0):
    return torch.randn(T, K, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).bfloat16()


@pytest.mark.parametrize("N,K", [(1, 64), (7, 128), (16, 192), (17, 1024), (250, 1088), (1000, 2112), (4999, 512)])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 33, 64])
def test_sizes(lib, N, K, T):
    codes, absmax = weight(lib, N, K, INT4)
    check(lib, tokens(T, K), codes, absmax, N, INT4)


@pytest.mark.parametrize("levels", [INT4, GRID, [-1.0, 0.25, 1.0], [-0.5, 0.5]])
def test_codebooks(lib, levels):
    codes, absmax = weight(lib, 333, 640, levels, seed=3)
    check(lib, tokens(3, 640), codes, absmax, 333, levels)
    any_codes = torch.randint(0, 256, codes.shape, device="cuda").to(torch.uint8)   # codes past the levels read 0
    check(lib, tokens(3, 640), any_codes, absmax, 333, levels)


def test_single_weight_equals_its_dequantized_product(lib):
    w = torch.from_numpy(synth.weight_f32(512, 1024, seed=1, tensor_id=92)).cuda()
    q = lib.quantize_single(w)
    X = tokens(5, 1024)
    Y = lib.linear_single(X, q)
    assert torch.equal(Y, lib.codebook_linear(X, q.codes, q.absmax, 512, lib.codebook()[0]))
    ref = X.double() @ lib.dequantize_single(q, torch.float32).double().t()
    assert float((Y.double() - ref).norm() / ref.norm()) <= 5e-3


def test_each_token_and_block_by_itself(lib):
    """One nonzero element of X at a time picks one column of the weight, exactly level * absmax in bf16 steps."""
    N, K = 40, 320
    codes, absmax = weight(lib, N, K, GRID, seed=4)
    W = R64.codebook_weight(codes, absmax, N, K, GRID)
    for ks in (range(0, 64), range(250, 314)):
        X = torch.zeros(64, K, device="cuda", dtype=torch.bfloat16)
        for t, k in enumerate(ks):
            X[t, k] = 1.0
        Y = lib.codebook_linear(X, codes, absmax, N, GRID)
        assert torch.equal(Y, W[:, list(ks)].t().float().bfloat16())   # eighths: the level is exact in bf16


def test_zero_blocks_and_large_constants(lib):
    N, K = 20, 256
    codes, absmax = weight(lib, N, K, INT4)
    absmax[::3] = 0.0
    absmax[1] = 1e30
    check(lib, tokens(4, K), codes, absmax, N, INT4)


def test_long_rows(lib):
    """X of two tokens past what stays in shared memory, and one token just inside and outside of it."""
    for T, K in ((2, 24576 + 64), (1, 24576), (1, 24576 + 512), (2, 12288), (2, 12288 + 256)):
        codes, absmax = weight(lib, 9, K, GRID, seed=K)
        check(lib, tokens(T, K), codes, absmax, 9, GRID)


def test_tokens_do_not_mix(lib):
    """An infinite or NaN token leaves the others as they are."""
    codes, absmax = weight(lib, 50, 512, INT4)
    for T in (2, 8, 16, 40):
        X = tokens(T, 512)
        ref = lib.codebook_linear(X, codes, absmax, 50, INT4)
        X[1, 7], X[1, 300] = float("inf"), float("nan")
        got = lib.codebook_linear(X, codes, absmax, 50, INT4)
        rest = [t for t in range(T) if t != 1]
        assert torch.equal(got[rest], ref[rest]) and not bool(torch.isfinite(got[1]).any())


@pytest.mark.parametrize("T", [1, 16])
def test_decode_shape(lib, T):
    lv = [float(v) for v in lib.codebook()[0]]
    w = torch.randn(8192, 8192, device="cuda", generator=torch.Generator("cuda").manual_seed(5)) * 0.02
    q = lib.quantize_single(w)
    del w
    a = check(lib, tokens(T, 8192), q.codes, q.absmax, 8192, lv)
    assert torch.equal(a, lib.codebook_linear(tokens(T, 8192), q.codes, q.absmax, 8192, lv))   # deterministic


@pytest.mark.parametrize("T,N,K", [(3, 37, 192), (1, 37, 192), (2, 300, 1024), (20, 300, 1024)])
def test_guards_capture_and_streams(lib, T, N, K):
    codes, absmax = weight(lib, N, K, INT4)
    X = tokens(T, K)
    ref = lib.codebook_linear(X, codes, absmax, N, INT4)
    buf = torch.full((T * N + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[2048:2048 + T * N].view(T, N)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lib.codebook_linear(X, codes, absmax, N, INT4, out=out)
    for seed in (0, 8):
        X.copy_(tokens(T, K, seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, lib.codebook_linear(X, codes, absmax, N, INT4))
    assert torch.equal(lib.codebook_linear(tokens(T, K), codes, absmax, N, INT4), ref)
    assert bool((buf[:2048] == 7).all()) and bool((buf[2048 + T * N:] == 7).all())
    with torch.cuda.stream(side):
        got = lib.codebook_linear(tokens(T, K), codes, absmax, N, INT4)
    side.synchronize()
    assert torch.equal(got, ref)


def test_refusals(lib):
    codes, absmax = weight(lib, 16, 128, INT4)
    X = tokens(2, 128)
    for bad in (dict(X=X.float()), dict(X=X[:, :64]), dict(X=X[0]), dict(N=17), dict(codes=codes[:-1]), dict(X=X.cpu()),
                dict(absmax=absmax.double()), dict(out=torch.empty(2, 8, device="cuda", dtype=torch.bfloat16))):
        a = dict(X=X, codes=codes, absmax=absmax, N=16, levels=INT4)
        a.update(bad)
        with pytest.raises(ValueError):
            lib.codebook_linear(**a)
    for bad, rc in ((dict(X=tokens(65, 128)), -2), (dict(levels=[0.0]), -10), (dict(levels=[0.5, -0.5]), -10)):
        a = dict(X=X, codes=codes, absmax=absmax, N=16, levels=INT4)
        a.update(bad)
        with pytest.raises(lib.QLoRAError) as e:
            lib.codebook_linear(**a)
        assert e.value.code == rc
    with pytest.raises(ValueError):
        lib.linear_single(tokens(2, 64), lib.quantize_single(torch.randn(16, 128, device="cuda")))
