"""The layer with counter-based LoRA dropout on the GPU: the mask bit for bit,
the layer against the fp64 oracle with that mask.

Tolerances, per value, counted from the roundings that are made:
  h    2^-8 (|h| + sum |us B|): h and us are rounded to bf16 once each
  us   2^-8 |us|
  dx   2^-8 (|dh W| + |dx| + sum |du A| k/(1-q)): the base product, du and dx
       are rounded to bf16
  dA, dB  no rounding below fp32
and for every fp32 sum of n terms (n + 64) 2^-23 times the sum of their
absolute values (an addition is off by at most one step; du's own sum enters
dA), with 2 % on top for products of these terms.
"""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_11_b200 as qmod
from bit_nf4_quantized_11_b200 import synth
from oracle import linear, nf4, philox
from parity import to_np

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


def rng_tensor(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("seed,offset,p,M,n", [
    (0, 0, 0.05, 3, 64),
    (-1, -2**63, 0.5, 2, 192),
    (2**62 + 12345, 2**40 + 7, 0.3, 17, 128),
    (5, 3, 0.0, 4, 64),
    (5, 3, 0.99999999, 4, 64),
    (9, 1, 0.1, 70000, 64),               # more rows than grid rows
    (9, 1, 0.1, 1, 8256),                 # a row of more than 256 words
])
def test_keep_bits(cuda_lib, seed, offset, p, M, n):
    got = cuda_lib.dropout_keep_bits(rng_tensor(seed, offset), p, M, n).cpu().numpy()
    rows = np.arange(M) if M < 100 else np.array([0, 1, 65534, 65535, 69999])
    for m in rows:
        # row m of the oracle's mask alone
        k = np.array([[((philox.philox4x32((g, int(m), offset & philox.MASK, (offset >> 32) & philox.MASK),
                                           (seed & philox.MASK, (seed >> 32) & philox.MASK), 7)[i // 2]
                         >> (16 * (i % 2))) & 0xFFFF) >= philox.threshold(p) for i in range(8)]
                      for g in range(n // 8)])
        assert np.array_equal(got[m], np.packbits(k, axis=1, bitorder="little")[:, 0])


@pytest.mark.parametrize("p", [1 / 65536, 0.25, 0.5, 32769 / 65536, 65534 / 65536, 65535 / 65536])
def test_keep_bits_of_a_whole_mask(cuda_lib, p):
    """262144 values per threshold, each half of a word four times on average:
    the comparison holds on both sides of T, at its ends too."""
    M, n, seed, offset = 64, 4096, 0x0123456789ABCDEF, 42
    u = np.uint64
    m32, sh = u(0xFFFFFFFF), u(32)
    c0, c1 = np.meshgrid(np.arange(n // 8, dtype=u), np.arange(M, dtype=u))
    c2, c3 = np.full_like(c0, u(offset)), np.zeros_like(c0)
    k0, k1 = u(seed) & m32, u(seed) >> sh
    for _ in range(7):
        a, b = c0 * u(philox.M0), c2 * u(philox.M1)
        c0, c1, c2, c3 = (b >> sh) ^ c1 ^ k0, b & m32, (a >> sh) ^ c3 ^ k1, a & m32
        k0, k1 = (k0 + u(philox.W0)) & m32, (k1 + u(philox.W1)) & m32
    words = np.stack([c0, c1, c2, c3], -1)
    halves = np.stack([words & u(0xFFFF), words >> u(16)], -1).reshape(M, n)
    keep = halves >= u(round(p * 65536))
    got = cuda_lib.dropout_keep_bits(rng_tensor(seed, offset), p, M, n).cpu().numpy()
    assert np.array_equal(got, np.packbits(keep, axis=1, bitorder="little"))


def run(q, M, n_in, n_out, r, alpha, p, seed=0, sample=None):
    prob = synth.problem(M, n_in, n_out, r, seed=seed)
    dev = torch.device("cuda")
    rng = rng_tensor(seed * 77 + 3, seed)
    w = q.quantize_nf4(prob["W"].to(dev))
    x, A, B, dh = (prob[k].to(dev) for k in ("x", "A", "B", "dh"))
    h, us = q.linear_fwd_dropout_rng(x, w, A, B, alpha, rng, p)
    dx, dA, dB = q.linear_bwd_dropout_rng(dh, x, us, w, A, B, alpha, rng, p)
    assert q.last_device_status() == 0

    keep = linear.unpack_keep(q.dropout_keep_bits(rng, p, M, n_in).cpu().numpy(), n_in)
    qo = nf4.quantize(prob["W"].numpy())
    W = nf4.dequantize(qo["codes"], qo["q8"], qo["step2"], qo["mean"]).astype(np.float64)
    xn, An, Bn, dhn, usn = (to_np(t) for t in (x, A, B, dh, us))
    drop = philox.threshold(p) / 65536
    s, inv = alpha / r, 1 / (1 - drop)
    rows = np.arange(M) if sample is None else np.asarray(sample)
    xd = xn * keep * inv

    h_ref, u_ref = linear.linear_fwd_dropout(xn[rows], W, An, Bn, alpha, keep[rows], drop)
    us_ref = s * u_ref
    us_size = s * np.abs(xd[rows]) @ np.abs(An).T
    g = lambda n: (n + 64) * 2.0 ** -23                                            # noqa: E731
    us_tol = 1.02 * (2.0 ** -8 * np.abs(us_ref) + g(n_in) * us_size)
    assert np.all(np.abs(usn[rows] - us_ref) <= us_tol)
    low = us_tol @ np.abs(Bn).T
    size = np.abs(xn[rows]) @ np.abs(W).T + np.abs(us_ref) @ np.abs(Bn).T
    tol = 1.02 * (2.0 ** -8 * np.abs(h_ref) + low + g(n_in + r) * size)
    err = np.abs(to_np(h)[rows] - h_ref)
    assert np.all(err <= tol), ("h", (err / tol).max())

    du = s * (dhn @ Bn)
    du_size = s * np.abs(dhn) @ np.abs(Bn)
    base, lowdx = dhn[rows] @ W, np.abs(du[rows]) @ np.abs(An) * keep[rows] * inv
    dx_ref = base + (du[rows] @ An) * keep[rows] * inv
    size = np.abs(dhn[rows]) @ np.abs(W) + (du_size[rows] @ np.abs(An)) * keep[rows] * inv
    tol = 1.02 * (2.0 ** -8 * (np.abs(base) + np.abs(dx_ref) + lowdx) + g(n_out + r) * size)
    err = np.abs(to_np(dx)[rows] - dx_ref)
    assert np.all(err <= tol), ("dx", (err / tol).max())

    dB_ref, dB_size = dhn.T @ usn, np.abs(dhn).T @ np.abs(usn)
    err, tol = np.abs(to_np(dB) - dB_ref), 1.02 * g(M) * dB_size
    assert np.all(err <= tol + 1e-300), ("dB", (err / tol).max())
    dA_ref, dA_size = du.T @ xd, np.abs(du).T @ np.abs(xd)
    tol = 1.02 * (g(M) * dA_size + g(n_out) * (du_size.T @ np.abs(xd)))
    err = np.abs(to_np(dA) - dA_ref)
    assert np.all(err <= tol + 1e-300), ("dA", (err / tol).max())
    # the norm-wise error of the fp32 gradients
    for got, ref in ((to_np(dA), dA_ref), (to_np(dB), dB_ref)):
        n = np.linalg.norm(ref)
        assert n == 0 or np.linalg.norm(got - ref) <= 4e-6 * n


@pytest.mark.parametrize("M,n_in,n_out,r,alpha,p", [
    (1, 64, 64, 1, 1.0, 0.5),            # the smallest layer
    (3, 128, 192, 8, 16.0, 0.0),         # nothing dropped
    (9, 1024, 768, 16, 32.0, 0.05),
    (16, 192, 320, 5, 10.0, 0.3),        # rank not a multiple of 8
    (17, 576, 320, 24, 24.0, 0.1),
    (64, 512, 512, 8, 16.0, 0.05),
    (129, 256, 768, 32, 8.0, 0.05),
    (200, 256, 192, 136, 16.0, 0.2),     # two column groups of the gradient
    (256, 640, 256, 64, 64.0, 0.25),
    (257, 320, 576, 80, 16.0, 0.5),
    (300, 640, 320, 12, 24.0, 0.1),
    (1500, 512, 448, 16, 32.0, 0.05),    # stages take turns over the accumulators
    (70, 256, 192, 256, 16.0, 0.1),      # the largest rank: four column groups
    (5000, 128, 192, 88, 16.0, 0.1),
])
def test_layer(cuda_lib, M, n_in, n_out, r, alpha, p):
    run(cuda_lib, M, n_in, n_out, r, alpha, p, seed=M)


def test_full_size_7b_attention(cuda_lib):
    rng = np.random.default_rng(0)
    run(cuda_lib, 4096, 4096, 4096, 16, 32.0, 0.05, seed=1, sample=np.sort(rng.choice(4096, 32, replace=False)))


@pytest.mark.parametrize("M", [7, 200, 600])
def test_equals_the_layer_with_that_mask(cuda_lib, M):
    """The stored-mask calls with the mask as bits and the rounded p: the same
    us up to the order of its sum, and gradients up to their bf16 du."""
    q = cuda_lib
    prob = synth.problem(M, 512, 384, 16, seed=M)
    w = q.quantize_nf4(prob["W"].cuda())
    x, A, B, dh = (prob[k].cuda() for k in ("x", "A", "B", "dh"))
    rng, p = rng_tensor(11, M), 0.1
    bits = q.dropout_keep_bits(rng, p, M, 512)
    drop = philox.threshold(p) / 65536
    h0, us0 = q.linear_fwd_dropout(x, w, A, B, 32.0, bits, drop)
    h1, us1 = q.linear_fwd_dropout_rng(x, w, A, B, 32.0, rng, p)
    assert (us0.float() - us1.float()).abs().max() <= 2.0 ** -7 * us0.float().abs().max()
    g0 = q.linear_bwd_dropout(dh, x, us0, w, A, B, 32.0, bits, drop)
    g1 = q.linear_bwd_dropout_rng(dh, x, us0, w, A, B, 32.0, rng, p)
    for a, b in zip((h0,) + g0, (h1,) + g1):
        assert (a.float() - b.float()).norm() <= 2.0 ** -7 * a.float().norm()


def test_gradient_against_differences(cuda_lib):
    """The layer is linear in A and in B: L(A) - L(0) = <dA, A> for
    L = sum dh h, and with us from the forward L(B) - L(0) = <dB, B>.  dh = h
    keeps L free of cancellation, so that the bf16 roundings of h (2^-8 each
    side) bound the difference by 2^-7 of L's terms."""
    q = cuda_lib
    prob = synth.problem(400, 256, 320, 16, seed=5)
    w = q.quantize_nf4(prob["W"].cuda())
    x, A, B = (prob[k].cuda() for k in ("x", "A", "B"))
    rng, p, alpha = rng_tensor(1, 2), 0.2, 16 * 64.0            # the adapter outweighs the base
    h, us = q.linear_fwd_dropout_rng(x, w, A, B, alpha, rng, p)
    zero, _ = q.linear_fwd_dropout_rng(x, w, torch.zeros_like(A), B, alpha, rng, p)
    dx, dA, dB = q.linear_bwd_dropout_rng(h, x, us, w, A, B, alpha, rng, p)
    diff = (h.double() * (h.double() - zero.double())).sum()
    size = (h.double().abs() * (h.double().abs() + zero.double().abs())).sum()
    assert (diff - (dA.double() * A.double()).sum()).abs() <= 2.0 ** -7 * size
    assert (diff - (dB.double() * B.double()).sum()).abs() <= 2.0 ** -7 * size
    assert diff > 0.3 * size                                    # the bounds above say something
    # x enters both products: L(x) - L(0) = <dx, x>
    assert ((h.double() ** 2).sum() - (dx.double() * x.double()).sum()).abs() <= 2.0 ** -6 * size


@pytest.mark.parametrize("M", [5, 100, 700])
def test_graph_draws_a_new_mask_when_the_state_changes(cuda_lib, M):
    q = cuda_lib
    prob = synth.problem(M, 512, 384, 16, seed=M)
    w = q.quantize_nf4(prob["W"].cuda())
    x, A, B, dh = (prob[k].cuda() for k in ("x", "A", "B", "dh"))
    rng = rng_tensor(3, 4)

    def step():
        h, us = q.linear_fwd_dropout_rng(x, w, A, B, 32.0, rng, 0.2)
        return (h, us) + q.linear_bwd_dropout_rng(dh, x, us, w, A, B, 32.0, rng, 0.2)
    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    rng[1] += 1
    graph.replay()
    torch.cuda.synchronize()
    again = step()
    assert all(torch.equal(a, b) for a, b in zip(again, out))
    assert not torch.equal(first[1], out[1])
    assert q.last_device_status() == 0


def test_train_two_adapters_then_serve_them(cuda_lib):
    """As they are used together: steps with dropout on two adapters of one
    base, then one batch of requests over both, each token as its adapter's
    layer alone gives it (bf16 h: one step apart at most)."""
    q = cuda_lib
    prob = synth.problem(320, 256, 384, 16, seed=8)
    w = q.quantize_nf4(prob["W"].cuda())
    x, A0, B0, dh = (prob[k].cuda() for k in ("x", "A", "B", "dh"))
    tables_a, tables_b = [], []
    for seed in (1, 2):
        A, B = A0.float().clone(), B0.float().clone()
        for step in range(3):
            a16, b16 = A.bfloat16(), B.bfloat16()
            rng = rng_tensor(seed, step)
            h, us = q.linear_fwd_dropout_rng(x, w, a16, b16, 32.0, rng, 0.05)
            _, dA, dB = q.linear_bwd_dropout_rng(dh, x, us, w, a16, b16, 32.0, rng, 0.05)
            A -= 1e-4 * dA
            B -= 1e-4 * dB
        tables_a.append(A.bfloat16())
        tables_b.append(B.bfloat16())
    ids = q.token_slots(torch.tensor([100, 0, 120], dtype=torch.int32, device="cuda"),
                        torch.tensor([1, 0, 0], dtype=torch.int32, device="cuda"), 230)
    scale = torch.full((2,), 2.0, device="cuda")
    y = q.linear_fwd_slots(x[:230].contiguous(), w, torch.stack(tables_a), torch.stack(tables_b), scale, ids)
    for a, rows in ((1, slice(0, 100)), (0, slice(100, 220))):
        ref, _ = q.linear_fwd(x[rows].contiguous(), w, tables_a[a], tables_b[a], 32.0)
        tol = 2.0 ** -7 * ref.float().abs() + 2.0 ** -8 * ref.float().abs().max() * 2.0 ** -4
        assert bool(((y[rows].float() - ref.float()).abs() <= tol).all())
    base, _ = q.linear_fwd(x[220:230].contiguous(), w, torch.zeros_like(A0), B0, 32.0)
    assert (y[220:230].float() - base.float()).norm() <= 2.0 ** -7 * base.float().norm()


def test_python_refusals(cuda_lib):
    q = cuda_lib
    prob = synth.problem(8, 128, 64, 8, seed=1)
    w = q.quantize_nf4(prob["W"].cuda())
    x, A, B, dh = (prob[k].cuda() for k in ("x", "A", "B", "dh"))
    rng = rng_tensor(1, 2)
    for bad in (rng.cpu(), rng.int(), rng[:1], 7):
        with pytest.raises((TypeError, ValueError)):
            q.linear_fwd_dropout_rng(x, w, A, B, 8.0, bad, 0.1)
        with pytest.raises((TypeError, ValueError)):
            q.dropout_keep_bits(bad, 0.1, 8, 128)
    for p in (-0.1, 1.0, float("nan")):
        with pytest.raises(q.QLoRAError):
            q.linear_fwd_dropout_rng(x, w, A, B, 8.0, rng, p)
        with pytest.raises(q.QLoRAError):
            q.dropout_keep_bits(rng, p, 8, 128)
    with pytest.raises(q.QLoRAError):
        q.dropout_keep_bits(rng, 0.1, 8, 72)
    h, us = q.linear_fwd_dropout_rng(x, w, A, B, 8.0, rng, 0.1)
    with pytest.raises(ValueError):
        q.linear_bwd_dropout_rng(dh, x, us[:4], w, A, B, 8.0, rng, 0.1)
    assert qmod.dropout_keep_bits(rng, 0.1, 0, 64).numel() == 0


def test_two_streams_at_once(cuda_lib):
    """Forward and backward calls of different shapes on two streams at a time."""
    q = cuda_lib
    cases = []
    for M, r in ((40, 16), (300, 88), (1100, 64), (200, 8)):
        prob = synth.problem(M, 512, 384, r, seed=M)
        w = q.quantize_nf4(prob["W"].cuda())
        x, A, B, dh = (prob[k].cuda() for k in ("x", "A", "B", "dh"))
        rng = rng_tensor(M, 1)

        def step(x=x, w=w, A=A, B=B, dh=dh, rng=rng):
            h, us = q.linear_fwd_dropout_rng(x, w, A, B, 32.0, rng, 0.1)
            return (h, us) + q.linear_bwd_dropout_rng(dh, x, us, w, A, B, 32.0, rng, 0.1)
        cases.append((step, step()))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for k in range(8):
        for st, j in ((s1, k % 4), (s2, (k + 2) % 4)):
            with torch.cuda.stream(st):
                got.append((cases[j][0](), cases[j][1]))
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert q.last_device_status() == 0


def test_infinities_in_dropped_places_change_nothing(cuda_lib):
    """The adapter branch never sees a dropped value, whatever it is: us, dA
    and dB stay as they are (the base product of h and dx does see x, dh)."""
    q = cuda_lib
    for M in (12, 300):
        prob = synth.problem(M, 256, 192, 16, seed=M)
        w = q.quantize_nf4(prob["W"].cuda())
        x, A, B, dh = (prob[k].cuda() for k in ("x", "A", "B", "dh"))
        rng = rng_tensor(5, M)
        bits = q.dropout_keep_bits(rng, 0.3, M, 256).cpu().numpy()
        drop = torch.from_numpy(linear.unpack_keep(bits, 256) == 0).cuda()
        _, us = q.linear_fwd_dropout_rng(x, w, A, B, 32.0, rng, 0.3)
        _, dA, dB = q.linear_bwd_dropout_rng(dh, x, us, w, A, B, 32.0, rng, 0.3)
        bad = torch.where(drop, torch.full_like(x, float("inf")), x)
        bad[0, drop[0].nonzero()[0]] = float("nan")
        _, us1 = q.linear_fwd_dropout_rng(bad, w, A, B, 32.0, rng, 0.3)
        _, dA1, dB1 = q.linear_bwd_dropout_rng(dh, bad, us1, w, A, B, 32.0, rng, 0.3)
        assert torch.equal(us, us1) and torch.equal(dA, dA1) and torch.equal(dB, dB1)


@pytest.mark.parametrize("M", [12, 300])
@pytest.mark.parametrize("r", [16, 136])
def test_a_dropped_column_of_dx_is_the_base_product(cuda_lib, M, r):
    """Where the mask drops an input, dx is dh W0 whatever the adapter's
    product is there, an infinity or NaN too; a kept one does see it."""
    q = cuda_lib
    prob = synth.problem(M, 256, 192, r, seed=M + r)
    w = q.quantize_nf4(prob["W"].cuda())
    x, A, B, dh = (prob[k].cuda() for k in ("x", "A", "B", "dh"))
    rng, p = rng_tensor(9, M), 0.3
    bits = q.dropout_keep_bits(rng, p, M, 256).cpu().numpy()
    keep = torch.from_numpy(linear.unpack_keep(bits, 256) == 1).cuda()
    us = torch.zeros(M, r, dtype=torch.bfloat16, device="cuda")
    base, _, _ = q.linear_bwd_dropout_rng(dh, x, us, w, torch.zeros_like(A), B, 32.0, rng, p)
    fine, _, _ = q.linear_bwd_dropout_rng(dh, x, us, w, A, B, 32.0, rng, p)
    assert torch.equal(fine[~keep], base[~keep])
    bad = A.clone()
    bad[3, 40:60] = float("inf")
    dx, _, _ = q.linear_bwd_dropout_rng(dh, x, us, w, bad, B, 32.0, rng, p)
    assert torch.equal(dx[~keep], base[~keep])
    hit = torch.zeros_like(keep)
    hit[:, 40:60] = True
    assert not bool(dx[keep & hit].isfinite().any()) and torch.equal(dx[keep & ~hit], fine[keep & ~hit])
    bad = B.clone()
    bad[5, 2] = float("nan")
    dx, _, _ = q.linear_bwd_dropout_rng(dh, x, us, w, A, bad, 32.0, rng, p)
    assert torch.equal(dx[~keep], base[~keep]) and bool(dx[keep].isnan().all())


@pytest.mark.parametrize("M,r", [(8193, 64), (20000, 136), (33000, 80), (33000, 256), (40000, 16), (70000, 12),
                                 (100001, 64), (262144, 64)])
def test_gradients_of_long_batches(cuda_lib, M, r):
    """The error of dA and dB does not grow with the tokens.  Positive data,
    where cut bits add up: dh and B are whole numbers up to 15, so that du is
    exact, and q = 1/2, s = 1 are powers of two.  What is left, in units of
    2^-23 of the sum: an accumulator takes at most 64 steps, each cutting less
    than one of its sum so far, which is half the whole on average; the rounded
    additions, half each, are those of at most 8 accumulators, 8 x 3 partial
    tiles and at most one round per 8192 tokens."""
    q = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(M + r)
    n = 64
    w = q.quantize_nf4(synth.problem(1, n, n, 8)["W"].cuda())
    dh = torch.randint(1, 16, (M, n), generator=g, device="cuda").bfloat16()
    B = torch.randint(1, 16, (n, r), generator=g, device="cuda").bfloat16()
    x = (torch.rand(M, n, generator=g, device="cuda") + 1).bfloat16()
    us = (torch.rand(M, r, generator=g, device="cuda") + 1).bfloat16()
    A = torch.zeros(r, n, dtype=torch.bfloat16, device="cuda")
    rng = rng_tensor(3, M)
    _, dA, dB = q.linear_bwd_dropout_rng(dh, x, us, w, A, B, float(r), rng, 0.5)
    bits = q.dropout_keep_bits(rng, 0.5, M, n)
    keep = (bits[:, :, None] >> torch.arange(8, device="cuda")) & 1
    xd = x.double() * keep.reshape(M, n) * 2
    tol = 2.0 ** -23 * (32 + (8 + 24 + -(-M // 8192)) / 2)
    dB_ref = dh.double().T @ us.double()
    dA_ref = (dh.double() @ B.double()).T @ xd
    for name, got, ref in (("dB", dB, dB_ref), ("dA", dA, dA_ref)):
        err = ((got.double() - ref).abs() / ref).max().item()
        print(name, M, r, err, tol)
        assert err <= tol, (name, err, tol)
    assert q.last_device_status() == 0


def test_du_of_many_features_and_tokens(cuda_lib):
    """The error of du does not grow with the tokens either: 28672 features of
    positive data, so many tokens that their tiles alone fill the chip.  Each
    column of x holds a single one, so dA shows du itself, column by column.
    In units of 2^-23: an accumulator takes at most 14 stages of 4 steps, each
    cutting less than one; the roundings of the sum over at most 8 accumulators
    and 8 CTAs, of the scale and of the three parts, half each."""
    q = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(1)
    M, n_in, n_out, r = 19200, 64, 28672, 64
    w = q.quantize_nf4(synth.problem(1, n_in, n_out, 8)["W"].cuda())
    dh = torch.rand(M, n_out, generator=g, device="cuda").add_(1).bfloat16()
    B = torch.rand(n_out, r, generator=g, device="cuda").add_(1).bfloat16()
    rows = torch.arange(n_in, device="cuda") * (M // n_in) + 7
    x = torch.zeros(M, n_in, dtype=torch.bfloat16, device="cuda")
    x[rows, torch.arange(n_in, device="cuda")] = 1
    us = torch.zeros(M, r, dtype=torch.bfloat16, device="cuda")
    A = torch.zeros(r, n_in, dtype=torch.bfloat16, device="cuda")
    _, dA, _ = q.linear_bwd_dropout_rng(dh, x, us, w, A, B, float(r), rng_tensor(1, 1), 0.0)
    ref = (dh[rows].double() @ B.double()).T
    err = ((dA.double() - ref).abs() / ref).max().item()
    tol = 2.0 ** -23 * (14 * 4 + (8 + 8 + 4) / 2)
    print("du", err, tol)
    assert err <= tol
    assert q.last_device_status() == 0


@pytest.mark.parametrize("M,n_in,n_out,r", [(20, 256, 40000, 16), (9, 1088, 8256, 16), (100, 1088, 8256, 12),
                                            (200, 256, 20032, 8)])
def test_layer_with_ctas_over_several_row_tiles(cuda_lib, M, n_in, n_out, r):
    """Few tokens and more row tiles than the SMs' even shares (148 SMs)."""
    run(cuda_lib, M, n_in, n_out, r, 32.0, 0.1, seed=M)


def test_keep_bits_of_more_than_2_32_words(cuda_lib):
    """A mask of 17 GB: the last rows lie past 2^32 words."""
    M, n, seed, offset, p = 2 ** 21 + 3, 65600, 12, 34, 0.25
    got = cuda_lib.dropout_keep_bits(rng_tensor(seed, offset), p, M, n)
    assert got.numel() // 4 > 2 ** 32
    for m in (0, 2 ** 20 + 1, M - 1):
        groups = list(range(0, n // 8, 97)) + [n // 8 - 1]
        row = got[m].cpu().numpy()
        for g in groups:
            w = philox.philox4x32((g, m, offset, 0), (seed, 0), 7)
            bits = sum((((w[i // 2] >> (16 * (i % 2))) & 0xFFFF) >= philox.threshold(p)) << i for i in range(8))
            assert row[g] == bits, (m, g)


def test_outputs_of_more_than_2_31_values(cuda_lib):
    """h and dx past 2^31 values without a mask (p = 0): the last 512 tokens
    against calls on them alone, bit for bit."""
    q = cuda_lib
    M, r = 512 * 157, 8
    g = torch.Generator(device="cuda").manual_seed(4)
    for n_in, n_out in ((64, 28672), (28672, 64)):
        prob = synth.problem(1, n_in, n_out, r, seed=4)
        w, A, B = q.quantize_nf4(prob["W"].cuda()), prob["A"].cuda(), prob["B"].cuda()
        rng = rng_tensor(1, 1)
        x = torch.randn(M, n_in, generator=g, device="cuda").bfloat16()
        h, us = q.linear_fwd_dropout_rng(x, w, A, B, 16.0, rng, 0.0)
        t = x[-512:].contiguous()
        h1, us1 = q.linear_fwd_dropout_rng(t, w, A, B, 16.0, rng, 0.0)
        us_same = torch.equal(us[-512:], us1)       # (K may be split differently)
        assert us_same or (us[-512:].float() - us1.float()).norm() <= 2.0 ** -8 * us1.float().norm()
        assert not us_same or torch.equal(h[-512:], h1)
        dh = torch.randn(M, n_out, generator=g, device="cuda").bfloat16()
        dx, _, _ = q.linear_bwd_dropout_rng(dh, x, us, w, torch.zeros_like(A), B, 16.0, rng, 0.0)
        dx1, _, _ = q.linear_bwd_dropout_rng(dh[-512:].contiguous(), t, us1, w, torch.zeros_like(A), B, 16.0, rng, 0.0)
        assert torch.equal(dx[-512:], dx1)
        assert max(h.numel(), dx.numel()) > 2 ** 31
        del x, h, dh, dx
    assert q.last_device_status() == 0
