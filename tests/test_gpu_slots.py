"""One adapter per request on the GPU against the fp64 oracle.

Tolerance, per output, counted from the roundings that the layer makes:
  2^-8 |h|            h is rounded to bf16 once (half a step)
  2^-8 sum |us B|     us is rounded to bf16 before the second product
  g (sum |x W| + sum |us B|), g = (in + 2 r + 64) 2^-23
                      fp32 sums of in + r terms; each addition is off by at
                      most one step (the tensor cores cut instead of rounding)
with 2 % on top for the products of these terms.
"""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_11_b200 as qmod
from bit_nf4_quantized_11_b200 import synth
from oracle import nf4, slots
from parity import to_np

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


@pytest.mark.parametrize("lengths,n_tokens", [
    ([1], 1),
    ([0, 0, 5, 0, 3, 0], 8),
    ([3, -4, 2], 9),                    # a negative length counts as zero; unused tokens
    ([5, 7], 6),                        # cut off
    ([0, 0], 3),
    ([1] * 1500, 1500),                 # more requests than one scan tile
    ([0] * 1030 + [2000, 0, 1] + [3] * 2000, 9000),
    ([2**31 - 1, 2**31 - 1, 4], 2000),  # the sum passes 32 bits
])
def test_token_slots(cuda_lib, lengths, n_tokens):
    rng = np.random.default_rng(len(lengths))
    s = rng.integers(-1, 60, len(lengths)).astype(np.int32)
    got = cuda_lib.token_slots(torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                               torch.from_numpy(s).cuda(), n_tokens)
    assert np.array_equal(got.cpu().numpy(), slots.token_slots(lengths, s, n_tokens))


def test_token_slots_no_requests_and_no_tokens(cuda_lib):
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert cuda_lib.token_slots(none, none, 70).tolist() == [-1] * 70
    assert cuda_lib.token_slots(none, none, 0).numel() == 0


def make(M, n_in, n_out, r, n, seed=0):
    g = torch.Generator().manual_seed(seed)
    p = synth.problem(M, n_in, n_out, 8, seed=seed)
    A = ((torch.rand(n, r, n_in, generator=g) * 2 - 1) / n_in ** 0.5).bfloat16()
    B = (torch.randn(n, n_out, r, generator=g) * 0.01).bfloat16()
    scale = torch.rand(n, generator=g) * 3 + 0.25
    return p["W"], p["x"], A, B, scale


def check(q, M, n_in, n_out, r, n, ids, seed=0, sample=None, **kw):
    W, x, A, B, scale = make(M, n_in, n_out, r, n, seed)
    w = q.quantize_nf4(W.cuda())
    ids_t = torch.from_numpy(np.asarray(ids, dtype=np.int32)).cuda()
    h = q.linear_fwd_slots(x.cuda(), w, A.cuda(), B.cuda(), scale.cuda(), ids_t, **kw)
    assert q.last_device_status() == 0
    qo = nf4.quantize(W.numpy())
    Wd = nf4.dequantize(qo["codes"], qo["q8"], qo["step2"], qo["mean"]).astype(np.float64)
    rows = np.arange(M) if sample is None else np.asarray(sample)
    xn = to_np(x)[rows]
    ref, low = slots.linear_fwd_slots(xn, Wd, to_np(A), to_np(B), scale.numpy(), np.asarray(ids)[rows])
    size = np.abs(xn) @ np.abs(Wd).T + low
    tol = 1.02 * (2.0 ** -8 * (np.abs(ref) + low) + (n_in + 2 * r + 64) * 2.0 ** -23 * size)
    err = np.abs(to_np(h)[rows] - ref)
    assert np.all(np.isfinite(to_np(h)))
    assert np.all(err <= tol), (err / tol).max()
    return h


def mixed(M, n, seed=0):
    """Slots in any order, some of them naming no adapter."""
    return np.random.default_rng(seed).integers(-1, n + 1, M)


@pytest.mark.parametrize("M,n_in,n_out,r,n", [
    (1, 512, 512, 16, 4),
    (1, 64, 64, 1, 1),                  # the smallest layer: one block, rank one
    (2, 192, 320, 8, 3),                # half a row tile at the end, three blocks
    (7, 1088, 192, 12, 5),              # rank not a multiple of 8; K ends inside a unit
    (16, 2048, 512, 16, 16),
    (17, 512, 768, 16, 20),
    (33, 1024, 256, 64, 40),
    (64, 512, 512, 24, 64),             # adapters across the 64-wide stages
    (100, 640, 320, 3, 7),
    (128, 4096, 256, 16, 200),
    (200, 576, 448, 40, 9),
    (256, 512, 384, 16, 300),           # a tile full of different adapters
    (257, 512, 512, 16, 4),
    (300, 640, 320, 20, 6),
    (500, 512, 768, 8, 40),
    (1100, 768, 512, 64, 5),
    (129, 256, 256, 136, 3),
    (20, 256, 192, 256, 2),             # the largest rank
])
def test_layer_mixed_slots(cuda_lib, M, n_in, n_out, r, n):
    check(cuda_lib, M, n_in, n_out, r, n, mixed(M, n, seed=M), seed=M)


@pytest.mark.parametrize("M", [3, 40, 150, 700])
def test_no_adapter_at_all(cuda_lib, M):
    check(cuda_lib, M, 512, 320, 16, 3, np.full(M, -1), seed=M)
    check(cuda_lib, M, 512, 320, 16, 3, np.full(M, 2**31 - 1), seed=M)


@pytest.mark.parametrize("M", [5, 90, 256, 800])
def test_one_adapter_equals_every_token(cuda_lib, M):
    check(cuda_lib, M, 512, 448, 16, 6, np.full(M, 4), seed=M)


@pytest.mark.parametrize("r,n", [(12, 9), (16, 40), (64, 40)])
def test_groups_of_one_to_nine_tokens(cuda_lib, r, n):
    """Adapter k has k + 1 tokens, in any order: full and partial groups of tokens that share an adapter's reading."""
    ids = np.random.default_rng(r).permutation(np.repeat(np.arange(9), np.arange(1, 10)))
    check(cuda_lib, len(ids), 576, 192, r, n, ids, seed=r + n)


@pytest.mark.parametrize("M,n_in,n_out,r,n", [(12, 512, 320, 16, 5), (90, 512, 320, 16, 5), (600, 512, 320, 16, 5)])
def test_unused_adapters_may_hold_anything(cuda_lib, M, n_in, n_out, r, n):
    """Infinities and NaN in slots that no token uses, and next to the used
    ones in memory, change nothing."""
    q = cuda_lib
    W, x, A, B, scale = make(M, n_in, n_out, r, n, seed=M)
    ids = torch.from_numpy(np.random.default_rng(M).choice([1, 3], M).astype(np.int32)).cuda()
    w = q.quantize_nf4(W.cuda())
    h0 = q.linear_fwd_slots(x.cuda(), w, A.cuda(), B.cuda(), scale.cuda(), ids)
    for a, v in ((0, float("nan")), (2, float("inf")), (4, float("nan"))):
        A[a], B[a], scale[a] = v, -v, v
    h1 = q.linear_fwd_slots(x.cuda(), w, A.cuda(), B.cuda(), scale.cuda(), ids)
    assert torch.equal(h0, h1)


@pytest.mark.parametrize("M", [6, 70, 700])
def test_a_token_with_nan_stays_alone(cuda_lib, M):
    """A NaN in one token's activations reaches that token's outputs only."""
    q = cuda_lib
    W, x, A, B, scale = make(M, 512, 320, 16, 4, seed=M)
    ids = torch.from_numpy(mixed(M, 4, M).astype(np.int32)).cuda()
    w = q.quantize_nf4(W.cuda())
    args = (w, A.cuda(), B.cuda(), scale.cuda(), ids)
    h0 = q.linear_fwd_slots(x.cuda(), *args)
    x[M // 2, 17] = float("nan")
    h1 = q.linear_fwd_slots(x.cuda(), *args)
    keep = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(h0[keep], h1[keep]) and bool(h1[M // 2].isnan().all())


@pytest.mark.parametrize("M", [1, 50, 300, 900])
def test_same_result_twice_streams_and_graph(cuda_lib, M):
    """Bit-identical when repeated, on a second stream, and replayed from a
    captured graph with new inputs and slots in the same buffers."""
    q = cuda_lib
    W, x, A, B, scale = make(M, 1024, 512, 16, 6, seed=M)
    w = q.quantize_nf4(W.cuda())
    x, A, B, scale = x.cuda(), A.cuda(), B.cuda(), scale.cuda()
    lens = torch.tensor([max(0, M // 3), 0, M - M // 3 - M // 5], dtype=torch.int32, device="cuda")
    sl = torch.tensor([5, 1, 2], dtype=torch.int32, device="cuda")

    def step():
        return q.linear_fwd_slots(x, w, A, B, scale, q.token_slots(lens, sl, M))
    h0 = step()
    assert torch.equal(h0, step())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        h1 = step()
    torch.cuda.synchronize()
    assert torch.equal(h0, h1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hg = step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h0, hg)
    x.mul_(0.5)
    sl.copy_(torch.tensor([0, 3, -1], dtype=torch.int32, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(hg, step())
    assert q.last_device_status() == 0


def test_output_rows_past_the_batch_are_left_alone(cuda_lib):
    q = cuda_lib
    W, x, A, B, scale = make(37, 512, 320, 16, 4, seed=1)
    w = q.quantize_nf4(W.cuda())
    buf = torch.full((60, 320), 7.0, dtype=torch.bfloat16, device="cuda")
    q.linear_fwd_slots(x.cuda(), w, A.cuda(), B.cuda(), scale.cuda(),
                       torch.zeros(37, dtype=torch.int32, device="cuda"), h=buf[:37])
    assert bool((buf[37:] == 7.0).all()) and not bool((buf[:37] == 7.0).all())


def test_python_refusals(cuda_lib):
    q = cuda_lib
    W, x, A, B, scale = (t.cuda() for t in make(4, 128, 64, 8, 2))
    w = q.quantize_nf4(W)
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        q.linear_fwd_slots(x.float(), w, A, B, scale, ids)
    with pytest.raises(TypeError):
        q.linear_fwd_slots(x, w, A, B, scale, ids.long())
    with pytest.raises(TypeError):
        q.linear_fwd_slots(x, w, A, B, scale.bfloat16(), ids)
    with pytest.raises(TypeError):
        q.linear_fwd_slots(x, w, A, B, scale, ids.cpu())
    with pytest.raises(ValueError):
        q.linear_fwd_slots(x, w, A, B, scale, ids[:3])
    with pytest.raises(ValueError):
        q.linear_fwd_slots(x, w, A, B.transpose(1, 2).contiguous(), scale, ids)
    with pytest.raises(ValueError):
        q.linear_fwd_slots(x.t().contiguous().t(), w, A, B, scale, ids)
    with pytest.raises(ValueError):
        q.token_slots(ids, ids[:2], 4)
    with pytest.raises(q.QLoRAError):
        q.linear_fwd_slots(x[:0], w, A, B, scale, ids[:0])


@pytest.mark.parametrize("M", [9, 140, 700])
def test_a_broken_adapter_reaches_its_own_tokens_only(cuda_lib, M):
    """An infinity or NaN in one used adapter changes its own tokens, in the
    features that it touches, and nobody else's."""
    q = cuda_lib
    W, x, A, B, scale = make(M, 512, 320, 16, 4, seed=M)
    ids_n = mixed(M, 4, M)
    ids_n[:2] = [2, 1]
    ids = torch.from_numpy(ids_n.astype(np.int32)).cuda()
    w = q.quantize_nf4(W.cuda())
    h0 = q.linear_fwd_slots(x.cuda(), w, A.cuda(), B.cuda(), scale.cuda(), ids)
    B[2, 130, 5] = float("inf")
    B[2, 7, 0] = float("nan")
    h1 = q.linear_fwd_slots(x.cuda(), w, A.cuda(), B.cuda(), scale.cuda(), ids)
    mine = torch.from_numpy(ids_n == 2).cuda()
    assert torch.equal(h0[~mine], h1[~mine])
    touched = torch.zeros(320, dtype=torch.bool, device="cuda")
    touched[[7, 130]] = True
    assert torch.equal(h0[mine][:, ~touched], h1[mine][:, ~touched])
    assert bool(h1[mine][:, 7].isnan().all()) and not bool(h1[mine][:, 130].isfinite().any())


def test_two_calls_at_once_and_graphs_that_share_a_workspace(cuda_lib):
    """Calls on two streams at a time, and two captured graphs over one
    workspace replayed in turn, give what single calls give."""
    q = cuda_lib
    cases = []
    for M, r, n in ((24, 16, 20), (200, 24, 3), (230, 16, 100), (600, 64, 6)):
        W, x, A, B, scale = (t.cuda() for t in make(M, 768, 640, r, n, seed=M))
        ids = torch.from_numpy(mixed(M, n, M).astype(np.int32)).cuda()
        args = (x, q.quantize_nf4(W), A, B, scale, ids)
        cases.append((args, q.linear_fwd_slots(*args)))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for k in range(12):
        for st, (args, _) in ((s1, cases[k % 4]), (s2, cases[(k + 1) % 4])):
            with torch.cuda.stream(st):
                got.append(q.linear_fwd_slots(*args))
    torch.cuda.synchronize()
    want = [c for k in range(12) for c in (cases[k % 4][1], cases[(k + 1) % 4][1])]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    graphs = []
    for args, h in cases[:3]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = q.linear_fwd_slots(*args, workspace=ws)
        graphs.append((g, out, h))
    for _ in range(3):
        for g, out, h in graphs:
            out.zero_()
            ws.fill_(0xFF)                  # what the workspace holds before does not matter
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, h)
    assert q.last_device_status() == 0


@pytest.mark.parametrize("M,n_in,n_out", [(8, 8192, 128), (64, 4160, 192), (100, 8192, 192), (200, 4160, 128)])
def test_long_rows_refill_the_operand_ring(cuda_lib, M, n_in, n_out):
    """Rows of 65 to 128 blocks go through the eight-block tensor-memory ring
    many times; the products that read a slot are over before it is written
    anew, so every run has the same bits."""
    q = cuda_lib
    ids = mixed(M, 3, M)
    h0 = check(q, M, n_in, n_out, 16, 3, ids, seed=M)
    W, x, A, B, scale = (t.cuda() for t in make(M, n_in, n_out, 16, 3, M))
    w = q.quantize_nf4(W)
    ids_t = torch.from_numpy(ids.astype(np.int32)).cuda()
    for _ in range(20):
        assert torch.equal(h0, q.linear_fwd_slots(x, w, A, B, scale, ids_t))


# Shapes whose row tiles are more than the SMs' even shares, on 148 SMs: CTAs
# begin and end inside tiles, hold the end of one and the start of another
# (1088 columns: tiles of six units over two to four CTAs) or whole tiles
# between two cut ones (256 columns: tiles of one or two units).
@pytest.mark.parametrize("M,n_in,n_out,r,n", [
    (1, 4096, 4096, 16, 3),
    (64, 1088, 8256, 16, 13),
    (100, 1088, 8256, 12, 4),
    (200, 1088, 8256, 24, 5),
    (20, 256, 40000, 16, 3),
    (100, 256, 40000, 8, 5),
    (200, 256, 40000, 16, 3),
])
def test_ctas_over_several_row_tiles(cuda_lib, M, n_in, n_out, r, n):
    check(cuda_lib, M, n_in, n_out, r, n, mixed(M, n, seed=M) if M > 1 else [1], seed=M)


@pytest.mark.parametrize("M", [9, 90, 180])
def test_base_alone_over_several_row_tiles(cuda_lib, M):
    check(cuda_lib, M, 256, 40000, 16, 3, np.full(M, -1), seed=M)


@pytest.mark.parametrize("M,n_in,n_out", [(12, 256, 40000), (100, 256, 40000), (200, 256, 40000),
                                          (12, 1088, 8256), (100, 1088, 8256), (200, 1088, 8256)])
def test_a_broken_adapter_in_whole_and_cut_row_tiles(cuda_lib, M, n_in, n_out):
    """Infinite and NaN B values in one adapter, in two of any three row tiles:
    they reach that adapter's tokens in their own features, and nothing else."""
    q = cuda_lib
    W, x, A, B, scale = make(M, n_in, n_out, 16, 4, seed=M)
    ids_n = mixed(M, 4, M)
    ids_n[:2] = [2, 1]
    ids = torch.from_numpy(ids_n.astype(np.int32)).cuda()
    w, x, A, scale = q.quantize_nf4(W.cuda()), x.cuda(), A.cuda(), scale.cuda()
    h0 = q.linear_fwd_slots(x, w, A, B.cuda(), scale, ids)
    first = torch.arange(0, n_out, 128)
    inf_rows = torch.cat([(first + 5)[0::3], (first + 63)[1::3]])
    nan_rows = (first + 31)[1::3]
    B[2, inf_rows, 3] = float("inf")
    B[2, nan_rows, 15] = float("nan")
    h1 = q.linear_fwd_slots(x, w, A, B.cuda(), scale, ids)
    mine = torch.from_numpy(ids_n == 2).cuda()
    touched = torch.zeros(n_out, dtype=torch.bool, device="cuda")
    touched[inf_rows.cuda()] = touched[nan_rows.cuda()] = True
    assert torch.equal(h0[~mine], h1[~mine])
    assert torch.equal(h0[mine][:, ~touched], h1[mine][:, ~touched])
    assert not bool(h1[mine][:, touched].isfinite().any())
    assert bool(h1[mine][:, nan_rows.cuda()].isnan().all())
    assert torch.equal(h1.isnan(), q.linear_fwd_slots(x, w, A, B.cuda(), scale, ids).isnan())
    assert q.last_device_status() == 0


@pytest.mark.parametrize("M", [20, 200, 300])
def test_tables_of_more_than_2_31_values(cuda_lib, M):
    """The last slot of an A table, then of a B table, past 2^31 values: the
    same bits as with that adapter in a table of 40 (more than 32, so that both
    calls form us the same way)."""
    q = cuda_lib
    r, n = 32, 2400
    for n_in, n_out in ((28672, 64), (64, 28672)):
        W, x, A, B, scale = (t.cuda() for t in make(M, n_in, n_out, r, 1, seed=M))
        w = q.quantize_nf4(W)
        ids = torch.zeros(M, dtype=torch.int32, device="cuda")
        want = q.linear_fwd_slots(x, w, A.repeat(40, 1, 1), B.repeat(40, 1, 1), scale.repeat(40), ids)
        big_a = torch.zeros(n, r, n_in, dtype=torch.bfloat16, device="cuda")
        big_b = torch.zeros(n, n_out, r, dtype=torch.bfloat16, device="cuda")
        assert max(big_a.numel(), big_b.numel()) > 2 ** 31
        big_a[-1], big_b[-1] = A[0], B[0]
        got = q.linear_fwd_slots(x, w, big_a, big_b, scale.repeat(n), ids + n - 1)
        assert torch.equal(got, want)
        del big_a, big_b
    assert q.last_device_status() == 0


def test_outputs_of_more_than_2_31_values(cuda_lib):
    """The last 512 tokens of a batch whose output passes 2^31 values, against
    a call on them alone: the same bits."""
    q = cuda_lib
    M, n_in, n_out, r, n = 512 * 157, 64, 28672, 8, 5
    g = torch.Generator(device="cuda").manual_seed(3)
    W, _, A, B, scale = (t.cuda() for t in make(1, n_in, n_out, r, n, seed=3))
    x = torch.randn(M, n_in, generator=g, device="cuda").bfloat16()
    ids = torch.randint(-1, n, (M,), generator=g, device="cuda").int()
    w = q.quantize_nf4(W)
    h = q.linear_fwd_slots(x, w, A, B, scale, ids)
    assert h.numel() > 2 ** 31
    for k in (-512, 512 * 149):                     # (token 149 * 512 begins just below 2^31)
        part = slice(k, k + 512 if k > 0 else None)
        assert torch.equal(h[part], q.linear_fwd_slots(x[part].contiguous(), w, A, B, scale, ids[part].contiguous()))
    assert q.last_device_status() == 0
