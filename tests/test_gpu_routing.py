"""GPU parity of the operators on rows grouped by expert: sort_tokens, moe_dispatch_*,
moe_combine and its gradient, against the plain fp64 forms of oracle/routing.py.

Indices, copies and quantised codes must be exact.  Rounded results: bf16 keeps 8
significant bits, so a rounding is off by at most 2^-8 of the value; combine's fp32 sum of
k products adds k roundings of 2^-24 of the largest partial sum, at most k * 2^-24 *
sum |w y| (and its own rounding's share); a dot product of H terms, in any order, at
most H * 2^-24 * sum |d y|."""
import numpy as np
import pytest
import torch

import block_scaled_precision_05_amd as bsg
from block_scaled_precision_05_amd import workloads
from oracle import routing

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U24, U8 = 2.0 ** -24, 2.0 ** -8


def _say(msg):
    print(f"[gpu-test] {msg}", flush=True)


def _ids(T, k, G, seed, missing=0.15, bad=True):
    """Skewed choices; some negative, some past G."""
    r = np.random.default_rng(seed)
    if G == 0:
        return r.integers(-2, 3, (T, k)).astype(np.int32)
    ids = np.minimum((G * r.random((T, k)) ** 2).astype(np.int32), G - 1)
    drop = r.random((T, k))
    ids[drop < missing] = -1
    if bad:
        ids[drop > 0.98] = G + 5
    return ids


def _np(t):
    return t.detach().cpu().numpy()


def _f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _check_plan(plan, ids, G, align, cap, rows=None):
    want = routing.sort_tokens(ids, G, align, cap, rows)
    for name, a, b in zip(plan._fields, plan, want):
        assert np.array_equal(_np(a), b), name


SORT = [(1, 1, 1, 1, 0), (1, 1, 1024, 128, 0), (33, 6, 48, 1, 0), (64, 1, 3, 16, 0),
        (500, 8, 384, 128, 0),              # 4000 pairs: one workgroup, four steps
        (4096, 1, 1000, 7, 0),              # the largest single-workgroup sort
        (4097, 1, 1024, 16, 0),             # the smallest sort in two launches
        (16384, 6, 256, 128, 0), (3001, 3, 2, 1, 0), (777, 64, 5, 3, 0),
        (70000, 4, 33, 16, 0),              # more than one step per chunk
        (100, 6, 8, 1, 16), (4096, 6, 48, 1, 512), (5, 2, 1024, 1, 1), (300, 20, 3, 1, 5000)]


@pytest.mark.parametrize("T,k,G,align,cap", SORT)
def test_sort_matches_oracle(T, k, G, align, cap):
    _say(f"sort_tokens T={T} k={k} G={G} align={align} cap={cap}")
    ids = _ids(T, k, G, T + G)
    plan = bsg.sort_tokens(torch.from_numpy(ids).to(DEV), G, align=align, cap=cap)
    _check_plan(plan, ids, G, align, cap)


def test_sort_edges():
    """No tokens, no groups, every pair dropped, every pair in one group, strided ids, spare
    rows, the largest and smallest int32 as ids."""
    for T, k, G, cap in ((0, 2, 5, 0), (0, 2, 5, 3), (3, 0, 4, 0), (7, 2, 0, 0), (0, 0, 0, 0)):
        _say(f"sort_tokens T={T} k={k} G={G} cap={cap}")
        ids = _ids(T, k, G, 1)
        _check_plan(bsg.sort_tokens(torch.from_numpy(ids).to(DEV), G, cap=cap), ids, G, 1, cap)
    for fill in (-1, 2, 3, 2 ** 31 - 1, -2 ** 31):
        for T in (50, 3000):
            ids = np.full((T, 4), fill, np.int32)
            plan = bsg.sort_tokens(torch.from_numpy(ids).to(DEV), 3, align=16)
            _check_plan(plan, ids, 3, 16, 0)
    wide = torch.from_numpy(_ids(900, 9, 10, 2)).to(DEV)
    _check_plan(bsg.sort_tokens(wide[:, 2:7], 10, align=4), _np(wide)[:, 2:7], 10, 4, 0)
    ids = _ids(2000, 3, 10, 5)
    e = lambda *s: torch.full(s, 77, dtype=torch.int32, device=DEV)
    out = bsg.TokenSort(e(11), e(2000, 3), e(9001), e(9001))
    ws = torch.full((bsg.lib().sort_tokens_workspace(6000, 10) // 4,), 77, dtype=torch.int32, device=DEV)
    plan = bsg.sort_tokens(torch.from_numpy(ids).to(DEV), 10, align=8, out=out, workspace=ws)
    assert plan.row_of.data_ptr() == out.row_of.data_ptr()
    _check_plan(plan, ids, 10, 8, 0, rows=9001)


def _case(T, k, G, align, H, seed, ld_pad=0, cap=0, rows_extra=5):
    """A plan with spare rows, X, Y, W and dO as bf16 / fp32 tensors whose rows are ld_pad
    apart from contiguous."""
    ids = _ids(T, k, G, seed)
    rows = routing.rows_needed(T, k, G, align, cap) + rows_extra
    plan = bsg.TokenSort(*(torch.from_numpy(x).to(DEV)
                           for x in routing.sort_tokens(ids, G, align, cap, rows)))
    g = torch.Generator(device=DEV).manual_seed(seed)

    def mat(n, h, dtype=torch.bfloat16):
        return torch.randn(n, h + ld_pad, generator=g, device=DEV).to(dtype)[:, :h]
    W = mat(T, k, torch.float32)
    return plan, mat(T, H), mat(rows, H), W, mat(T, H), rows


SHAPES = [(1, 1, 1, 1, 8, 0), (3, 2, 4, 16, 1, 0), (33, 8, 16, 1, 520, 0), (65, 3, 5, 16, 1000, 0),
          (40, 9, 20, 4, 776, 8),            # more than eight choices a token, padded rows
          (17, 2, 3, 128, 513, 0),           # odd width: element-wise accesses
          (29, 5, 7, 3, 1024, 3),            # leading dimension not a multiple of 8
          (257, 6, 48, 16, 2056, 0), (130, 64, 9, 1, 128, 0)]


@pytest.mark.parametrize("T,k,G,align,H,pad", SHAPES)
def test_dispatch_bf16(T, k, G, align, H, pad):
    _say(f"moe_dispatch_bf16 T={T} k={k} G={G} align={align} H={H} pad={pad}")
    plan, X, _, _, _, rows = _case(T, k, G, align, H, T + H, pad)
    X[0, 0], X[0, H // 2] = float("nan"), float("-inf")     # copies are bits
    buf = torch.full((rows, H + pad), 3.0, dtype=torch.bfloat16, device=DEV)
    out = bsg.moe_dispatch_bf16(X, plan, out=buf[:, :H])
    bits = lambda t: _np(t.contiguous().view(torch.int16))
    want = routing.dispatch(bits(X), _np(plan.row_of), _np(plan.pair_of),
                            np.full((rows, H), 0x4040, np.int16))
    assert np.array_equal(bits(out), want)
    assert torch.all(buf[:, H:] == 3.0)


@pytest.mark.parametrize("rule", ["ceil", "ocp_mx"])
@pytest.mark.parametrize("fmt,T,k,G,align,H,cap", [
    ("fp8", 1, 1, 1, 1, 128, 0), ("fp8", 70, 6, 9, 16, 1152, 0), ("fp8", 33, 3, 200, 128, 7168, 0),
    ("fp8", 50, 17, 4, 1, 1024, 0), ("fp8", 96, 6, 8, 1, 640, 64), ("fp8", 700, 6, 32, 128, 2048, 0),
    ("fp4", 1, 1, 1, 1, 32, 0), ("fp4", 70, 6, 9, 16, 1120, 0), ("fp4", 33, 9, 30, 7, 2080, 0),
    ("fp4", 96, 6, 8, 1, 608, 64), ("fp4", 600, 4, 32, 128, 4096, 0)])
def test_dispatch_quantised(fmt, T, k, G, align, H, cap, rule):
    """Codes and scales are those of the per-token quantisers (checked against the oracle
    by their own tests), row by row; padding is a quantised zero row; rows of no group keep
    the fill in Q and in the scales."""
    _say(f"moe_dispatch_{fmt} T={T} k={k} G={G} align={align} H={H} cap={cap} {rule}")
    plan, _, _, _, _, rows = _case(T, k, G, align, 8, T + H, cap=cap)
    X = workloads.activations(T, H, seed=T + H, device=DEV)
    if T > 2:
        X[1] = 0.0
        X[2] = (X[2].float() * 2.0 ** -120).to(torch.bfloat16)
    per, gk = (1, 128) if fmt == "fp8" else (2, 32)
    quant = bsg.quantize_fp8_per_token if fmt == "fp8" else bsg.quantize_fp4_per_token
    disp = bsg.moe_dispatch_fp8 if fmt == "fp8" else bsg.moe_dispatch_fp4
    Qx, Px = quant(X, rule)
    Q0, P0 = quant(torch.zeros(1, H, dtype=torch.bfloat16, device=DEV), rule)
    buf = torch.full((rows, H // per + 16), 0xA5, dtype=torch.uint8, device=DEV)
    sf = torch.full(((H // gk + 1) // 2, rows + 3), 0x5A5A, dtype=torch.int16, device=DEV)
    Q, P = disp(X, plan, rule, out=buf[:, :H // per], sf_out=sf)
    pair = _np(plan.pair_of)
    for what, got, src, zero, fill in (
            ("codes", _np(Q), _np(Qx), _np(Q0)[0], 0xA5),
            ("scales", _np(P)[:, :rows].T, _np(Px).T, _np(P0)[:, 0], 0x5A5A)):
        want = np.full(got.shape, fill, got.dtype)
        want[pair == -1] = zero
        want[pair >= 0] = src[pair[pair >= 0] // k]
        assert np.array_equal(got, want), what
    assert torch.all(buf[:, H // per:] == 0xA5) and torch.all(sf[:, rows:] == 0x5A5A)


def _close(got, want, tol, what):
    d = np.abs(got - want)
    assert np.all(np.isfinite(got)) and np.all(d <= tol), \
        f"{what}: off by {np.max(d - tol):.3e} over the bound at {np.argmax(d - tol)}"
    _say(f"  {what}: {np.max(np.where(tol > 0, d / np.where(tol > 0, tol, 1), 0)):.2f} of the bound")


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,G,align,H,pad", SHAPES)
def test_combine(T, k, G, align, H, pad, weighted):
    _say(f"moe_combine T={T} k={k} G={G} align={align} H={H} pad={pad} weighted={weighted}")
    plan, _, Y, W, _, rows = _case(T, k, G, align, H, T + H, pad)
    W[plan.row_of < 0] = float("nan")            # weights of pairs without a row: not used
    Y[plan.pair_of < 0] = float("nan")           # rows without a pair: not read
    buf = torch.full((T, H + pad), 3.0, dtype=torch.bfloat16, device=DEV)
    out = bsg.moe_combine(Y, plan, W if weighted else None, out=buf[:, :H])
    want, mag = routing.combine(_f64(Y), _np(plan.row_of), _np(W) if weighted else None)
    _close(_f64(out), want, U8 * np.abs(want) + (1 + U8) * k * U24 * mag, "out")
    assert torch.all(buf[:, H:] == 3.0)


@pytest.mark.parametrize("T,k,G,align,H,pad", SHAPES)
def test_combine_backward(T, k, G, align, H, pad):
    _say(f"moe_combine_backward T={T} k={k} G={G} align={align} H={H} pad={pad}")
    plan, _, Y, W, dO, rows = _case(T, k, G, align, H, T + H, pad)
    none = plan.row_of < 0
    W[none] = float("nan")
    Y[plan.pair_of < 0] = float("nan")
    buf = torch.full((rows, H + pad), 3.0, dtype=torch.bfloat16, device=DEV)
    dY, dW = bsg.moe_combine_backward(dO, Y, plan, W, out=buf[:, :H])
    row_of, pair_of = _np(plan.row_of), _np(plan.pair_of)
    want, want_w, mag = routing.combine_backward(_f64(dO), _f64(Y), row_of, pair_of, _np(W),
                                                 np.full((rows, H), 3.0))
    _close(_f64(dY), want, (U8 + 2 * U24) * np.abs(want), "dY")
    _close(_f64(dW), want_w, H * U24 * mag, "dW")
    assert torch.all(buf[:, H:] == 3.0)
    # without the weights' gradient Y is not read; without weights dY is dO's rows
    dY1, none_w = bsg.moe_combine_backward(dO, None, plan, None, need_weights=False)
    assert none_w is None
    kept = plan.pair_of >= 0
    assert torch.equal(dY1[kept], dO[(plan.pair_of[kept] // k).long()])
    assert torch.all(dY1[plan.pair_of == -1] == 0)


def test_dropped_pairs_of_infinite_gradients_are_zero():
    """dO holds infinities: pairs without a row still have the gradient 0."""
    plan, _, Y, W, dO, rows = _case(20, 4, 3, 1, 512, 9)
    dO[:, 7] = float("inf")
    _, dW = bsg.moe_combine_backward(dO, Y, plan, W)
    assert torch.all(dW[plan.row_of < 0] == 0)
    assert not torch.any(torch.isfinite(dW[plan.row_of >= 0]))


@pytest.mark.parametrize("T", [0, 5])
def test_empty(T):
    """No tokens; tokens without any row; no groups at all."""
    _say(f"empty plans, T={T}")
    ids = torch.full((T, 3), -1, dtype=torch.int32, device=DEV)
    for G in (0, 4):
        plan = bsg.sort_tokens(ids, G, align=16)
        rows = plan.pair_of.numel()
        X = torch.ones(T, 256, dtype=torch.bfloat16, device=DEV)
        Y = torch.ones(rows, 256, dtype=torch.bfloat16, device=DEV)
        out = torch.full((rows, 256), 2.0, dtype=torch.bfloat16, device=DEV)
        assert torch.all(bsg.moe_dispatch_bf16(X, plan, out=out) == 2.0)
        bsg.moe_dispatch_fp8(X, plan)
        assert torch.all(bsg.moe_combine(Y, plan) == 0)
        dY, dW = bsg.moe_combine_backward(X, Y, plan, out=out)
        assert torch.all(dY == 2.0) and torch.all(dW == 0)


def test_broken_plans_stay_in_bounds():
    """Indices outside their arrays are skipped: rows past the end, pairs past the end."""
    _say("plans with indices out of range")
    plan, X, Y, W, dO, rows = _case(30, 3, 4, 16, 256, 3)
    plan.row_of[::3] = rows
    plan.row_of[1::3] = 2 ** 31 - 1
    plan.pair_of[::5] = 2 ** 31 - 1
    out = torch.full((rows, 256), 2.0, dtype=torch.bfloat16, device=DEV)
    bsg.moe_dispatch_bf16(X, plan, out=out)
    bsg.moe_dispatch_fp8(X, plan)
    got = bsg.moe_combine(Y, plan, W)
    want, mag = routing.combine(_f64(Y), np.where(_np(plan.row_of) < rows, _np(plan.row_of), -1), _np(W))
    _close(_f64(got), want, U8 * np.abs(want) + (1 + U8) * 3 * U24 * mag, "out")
    _, dW = bsg.moe_combine_backward(dO, Y, plan, W)
    assert torch.all(dW[plan.row_of >= rows] == 0)


def test_rows_past_32_bit_offsets():
    """Rows more than 2^32 bytes into the matrix."""
    rows, H, T = 1 << 17, 1 << 15, 4          # 8 GiB a matrix
    _say(f"rows past 4 GiB: {rows} x {H}")
    Y = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    X = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    row_of = torch.tensor([[rows - 1], [3], [rows // 2 + 1], [rows - 2]], dtype=torch.int32, device=DEV)
    pair_of = torch.full((rows,), -2, dtype=torch.int32, device=DEV)
    pair_of[row_of[:, 0].long()] = torch.arange(T, dtype=torch.int32, device=DEV)
    pair_of[rows - 3] = -1
    Y[rows - 3] = 5.0
    plan = (torch.zeros(2, dtype=torch.int32, device=DEV), row_of, pair_of, torch.zeros_like(pair_of))
    bsg.moe_dispatch_bf16(X, plan, out=Y)
    assert torch.equal(Y[row_of[:, 0].long()], X) and torch.all(Y[rows - 3] == 0)
    assert int(torch.count_nonzero(Y.any(1))) == T
    assert torch.equal(bsg.moe_combine(Y, plan), X)
    _, dW = bsg.moe_combine_backward(X, Y, plan, out=Y.new_empty(rows, H))
    want = (X.double() ** 2).sum(1, keepdim=True)
    assert torch.all((dW.double() - want).abs() <= H * U24 * want)


def test_same_result_every_run_other_stream_and_captured():
    """The chain sort -> dispatch -> combine -> backward: run twice, on a side stream, and
    captured into a graph that is replayed on new ids with eager calls in between."""
    _say("determinism, side stream, graph")
    T, k, G, H, align = 1500, 6, 40, 1024, 16
    rows = routing.rows_needed(T, k, G, align)
    g = torch.Generator(device=DEV).manual_seed(5)
    X = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    W = torch.rand(T, k, generator=g, device=DEV)
    ids = torch.from_numpy(_ids(T, k, G, 1)).to(DEV)
    A = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)
    Q = torch.zeros(rows, H, dtype=torch.uint8, device=DEV)
    P = torch.zeros(H // 256, rows, dtype=torch.int16, device=DEV)
    dA = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)

    def chain(stream=None):
        plan = bsg.sort_tokens(ids, G, align=align, stream=stream)
        bsg.moe_dispatch_bf16(X, plan, out=A, stream=stream)
        bsg.moe_dispatch_fp8(X, plan, out=Q, sf_out=P, stream=stream)
        out = bsg.moe_combine(A, plan, W, stream=stream)
        _, dW = bsg.moe_combine_backward(out, A, plan, W, out=dA, stream=stream)
        return (*plan, out, dW)

    def snap(res):
        torch.cuda.synchronize()
        return [t.clone() for t in (*res, A, Q, P, dA)]

    def clear():
        for t in (A, Q, P, dA):
            t.zero_()
        torch.cuda.synchronize()

    first = snap(chain())
    clear()
    for a, b in zip(first, snap(chain())):
        assert torch.equal(a, b)
    clear()
    side = torch.cuda.Stream()
    for a, b in zip(first, snap(chain(side))):
        assert torch.equal(a, b)
    clear()
    for a, b in zip(first, snap(chain(side.cuda_stream))):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = chain()
    for seed in (1, 2, 3, 2):
        ids.copy_(torch.from_numpy(_ids(T, k, G, seed)))
        clear()
        graph.replay()
        got = snap(captured)
        clear()
        for a, b in zip(got, snap(chain())):
            assert torch.equal(a, b)


def test_fp8_expert_layer():
    """The operators as they are used: sort, quantising dispatch, the FFN core, combine; each
    expert's rows and the output compared with the same steps without the sort."""
    _say("sort -> moe_dispatch_fp8 -> moe_ffn_fp8 -> moe_combine")
    T, k, G, hidden, inter = 300, 3, 6, 512, 256
    w = workloads.moe_ffn(11, device=DEV, hidden=hidden, inter=inter, counts=[128] * G)
    t = w.tensors
    sfw13 = torch.stack([bsg.ensure_packed(x, 2 * inter // 128, hidden // 128) for x in t["sfw13"]])
    sfw2 = torch.stack([bsg.ensure_packed(x, hidden // 128, inter // 128) for x in t["sfw2"]])
    X = workloads.activations(T, hidden, seed=3, device=DEV)
    ids = torch.from_numpy(_ids(T, k, G, 4)).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    W = torch.rand(T, k, generator=g, device=DEV)
    plan = bsg.sort_tokens(ids, G, align=128)
    A, sfa = bsg.moe_dispatch_fp8(X, plan)
    Y = bsg.moe_ffn_fp8(A, sfa, t["W13"], sfw13, t["W2"], sfw2, plan.offsets)
    out = bsg.moe_combine(Y, plan, W)
    # every token through every expert, one expert at a time
    Qx, Px = bsg.quantize_fp8_per_token(X)
    one = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    per = torch.stack([bsg.moe_ffn_fp8(Qx, Px, t["W13"][e:e + 1], sfw13[e:e + 1], t["W2"][e:e + 1],
                                       sfw2[e:e + 1], one) for e in range(G)])
    row_of = _np(plan.row_of)
    rows_want = torch.zeros_like(Y)
    for i, j in np.argwhere(row_of >= 0):
        rows_want[row_of[i, j]] = per[ids[i, j], i]
    kept = plan.pair_of >= 0
    assert torch.equal(Y[kept], rows_want[kept])
    want, mag = routing.combine(_f64(rows_want), row_of, _np(W))
    _close(_f64(out), want, U8 * np.abs(want) + (1 + U8) * k * U24 * mag, "out")


def test_masked_decode_layer():
    """The masked layout: sort with a capacity, quantising dispatch into [G, cap, K], the
    masked GEMM, combine."""
    _say("sort(cap) -> moe_dispatch_fp8 -> m_grouped_gemm_fp8_masked -> moe_combine")
    T, k, G, cap, N, K = 40, 4, 5, 24, 384, 512
    w = workloads.masked(7, device=DEV, G=G, cap=cap, N=N, K=K)
    t = w.tensors
    sfb = torch.stack([bsg.ensure_packed(x, N // 128, K // 128) for x in t["sfb"]])
    X = workloads.activations(T, K, seed=8, device=DEV)
    ids = torch.from_numpy(_ids(T, k, G, 6)).to(DEV)
    W = torch.rand(T, k, device=DEV)
    plan = bsg.sort_tokens(ids, G, cap=cap)
    assert int((plan.row_of < 0).sum()) > int(((ids < 0) | (ids >= G)).sum())   # some over capacity
    A, sfa = bsg.moe_dispatch_fp8(X, plan)
    Y = bsg.m_grouped_gemm_fp8_masked(A.view(G, cap, K), sfa, t["B"], sfb, plan.offsets).view(G * cap, N)
    out = bsg.moe_combine(Y, plan, W)
    Qx, Px = bsg.quantize_fp8_per_token(X)
    row_of = _np(plan.row_of)
    want_rows = np.zeros((G * cap, N))
    every = torch.tensor([T], dtype=torch.int32, device=DEV)
    for e in range(G):                 # every token through expert e alone
        D = _f64(bsg.m_grouped_gemm_fp8_masked(Qx.view(1, T, K), Px, t["B"][e:e + 1], sfb[e:e + 1],
                                               every))[0]
        for i, j in np.argwhere((row_of >= 0) & (_np(ids) == e)):
            want_rows[row_of[i, j]] = D[i]
    kept = _np(plan.pair_of) >= 0
    assert np.array_equal(_f64(Y)[kept], want_rows[kept])
    want, mag = routing.combine(want_rows, row_of, _np(W))
    _close(_f64(out), want, U8 * np.abs(want) + (1 + U8) * k * U24 * mag, "out")


@pytest.mark.parametrize("T,k,G,align,cap", [
    (64, 6, 256, 1, 1024), (700, 4, 37, 1, 3001), (30, 2, 1024, 512, 0), (900, 4, 64, 4096, 0), (1, 1, 3, 1, 70000)])
def test_sort_with_many_more_rows_than_pairs(T, k, G, align, cap):
    _say(f"sort_tokens T={T} k={k} G={G} align={align} cap={cap}")
    ids = _ids(T, k, G, T + G)
    rows = routing.rows_needed(T, k, G, align, cap) + 8192
    e = lambda *s: torch.full(s, 77, dtype=torch.int32, device=DEV)
    out = bsg.TokenSort(e(G if cap else G + 1), e(T, k), e(rows), e(rows))
    bsg.sort_tokens(torch.from_numpy(ids).to(DEV), G, align=align, cap=cap, out=out)
    _check_plan(out, ids, G, align, cap, rows=rows)


def test_calls_with_and_without_a_stream_agree():
    """A call on the current stream goes through the compiled marshalling, one that names its
    stream does not: same results, with and without given outputs, contiguous or not."""
    _say("both ways into the library")
    cur = torch.cuda.current_stream()
    T, k, G, H = 300, 4, 12, 512

    def agree(f, *args, **kw):
        def run(**more):
            for n in ("out", "sf_out"):
                if n in kw:
                    kw[n].zero_()
            r = f(*args, **kw, **more)
            return [x.clone() for x in ((r,) if torch.is_tensor(r) else r)]
        a, b = run(), run(stream=cur)
        for x, y in zip(a, b, strict=True):
            assert x.dtype == y.dtype and x.shape == y.shape and torch.equal(x, y), f.__name__
        return a

    def filled(*s, dtype=torch.bfloat16):
        return torch.zeros(s, dtype=dtype, device=DEV)
    plan, X, Y, W, dO, rows = _case(T, k, G, 16, H, 3, ld_pad=8)
    ids = torch.from_numpy(_ids(T, k, G, 3)).to(DEV)
    for kw in ({}, {"align": 32}, {"cap": 40}):
        assert isinstance(bsg.sort_tokens(ids, G, **kw), bsg.TokenSort)
        agree(bsg.sort_tokens, ids, G, **kw)
    # (rows of no group are not written: outputs that held zeros are compared whole)
    agree(bsg.moe_dispatch_bf16, X, plan, out=filled(rows, H))
    assert bsg.moe_dispatch_bf16(X, plan).shape == (rows, H)
    for f, per, gk in ((bsg.moe_dispatch_fp8, 1, 128), (bsg.moe_dispatch_fp4, 2, 32)):
        for rule in ("ceil", "ocp_mx"):
            q, sf = filled(rows, H // per, dtype=torch.uint8), filled(H // gk // 2, rows + 3, dtype=torch.int16)
            agree(f, X, plan, rule, out=q, sf_out=sf)
            got = f(X, plan, rule)
            real = plan.pair_of > -2
            assert torch.equal(got[0][real], q[real]) and torch.equal(got[1][:, real], sf[:, :rows][:, real])
    e4m3 = filled(rows, H, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert torch.equal(bsg.moe_dispatch_fp8(X, plan, out=e4m3)[0].view(torch.uint8), agree(
        bsg.moe_dispatch_fp8, X, plan, out=filled(rows, H, dtype=torch.uint8), sf_out=sf.new_zeros(2, rows))[0])
    agree(bsg.moe_combine, Y, plan, W)
    agree(bsg.moe_combine, Y, tuple(plan))
    wide = filled(T, H + 5)
    agree(bsg.moe_combine, Y, plan, W, out=wide[:, :H])
    assert torch.all(wide[:, H:] == 0)
    agree(bsg.moe_combine_backward, dO, Y, plan, W, out=filled(rows, H))
    agree(bsg.moe_combine_backward, dO, Y, plan, out=filled(rows, H))
    dY, none = bsg.moe_combine_backward(dO, None, plan, W, need_weights=False, out=filled(rows, H))
    assert none is None and torch.equal(dY, bsg.moe_combine_backward(dO, Y, plan, W, out=filled(rows, H))[0])


def test_wrong_arguments_raise_on_the_gpu():
    _say("refusals with tensors on the GPU")
    plan, X, Y, W, dO, rows = _case(20, 3, 4, 16, 256, 3)
    ids = torch.from_numpy(_ids(20, 3, 4, 3)).to(DEV)
    half, host = X.half(), X.cpu()
    bad_plan = bsg.TokenSort(plan.offsets, plan.row_of.long(), plan.pair_of, plan.row_group)
    short = torch.zeros(rows - 1, 256, dtype=torch.bfloat16, device=DEV)
    every_second = torch.zeros(rows, 512, dtype=torch.bfloat16, device=DEV)[:, ::2]
    for f, error in (
            (lambda: bsg.sort_tokens(ids.long(), 4), TypeError),
            (lambda: bsg.sort_tokens(ids[:, 0], 4), TypeError),
            (lambda: bsg.sort_tokens(ids, 4, align=0), ValueError),
            (lambda: bsg.sort_tokens(ids, -1), ValueError),
            (lambda: bsg.sort_tokens(ids, 1025), bsg.BsgError),
            (lambda: bsg.sort_tokens(ids, 4, align=16, cap=8), bsg.BsgError),
            (lambda: bsg.moe_dispatch_bf16(half, plan), TypeError),
            (lambda: bsg.moe_dispatch_bf16(X, bad_plan), TypeError),
            (lambda: bsg.moe_dispatch_bf16(X[:19], plan), ValueError),
            (lambda: bsg.moe_dispatch_bf16(X, plan, out=short), ValueError),
            (lambda: bsg.moe_dispatch_bf16(X, plan, out=every_second), ValueError),
            (lambda: bsg.moe_dispatch_bf16(host, plan), ValueError),
            (lambda: bsg.moe_dispatch_fp8(X, plan, rule="floor"), ValueError),
            (lambda: bsg.moe_dispatch_fp8(X[:, :200], plan), bsg.BsgError),
            (lambda: bsg.moe_dispatch_fp8(X[:, 4:132], plan), bsg.BsgError),
            (lambda: bsg.moe_dispatch_fp8(X, plan, sf_out=torch.zeros(1, rows - 1, dtype=torch.int16, device=DEV)),
             ValueError),
            (lambda: bsg.moe_combine(short, plan), ValueError),
            (lambda: bsg.moe_combine(Y, plan, W.bfloat16()), TypeError),
            (lambda: bsg.moe_combine(Y, plan, W[:, :2]), ValueError),
            (lambda: bsg.moe_combine_backward(dO, None, plan, W), ValueError),
            (lambda: bsg.moe_combine_backward(dO, short, plan, W), ValueError)):
        with pytest.raises(error):
            f()


# choices shared out to several workgroups, and a wave a token: few and many tokens, short
# rows, more than eight choices, tokens without rows, unweighted, without the weights' gradient
@pytest.mark.parametrize("T,k,G,H", [(1, 8, 64, 7168), (2, 3, 5, 2048), (7, 7, 9, 1024), (40, 20, 30, 520), (100, 64, 70, 256),
                                     (255, 2, 8, 512), (256, 5, 8, 1024), (700, 9, 12, 136), (3000, 6, 20, 512),
                                     (1200, 1, 4, 8), (9000, 4, 40, 512), (5000, 8, 30, 1024)])
def test_combine_backward_shared_out(T, k, G, H):
    _say(f"moe_combine_backward T={T} k={k} G={G} H={H}")
    plan, _, Y, W, dO, rows = _case(T, k, G, 16, H, T + k)
    row_of, pair_of = _np(plan.row_of), _np(plan.pair_of)
    for w in (W, None):
        out = torch.full((rows, H), 3.0, dtype=torch.bfloat16, device=DEV)
        dY, dW = bsg.moe_combine_backward(dO, Y, plan, w, out=out)
        again, none = bsg.moe_combine_backward(dO, None, plan, w, need_weights=False, out=torch.full_like(out, 3.0))
        assert none is None and torch.equal(again, dY)
        have = torch.from_numpy(row_of >= 0).to(DEV)
        t, j = torch.nonzero(have, as_tuple=True)
        r = plan.row_of[t, j].long()
        f = 1.0 if w is None else w[t, j][:, None]
        assert torch.equal(dY[r], (f * dO[t].float()).to(torch.bfloat16))     # one product, rounded once
        assert torch.all(dY[plan.pair_of == -1] == 0) and torch.all(dY[plan.pair_of == -2] == 3.0)
        prod = dO[t].double() * Y[r].double()
        want, mag = torch.zeros(T, k, dtype=torch.float64, device=DEV), torch.zeros(T, k, dtype=torch.float64, device=DEV)
        want[t, j], mag[t, j] = prod.sum(1), prod.abs().sum(1)
        assert torch.all((dW.double() - want).abs() <= H * U24 * mag)
        assert torch.all(dW[~have] == 0)


# ---------------------------------------------------------------------------
# Matrices past 32 MiB: copies with the non-temporal hint, and in the quantising dispatch
# another order of the workgroups.  Widths whose last segment is partial (and an odd number
# of scale blocks), numbers of workgroups that are no multiple of 8, padding and spare rows,
# tokens without rows; k up to, at and past eight.
# ---------------------------------------------------------------------------
STREAM = 32 << 20


def _stream_case(T, k, G, align, H, cap=0):
    """_case with every 17th token without a row."""
    ids = _ids(T, k, G, T + k)
    ids[::17] = -1
    rows = routing.rows_needed(T, k, G, align, cap) + 5
    plan = bsg.TokenSort(*(torch.from_numpy(x).to(DEV)
                           for x in routing.sort_tokens(ids, G, align, cap, rows)))
    g = torch.Generator(device=DEV).manual_seed(T)
    mat = lambda n, h: torch.randn(n, h, generator=g, device=DEV).to(torch.bfloat16)
    return plan, mat, rows, torch.randn(T, k, generator=g, device=DEV)


@pytest.mark.parametrize("T,k", [(8170, 1), (4099, 2), (2731, 3), (2049, 4), (1640, 5), (1367, 6), (1171, 7),
                                 (1025, 8), (750, 11), (130, 64)])
def test_streamed_dispatch_bf16_and_combine(T, k):
    H, G, align = 2056, 30, 16
    assert 2 * T * k * H >= STREAM
    _say(f"past 32 MiB: moe_dispatch_bf16, moe_combine T={T} k={k} H={H}")
    plan, mat, rows, W = _stream_case(T, k, G, align, H)
    pair = plan.pair_of.long()
    holds, pad = pair >= 0, pair == -1
    X = mat(T, H)
    buf = torch.full((rows, H + 8), 3.0, dtype=torch.bfloat16, device=DEV)
    bsg.moe_dispatch_bf16(X, plan, out=buf[:, :H])
    want = torch.full_like(buf, 3.0)
    want[pad, :H] = 0
    want[holds, :H] = X[pair[holds] // k]
    assert torch.equal(buf, want)

    Y = mat(rows, H)
    Y[~holds] = float("nan")                     # rows without a pair: not read
    have = plan.row_of >= 0
    W[~have] = float("nan")                      # weights of pairs without a row: not used
    for w in (W, None):
        buf = torch.full((T, H + 8), 3.0, dtype=torch.bfloat16, device=DEV)
        out = bsg.moe_combine(Y, plan, w, out=buf[:, :H])
        sum_, mag = (torch.zeros(T, H, dtype=torch.float64, device=DEV) for _ in range(2))
        for j in range(k):
            m = have[:, j]
            v = Y[plan.row_of[m, j].long()].double() * (1.0 if w is None else w[m, j, None].double())
            sum_[m] += v
            mag[m] += v.abs()
        assert torch.all((out.double() - sum_).abs() <= U8 * sum_.abs() + (1 + U8) * k * U24 * mag)
        assert torch.all(buf[:, H:] == 3.0)


@pytest.mark.parametrize("rule", ["ceil", "ocp_mx"])
@pytest.mark.parametrize("fmt,T,k,G,align,H,cap", [
    ("fp8", 29131, 1, 12, 16, 1152, 0), ("fp8", 4863, 6, 40, 16, 1152, 0), ("fp8", 3240, 9, 40, 1, 1152, 0),
    ("fp8", 4863, 6, 40, 1, 1152, 700), ("fp8", 670, 7, 9, 128, 7168, 0),
    ("fp4", 9987, 6, 40, 16, 1120, 0), ("fp4", 3525, 17, 30, 7, 1120, 0), ("fp4", 2710, 6, 20, 1, 4128, 800)])
def test_streamed_dispatch_quantised(fmt, T, k, G, align, H, cap, rule):
    per, gk = (1, 128) if fmt == "fp8" else (2, 32)
    assert T * k * H // per >= STREAM
    _say(f"past 32 MiB: moe_dispatch_{fmt} T={T} k={k} G={G} align={align} H={H} cap={cap} {rule}")
    plan, _, rows, _ = _stream_case(T, k, G, align, H, cap)
    X = workloads.activations(T, H, seed=T + H, device=DEV)
    X[1] = 0.0
    X[2] = (X[2].float() * 2.0 ** -120).to(torch.bfloat16)
    quant = bsg.quantize_fp8_per_token if fmt == "fp8" else bsg.quantize_fp4_per_token
    disp = bsg.moe_dispatch_fp8 if fmt == "fp8" else bsg.moe_dispatch_fp4
    Qx, Px = quant(X, rule)
    Q0, P0 = quant(torch.zeros(1, H, dtype=torch.bfloat16, device=DEV), rule)
    buf = torch.full((rows, H // per + 16), 0xA5, dtype=torch.uint8, device=DEV)
    sf = torch.full(((H // gk + 1) // 2, rows + 3), 0x5A5A, dtype=torch.int16, device=DEV)
    disp(X, plan, rule, out=buf[:, :H // per], sf_out=sf)
    pair = plan.pair_of.long()
    holds, pad = pair >= 0, pair == -1
    want = torch.full_like(buf, 0xA5)
    want[pad, :H // per] = Q0
    want[holds, :H // per] = Qx[pair[holds] // k]
    assert torch.equal(buf, want), "codes"
    # scales with a row's words side by side
    want = torch.full_like(sf, 0x5A5A).t().contiguous()
    of_x, of_0 = Px.t().contiguous(), P0.t().contiguous()
    want[:rows][pad] = of_0
    want[:rows][holds] = of_x[pair[holds] // k]
    assert torch.equal(sf.t().contiguous(), want), "scales"


def test_streamed_chain_captured():
    """sort -> FP8 dispatch and bf16 dispatch -> combine past 32 MiB, captured and replayed on
    new ids and tokens, with the same calls made eagerly in between."""
    T, k, G, H, align = 4870, 6, 40, 1152, 16
    assert T * k * H >= STREAM
    rows = routing.rows_needed(T, k, G, align)
    ids = torch.from_numpy(_ids(T, k, G, 1)).to(DEV)
    X = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    W = torch.rand(T, k, device=DEV)
    A = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)
    Q = torch.zeros(rows, H, dtype=torch.uint8, device=DEV)
    P = torch.zeros((H // 128 + 1) // 2, rows, dtype=torch.int16, device=DEV)

    def chain():
        plan = bsg.sort_tokens(ids, G, align=align)
        bsg.moe_dispatch_bf16(X, plan, out=A)
        bsg.moe_dispatch_fp8(X, plan, out=Q, sf_out=P)
        return bsg.moe_combine(A, plan, W)

    def snap(out):
        torch.cuda.synchronize()
        r = [t.clone() for t in (out, A, Q, P)]
        for t in (A, Q, P):
            t.zero_()
        torch.cuda.synchronize()
        return r
    snap(chain())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = chain()
    snap(captured)
    for seed in (1, 2, 3, 2):
        ids.copy_(torch.from_numpy(_ids(T, k, G, seed)))
        X.copy_(workloads.activations(T, H, seed=seed, device=DEV))
        torch.cuda.synchronize()
        graph.replay()
        got = snap(captured)
        for a, b in zip(got, snap(chain()), strict=True):
            assert torch.equal(a, b)


def test_expert_layer_under_autograd():
    """The functions record no graph; in training they stand in autograd Functions.  All
    values are integers and powers of two, so that every sum is exact: equal to fp64."""
    _say("dispatch -> experts -> combine, trained")
    T, k, G, H, align = 70, 3, 6, 64, 16
    g = torch.Generator(device=DEV).manual_seed(6)
    ids = torch.from_numpy(_ids(T, k, G, 9)).to(DEV)
    plan = bsg.sort_tokens(ids, G, align=align)
    rows = plan.pair_of.numel()

    class Dispatch(torch.autograd.Function):
        @staticmethod
        def forward(ctx, X):
            return bsg.moe_dispatch_bf16(X, plan, out=X.new_zeros(rows, H))

        @staticmethod
        def backward(ctx, dA):
            return bsg.moe_combine(dA.contiguous(), plan)

    class Combine(torch.autograd.Function):
        @staticmethod
        def forward(ctx, Y, W):
            ctx.save_for_backward(Y, W)
            return bsg.moe_combine(Y, plan, W)

        @staticmethod
        def backward(ctx, dO):
            Y, W = ctx.saved_tensors
            return bsg.moe_combine_backward(dO.contiguous(), Y, plan, W, out=torch.zeros_like(Y))

    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device=DEV)
    X, dO = ints(T, H).to(torch.bfloat16), ints(T, H).to(torch.bfloat16)
    W = torch.exp2(-torch.randint(0, 3, (T, k), generator=g, device=DEV).float())
    s = torch.exp2(torch.randint(-1, 2, (G,), generator=g, device=DEV).float())
    assert not bsg.moe_dispatch_bf16(X.clone().requires_grad_(), plan).requires_grad
    X.requires_grad_(), W.requires_grad_()
    Y = Dispatch.apply(X) * s[plan.row_group.clamp_min(0).long(), None].to(torch.bfloat16)
    out = Combine.apply(Y, W)
    out.backward(dO)

    Xd, Wd = X.detach().double().requires_grad_(), W.detach().double().requires_grad_()
    kept = (ids >= 0) & (ids < G)
    f = torch.where(kept, s.double()[ids.clamp(0, G - 1).long()], 0.0)
    want = (Wd * f).sum(1, keepdim=True) * Xd
    want.backward(dO.double())
    assert torch.equal(out.double(), want)
    assert torch.equal(X.grad.double(), Xd.grad) and torch.equal(W.grad.double(), Wd.grad)
