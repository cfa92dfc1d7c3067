"""Host-side checks of the operators on grouped rows that need no GPU: bad arguments are
refused with the documented status before any HIP call, and the binding refuses wrong
types, shapes and devices."""
import pytest
import torch

import block_scaled_precision_05_amd as bsg

INV, SHAPE, ALIGN, OK = (bsg.BSG_ERR_INVALID_ARG, bsg.BSG_ERR_UNSUPPORTED_SHAPE,
                         bsg.BSG_ERR_MISALIGNED, bsg.BSG_OK)
# fake, never-dereferenced device addresses: validation fails before any HIP call
P, P2, P3, P4, P5 = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000


def _try(f, good, changes):
    """Each change ({index: value}, status) of the good arguments gives that status."""
    for change, status in changes:
        a = list(good)
        for i, v in change.items():
            a[i] = v
        assert f(*a) == status, (change, status)


def test_sort_refusals():
    L = bsg.lib()
    #       ids ld T    k  G  al cap off row pair grp rows ws bytes stream
    good = [P, 4, 100, 4, 8, 16, 0, P2, P3, P4, P5, 520, 0, 0, None]
    _try(L.sort_tokens, good, [
        ({2: -1}, INV), ({3: -1}, INV), ({4: -1}, INV), ({5: 0}, INV), ({6: -1}, INV), ({11: -1}, INV),
        ({1: 3}, INV),                        # ld_ids < k
        ({0: 0}, INV), ({7: 0}, INV), ({8: 0}, INV), ({9: 0}, INV), ({10: 0}, INV),
        ({11: 519}, INV),                     # 400 pairs + 8 * 15 padding rows
        ({4: 1025}, SHAPE), ({3: 65, 1: 65}, SHAPE),
        ({2: 1 << 31, 11: 1 << 40}, SHAPE), ({11: 1 << 31}, SHAPE),
        ({5: 1 << 30}, SHAPE),
        ({6: 8}, INV),                        # masked layout takes align 1
        ({6: 100, 5: 1}, INV),                # 8 * 100 rows do not fit 520
        ({6: 1 << 30, 5: 1}, SHAPE),
        ({0: P + 2}, ALIGN), ({7: P2 + 1}, ALIGN), ({8: P3 + 2}, ALIGN), ({9: P4 + 2}, ALIGN),
        ({10: P5 + 2}, ALIGN),
    ])
    # many pairs need a workspace
    assert L.sort_tokens_workspace(400, 8) == 0
    need = L.sort_tokens_workspace(40000, 8)
    assert need > 0
    big = list(good)
    big[2], big[11] = 10000, 40120
    _try(L.sort_tokens, big, [({}, INV), ({12: P, 13: need - 1}, INV), ({12: 0, 13: need}, INV),
                              ({12: P + 1, 13: need}, ALIGN)])


def test_dispatch_refusals():
    L = bsg.lib()
    #       X  ldx  row pair T   k  rows H    out ldo stream
    good = [P, 256, P2, P3, 100, 4, 500, 256, P4, 256, None]
    _try(L.moe_dispatch_bf16, good, [
        ({4: -1}, INV), ({5: -1}, INV), ({6: -1}, INV), ({7: -1}, INV),
        ({0: 0}, INV), ({2: 0}, INV), ({3: 0}, INV), ({8: 0}, INV), ({1: 255}, INV), ({9: 255}, INV),
        ({5: 65}, SHAPE), ({6: 1 << 31}, SHAPE), ({7: 1 << 29, 1: 1 << 29, 9: 1 << 29}, SHAPE),
        ({4: 1 << 30}, SHAPE), ({0: P + 1}, ALIGN), ({8: P4 + 1}, ALIGN), ({2: P2 + 2}, ALIGN),
        ({6: 0}, OK), ({7: 0}, OK),           # nothing to write
    ])
    for name, H in (("moe_dispatch_fp8", 256), ("moe_dispatch_fp4", 256)):
        per = 1 if name.endswith("fp8") else 2
        #       X  ldx  row pair T   k  rows H  Q   ldq      sf  ld_sf rule stream
        good = [P, 256, P2, P3, 100, 4, 500, H, P4, H // per, P5, 500, 0, None]
        _try(getattr(L, name), good, [
            ({4: -1}, INV), ({0: 0}, INV), ({8: 0}, INV), ({10: 0}, INV), ({12: 2}, INV),
            ({9: H // per - 1}, INV), ({11: 499}, INV), ({1: 248}, INV),
            ({7: 240}, SHAPE), ({5: 65}, SHAPE),
            ({0: P + 8}, ALIGN), ({1: 260}, ALIGN), ({8: P4 + 4}, ALIGN), ({9: H // per + 4}, ALIGN),
            ({10: P5 + 1}, ALIGN), ({6: 0}, OK), ({7: 0}, OK),
        ])


def test_combine_refusals():
    L = bsg.lib()
    #       Y  ldy  row W  ldw T   k  rows H    out ldo stream
    good = [P, 256, P2, P3, 4, 100, 4, 500, 256, P4, 256, None]
    _try(L.moe_combine, good, [
        ({5: -1}, INV), ({6: -1}, INV), ({7: -1}, INV), ({8: -1}, INV),
        ({0: 0}, INV), ({2: 0}, INV), ({9: 0}, INV), ({1: 255}, INV), ({10: 255}, INV), ({4: 3}, INV),
        ({6: 65}, SHAPE), ({0: P + 1}, ALIGN), ({3: P3 + 2}, ALIGN), ({9: P4 + 1}, ALIGN),
        ({5: 0}, OK), ({8: 0}, OK),
    ])
    #       dO ldo  Y  ldy  row pair W  ldw T   k  rows H    dY  lddy dW  lddw stream
    good = [P, 256, P, 256, P2, P3, P4, 4, 100, 4, 500, 256, P5, 256, P2, 4, None]
    _try(L.moe_combine_backward, good, [
        ({8: -1}, INV), ({9: -1}, INV), ({10: -1}, INV), ({11: -1}, INV),
        ({0: 0}, INV), ({2: 0}, INV), ({4: 0}, INV), ({5: 0}, INV), ({12: 0}, INV),
        ({1: 255}, INV), ({3: 255}, INV), ({13: 255}, INV), ({7: 3}, INV), ({15: 3}, INV),
        ({9: 65}, SHAPE), ({0: P + 1}, ALIGN), ({12: P5 + 1}, ALIGN), ({14: P2 + 2}, ALIGN),
        ({6: P4 + 1}, ALIGN), ({8: 0, 10: 0}, OK),
    ])


def test_lora_refusals():
    L = bsg.lib()
    assert L.lora_add_workspace(100, 0, 4, 256, 512, 16) == 0
    need = L.lora_add_workspace(100, 256, 4, 256, 512, 16)
    assert need >= 256 * 16 * 4
    names = ("X ldx A lda stride_a B ldb stride_b scale off row pair grp rows base ldbase out ldo T G N K r ws "
             "wsbytes stream").split()
    at = {n: i for i, n in enumerate(names)}

    def args(**kw):
        return [kw[n] for n in names]

    def refuse(good, changes):
        _try(L.lora_add_bf16, good, [({at[n]: v for n, v in c.items()}, st) for c, st in changes])
    good = args(X=P, ldx=512, A=P, lda=512, stride_a=16 * 512, B=P, ldb=16, stride_b=256 * 16, scale=P2, off=P2, row=P2,
                pair=P3, grp=P4, rows=256, base=P5, ldbase=256, out=0x90000, ldo=256, T=100, G=4, N=256, K=512, r=16,
                ws=0x80000, wsbytes=need, stream=None)
    refuse(good, [
        ({"ws": 0}, INV), ({"wsbytes": need - 1}, INV),
        *[({n: -1}, INV) for n in ("T", "G", "N", "K", "r", "rows", "wsbytes")],
        *[({n: 0}, INV) for n in ("X", "A", "B", "off", "row", "pair", "grp", "out")],
        ({"ldx": 504}, INV), ({"lda": 504}, INV), ({"ldb": 8}, INV), ({"ldbase": 255}, INV), ({"ldo": 255}, INV),
        ({"stride_a": 16 * 512 - 8}, INV), ({"stride_b": 256 * 16 - 8}, INV),
        ({"out": P5, "ldo": 264}, INV),       # in place with another leading dimension
        ({"r": 12}, SHAPE), ({"r": 136, "ldb": 136}, SHAPE), ({"K": 508}, SHAPE), ({"G": 1025}, SHAPE),
        *[({n: P + 8}, ALIGN) for n in ("X", "A", "B")],
        *[({n: P2 + 2}, ALIGN) for n in ("scale", "off", "row", "pair", "grp")],
        ({"ldx": 516}, ALIGN), ({"lda": 516, "stride_a": 16 * 516}, ALIGN), ({"ldb": 20, "stride_b": 256 * 24}, ALIGN),
        ({"ws": 0x80008}, ALIGN), ({"out": 0x90001}, ALIGN), ({"base": P5 + 1}, ALIGN),
        ({"T": 0}, OK), ({"N": 0}, OK),
    ])
    for T, rows, K, N, r in ((100, 256, 8192, 4096, 128), (8192, 8256, 512, 256, 16)):
        need = L.lora_add_workspace(T, rows, 4, N, K, r)
        assert need >= rows * r * 4
        big = args(X=P, ldx=K, A=P, lda=K, stride_a=r * K, B=P, ldb=r, stride_b=N * r, scale=P2, off=P2, row=P2, pair=P3,
                   grp=P4, rows=rows, base=P5, ldbase=N, out=0x90000, ldo=N, T=T, G=4, N=N, K=K, r=r, ws=0x80000,
                   wsbytes=need, stream=None)
        refuse(big, [({"ws": 0}, INV), ({"wsbytes": need - 1}, INV), ({"ws": 0x80008}, ALIGN)])


def test_launches_past_the_grid_limit_are_refused():
    """2^24 workgroups of 256 work-items would not fit a launch."""
    L = bsg.lib()
    #                         X  ldx   row pair T        k  rows     H     out ldo   stream
    _try(L.moe_dispatch_bf16, [P, 2048, P2, P3, 1 << 24, 1, 1, 2048, P4, 2048, None], [({}, SHAPE)])
    _try(L.moe_dispatch_bf16, [P, 8, P2, P3, 1, 1, 1 << 28, 8, P4, 8, None], [({}, SHAPE)])
    _try(L.moe_dispatch_fp8, [P, 4096, P2, P3, 1 << 24, 1, 1, 4096, P4, 4096, P5, 1, 0, None], [({}, SHAPE)])
    #                   Y  ldy   row W  ldw T        k  rows H     out ldo   stream
    _try(L.moe_combine, [P, 2048, P2, P3, 1, 1 << 24, 1, 1, 2048, P4, 2048, None],
         [({}, SHAPE), ({5: 1 << 23, 8: 2047}, SHAPE)])      # an odd width: element-wise
    #                            dO ldo Y ldy row pair W  ldw T      k  rows H  dY lddy dW  lddw stream
    _try(L.moe_combine_backward, [P, 8, P, 8, P2, P3, P4, 1, 1 << 24, 1, 1, 8, P5, 8, P2, 1, None], [({}, SHAPE)])
    T, G, N, K, r = 1 << 20, 4, 1 << 22, 64, 16
    need = L.lora_add_workspace(T, T, G, N, K, r)
    #                     X  ldx A  lda sa      B  ldb sb      sc off row pair grp rows base ldb out ldo
    _try(L.lora_add_bf16, [P, K, P, K, r * K, P, r, N * r, 0, P2, P2, P3, P4, T, P5, N, 0x90000, N, T, G, N, K, r,
                           0x80000, need, None],
         [({}, SHAPE), ({13: (1 << 26) + 1}, SHAPE), ({18: (1 << 26) + 1}, SHAPE), ({20: (1 << 23) + 8}, SHAPE)])


def _plan(T=4, k=2, rows=8):
    e = lambda *s: torch.zeros(s, dtype=torch.int32)
    return bsg.TokenSort(e(3), e(T, k), e(rows), e(rows))


def test_binding_refuses_host_tensors():
    X = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bsg.sort_tokens(torch.zeros(4, 2, dtype=torch.int32), 2)
    for f in (bsg.moe_dispatch_bf16, bsg.moe_dispatch_fp8, bsg.moe_dispatch_fp4, bsg.moe_combine):
        with pytest.raises(ValueError):
            f(X, _plan())
    with pytest.raises(ValueError):
        bsg.moe_combine_backward(X, X, _plan())
    with pytest.raises(ValueError):
        bsg.lora_add_bf16(X, X[None], X[None], _plan(k=1))


def test_sort_refuses_rows_that_a_grid_could_step_past():
    """Rows are walked in 32 bits by up to 2^18 work-items: the step past the last row must
    not wrap, so plans of more than 2^31 - 2^18 rows are refused.  (A workspace that is
    missing is refused after the sizes, so that nothing here launches.)"""
    L = bsg.lib()
    most = 2 ** 31 - 2 ** 18
    for T, k, align, cap in ((1, 1, 1, 0), (10000, 4, 16, 0), (10000, 4, 1, 5)):
        #       ids ld T  k  G  al     cap  off row pair grp rows ws bytes stream
        args = [P, k, T, k, 8, align, cap, P2, P3, P4, P5, most, 0, 0, None]
        for rows in (most + 1, 2 ** 31 - 1025, 2 ** 31 - 1, 2 ** 31):
            args[11] = rows
            assert L.sort_tokens(*args) == SHAPE, (T, rows)
        if T > 1:
            args[11] = most
            assert L.sort_tokens(*args) == INV


def _tiles_apart(T, rows, G, N, K, r):
    """Whether lora_add_bf16 takes the plan's tiles one by one: its workspace is then S slabs
    of fp32 sums, a slice of at least 1024 elements of K each, and nothing behind them."""
    tiles = -(-rows // 16)
    S = max(1, min(512 // tiles, -(-K // 1024)))
    return bsg.lib().lora_add_workspace(T, rows, G, N, K, r) == 4 * S * tiles * 16 * r


def test_lora_groups_no_more_tiles_than_it_can_count():
    """Grouped tiles are taken by stages of K that are counted in 32 bits.  A plan that is
    mostly padding can have more than 2^30 of them: its tiles are not grouped, whatever the
    number of its tokens."""
    K = 1 << 22                               # 65536 stages an item of four tiles
    rows = 64 * ((1 << 14) - 2)
    assert not _tiles_apart(16, rows, 2, 8, K, 8)           # 2^14 items
    assert _tiles_apart(16, rows + 64, 2, 8, K, 8)          # one more
    assert _tiles_apart(1 << 20, 1 << 26, 1024, 1024, 1 << 20, 128)


def test_lora_limits_follow_the_form():
    """The limit of a launch's workgroups is that of grouped tiles: a call that takes its
    tiles one by one is not refused for it.  (The missing workspace is refused after the
    sizes, so that nothing here launches.)"""
    L = bsg.lib()

    def status(T, rows, G, N, K, r):
        #                      X  ldx A  lda sa     B  ldb sb     sc off row pair grp rows  base ldb out ldo
        return L.lora_add_bf16(P, K, P, K, r * K, P, r, N * r, 0, P2, P2, P3, P4, rows, P5, N, 0x90000, N,
                               T, G, N, K, r, 0, 0, None)
    for T, rows, G, N, K, r in ((1, 16, 1024, 1 << 22, 8, 8),       # many adapters, a wide output
                                (1, 16, 1024, 1 << 23, 8, 8),
                                (1, 1 << 26, 1, 4096, 8, 8),        # many spare rows
                                (4, 64, 1024, 1 << 23, 8, 8),       # the widest
                                (5, 80, 1024, 1 << 23, 8, 8)):      # grouped: 2 + 5 items of 2^15 blocks
        assert status(T, rows, G, N, K, r) == INV, (T, rows, G, N)
    # grouped: 4096 items and one more per adapter, 4096 blocks of 256 columns
    assert status(1 << 16, 1 << 18, 4, 1 << 20, 64, 8) == SHAPE      # 4100 * 4096
    assert status(1 << 16, (1 << 18) - 320, 4, 1 << 20, 64, 8) == INV  # 4095 * 4096


def test_empty_operands():
    """The matrix operands of the products keep their check of the strides when they are
    empty; the operators on grouped rows take empty operands of any stride."""
    odd = torch.zeros(8, 16, dtype=torch.bfloat16)[:0, ::2]       # [0, 8], every second column
    with pytest.raises(ValueError, match="unit stride"):
        bsg._mat(odd, "A")
    assert bsg._mat(torch.zeros(8, 16)[:0, :8], "A") == 16
    assert bsg._ld(odd, "X", torch.bfloat16, 0, 8) == 8
    assert bsg._ld(torch.zeros(0, 5, dtype=torch.bfloat16).t(), "X", torch.bfloat16, 5, 0) == 0


def test_a_missing_binding_is_named(monkeypatch, tmp_path):
    """Without _binding.so (a library built before there was one) the operators that use it
    raise as every call does without libbsg.so: naming the file and the build command."""
    monkeypatch.setattr(bsg, "BINDING_PATH", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(bsg, "_native_module", None)
    for f in (lambda: bsg.sort_tokens(torch.zeros(4, 2, dtype=torch.int32), 2),
              lambda: bsg.moe_combine(torch.zeros(8, 128, dtype=torch.bfloat16), _plan())):
        with pytest.raises(RuntimeError, match="_binding.so is missing: build it with"):
            f()


def test_lora_workspace_refusals_of_grouped_tiles():
    """As in test_lora_refusals, at sizes that group tiles (with the slabs added by the second
    product, and joined)."""
    L = bsg.lib()
    G = 4
    for T, rows, K, N, r in ((8192, 8256, 512, 512, 48), (1024, 1104, 8192, 4096, 128)):
        assert not _tiles_apart(T, rows, G, N, K, r)
        need = L.lora_add_workspace(T, rows, G, N, K, r)
        for ws, size, status in ((0, need, INV), (0x80000, need - 1, INV), (0x80000, 0, INV), (0x80008, need, ALIGN)):
            assert L.lora_add_bf16(P, K, P, K, r * K, P, r, N * r, P2, P2, P2, P3, P4, rows, P5, N, 0x90000, N,
                                   T, G, N, K, r, ws, size, None) == status, (T, ws, size)


def test_documented_limits_are_the_checked_ones():
    """The largest sizes that the header allows pass the check of the sizes (a missing pointer
    is refused after it, so that nothing launches), the next ones do not."""
    L = bsg.lib()

    def sort(T=10000, G=8, align=1, cap=0, rows=2 ** 31 - 2 ** 18):
        return L.sort_tokens(P, 4, T, 4, G, align, cap, P2, P3, P4, P5, rows, 0, 0, None)
    assert sort(align=2 ** 20 - 1) == INV and sort(align=2 ** 20) == SHAPE
    assert sort(cap=2 ** 27 - 1) == INV and sort(cap=2 ** 27) == SHAPE
    assert sort(T=2 ** 21) == INV and sort(T=2 ** 21 + 1) == SHAPE
    assert sort(G=1024) == INV and sort(G=1025) == SHAPE

    def dispatch(T=100, k=4, rows=500, H=256, ldx=2 ** 40):
        return L.moe_dispatch_bf16(P, ldx, P2, P3, T, k, rows, H, 0, 2 ** 40, None)

    def combine(T=100, k=4, rows=500, H=256, ldx=2 ** 40):
        return L.moe_combine(P, ldx, P2, P3, k, T, k, rows, H, 0, 2 ** 40, None)
    for f in (dispatch, combine):
        assert f() == INV and f(ldx=2 ** 40 + 1) == SHAPE
        assert f(k=64) == INV and f(k=65) == SHAPE
        assert f(H=2 ** 28) == INV and f(H=2 ** 28 + 1) == SHAPE
        assert f(rows=2 ** 31 - 1025) == INV and f(rows=2 ** 31 - 1024) == SHAPE
        assert f(T=2 ** 31 - 1025, k=1) == INV and f(T=2 ** 31 - 1024, k=1) == SHAPE
