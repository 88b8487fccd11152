"""Experts (moe.py): the sort against a plain one, dispatch, combine and its
gradient against float64, the sorted casts bit for bit against the oracle, the
grouped products against float64 and bit for bit against fp8_gemm_scaled on
each expert's own rows, the layer's gradients, and a captured step.

Tolerances, derived before the first run: one rounding to a type with half step
u is off by u |ref| (bf16 2^-8, fp32 2^-24); a binary32 sum of n products in
any order by (n + 2) 2^-24 of the sum of their magnitudes; the products keep
fp8_gemm_scaled's 2^-10 of the sum of magnitudes (+ 2^-8 |ref| in bf16)."""
import numpy as np
import pytest
import torch

import fp8_scaled_quantization_scale_amd as fm
import oracle
from fp8_scaled_quantization_scale_amd import linear, moe, norm
from gpu_util import FMT_NAME, host, need_gpu, same_f32

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
B, F = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _routing(tokens, topk, experts, seed, kind="random", dtype=torch.int64):
    g = _gen(seed)
    if kind == "one":  # everything to the last expert, the others empty
        e = torch.full((tokens, topk), experts - 1, device="cuda")
    elif kind == "none":
        e = torch.full((tokens, topk), -1, device="cuda")
    else:
        e = torch.randint(0, experts, (tokens, topk), generator=g, device="cuda")
        if kind == "dropped":
            far = torch.tensor([-1, experts, -(1 << 31), (1 << 31) - 1], device="cuda")
            e = torch.where(torch.rand(tokens, topk, generator=g, device="cuda") < 0.3,
                            far[torch.randint(0, 4, (tokens, topk), generator=g, device="cuda")], e)
        if kind == "half":  # only even experts
            e = e // 2 * 2
    w = torch.rand(tokens, topk, generator=g, device="cuda") + 0.1
    return e.to(dtype), w


def _plain_sort(e, experts):
    e = e.cpu().numpy().reshape(-1).astype(np.int64)
    rows = int(fm.fp8_moe_rows(e.size, 1, experts))
    counts = np.array([(e == x).sum() for x in range(experts)])
    offsets = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    row_slot, slot_row = np.full(rows, -1), np.full(e.size, -1)
    for x in range(experts):
        s = np.nonzero(e == x)[0]
        slot_row[s] = offsets[x] + np.arange(s.size)
        row_slot[slot_row[s]] = s
    return offsets, counts, row_slot, slot_row


ROUTINGS = [
    (1, 1, 1, "random"), (1, 1, 7, "random"), (3, 2, 5, "random"), (200, 2, 8, "random"), (129, 1, 1, "random"),
    (128, 1, 1, "random"), (333, 8, 64, "dropped"), (257, 6, 129, "half"), (500, 2, 4, "one"), (70, 3, 9, "none"),
    (1000, 4, 1024, "random"), (5000, 8, 256, "dropped"), (4097, 1, 3, "random"), (40000, 8, 33, "random"),
]


@pytest.mark.parametrize("tokens,topk,experts,kind", ROUTINGS)
@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
def test_sort(tokens, topk, experts, kind, dtype):
    need_gpu()
    e, _ = _routing(tokens, topk, experts, 11, kind, dtype)
    p = moe.sort(e, experts)
    offsets, counts, row_slot, slot_row = _plain_sort(e, experts)
    assert np.array_equal(host(p.offsets), offsets) and np.array_equal(host(p.counts), counts)
    assert p.rows >= offsets[-1] and p.rows == fm.fp8_moe_rows(tokens, topk, experts)
    assert np.array_equal(host(p.slot_row).reshape(-1), slot_row)
    want = np.full(p.rows, -1)
    want[:min(row_slot.size, p.rows)] = row_slot[:p.rows]
    assert np.array_equal(host(p.row_slot), want)


def test_sort_strided_and_empty():
    need_gpu()
    wide, _ = _routing(700, 9, 13, 5)
    p, q = moe.sort(wide[:, 2:5], 13), moe.sort(wide[:, 2:5].contiguous(), 13)
    for name in ("offsets", "counts", "row_slot", "slot_row"):
        assert torch.equal(getattr(p, name), getattr(q, name))
    p = moe.sort(wide[:0], 13)
    assert p.rows == 0 and not p.offsets.any() and not p.counts.any()


def test_rows_hold_any_routing():
    """fp8_moe_rows is enough for the worst routing and no more than the worst needs."""
    for slots, experts in ((1, 1), (1, 9), (5, 3), (128, 2), (129, 2), (300, 300), (1000, 64)):
        worst = 0
        for used in range(1, min(slots, experts) + 1):  # `used` experts with one slot each but the first
            first = slots - used + 1
            for extra in range(used):  # 1 .. used of them with one more
                n = [first - extra] + [2] * extra + [1] * (used - 1 - extra) if first > extra else [slots]
                worst = max(worst, sum(-(-v // 128) * 128 for v in n))
        assert worst <= fm.fp8_moe_rows(slots, 1, experts) <= worst + 127


def _within(got, ref, err, what):
    bad = (got.double() - ref).abs() > U[got.dtype] * ref.abs() + err
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance"


ROWS = [(1, 1, 1, 1, "random", B), (5, 2, 3, 7, "random", F), (200, 2, 8, 512, "dropped", B), (333, 8, 64, 1000, "random", B),
        (130, 3, 4, 2049, "one", F), (64, 9, 16, 4096, "dropped", B), (77, 12, 12, 130, "half", F), (40, 2, 6, 33, "none", B)]


@pytest.mark.parametrize("tokens,topk,experts,cols,kind,dt", ROWS)
def test_dispatch_combine_and_gradient(tokens, topk, experts, cols, kind, dt):
    need_gpu()
    e, w = _routing(tokens, topk, experts, 23, kind)
    p = moe.sort(e, experts)
    g = _gen(3)
    pad = 3  # strided inputs
    x = torch.randn(tokens, cols + pad, generator=g, device="cuda").to(dt)[:, :cols]
    ys = torch.randn(p.rows, cols + pad, generator=g, device="cuda").to(dt)[:, :cols]
    dy = torch.randn(tokens, cols + pad, generator=g, device="cuda").to(dt)[:, :cols]
    end = int(p.offsets[-1])
    ys[end:] = float("nan")  # nobody's rows
    slot, row = p.row_slot.long(), p.slot_row.long()
    for w_ in (None, w):
        wf = torch.ones_like(w) if w_ is None else w
        got = moe.dispatch(x, p, w_)
        src = x.double()[slot.clamp(min=0) // topk] * wf.double().reshape(-1)[slot.clamp(min=0)][:, None]
        ref = torch.where(slot[:, None] >= 0, src, 0.0)
        _within(got[:end], ref[:end], 0.0 if w_ is None else E32 * ref[:end].abs(), "dispatch")
        held = (row >= 0)[..., None]
        picked = torch.where(held, ys.double()[row.clamp(min=0)], 0.0) if p.rows else held.double().expand(-1, -1, cols)
        terms = picked * wf.double()[..., None]
        _within(moe.combine(ys, p, w_), terms.sum(1), (topk + 2) * E32 * terms.abs().sum(1), "combine")
        dys, dw = moe.combine_backward(dy, ys, p, w_)
        src = dy.double()[slot.clamp(min=0) // topk] * wf.double().reshape(-1)[slot.clamp(min=0)][:, None]
        ref = torch.where(slot[:, None] >= 0, src, 0.0)
        _within(dys[:end], ref[:end], 0.0 if w_ is None else E32 * ref[:end].abs(), "dys")
        dots = picked * dy.double()[:, None]
        _within(dw, dots.sum(2), (cols + 2) * E32 * dots.abs().sum(2), "dweights")
        assert not dw[row < 0].any()
    only_rows, none = moe.combine_backward(dy, None, p, w, dots=False)
    assert none is None and torch.equal(only_rows[:end], dys[:end])
    none, only_dots = moe.combine_backward(dy, ys, p, w, rows=False)
    assert none is None and torch.equal(only_dots, dw)


def test_rows_behind_the_last_segment_are_left_alone():
    need_gpu()
    e, w = _routing(150, 2, 6, 4)
    p = moe.sort(e, 6)
    end, cols = int(p.offsets[-1]), 256
    assert end < p.rows
    x = torch.randn(150, cols, device="cuda").bfloat16()
    buf = torch.full((p.rows, cols), 7.0, dtype=B, device="cuda")
    assert fm.fp8_moe_dispatch(x, fm.IN_BF16, 150, cols, cols, 2, w, p.slot_row, p.offsets, p.counts, 6, buf, p.rows, cols) == fm.OK
    assert (buf[end:] == 7).all() and torch.equal(buf[:end], moe.dispatch(x, p, w)[:end])
    buf.fill_(7.0)
    dw = torch.empty(150, 2, device="cuda")
    assert fm.fp8_moe_combine_backward(x, fm.IN_BF16, 150, cols, cols, x.new_zeros(p.rows, cols), cols, p.slot_row, p.offsets,
                                       p.counts, 6, 2, w, buf, p.rows, cols, dw) == fm.OK
    assert (buf[end:] == 7).all()
    q_row = torch.full((p.rows, cols), 0xAB, dtype=torch.uint8, device="cuda")
    q_col = torch.full((cols, p.rows), 0xAB, dtype=torch.uint8, device="cuda")
    s_row = torch.full((p.rows, 2), 7.0, device="cuda")
    s_col = torch.full((cols, p.rows // 128), 7.0, device="cuda")
    assert fm.fp8_moe_quantize(x, fm.IN_BF16, 150, cols, cols, p.row_slot, 2, w, p.offsets, 6, p.rows, fm.BLOCK_1x128, fm.E4M3,
                               fm.ROW_AND_COL, 0, q_row, cols, s_row, q_col, p.rows, s_col, None) == fm.OK
    assert (q_row[end:] == 0xAB).all() and (q_col[:, end:] == 0xAB).all()
    assert (s_row[end:] == 7).all() and (s_col[:, end // 128:] == 7).all() and (s_row[:end] != 7).all()
    c = torch.full((p.rows, 128), 7.0, device="cuda")
    wq = fm.quantize(torch.randn(6 * 128, cols, device="cuda"), fm.BLOCK_128x128, fm.E4M3)
    moe.gemm(q_row, fm.E4M3, s_row, wq.q_row.view(6, 128, cols), fm.E4M3, wq.s_row.view(6, 1, 2), fm.GEMM_BLOCK_1x128_128x128,
             p.offsets, c=c)
    assert (c[end:] == 7).all() and c[:end].isfinite().all()


CASTS = [(1, 1, 1, 16, "random", B), (200, 2, 8, 512, "dropped", B), (150, 3, 5, 1000, "half", F), (130, 2, 3, 136, "one", B),
         (64, 1, 70, 384, "random", F), (64, 1, 70, 384, "random", B), (2500, 4, 9, 1408, "dropped", B)]


@pytest.mark.parametrize("tokens,topk,experts,cols,kind,dt", CASTS)
@pytest.mark.parametrize("recipe", [fm.BLOCK_1x128, fm.MX_1x32, fm.MX_1x32_OCP])
@pytest.mark.parametrize("fmt", [fm.E4M3, fm.E5M2])
def test_quantize_matches_the_oracle(tokens, topk, experts, cols, kind, dt, recipe, fmt):
    need_gpu()
    e, w = _routing(tokens, topk, experts, 31, kind)
    p = moe.sort(e, experts)
    end = int(p.offsets[-1])
    x = (torch.randn(tokens, cols, generator=_gen(9), device="cuda") * torch.exp(torch.randn(1, cols, generator=_gen(8), device="cuda")))
    x[0, 0] = 0.0
    x = x.to(dt)
    slot = p.row_slot.long()[:end]
    for w_ in (None, w):
        rows = x.float()[slot.clamp(min=0) // topk]
        if w_ is not None:
            rows = rows * w.reshape(-1)[slot.clamp(min=0)][:, None]
        rows = host(torch.where(slot[:, None] >= 0, rows, 0.0))
        for orient in (fm.ROW, fm.COL, fm.ROW_AND_COL):
            q = moe.quantize(x, p, recipe, fmt, orient, weights=w_)
            for codes, scales, m in ((q.q_row, q.s_row, rows), (q.q_col, q.s_col, rows.T)):
                if codes is None:
                    continue
                lines, n = m.shape
                codes = host(codes)[:lines, :n]
                if recipe == fm.BLOCK_1x128:
                    oc, og, _ = oracle.quantize_blocks(FMT_NAME[fmt], np.ascontiguousarray(m), 1, 128)
                    assert same_f32(host(scales)[:lines, :og.shape[1]], og)
                else:
                    oc, og, _ = oracle.quantize_mx(FMT_NAME[fmt], np.ascontiguousarray(m), 1, 32,
                                                       "floor" if recipe == fm.MX_1x32_OCP else "ceil")
                    assert np.array_equal(host(scales)[:lines, :og.shape[1]], og)
                assert np.array_equal(codes, oc)


def test_quantize_sorted_rows_and_nonfinite():
    """gather=False reads the rows as they are; NaN and Inf mark their own blocks."""
    need_gpu()
    e, w = _routing(300, 2, 4, 2)
    p = moe.sort(e, 4)
    x = torch.randn(300, 256, device="cuda").bfloat16()
    a, b = moe.quantize(x, p, fm.BLOCK_1x128, fm.E4M3, fm.ROW_AND_COL), None
    xs = moe.dispatch(x, p)
    end = int(p.offsets[-1])
    xs[end:] = float("nan")
    b = moe.quantize(xs, p, fm.BLOCK_1x128, fm.E4M3, fm.ROW_AND_COL, gather=False)
    assert torch.equal(a.q_row[:end], b.q_row[:end]) and torch.equal(a.s_row[:end], b.s_row[:end])
    assert torch.equal(a.q_col[:, :end], b.q_col[:, :end]) and torch.equal(a.s_col[:, :end // 128], b.s_col[:, :end // 128])
    x[7, 3], x[9, 200] = float("nan"), float("inf")
    xs = moe.dispatch(x, p)
    xs[end:] = 0.0
    for recipe in (fm.BLOCK_1x128, fm.MX_1x32, fm.MX_1x32_OCP):
        for w_ in (None, torch.ones_like(w)):
            for cols in (256, 232):  # whole tiles, and rows that end inside one
                count, ref = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
                q = moe.quantize(x[:, :cols], p, recipe, fm.E5M2, fm.ROW_AND_COL, weights=w_, nonfinite=count)
                f = fm.quantize(xs[:end, :cols], recipe, fm.E5M2, fm.ROW_AND_COL, nonfinite=ref)
                assert int(count) == int(ref) > 0
                n = f.s_col.shape[1]
                assert torch.equal(q.q_row[:end, :cols], f.q_row[:, :cols]) and torch.equal(q.q_col[:, :end], f.q_col[:, :end])
                assert torch.equal(q.s_row[:end], f.s_row) and torch.equal(q.s_col[:, :n], f.s_col)
    r = p.slot_row[7, 0]
    q = moe.quantize(x, p, fm.BLOCK_1x128, fm.E4M3, fm.ROW)
    assert int(q.q_row[r, 3]) == 0x7F and float(q.s_row[r, 0]) == 1.0


def _codes(shape, fmt, seed):
    """Finite codes [.., n] with rows a multiple of 16 bytes apart."""
    c = torch.randint(0, 256, shape, generator=_gen(seed), device="cuda", dtype=torch.int32)
    top = 0x7F if fmt == fm.E4M3 else 0x7C
    return torch.where((c & 0x7F) >= top, c & 0x80, c).to(torch.uint8)


def _scales(shape, mx, seed):
    g = _gen(seed)
    if mx:
        return torch.randint(120, 134, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    return torch.rand(shape, generator=g, device="cuda") + 0.25


PRODUCTS = [  # tokens, topk, experts, n, k, kind
    (1, 1, 1, 1, 16, "random"), (200, 2, 8, 256, 512, "random"), (300, 2, 3, 100, 144, "dropped"), (700, 1, 5, 513, 272, "half"),
    (90, 4, 40, 384, 1040, "random"), (600, 2, 2, 130, 4096, "one"), (1500, 2, 4, 1000, 640, "random"), (50, 2, 4, 64, 128, "none"),
]


@pytest.mark.parametrize("tokens,topk,experts,n,k,kind", PRODUCTS)
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("fa,fb,out", [(fm.E4M3, fm.E4M3, B), (fm.E5M2, fm.E4M3, F), (fm.E4M3, fm.E5M2, F), (fm.E5M2, fm.E5M2, B)])
def test_gemm_rows(tokens, topk, experts, n, k, kind, mx, fa, fb, out):
    need_gpu()
    p = moe.sort(_routing(tokens, topk, experts, 41, kind)[0], experts)
    off = host(p.offsets)
    per = 32 if mx else 128
    kb, nb = -(-k // per), n if mx else -(-n // 128)
    a, b = _codes((p.rows, k), fa, 1), _codes((experts, n, k), fb, 2)
    s_a, s_b = _scales((p.rows, kb), mx, 3), _scales((experts, nb, kb), mx, 4)
    a[off[-1]:] = 0x7F
    recipe = fm.GEMM_MX_1x32 if mx else fm.GEMM_BLOCK_1x128_128x128
    c = moe.gemm(a, fa, s_a, b, fb, s_b, recipe, p.offsets, out)
    # the same product with B's and its scales' rows of all experts interleaved
    bt, st = b.permute(1, 0, 2).contiguous().permute(1, 0, 2), s_b.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    ct = moe.gemm(a, fa, s_a, bt, fb, st, recipe, p.offsets, out)
    assert torch.equal(c[:off[-1]], ct[:off[-1]])
    for e in range(experts):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        want = fm.gemm(a[lo:hi], fa, s_a[lo:hi].contiguous(), b[e], fb, s_b[e].clone(), recipe, k, out)
        assert torch.equal(c[lo:hi], want), f"expert {e}"
    if experts <= 8 and off[-1]:
        lo, hi = off[experts - 1], off[experts]
        if lo < hi:
            _check_product(c[lo:hi], _values(a[lo:hi], fa, s_a[lo:hi], mx), _values(b[-1], fb, s_b[-1], mx, not mx))


@pytest.mark.parametrize("tokens,topk,experts,n,k", [(300, 2, 3, 1300, 1024), (900, 1, 2, 2100, 512), (130, 2, 5, 1030, 2048)])
@pytest.mark.parametrize("mx", [False, True])
def test_gemm_rows_of_whole_step_groups(tokens, topk, experts, n, k, mx):
    """K a multiple of 512: the column tiles start at different steps of K, so
    the sums are in another order than fp8_gemm_scaled's; the same in two calls."""
    need_gpu()
    p = moe.sort(_routing(tokens, topk, experts, 47)[0], experts)
    off = host(p.offsets)
    per = 32 if mx else 128
    kb, nb = k // per, n if mx else -(-n // 128)
    a, b = _codes((p.rows, k), fm.E5M2, 1), _codes((experts, n, k), fm.E4M3, 2)
    s_a, s_b = _scales((p.rows, kb), mx, 3), _scales((experts, nb, kb), mx, 4)
    recipe = fm.GEMM_MX_1x32 if mx else fm.GEMM_BLOCK_1x128_128x128
    c = moe.gemm(a, fm.E5M2, s_a, b, fm.E4M3, s_b, recipe, p.offsets, F)
    assert torch.equal(c[:off[-1]], moe.gemm(a, fm.E5M2, s_a, b, fm.E4M3, s_b, recipe, p.offsets, F)[:off[-1]])
    for e in range(experts):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            _check_product(c[lo:hi], _values(a[lo:hi], fm.E5M2, s_a[lo:hi], mx), _values(b[e], fm.E4M3, s_b[e], mx, not mx))


@pytest.mark.parametrize("tokens,topk,experts,n,k", [(4500, 2, 4, 2100, 400), (2600, 2, 3, 2180, 1024), (5000, 1, 2, 1700, 130 * 16)])
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("fa,fb,out", [(fm.E4M3, fm.E4M3, B), (fm.E5M2, fm.E4M3, F)])
def test_gemm_rows_of_many_tiles(tokens, topk, experts, n, k, mx, fa, fb, out):
    """More than 256 rows per expert and more tiles than run at once: the large
    tiles, in which segments end halfway."""
    need_gpu()
    p = moe.sort(_routing(tokens, topk, experts, 53)[0], experts)
    off = host(p.offsets)
    per = 32 if mx else 128
    kb, nb = -(-k // per), n if mx else -(-n // 128)
    a, b = _codes((p.rows, k), fa, 1), _codes((experts, n, k), fb, 2)
    s_a, s_b = _scales((p.rows, kb), mx, 3), _scales((experts, nb, kb), mx, 4)
    recipe = fm.GEMM_MX_1x32 if mx else fm.GEMM_BLOCK_1x128_128x128
    base = torch.full((p.rows + 128, n), 7.0, dtype=out, device="cuda")
    c = moe.gemm(a, fa, s_a, b, fb, s_b, recipe, p.offsets, c=base[:p.rows])
    for e in range(experts):
        lo, hi = off[e], off[e + 1]
        if k % 512:
            want = fm.gemm(a[lo:hi], fa, s_a[lo:hi].contiguous(), b[e], fb, s_b[e].clone(), recipe, k, out)
            assert torch.equal(c[lo:hi], want), f"expert {e}"
    _check_product(c[lo:hi], _values(a[lo:hi], fa, s_a[lo:hi], mx), _values(b[-1], fb, s_b[-1], mx, not mx))
    assert (base[off[-1]:] == 7).all()


def test_many_tiles_offsets_outside_the_buffers_are_clamped():
    """Whatever an offsets array holds, for a product in the large tiles."""
    need_gpu()
    rows, n, k, experts = 4096, 2200, 128, 4
    a, b = _codes((rows, k), fm.E4M3, 1), _codes((experts, n, k), fm.E4M3, 2)
    s_a, s_b = _scales((rows, 1), False, 3), _scales((experts, 18, 1), False, 4)
    base = torch.full((rows + 512, n), 7.0, device="cuda")
    off = torch.tensor([-5, 1601, 1 << 30, 130, 2000000000], dtype=torch.int32, device="cuda")
    moe.gemm(a, fm.E4M3, s_a, b, fm.E4M3, s_b, fm.GEMM_BLOCK_1x128_128x128, off, c=base[:rows])
    assert (base[rows:] == 7).all()
    want = [fm.gemm(a, fm.E4M3, s_a, b[e], fm.E4M3, s_b[e].clone(), fm.GEMM_BLOCK_1x128_128x128, k, F) for e in (0, 1, 3)]
    assert torch.equal(base[:128], want[0][:128])
    some = base[:rows] == want[0]
    for w in want[1:]:
        some |= base[:rows] == w
    assert some.all()


def test_gemm_of_nothing_is_zero():
    """K = 0 writes zeros to the segments' rows; no rows, nothing."""
    need_gpu()
    p = moe.sort(_routing(100, 1, 2, 5)[0], 2)
    end = int(p.offsets[-1])
    u8 = dict(dtype=torch.uint8, device="cuda")
    c = torch.full((p.rows, 40), 7.0, device="cuda")
    moe.gemm(torch.empty(p.rows, 0, **u8), 0, torch.empty(p.rows, 0, device="cuda"), torch.empty(2, 40, 0, **u8), 0,
             torch.empty(2, 1, 0, device="cuda"), fm.GEMM_BLOCK_1x128_128x128, p.offsets, c=c)
    assert not c[:end].any() and (c[end:] == 7).all()
    p = moe.sort(torch.empty(0, 2, dtype=torch.int64, device="cuda"), 3)
    q = moe.quantize(torch.empty(0, 128, dtype=B, device="cuda"), p, fm.BLOCK_1x128, fm.E4M3, fm.ROW_AND_COL)
    y = moe.gemm(q.q_row, 0, q.s_row, torch.zeros(3, 64, 128, **u8), 0, torch.ones(3, 1, 1, device="cuda"),
                 fm.GEMM_BLOCK_1x128_128x128, p.offsets)
    assert y.shape == (0, 64) and moe.combine(y, p).shape == (0, 64)
    g = moe.gemm_wgrad(q.q_col[:, :0], 0, q.s_col, q.q_col[:, :0], 0, q.s_col, fm.GEMM_BLOCK_1x128_1x128, p.offsets)
    assert g.shape == (3, 128, 128) and not g.any()


def _values(codes, fmt, scales, mx, tiles=False):
    v = codes.view(fm.TORCH_FP8[fmt]).float().double()
    s = 2.0 ** (scales.double() - 127) if mx else scales.double()
    if tiles:
        s = s.repeat_interleave(128, 0)[:v.shape[0]]
    return v * s.repeat_interleave(32 if mx else 128, 1)[:, :v.shape[1]]


def _check_product(c, a, b):
    ref, size = a @ b.t(), a.abs() @ b.abs().t()
    bad = (c.double() - ref).abs() > 2.0 ** -10 * size + (2.0 ** -8 * ref.abs() if c.dtype == B else 0.0)
    assert not bad.any()


@pytest.mark.parametrize("tokens,topk,experts,m,n,kind", PRODUCTS)
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("fa,fb,out", [(fm.E5M2, fm.E4M3, B), (fm.E4M3, fm.E4M3, F)])
def test_gemm_contract(tokens, topk, experts, m, n, kind, mx, fa, fb, out):
    need_gpu()
    p = moe.sort(_routing(tokens, topk, experts, 43, kind)[0], experts)
    off = host(p.offsets)
    per = 32 if mx else 128
    a, b = _codes((m, p.rows), fa, 1), _codes((n, p.rows), fb, 2)
    s_a, s_b = _scales((m, p.rows // per), mx, 3), _scales((n, p.rows // per), mx, 4)
    a[:, off[-1]:], b[:, off[-1]:] = 0x7F, 0x7F
    recipe = fm.GEMM_MX_1x32 if mx else fm.GEMM_BLOCK_1x128_1x128
    c = moe.gemm_wgrad(a, fa, s_a, b, fb, s_b, recipe, p.offsets, out)
    assert c.shape == (experts, m, n)
    wide = torch.full((experts, m + 1, n + 5), 7.0, dtype=out, device="cuda")
    moe.gemm_wgrad(a, fa, s_a, b, fb, s_b, recipe, p.offsets, c=wide[:, :m, :n])
    assert torch.equal(wide[:, :m, :n], c) and (wide[:, m] == 7).all() and (wide[:, :, n:] == 7).all()
    for e in range(experts):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            assert not c[e].any()
            continue
        if e > 8 and e < experts - 2:
            continue
        sl = slice(lo // per, hi // per)
        want = fm.gemm(a[:, lo:hi].contiguous(), fa, s_a[:, sl].contiguous(), b[:, lo:hi].contiguous(), fb,
                       s_b[:, sl].contiguous(), recipe, int(hi - lo), out)
        assert torch.equal(c[e], want), f"expert {e}"
        if e == experts - 1:
            _check_product(c[e], _values(a[:, lo:hi], fa, s_a[:, sl], mx), _values(b[:, lo:hi], fb, s_b[:, sl], mx))


@pytest.mark.parametrize("lens", [(1, 0, 9, 2, 0, 0, 5, 1, 1, 4, 0, 8), (1,), (0, 0, 0, 3, 0), (4, 5, 1)])
@pytest.mark.parametrize("mx", [False, True])
def test_gemm_contract_of_many_tiles(lens, mx):
    """Two tiles and more per workgroup, with contractions of every length after
    each other: none, one step, odd and even numbers, whole groups of four."""
    need_gpu()
    m, n, experts = 700, 520, 70
    seg = [lens[e % len(lens)] * 128 for e in range(experts)]
    off = np.concatenate([[0], np.cumsum(seg)])
    rows, per = int(off[-1]), 32 if mx else 128
    a, b = _codes((m, rows), fm.E5M2, 1), _codes((n, rows), fm.E4M3, 2)
    s_a, s_b = _scales((m, rows // per), mx, 3), _scales((n, rows // per), mx, 4)
    recipe = fm.GEMM_MX_1x32 if mx else fm.GEMM_BLOCK_1x128_1x128
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    c = moe.gemm_wgrad(a, fm.E5M2, s_a, b, fm.E4M3, s_b, recipe, offsets, F)
    for e in range(experts):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            assert not c[e].any()
            continue
        sl = slice(lo // per, hi // per)
        want = fm.gemm(a[:, lo:hi].contiguous(), fm.E5M2, s_a[:, sl].contiguous(), b[:, lo:hi].contiguous(), fm.E4M3,
                       s_b[:, sl].contiguous(), recipe, hi - lo, F)
        assert torch.equal(c[e], want), f"expert {e}"


@pytest.mark.parametrize("tokens", [300, 300000])
def test_products_of_the_most_experts(tokens):
    """1024 experts, a few slots each and a few hundred: both tile sizes and the
    contraction, on sampled experts."""
    need_gpu()
    experts, n, k = 1024, 130, 16
    p = moe.sort(_routing(tokens, 1, experts, 91)[0], experts)
    off = host(p.offsets)
    a, b = _codes((p.rows, k), fm.E4M3, 1), _codes((experts, n, k), fm.E4M3, 2)
    s_a, s_b = _scales((p.rows, 1), False, 3), _scales((experts, 2, 1), False, 4)
    c = moe.gemm(a, fm.E4M3, s_a, b, fm.E4M3, s_b, fm.GEMM_BLOCK_1x128_128x128, p.offsets, F)
    at, bt = _codes((40, p.rows), fm.E4M3, 5), _codes((24, p.rows), fm.E4M3, 6)
    s_at, s_bt = _scales((40, p.rows // 128), False, 7), _scales((24, p.rows // 128), False, 8)
    g = moe.gemm_wgrad(at, fm.E4M3, s_at, bt, fm.E4M3, s_bt, fm.GEMM_BLOCK_1x128_1x128, p.offsets, F)
    for e in (0, 1, 62, 63, 64, 65, 511, 512, 1000, 1022, 1023):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            assert not g[e].any()
            continue
        want = fm.gemm(a[lo:hi], fm.E4M3, s_a[lo:hi].contiguous(), b[e], fm.E4M3, s_b[e].clone(),
                       fm.GEMM_BLOCK_1x128_128x128, k, F)
        assert torch.equal(c[lo:hi], want), f"expert {e}"
        sl = slice(lo // 128, hi // 128)
        want = fm.gemm(at[:, lo:hi].contiguous(), fm.E4M3, s_at[:, sl].contiguous(), bt[:, lo:hi].contiguous(), fm.E4M3,
                       s_bt[:, sl].contiguous(), fm.GEMM_BLOCK_1x128_1x128, hi - lo, F)
        assert torch.equal(g[e], want), f"expert {e}"


def test_offsets_outside_the_buffers_are_clamped():
    """Whatever an offsets array holds, only the buffers' own rows are touched."""
    need_gpu()
    rows, n, k, experts = 512, 64, 128, 4
    a, b = _codes((rows, k), fm.E4M3, 1), _codes((experts, n, k), fm.E4M3, 2)
    s_a, s_b = _scales((rows, 1), False, 3), _scales((experts, 1, 1), False, 4)
    base = torch.full((rows + 512, n), 7.0, device="cuda")
    off = torch.tensor([-5, 200, 1 << 30, 130, 2000000000], dtype=torch.int32, device="cuda")
    moe.gemm(a, fm.E4M3, s_a, b, fm.E4M3, s_b, fm.GEMM_BLOCK_1x128_128x128, off, c=base[:rows])
    assert (base[rows:] == 7).all()
    # segments 0 .. 128, 128 .. 512, none (it would end before it begins), 128 .. 512: the
    # rows of two experts hold one's or the other's product
    want = [fm.gemm(a, fm.E4M3, s_a, b[e], fm.E4M3, s_b[e].clone(), fm.GEMM_BLOCK_1x128_128x128, k, F) for e in (0, 1, 3)]
    assert torch.equal(base[:128], want[0][:128])
    assert ((base[128:rows] == want[1][128:]) | (base[128:rows] == want[2][128:])).all()


def _layer_case(dt, seed=0):
    g = _gen(seed)
    tokens, topk, experts, d, h = 300, 2, 5, 256, 384
    e, w = _routing(tokens, topk, experts, 77, "dropped")
    x = torch.randn(tokens, d, generator=g, device="cuda").to(dt)
    return e, w, x, tokens, topk, experts, d, h


@pytest.mark.parametrize("recipe", [linear.Float8BlockScaling(), linear.MXFP8BlockScaling(fp8_format=linear.Format.HYBRID)])
@pytest.mark.parametrize("dt", [B, F])
def test_layer_matches_linear_per_expert(recipe, dt):
    """GroupedLinear gives each expert's tokens what Linear with that expert's
    weight gives them, forward and backward, bit for bit in y and dx (the
    products are the same), and dx of a gathered input is their sum."""
    need_gpu()
    e, w, x, tokens, topk, experts, d, h = _layer_case(dt)
    p = moe.sort(e, experts)
    layer = moe.GroupedLinear(experts, d, h, recipe, device="cuda", dtype=dt)
    xs = moe.dispatch(x, p).requires_grad_()
    dy = torch.randn(p.rows, h, generator=_gen(2), device="cuda").to(dt) * (p.row_slot >= 0)[:, None]
    y = layer(xs, p)
    y.backward(dy)
    off = host(p.offsets)
    for i in range(experts):
        lo, hi = off[i], off[i + 1]
        one = linear.Linear(d, h, recipe=recipe, device="cuda", dtype=dt)
        with torch.no_grad():
            one.weight.copy_(layer.weight[i])
        xi = xs.detach()[lo:hi].requires_grad_()
        yi = one(xi)
        yi.backward(dy[lo:hi])
        assert torch.equal(y[lo:hi], yi) and torch.equal(xs.grad[lo:hi], xi.grad)
        assert torch.equal(layer.weight.grad[i], one.weight.grad)
    layer.weight.grad = None
    xg = x.clone().requires_grad_()
    layer(xg, p, gather=True).backward(dy)
    assert torch.equal(xg.grad, moe.combine(xs.grad, p))


def test_dispatch_and_combine_gradients():
    """autograd through dispatch and combine against float64."""
    need_gpu()
    e, w, x, tokens, topk, experts, d, _ = _layer_case(F, 1)
    p = moe.sort(e, experts)
    xv, wv = x.clone().requires_grad_(), w.clone().requires_grad_()
    w2 = (w.flip(0) + 0.5).requires_grad_()
    dy = torch.randn(tokens, d, generator=_gen(6), device="cuda")
    moe.combine(torch.tanh(moe.dispatch(xv, p, wv)), p, w2).backward(dy)
    xr, wr, w2r = (t.detach().double().requires_grad_() for t in (xv, wv, w2))
    kept = (p.slot_row >= 0).double()
    y = (torch.tanh(xr[:, None] * wr[..., None]) * (w2r * kept)[..., None]).sum(1)
    y.backward(dy.double())
    for got, ref in ((xv.grad, xr.grad), (wv.grad, wr.grad), (w2.grad, w2r.grad)):
        # sums of at most d = 256 terms of size about 1
        assert ((got.double() - ref).abs() <= 400 * E32 * (1 + ref.abs().max())).all()


def test_run_of_the_operators_captured_and_replayed():
    """Norm, sort, grouped layers, combine and their backward, as a block of a
    model uses them: captured once, replayed with other inputs and routings
    between eager runs, each replay equal to the eager result bit for bit."""
    need_gpu()
    tokens, topk, experts, d, h = 256, 2, 6, 256, 512
    rec = linear.Float8BlockScaling()
    ln = norm.LayerNorm(d, device="cuda", dtype=F)
    up = moe.GroupedLinear(experts, d, h, rec, device="cuda")
    down = moe.GroupedLinear(experts, h, d, rec, device="cuda")
    params = [ln.weight, ln.bias, up.weight, down.weight]

    def block(x, e, w, dy):
        x, w = x.detach().requires_grad_(), w.detach().requires_grad_()
        plan = moe.sort(e, experts)
        hid = up(ln(x), plan, gather=True)
        y = x + moe.combine(down(torch.nn.functional.silu(hid), plan), plan, w)
        return (y.detach(),) + torch.autograd.grad(y, [x, w] + params, dy)

    def inputs(seed):
        e, w = _routing(tokens, topk, experts, seed, "dropped")
        g = _gen(seed)
        return (torch.randn(tokens, d, generator=g, device="cuda").bfloat16(), e, w,
                torch.randn(tokens, d, generator=g, device="cuda").bfloat16())

    static = inputs(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(*static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(*static)
    for seed in (2, 3, 4, 1):
        fresh = inputs(seed)
        want = block(*fresh)
        torch.cuda.synchronize()
        for s, f in zip(static, fresh):
            s.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), seed
        assert all(t.isfinite().all() for t in want)


def test_no_second_derivative():
    """The backward passes are kernels of their own: asking for their gradient
    raises instead of giving none."""
    need_gpu()
    e, w = _routing(40, 2, 3, 1)
    p = moe.sort(e, 3)
    x = torch.randn(40, 128, device="cuda", requires_grad=True)
    ln = norm.LayerNorm(128, device="cuda", dtype=F)
    for f in (lambda: moe.dispatch(x, p), lambda: moe.combine(moe.dispatch(x, p), p, w), lambda: ln(x)):
        g, = torch.autograd.grad(f().square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            g.sum().backward()


def test_side_stream():
    """On a stream of its own, as an argument and as the current one."""
    need_gpu()
    e, w = _routing(500, 4, 16, 3)
    x = torch.randn(500, 512, device="cuda").bfloat16()
    p = moe.sort(e, 16)
    want = moe.combine(moe.dispatch(x, p, w), p, w)
    torch.cuda.synchronize()
    for raw in (False, True):
        s = torch.cuda.Stream()
        arg = s.cuda_stream if raw else s
        q = moe.sort(e, 16, stream=arg)
        got = moe.combine(moe.dispatch(x, q, w, stream=arg), q, w, stream=arg)
        y, *_ = norm.layer_norm_forward(x, None, None, stream=arg)
        s.synchronize()
        assert torch.equal(got, want) and torch.equal(q.row_slot, p.row_slot)
        assert torch.equal(y, norm.layer_norm_forward(x)[0])


def test_offsets_past_32_bits():
    """Sorted buffers of more than 4 GiB: the last expert's rows lie behind 2^32
    bytes of codes, rows and products."""
    need_gpu()
    tokens, topk, experts, cols, n = 66000, 8, 3, 8192, 256
    e = torch.full((tokens, topk), 1, device="cuda")
    e[-100:] = 2
    e[0] = 0
    p = moe.sort(e, experts)
    last = int(p.offsets[2])
    assert last * cols > 1 << 32
    x = torch.randn(tokens, cols, generator=_gen(1), device="cuda").bfloat16()
    w = torch.rand(tokens, topk, generator=_gen(2), device="cuda")
    src = x[-100:].repeat_interleave(topk, 0)  # the last segment's rows
    q = moe.quantize(x, p, fm.BLOCK_1x128, fm.E4M3, fm.ROW_AND_COL)
    want = fm.quantize(src, fm.BLOCK_1x128, fm.E4M3, fm.ROW)
    assert torch.equal(q.q_row[last:last + 800], want.q_row) and torch.equal(q.s_row[last:last + 800], want.s_row)
    pad = torch.nn.functional.pad(src, (0, 0, 0, 96))
    want = fm.quantize(pad, fm.BLOCK_1x128, fm.E4M3, fm.COL)
    assert torch.equal(q.q_col[:, last:last + 896], want.q_col)
    assert torch.equal(q.s_col[:, last // 128:last // 128 + 7], want.s_col)
    wq = fm.quantize(torch.randn(experts * n, cols, generator=_gen(3), device="cuda"), fm.BLOCK_128x128, fm.E4M3)
    b, s_b = wq.q_row.view(experts, n, cols), wq.s_row.view(experts, 2, -1)
    c = moe.gemm(q.q_row, fm.E4M3, q.s_row, b, fm.E4M3, s_b, fm.GEMM_BLOCK_1x128_128x128, p.offsets)
    for rows in (slice(last, last + 800), slice(last - 256, last)):
        a = _values(q.q_row[rows], fm.E4M3, q.s_row[rows], False)
        _check_product(c[rows], a, _values(b[2 if rows.start == last else 1], fm.E4M3, s_b[2 if rows.start == last else 1], False, True))
    del q, wq, b, s_b, c
    xs = moe.dispatch(x, p)
    assert torch.equal(xs[last:last + 800], src) and torch.equal(xs[:topk], x[:1].expand(topk, -1))
    y = moe.combine(xs, p, w)
    ref = src.view(100, topk, cols).double() * w[-100:].double()[..., None]
    _within(y[-100:], ref.sum(1), (topk + 2) * E32 * ref.abs().sum(1), "combine")
    dys, dw = moe.combine_backward(x, xs, p, w)
    ref = (src.double() * w[-100:].reshape(-1, 1).double())
    _within(dys[last:last + 800], ref, E32 * ref.abs(), "dys")
    dots = x[-100:].double().square()
    _within(dw[-100:], dots.sum(1, keepdim=True).expand(-1, topk), (cols + 2) * E32 * dots.sum(1, keepdim=True), "dweights")


def test_refusals():
    need_gpu()
    e, w = _routing(100, 2, 4, 3)
    p = moe.sort(e, 4)
    x = torch.randn(100, 128, device="cuda").bfloat16()
    xs = moe.dispatch(x, p)
    a = torch.zeros(p.rows, 128, dtype=torch.uint8, device="cuda")
    b = torch.zeros(4, 128, 128, dtype=torch.uint8, device="cuda")
    sa, sb = torch.ones(p.rows, 1, device="cuda"), torch.ones(4, 1, 1, device="cuda")
    rec = fm.GEMM_BLOCK_1x128_128x128
    layer = moe.GroupedLinear(4, 128, 128, device="cuda")
    for bad in (lambda: moe.sort(e.float(), 4), lambda: moe.sort(e[:, 0], 4), lambda: moe.sort(e, 0), lambda: moe.sort(e, 1025),
                lambda: moe.sort(e.cpu(), 4), lambda: moe.sort(e.t(), 4), lambda: moe.sort(e[:, :0], 4),
                lambda: moe.dispatch(x[:99], p), lambda: moe.dispatch(x, p, w[:99]), lambda: moe.dispatch(x, p, w.double()),
                lambda: moe.dispatch(x.half(), p), lambda: moe.combine(xs[:128], p, w), lambda: moe.combine(xs.t(), p),
                lambda: moe.combine_backward(x, xs.float(), p, w), lambda: moe.combine_backward(x, None, p, w),
                lambda: moe.quantize(x, p, fm.TENSOR_CURRENT, fm.E4M3), lambda: moe.quantize(x, p, fm.BLOCK_128x128, fm.E4M3),
                lambda: moe.quantize(x, p, fm.CHANNEL, fm.E4M3), lambda: moe.quantize(x[:, :100], p, fm.BLOCK_1x128, 7),
                lambda: moe.quantize(x, p, fm.BLOCK_1x128, fm.E4M3, gather=False),
                lambda: moe.quantize(xs, p, fm.BLOCK_1x128, fm.E4M3, gather=False, weights=w),
                lambda: moe.quantize(x[:, 1:], p, fm.BLOCK_1x128, fm.E4M3),
                lambda: moe.gemm(a[:, :120], 0, sa, b, 0, sb, rec, p.offsets), lambda: moe.gemm(a, 0, sa, b[:3], 0, sb, rec, p.offsets),
                lambda: moe.gemm(a, 0, sa[:5], b, 0, sb, rec, p.offsets), lambda: moe.gemm(a, 0, sa, b, 0, sb[:, :, :0], rec, p.offsets),
                lambda: moe.gemm(a, 0, sa, b, 0, sb, fm.GEMM_TENSOR, p.offsets), lambda: moe.gemm(a, 0, sa, b, 0, sb, rec, p.offsets.long()),
                lambda: moe.gemm(a[:100], 0, sa, b, 0, sb, rec, p.offsets),
                lambda: moe.gemm(a, 0, sa, b, 0, sb, fm.GEMM_BLOCK_1x128_1x128, p.offsets),
                lambda: moe.gemm_wgrad(a.t().contiguous(), 0, sa, a.t().contiguous(), 0, sa, rec, p.offsets),
                lambda: moe.gemm_wgrad(a.t(), 0, sa, a.t(), 0, sa, fm.GEMM_BLOCK_1x128_1x128, p.offsets),
                lambda: moe.GroupedLinear(256, 128, 1 << 15), lambda: moe.GroupedLinear(1025, 128, 128),
                lambda: layer(xs, p), lambda: moe.GroupedLinear(4, 100, 128), lambda: moe.GroupedLinear(0, 128, 128),
                lambda: moe.GroupedLinear(3, 128, 128, linear.Float8BlockScaling(), device="cuda")(xs, p),
                lambda: moe.GroupedLinear(4, 128, 128, linear.Float8CurrentScaling(), device="cuda")(xs, p),
                lambda: moe.GroupedLinear(4, 128, 128, linear.Float8BlockScaling(), device="cuda")(x, p)):
        with pytest.raises(fm.Fp8Error):
            bad()
