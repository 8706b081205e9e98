"""GPU: the weighted combine of the experts' rows and its gradient against the
64-bit definitions of oracle/moe.py.

Tolerances.  A token's sum of k products and a residual in fp32 is off by at
most (k + 1) 2^-24 of the sum of the magnitudes; a bf16 output must be the
rounding of a value within that bound.  dy is one fp32 product rounded once: it must be
equal to numpy's.  dweights sums cols products in any order: cols 2^-24 of the
sum of the magnitudes."""
import numpy as np
import pytest

import oracle
from mxfp4_precision_numerics_amd import mx, synth
from oracle import moe
from gpu_util import bf16_bits_to_f64, dev, host, torch

pytestmark = pytest.mark.gpu


def values(shape, dtype, seed, scale=1.0):
    """(64-bit values, device tensor) representable in dtype."""
    tt = torch()
    x = tt.from_numpy((np.random.default_rng(seed).normal(size=shape) * scale).astype(np.float32)).to(dtype)
    return x.double().numpy(), x.cuda()


def placed(x, pad):
    """x with its rows pad elements further apart; odd pads also start off any
    16-byte boundary."""
    tt = torch()
    t, c = x.shape
    buf = tt.full((t * (c + pad) + 1,), float("nan"), dtype=x.dtype, device="cuda")
    view = buf[pad % 2:pad % 2 + t * (c + pad)].view(t, c + pad)[:, :c]
    view.copy_(x)
    return view


def slots_of(t, k, rows, seed):
    """Distinct slots, some assignments without one (-1 or past the rows)."""
    rng = np.random.default_rng(seed)
    slot = np.full(t * k, -1, dtype=np.int32)
    n = min(rows, t * k)
    slot[rng.permutation(t * k)[:n]] = rng.permutation(rows)[:n]
    gone = rng.random(t * k) < 0.1
    slot[gone] = rng.choice([-1, -2 ** 31, rows, 2 ** 31 - 1], size=int(gone.sum()))
    if t > 2:
        slot[k:2 * k] = -1                                 # a token that went nowhere
    return slot.reshape(t, k)


CASES = [
    # tokens, k, rows, cols, y dtype, out dtype, weights, residual, pad
    (1, 4, 4, 2880, "bf16", "bf16", True, False, 0),
    (1, 1, 1, 1, "f32", "f32", False, False, 0),
    (3, 2, 6, 7, "bf16", "f32", True, True, 1),
    (5, 8, 40, 96, "f32", "f32", True, True, 4),
    (9, 3, 20, 1001, "f32", "bf16", True, False, 0),
    (33, 4, 140, 512, "bf16", "bf16", False, True, 8),
    (17, 4, 68, 513, "bf16", "bf16", True, True, 3),
    (40, 9, 360, 136, "f32", "f32", False, False, 0),
    (7, 6, 0, 64, "bf16", "bf16", True, True, 0),
    (64, 5, 300, 2048, "f32", "bf16", True, True, 8),
    (300, 4, 1200, 2880, "bf16", "f32", True, False, 0),
    (21, 2, 42, 8200, "bf16", "bf16", True, False, 0),
]


def types(case):
    tt = torch()
    return tuple(tt.bfloat16 if v == "bf16" else tt.float32 for v in case[4:6])


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_combine(case):
    t, k, rows, cols, _, _, with_w, with_res, pad = case
    tt = torch()
    yt, ot = types(case)
    y64, y = values((rows, cols), yt, 1)
    slot = slots_of(t, k, rows, 2)
    w = np.random.default_rng(3).normal(size=(t, k)).astype(np.float32) if with_w else None
    r64, res = values((t, cols), ot, 4) if with_res else (None, None)
    out = placed(tt.zeros((t, cols), dtype=ot, device="cuda"), pad) if pad else None
    got = mx.combine(placed(y, pad), dev(slot), None if w is None else dev(w),
                     residual=None if res is None else placed(res, pad), out=out, out_dtype=ot)
    assert got.dtype == ot
    want = moe.combine(y64, slot, w, r64)
    size = moe.combine(np.abs(y64), slot, np.ones((t, k)) if w is None else np.abs(w), None if r64 is None else np.abs(r64))
    tol = (k + 1) * 2.0 ** -24 * size + 1e-38
    low, high = want - tol, want + tol
    if ot == tt.bfloat16:                                  # rounding keeps the order
        low, high = (bf16_bits_to_f64(oracle.round_bf16_bits(v)) for v in (low, high))
    value = got.double().cpu().numpy()
    assert ((low <= value) & (value <= high)).all()
    if with_res:                                           # the residual updated in place
        mx.combine(y, dev(slot), None if w is None else dev(w), residual=res, out=res)
        assert tt.equal(res, got)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
@pytest.mark.parametrize("cleared", [True, False])
def test_combine_gradient(case, cleared):
    t, k, rows, cols, _, _, with_w, _, pad = case
    tt = torch()
    yt, dt = types(case)
    y64, y = values((rows, cols), yt, 5)
    d64, dout = values((t, cols), dt, 6, 1e-3)
    slot = slots_of(t, k, rows, 7)
    w = np.random.default_rng(8).normal(size=(t, k)).astype(np.float32) if with_w else None
    named = (slot >= 0) & (slot < rows)
    used = int(slot[named].max()) + 1 if named.any() else 0
    dy = placed(tt.full((rows, cols), 7.0, dtype=yt, device="cuda"), pad) if rows else None
    dy, dw = mx.combine_bwd(placed(dout, pad), placed(y, pad), dev(slot), None if w is None else dev(w), dy=dy,
                            used_rows=dev(np.array([used], np.int32)) if cleared else None)
    want_dy, want_dw = moe.combine_bwd(d64, y64, slot, w)
    size = moe.combine_bwd(np.abs(d64), np.abs(y64), slot)[1]
    assert (np.abs(host(dw) - want_dw) <= cols * 2.0 ** -24 * size + 1e-38).all()
    # one product, rounded once; rows no slot names are left alone, or zero from the used ones on
    expect = np.full((rows, cols), 7.0, dtype=np.float32)
    for i, j in zip(*np.nonzero(named)):
        expect[slot[i, j]] = np.float32(1.0 if w is None else w[i, j]) * d64[i].astype(np.float32)
    expect = tt.from_numpy(expect).to(yt)
    if cleared:
        expect[used:] = 0
    assert tt.equal(dy.cpu(), expect)
    if rows:                                               # without dweights y is not read
        again, none = mx.combine_bwd(dout, y, dev(slot), None if w is None else dev(w), need_dweights=False,
                                     dy=tt.full((rows, cols), 7.0, dtype=yt, device="cuda"))
        assert none is None
        mine = tt.from_numpy(~np.isnan(want_dy[:, 0]))
        assert tt.equal(again.cpu()[mine], expect[mine])


# more rows a token than a wave reads at once, over columns that leave its last piece ragged or only one to three of
# its lanes with a piece (8 bf16 or 4 fp32 elements each, 64 lanes)
MANY = ([(k, cols, "bf16") for k in (5, 8, 9, 17) for cols in (1, 7, 8, 24, 513, 520, 1001, 2056)] +
        [(k, cols, "f32") for k in (5, 8, 9, 17) for cols in (1, 3, 4, 12, 257, 260, 1001, 1028)])


@pytest.mark.parametrize("k,cols,dtype", MANY)
@pytest.mark.parametrize("residual", [False, True])
def test_many_rows_a_token(k, cols, dtype, residual):
    rows = 13 * k - (9 if residual else 0)
    out = {"bf16": "f32", "f32": "bf16"}[dtype] if residual else dtype
    case = (13, k, rows, cols, dtype, out, k != 9, residual, cols % 3)
    test_combine(case)
    test_combine_gradient(case, cleared=residual)


def test_rows_that_no_token_names_do_not_matter():
    tt = torch()
    y = tt.randn((8, 64), device="cuda", generator=tt.Generator("cuda").manual_seed(1))
    y[0] = float("nan")
    y[7] = float("inf")
    slot = np.array([[1, -1], [-1, -1], [8, 6]], dtype=np.int32)
    out = host(mx.combine(y, dev(slot)))
    assert np.array_equal(out[0], host(y[1])) and not out[1].any() and np.array_equal(out[2], host(y[6]))
    # a weight of 0 is a factor like any other: 0 * nan is nan
    out = host(mx.combine(y, dev(np.array([[0]], np.int32)), tt.zeros((1, 1), device="cuda")))
    assert np.isnan(out).all()


@pytest.mark.parametrize("cols", [96, 2880, 1001])
def test_gradient_in_place_of_y(cols):
    tt = torch()
    _, y = values((420, cols), tt.bfloat16, 20)
    _, dout = values((100, cols), tt.bfloat16, 21)
    slot = dev(slots_of(100, 4, 400, 22))
    w = dev(np.random.default_rng(23).normal(size=(100, 4)).astype(np.float32))
    used = dev(np.array([400], np.int32))
    named = host(slot)[(host(slot) >= 0) & (host(slot) < 400)]
    dy, dw = mx.combine_bwd(dout, y, slot, w, used_rows=used)
    same, dw2 = mx.combine_bwd(dout, y, slot, w, used_rows=used, dy=y)
    assert same is y and tt.equal(dw, dw2) and tt.equal(y[named], dy[named]) and not y[400:].any()


def test_no_tokens():
    tt = torch()
    y = tt.ones((6, 40), device="cuda")
    slot = tt.zeros((0, 4), dtype=tt.int32, device="cuda")
    assert mx.combine(y, slot).shape == (0, 40)
    dy, dw = mx.combine_bwd(tt.zeros((0, 40), device="cuda"), y, slot, used_rows=dev(np.array([2], np.int32)),
                            dy=tt.full((6, 40), 7.0, device="cuda"))
    assert dw.shape == (0, 4) and (dy[:2] == 7.0).all() and not dy[2:].any()


def test_gradient_of_the_token_gather():
    """weights None sums the gradients that the experts' copies of a token
    send back; against the plan that gathered them."""
    tt = torch()
    rng = np.random.default_rng(9)
    ids = np.stack([rng.permutation(32)[:4] for _ in range(200)]).astype(np.int32)
    offsets, row_index, slot = mx.route_plan(dev(ids), 32)
    d64, dx = values((800, 256), tt.float32, 10)
    want = np.zeros((200, 256))
    np.add.at(want, host(row_index), d64)
    assert np.allclose(host(mx.combine(dx, slot)), want, rtol=0, atol=5 * 2.0 ** -24 * 20)


def test_full_size_step():
    """16384 tokens, top 4 of 32 experts, 2880 columns: every row against a
    vectorised 64-bit form."""
    tt = torch()
    gen = tt.Generator("cuda").manual_seed(2)
    t, k, d = 16384, 4, 2880
    counts = synth.zipf_counts()
    # expert e's rows are consecutive tokens; slots of a token in expert order
    token = tt.from_numpy(synth.routing_row_index(counts)).cuda().long()
    order = tt.sort(token, stable=True).indices
    slot = order.view(t, k).to(tt.int32).contiguous()
    y = tt.randn((t * k, d), device="cuda", generator=gen).to(tt.bfloat16)
    w = tt.rand((t, k), device="cuda", generator=gen)
    dout = (1e-3 * tt.randn((t, d), device="cuda", generator=gen)).to(tt.bfloat16)
    out = mx.combine(y, slot, w, out_dtype=tt.float32)
    dy, dw = mx.combine_bwd(dout, y, slot, w)
    for a in range(0, t, 2048):
        s = slot[a:a + 2048].long()
        rows, ww, g = y[s].double(), w[a:a + 2048].double()[:, :, None], dout[a:a + 2048].double()[:, None, :]
        assert ((out[a:a + 2048] - (ww * rows).sum(1)).abs() <= 5 * 2.0 ** -24 * (ww * rows).abs().sum(1)).all()
        assert tt.equal(dy[s], (w[a:a + 2048][:, :, None] * dout[a:a + 2048].float()[:, None, :]).to(tt.bfloat16))
        assert ((dw[a:a + 2048] - (g * rows).sum(2)).abs() <= d * 2.0 ** -24 * (g * rows).abs().sum(2)).all()


def test_offsets_past_32_bits():
    """Rows whose byte offsets pass 4 GiB."""
    tt = torch()
    rows, cols = 600_000, 8192                             # 9.8 GB in bf16
    y = tt.empty((rows, cols), dtype=tt.bfloat16, device="cuda")
    at = [0, 131_071, 131_072, 262_143, 262_144, 300_001, rows - 1]
    for i, r in enumerate(at):
        y[r] = i + 1
    slot = dev(np.array([at], dtype=np.int32))
    assert (host(mx.combine(y, slot, out_dtype=tt.float32)) == sum(range(1, len(at) + 1))).all()
    dout = tt.ones((1, cols), dtype=tt.bfloat16, device="cuda")
    w = dev(np.arange(2, 2 + len(at), dtype=np.float32)[None])
    dy, dw = mx.combine_bwd(dout, y, slot, w)
    assert host(dw)[0].tolist() == [cols * (i + 1.0) for i in range(len(at))]
    for i, r in enumerate(at):
        assert (dy[r] == i + 2).all()


def test_most_pieces():
    """2^25 pieces of 1 KiB, one a token; one more is refused."""
    tt = torch()
    t = 2 ** 25
    y = tt.arange(1, 1001, dtype=tt.float32, device="cuda").view(1000, 1)
    slot = (tt.arange(t, dtype=tt.int32, device="cuda") % 1001).view(t, 1)     # (1000 names no row)
    out = mx.combine(y, slot)
    assert tt.equal(out.view(-1), tt.where(slot.view(-1) < 1000, slot.view(-1) + 1, 0).float())
    with pytest.raises(mx.MXError):
        mx.combine(y, tt.zeros((t + 1, 1), dtype=tt.int32, device="cuda"))


def test_most_tokens_of_the_gradient():
    """2^23 - 1 tokens, with rows to clear; one more is refused."""
    tt = torch()
    t, rows = 2 ** 23 - 1, 2 ** 23 + 5000
    slot = (tt.arange(t, dtype=tt.int32, device="cuda") + 7).view(t, 1)
    y = (tt.arange(rows, dtype=tt.float32, device="cuda") % 1024).view(rows, 1)
    dout = (tt.arange(t, dtype=tt.float32, device="cuda") % 31).view(t, 1)
    used = dev(np.array([t + 7 - 3], np.int32))            # the last three slots count as none
    dy, dw = mx.combine_bwd(dout, y, slot, used_rows=used, dy=tt.full_like(y, 7.0))
    want = tt.full_like(y, 7.0)
    want[7:7 + t] = dout
    want[t + 4:] = 0
    assert tt.equal(dy, want)
    want = dout * y[7:7 + t]
    want[-3:] = 0
    assert tt.equal(dw, want)
    with pytest.raises(mx.MXError):
        mx.combine_bwd(tt.zeros((t + 1, 1), device="cuda"), y, tt.zeros((t + 1, 1), dtype=tt.int32, device="cuda"))


def test_other_stream_and_graph():
    tt = torch()
    gen = tt.Generator("cuda").manual_seed(8)
    y = tt.randn((400, 320), device="cuda", generator=gen)
    dout = tt.randn((100, 320), device="cuda", generator=gen)
    w = tt.rand((100, 4), device="cuda", generator=gen)
    slot = dev(slots_of(100, 4, 400, 1))
    used = dev(np.array([390], np.int32))
    dy = tt.zeros_like(y)
    tt.cuda.synchronize()

    def step(dy):
        return (mx.combine(y, slot, w),) + mx.combine_bwd(dout, y, slot, w, used_rows=used, dy=dy)

    side = tt.cuda.Stream()
    with tt.cuda.stream(side):
        got = step(dy)
    side.synchronize()
    for a, b in zip(got, step(tt.zeros_like(y))):
        assert tt.equal(a, b)
    graph = tt.cuda.CUDAGraph()
    with tt.cuda.graph(graph):
        held = step(dy)
    for n in range(3):
        y.copy_(tt.randn((400, 320), device="cuda", generator=gen))
        w.copy_(tt.rand((100, 4), device="cuda", generator=gen))
        graph.replay()
        tt.cuda.synchronize()
        for a, b in zip(held, step(tt.zeros_like(y))):
            assert tt.equal(a, b), n


def test_slots_at_or_past_the_used_rows_count_as_none():
    tt = torch()
    y = tt.ones((10, 64), device="cuda")
    dout = tt.ones((3, 64), device="cuda")
    slot = dev(np.array([[0, 9], [6, 7], [3, -1]], dtype=np.int32))
    dy, dw = mx.combine_bwd(dout, y, slot, used_rows=dev(np.array([7], np.int32)))
    assert host(dw).tolist() == [[64.0, 0.0], [64.0, 0.0], [64.0, 0.0]]
    assert not dy[7:].any() and (dy[[0, 3, 6]] == 1.0).all()
    dy, dw = mx.combine_bwd(dout, y, slot, used_rows=dev(np.array([-5], np.int32)))
    assert not dy.any() and not dw.any()


def test_refusals():
    tt = torch()
    y = tt.zeros((8, 64), device="cuda")
    slot = tt.zeros((2, 4), dtype=tt.int32, device="cuda")
    w = tt.zeros((2, 4), device="cuda")
    with pytest.raises(ValueError):
        mx.combine(y.cpu(), slot)
    with pytest.raises(TypeError):
        mx.combine(y.half(), slot)
    with pytest.raises(TypeError):
        mx.combine(y, slot.long())
    with pytest.raises(ValueError):
        mx.combine(y, slot, w[:1])
    with pytest.raises(TypeError):
        mx.combine(y, slot, w.bfloat16())
    with pytest.raises(TypeError):
        mx.combine(y, slot, residual=tt.zeros((2, 64), dtype=tt.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        mx.combine(y, slot, out=tt.zeros((3, 64), device="cuda"))
    with pytest.raises(ValueError):
        mx.combine(y.t(), slot)
    with pytest.raises(ValueError):
        mx.combine_bwd(tt.zeros((2, 63), device="cuda"), y, slot)
    with pytest.raises(ValueError):
        mx.combine_bwd(tt.zeros((2, 64), device="cuda"), y, slot, used_rows=tt.zeros(1, device="cuda"))
    with pytest.raises(TypeError):
        mx.combine_bwd(tt.zeros((2, 64), device="cuda"), y, slot, dy=tt.zeros((8, 64), dtype=tt.bfloat16, device="cuda"))
