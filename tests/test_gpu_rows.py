"""The row operators on the GPU (moe_permute, moe_unpermute and their gradients)
against oracle/rows.py in float64, on the routing that moe_route_static computes.

Tolerances, with u the unit roundoff 2^-24 of fp32 and e the type's half step
(bf16 2^-8 relative to the value at most, fp16 2^-11, fp32 2^-24), `tiny` half the
type's smallest subnormal:
  copies          bitwise
  sums over slots k fused multiply-adds: k * u * sum |w r|, then one rounding
  drows           one fp32 product, one rounding
  dw              each thread adds at most `chain` products, five shuffles and
                  eight warps: (chain + 13) * u * sum |d r|
(1.01 covers the second-order terms.)"""
import numpy as np
import pytest
import torch

import moe_expert_ffn_permute_b200 as moe
from oracle import rows as O

from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}
U = 2.0 ** -24


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _route(T, k, E, masked, g):
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    if masked:
        ids[torch.rand(T, k, generator=g, device="cuda") < masked] = -1
    ids = ids.contiguous()
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, offsets, perm, inv = i32(E), i32(E + 1), i32(T * k), i32(T * k)
    moe.moe_route_static(ids, T, k, E, counts, offsets, perm, inv)
    return inv.reshape(T, k), offsets


def _np(t):
    return t.double().cpu().numpy()


def _close(got, want, tol):
    got = _np(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


# Rows of one vector, of odd vector counts, of more than a block's threads; one
# token; more slots than a group of eight; every slot masked.
SIZES = [("bf16", 1, 8, 1, 1, 0.0), ("bf16", 1, 7168, 8, 32, 0.0), ("fp16", 3, 24, 2, 4, 0.3),
         ("fp32", 17, 12, 3, 5, 0.2), ("bf16", 300, 520, 4, 64, 0.1), ("fp32", 297, 1544, 9, 16, 0.5),
         ("fp16", 37, 4104, 6, 48, 0.0), ("bf16", 64, 256, 17, 32, 0.0), ("bf16", 5, 64, 2, 8, 1.1),
         ("fp32", 513, 4, 1, 1, 0.4), ("fp16", 400, 8, 8, 256, 0.05)]
IDS = [f"{d}-T{T}-H{H}-k{k}-E{E}-m{m}" for d, T, H, k, E, m in SIZES]


@pytest.mark.parametrize("dtype,T,H,k,E,masked", SIZES, ids=IDS)
def test_permute_and_its_gradient(dtype, T, H, k, E, masked):
    ensure_built()
    g = _gen(T * 131 + H)
    inv, _ = _route(T, k, E, masked, g)
    x = torch.randn(T, H, generator=g, device="cuda").to(DT[dtype])
    rows = torch.full((T * k, H), 7.0, dtype=DT[dtype], device="cuda")
    moe.moe_permute(x, T, H * x.element_size(), k, inv, rows)
    want = O.permute(_np(x), inv.cpu().numpy(), np.full((T * k, H), 7.0))
    np.testing.assert_array_equal(_np(rows), want)

    drows = torch.randn(T * k, H, generator=g, device="cuda").to(DT[dtype])
    n = int((inv >= 0).sum())
    drows[n:] = float("nan")                         # rows no slot names are not read
    dx = torch.full((T, H), float("nan"), dtype=DT[dtype], device="cuda")
    moe.moe_permute_backward(drows, dtype, T, H, k, inv, dx)
    d, iv = _np(drows), inv.cpu().numpy()
    want = O.unpermute(d, iv, np.ones((T, k)))
    mag = O.unpermute(np.abs(d), iv, np.ones((T, k)))
    _close(dx, want, 1.01 * (k * U * mag + HALF[dtype] * np.abs(want)) + TINY[dtype])


@pytest.mark.parametrize("dtype,T,H,k,E,masked", SIZES, ids=IDS)
def test_unpermute_and_its_gradient(dtype, T, H, k, E, masked):
    ensure_built()
    g = _gen(T * 137 + H)
    inv, _ = _route(T, k, E, masked, g)
    rows = torch.randn(T * k, H, generator=g, device="cuda").to(DT[dtype])
    n = int((inv >= 0).sum())
    rows[n:] = float("nan")
    w = torch.randn(T, k, generator=g, device="cuda")
    w[inv < 0] = float("nan")                        # nor are the weights of masked slots
    out = torch.full((T, H), float("nan"), dtype=DT[dtype], device="cuda")
    moe.moe_unpermute(rows, dtype, T, H, k, inv, w, out)
    r, iv, wn = _np(rows), inv.cpu().numpy(), _np(w)
    want, mag = O.unpermute(r, iv, wn), O.unpermute(np.abs(r), iv, np.abs(wn))
    _close(out, want, 1.01 * (k * U * mag + HALF[dtype] * np.abs(want)) + TINY[dtype])

    dout = torch.randn(T, H, generator=g, device="cuda").to(DT[dtype])
    drows = torch.full((T * k, H), 7.0, dtype=DT[dtype], device="cuda")
    dw = torch.full((T, k), float("nan"), device="cuda")
    moe.moe_unpermute_backward(dout, rows, dtype, T, H, k, inv, w, drows, dw)
    dn = _np(dout)
    want_r, want_w = O.unpermute_backward(dn, r, iv, wn, np.full((T * k, H), 7.0))
    tol = 1.01 * (HALF[dtype] + U) * np.abs(want_r) + TINY[dtype]
    tol[n:] = 0
    _close(drows, want_r, tol)
    _, mag_w = O.unpermute_backward(np.abs(dn), np.abs(r), iv, wn, np.zeros((T * k, H)))
    per = 4 if dtype == "fp32" else 8
    chain = per * -(-(H // per) // 32)     # at least a warp shares a row
    _close(dw, want_w, 1.01 * (chain + 13) * U * mag_w + 2.0 ** -140)

    # Either gradient alone is the same; without dw the rows are not needed.
    only_r, only_w = torch.full_like(drows, 7.0), torch.empty_like(dw)
    moe.moe_unpermute_backward(dout, None, dtype, T, H, k, inv, w, only_r, None)
    moe.moe_unpermute_backward(dout, rows, dtype, T, H, k, inv, w, None, only_w)
    assert torch.equal(only_r, drows) and torch.equal(only_w, dw)


@pytest.mark.parametrize("row_bytes", [4, 12, 16, 20, 224, 256])
def test_permute_of_byte_rows(row_bytes):
    """Codes and scale bytes: rows that are not whole 16-byte vectors."""
    ensure_built()
    g = _gen(row_bytes)
    T, k, E = 33, 3, 8
    inv, _ = _route(T, k, E, 0.2, g)
    x = torch.randint(0, 256, (T, row_bytes), generator=g, device="cuda", dtype=torch.uint8)
    rows = torch.zeros(T * k, row_bytes, dtype=torch.uint8, device="cuda")
    moe.moe_permute(x, T, row_bytes, k, inv, rows)
    want = O.permute(x.cpu().numpy(), inv.cpu().numpy(), np.zeros((T * k, row_bytes), np.uint8))
    np.testing.assert_array_equal(rows.cpu().numpy(), want)


def test_infinities_and_zero_weights_follow_ieee():
    ensure_built()
    inv = torch.tensor([[0, 1], [2, -1]], dtype=torch.int32, device="cuda")
    rows = torch.zeros(4, 8, device="cuda")
    rows[0], rows[1], rows[2] = float("inf"), 1.0, float("inf")
    w = torch.tensor([[1.0, 2.0], [0.0, 5.0]], device="cuda")
    out = torch.empty(2, 8, device="cuda")
    moe.moe_unpermute(rows, "fp32", 2, 8, 2, inv, w, out)
    assert torch.isinf(out[0]).all() and torch.isnan(out[1]).all()    # 0 * inf
    rows = torch.full((4, 8), 60000.0, device="cuda").half()
    out = torch.empty(2, 8, dtype=torch.float16, device="cuda")
    moe.moe_unpermute(rows, "fp16", 2, 8, 2, inv, w, out)
    assert torch.isinf(out[0]).all() and (out[1] == 0).all()          # overflow of the type


def test_positions_out_of_range_are_skipped():
    ensure_built()
    T, H, k = 4, 64, 2
    inv = torch.tensor([[0, 8], [1, -7], [2, 1 << 30], [3, -(1 << 31)]], dtype=torch.int32,
                       device="cuda")
    x = torch.arange(T * H, device="cuda", dtype=torch.float32).reshape(T, H)
    rows = torch.full((T * k, H), -1.0, device="cuda")
    moe.moe_permute(x, T, H * 4, k, inv, rows)
    assert torch.equal(rows[:4], x) and (rows[4:] == -1).all()
    dx = torch.empty(T, H, device="cuda")
    moe.moe_permute_backward(rows, "fp32", T, H, k, inv, dx)
    assert torch.equal(dx, x)
    dw = torch.full((T, k), 9.0, device="cuda")
    ones = torch.ones(T, k, device="cuda")
    moe.moe_unpermute_backward(x, rows, "fp32", T, H, k, inv, ones, None, dw)
    assert (dw[:, 1] == 0).all() and (dw[1:, 0] > 0).all()


def test_offsets_past_32_bits():
    """Rows whose byte offsets (and, in bf16, element offsets) pass 2^31 and 2^32."""
    ensure_built()
    T, H, k = 300, 8192, 1024           # 307,200 rows of 16 KB: 5 GB
    S = T * k
    rows = torch.zeros(S, H, dtype=torch.bfloat16, device="cuda")
    pos = torch.randperm(S, generator=_gen(1), device="cuda").to(torch.int32).reshape(T, k)
    inv = pos.contiguous()
    x = torch.randint(-8, 8, (T, H), generator=_gen(2), device="cuda").to(torch.bfloat16)
    moe.moe_permute(x, T, H * 2, k, inv, rows)
    flat = inv.reshape(-1).long()
    for t in (0, 7, T - 1):
        assert torch.equal(rows[inv[t].long()], x[t].expand(k, H))
    assert torch.equal(rows[flat[-5:]], x[-1].expand(5, H))
    dx = torch.empty_like(x)
    moe.moe_permute_backward(rows, "bf16", T, H, k, inv, dx)
    assert torch.equal(dx, (x.float() * k).to(torch.bfloat16))    # whole numbers: exact sums
    dw = torch.empty(T, k, device="cuda")
    moe.moe_unpermute_backward(x, rows, "bf16", T, H, k, inv, torch.ones_like(dw), None, dw)
    assert torch.equal(dw, (x.float() * x.float()).sum(1, keepdim=True).expand(T, k))


def test_gradients_against_differences():
    """<dout, out> is linear in rows and in w: differences along a random direction."""
    ensure_built()
    T, H, k, E = 23, 192, 3, 8
    g = _gen(5)
    inv, _ = _route(T, k, E, 0.2, g)
    rows, drow = (torch.randn(T * k, H, generator=g, device="cuda") for _ in range(2))
    w, dwt = (torch.randn(T, k, generator=g, device="cuda") for _ in range(2))
    dout = torch.randn(T, H, generator=g, device="cuda")
    drows, dw = torch.zeros_like(rows), torch.empty_like(w)
    moe.moe_unpermute_backward(dout, rows, "fp32", T, H, k, inv, w, drows, dw)

    def value(r, v):
        out = torch.empty(T, H, device="cuda")
        moe.moe_unpermute(r.contiguous(), "fp32", T, H, k, inv, v.contiguous(), out)
        return (out.double() * dout.double()).sum()

    n = int((inv >= 0).sum())
    drow[n:] = 0
    a = (value(rows + drow, w) - value(rows - drow, w)) / 2
    b = (value(rows, w + dwt) - value(rows, w - dwt)) / 2
    routed = (inv >= 0)
    # fp32 steps: u relative on inputs and outputs of sums of T * H terms of size ~ k.
    bound = 16 * U * float((dout.abs().double().sum() * k * 16))
    assert abs(float(a - (drows.double() * drow.double()).sum())) < bound
    assert abs(float(b - (dw.double() * dwt.double())[routed].sum())) < bound


def test_captured_replayed_and_on_another_stream():
    """The training pass (copy, weighted sum, both gradients) captured once and
    replayed on new contents equals the eager calls, bitwise; so does a run on a
    side stream."""
    ensure_built()
    T, H, k, E = 130, 1024, 4, 16
    g = _gen(9)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    w, dout = torch.empty(T, k, device="cuda"), torch.empty_like(x)
    rows, out = torch.zeros(T * k, H, dtype=x.dtype, device="cuda"), torch.empty_like(x)
    drows, dw, dx = torch.zeros_like(rows), torch.empty_like(w), torch.empty_like(x)
    inv, _ = _route(T, k, E, 0.1, g)

    def step():
        moe.moe_permute(x, T, H * 2, k, inv, rows)
        moe.moe_unpermute(rows, "bf16", T, H, k, inv, w, out)
        moe.moe_unpermute_backward(dout, rows, "bf16", T, H, k, inv, w, drows, dw)
        moe.moe_permute_backward(drows, "bf16", T, H, k, inv, dx)

    def fill(seed):
        gg = _gen(seed)
        for t in (x, w, dout):
            t.copy_(torch.randn(t.shape, generator=gg, device="cuda"))
        for t in (rows, out, drows, dw, dx):
            t.zero_()

    outs = (rows, out, drows, dw, dx)
    want = {}
    for seed in (1, 2):
        fill(seed)
        step()
        torch.cuda.synchronize()
        want[seed] = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    fill(1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want[1]))
    graph = torch.cuda.CUDAGraph()
    fill(1)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for seed in (2, 1, 2):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[seed]))


def test_tensor_checks_on_the_gpu():
    ensure_built()
    T, H, k = 4, 64, 2
    inv = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(T, k, device="cuda")
    bad = [lambda: moe.moe_permute(x, T, H * 2, k, inv.long(), rows),
           lambda: moe.moe_permute(x, T, H * 2, k, inv, rows[1:]),
           lambda: moe.moe_permute(x.t(), T, H * 2, k, inv, rows),
           lambda: moe.moe_permute(x, T + 1, H * 2, k, inv, rows),
           lambda: moe.moe_unpermute(rows, "fp16", T, H, k, inv, w, x),
           lambda: moe.moe_unpermute(rows, "bf16", T, H, k, inv, w.half(), x),
           lambda: moe.moe_unpermute(rows, "bf16", T, H, k, inv, w, x.cpu()),
           lambda: moe.moe_unpermute(rows, "bf16", T, H, k, inv, w, rows[:T]),
           lambda: moe.moe_unpermute_backward(x, rows, "bf16", T, H, k, inv, w, rows, w)]
    for call in bad:
        with pytest.raises(moe.MoEError) as e:
            call()
        assert e.value.status == moe.MOE_ERR_INVALID_ARG


def _at(offset, shape, dtype, fill=None):
    """A contiguous tensor `offset` bytes into an allocation (512-byte aligned)."""
    n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    base = torch.zeros(n + 1024, dtype=torch.uint8, device="cuda")
    t = base[offset:offset + n].view(dtype).view(shape)
    assert t.data_ptr() % 512 == offset and t.is_contiguous()
    if fill is not None:
        t.copy_(fill)
    return t


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_buffers_at_the_least_alignment(dtype):
    """Rows 16 bytes and indices 4 bytes off a larger boundary give the same bytes."""
    ensure_built()
    T, H, k, E = 45, 264, 5, 8
    g = _gen(31)
    inv, _ = _route(T, k, E, 0.1, g)
    x = torch.randn(T, H, generator=g, device="cuda").to(DT[dtype])
    w = torch.randn(T, k, generator=g, device="cuda")
    dout = torch.randn(T, H, generator=g, device="cuda").to(DT[dtype])

    def run(make):
        a, iv, wt, do = (make(16, x.shape, x.dtype, x), make(4, inv.shape, inv.dtype, inv),
                         make(12, w.shape, w.dtype, w), make(48, dout.shape, dout.dtype, dout))
        rows, out = make(80, (T * k, H), x.dtype), make(16, (T, H), x.dtype)
        drows, dw, dx = make(112, (T * k, H), x.dtype), make(20, (T, k), torch.float32), make(16, (T, H), x.dtype)
        moe.moe_permute(a, T, H * x.element_size(), k, iv, rows)
        moe.moe_unpermute(rows, dtype, T, H, k, iv, wt, out)
        moe.moe_unpermute_backward(do, rows, dtype, T, H, k, iv, wt, drows, dw)
        moe.moe_permute_backward(drows, dtype, T, H, k, iv, dx)
        return rows, out, drows, dw, dx

    plain = run(lambda off, shape, dt, fill=None: torch.zeros(shape, dtype=dt, device="cuda")
                if fill is None else fill.clone())
    for a, b in zip(run(_at), plain):
        assert torch.equal(a, b)


def test_two_calls_at_once():
    """The same operators on two streams at once, on shared inputs."""
    ensure_built()
    T, H, k, E = 700, 2048, 6, 32
    g = _gen(41)
    inv, _ = _route(T, k, E, 0.05, g)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(T, k, generator=g, device="cuda")
    bufs = []
    for _ in range(3):
        bufs.append([torch.zeros(T * k, H, dtype=x.dtype, device="cuda"), torch.zeros_like(x),
                     torch.zeros(T * k, H, dtype=x.dtype, device="cuda"), torch.zeros_like(w)])
    torch.cuda.synchronize()

    def run(b):
        moe.moe_permute(x, T, H * 2, k, inv, b[0])
        moe.moe_unpermute(b[0], "bf16", T, H, k, inv, w, b[1])
        moe.moe_unpermute_backward(x, b[0], "bf16", T, H, k, inv, w, b[2], b[3])

    run(bufs[0])
    torch.cuda.synchronize()
    for _ in range(10):
        streams = [torch.cuda.Stream() for _ in range(2)]
        for s, b in zip(streams, bufs[1:]):
            with torch.cuda.stream(s):
                run(b)
        torch.cuda.synchronize()
        for b in bufs[1:]:
            assert all(torch.equal(p, q) for p, q in zip(b, bufs[0]))
