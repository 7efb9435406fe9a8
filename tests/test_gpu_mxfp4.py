"""MXFP4 on the GPU: the quantiser byte for byte and the grouped product against
oracle/rows.py in float64, and the chain of both with the row operators.

The product's tolerance: every E2M1 x E2M1 product with power-of-two scales is
exact in fp32; a K = 64 step of the tensor core adds 64 of them and the running
sum, ceil(K / 64) times.  Taking each of those additions to keep 24 bits, rounded
or cut (2^-23 relative to the magnitudes added), the sum is off by at most
(64 + K / 64) * 2^-23 * sum |a w|; then one rounding to the output type (bf16
2^-8, fp16 2^-11).  Whole-number cases, whose sums fit 24 bits, are bitwise."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import moe_expert_ffn_permute_b200 as moe
from oracle import rows as O

from gpu_helpers import ensure_built
from test_gpu_rows import DT, HALF, TINY, _gen, _np, _route

pytestmark = pytest.mark.gpu


def _quantize(x, dtype, layout, k=1, inv=None, fill=0xEE):
    T, K = x.shape
    R = T * k
    codes = torch.full((R, K // 2), fill, dtype=torch.uint8, device="cuda")
    scales = torch.full(moe.mxfp4_scale_shape(R, K, layout), fill, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mxfp4(x, dtype, T, K, k, inv, codes, scales, layout)
    return codes, scales


def _hard(T, K, dtype, seed):
    """Values of many magnitudes with exact ties, zeros, block maxima on a
    boundary, subnormals and blocks that are not finite."""
    g = _gen(seed)
    x = torch.randn(T, K, generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-12, 13, (T, K // 32, 1), generator=g, device="cuda").float()
                       ).expand(T, K // 32, 32).reshape(T, K)
    b = x.view(T, K // 32, 32)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], device="cuda").repeat(4)
    b[0, 0] = ties
    if T > 1:
        b[1, 0] = -ties * 2.0 ** -10
        b[1, -1] = 0.0
    if T > 2:
        b[2, 0] = 0.0
        b[2, 0, 5] = 6.0 * 2.0 ** -14 if dtype == "fp16" else 6.0 * 2.0 ** -120
        b[2, -1, 0] = float("nan")
    if T > 3:
        b[3, 0, 31] = float("inf")
        b[3, -1, :] = 2.0 ** -24 if dtype == "fp16" else 2.0 ** -133
    if T > 4:
        b[4, 0, 7] = 65504.0 if dtype == "fp16" else 3.0e38
    return x.to(DT[dtype])


@pytest.mark.parametrize("layout", ["row", "group"])
@pytest.mark.parametrize("dtype,T,K", [("bf16", 1, 32), ("fp16", 5, 32), ("fp32", 7, 64),
                                       ("bf16", 300, 96), ("bf16", 6, 7168), ("fp32", 33, 1568),
                                       ("fp16", 129, 160), ("bf16", 9, 128)])
def test_quantize_and_dequantize(dtype, T, K, layout):
    ensure_built()
    x = _hard(T, K, dtype, T * 17 + K)
    codes, scales = _quantize(x, dtype, layout)
    want_c, want_s = O.quantize_mxfp4(_np(x))
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)
    np.testing.assert_array_equal(scales.cpu().numpy(),
                                  want_s if layout == "row" else O.group_major(want_s))
    val = O.dequantize_mxfp4(want_c, want_s)
    for out_t in ("bf16", "fp32", "fp16"):
        out = torch.empty(T, K, dtype=DT[out_t], device="cuda")
        moe.moe_dequantize_mxfp4(codes, scales, layout, T, K, out_t, out)
        # Exact but for the range: codes of values near fp32's largest can stand for
        # 4 * 2^126 = 2^128, which rounds to infinity in bf16 and fp32 too.
        with np.errstate(over="ignore"):
            want = val.astype(np.float16 if out_t == "fp16" else np.float32).astype(np.float64)
        np.testing.assert_array_equal(_np(out), want)


def test_every_code_and_scale():
    ensure_built()
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None].expand(256, 16).contiguous()
    scales = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None].contiguous()
    for flip in (0, 85):
        c = torch.roll(codes, flip, 0).contiguous()
        out = torch.empty(256, 32, dtype=torch.float32, device="cuda")
        moe.moe_dequantize_mxfp4(c, scales, "row", 256, 32, "fp32", out)
        with np.errstate(over="ignore"):
            want = O.dequantize_mxfp4(c.cpu().numpy(), scales.cpu().numpy()).astype(np.float32)
        np.testing.assert_array_equal(out.cpu().numpy(), want)


@pytest.mark.parametrize("layout", ["row", "group"])
@pytest.mark.parametrize("dtype,T,K,k,E,masked", [("bf16", 1, 7168, 8, 32, 0.0),
                                                   ("fp16", 37, 96, 3, 8, 0.3),
                                                   ("fp32", 130, 288, 12, 16, 0.5),
                                                   ("bf16", 9, 64, 2, 4, 1.1)])
def test_quantize_into_expert_order(dtype, T, K, k, E, masked, layout):
    """Equals quantising in token order and copying; other rows are untouched."""
    ensure_built()
    g = _gen(T + K)
    inv, _ = _route(T, k, E, masked, g)
    x = _hard(T, K, dtype, 3)
    codes, scales = _quantize(x, dtype, layout, k, inv)
    want_c, want_s = O.quantize_mxfp4(_np(x))
    iv = inv.cpu().numpy()
    rc = O.permute(want_c, iv, np.full((T * k, K // 2), 0xEE, np.uint8))
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)
    if layout == "row":
        rs = O.permute(want_s, iv, np.full((T * k, K // 32), 0xEE, np.uint8))
    else:
        gm = O.group_major(want_s)
        rs = np.stack([O.permute(gm[i], iv, np.full((T * k, 4), 0xEE, np.uint8))
                       for i in range(len(gm))])
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)


def test_quantize_offsets_past_32_bits():
    """More than 2^32 codes and 2^31 bytes of them; checked on rows from both ends."""
    ensure_built()
    T, K, k = 640, 7168, 1024
    g = _gen(4)
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    inv = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).reshape(T, k).contiguous()
    codes, scales = _quantize(x, "bf16", "group", k, inv)
    base_c, base_s = _quantize(x, "bf16", "group")
    for t in (0, 1, 320, T - 1):
        at = inv[t].long()
        assert torch.equal(codes[at], base_c[t].expand(k, -1))
        assert torch.equal(scales[:, at], base_s[:, t:t + 1].expand(-1, k, -1))
    R = T * k
    out = torch.empty(R, K, dtype=torch.bfloat16, device="cuda")
    moe.moe_dequantize_mxfp4(codes, scales, "group", R, K, "bf16", out)
    one = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    moe.moe_dequantize_mxfp4(base_c, base_s, "group", T, K, "bf16", one)
    for t in (0, T - 1):
        assert torch.equal(out[inv[t].long()], one[t].expand(k, -1))


# --------------------------------------------------------------------- product
def _operands(R, E, N, K, seed, whole=False):
    """Codes and row-major scales of rows and weights (numpy).  whole: scales
    2^-1 .. 2^1, so that all sums are exact in fp32 for K <= 1024."""
    g = np.random.default_rng(seed)

    def draw(n):
        codes = g.integers(0, 256, (n, K // 2), dtype=np.uint8)
        lo, hi = (126, 129) if whole else (118, 126)
        return codes, g.integers(lo, hi, (n, K // 32)).astype(np.uint8)

    a, sa = draw(R)
    w, sw = draw(E * N)
    return a, sa, w.reshape(E, N, K // 2), sw.reshape(E, N, K // 32)


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Product:
    def __init__(self, R, E, N, K, a, sa, w, sw):
        self.R, self.E, self.N, self.K = R, E, N, K
        self.codes, self.scales = _cuda(a), _cuda(O.group_major(sa))
        self.w = torch.empty(moe.moe_mxfp4_weight_bytes(E, N, K), dtype=torch.uint8, device="cuda")
        self.ws = torch.empty(moe.moe_mxfp4_weight_scale_bytes(E, N, K), dtype=torch.uint8,
                              device="cuda")
        moe.moe_mxfp4_prepack(_cuda(w), _cuda(sw), E, N, K, self.w, self.ws)
        self.workspace = torch.zeros(moe.moe_mxfp4_workspace_bytes(R, E, N, K), dtype=torch.uint8,
                                     device="cuda")

    def __call__(self, offsets, dtype, out=None):
        if out is None:
            out = torch.full((self.R, self.N), 7.0, dtype=DT[dtype], device="cuda")
        moe.moe_mxfp4_gemm(self.codes, self.scales, offsets, self.R, self.E, self.N, self.K, self.w,
                           self.ws, dtype, out, self.workspace)
        return out

    def check(self):
        assert moe.moe_mxfp4_check_error(self.workspace) == 0


def _offsets(counts, lead=0):
    return np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int32)


# (counts, rows behind the last group, N, K): tile edges of 16, 64, 128 and 256
# rows on both tile variants (few rows per expert, many), groups without rows at
# the ends and in between, K inside and across the 128- and 256-wide blocks, N
# inside and across the 128-row weight blocks.
PRODUCTS = [
    ([1], 0, 8, 32), ([1], 3, 128, 256), ([2, 0, 1], 0, 136, 64), ([0, 15, 16, 17, 0], 2, 128, 96),
    ([63, 64, 65], 1, 264, 288), ([0, 0, 0], 4, 128, 128), ([33] * 40, 0, 64, 160),
    ([127, 1, 128], 0, 128, 512), ([129, 255, 256, 257], 5, 120, 320), ([700], 0, 384, 224),
    ([0, 513, 0, 3], 0, 256, 1024), ([2] * 256, 0, 40, 96), ([300, 0, 1], 0, 1160, 672),
]
PIDS = [f"p{i}-N{p[2]}-K{p[3]}" for i, p in enumerate(PRODUCTS)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("counts,behind,N,K", PRODUCTS, ids=PIDS)
def test_product_whole_numbers_bitwise(counts, behind, N, K, dtype):
    ensure_built()
    E, R = len(counts), sum(counts) + behind
    a, sa, w, sw = _operands(R, E, N, K, R + N + K, whole=True)
    off = _offsets(counts)
    p = Product(R, E, N, K, a, sa, w, sw)
    out = p(_cuda(off), dtype)
    p.check()
    want = O.grouped_product(O.dequantize_mxfp4(a, sa), O.dequantize_mxfp4(w.reshape(E * N, -1),
                             sw.reshape(E * N, -1)).reshape(E, N, K), off, np.full((R, N), 7.0))
    want = torch.from_numpy(want).to(DT[dtype])       # exact sums: one rounding
    assert torch.equal(out.cpu(), want), (out.cpu() != want).nonzero()[:8]
    if E == 1 and behind == 0:
        assert torch.equal(p(None, dtype), out)       # one group: offsets not needed


# Products on both sides of the CTA-pair kernel's rule (224 rows per group on average,
# and two waves of 256 x 256 tiles at K > 2560 or forty at less): the first seven run
# on single CTAs, the others on pairs.  Halves of 8 to 128 tokens, an odd number of
# weight blocks (a pair's second block past N), groups without rows, one K block, K
# that ends inside a block, several tiles per pair.  (Whole-number sums reach
# 144 * 7168 < 2^20 in steps of 2^-4: 24 bits.)
PAIRS = [
    ([5000], 3, 4104, 32), ([250, 33, 5120, 1, 0], 0, 4096, 96),
    ([1024, 0, 2050, 255, 17], 7, 6280, 288), ([300] * 10, 0, 7048, 160),
    ([2000, 31, 32, 33], 0, 10760, 64), ([77000], 0, 136, 32), ([2600, 700], 0, 6152, 1024),
    ([5000], 3, 2056, 2848), ([250, 33, 5120, 1, 0], 0, 2048, 2816),
    ([1024, 0, 2050, 255, 17], 7, 3080, 3104), ([300] * 10, 0, 3592, 2848),
    ([2000, 31, 32, 33], 0, 5384, 2816), ([2600, 700], 0, 3336, 7168), ([77000], 0, 2456, 32),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("counts,behind,N,K", PAIRS, ids=[f"q{i}-N{p[2]}-K{p[3]}" for i, p in enumerate(PAIRS)])
def test_product_on_pairs_whole_numbers_bitwise(counts, behind, N, K, dtype):
    test_product_whole_numbers_bitwise(counts, behind, N, K, dtype)


@pytest.mark.parametrize("counts,behind,N,K", [([5, 40, 0, 9], 0, 264, 2080), ([200, 90], 0, 128, 7168),
                                               ([1], 0, 512, 7168), ([777], 0, 136, 2048),
                                               ([3] * 32, 1, 256, 1536)])
def test_product_of_quantised_values(counts, behind, N, K):
    """Normal values quantised on the GPU, within the derived tolerance."""
    ensure_built()
    E, R = len(counts), sum(counts) + behind
    g = _gen(R + K)
    x = torch.randn(R, K, generator=g, device="cuda").to(torch.bfloat16)
    wt = (torch.randn(E * N, K, generator=g, device="cuda") * 0.02)
    a, sa = _quantize(x, "bf16", "row")
    w, sw = _quantize(wt, "fp32", "row")
    a, sa, w, sw = (t.cpu().numpy() for t in (a, sa, w, sw))
    off = _offsets(counts)
    p = Product(R, E, N, K, a, sa, w.reshape(E, N, -1), sw.reshape(E, N, -1))
    av, wv = O.dequantize_mxfp4(a, sa), O.dequantize_mxfp4(w, sw).reshape(E, N, K)
    want = O.grouped_product(av, wv, off, np.full((R, N), 7.0))
    mag = O.grouped_product(np.abs(av), np.abs(wv), off, np.zeros((R, N)))
    for dtype in ("bf16", "fp16"):
        out = p(_cuda(off), dtype)
        p.check()
        tol = 1.01 * ((64 + K / 64) * 2.0 ** -23 * mag + HALF[dtype] * np.abs(want)) + TINY[dtype]
        err = np.abs(_np(out) - want)
        assert (err <= tol).all(), (err.max(), (err / tol).max())
        assert torch.equal(p(_cuda(off), dtype), out)      # repeats bitwise


def test_product_offsets_that_are_not_prefix_sums():
    """Offsets that start late, run backwards or out of range stay in bounds and
    mean what their clamped, non-decreasing values say."""
    ensure_built()
    R, E, N, K = 100, 4, 128, 256
    a, sa, w, sw = _operands(R, E, N, K, 1, whole=True)
    p = Product(R, E, N, K, a, sa, w, sw)
    av = O.dequantize_mxfp4(a, sa)
    wv = O.dequantize_mxfp4(w.reshape(E * N, -1), sw.reshape(E * N, -1)).reshape(E, N, K)
    for off in ([10, 20, 20, 90, 95], [-5, 30, 7, 60, 1 << 30], [100] * 5, [50, 0, 0, 0, 0],
                [0, 1 << 31 - 1, 3, 5, 100]):
        off = np.array(off, np.int64).astype(np.int32)
        out = p(_cuda(off), "bf16")
        p.check()
        want = torch.from_numpy(O.grouped_product(av, wv, off, np.full((R, N), 7.0))).bfloat16()
        assert torch.equal(out.cpu(), want), off


@pytest.mark.parametrize("N,K", [(5128, 320), (2568, 2848)], ids=["single", "pairs"])
def test_product_on_pairs_offsets_and_nan_rows(N, K):
    """Offsets that are not prefix sums, and NaN scales, on large products."""
    ensure_built()
    R, E = 4000, 4
    a, sa, w, sw = _operands(R, E, N, K, 1, whole=True)
    p = Product(R, E, N, K, a, sa, w, sw)
    av = O.dequantize_mxfp4(a, sa)
    wv = O.dequantize_mxfp4(w.reshape(E * N, -1), sw.reshape(E * N, -1)).reshape(E, N, K)
    for off in ([10, 20, 20, 3900, 3950], [-5, 300, 70, 600, 1 << 30], [4000] * 5,
                [0, (1 << 31) - 1, 3, 5, 4000]):
        off = np.array(off, np.int64).astype(np.int32)
        out = p(_cuda(off), "bf16")
        p.check()
        want = torch.from_numpy(O.grouped_product(av, wv, off, np.full((R, N), 7.0))).bfloat16()
        assert torch.equal(out.cpu(), want), off
    off = _cuda(_offsets([1000, 1000, 1000, 1000]))
    clean = p(off, "bf16")
    sa[2717, 3], sw[1, 130, 9] = 255, 255
    out = Product(R, E, N, K, a, sa, w, sw)(off, "bf16")
    want = torch.zeros(R, N, dtype=torch.bool, device="cuda")
    want[2717], want[1000:2000, 130] = True, True
    assert torch.equal(torch.isnan(out), want)
    assert torch.equal(out[~want], clean[~want])


@pytest.mark.parametrize("N,K", [(5128, 512), (2568, 2816)], ids=["single", "pairs"])
def test_product_on_pairs_in_a_graph_beside_another(N, K):
    """A captured large product (two launches on pairs) and a captured small one,
    workspaces of their own, replayed on two streams at once, equal the eager calls."""
    ensure_built()
    cases = [([1500, 2500], N, K), ([40] * 32, 256, 1024)]
    runs = []
    for i, (counts, N, K) in enumerate(cases):
        p = Product(sum(counts), len(counts), N, K, *_operands(sum(counts), len(counts), N, K, 60 + i))
        off = _cuda(_offsets(counts))
        want = p(off, "bf16")
        out = torch.zeros_like(want)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                p(off, "bf16", out)
        runs.append((p, off, want, out, graph, torch.cuda.Stream()))
    for _ in range(5):
        for r in runs:
            r[3].zero_()
        torch.cuda.synchronize()
        for r in runs:
            with torch.cuda.stream(r[5]):
                r[4].replay()
        torch.cuda.synchronize()
        for p, _, want, out, _, _ in runs:
            assert torch.equal(out, want)
            p.check()


def test_product_keeps_nan_rows_apart():
    """A NaN scale (a row whose block was not finite) makes that row NaN and no
    other; a NaN weight scale that output feature."""
    ensure_built()
    R, E, N, K = 40, 1, 136, 320
    a, sa, w, sw = _operands(R, E, N, K, 2, whole=True)
    clean = Product(R, E, N, K, a, sa, w, sw)(None, "bf16")
    sa[17, 3], sw[0, 130, 9] = 255, 255
    out = Product(R, E, N, K, a, sa, w, sw)(None, "bf16")
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[17], want[:, 130] = True, True
    assert torch.equal(nan, want)
    assert torch.equal(out[~want], clean[~want])


def test_product_in_two_graphs_and_on_two_streams():
    """Two captured products with workspaces of their own, replayed on two streams
    at once, equal the eager calls; one workspace serves calls in order."""
    ensure_built()
    cases = [([40] * 32, 256, 1024), ([600, 300], 512, 768)]
    ps, offs, want, outs, graphs = [], [], [], [], []
    for i, (counts, N, K) in enumerate(cases):
        R, E = sum(counts), len(counts)
        ps.append(Product(R, E, N, K, *_operands(R, E, N, K, 50 + i)))
        offs.append(_cuda(_offsets(counts)))
        want.append(ps[i](offs[i], "bf16"))
        outs.append(torch.zeros_like(want[i]))
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                ps[i](offs[i], "bf16", outs[i])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[i])
            ps[i].check()


def test_expert_ffn_chain():
    """The operators as a user runs them: route, quantise into expert order, gate-up
    product, SwiGLU, quantise, down product, weighted sum back -- against the same
    chain in float64 (on the GPU's own 4-bit codes of the activation, which rounding
    decides)."""
    ensure_built()
    T, H, I, E, k = 70, 512, 256, 8, 3
    g = _gen(77)
    inv, offsets = _route(T, k, E, 0.1, g)
    S = T * k
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    tw = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
    ws = []
    for rows, cols in ((2 * I, H), (H, I)):
        wt = torch.randn(E * rows, cols, generator=g, device="cuda") * 0.05
        c, s = _quantize(wt, "fp32", "row")
        ws.append((c.reshape(E, rows, -1), s.reshape(E, rows, -1)))

    def layer(w, sw, N, K):
        wt = torch.empty(moe.moe_mxfp4_weight_bytes(E, N, K), dtype=torch.uint8, device="cuda")
        st = torch.empty(moe.moe_mxfp4_weight_scale_bytes(E, N, K), dtype=torch.uint8, device="cuda")
        moe.moe_mxfp4_prepack(w, sw, E, N, K, wt, st)
        return wt, st

    w1, w2 = layer(*ws[0], 2 * I, H), layer(*ws[1], H, I)
    space = torch.zeros(max(moe.moe_mxfp4_workspace_bytes(S, E, 2 * I, H),
                            moe.moe_mxfp4_workspace_bytes(S, E, H, I)), dtype=torch.uint8,
                        device="cuda")
    codes = torch.zeros(S, H // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(moe.mxfp4_scale_shape(S, H, "group"), dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mxfp4(x, "bf16", T, H, k, inv, codes, scales, "group")
    h = torch.zeros(S, 2 * I, dtype=torch.bfloat16, device="cuda")
    moe.moe_mxfp4_gemm(codes, scales, offsets, S, E, 2 * I, H, *w1, "bf16", h, space)
    act = (torch.nn.functional.silu(h[:, :I].float()) * h[:, I:].float()).to(torch.bfloat16)
    c2, s2 = _quantize(act, "bf16", "group")
    y = torch.zeros(S, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_mxfp4_gemm(c2, s2, offsets, S, E, H, I, *w2, "bf16", y, space)
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_unpermute(y, "bf16", T, H, k, inv, tw, out)
    assert moe.moe_mxfp4_check_error(space) == 0

    iv, off = inv.cpu().numpy(), offsets.cpu().numpy()
    qc, qs = O.quantize_mxfp4(_np(x))
    a = O.permute(O.dequantize_mxfp4(qc, qs), iv, np.zeros((S, H)))
    val = [O.dequantize_mxfp4(c.cpu().numpy(), s.cpu().numpy()) for c, s in ws]
    h64 = O.grouped_product(a, val[0], off, np.zeros((S, 2 * I)))
    mag = O.grouped_product(np.abs(a), np.abs(val[0]), off, np.zeros((S, 2 * I)))
    tol = 1.01 * ((64 + H / 64) * 2.0 ** -23 * mag + HALF["bf16"] * np.abs(h64)) + TINY["bf16"]
    assert (np.abs(_np(h) - h64) <= tol).all()
    a2c, a2s = O.quantize_mxfp4(_np(act))
    np.testing.assert_array_equal(c2.cpu().numpy(), a2c)
    a2 = O.dequantize_mxfp4(a2c, a2s)
    y64 = O.grouped_product(a2, val[1], off, np.zeros((S, H)))
    mag = O.grouped_product(np.abs(a2), np.abs(val[1]), off, np.zeros((S, H)))
    tol = 1.01 * ((64 + I / 64) * 2.0 ** -23 * mag + HALF["bf16"] * np.abs(y64)) + TINY["bf16"]
    assert (np.abs(_np(y) - y64) <= tol).all()
    # The sum takes the GPU's rows: k multiply-adds and one rounding.
    w64 = _np(tw)
    want = O.unpermute(_np(y), iv, w64)
    mag = O.unpermute(np.abs(_np(y)), iv, np.abs(w64))
    assert (np.abs(_np(out) - want) <= 1.01 * (k * 2.0 ** -24 * mag + HALF["bf16"] * np.abs(want))
            + TINY["bf16"]).all()


def test_tensor_checks_on_the_gpu():
    ensure_built()
    R, E, N, K = 8, 2, 64, 64
    p = Product(R, E, N, K, *_operands(R, E, N, K, 3))
    off = _cuda(_offsets([4, 4]))
    out = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
    args = dict(codes=p.codes, scales=p.scales, offsets=off, R=R, E=E, N=N, K=K, w_tiled=p.w,
                w_scales_chunked=p.ws, dtype="bf16", out=out, workspace=p.workspace)
    moe.moe_mxfp4_gemm(**args)
    for over in (dict(codes=p.codes[:4]), dict(scales=p.scales[:, :4]), dict(offsets=off.long()),
                 dict(offsets=off[:2]), dict(w_tiled=p.w[:-1]), dict(w_scales_chunked=p.ws[:512]),
                 dict(dtype="fp16"), dict(out=out[:4]), dict(out=out.t()), dict(workspace=p.workspace[:128]),
                 dict(R=9), dict(N=72, out=torch.zeros(R, 72, dtype=torch.bfloat16).cuda(), w_tiled=p.w[:1])):
        with pytest.raises(moe.MoEError) as e:
            moe.moe_mxfp4_gemm(**{**args, **over})
        assert e.value.status == moe.MOE_ERR_INVALID_ARG, over


def test_buffers_at_the_least_alignment():
    """Codes 16, scales and offsets 4, quantiser inputs 32 bytes off a larger
    boundary give the same bytes."""
    from test_gpu_rows import _at
    ensure_built()
    T, K, k, E, N = 29, 352, 3, 4, 136
    g = _gen(51)
    inv, offsets = _route(T, k, E, 0.1, g)
    S = T * k
    x = _hard(T, K, "bf16", 8)
    x = torch.where(torch.isfinite(x.float()) & (x.float().abs() < 1e4), x, 1.0)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.randint(120, 128, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)

    def run(make):
        a, iv, off = (make(32, x.shape, x.dtype, x), make(4, inv.shape, inv.dtype, inv),
                      make(12, offsets.shape, offsets.dtype, offsets))
        codes = make(16, (S, K // 2), torch.uint8)
        scales = make(4, moe.mxfp4_scale_shape(S, K, "group"), torch.uint8)
        moe.moe_quantize_mxfp4(a, "bf16", T, K, k, iv, codes, scales, "group")
        val = make(32, (S, K), torch.float32)
        moe.moe_dequantize_mxfp4(codes, scales, "group", S, K, "fp32", val)
        wt = make(16, (moe.moe_mxfp4_weight_bytes(E, N, K),), torch.uint8)
        st = make(48, (moe.moe_mxfp4_weight_scale_bytes(E, N, K),), torch.uint8)
        moe.moe_mxfp4_prepack(make(16, w.shape, w.dtype, w), make(1, ws.shape, ws.dtype, ws), E, N, K, wt, st)
        out = make(16, (S, N), torch.bfloat16)
        space = torch.zeros(moe.moe_mxfp4_workspace_bytes(S, E, N, K), dtype=torch.uint8, device="cuda")
        moe.moe_mxfp4_gemm(codes, scales, off, S, E, N, K, wt, st, "bf16", out, space)
        assert moe.moe_mxfp4_check_error(space) == 0
        return codes, scales, val, out

    plain = run(lambda off, shape, dt, fill=None: torch.zeros(shape, dtype=dt, device="cuda")
                if fill is None else fill.clone())
    for a, b in zip(run(_at), plain):
        assert torch.equal(a, b)


@pytest.mark.parametrize("R,E,N,K", [(300000, 2, 8192, 64), (56000, 256, 40960, 32), (1100000, 1, 8, 8192)],
                         ids=["pairs-out", "single-out", "codes"])
def test_product_offsets_past_32_bits(R, E, N, K):
    """Outputs or codes of more than 2^32 bytes, on both kernels; rows from every
    part of the range against the oracle, bitwise (whole-number operands)."""
    ensure_built()
    g = _gen(R)
    rnd = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    codes, w = rnd(R, K // 2), rnd(E, N, K // 2)
    if K > 1024:       # sparse rows: the sums stay within 24 bits
        codes[:, 16:] = 0
        codes[:, -16:] = rnd(R, 16)
    one = lambda *s: torch.full(s, 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    scales, ws = one((K + 127) // 128, R, 4), one(E, N, K // 32)
    if K % 128:
        scales[-1, :, (K % 128) // 32:] = 0
    cut = np.sort(np.random.default_rng(R).integers(0, R, E - 1))
    off = np.concatenate([[0], cut, [R]]).astype(np.int32)
    p = Product.__new__(Product)
    p.R, p.E, p.N, p.K, p.codes, p.scales = R, E, N, K, codes, scales
    p.w = torch.empty(moe.moe_mxfp4_weight_bytes(E, N, K), dtype=torch.uint8, device="cuda")
    p.ws = torch.empty(moe.moe_mxfp4_weight_scale_bytes(E, N, K), dtype=torch.uint8, device="cuda")
    moe.moe_mxfp4_prepack(w, ws, E, N, K, p.w, p.ws)
    p.workspace = torch.zeros(moe.moe_mxfp4_workspace_bytes(R, E, N, K), dtype=torch.uint8, device="cuda")
    out = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    p(_cuda(off), "bf16", out)
    p.check()
    for r in [0, 1, R // 3, R // 2 + 7, R - 300, R - 2, R - 1]:
        e = int(np.searchsorted(off, r, side="right")) - 1
        a = O.dequantize_mxfp4(codes[r:r + 1].cpu().numpy(), np.full((1, K // 32), 127, np.uint8))
        b = O.dequantize_mxfp4(w[e].cpu().numpy(), np.full((N, K // 32), 127, np.uint8))
        assert torch.equal(out[r].cpu(), torch.from_numpy((a @ b.T)[0]).bfloat16()), r


@pytest.mark.parametrize("counts,other,N,K", [([40, 0, 9, 15] * 4, [1, 100, 0, 3] * 4, 264, 288),
                                              ([3000, 1000], [17, 3983], 5128, 64),
                                              ([3000, 1000], [17, 3983], 2568, 2816)],
                         ids=["single", "single-large", "pairs"])
def test_replay_on_other_groups(counts, other, N, K):
    """A captured product replayed on other row offsets (and other rows): the launch
    is sized by R and E alone."""
    ensure_built()
    E, R = len(counts), max(sum(counts), sum(other))
    a, sa, w, sw = _operands(R, E, N, K, 9, whole=True)
    p = Product(R, E, N, K, a, sa, w, sw)
    off = _cuda(_offsets(counts))
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    p(off, "bf16", out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p(off, "bf16", out)
    for c in (other, counts, other):
        off.copy_(_cuda(_offsets(c)))
        p.codes.copy_(torch.roll(p.codes, 1, 0))
        out.fill_(7.0)
        graph.replay()
        got = out.clone()
        want = p(off, "bf16")
        assert torch.equal(got, want)
        assert (got[sum(c):] == 7.0).all() and not (got[:sum(c)] == 7.0).all()
    p.check()


def test_operators_on_a_plan_s_routing():
    """The routing in a plan's workspace (moe_route, raw addresses from the view)
    drives the operators as moe_route_static's does."""
    ensure_built()
    T, H, k, E, N = 96, 512, 2, 8, 136
    g = _gen(61)
    lay = moe.MoELayer(T, H, 256, E, k)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32).contiguous()
    ids[3, 1] = -1
    moe.moe_route(lay.plan, ids, lay.workspace)
    v = lay.view()
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, offsets, perm, inv = i32(E), i32(E + 1), i32(T * k), i32(T * k)
    moe.moe_route_static(ids, T, k, E, counts, offsets, perm, inv)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    _, _, w, sw = _operands(1, E, N, H, 4)
    res = []
    for iv, off in ((v.inv, v.offsets), (inv, offsets)):
        codes = torch.zeros(T * k, H // 2, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(moe.mxfp4_scale_shape(T * k, H, "group"), dtype=torch.uint8, device="cuda")
        moe.moe_quantize_mxfp4(x, "bf16", T, H, k, iv, codes, scales, "group")
        p = Product(T * k, E, N, H, np.zeros((T * k, H // 2), np.uint8),
                    np.zeros((T * k, H // 32), np.uint8), w, sw)
        p.codes, p.scales = codes, scales
        out = torch.zeros(T * k, N, dtype=torch.bfloat16, device="cuda")
        p(off, "bf16", out)
        rows = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
        moe.moe_permute(x, T, H * 2, k, iv, rows)
        res.append((codes, scales, out, rows))
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert lay.check() == 0


def test_product_of_the_most_rows():
    """2^31 - 1 rows (95 GB of buffers), in one group and with a last group of a single
    row whose second half would lie past 2^31 - 1: every row written, bitwise."""
    ensure_built()
    R, E, N, K = (1 << 31) - 1, 2, 8, 32
    torch.cuda.empty_cache()
    g = _gen(21)
    codes = torch.randint(0, 256, (R, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.zeros(1, R, 4, dtype=torch.uint8, device="cuda")
    scales[:, :, 0] = 127
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.full((E, N, 1), 127, dtype=torch.uint8, device="cuda")
    out = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    table = torch.cat([table, -table])
    value = lambda c: table[torch.stack([c & 15, c >> 4], -1).flatten(-2).int()]  # noqa: E731
    for counts in ([R], [R - 1, 1]):
        n = len(counts)
        wt = torch.empty(moe.moe_mxfp4_weight_bytes(n, N, K), dtype=torch.uint8, device="cuda")
        st = torch.empty(moe.moe_mxfp4_weight_scale_bytes(n, N, K), dtype=torch.uint8, device="cuda")
        moe.moe_mxfp4_prepack(w[:n], ws[:n], n, N, K, wt, st)
        space = torch.zeros(moe.moe_mxfp4_workspace_bytes(R, n, N, K), dtype=torch.uint8, device="cuda")
        out.fill_(float("nan"))
        off = _cuda(_offsets(np.array(counts, np.int64)))
        moe.moe_mxfp4_gemm(codes, scales, off, R, n, N, K, wt, st, "bf16", out, space)
        assert moe.moe_mxfp4_check_error(space) == 0
        del space
        step = 1 << 24
        for e, lo, hi in ((0, 0, counts[0]),) + (((1, R - 1, R),) if n == 2 else ()):
            for r in range(lo, hi, step):
                rows = slice(r, min(r + step, hi))
                want = (value(codes[rows]) @ value(w[e]).T).bfloat16()      # exact in fp32
                assert torch.equal(out[rows], want), (n, r)
    del codes, scales, out
    torch.cuda.empty_cache()


# One product for each kernel: groups of few rows, of more, and on CTA pairs.
VARIANTS = [([40, 0, 9, 15] * 4, 264, 288), ([300, 500], 264, 288), ([1500, 2500], 2568, 2816)]


@pytest.mark.timeout(120)
@pytest.mark.parametrize("counts,N,K", VARIANTS, ids=["few", "many", "pairs"])
def test_waits_that_run_out_end_the_product(counts, N, K):
    """The issuers' wait runs out (debug hook): the launch stops with a timeout in the
    workspace's error word, the context stays usable, and the word stays until it is
    cleared."""
    ensure_built()
    E, R = len(counts), sum(counts)
    a, sa, w, sw = _operands(R, E, N, K, 31, whole=True)
    off = _cuda(_offsets(counts))
    p = Product(R, E, N, K, a, sa, w, sw)
    assert (p.workspace.numel() > 256) == (R == 4000)
    want = p(off, "bf16")
    p.check()
    try:
        moe.moe_mxfp4_set_debug(1)
        p(off, "bf16")
        torch.cuda.synchronize()
    finally:
        moe.moe_mxfp4_set_debug(0)
    assert moe.moe_mxfp4_check_error(p.workspace) == 5          # MOE_ERR_DEVICE_TIMEOUT
    assert torch.equal(p(off, "bf16"), want)
    assert moe.moe_mxfp4_check_error(p.workspace) == 5
    moe.moe_mxfp4_clear_error(p.workspace)
    assert torch.equal(p(off, "bf16"), want)
    p.check()


def test_error_word_is_read_and_cleared():
    """The error word as the kernels write it (bit 5), written from the host."""
    ensure_built()
    counts, N, K = VARIANTS[0]
    E, R = len(counts), sum(counts)
    p = Product(R, E, N, K, *_operands(R, E, N, K, 33, whole=True))
    off = _cuda(_offsets(counts))
    want = p(off, "bf16")
    p.check()
    p.workspace[:4] = torch.tensor([32, 0, 0, 0], dtype=torch.uint8, device="cuda")
    assert moe.moe_mxfp4_check_error(p.workspace) == 5
    assert torch.equal(p(off, "bf16"), want)
    assert moe.moe_mxfp4_check_error(p.workspace) == 5
    moe.moe_mxfp4_clear_error(p.workspace)
    p.check()
    assert torch.equal(p(off, "bf16"), want)
    p.check()


# Sizes on pairs (the last of VARIANTS) and on single CTAs, with the kernel that takes them.
def _on_pairs(R, E, N, K):
    return moe.moe_mxfp4_workspace_bytes(R, E, N, K) > 256


def test_cases_reach_the_kernels_they_are_for():
    """PRODUCTS and the first seven of PAIRS run on single CTAs, the others on pairs."""
    ensure_built()
    sizes = [(sum(c) + b, len(c), N, K) for c, b, N, K in PRODUCTS + PAIRS]
    assert [_on_pairs(*s) for s in sizes] == [False] * (len(PRODUCTS) + 7) + [True] * (len(PAIRS) - 7)


@pytest.mark.parametrize("shift", [-125, -93, 93, 125])
@pytest.mark.parametrize("counts,N,K", VARIANTS, ids=["few", "many", "pairs"])
def test_product_of_distant_scales_bitwise(counts, N, K, shift):
    """Scale bytes from 1 to 253 on one side and as far from 127 the other way on the
    other: the products of two scales are 2^-2 to 2^2, and the sums exact."""
    ensure_built()
    E, R = len(counts), sum(counts)
    a, sa, w, sw = _operands(R, E, N, K, 71, whole=True)
    sa, sw = (sa.astype(int) + shift).astype(np.uint8), (sw.astype(int) - shift).astype(np.uint8)
    off = _offsets(counts)
    p = Product(R, E, N, K, a, sa, w, sw)
    assert _on_pairs(R, E, N, K) == (R == 4000)
    want = O.grouped_product(O.dequantize_mxfp4(a, sa), O.dequantize_mxfp4(w.reshape(E * N, -1),
                             sw.reshape(E * N, -1)).reshape(E, N, K), off, np.full((R, N), 7.0))
    for dtype in ("bf16", "fp16"):
        out = p(_cuda(off), dtype)
        p.check()
        assert torch.equal(out.cpu(), torch.from_numpy(want).to(DT[dtype]))


@pytest.mark.parametrize("counts,behind,N,K", [([1400, 0, 2600], 2, 2568, 2848), ([3000], 0, 4104, 7168),
                                               ([300] * 6, 1, 6152, 2912)])
def test_product_on_pairs_of_quantised_values(counts, behind, N, K):
    ensure_built()
    assert _on_pairs(sum(counts) + behind, len(counts), N, K)
    test_product_of_quantised_values(counts, behind, N, K)


def test_product_codes_past_32_bits_on_single_ctas():
    ensure_built()
    assert not _on_pairs(57000, 256, 8, 151552)
    test_product_offsets_past_32_bits(57000, 256, 8, 151552)


FIRST_CALLS = """
import sys
import torch
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import moe_expert_ffn_permute_b200 as moe
u8, bf16 = torch.uint8, torch.bfloat16
rnd = lambda *s: torch.randint(0, 256, s, device="cuda", dtype=u8)
for R, N, K in ((64, 264, 288), (1024, 264, 288), (4000, 2568, 2816)):
    x, T, k = torch.randn(R, K, device="cuda").to(bf16), R // 2, 2
    inv = torch.arange(R, device="cuda", dtype=torch.int32)
    tw = torch.rand(T, k, device="cuda")
    w = torch.zeros(moe.moe_mxfp4_weight_bytes(1, N, K), dtype=u8, device="cuda")
    ws = torch.zeros(moe.moe_mxfp4_weight_scale_bytes(1, N, K), dtype=u8, device="cuda")
    raw, raw_s = rnd(1, N, K // 2), torch.full((1, N, K // 32), 127, dtype=u8, device="cuda")
    codes = torch.zeros(R, K // 2, dtype=u8, device="cuda")
    scales = torch.zeros(moe.mxfp4_scale_shape(R, K, "group"), dtype=u8, device="cuda")
    space = torch.zeros(moe.moe_mxfp4_workspace_bytes(R, 1, N, K), dtype=u8, device="cuda")
    out, y = torch.zeros(R, N, dtype=bf16, device="cuda"), torch.zeros(T, N, dtype=bf16, device="cuda")
    def step():
        moe.moe_mxfp4_prepack(raw, raw_s, 1, N, K, w, ws)
        moe.moe_quantize_mxfp4(x, "bf16", T, K, k, inv, codes, scales, "group")
        moe.moe_mxfp4_gemm(codes, scales, None, R, 1, N, K, w, ws, "bf16", out, space)
        moe.moe_unpermute(out, "bf16", T, N, k, inv, tw, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    got = [t.clone() for t in (codes, scales, w, ws, out, y)]
    assert moe.moe_mxfp4_check_error(space) == 0 and got[-1].abs().sum() > 0
    for t in (codes, scales, w, ws, out, y):
        t.zero_()
    step()
    assert all(torch.equal(a, b) for a, b in zip(got, (codes, scales, w, ws, out, y)))
print("captured ok")
"""


def test_first_calls_of_a_process_are_captured():
    """Every launch's first use inside a capture (kernels are loaded and set up there)."""
    ensure_built()
    root = os.path.abspath(os.path.join(os.path.dirname(__file__), ".."))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=root)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("captured ok"), r.stdout + r.stderr


@pytest.mark.parametrize("T,H,N,k", [(1, 512, 264, 4), (37, 1024, 136, 2), (600, 288, 264, 3), (2000, 2816, 2568, 2)])
def test_launches_that_overlap_read_what_the_last_one_wrote(T, H, N, k):
    """Forty rounds on other tokens through the same buffers, captured without a gap: each
    launch starts while those before it run, and rereads addresses that they rewrite."""
    ensure_built()
    g, n, S = _gen(T + H), 40, T * k
    xs = torch.randn(n, T, H, generator=g, device="cuda").to(torch.bfloat16)
    invs = [torch.randperm(S, generator=g, device="cuda").reshape(T, k).int() for _ in range(n)]
    tw = [torch.rand(T, k, generator=g, device="cuda") for _ in range(n)]
    p = Product(S, 1, N, H, *_operands(S, 1, N, H, 81))
    rows, inv, w = torch.zeros(S, H, dtype=xs.dtype, device="cuda"), torch.empty_like(invs[0]), torch.empty_like(tw[0])
    drows, y = torch.zeros_like(rows), torch.zeros(S, N, dtype=xs.dtype, device="cuda")

    def make():
        return [torch.zeros(n, T, H, dtype=xs.dtype, device="cuda"), torch.zeros(n, T, k, device="cuda"),
                torch.zeros(n, T, H, dtype=xs.dtype, device="cuda"), torch.zeros(n, T, N, dtype=xs.dtype, device="cuda")]

    def step(i, o, wait):
        calls = (lambda: moe.moe_permute(invs[i], T, 4 * k, 1, first, inv),
                 lambda: moe.moe_permute(tw[i], T, 4 * k, 1, first, w),
                 lambda: moe.moe_permute(xs[i], T, H * 2, k, inv, rows),
                 lambda: moe.moe_unpermute(rows, "bf16", T, H, k, inv, w, o[0][i]),
                 lambda: moe.moe_unpermute_backward(xs[i], rows, "bf16", T, H, k, inv, w, drows, o[1][i]),
                 lambda: moe.moe_permute_backward(drows, "bf16", T, H, k, inv, o[2][i]),
                 lambda: moe.moe_quantize_mxfp4(xs[i], "bf16", T, H, k, inv, p.codes, p.scales, "group"),
                 lambda: p(None, "bf16", y),
                 lambda: moe.moe_unpermute(y, "bf16", T, N, k, inv, w, o[3][i]))
        for call in calls:
            call()
            if wait:
                torch.cuda.synchronize()

    first = torch.arange(T, dtype=torch.int32, device="cuda")
    want, got = make(), make()
    for i in range(n):
        step(i, want, True)
    p.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(n):
            step(i, got, False)
    for _ in range(5):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    for t in got:
        t.zero_()
    for i in range(n):
        step(i, got, False)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    p.check()
