"""Refusals of the row operators and the MXFP4 operators, without a GPU: sizes,
pointers, alignment and overlap by the C ABI (raw addresses; nothing is launched),
tensors by the binding."""
import pytest
import torch

import moe_expert_ffn_permute_b200 as moe
from moe_expert_ffn_permute_b200.build import build

INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 3
A, B, C, D, E_, F_, G = (1 << 40, 2 << 40, 3 << 40, 4 << 40, 5 << 40, 6 << 40, 7 << 40)


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _refused(status, fn, **over):
    base = {
        "moe_permute": dict(x=A, T=4, row_bytes=256, k=2, inv=B, rows=C),
        "moe_permute_backward": dict(drows=A, dtype="bf16", T=4, H=64, k=2, inv=B, dx=C),
        "moe_unpermute": dict(rows=A, dtype="bf16", T=4, H=64, k=2, inv=B, topk_w=C, out=D),
        "moe_unpermute_backward": dict(dout=A, rows=B, dtype="bf16", T=4, H=64, k=2, inv=C,
                                       topk_w=D, drows=E_, dw=F_),
        "moe_quantize_mxfp4": dict(x=A, dtype="bf16", T=4, K=64, k=2, inv=B, codes=C, scales=D,
                                   scale_layout="group"),
        "moe_dequantize_mxfp4": dict(codes=A, scales=B, scale_layout="row", R=4, K=64,
                                     dtype="bf16", out=C),
        "moe_mxfp4_prepack": dict(w=A, w_scales=B, E=2, N=64, K=64, w_tiled=C,
                                  w_scales_chunked=D),
        "moe_mxfp4_gemm": dict(codes=A, scales=B, offsets=C, R=8, E=2, N=64, K=64, w_tiled=D,
                               w_scales_chunked=E_, dtype="bf16", out=F_, workspace=G),
    }[fn]
    base.update(over)
    with pytest.raises(moe.MoEError) as e:
        getattr(moe, fn)(**base, stream=0)
    assert e.value.status == status, (fn, over, e.value)


CASES = [
    ("moe_permute", INVALID, dict(x=None)), ("moe_permute", INVALID, dict(inv=None)),
    ("moe_permute", INVALID, dict(rows=None)), ("moe_permute", INVALID, dict(T=0)),
    ("moe_permute", INVALID, dict(k=0)), ("moe_permute", INVALID, dict(row_bytes=0)),
    ("moe_permute", INVALID, dict(T=1 << 30, k=2)), ("moe_permute", INVALID, dict(T=1 << 31)),
    ("moe_permute", UNSUPPORTED, dict(row_bytes=18)), ("moe_permute", ALIGNMENT, dict(x=A + 8)),
    ("moe_permute", ALIGNMENT, dict(rows=C + 4)), ("moe_permute", ALIGNMENT, dict(inv=B + 2)),
    ("moe_permute", INVALID, dict(rows=A)), ("moe_permute", INVALID, dict(rows=A + 1008)),
    ("moe_permute", UNSUPPORTED, dict(T=1 << 30, k=1, row_bytes=1 << 44)),
    ("moe_permute_backward", INVALID, dict(drows=None)),
    ("moe_permute_backward", INVALID, dict(dx=None)),
    ("moe_permute_backward", INVALID, dict(dtype="fp8")),
    ("moe_permute_backward", INVALID, dict(dx=A + 16)),
    ("moe_permute_backward", UNSUPPORTED, dict(H=63)),
    ("moe_permute_backward", UNSUPPORTED, dict(dtype="fp32", H=62)),
    ("moe_permute_backward", ALIGNMENT, dict(dx=C + 8)),
    ("moe_unpermute", INVALID, dict(topk_w=None)), ("moe_unpermute", INVALID, dict(inv=None)),
    ("moe_unpermute", INVALID, dict(T=-1)), ("moe_unpermute", INVALID, dict(H=0)),
    ("moe_unpermute", INVALID, dict(k=-3)), ("moe_unpermute", INVALID, dict(dtype=torch.bfloat16)),
    ("moe_unpermute", ALIGNMENT, dict(topk_w=C + 1)), ("moe_unpermute", UNSUPPORTED, dict(H=4)),
    ("moe_unpermute_backward", INVALID, dict(drows=None, dw=None)),
    ("moe_unpermute_backward", INVALID, dict(rows=None)),
    ("moe_unpermute_backward", INVALID, dict(topk_w=None)),
    ("moe_unpermute_backward", INVALID, dict(drows=A)),
    ("moe_unpermute_backward", INVALID, dict(drows=B)),
    ("moe_unpermute_backward", INVALID, dict(dw=E_ + 16)),
    ("moe_unpermute_backward", ALIGNMENT, dict(dw=F_ + 2)),
    ("moe_unpermute_backward", UNSUPPORTED, dict(H=20)),
    ("moe_permute", INVALID, dict(rows=B)), ("moe_permute", UNSUPPORTED, dict(T=1, k=(1 << 31) - 1, row_bytes=1 << 40)),
    ("moe_permute", UNSUPPORTED, dict(T=1, k=(1 << 24) + 1)), ("moe_unpermute", UNSUPPORTED, dict(T=1, k=(1 << 24) + 1)),
    ("moe_unpermute_backward", UNSUPPORTED, dict(T=1, k=1 << 30)), ("moe_quantize_mxfp4", UNSUPPORTED, dict(T=1, k=1 << 30)),
    ("moe_unpermute", INVALID, dict(out=C)), ("moe_unpermute", INVALID, dict(out=B + 16)),
    ("moe_unpermute_backward", INVALID, dict(dw=D)), ("moe_unpermute_backward", INVALID, dict(dw=C)),
    ("moe_unpermute_backward", INVALID, dict(drows=C)),
    ("moe_unpermute_backward", INVALID, dict(drows=D, dw=None)),
    ("moe_quantize_mxfp4", INVALID, dict(codes=B)), ("moe_quantize_mxfp4", INVALID, dict(scales=B)),
    ("moe_mxfp4_gemm", INVALID, dict(out=C)), ("moe_mxfp4_gemm", INVALID, dict(out=D)),
    ("moe_mxfp4_gemm", INVALID, dict(out=E_)), ("moe_mxfp4_gemm", INVALID, dict(out=G)),
    ("moe_mxfp4_gemm", INVALID, dict(workspace=A)),
    ("moe_quantize_mxfp4", INVALID, dict(inv=None)), ("moe_quantize_mxfp4", INVALID, dict(x=None)),
    ("moe_quantize_mxfp4", INVALID, dict(scale_layout="col")),
    ("moe_quantize_mxfp4", INVALID, dict(T=0)), ("moe_quantize_mxfp4", INVALID, dict(codes=A)),
    ("moe_quantize_mxfp4", INVALID, dict(scales=C)),
    ("moe_quantize_mxfp4", UNSUPPORTED, dict(K=48)),
    ("moe_quantize_mxfp4", ALIGNMENT, dict(scales=D + 2)),
    ("moe_quantize_mxfp4", ALIGNMENT, dict(codes=C + 8)),
    ("moe_quantize_mxfp4", ALIGNMENT, dict(x=A + 16)),
    ("moe_quantize_mxfp4", UNSUPPORTED, dict(T=1, k=1, inv=None, K=(1 << 28) + 32)),
    ("moe_dequantize_mxfp4", ALIGNMENT, dict(out=C + 16)),
    ("moe_dequantize_mxfp4", UNSUPPORTED, dict(R=1, K=(1 << 28) + 32)),
    ("moe_dequantize_mxfp4", INVALID, dict(R=0)), ("moe_dequantize_mxfp4", INVALID, dict(out=A)),
    ("moe_dequantize_mxfp4", INVALID, dict(out=B)), ("moe_dequantize_mxfp4", INVALID, dict(scales=None)),
    ("moe_dequantize_mxfp4", UNSUPPORTED, dict(K=16)),
    ("moe_dequantize_mxfp4", ALIGNMENT, dict(out=C + 4)),
    ("moe_mxfp4_prepack", INVALID, dict(w=None)), ("moe_mxfp4_prepack", INVALID, dict(E=0)),
    ("moe_mxfp4_prepack", UNSUPPORTED, dict(E=257)), ("moe_mxfp4_prepack", UNSUPPORTED, dict(N=12)),
    ("moe_mxfp4_prepack", UNSUPPORTED, dict(K=40)), ("moe_mxfp4_prepack", ALIGNMENT, dict(w=A + 8)),
    ("moe_mxfp4_prepack", INVALID, dict(w_tiled=A)), ("moe_mxfp4_prepack", INVALID, dict(w_tiled=B)),
    ("moe_mxfp4_prepack", INVALID, dict(w_scales_chunked=C)),
    ("moe_mxfp4_gemm", INVALID, dict(offsets=None)), ("moe_mxfp4_gemm", INVALID, dict(workspace=None)),
    ("moe_mxfp4_gemm", INVALID, dict(R=0)), ("moe_mxfp4_gemm", INVALID, dict(dtype="fp8")),
    ("moe_mxfp4_gemm", UNSUPPORTED, dict(dtype="fp32")), ("moe_mxfp4_gemm", UNSUPPORTED, dict(N=4)),
    ("moe_mxfp4_gemm", UNSUPPORTED, dict(K=16)), ("moe_mxfp4_gemm", UNSUPPORTED, dict(E=300)),
    ("moe_mxfp4_gemm", INVALID, dict(out=A)), ("moe_mxfp4_gemm", INVALID, dict(out=B)),
    ("moe_mxfp4_gemm", ALIGNMENT, dict(workspace=G + 128)),
    ("moe_mxfp4_gemm", ALIGNMENT, dict(codes=A + 8)), ("moe_mxfp4_gemm", ALIGNMENT, dict(out=F_ + 2)),
]


@pytest.mark.parametrize("fn,status,over", CASES,
                         ids=[f"{f[4:]}-{'-'.join(map(str, o))}-{i}" for i, (f, _, o) in enumerate(CASES)])
def test_refused(fn, status, over):
    _refused(status, fn, **over)


def test_tensors_on_the_cpu_are_refused():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    _refused(INVALID, "moe_permute", x=x)
    _refused(INVALID, "moe_unpermute", out=x)
    _refused(INVALID, "moe_quantize_mxfp4", x=x)
    _refused(INVALID, "moe_mxfp4_gemm", codes=torch.zeros(8, 32, dtype=torch.uint8))


def test_other_objects_are_a_type_error():
    import numpy as np
    with pytest.raises(TypeError):
        moe.moe_permute(np.zeros(4), 1, 16, 1, B, C, stream=0)


def test_default_stream_without_a_gpu():
    """No stream given: the refusal is the library's, with or without CUDA in torch."""
    with pytest.raises(moe.MoEError) as e:
        moe.moe_permute(A, 4, 255, 2, B, C)
    assert e.value.status == UNSUPPORTED


def test_sizes_that_do_not_fit_are_refused():
    _refused(INVALID, "moe_unpermute", T=(1 << 32) + 4)
    _refused(INVALID, "moe_mxfp4_gemm", K=(1 << 32) + 64)


def test_sizes_of_prepacked_weights():
    assert moe.moe_mxfp4_weight_bytes(3, 136, 288) == 3 * 2 * 2 * 16384
    assert moe.moe_mxfp4_weight_scale_bytes(3, 128, 288) == 3 * 1 * 2 * 1024
    for E, N, K in ((0, 128, 256), (257, 128, 256), (1, 12, 256), (1, 128, 48), (1, 0, 256),
                    (1, 128, 0), (1, -8, 256), (1, (1 << 20) + 8, 256), (1, 8, (1 << 20) + 32)):
        assert moe.moe_mxfp4_weight_bytes(E, N, K) == 0
        assert moe.moe_mxfp4_weight_scale_bytes(E, N, K) == 0
        assert moe.moe_mxfp4_workspace_bytes(4, E, N, K) == 0
    assert moe.moe_mxfp4_workspace_bytes(0, 1, 128, 256) == 0
    assert moe.moe_mxfp4_workspace_bytes(1, 1, 128, 256) >= 256


def test_debug_flags_of_the_product():
    for flags in (2, -1, 1 << 20):
        with pytest.raises(moe.MoEError) as e:
            moe.moe_mxfp4_set_debug(flags)
        assert e.value.status == INVALID
    moe.moe_mxfp4_set_debug(0)


# Sizes whose products pass 2^31, as NumPy integers of 32 bits: in their own arithmetic
# the buffers' lengths would wrap around to zero and short tensors pass for whole ones.
WRAPPING = [
    ("moe_permute", dict(x="u8", T=1 << 12, row_bytes=1 << 20, k=2, inv="i32", rows="u8"), "x"),
    ("moe_permute_backward", dict(drows="bf16", dtype="bf16", T=1 << 12, H=1 << 19, k=2, inv="i32",
                                  dx="bf16"), "drows"),
    ("moe_unpermute", dict(rows="bf16", dtype="bf16", T=1 << 12, H=1 << 19, k=2, inv="i32",
                           topk_w="f32", out="bf16"), "rows"),
    ("moe_unpermute_backward", dict(dout="bf16", rows="bf16", dtype="bf16", T=1 << 12, H=1 << 19, k=2,
                                    inv="i32", topk_w="f32", drows="bf16", dw="f32"), "dout"),
    ("moe_quantize_mxfp4", dict(x="bf16", dtype="bf16", T=1 << 12, K=1 << 21, k=1, inv=None, codes="u8",
                                scales="u8", scale_layout="group"), "x"),
    ("moe_dequantize_mxfp4", dict(codes="u8", scales="u8", scale_layout="row", R=1 << 12, K=1 << 25,
                                  dtype="bf16", out="bf16"), "codes"),
    ("moe_mxfp4_prepack", dict(w="u8", w_scales="u8", E=1 << 8, N=1 << 10, K=1 << 15, w_tiled="u8",
                               w_scales_chunked="u8"), "w"),
    ("moe_mxfp4_gemm", dict(codes="u8", scales="u8", offsets="i32", R=1 << 20, E=2, N=1 << 12, K=1 << 13,
                            w_tiled="u8", w_scales_chunked="u8", dtype="bf16", out="bf16",
                            workspace="u8"), "codes"),
]


@pytest.mark.parametrize("fn,args,first", WRAPPING, ids=[w[0][4:] for w in WRAPPING])
def test_sizes_as_numpy_integers_do_not_wrap(fn, args, first, monkeypatch):
    import numpy as np
    monkeypatch.setattr(moe, "_here", lambda stream: (-1, 0))      # tensors of the CPU pass for the GPU's
    kinds = {"u8": torch.uint8, "i32": torch.int32, "f32": torch.float32, "bf16": torch.bfloat16}
    long = [a for a, v in args.items() if v in ("i32", "f32")]
    call = {a: torch.zeros(1 << 14 if a in long else 64, dtype=kinds[v]) if v in kinds and a != "dtype" else v
            for a, v in args.items()}
    for a, v in args.items():
        if isinstance(v, int):
            call[a] = np.int32(v)
    with pytest.raises(moe.MoEError) as e:
        getattr(moe, fn)(**call)
    assert e.value.status == INVALID and f"{first} holds" in str(e.value), e.value


def test_sizes_as_numpy_integers_are_taken():
    import numpy as np
    for n in (np.int32, np.int64, np.uint8, torch.tensor):
        _refused(UNSUPPORTED, "moe_unpermute", T=n(4), H=n(20), k=n(2))
        _refused(UNSUPPORTED, "moe_mxfp4_gemm", R=n(8), K=n(48))
        _refused(INVALID, "moe_permute", T=n(0))
    _refused(INVALID, "moe_unpermute", T=np.int64(1 << 31))
    _refused(INVALID, "moe_unpermute", H=np.int64(-8))


def test_row_bytes_past_64_bits_are_refused():
    """(1 << 64) + 255 would reach the library as 255, a size it refuses for another reason."""
    for row_bytes in ((1 << 64) + 255, (1 << 63) + 1, -(1 << 64) + 255, -4):
        _refused(INVALID, "moe_permute", row_bytes=row_bytes)


@pytest.mark.parametrize("fn", [moe.moe_mxfp4_clear_error, moe.moe_mxfp4_check_error],
                         ids=["clear", "check"])
def test_error_word_of_a_tensor_that_is_no_workspace(fn, monkeypatch):
    """One on the CPU, one shorter than the 256 bytes that are written, one with gaps."""
    with pytest.raises(moe.MoEError) as e:
        fn(torch.zeros(256, dtype=torch.uint8))
    assert e.value.status == INVALID
    monkeypatch.setattr(moe, "_here", lambda stream: (-1, 0))      # tensors of the CPU pass for the GPU's
    for t in (torch.zeros(255, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)[::2]):
        with pytest.raises(moe.MoEError) as e:
            fn(t)
        assert e.value.status == INVALID


def test_scale_shapes():
    assert moe.mxfp4_scale_shape(5, 288, "row") == (5, 9)
    assert moe.mxfp4_scale_shape(5, 288, "group") == (3, 5, 4)
    for layout in ("rows", "row-major", 0, None):
        with pytest.raises(moe.MoEError) as e:
            moe.mxfp4_scale_shape(5, 288, layout)
        assert e.value.status == INVALID
