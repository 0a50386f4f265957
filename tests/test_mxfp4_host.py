"""Refusals of the MXFP4 and expert-layer entry points, on the CPU: no call here validates, so none launches."""
import ctypes

import pytest
import torch

from weight_only_quantized_int8_amd import Mxfp4Weight, moe_layer
from weight_only_quantized_int8_amd import binding as B

A = 1 << 20  # fake, 256-byte aligned "device" addresses, never dereferenced


def mx(rows=64, k=256, codes=A, scales=2 * A):
    return B.Mxfp4Desc(codes, scales, rows, k)


def err(rc):
    assert rc != B.INT8W_OK
    return rc, B.load_library().int8w_last_error().decode()


@pytest.mark.parametrize("d,code,text", [
    (mx(codes=0), B.INT8W_ERR_NULL, "missing a tensor"),
    (mx(scales=0), B.INT8W_ERR_NULL, "missing a tensor"),
    (mx(rows=0), B.INT8W_ERR_SHAPE, "zero dimension"),
    (mx(k=0), B.INT8W_ERR_SHAPE, "zero dimension"),
    (mx(k=48), B.INT8W_ERR_SHAPE, "not a multiple of 32"),
    (mx(k=1 << 22), B.INT8W_ERR_SHAPE, "too large"),
    (mx(rows=1 << 24, k=1 << 16), B.INT8W_ERR_SHAPE, "too large"),
    (mx(codes=A + 8), B.INT8W_ERR_ALIGN, "not 16-byte aligned"),
])
def test_a_bad_matrix_is_refused_everywhere(d, code, text):
    for call in (lambda: B.int8w_mxfp4_dequantize_to(d, 4 * A, 0), lambda: B.int8w_mxfp4_gemm(d, 4 * A, 5 * A, 3, 0),
                 lambda: B.int8w_mxfp4_gemm_mx(d, mx(codes=6 * A, scales=7 * A), 5 * A, 0),
                 lambda: B.int8w_mxfp4_moe_layer(d, d, d, 1, moe_call(), 9 * A, 1 << 30, 0),
                 lambda: B.int8w_mxfp4_quantize(4 * A, 0, d.rows, d.k, d.codes, d.scales, 0)):
        if d.rows == 0 and call.__code__.co_names[1] == "int8w_mxfp4_quantize":
            continue  # no rows: nothing to do there
        rc, msg = err(call())
        assert rc == code and text in msg, (rc, msg)


@pytest.mark.parametrize("call,code,text", [
    (lambda: B.int8w_mxfp4_quantize(0, 0, 4, 64, A, 2 * A, 0), B.INT8W_ERR_NULL, "x is NULL"),
    (lambda: B.int8w_mxfp4_quantize(A, 2, 4, 64, 2 * A, 3 * A, 0), B.INT8W_ERR_UNSUPPORTED, "x_format"),
    (lambda: B.int8w_mxfp4_quantize(A + 4, 0, 4, 64, 2 * A, 3 * A, 0), B.INT8W_ERR_ALIGN, "x is not"),
    (lambda: B.int8w_mxfp4_quantize(A, 0, 4, 64, A + 256, 3 * A, 0), B.INT8W_ERR_ALIAS, "overlaps"),
    (lambda: B.int8w_mxfp4_quantize(A, 1, 4, 64, A + 1008, 3 * A, 0), B.INT8W_ERR_ALIAS, "overlaps"),
    (lambda: B.int8w_mxfp4_quantize(A, 0, 4, 64, 2 * A, 2 * A + 100, 0), B.INT8W_ERR_ALIAS, "overlap"),
    (lambda: B.int8w_mxfp4_dequantize_to(mx(), 0, 0), B.INT8W_ERR_NULL, "out is NULL"),
    (lambda: B.int8w_mxfp4_dequantize_to(mx(), 4 * A + 8, 0), B.INT8W_ERR_ALIGN, "out is not"),
    (lambda: B.int8w_mxfp4_dequantize_to(mx(), A + 4096, 0), B.INT8W_ERR_ALIAS, "overlaps"),
    (lambda: B.int8w_mxfp4_gemm(mx(), 0, 5 * A, 1, 0), B.INT8W_ERR_NULL, "X or Y is NULL"),
    (lambda: B.int8w_mxfp4_gemm(mx(), 4 * A + 2, 5 * A, 1, 0), B.INT8W_ERR_ALIGN, "X is not"),
    (lambda: B.int8w_mxfp4_gemm(mx(), 4 * A, 5 * A + 1, 1, 0), B.INT8W_ERR_ALIGN, "Y is not"),
    (lambda: B.int8w_mxfp4_gemm(mx(), 4 * A, 2 * A + 2, 1, 0), B.INT8W_ERR_ALIAS, "scales"),
    (lambda: B.int8w_mxfp4_gemm(mx(), 4 * A, 4 * A + 16, 1, 0), B.INT8W_ERR_ALIAS, "input X"),
    (lambda: B.int8w_mxfp4_gemm(mx(), 4 * A, 5 * A, 1 << 25, 0), B.INT8W_ERR_SHAPE, "too many"),
    (lambda: B.int8w_mxfp4_gemm_mx(mx(), mx(k=512), 5 * A, 0), B.INT8W_ERR_SHAPE, "k=512"),
    (lambda: B.int8w_mxfp4_gemm_mx(mx(), mx(codes=0), 5 * A, 0), B.INT8W_ERR_NULL, "missing"),
    (lambda: B.int8w_mxfp4_gemm_mx(mx(), mx(codes=6 * A, scales=7 * A), 0, 0), B.INT8W_ERR_NULL, "Y is NULL"),
    (lambda: B.int8w_mxfp4_gemm_mx(mx(), mx(codes=6 * A, scales=7 * A), 7 * A, 0), B.INT8W_ERR_ALIAS, "X scales"),
])
def test_calls_are_refused(call, code, text):
    rc, msg = err(call())
    assert rc == code and text in msg, (rc, msg)


def test_nothing_to_do_is_ok():
    assert B.int8w_mxfp4_gemm(mx(), 0, 0, 0, 0) == B.INT8W_OK
    assert B.int8w_mxfp4_gemm_mx(mx(), mx(rows=0, codes=0, scales=0), 0, 0) == B.INT8W_OK
    assert B.int8w_mxfp4_quantize(0, 0, 0, 64, 0, 0, 0) == B.INT8W_OK
    g, u, d = layer()
    assert B.int8w_mxfp4_moe_layer(g, u, d, 4, moe_call(tokens=0), 0, 0, 0) == B.INT8W_OK


E, I, H = 4, 96, 64


def layer(e=E, i=I, h=H):
    return (mx(e * i, h, 10 * A, 11 * A), mx(e * i, h, 12 * A, 13 * A), mx(e * h, i, 14 * A, 15 * A))


def moe_call(x=20 * A, logits=21 * A, resid=None, y=22 * A, tokens=3, topk=2, fmt=B.VALUES_F32):
    return B.MoeCall(x, logits, resid, y, tokens, topk, fmt, 1, 1.0)


WS, BIG = 30 * A, 1 << 19


@pytest.mark.parametrize("w,n,call,ws,nbytes,code,text", [
    (layer(), 0, moe_call(), WS, BIG, B.INT8W_ERR_SHAPE, "num_experts"),
    (layer(), 513, moe_call(), WS, BIG, B.INT8W_ERR_SHAPE, "num_experts"),
    (layer(), 3, moe_call(), WS, BIG, B.INT8W_ERR_SHAPE, "not 3 experts"),
    ((layer()[0], layer(i=128)[1], layer()[2]), E, moe_call(), WS, BIG, B.INT8W_ERR_SHAPE, "up is not"),
    ((*layer()[:2], layer(h=96)[2]), E, moe_call(), WS, BIG, B.INT8W_ERR_SHAPE, "down"),
    (layer(), E, moe_call(topk=0), WS, BIG, B.INT8W_ERR_SHAPE, "topk"),
    (layer(), E, moe_call(topk=5), WS, BIG, B.INT8W_ERR_SHAPE, "topk"),
    (layer(e=32), 32, moe_call(topk=17), WS, BIG, B.INT8W_ERR_SHAPE, "topk"),
    (layer(), E, moe_call(fmt=2), WS, BIG, B.INT8W_ERR_UNSUPPORTED, "logits_format"),
    (layer(), E, moe_call(x=0), WS, BIG, B.INT8W_ERR_NULL, "NULL"),
    (layer(), E, moe_call(logits=0), WS, BIG, B.INT8W_ERR_NULL, "NULL"),
    (layer(), E, moe_call(y=0), WS, BIG, B.INT8W_ERR_NULL, "NULL"),
    (layer(), E, moe_call(), 0, BIG, B.INT8W_ERR_NULL, "NULL"),
    (layer(), E, moe_call(x=20 * A + 8), WS, BIG, B.INT8W_ERR_ALIGN, "x is not"),
    (layer(), E, moe_call(logits=21 * A + 2), WS, BIG, B.INT8W_ERR_ALIGN, "logits"),
    (layer(), E, moe_call(), WS + 16, BIG, B.INT8W_ERR_ALIGN, "workspace"),
    (layer(), E, moe_call(), WS, 1024, B.INT8W_ERR_SHAPE, "workspace of 1024"),
    (layer(), E, moe_call(y=20 * A), WS, BIG, B.INT8W_ERR_ALIAS, "input x"),
    (layer(), E, moe_call(resid=22 * A + 2), WS, BIG, B.INT8W_ERR_ALIAS, "x_resid"),
    (layer(), E, moe_call(y=WS + 64), WS, BIG, B.INT8W_ERR_ALIAS, "workspace"),
    (layer(), E, moe_call(y=14 * A), WS, BIG, B.INT8W_ERR_ALIAS, "codes"),
])
def test_layer_calls_are_refused(w, n, call, ws, nbytes, code, text):
    rc, msg = err(B.int8w_mxfp4_moe_layer(*w, n, call, ws, nbytes, 0))
    assert rc == code and text in msg, (rc, msg)


def test_int8_layer_refuses_mixed_group_sizes_and_null():
    def w(rows, k, gs, at):
        return B.WeightDesc(at, at + A, at + 2 * A, rows, k, gs)
    g, u, d = w(E * 128, 256, 64, 40 * A), w(E * 128, 256, 64, 44 * A), w(E * 256, 128, 64, 48 * A)
    u32 = w(E * 128, 256, 32, 44 * A)
    rc, msg = err(B.int8_moe_layer(g, u32, d, E, moe_call(), WS, BIG, 0))
    assert rc == B.INT8W_ERR_SHAPE and "group sizes" in msg
    rc, msg = err(B.int8_moe_layer(g, u, d, E, ctypes.POINTER(B.MoeCall)(), WS, BIG, 0))
    assert rc == B.INT8W_ERR_NULL and "call is NULL" in msg


def test_workspace_bytes_grow_with_the_pass_and_stop_at_it():
    f = B.int8w_moe_workspace_bytes
    assert f(0, 2, 64, 64) == 0
    assert f(2, 2, 64, 32) - f(1, 2, 64, 32) == 2 * (64 * 2 + 32 * 4)
    assert f(64, 4, 96, 32) == f(1000, 4, 96, 32)


def test_python_checks():
    u8, bf = torch.uint8, torch.bfloat16
    with pytest.raises(ValueError, match="2-D uint8"):
        Mxfp4Weight(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4, 2, dtype=u8))
    with pytest.raises(ValueError, match="multiple of 32"):
        Mxfp4Weight(torch.zeros(4, 24, dtype=u8), torch.zeros(4, 1, dtype=u8))
    with pytest.raises(ValueError, match="scales must be"):
        Mxfp4Weight(torch.zeros(4, 32, dtype=u8), torch.zeros(4, 3, dtype=u8))
    with pytest.raises(ValueError, match="contiguous"):
        Mxfp4Weight(torch.zeros(4, 64, dtype=u8)[:, ::2], torch.zeros(4, 2, dtype=u8))
    with pytest.raises(ValueError, match="on one GPU"):
        Mxfp4Weight(torch.zeros(4, 32, dtype=u8), torch.zeros(4, 2, dtype=u8))
    for bad in (torch.zeros(4, 64, dtype=torch.float16), torch.zeros(64, dtype=bf), torch.zeros(4, 64, dtype=bf)):
        with pytest.raises(ValueError, match="GPU tensor"):
            Mxfp4Weight.quantize(bad)
    with pytest.raises(TypeError, match="three Int8Weight or three Mxfp4Weight"):
        moe_layer(None, None, None, 4, torch.zeros(1, 64, dtype=bf), torch.zeros(1, 4), 2)


def host_matrix(rows, k):
    """An Mxfp4Weight on the CPU: enough for the checks that come before a launch."""
    codes, scales = torch.zeros(rows, k // 2, dtype=torch.uint8), torch.zeros(rows, k // 32, dtype=torch.uint8)
    w = Mxfp4Weight.__new__(Mxfp4Weight)
    w._set(codes, scales, rows, k, codes.device, codes.data_ptr(), scales.data_ptr())
    return w


@pytest.mark.parametrize("topk", [-(1 << 31), -1, 0, 5, 17, 1 << 20, (1 << 32) + 1])
def test_a_wrong_topk_is_refused_before_it_sizes_the_scratch(topk, monkeypatch):
    monkeypatch.setattr(B, "int8w_moe_workspace_bytes", lambda *a: pytest.fail(f"scratch sized for topk {topk}"))
    gate, up, down = host_matrix(E * I, H), host_matrix(E * I, H), host_matrix(E * H, I)
    with pytest.raises(B.Int8wError, match="topk") as e:
        moe_layer(gate, up, down, E, torch.zeros(3, H, dtype=torch.bfloat16), torch.zeros(3, E), topk)
    assert e.value.code == B.INT8W_ERR_SHAPE


def test_dequantizing_no_rows_gives_no_rows():
    q = host_matrix(0, 64)
    y = q.dequantize_to()
    assert y.shape == (0, 64) and y.dtype == torch.bfloat16
    out = torch.ones(5, dtype=torch.bfloat16)
    assert q.dequantize_to(out) is out and (out == 1).all()
    with pytest.raises(TypeError, match="bfloat16"):
        q.dequantize_to(torch.ones(5))


def test_streams_without_the_private_torch_function(monkeypatch):
    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: Stream(1000 + index))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert B._stream_of(torch.device("cuda", 1)) == 1001
    assert B._stream_of(torch.device("cuda")) == 1003
