"""Host-side refusals of the MXFP4 and expert-order row entry points (no GPU,
nothing is launched)."""
import ctypes
import pathlib
import types

import numpy as np
import pytest
import torch

NULL = None
FAKE, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4100)   # never dereferenced: every call fails its checks


@pytest.fixture(scope="module")
def m():
    import mixture_experts_layer_lds_amd as mod
    return mod


def test_layouts(m):
    # decode: x codes, h blocks of max_tasks 16-row tiles, no down rows at one token
    for T, k, E, H, I in ((1, 8, 256, 7168, 2048), (16, 8, 256, 7168, 2048), (4096, 8, 256, 7168, 2048), (300, 2, 4, 384, 640)):
        R, W = m.moe_routing_layout(T, k, E, H, I, "mxfp4"), m.moe_workspace_layout(T, k, E, H, I, "mxfp4")
        none = 2 ** 64 - 1
        assert W["xq"] == 0 and W["x_scale"] >= T * H // 2 and W["h"] >= W["x_scale"] + T * H // 32
        assert W["g"] == W["h_scale"] == W["x_scale_rows"] == none
        end = W["h"] + R["max_tasks"] * R["block_m"] * I * 17 // 32
        if T == 1:
            assert W["y"] == none and end <= W["total_bytes"]
        else:
            assert W["y"] >= end and W["y"] + 2 * T * k * H <= W["total_bytes"]
        assert all(W[n] == none or W[n] % 256 == 0 for n in ("xq", "x_scale", "h", "y"))
        assert R["max_tasks"] == T * k // R["block_m"] + min(E, T * k)
    for bad in ((4, 2, 8, 64, 128), (4, 2, 8, 128, 192), (8193, 8, 8, 128, 128)):
        with pytest.raises(m.MoeError) as e:
            m.moe_workspace_layout(*bad, "mxfp4")
        assert e.value.status == -2


def test_quantize_refusals(m):
    q, d = m._lib.moe_quantize_mxfp4, m._lib.moe_dequantize_mxfp4
    assert q(FAKE, 3, 4, 64, 64, FAKE, FAKE, NULL) == -1      # no such row type
    assert q(FAKE, -1, 4, 64, 64, FAKE, FAKE, NULL) == -1
    assert q(FAKE, 0, -1, 64, 64, FAKE, FAKE, NULL) == -1
    assert q(FAKE, 0, 4, 0, 64, FAKE, FAKE, NULL) == -1
    assert q(FAKE, 0, 4, 64, 32, FAKE, FAKE, NULL) == -1      # rows would overlap
    assert q(FAKE, 0, 4, 48, 64, FAKE, FAKE, NULL) == -2
    assert q(FAKE, 0, 4, 64, 68, FAKE, FAKE, NULL) == -2      # rows not 16-byte aligned
    assert q(FAKE, 0, 0, 64, 64, NULL, NULL, NULL) == 0
    for args in ((NULL, FAKE, FAKE), (FAKE, NULL, FAKE), (FAKE, FAKE, NULL), (ODD, FAKE, FAKE)):
        assert q(args[0], 0, 4, 64, 64, args[1], args[2], NULL) == -1
    assert q(FAKE, 0, 4, 64, 64, ctypes.c_void_p(4098), FAKE, NULL) == -1
    assert d(FAKE, FAKE, 4, 48, 0, FAKE, NULL) == -2 and d(FAKE, FAKE, 4, 64, 5, FAKE, NULL) == -1
    assert d(FAKE, FAKE, 4, 64, 0, ODD, NULL) == -1 and d(NULL, FAKE, 4, 64, 0, FAKE, NULL) == -1
    assert d(NULL, NULL, 0, 64, 0, NULL, NULL) == 0


def test_pack_and_forward_refusals(m):
    lib = m._lib
    desc = m.PackedWeightsDesc()
    D = ctypes.byref(desc)
    big = ctypes.c_void_p(1 << 30)
    pack = lib.moe_pack_weights_mxfp4
    assert pack(FAKE, FAKE, 8, 256, 128, big, NULL, NULL) == -1
    assert pack(FAKE, FAKE, 8, 48, 128, big, D, NULL) == -2 and pack(FAKE, FAKE, 8, 64, 192, big, D, NULL) == -2
    assert pack(FAKE, FAKE, 0, 64, 128, big, D, NULL) == -1
    assert pack(NULL, FAKE, 8, 64, 128, big, D, NULL) == -1 and pack(FAKE, NULL, 8, 64, 128, big, D, NULL) == -1
    assert pack(FAKE, FAKE, 8, 64, 128, NULL, D, NULL) == -1 and pack(ODD, FAKE, 8, 64, 128, big, D, NULL) == -1
    assert pack(FAKE, big, 8, 64, 128, FAKE, D, NULL) == -1                                   # codes overlap
    assert pack(big, ctypes.c_void_p(4096 + 64), 8, 64, 128, FAKE, D, NULL) == -1             # scales overlap
    assert desc.data is None and desc.check == 0
    # the generic pack has no scales to pack
    assert lib.moe_pack_weights(FAKE, 8, 64, 128, m.MOE_DTYPE_MXFP4, big, D, NULL) == -1

    E, H, I, T, k = 8, 128, 128, 4, 2

    def describe(rows, cols, dtype):
        d = m.PackedWeightsDesc()
        assert lib.moe_describe_packed_weights(FAKE, E, rows, cols, m.DTYPES[dtype], ctypes.byref(d)) == 0
        return ctypes.byref(d)

    w1, w2, f1 = describe(2 * I, H, "mxfp4"), describe(H, I, "mxfp4"), describe(2 * I, H, "fp8")
    n, W = m.moe_routing_layout(T, k, E, H, I, "mxfp4")["total_bytes"], m.moe_workspace_layout(T, k, E, H, I, "mxfp4")["total_bytes"]
    fwd, rfw, bld = lib.moe_forward_mxfp4, lib.moe_route_forward_mxfp4, lib.moe_build_routing_mxfp4
    good = [FAKE, FAKE, FAKE, w1, w2, T, k, E, H, I, FAKE, W, FAKE, NULL]
    for at, value, code in ((0, NULL, -1), (1, NULL, -1), (2, NULL, -1), (3, NULL, -1), (3, f1, -1), (3, w2, -1), (4, w1, -1),
                            (10, NULL, -1), (10, ODD, -1), (11, W - 1, -3), (12, NULL, -1), (12, ODD, -1), (8, 192, -2), (9, 64, -2),
                            (6, 17, -1), (5, -1, -1), (7, 0, -1)):
        a = list(good)
        a[at] = value
        assert fwd(*a) == code, (at, value)
        b = [FAKE, a[0], a[1], a[2], n, *a[3:]]
        assert rfw(*b) == code, (at, value)
    assert fwd(*[NULL] * 5, 0, k, E, H, I, NULL, 0, NULL, NULL) == 0
    assert rfw(*[FAKE, FAKE, FAKE, FAKE, n - 1], *good[3:]) == -3 and rfw(NULL, FAKE, FAKE, FAKE, n, *good[3:]) == -1
    assert bld(FAKE, T, k, E, H, I, FAKE, n - 1, NULL) == -3 and bld(FAKE, T, k, E, 192, I, FAKE, n, NULL) == -2
    # MXFP4 weights do not pass for another dtype's
    assert lib.moe_forward_mxfp8(FAKE, FAKE, FAKE, w1, FAKE, w2, FAKE, T, k, E, H, I, FAKE, 1 << 30, FAKE, NULL) == -1


def test_row_operator_refusals(m):
    lib = m._lib
    T, k, E, H = 4, 2, 8, 64
    n = m.moe_routing_layout(T, k, E, 128, 128, "bf16")["tasks"]
    for name in ("moe_dispatch", "moe_combine"):
        f = getattr(lib, name)
        good = [FAKE, 0, FAKE, FAKE, n, T, k, E, H, FAKE, NULL]
        for at, value, code in ((0, NULL, -1), (0, ODD, -1), (1, 3, -1), (1, -1, -1), (2, ctypes.c_void_p(4098), -1), (3, NULL, -1), (3, ODD, -1),
                                (4, n - 1, -3), (5, -1, -1), (5, 40000, -2), (6, 0, -1), (6, 17, -1), (7, 0, -1), (7, 512, -1), (8, 0, -1),
                                (8, 12, -2), (8, 65544, -2), (9, NULL, -1), (9, ODD, -1)):
            a = list(good)
            a[at] = value
            assert f(*a) == code, (name, at, value)
        assert f(NULL, 0, NULL, NULL, 0, 0, k, E, H, NULL, NULL) == 0
    for name in ("moe_dispatch_grad", "moe_combine_grad"):
        f = getattr(lib, name)
        good = [FAKE, FAKE, 0, FAKE, FAKE, n, T, k, E, H, FAKE, FAKE, NULL]
        for at, value, code in ((0, NULL, -1), (1, NULL, -1), (1, ODD, -1), (2, 7, -1), (3, NULL, -1), (4, NULL, -1), (5, n - 1, -3),
                                (9, 12, -2), (10, NULL, -1), (11, ctypes.c_void_p(4097), -1)):
            a = list(good)
            a[at] = value
            assert f(*a) == code, (name, at, value)
        # without the weights' gradient the second operand is not needed, the rest still is
        assert f(FAKE, NULL, 0, NULL, FAKE, n, T, k, E, H, NULL, NULL, NULL) == -1
    g = lib.moe_router_topk_grad
    good = [FAKE, FAKE, FAKE, FAKE, T, E, k, 1, 0, FAKE, NULL]
    for at, value, code in ((1, NULL, -1), (2, NULL, -1), (3, NULL, -1), (4, -1, -1), (5, 0, -1), (5, 257, -2), (6, 0, -1), (6, 9, -1),
                            (7, 2, -1), (8, -1, -1), (8, 15, -2), (9, NULL, -1), (9, ctypes.c_void_p(4097), -1)):
        a = list(good)
        a[at] = value
        assert g(*a) == code, (at, value)
    assert g(NULL, FAKE, FAKE, FAKE, T, E, k, 0, 0, FAKE, NULL) == -1      # the full softmax needs the scores
    assert g(NULL, NULL, NULL, NULL, 0, E, k, 1, 0, NULL, NULL) == 0


def test_counts_past_the_launch_limits(m):
    lib = m._lib
    # rows of 2^38 bytes and more
    for rows, cols, row_type in ((1 << 32, 32, 0), (1 << 31, 32, 2), (1 << 62, 64, 0), (64, 1 << 30, 2), ((1 << 63) - 1, 32, 1)):
        assert lib.moe_quantize_mxfp4(FAKE, row_type, rows, cols, cols, FAKE, FAKE, NULL) == -2, (rows, cols)
        assert lib.moe_dequantize_mxfp4(FAKE, FAKE, rows, cols, row_type, FAKE, NULL) == -2, (rows, cols)
    for T in ((1 << 25) + 1, (1 << 31) - 1):
        assert lib.moe_router_topk_grad(FAKE, FAKE, FAKE, FAKE, T, 8, 2, 1, 0, FAKE, NULL) == -2


def test_binding_refuses_wrong_tensors(m):
    """Shapes, types, strides and devices are refused before the library is called."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    r = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="current GPU"):
        m.moe_quantize_mxfp4(x)
    with pytest.raises(ValueError, match="current GPU"):
        m.moe_dispatch(x, r, 2, 8)
    with pytest.raises(ValueError, match="32 values"):
        m.moe_quantize_mxfp4(x[:, :48])
    with pytest.raises(ValueError, match="contiguous rows"):
        m.moe_quantize_mxfp4(torch.zeros(64, 64).t()[:, :32])
    with pytest.raises(ValueError, match="contiguous rows"):
        m.moe_quantize_mxfp4(torch.zeros(1, 64).expand(4, 64))
    with pytest.raises(ValueError, match="rows"):
        m.moe_quantize_mxfp4(x.double())
    with pytest.raises(ValueError, match="codes"):
        m.moe_dequantize_mxfp4(torch.zeros(4, 24, dtype=torch.uint8), r)
    with pytest.raises(ValueError, match="scales"):
        m.moe_pack_weights_mxfp4(torch.zeros(1, 32, 64, dtype=torch.uint8), torch.zeros(1, 32, 5, dtype=torch.uint8))
    with pytest.raises(ValueError, match="y: expected"):
        m.moe_combine(torch.zeros(7, 64), r, 2, 8)
    with pytest.raises(ValueError, match="topk_w"):
        m.moe_dispatch(x, r, 2, 8, topk_w=torch.zeros(4, 3))
    with pytest.raises(ValueError, match="topk_w"):
        m.moe_dispatch_grad(torch.zeros(8, 64), r, 2, 8, x=torch.zeros(4, 64))
    with pytest.raises(ValueError, match="dtopk_w needs"):
        m.moe_combine_grad(torch.zeros(4, 64), r, 2, 8, topk_w=torch.zeros(4, 2), dtopk_w=torch.zeros(4, 2))
    with pytest.raises(ValueError, match="x: expected"):
        m.moe_dispatch_grad(torch.zeros(8, 64), r, 2, 8, x=torch.zeros(5, 64), topk_w=torch.zeros(4, 2))
    with pytest.raises(ValueError, match="dtopk_w"):
        m.moe_router_topk_grad(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(4, 3))
    with pytest.raises(ValueError, match="packed MXFP4"):
        m.moe_describe_packed_weights(torch.zeros(1, 32, 64, dtype=torch.uint8), "mxfp4")


def test_sizes_past_32_bits_are_refused(m, monkeypatch):
    """Sizes whose low 32 bits are good ones: none may reach the library as those."""
    lib, over = m._lib, 1 << 32
    n = m.moe_routing_layout(4, 2, 8, 128, 128, "bf16")["total_bytes"]
    # of sizes that would return MOE_OK without a launch, or describe nothing
    for f, args in ((lib.moe_quantize_mxfp4, (FAKE, 0, 0, over + 64, over + 64, FAKE, FAKE, NULL)),
                    (lib.moe_dequantize_mxfp4, (FAKE, FAKE, 0, over + 64, 0, FAKE, NULL)),
                    (lib.moe_dispatch, (FAKE, 0, NULL, FAKE, n, over, 2, 8, 64, FAKE, NULL)),
                    (lib.moe_combine, (FAKE, 0, NULL, FAKE, n, 0, over + 2, 8, 64, FAKE, NULL)),
                    (lib.moe_dispatch_grad, (FAKE, NULL, 0, NULL, FAKE, n, 0, 2, over + 8, 64, FAKE, NULL, NULL)),
                    (lib.moe_combine_grad, (FAKE, NULL, 0, NULL, FAKE, n, 0, 2, 8, over + 64, FAKE, NULL, NULL)),
                    (lib.moe_router_topk_grad, (FAKE, FAKE, FAKE, FAKE, over, 8, 2, 1, 0, FAKE, NULL)),
                    (lib.moe_router_topk, (FAKE, over, 8, 2, 1, 0, FAKE, FAKE, NULL)),
                    (lib.moe_build_routing_mxfp4, (FAKE, over, 2, 8, 128, 128, FAKE, n, NULL)),
                    (lib.moe_build_routing_bf16, (FAKE, -over, 2, 8, 128, 128, FAKE, n, NULL)),
                    (lib.moe_forward_bf16, (FAKE, FAKE, FAKE, NULL, NULL, over, 2, 8, 128, 128, FAKE, n, FAKE, NULL))):
        with pytest.raises(ctypes.ArgumentError, match="32-bit"):
            f(*args)
    for f, args in ((m.moe_routing_layout, (over + 4, 2, 8, 128, 128)), (m.moe_workspace_layout, (4, 2, 8, over + 128, 128, "mxfp4")),
                    (m.alloc_routing, (4, 2, over + 8, 128, 128)), (m.moe_router_pair_bytes, (over + 8, 64))):
        with pytest.raises(ctypes.ArgumentError, match="32-bit"):
            f(*args)
    # through the binding, on tensors without memory
    monkeypatch.setattr(m, "_check_device", lambda *t: 0)
    monkeypatch.setattr(m, "_here", lambda dev, stream: None)
    r = torch.zeros(n, dtype=torch.uint8)
    rows = torch.empty(1, over + 64, dtype=torch.bfloat16, device="meta")
    tall = torch.empty(over + 4, 64, dtype=torch.bfloat16, device="meta")
    codes = torch.empty(1, over + 64, dtype=torch.uint8, device="meta")
    scores = torch.empty(over + 5, 1, device="meta")
    for f, args in ((m.moe_quantize_mxfp4, (rows,)),
                    (m.moe_dequantize_mxfp4, (codes, torch.empty(1, (over + 64) // 16, dtype=torch.uint8, device="meta"))),
                    (m.moe_dispatch, (tall, r, 1, 8)), (m.moe_combine, (tall, r, 1, 8)),
                    (m.moe_dispatch_grad, (tall, r, 1, 8)), (m.moe_combine_grad, (tall, r, 1, 8)),
                    (m.moe_router_topk_grad, (scores, torch.empty(over + 5, 1, dtype=torch.int32, device="meta"), scores, scores))):
        with pytest.raises(ctypes.ArgumentError, match="32-bit"):
            f(*args)
    # every size that fits still reaches the library's own checks, numpy's integers too
    assert lib.moe_router_topk_grad(FAKE, FAKE, FAKE, FAKE, (1 << 31) - 1, 8, 2, 1, 0, FAKE, NULL) == -2
    assert lib.moe_router_topk_grad(FAKE, FAKE, FAKE, FAKE, -(1 << 31), 8, 2, 1, 0, FAKE, NULL) == -1
    assert m.moe_routing_layout(np.int64(4), np.int32(2), 8, 128, 128) == m.moe_routing_layout(4, 2, 8, 128, 128)


def test_mxfp4_routing_refuses_host_tensors(m):
    # host ids would be read, and a host routing buffer written, by the kernel
    ids, r = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8)
    w = m.moe_describe_packed_weights(torch.zeros(8, 256, 68, dtype=torch.uint8), "mxfp4")
    for call in (lambda: m.moe_build_routing_mxfp4(ids, 8, 128, 128, r), lambda: m.build_routing(ids, 8, 128, 128, r, "mxfp4"),
                 lambda: m.moe_layer(torch.zeros(4, 128, dtype=torch.bfloat16), ids, torch.zeros(4, 2), {"w1": w, "w2": w}, "mxfp4")):
        with pytest.raises(ValueError, match="current GPU"):
            call()


def test_streams_of_another_gpu_are_refused(m, monkeypatch):
    # a launch goes to the current device, where the tensors are
    monkeypatch.setattr(m, "_check_device", lambda *t: 0)
    here, there = types.SimpleNamespace(device_index=0, cuda_stream=4096), types.SimpleNamespace(device_index=1, cuda_stream=4096)
    assert m._here(0, here) == 4096
    r = torch.zeros(4096, dtype=torch.uint8)
    x, y, w = torch.zeros(4, 64), torch.zeros(8, 64), torch.zeros(4, 2)
    ids, codes = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(1, 32, 64, dtype=torch.uint8)
    scales = torch.zeros(1, 32, 4, dtype=torch.uint8)
    for f, args in ((m.moe_quantize_mxfp4, (x, torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))),
                    (m.moe_dequantize_mxfp4, (codes, scales, None, torch.zeros(1, 32, 128))),
                    (m.moe_pack_weights_mxfp4, (codes, scales, torch.zeros(1, 32, 68, dtype=torch.uint8))),
                    (m.moe_build_routing_mxfp4, (ids, 8, 128, 128, r)),
                    (m.moe_dispatch, (x, r, 2, 8, None, y)), (m.moe_combine, (y, r, 2, 8, None, x)),
                    (m.moe_dispatch_grad, (y, r, 2, 8, None, None, x)), (m.moe_combine_grad, (x, r, 2, 8, None, None, y)),
                    (m.moe_router_topk_grad, (torch.zeros(4, 8), ids, w, w, True, 0, torch.zeros(4, 8)))):
        with pytest.raises(ValueError, match="stream"):
            f(*args, stream=there)


def test_buffers_that_are_no_run_of_bytes_are_refused(m, monkeypatch):
    # an expanded tensor counts bytes that it does not have
    monkeypatch.setattr(m, "_check_device", lambda *t: 0)
    monkeypatch.setattr(m, "_here", lambda dev, stream: None)
    E, H, I, T, k = 8, 128, 128, 4, 2
    r, bad = torch.zeros(4096, dtype=torch.uint8), torch.zeros(1, dtype=torch.uint8).expand(1 << 20)
    x, out, ids, w = torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k)
    y = torch.zeros(T * k, H, dtype=torch.bfloat16)
    w1 = m.moe_describe_packed_weights(torch.zeros(E, 2 * I, 68, dtype=torch.uint8), "mxfp4")
    w2 = m.moe_describe_packed_weights(torch.zeros(E, H, 68, dtype=torch.uint8), "mxfp4")
    for f, args, name in ((m.moe_build_routing_mxfp4, (ids, E, H, I, bad), "routing"), (m.moe_dispatch, (x, bad, k, E), "routing"),
                          (m.moe_combine, (y, r.repeat(2)[::2], k, E), "routing"), (m.moe_dispatch_grad, (y, bad, k, E), "routing"),
                          (m.moe_combine_grad, (x, bad, k, E), "routing"), (m.moe_forward_mxfp4, (x, w, r, w1, w2, bad, out), "workspace"),
                          (m.moe_route_forward_mxfp4, (ids, x, w, bad, w1, w2, r, out), "routing"),
                          (m.moe_route_forward_mxfp4, (ids, x, w, r, w1, w2, bad, out), "workspace")):
        with pytest.raises(ValueError, match=name + ": expected a contiguous buffer"):
            f(*args)


def test_headers_define_no_external_device_function(m):
    # a header in two sources would define it twice under relocatable device code
    for path in pathlib.Path(m.LIB_PATH).parent.glob("csrc/*.h"):
        lines = path.read_text().splitlines()
        for i, line in enumerate(lines):
            if line.startswith("__device__") and not lines[i - 1].startswith("template"):
                assert "__forceinline__" in line or "inline" in line, f"{path.name}: {line}"
