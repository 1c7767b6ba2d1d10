"""Host-side refusals of the linear layers and their gradients (no GPU, nothing
is launched)."""
import ctypes
import types

import pytest
import torch

NULL = None
FAKE, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4104)   # never dereferenced: every call fails its checks


@pytest.fixture(scope="module")
def m():
    import mixture_experts_layer_lds_amd as mod
    return mod


T, k, E, N, K = 4, 2, 8, 64, 128


def each(f, good, bad):
    for at, value, code in bad:
        a = list(good)
        a[at] = value
        assert f(*a) == code, (f, at, value)


def test_forward_refusals(m):
    lib, n = m._lib, m.moe_routing_layout(T, k, E, 128, 128, "bf16")["tasks"]
    good = [FAKE, FAKE, FAKE, FAKE, 0, 0, FAKE, n, T, k, E, N, K, FAKE, FAKE, NULL]
    each(lib.moe_grouped_linear, good, (
        (0, NULL, -1), (0, ODD, -1), (1, NULL, -1), (1, ODD, -1), (2, ODD, -1), (3, ODD, -1), (4, 2, -1), (4, 3, -1), (4, -1, -1),
        (5, -1, -1), (5, 4, -1), (6, NULL, -1), (6, ODD, -1), (7, n - 1, -3), (8, -1, -1), (8, 40000, -2), (9, 0, -1), (9, 17, -1),
        (10, 0, -1), (10, 512, -1), (11, 0, -1), (11, 12, -2), (11, 65544, -2), (12, -8, -1), (12, 20, -2), (12, 65544, -2),
        (13, ODD, -1), (14, NULL, -1), (14, ODD, -1)))
    gated = list(good)
    gated[5], gated[11] = 3, 72                       # halves of 36
    assert lib.moe_grouped_linear(*gated) == -2
    large = list(good)
    large[11], large[12] = 16392, 65536               # 2^30 values and a few rows more
    assert lib.moe_grouped_linear(*large) == -2
    good[8] = 0
    for at in (0, 1, 2, 3, 6, 13, 14):
        good[at] = NULL
    assert lib.moe_grouped_linear(*good) == 0
    plain = [FAKE, FAKE, FAKE, FAKE, 0, 0, T, N, K, FAKE, FAKE, NULL]
    each(lib.moe_linear, plain, (
        (0, NULL, -1), (1, ODD, -1), (2, ODD, -1), (3, ODD, -1), (4, 2, -1), (5, 4, -1), (6, -1, -1), (6, (1 << 24) + 1, -2),
        (7, 0, -1), (7, 4, -2), (8, 65544, -2), (9, ODD, -1), (10, NULL, -1)))
    assert lib.moe_linear(NULL, NULL, NULL, NULL, 1, 3, 0, N, K, NULL, NULL, NULL) == 0


def test_gradient_refusals(m):
    lib, n = m._lib, m.moe_routing_layout(T, k, E, 128, 128, "bf16")["tasks"]
    good = [FAKE, FAKE, FAKE, 1, 1, FAKE, n, T, k, E, N, K, FAKE, NULL]
    each(lib.moe_grouped_linear_grad_x, good, (
        (0, NULL, -1), (0, ODD, -1), (1, NULL, -1), (1, ODD, -1), (2, NULL, -1), (2, ODD, -1), (3, 2, -1), (4, 4, -1), (5, NULL, -1),
        (6, n - 1, -3), (7, 40000, -2), (8, 0, -1), (9, 512, -1), (10, 12, -2), (11, 12, -2), (12, NULL, -1), (12, ODD, -1)))
    wide = list(good)
    wide[4], wide[11] = 3, 32776                      # dx of 2 K values
    assert lib.moe_grouped_linear_grad_x(*wide) == -2
    plain = [FAKE, FAKE, FAKE, 1, 3, T, N, K, FAKE, NULL]
    each(lib.moe_linear_grad_x, plain, ((0, NULL, -1), (1, NULL, -1), (2, NULL, -1), (4, 9, -1), (5, -1, -1), (6, 4, -2), (8, ODD, -1)))
    assert lib.moe_linear_grad_x(NULL, NULL, NULL, 0, 0, 0, N, K, NULL, NULL) == 0
    good = [FAKE, FAKE, 0, 0, 0, FAKE, n, T, k, E, N, K, FAKE, FAKE, NULL]
    each(lib.moe_grouped_linear_grad_w, good, (
        (0, NULL, -1), (0, ODD, -1), (1, NULL, -1), (1, ODD, -1), (2, 2, -1), (3, 1, -1), (3, 3, -1), (4, 2, -1), (4, -1, -1),
        (5, NULL, -1), (6, n - 1, -3), (7, 40000, -2), (8, 0, -1), (9, 0, -1), (10, 12, -2), (11, 0, -1), (12, NULL, -1), (12, ODD, -1),
        (13, ODD, -1)))
    plain = [FAKE, FAKE, 1, 2, 1, T, N, K, FAKE, FAKE, NULL]
    each(lib.moe_linear_grad_w, plain, ((0, NULL, -1), (1, ODD, -1), (2, 2, -1), (3, 0, -1), (4, 2, -1), (5, -1, -1), (6, 4, -2), (8, NULL, -1),
                                        (9, ODD, -1)))
    assert lib.moe_linear_grad_w(NULL, NULL, 0, 0, 1, 0, N, K, FAKE, NULL, NULL) == 0       # nothing to add
    assert lib.moe_linear_grad_w(NULL, NULL, 0, 0, 0, 0, N, K, NULL, NULL, NULL) == -1      # zeros have to go somewhere
    good = [FAKE, FAKE, 0, 1, FAKE, n, T, k, E, N, FAKE, NULL]
    each(lib.moe_grouped_act_grad, good, (
        (0, NULL, -1), (0, ODD, -1), (1, NULL, -1), (2, 2, -1), (3, 0, -1), (3, 4, -1), (4, NULL, -1), (5, n - 1, -3), (6, 40000, -2),
        (7, 17, -1), (8, 0, -1), (9, 0, -1), (9, 12, -2), (9, 65544, -2), (10, ODD, -1)))
    assert lib.moe_act_grad(FAKE, FAKE, 0, 3, T, 32776, FAKE, NULL) == -2
    assert lib.moe_act_grad(FAKE, NULL, 0, 3, T, 64, FAKE, NULL) == -1
    assert lib.moe_act_grad(NULL, NULL, 0, 3, 0, 64, NULL, NULL) == 0


def test_sizes_past_32_bits_are_refused(m, monkeypatch):
    lib, over = m._lib, 1 << 32
    for f, args in ((lib.moe_linear, (FAKE, FAKE, NULL, NULL, 0, 0, over, N, K, NULL, FAKE, NULL)),
                    (lib.moe_linear_grad_x, (FAKE, FAKE, NULL, 0, 0, over, N, K, FAKE, NULL)),
                    (lib.moe_linear_grad_w, (FAKE, FAKE, 0, 0, 1, 0, over + N, K, FAKE, NULL, NULL)),
                    (lib.moe_act_grad, (FAKE, FAKE, 0, 1, over, 64, FAKE, NULL)),
                    (lib.moe_grouped_act_grad, (FAKE, FAKE, 0, 1, FAKE, 4096, over, 2, 8, 64, FAKE, NULL))):
        with pytest.raises(ctypes.ArgumentError, match="32-bit"):
            f(*args)
    monkeypatch.setattr(m, "_check_device", lambda *t: 0)
    monkeypatch.setattr(m, "_here", lambda dev, stream: None)
    tall = torch.empty(over + 4, 64, dtype=torch.bfloat16, device="meta")
    w = torch.empty(64, 64, dtype=torch.bfloat16, device="meta")
    for f in (lambda: m.moe_linear(tall, w), lambda: m.moe_linear_grad_x(tall, w), lambda: m.moe_linear_grad_w(tall, tall),
              lambda: m.moe_act_grad(tall, tall, "silu")):
        with pytest.raises(ctypes.ArgumentError, match="32-bit"):
            f()


def test_binding_refusals(m, monkeypatch):
    r = torch.zeros(4096, dtype=torch.uint8)
    bf = torch.bfloat16
    x, w3, w2, dy = torch.zeros(8, 64, dtype=bf), torch.zeros(4, 32, 64, dtype=bf), torch.zeros(32, 64, dtype=bf), torch.zeros(8, 32, dtype=bf)
    cases = [
        (lambda: m.moe_linear(x, w2), "current GPU"), (lambda: m.moe_grouped_linear(x, w3, r, 2), "current GPU"),
        (lambda: m.moe_linear(x.float(), w2.float()), "bf16 or fp16"), (lambda: m.moe_linear(x, w3), r"\[N\]\[K\]"),
        (lambda: m.moe_grouped_linear(x, w2, r, 2), r"\[E\]\[N\]\[K\]"), (lambda: m.moe_linear(x, w2, act="relu"), "act"),
        (lambda: m.moe_linear(x, w2.half()), "w: expected"), (lambda: m.moe_linear(x[:, :32], w2), "x: expected"),
        (lambda: m.moe_linear(x[0], w2), "x: expected"), (lambda: m.moe_linear(x, w2.t()), "x: expected"),
        (lambda: m.moe_linear(x, w2, bias=torch.zeros(31, dtype=bf)), "bias"),
        (lambda: m.moe_linear(x, w2, act="swiglu", residual=dy), "residual"),
        (lambda: m.moe_linear_grad_x(dy, w2, z=x), "z goes with"), (lambda: m.moe_linear_grad_x(dy, w2, act="silu"), "z goes with"),
        (lambda: m.moe_linear_grad_x(dy, w2, act="swiglu", z=x), "z: expected"),
        (lambda: m.moe_linear_grad_w(dy, x[:4]), "x: expected"), (lambda: m.moe_linear_grad_w(dy, x, dtype=torch.float16), "dtype"),
        (lambda: m.moe_linear_grad_w(dy, x, accumulate=True), "accumulate"),
        (lambda: m.moe_linear_grad_w(dy, x, dw=w2, want_bias=True, accumulate=True), "accumulate"),
        (lambda: m.moe_act_grad(dy, x, "silu"), "z: expected"), (lambda: m.moe_act_grad(dy, dy, "tanh"), "act"),
    ]
    for call, match in cases:
        with pytest.raises(ValueError, match=match):
            call()
    monkeypatch.setattr(m, "_check_device", lambda *t: 0)
    monkeypatch.setattr(m, "_here", lambda dev, stream: None)
    for call, match in ((lambda: m.moe_grouped_linear(x, w3, r, 3), "T \\* k rows"), (lambda: m.moe_grouped_linear(x, w3, r, 0), "T \\* k rows"),
                        (lambda: m.moe_grouped_linear(x, w3, r[::2], 2), "contiguous buffer"),
                        (lambda: m.moe_linear(x, w2, out=torch.zeros(8, 31, dtype=bf)), "out"),
                        (lambda: m.moe_linear(x, w2, z=torch.zeros(8, 32)), "z"),
                        (lambda: m.moe_grouped_linear_grad_w(dy, x, r, 2, 4, dw=w2), "dw"),
                        (lambda: m.moe_grouped_act_grad(dy, dy, r, 2, 4, "silu", dz=x), "dz")):
        with pytest.raises(ValueError, match=match):
            call()


def test_streams_of_another_gpu_are_refused(m, monkeypatch):
    monkeypatch.setattr(m, "_check_device", lambda *t: 0)
    there = types.SimpleNamespace(device_index=1, cuda_stream=4096)
    r, bf = torch.zeros(4096, dtype=torch.uint8), torch.bfloat16
    x, w, dy = torch.zeros(8, 64, dtype=bf), torch.zeros(4, 32, 64, dtype=bf), torch.zeros(8, 32, dtype=bf)
    for call in (lambda: m.moe_grouped_linear(x, w, r, 2, out=dy, stream=there), lambda: m.moe_linear(x, w[0], out=dy, stream=there),
                 lambda: m.moe_grouped_linear_grad_x(dy, w, r, 2, dx=x, stream=there),
                 lambda: m.moe_linear_grad_w(dy, x, dw=w[0], stream=there),
                 lambda: m.moe_grouped_act_grad(dy, dy, r, 2, 4, "gelu", dz=dy, stream=there)):
        with pytest.raises(ValueError, match="stream"):
            call()
