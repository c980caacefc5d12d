"""Refusals of the microscaled 4-bit and the routing calls, and their host-side bookkeeping (no GPU needed: every case fails
validation, or gets exactly as far as the device check, before anything is launched)."""

import ctypes
import os

import pytest
import torch

import bit_blockwise_weight_amd as qk

A = 0x40000000                                 # addresses that are never dereferenced, 1 GiB apart
B = ctypes.byref
INVALID = qk.QK_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(qk.LIB_PATH):
        pytest.fail("libqk.so is not built; run python -m bit_blockwise_weight_amd.build")
    return qk.lib()


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can launch")


def _state(L, rows=64, cols=256, codes=16 * A, cstride=128, scales=17 * A, sstride=8):
    st = qk.Mx4State()
    return L.qk_mx4_state_init(B(st), rows, cols, codes, cstride, scales, sstride), st


def test_state_init_accepts_and_refuses(L):
    rc, st = _state(L)
    assert rc == qk.QK_OK and st.magic == qk.QK_MX4_MAGIC and st.version == qk.QK_MX4_VERSION
    assert st.struct_bytes == ctypes.sizeof(qk.Mx4State) == 64
    for good in (dict(cols=1), dict(cols=255), dict(rows=1 << 30), dict(cstride=4096), dict(sstride=4096),
                 dict(cols=1 << 22, cstride=1 << 21, sstride=1 << 17), dict(scales=17 * A + 4)):
        assert _state(L, **good)[0] == qk.QK_OK, good
    for bad in (dict(rows=0), dict(rows=(1 << 30) + 1), dict(cols=0), dict(cols=(1 << 22) + 1, cstride=1 << 22, sstride=1 << 18),
                dict(codes=None), dict(scales=None), dict(cstride=112), dict(cstride=136), dict(cstride=0), dict(cstride=-128),
                dict(cstride=(1 << 22) + 16), dict(sstride=4), dict(sstride=9), dict(sstride=10), dict(sstride=-8),
                dict(sstride=(1 << 22) + 4), dict(codes=16 * A + 8), dict(scales=17 * A + 2), dict(cols=257)):
        assert _state(L, **bad)[0] == INVALID, bad
    assert L.qk_mx4_state_init(None, 1, 1, A, 16, A, 4) == INVALID


@needs_no_gpu
def test_good_arguments_reach_the_device_check(L):
    _, x = _state(L)
    _, w = _state(L, rows=96, codes=18 * A, scales=19 * A)
    no = qk.QK_ERR_NO_DEVICE
    assert L.qk_mx4_quantize(A, qk.QK_BF16, 64, 256, 256, 16 * A, 128, 17 * A, 8, None) == no
    assert L.qk_mx4_quantize(A + 2, qk.QK_F16, 64, 255, 1000, 16 * A, 128, 17 * A, 8, None) == no
    assert L.qk_mx4_dequantize(B(x), A, qk.QK_F32, None) == no
    assert L.qk_gemm_mx4(B(x), B(w), A, qk.QK_F16, None) == no and L.qk_gemm_mx4(B(x), B(x), A + 2, qk.QK_BF16, None) == no
    assert L.qk_gemv_mx4(A, qk.QK_F16, 16, B(w), 2 * A, None) == no
    assert L.qk_moe_route(A, qk.QK_BF16, 5, 64, 2 * A, qk.SIGMOID, 8, 4, 8, 1, 2.5, 3 * A,
                          4 * A, None) == no
    assert L.qk_moe_route_backward(A, qk.QK_F32, 5, 64, qk.SOFTMAX, 8, 1, 1.0, 2 * A, 3 * A, A, None) == no
    assert L.qk_moe_plan(A, 5, 8, 64, 2 * A, None) == no
    assert _up(L) == no and _down(L) == no


def test_a_broken_descriptor_is_refused_by_every_call(L):
    for field, value in (("magic", 1), ("version", 2), ("struct_bytes", 72), ("reserved", 1), ("rows", 0), ("cols", 0),
                         ("cols", (1 << 22) + 1), ("code_stride", 24), ("code_stride", 112), ("scale_stride", 4),
                         ("scale_stride", 9), ("codes", None), ("scales", None), ("codes", 16 * A + 4), ("scales", 17 * A + 1)):
        _, good = _state(L, codes=20 * A, scales=21 * A)
        _, bad = _state(L)
        setattr(bad, field, value)
        for rc in (L.qk_mx4_dequantize(B(bad), A, qk.QK_F32, None), L.qk_gemm_mx4(B(bad), B(good), A, qk.QK_F32, None),
                   L.qk_gemm_mx4(B(good), B(bad), A, qk.QK_F32, None), L.qk_gemv_mx4(A, qk.QK_BF16, 1, B(bad), 2 * A, None),
                   L.qk_moe_up_mx4(B(bad), B(good), A, 1, 1, 2 * A, qk.QK_F32, None),
                   L.qk_moe_up_mx4(B(good), B(bad), A, 1, 1, 2 * A, qk.QK_F32, None),
                   L.qk_moe_down_mx4(B(bad), B(good), A, 2 * A, 1, 1, 3 * A, qk.QK_F32, 4 * A, 1 << 30, None),
                   L.qk_moe_down_mx4(B(good), B(bad), A, 2 * A, 1, 1, 3 * A, qk.QK_F32, 4 * A, 1 << 30, None)):
            assert rc == qk.QK_ERR_BAD_STATE, field
        assert "mx4 state" in qk.qk_last_error()
    _, good = _state(L)
    for rc in (L.qk_mx4_dequantize(None, A, qk.QK_F32, None), L.qk_gemm_mx4(None, B(good), A, qk.QK_F32, None),
               L.qk_gemm_mx4(B(good), None, A, qk.QK_F32, None), L.qk_gemv_mx4(A, qk.QK_BF16, 1, None, 2 * A, None)):
        assert rc == INVALID


def test_quantize_refusals(L):
    def call(x=A, dt=qk.QK_BF16, rows=64, cols=256, pitch=256, codes=16 * A, cs=128, scales=17 * A, ss=8):
        return L.qk_mx4_quantize(x, dt, rows, cols, pitch, codes, cs, scales, ss, None)

    for bad in (dict(x=None), dict(x=A + 1), dict(dt=3), dict(dt=-1), dict(dt=qk.QK_F32, x=A + 2), dict(rows=0), dict(rows=-1),
                dict(cols=0), dict(pitch=255), dict(pitch=-256), dict(pitch=(1 << 40) + 1), dict(codes=None), dict(scales=None),
                dict(cs=120), dict(cs=112), dict(ss=6), dict(ss=4), dict(codes=16 * A + 8), dict(scales=17 * A + 1),
                dict(rows=1 << 30, pitch=1 << 40), dict(x=16 * A + 64), dict(x=17 * A), dict(scales=16 * A + 64)):
        assert call(**bad) == INVALID, bad


def test_dequantize_and_gemm_refusals(L):
    _, x = _state(L)
    _, w = _state(L, rows=96, codes=18 * A, scales=19 * A)
    _, other = _state(L, rows=96, cols=255, codes=18 * A, scales=19 * A)
    for out, dt in ((None, qk.QK_F32), (A, 3), (A + 2, qk.QK_F32), (A + 1, qk.QK_BF16), (16 * A + 16, qk.QK_F32),
                    (17 * A - 64, qk.QK_F16)):
        assert L.qk_mx4_dequantize(B(x), out, dt, None) == INVALID, (out, dt)
        assert L.qk_gemm_mx4(B(x), B(w), out, dt, None) == INVALID, (out, dt)
    assert L.qk_gemm_mx4(B(x), B(w), 18 * A + 4, qk.QK_F32, None) == INVALID and "overlaps" in qk.qk_last_error()
    assert L.qk_gemm_mx4(B(x), B(w), 19 * A, qk.QK_F32, None) == INVALID
    assert L.qk_gemm_mx4(B(x), B(other), A, qk.QK_F32, None) == INVALID and "columns" in qk.qk_last_error()


def test_gemv_refusals(L):
    _, w = _state(L)
    p = B(w)
    for args in ((None, qk.QK_BF16, 1, p, 2 * A), (A, qk.QK_BF16, 1, p, None), (A, qk.QK_F32, 1, p, 2 * A), (A, 9, 1, p, 2 * A),
                 (A, qk.QK_BF16, 0, p, 2 * A), (A, qk.QK_BF16, 17, p, 2 * A), (A + 1, qk.QK_BF16, 1, p, 2 * A),
                 (A, qk.QK_BF16, 1, p, 2 * A + 1), (A, qk.QK_BF16, 2, p, A + 512), (A, qk.QK_BF16, 1, p, 16 * A),
                 (A, qk.QK_F16, 1, p, 17 * A)):
        assert L.qk_gemv_mx4(*args, None) == INVALID, args
    _, big = _state(L, rows=(1 << 28) + 1)
    assert L.qk_gemv_mx4(A, qk.QK_BF16, 1, B(big), 40 * A, None) == INVALID


def test_route_refusals(L):
    def call(z=A, dt=qk.QK_F32, T=5, E=64, bias=2 * A, score=qk.SOFTMAX, groups=8, top=4, k=8, scale=1.0, ids=3 * A, w=4 * A):
        return L.qk_moe_route(z, dt, T, E, bias, score, groups, top, k, 1, scale, ids, w, None)

    for bad in (dict(z=None), dict(ids=None), dict(w=None), dict(dt=3), dict(T=0), dict(T=-1), dict(T=(1 << 26) // 8 + 1), dict(E=0),
                dict(E=513, groups=1, top=1), dict(score=2), dict(score=-1), dict(groups=0), dict(groups=65, E=130, top=1),
                dict(groups=7), dict(top=0), dict(top=9), dict(k=0), dict(k=33), dict(k=9, top=1), dict(scale=float("inf")),
                dict(scale=float("nan")), dict(z=A + 2), dict(bias=2 * A + 1), dict(ids=3 * A + 2), dict(w=4 * A + 1), dict(ids=A),
                dict(w=A + 64), dict(w=3 * A), dict(ids=2 * A), dict(w=2 * A), dict(E=4, groups=1, top=1, k=5)):
        assert call(**bad) == INVALID, bad


def test_route_backward_refusals(L):
    def call(z=A, dt=qk.QK_F32, T=5, E=64, score=qk.SOFTMAX, k=8, scale=1.0, ids=2 * A, dw=3 * A, dz=4 * A):
        return L.qk_moe_route_backward(z, dt, T, E, score, k, 1, scale, ids, dw, dz, None)

    for bad in (dict(z=None), dict(ids=None), dict(dw=None), dict(dz=None), dict(dt=3), dict(T=0), dict(E=0), dict(E=513), dict(score=2),
                dict(k=0), dict(k=33), dict(scale=float("nan")), dict(z=A + 2), dict(dz=4 * A + 2), dict(ids=2 * A + 2),
                dict(dw=3 * A + 2), dict(dz=A + 4), dict(dz=2 * A), dict(dz=3 * A + 64)):
        assert call(**bad) == INVALID, bad


def test_plan_refusals(L):
    n = ctypes.c_size_t(0)
    assert L.qk_moe_plan_size(5, 8, 64, B(n)) == qk.QK_OK and n.value >= 4 * (68 + 40)
    assert L.qk_moe_plan_size(1, 1, 3, B(n)) == qk.QK_OK and n.value >= 4 * (4 + 1)
    assert L.qk_moe_plan_size(5, 8, 64, None) == INVALID
    for bad in ((0, 8, 64), (5, 0, 64), (5, 33, 64), (5, 8, 0), (5, 8, 513), ((1 << 26) // 8 + 1, 8, 64)):
        assert L.qk_moe_plan_size(*bad, B(n)) == INVALID, bad
        assert L.qk_moe_plan(A, *bad, 2 * A, None) == INVALID, bad
    for ids, plan in ((None, A), (A, None), (A + 2, 2 * A), (A, 2 * A + 8), (A, A), (A + 16, A)):
        assert L.qk_moe_plan(ids, 5, 8, 64, plan, None) == INVALID, (ids, plan)


def _experts(L, T=6, k=2, E=4, H=64, I=96, **kw):
    """states of x, gate_up, h, down"""
    def st(rows, cols, at):
        rc, s = _state(L, rows, cols, at, -(-cols // 32) * 16, at + A // 2, (-(-cols // 32) + 3) // 4 * 4)
        assert rc == qk.QK_OK
        return s
    return st(T, H, 16 * A), st(E * 2 * I, H, 17 * A), st(T * k, I, 18 * A), st(E * H, I, 19 * A)


def _up(L, x=None, w=None, plan=A, k=2, E=4, h=2 * A, dt=qk.QK_BF16):
    s = _experts(L)
    return L.qk_moe_up_mx4(B(x or s[0]), B(w or s[1]), plan, k, E, h, dt, None)


def _down(L, h=None, w=None, plan=A, weights=3 * A, k=2, E=4, y=2 * A, dt=qk.QK_BF16, ws=4 * A, wsb=6 * 2 * 64 * 4):
    s = _experts(L)
    return L.qk_moe_down_mx4(B(h or s[2]), B(w or s[3]), plan, weights, k, E, y, dt, ws, wsb, None)


def test_experts_refusals(L):
    x, up, h, down = _experts(L)
    for bad in (dict(plan=None), dict(plan=A + 8), dict(k=0), dict(k=33), dict(E=0), dict(E=513), dict(E=5), dict(h=None), dict(h=2 * A + 1),
                dict(dt=3), dict(h=16 * A), dict(h=17 * A + 64), dict(h=A), dict(x=h)):
        assert _up(L, **bad) == INVALID, bad
    for bad in (dict(plan=None), dict(plan=A + 8), dict(weights=None), dict(weights=3 * A + 2), dict(k=0), dict(k=33), dict(k=5), dict(E=0),
                dict(E=513), dict(E=5), dict(y=None), dict(y=2 * A + 1), dict(dt=3), dict(y=18 * A), dict(y=19 * A), dict(y=A), dict(y=3 * A),
                dict(y=4 * A), dict(ws=4 * A + 8), dict(ws=A), dict(ws=3 * A), dict(ws=18 * A), dict(ws=19 * A), dict(h=x)):
        assert _down(L, **bad) == INVALID, bad
    for bad in (dict(ws=None), dict(wsb=6 * 2 * 64 * 4 - 1), dict(wsb=0)):
        assert _down(L, **bad) == qk.QK_ERR_WORKSPACE, bad
    n = ctypes.c_size_t(0)
    assert L.qk_moe_down_mx4_workspace_size(6, 2, 64, B(n)) == qk.QK_OK and n.value == 6 * 2 * 64 * 4
    assert L.qk_moe_down_mx4_workspace_size(6, 2, 64, None) == INVALID
    for bad in ((0, 2, 64), (6, 0, 64), (6, 33, 64), (6, 2, 0), (6, 2, (1 << 30) + 1)):
        assert L.qk_moe_down_mx4_workspace_size(*bad, B(n)) == INVALID, bad


def test_rows_that_pass_32_bit_offsets_are_refused(L):
    far = 1 << 46
    _, x = _state(L, rows=1 << 20, cols=8192, codes=far, cstride=4096, scales=2 * far, sstride=256)
    _, up = _state(L, rows=4 * 2 * 96, cols=8192, codes=3 * far, cstride=4096, scales=4 * far, sstride=256)
    assert L.qk_moe_up_mx4(B(x), B(up), A, 2, 4, 5 * far, qk.QK_BF16, None) == qk.QK_ERR_UNSUPPORTED
    _, x = _state(L, rows=4, cols=1 << 22, codes=far, cstride=1 << 21, scales=2 * far, sstride=1 << 17)
    _, up = _state(L, rows=2 * 1100, cols=1 << 22, codes=3 * far, cstride=1 << 21, scales=4 * far, sstride=1 << 17)
    assert L.qk_moe_up_mx4(B(x), B(up), A, 1, 1, 5 * far, qk.QK_BF16, None) == qk.QK_ERR_UNSUPPORTED
    assert "expert" in qk.qk_last_error()
    _, h = _state(L, rows=1 << 20, cols=8192, codes=far, cstride=4096, scales=2 * far, sstride=256)
    _, down = _state(L, rows=4 * 64, cols=8192, codes=3 * far, cstride=4096, scales=4 * far, sstride=256)
    assert L.qk_moe_down_mx4(B(h), B(down), A, 3 * A, 2, 4, 5 * far, qk.QK_BF16, 6 * far, 1 << 40, None) == qk.QK_ERR_UNSUPPORTED


def test_wrappers_check_shapes_and_devices():
    u8 = torch.zeros((4, 32), dtype=torch.uint8)
    with pytest.raises(ValueError, match="codes"):
        qk.qk_mx4_state_init(4, 65, u8, u8)                      # 33 bytes needed
    with pytest.raises(ValueError, match="codes"):
        qk.qk_mx4_state_init(5, 64, u8, u8)
    with pytest.raises(ValueError, match="scales"):
        qk.qk_mx4_state_init(4, 64, u8, u8[:, :3])
    with pytest.raises(ValueError, match="HIP device"):
        qk.qk_mx4_state_init(4, 64, u8, u8)
    with pytest.raises(ValueError, match="HIP device"):
        qk.qk_mx4_quantize(torch.zeros((4, 64)))
    with pytest.raises(ValueError, match="dtype"):
        qk.qk_mx4_quantize(torch.zeros((4, 64), dtype=torch.float64))
    with pytest.raises(ValueError, match="HIP device"):
        qk.qk_moe_route(torch.zeros((4, 64)), 2)
    with pytest.raises(ValueError, match="logits"):
        qk.qk_moe_route(torch.zeros((4, 64), dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="int32"):
        qk.qk_moe_plan(torch.zeros((4, 2), dtype=torch.int64), 8)
    with pytest.raises(ValueError, match="HIP device"):
        qk.qk_moe_plan(torch.zeros((4, 2), dtype=torch.int32), 8)
    with pytest.raises(ValueError, match="row per token"):
        qk.qk_moe_route_backward(torch.zeros((5, 64)), torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2)))
    with pytest.raises(ValueError, match="dweights"):
        qk.qk_moe_route_backward(torch.zeros((4, 64)), torch.zeros((4, 2), dtype=torch.int32), torch.zeros((2, 4)))
    assert qk.qk_moe_plan_size(5, 8, 64) >= 4 * (68 + 40)
    with pytest.raises(qk.QKError):
        qk.qk_moe_plan_size(5, 8, 513)


def test_a_plan_has_a_buffer_that_holds_it():
    words = qk.qk_moe_plan_size(5, 8, 64) // 4
    p = qk.MoePlan(torch.zeros(words, dtype=torch.int32), 5, 8, 64)
    assert p.first.shape == (65,) and p.slots.shape == (40,)
    for bad in (torch.zeros(words - 1, dtype=torch.int32), torch.zeros(words, dtype=torch.int64), torch.zeros(words)):
        with pytest.raises(ValueError, match="plan must be int32"):
            qk.MoePlan(bad, 5, 8, 64)
    with pytest.raises(qk.QKError):
        qk.MoePlan(torch.zeros(words, dtype=torch.int32), 5, 33, 64)
