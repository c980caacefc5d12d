"""Refusals of the int4 GEMV and the mixture-of-experts calls, and their host-side bookkeeping (no GPU needed:
every case fails validation, or gets exactly as far as the device check, before anything is launched)."""

import ctypes
import os

import pytest
import torch

import bit_blockwise_weight_amd as qk

A = 0x100000                                   # addresses that are never dereferenced
X, Y, LG, WS = A, 2 * A, 3 * A, 4 * A


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(qk.LIB_PATH):
        pytest.fail("libqk.so is not built; run python -m bit_blockwise_weight_amd.build")
    return qk.lib()


def _init(L, rows=64, cols=128, group=128, codes=16 * A, stride=64, scales=17 * A, sdt=qk.QK_F16, zeros=18 * A):
    st = qk.Int4State()
    return L.qk_int4_state_init(ctypes.byref(st), rows, cols, group, codes, stride, scales, sdt, zeros), st


def test_state_init_accepts_and_refuses(L):
    rc, st = _init(L)
    assert rc == qk.QK_OK and st.magic == qk.QK_INT4_MAGIC and st.version == qk.QK_INT4_VERSION
    assert st.struct_bytes == ctypes.sizeof(qk.Int4State) == 72
    for group in (0, 32, 64, 128, 256):
        assert _init(L, group=group)[0] == qk.QK_OK
    assert _init(L, cols=127)[0] == qk.QK_OK and _init(L, zeros=None)[0] == qk.QK_OK
    assert _init(L, stride=4096)[0] == qk.QK_OK
    for bad in (dict(rows=0), dict(rows=(1 << 28) + 1), dict(cols=0), dict(cols=(1 << 24) + 1), dict(group=16),
                dict(group=96), dict(group=-1), dict(group=512), dict(codes=None), dict(scales=None), dict(stride=48),
                dict(stride=72), dict(stride=0), dict(stride=-64), dict(sdt=qk.QK_F32), dict(sdt=7),
                dict(codes=16 * A + 8), dict(scales=17 * A + 1), dict(cols=129)):
        assert _init(L, **bad)[0] == qk.QK_ERR_INVALID_ARG, bad
    assert L.qk_int4_state_init(None, 1, 1, 0, A, 16, A, qk.QK_F16, None) == qk.QK_ERR_INVALID_ARG


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can launch")


@needs_no_gpu
def test_good_arguments_reach_the_device_check(L):
    _, st = _init(L)
    assert L.qk_gemv_int4(X, qk.QK_BF16, 16, ctypes.byref(st), Y, None) == qk.QK_ERR_NO_DEVICE
    assert L.qk_gemv_int4(X + 2, qk.QK_F16, 1, ctypes.byref(st), Y + 6, None) == qk.QK_ERR_NO_DEVICE
    up, down = _experts(L)
    assert _moe(L, up, down) == qk.QK_ERR_NO_DEVICE and _moe(L, up, down, y=X) == qk.QK_ERR_NO_DEVICE
    un, dn = _nf4_experts(L)
    assert _moe_nf4(L, un, dn) == qk.QK_ERR_NO_DEVICE


def test_gemv_refusals(L):
    _, st = _init(L)
    p = ctypes.byref(st)
    for args in ((None, qk.QK_BF16, 1, p, Y), (X, qk.QK_BF16, 1, p, None), (X, qk.QK_F32, 1, p, Y), (X, 9, 1, p, Y),
                 (X, qk.QK_BF16, 0, p, Y), (X, qk.QK_BF16, 17, p, Y), (X, qk.QK_BF16, 1, None, Y),
                 (X + 1, qk.QK_BF16, 1, p, Y), (X, qk.QK_BF16, 1, p, Y + 1), (X, qk.QK_BF16, 2, p, X + 256)):
        assert L.qk_gemv_int4(*args, None) == qk.QK_ERR_INVALID_ARG, args
    assert "overlaps" in qk.qk_last_error()
    for field, value in (("magic", 1), ("version", 2), ("struct_bytes", 160), ("group", 48), ("rows", 0), ("cols", 0),
                         ("code_stride", 24), ("scale_dtype", qk.QK_F32), ("reserved", 1), ("codes", None),
                         ("scales", None), ("codes", 16 * A + 4)):
        _, bad = _init(L)
        setattr(bad, field, value)
        assert L.qk_gemv_int4(X, qk.QK_BF16, 1, ctypes.byref(bad), Y, None) == qk.QK_ERR_BAD_STATE, field
        assert "int4 state" in qk.qk_last_error()


def test_grouped_gemv_refusals(L):
    _, st = _init(L)

    def call(n, ys=(Y, 5 * A), xs=(X, 6 * A), states=(st, st), M=4):
        arr = (qk.GemvInt4Task * 2)()
        for i in range(2):
            arr[i].x, arr[i].y = xs[i], ys[i]
            arr[i].st = ctypes.addressof(states[i]) if states[i] is not None else None
        return L.qk_gemv_int4_grouped(arr, n, qk.QK_F16, M, None)

    for bad in (dict(n=0), dict(n=257), dict(n=2, M=17), dict(n=2, ys=(Y, Y)), dict(n=2, ys=(Y, Y + 128)),
                dict(n=2, ys=(Y, X + 2)), dict(n=2, xs=(X, None)), dict(n=2, ys=(Y, None)), dict(n=2, states=(st, None))):
        assert call(**bad) == qk.QK_ERR_INVALID_ARG, bad
    corrupt = qk.Int4State()
    assert call(n=2, states=(st, corrupt)) == qk.QK_ERR_BAD_STATE
    assert L.qk_gemv_int4_grouped(None, 1, qk.QK_F16, 1, None) == qk.QK_ERR_INVALID_ARG


def _experts(L, E=4, H=128, I=64):
    return (_init(L, rows=E * 2 * I, cols=H, stride=H // 2)[1],
            _init(L, rows=E * H, cols=I, stride=64, codes=32 * A)[1])


def _moe(L, up, down, x=X, dtype=qk.QK_BF16, T=2, logits=LG, ldt=qk.QK_F32, E=4, top_k=2, y=Y, ws=WS, bytes_=1 << 19):
    return L.qk_moe_int4(x, dtype, T, logits, ldt, E, top_k, 1, ctypes.byref(up) if up is not None else None,
                         ctypes.byref(down) if down is not None else None, y, ws, bytes_, None)


def _nf4_state(L, rows, cols, codes=16 * A, block=64):
    st = qk.QuantState()
    lv = (ctypes.c_float * 16)(*qk.qk_make_codebook(qk.NF4).tolist())
    assert L.qk_state_init(ctypes.byref(st), qk.NF4, lv, rows, cols, block, codes, 24 * A, None, None, None) == qk.QK_OK
    return st


def _nf4_experts(L, E=4, H=128, I=64, **kw):
    return _nf4_state(L, E * 2 * I, H, **kw), _nf4_state(L, E * H, I, 32 * A)


def _moe_nf4(L, up, down, T=2, E=4, top_k=2, x=X, y=Y, ws=WS, bytes_=1 << 19):
    return L.qk_moe_nf4(x, T, LG, qk.QK_F32, E, top_k, 1, ctypes.byref(up), ctypes.byref(down), y, ws, bytes_, None)


def test_workspace_size(L):
    assert qk.qk_moe_workspace_size(16, 8, 4096, 11008) >= 16 * 8 * (4096 + 11008) * 4
    w = qk.qk_moe_workspace_size
    assert w(1, 1, 1, 1) <= w(1, 1, 1, 129) <= w(2, 1, 1, 129) <= w(2, 1, 200, 129)
    out = ctypes.c_size_t()
    big = (1 << 20) + 1
    for a in ((0, 1, 1, 1), (17, 1, 1, 1), (1, 0, 1, 1), (1, 17, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (1, 1, 1, big),
              (1, 1, big, 1)):
        assert L.qk_moe_workspace_size(*a, ctypes.byref(out)) == qk.QK_ERR_INVALID_ARG
    assert L.qk_moe_workspace_size(1, 1, 1, 1, None) == qk.QK_ERR_INVALID_ARG


def test_moe_refusals(L):
    up, down = _experts(L)
    for bad in (dict(x=None), dict(logits=None), dict(y=None), dict(T=0), dict(T=17), dict(E=3), dict(E=0), dict(E=257),
                dict(top_k=0), dict(top_k=5), dict(top_k=17), dict(dtype=qk.QK_F32), dict(ldt=5), dict(x=X + 1),
                dict(y=Y + 1), dict(logits=LG + 2), dict(ws=WS + 8), dict(ws=X - 64), dict(y=WS + 64),
                dict(logits=WS + 4096), dict(y=X + 256)):
        assert _moe(L, up, down, **bad) == qk.QK_ERR_INVALID_ARG, bad
    need = qk.qk_moe_workspace_size(2, 2, 128, 64)
    assert _moe(L, up, down, bytes_=need - 1) == qk.QK_ERR_WORKSPACE
    assert _moe(L, up, down, ws=None) == qk.QK_ERR_WORKSPACE
    assert _moe(L, None, down) == qk.QK_ERR_INVALID_ARG and _moe(L, up, None) == qk.QK_ERR_INVALID_ARG
    assert _moe(L, up, up) == qk.QK_ERR_INVALID_ARG          # not the stack [E * H, I]
    bad = qk.Int4State()
    assert _moe(L, bad, down) == qk.QK_ERR_BAD_STATE and _moe(L, up, bad) == qk.QK_ERR_BAD_STATE


def test_moe_nf4_refusals(L):
    up, down = _nf4_experts(L)
    assert _moe_nf4(L, up, down, T=17) == qk.QK_ERR_INVALID_ARG
    assert _moe_nf4(L, up, down, E=5) == qk.QK_ERR_INVALID_ARG
    assert _moe_nf4(L, up, down, bytes_=64) == qk.QK_ERR_WORKSPACE
    u2, d2 = _nf4_state(L, 4 * 2 * 96, 128), _nf4_state(L, 4 * 128, 96)
    assert _moe_nf4(L, u2, d2) == qk.QK_ERR_UNSUPPORTED and "multiples of 64" in qk.qk_last_error()
    u3, _ = _nf4_experts(L, codes=16 * A + 4)
    assert _moe_nf4(L, u3, down) == qk.QK_ERR_INVALID_ARG
    bad = qk.QuantState()
    assert _moe_nf4(L, bad, down) == qk.QK_ERR_BAD_STATE and _moe_nf4(L, up, bad) == qk.QK_ERR_BAD_STATE


def test_moe_refuses_experts_that_pass_32_bit_offsets(L):
    """(I + 16) rows of gate_up codes, (H + 16) of down: under 2^31 - 2^16 bytes, whatever a row's padding."""
    ws = dict(E=1, top_k=1, T=1, bytes_=1 << 30, ws=1 << 40)
    top = (1 << 31) - (1 << 16)
    for I, stride, good in ((48, 1 << 24, True), (112, 1 << 24, False), (241, (top // 257 // 16) * 16, True),
                            (241, (top // 257 // 16 + 1) * 16, False)):
        up, down = _init(L, rows=2 * I, cols=128, stride=stride)[1], _init(L, rows=128, cols=I, stride=128)[1]
        if good:
            if not torch.cuda.is_available():
                assert _moe(L, up, down, **ws) == qk.QK_ERR_NO_DEVICE
        else:
            assert _moe(L, up, down, **ws) == qk.QK_ERR_UNSUPPORTED and "gate_up" in qk.qk_last_error()
        up, down = _init(L, rows=256, cols=I, stride=128)[1], _init(L, rows=I, cols=128, stride=stride)[1]
        if good:
            if not torch.cuda.is_available():
                assert _moe(L, up, down, **ws) == qk.QK_ERR_NO_DEVICE
        else:
            assert _moe(L, up, down, **ws) == qk.QK_ERR_UNSUPPORTED and "down" in qk.qk_last_error()
    big = 1 << 20
    ws.update(x=1 << 36, y=1 << 37)
    for H, I, rc in ((big, 2048, qk.QK_ERR_UNSUPPORTED), (2048, big, qk.QK_ERR_UNSUPPORTED), (big, 1024, qk.QK_ERR_NO_DEVICE)):
        if rc == qk.QK_ERR_NO_DEVICE and torch.cuda.is_available():
            continue
        assert _moe_nf4(L, _nf4_state(L, 2 * I, H), _nf4_state(L, H, I, 32 * A), **ws) == rc, (H, I)


def test_binding_refuses_host_tensors_and_wrong_shapes(L):
    z = torch.zeros
    codes, scales = z((4, 16), dtype=torch.uint8), z((4, 1), dtype=torch.float16)
    with pytest.raises(ValueError, match="HIP device"):
        qk.qk_int4_state_init(4, 32, 32, codes, scales)
    for args in ((5, 32, 32, codes, scales), (4, 64, 32, codes, scales), (4, 32, 32, codes.int(), scales),
                 (4, 32, 32, codes, scales.float()), (4, 32, 32, codes, scales, z((4, 2), dtype=torch.uint8)),
                 (4, 32, 32, codes, scales, z((4, 1), dtype=torch.int8))):
        with pytest.raises(ValueError):
            qk.qk_int4_state_init(*args)
    with pytest.raises(ValueError):
        qk.Int4Weight(z((4, 32)), scales, None, 32)
    with pytest.raises(ValueError):
        qk.qk_gemv_int4_grouped([])
    _, st = _init(L)
    st._device, st._shape, st._address = torch.device("cuda", 0), (64, 128), ctypes.addressof(st)
    with pytest.raises(ValueError, match="bf16 or fp16"):
        qk.qk_gemv_int4(z((1, 128)), st)
    with pytest.raises(ValueError, match="128 columns"):
        qk.qk_gemv_int4(z((1, 64), dtype=torch.float16), st)
    with pytest.raises(ValueError, match="HIP device"):
        qk.qk_gemv_int4(z((1, 128), dtype=torch.float16), st)
    with pytest.raises(ValueError, match="2 outputs"):
        qk.qk_gemv_int4_grouped([(z((1, 128)), st)], [None, None])
