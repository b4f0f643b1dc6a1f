"""Refusals of the operators around the layer: bad arguments are rejected on
the host before anything is launched.  No GPU is needed: the pointers are made
up and no call reaches the device."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def deco():
    import sparse_moe_ffn_relu_b200 as d
    return d


X, Y, GP, GQ, GATE, OUT, H, WS = (0x100000 * (i + 1) for i in range(8))


def norm(deco, T=4, D=64, dtype=1, eps=1e-6, c=1.0, gate=0, lds=(0,) * 5, dh=1, dout=1):
    return deco.BlockNorm(T, D, dtype, eps, c, gate, *lds, dh, dout)


def fwd(deco, s, x=X, y=Y, gq=GQ, gate=None, gp=GP, out=OUT, h=H):
    return deco._lib.deco_block_norm_forward(s, x, y, gq, gate, gp, out, h, None)


def test_norm_forward_refusals(deco):
    n = lambda **k: norm(deco, **k)  # noqa: E731
    assert fwd(deco, n(T=0)) == OK                                        # an empty batch launches nothing
    for s in (n(T=-1), n(D=0), n(dtype=2), n(eps=-1.0), n(eps=float("nan")), n(c=float("inf")), n(gate=4), n(gate=-1)):
        assert fwd(deco, s, gate=GATE if s.gate else None) == INVALID
    for s in (n(D=16385), n(T=(1 << 20) + 1), n(lds=(1 << 31, 0, 0, 0, 0)), n(lds=(0, 0, 0, 0, 1 << 31))):   # rows of 4 GB
        assert fwd(deco, s) == UNSUPPORTED
    for kw in (dict(out=None), dict(y=None), dict(h=None), dict(gp=None), dict(y=None, out=None), dict(x=None), dict(gate=GATE),
               dict(y=None, out=None, gq=None, gp=None, h=None), dict(x=X + 1), dict(gq=GQ + 2), dict(h=X), dict(h=Y), dict(h=OUT), dict(out=Y)):
        assert fwd(deco, n(), **kw) == INVALID, kw
    assert fwd(deco, n(gate=1)) == INVALID                                # a gate kind without a gate
    assert fwd(deco, n(gate=3), gate=OUT) == INVALID                      # out on the gate
    assert fwd(deco, n(gate=2), gate=GATE + 2) == INVALID                 # an fp32 gate off its alignment
    for i in range(5):
        lds = [0] * 5
        lds[i] = 63
        assert fwd(deco, n(lds=tuple(lds), gate=3), gate=GATE) == INVALID, i   # rows would overlap
    assert fwd(deco, n(lds=(128, 0, 0, 64, 0)), out=X) == INVALID         # in place needs one stride
    assert deco._lib.deco_block_norm_forward(None, X, Y, GQ, None, GP, OUT, H, None) == INVALID


def bwd(deco, s, x=X, y=Y, gq=GQ, gate=None, gp=GP, dout=OUT, dh=H, grads=None, ws=WS, n=1 << 30):
    g = dict(dx=0x1100000, dy=0x1200000, dg_pre=0x1300000, dg_post=0x1400000, dgate=None)
    g.update(grads or {})
    gs = deco.BlockNormGrads(*[g[k] for k in ("dx", "dy", "dg_pre", "dg_post", "dgate")])
    return deco._lib.deco_block_norm_backward(s, x, y, gq, gate, gp, dout, dh, gs, ws, n, None)


def test_norm_backward_refusals(deco):
    s = norm(deco)
    need = ctypes.c_size_t(0)
    size = deco._lib.deco_block_norm_backward_workspace_size
    assert size(s, need) == OK and need.value > 0
    assert size(s, None) == INVALID and size(norm(deco, D=0), need) == INVALID and size(norm(deco, D=20000), need) == UNSUPPORTED
    for kw in (dict(dout=None, dh=None), dict(gp=None), dict(dh=None), dict(y=None), dict(x=None), dict(gate=GATE), dict(grads=dict(dx=None)),
               dict(grads=dict(dy=None)), dict(grads=dict(dg_pre=None)), dict(grads=dict(dg_post=None)), dict(grads=dict(dgate=0x1500000)),
               dict(grads=dict(dx=X)), dict(grads=dict(dx=H)), dict(grads=dict(dy=OUT)), dict(grads=dict(dy=Y)), dict(grads=dict(dx=0x1200000)),
               dict(x=X + 1), dict(grads=dict(dg_pre=0x1300002))):
        assert bwd(deco, s, **kw) == INVALID, kw
    assert bwd(deco, norm(deco, lds=(0, 0, 0, 128, 0)), grads=dict(dx=OUT)) == INVALID     # in place over gaps
    assert bwd(deco, norm(deco, dtype=0, dh=1)) == UNSUPPORTED                             # fp32 storage, bf16 gradient
    assert bwd(deco, norm(deco, dh=5)) == INVALID
    for ws, n in ((None, need.value), (WS + 16, need.value), (WS, need.value - 1)):
        assert bwd(deco, s, ws=ws, n=n) == WORKSPACE


def disp(deco, T=4, S=8, E=16, D=64, dtype=1, experts=X, active=None, x=Y, ld_x=0, ws=None, nws=0, **out):
    o = dict(counts=0x1000, offsets=0x2000, slot_of=0x3000, row_of=0x4000, n_pairs=0x5000, xs=OUT, ld_xs=0, capacity=32)
    o.update(out)
    t = deco.Dispatch(*[o[k] for k in ("counts", "offsets", "slot_of", "row_of", "n_pairs", "xs", "ld_xs", "capacity")])
    return deco._lib.deco_moe_dispatch(T, S, E, D, dtype, experts, active, x, ld_x, t, ws, nws, None)


def test_dispatch_refusals(deco):
    for kw in (dict(T=-1), dict(S=0), dict(E=0), dict(D=0), dict(dtype=3), dict(experts=None), dict(active=X), dict(experts=None, active=X),
               dict(experts=X + 2), dict(x=None), dict(x=OUT), dict(x=Y + 1), dict(ld_x=63), dict(ld_xs=1), dict(capacity=-1), dict(counts=None),
               dict(offsets=None), dict(n_pairs=None), dict(row_of=None), dict(slot_of=None), dict(counts=0x1002)):
        assert disp(deco, **kw) == INVALID, kw
    for kw in (dict(S=257), dict(E=257), dict(T=(1 << 20) + 1), dict(T=1 << 20, S=256, E=256, capacity=1), dict(D=(1 << 20) + 1), dict(capacity=1 << 31)):
        assert disp(deco, **kw) in (UNSUPPORTED, WORKSPACE), kw
    need = ctypes.c_size_t(0)
    size = deco._lib.deco_moe_dispatch_workspace_size
    assert size(16, 64, 64, 2048, 1, need) == OK and need.value == 0
    assert size(2048, 8, 64, 64, 1, need) == OK and need.value == 0        # 16384 slots, 2 MB of rows: one launch
    assert size(2049, 8, 64, 64, 1, need) == OK and need.value > 0
    assert size(2048, 8, 64, 2048, 1, need) == OK and need.value > 0       # 64 MB of rows
    # the binding asks unless no row could be too long
    assert size(deco._NO_WORKSPACE, 1, 64, 8192, 0, need) == OK and need.value == 0
    assert size(4096, 13, 300, 64, 1, need) == UNSUPPORTED and size(4, 4, 4, 64, 1, None) == INVALID
    assert size(4, 4, 4, 0, 1, need) == INVALID and size(4, 4, 4, 64, 2, need) == INVALID
    assert size(4096, 13, 64, 64, 1, need) == OK and need.value > 0
    for ws, n in ((None, need.value), (WS + 16, need.value), (WS, need.value - 1)):
        assert disp(deco, T=4096, S=13, E=64, ws=ws, nws=n) == WORKSPACE
    # the count of tiles, and with it the workspace, is bounded
    assert size(1 << 20, 256, 256, 64, 1, need) == OK and need.value <= 300 * 256 * 4


def test_combine_refusals(deco):
    def comb(T=4, S=8, D=64, dtype=1, ot=1, row_of=X, w=GP, ys=Y, n=32, ld_ys=0, base=None, ld_base=0, y=OUT, ld_y=0):
        return deco._lib.deco_moe_combine(T, S, D, dtype, ot, row_of, w, ys, n, ld_ys, base, ld_base, y, ld_y, None)
    assert comb(T=0) == OK
    for kw in (dict(T=-1), dict(S=0), dict(D=0), dict(dtype=2), dict(ot=7), dict(n=-1), dict(row_of=None), dict(ys=None), dict(y=None), dict(y=Y),
               dict(ys=Y + 1), dict(w=GP + 1), dict(ld_ys=8), dict(ld_y=8), dict(base=GQ, ld_base=8), dict(base=OUT, ld_base=128),
               dict(base=OUT, ot=0)):
        assert comb(**kw) == INVALID, kw
    assert comb(dtype=0, ot=1) == UNSUPPORTED and comb(S=300) == UNSUPPORTED

    def back(T=4, S=8, D=64, dtype=1, row_of=X, w=GP, ys=Y, n=32, ld_ys=0, dy=GQ, ld_dy=0, dys=OUT, ld_dys=0, dw=H):
        return deco._lib.deco_moe_combine_backward(T, S, D, dtype, row_of, w, ys, n, ld_ys, dy, ld_dy, dys, ld_dys, dw, None)
    assert back(T=0) == OK
    for kw in (dict(row_of=None), dict(dy=None), dict(ys=None), dict(dys=None), dict(dys=Y), dict(dys=GQ), dict(dw=H + 2), dict(ld_dy=3),
               dict(dys=OUT + 1), dict(S=0), dict(n=-1)):
        assert back(**kw) == INVALID, kw


def test_q4_refusals(deco):
    lib = deco._lib

    def mv(T=4, N=32, K=128, group=64, dtype=1, ot=1, x=X, ld_x=0, q=Y, scale=GP, zero=None, y=OUT, ld_y=0):
        return lib.deco_q4_matvec(T, N, K, group, dtype, ot, x, ld_x, q, scale, zero, y, ld_y, None)
    assert mv(T=0) == OK
    for kw in (dict(T=-1), dict(N=0), dict(K=0), dict(dtype=2), dict(ot=4), dict(x=None), dict(q=None), dict(scale=None), dict(y=None), dict(y=X),
               dict(q=Y + 8), dict(scale=GP + 4), dict(zero=GQ + 1), dict(x=X + 1), dict(ld_x=127), dict(ld_y=31)):
        assert mv(**kw) == INVALID, kw
    for kw in (dict(group=48), dict(K=(1 << 20) + 1), dict(dtype=0, ot=1), dict(T=(1 << 28) + 1), dict(N=(1 << 28) + 1), dict(T=1 << 28, N=1 << 20)):
        assert mv(**kw) == UNSUPPORTED, kw

    def ex(E=8, N=32, K=128, group=64, off=GQ, perm=None, rx=4, x=X, ry=16, y=OUT):
        return lib.deco_q4_expert_matvec(E, N, K, group, 1, 1, off, perm, rx, x, 0, Y, GP, None, ry, y, 0, None)
    assert ex(rx=0) == OK and ex(ry=0) == OK
    for kw in (dict(E=0), dict(off=None), dict(off=GQ + 2), dict(perm=H + 2), dict(rx=-1), dict(ry=-1), dict(N=0)):
        assert ex(**kw) == INVALID, kw
    assert ex(E=257) == UNSUPPORTED and ex(ry=(1 << 28) + 1) == UNSUPPORTED and ex(rx=(1 << 28) + 1) == UNSUPPORTED
    for rc in (lib.deco_q4_quantize(4, 64, 64, 1, None, Y, GP, None, None), lib.deco_q4_quantize(0, 64, 64, 1, X, Y, GP, None, None),
               lib.deco_q4_quantize(4, 64, 64, 1, X, Y + 4, GP, None, None), lib.deco_q4_pack(4, 64, X, None, None), lib.deco_q4_pack(4, 64, X, X, None),
               lib.deco_q4_dequantize(4, 64, 64, 1, Y, GP, None, None, None), lib.deco_q4_dequantize(4, 64, 64, 9, Y, GP, None, X, None)):
        assert rc == INVALID
    assert lib.deco_q4_quantize(4, 64, 16, 1, X, Y, GP, None, None) == UNSUPPORTED


def test_the_binding_checks_its_tensors(deco):
    """Python-level checks that come before the library (tensors on the CPU: no
    call gets as far as a launch)."""
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        deco.block_norm(x, torch.ones(64))
    with pytest.raises(ValueError, match="either"):
        deco.dispatch(x)
    with pytest.raises(ValueError, match="group"):
        deco._q4_sizes(64, 16)
    f32 = torch.float32
    with pytest.raises(ValueError, match="contiguous"):
        deco._whole(x.T, "x", (64, 4), f32, -1)
    with pytest.raises(ValueError, match="gaps"):
        deco._rows(x.T, "x", (64, 4), f32, -1)
    with pytest.raises(ValueError, match="overlap"):
        deco._rows(torch.zeros(64).expand(4, 64), "x", (4, 64), f32, -1)
    for shape, dtype, dev in (((4, 65), f32, -1), ((4, 64), torch.bfloat16, -1), ((4, 64), f32, 0)):
        for check in (deco._whole, deco._rows):
            with pytest.raises(ValueError, match="expected"):
                check(x, "x", shape, dtype, dev)
    wide = torch.zeros(4, 80)
    assert deco._rows(wide[:, 3:67], "x", (4, 64), f32, -1) == (wide.data_ptr() + 12, 80)
    assert deco._rows(wide[:1, :64], "x", (1, 64), f32, -1)[1] == 64
    assert deco._rows(None, "x", (1, 64), f32, -1) == (None, 0) and deco._whole(None, "x", (64,), f32, -1) is None
    assert [deco._gate_kind(g, 4, 64) for g in (None, torch.zeros(64), torch.zeros(4), torch.zeros(4, 1), torch.zeros(4, 64))] == [0, 1, 2, 2, 3]
    with pytest.raises(ValueError, match="gate"):
        deco._gate_kind(torch.zeros(5), 4, 64)


def test_a_gate_of_as_many_tokens_as_channels_is_named(deco):
    """[n] with n = T = D could be a gate per channel or per token: the binding
    asks for its kind instead of taking one of them."""
    n, kind = torch.zeros(8), deco._gate_kind
    with pytest.raises(ValueError, match="gate_kind"):
        kind(n, 8, 8)
    assert [kind(n, 8, 8, k) for k in ("channel", "token")] == [1, 2]
    assert kind(torch.zeros(8, 1), 8, 8) == kind(torch.zeros(8, 1), 8, 8, "token") == 2       # shapes that say it
    assert kind(torch.zeros(8, 8), 8, 8) == kind(torch.zeros(8, 8), 8, 8, "full") == 3
    assert kind(torch.zeros(1), 1, 1) == 1                                                    # one value: the same either way
    assert [kind(torch.zeros(s), 4, 8, k) for s, k in (((8,), "channel"), ((4,), "token"), ((4, 1), "token"), ((4, 8), "full"))] == [1, 2, 2, 3]
    assert [kind(torch.zeros(4, 1), 4, 1, k) for k in ("token", "full")] == [2, 3]            # of one channel
    for shape, k in (((8,), "token"), ((4,), "channel"), ((4, 8), "token"), ((8,), "full"), ((4, 1), "full"), ((8,), "rows")):
        with pytest.raises(ValueError, match="gate"):
            kind(torch.zeros(shape), 4, 8, k)
    with pytest.raises(ValueError, match="gate"):
        kind(None, 4, 8, "token")
    assert kind(None, 4, 8) == 0


def test_q4_experts_without_rows_of_x_still_check_perm(deco):
    """perm into an x of no rows asks for zero rows, so its call is one like
    others; without perm there is nothing to do.  (Refusals alone: nothing
    here reaches a device.)"""
    def ex(rx=0, x=None, off=GQ, perm=H, y=OUT, ry=16, q=Y):
        return deco._lib.deco_q4_expert_matvec(8, 32, 128, 64, 1, 1, off, perm, rx, x, 0, q, GP, None, ry, y, 0, None)
    for kw in (dict(perm=H + 2), dict(off=None), dict(y=None), dict(q=None), dict(rx=4), dict(y=OUT + 1)):
        assert ex(**kw) == INVALID, kw
    assert ex(perm=None) == OK and ex(ry=0) == OK


def test_import_needs_no_private_name_of_pytorch():
    """Where a build of PyTorch lacks the quick accessors of device and stream,
    the public ones serve."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import sparse_moe_ffn_relu_b200 as deco
assert deco._current_device is torch.cuda.current_device
class Stream:
    cuda_stream = 1234
torch.cuda.current_stream = lambda device: Stream() if device == 3 else None
assert deco._raw_stream(3) == 1234
assert deco.sparsity_controller(1.0, 0.3, 0.2) > 1.0      # calls that need no GPU
print("imported")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "imported", r.stdout + r.stderr


def test_sizes_beyond_32_bits_are_refused(deco):
    """The C side takes sizes as 32-bit integers, which ctypes fills with the
    low bits of what it gets: 2^32 + 4 rows must not become four."""
    far = 2 ** 32 + 4
    for shape in ((far, 1), (2 ** 31, 1), (1, far), (3, 2 ** 31)):
        with pytest.raises(ValueError, match="2\\^31"):
            deco._matrix(torch.empty(shape, device="meta"), "x")
    assert deco._matrix(torch.empty(2 ** 31 - 1, 1, device="meta"), "x") == (2 ** 31 - 1, 1)
    # rows that only a table of int32 names may be more: their number is 64 bits wide in C
    assert deco._matrix(torch.empty(far, 1, device="meta"), "ys", 63) == (far, 1)
    with pytest.raises(ValueError, match="2\\^31"):
        deco._matrix(torch.empty(1, far, device="meta"), "ys", 63)
    for K in (2 ** 32 + 128, 2 ** 31):
        with pytest.raises(ValueError, match="2\\^31"):
            deco._q4_sizes(K, 64)
    with pytest.raises(ValueError, match="dimensions"):
        deco._matrix(torch.zeros(4), "x")
    # every size that a call takes goes through one of these, but for dispatch's E
    with pytest.raises(ValueError, match="2\\^31"):
        deco._experts(2 ** 32 + 3)
    assert deco._experts(256) == 256
