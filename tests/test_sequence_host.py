"""The sequence operators' entry points on the host (CPU only): argument structures, sizes of
workspaces and every refusal, none of which touches the device.  Addresses are made up; a call that
should be refused is refused before anything reads them."""
import ctypes
import os
import subprocess

import pytest

import sparse_weight_direct_amd as sc
from sparse_weight_direct_amd import sequence as sq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A0 = 1 << 20  # addresses far apart


def _conv(**kw):
    v = dict(x=A0, out=2 * A0, weight=3 * A0, bias=4 * A0, initial=5 * A0, final=6 * A0, lengths=7 * A0, slots=0, x_batch=8 * 16,
             x_channel=16, out_batch=8 * 16, out_channel=16, initial_stride=8 * 3, final_stride=8 * 3, dtype=0, B=2, D=8, L=16,
             K=4, num_slots=2, flags=sq.SC_SEQ_SILU, reserved=0)
    assert set(kw) <= set(v)
    return sq.sc_causal_conv.pack(*{**v, **kw}.values())


def _scan(**kw):
    v = dict(x=A0, dt=2 * A0, z=3 * A0, b=4 * A0, c=5 * A0, out=6 * A0, A=7 * A0, skip=8 * A0, dt_bias=9 * A0, initial=10 * A0,
             final=11 * A0, lengths=12 * A0, slots=13 * A0, workspace=0, workspace_bytes=0, x_batch=128, x_channel=16,
             dt_batch=128, dt_channel=16, z_batch=128, z_channel=16, out_batch=128, out_channel=16, b_batch=64, b_group=64,
             b_state=16, c_batch=64, c_group=64, c_state=16, initial_stride=32, final_stride=32, dtype=0, B=2, D=8, L=16, N=4,
             G=1, num_slots=2, flags=sq.SC_SEQ_SOFTPLUS)
    assert set(kw) <= set(v)
    return sq.sc_selective_scan.pack(*{**v, **kw}.values())


def _adapter(**kw):
    v = dict(x=A0, base=2 * A0, out=3 * A0, down=4 * A0, up=5 * A0, scale=6 * A0, index=7 * A0, workspace=8 * A0,
             workspace_bytes=1 << 19, x_batch=8 * 16, x_channel=16, base_batch=6 * 16, base_channel=16, out_batch=6 * 16,
             out_channel=16, dtype=0, B=2, C=8, M=6, L=16, R=2, adapters=3, reserved=0)
    assert set(kw) <= set(v)
    return sq.sc_adapter.pack(*{**v, **kw}.values())


EINVAL, ESHAPE, EUNSUPPORTED = sc.SC_EINVAL, sc.SC_ESHAPE, sc.SC_EUNSUPPORTED


def _status(call, args):
    with pytest.raises(sc.SparseConvError) as e:
        call(args, 0)
    assert str(e.value).split(": ", 2)[2], "a message"
    return e.value.status


CONV = [(dict(dtype=3), EINVAL), (dict(dtype=-1), EINVAL), (dict(flags=2), EINVAL), (dict(reserved=1), EINVAL),
        (dict(B=-1), ESHAPE), (dict(L=-1), ESHAPE), (dict(D=0), ESHAPE), (dict(K=0), ESHAPE), (dict(K=9), EUNSUPPORTED),
        (dict(B=1 << 20, D=1 << 12), EUNSUPPORTED), (dict(x=0), EINVAL), (dict(out=0), EINVAL), (dict(weight=0), EINVAL),
        (dict(x=A0 + 2), EINVAL), (dict(out=2 * A0 + 1), EINVAL), (dict(weight=3 * A0 + 2), EINVAL), (dict(bias=4 * A0 + 1), EINVAL),
        (dict(lengths=7 * A0 + 2), EINVAL), (dict(slots=7 * A0 + 1), EINVAL), (dict(initial=5 * A0 + 2), EINVAL),
        (dict(x_batch=-1), ESHAPE), (dict(x_channel=-16), ESHAPE), (dict(out_channel=1 << 41), ESHAPE),
        (dict(out_channel=15), EINVAL), (dict(out_batch=0), EINVAL), (dict(num_slots=1), ESHAPE), (dict(num_slots=-1), ESHAPE),
        (dict(initial_stride=23), ESHAPE), (dict(num_slots=1 << 30, initial_stride=1 << 39), ESHAPE),
        (dict(final_stride=0), ESHAPE), (dict(final=5 * A0 + 4), EINVAL),
        (dict(final=5 * A0, final_stride=48), EINVAL), (dict(out=A0), EINVAL), (dict(out=A0 + 64), EINVAL),
        (dict(out=5 * A0), EINVAL), (dict(out=6 * A0 - 4), EINVAL), (dict(final=A0), EINVAL), (dict(out=3 * A0), EINVAL),
        (dict(out=4 * A0 + 16), EINVAL), (dict(final=7 * A0 - 4), EINVAL)]


@pytest.mark.parametrize("kw,status", CONV)
def test_conv_refusals(kw, status):
    assert _status(sc.sparseconv_causal_conv, _conv(**kw)) == status


SCAN = [(dict(dtype=7), EINVAL), (dict(flags=4), EINVAL), (dict(B=-1), ESHAPE), (dict(N=0), ESHAPE), (dict(G=3), ESHAPE),
        (dict(G=0), ESHAPE), (dict(D=0), ESHAPE), (dict(L=-2), ESHAPE), (dict(N=257), EUNSUPPORTED), (dict(L=1 << 30), EUNSUPPORTED),
        (dict(B=1 << 29, D=8), EUNSUPPORTED)] + \
       [({k: 0}, EINVAL) for k in ("x", "dt", "b", "c", "out", "A")] + \
       [({k: A0 * i + 2}, EINVAL) for i, k in enumerate(("x", "dt", "z", "b", "c", "out", "A", "skip", "dt_bias", "initial", "final",
                                                        "lengths", "slots"), 1)] + \
       [({k: -1}, ESHAPE) for k in ("x_batch", "dt_channel", "z_batch", "b_batch", "b_group", "b_state", "c_state", "out_batch")] + \
       [(dict(out_channel=8), EINVAL), (dict(initial_stride=31), ESHAPE), (dict(out=A0), EINVAL), (dict(out=4 * A0), EINVAL),
        (dict(out=7 * A0 - 4), EINVAL), (dict(final=8 * A0 - 4), EINVAL), (dict(final=10 * A0 + 16), EINVAL),
        (dict(final=6 * A0), EINVAL), (dict(slots=0, num_slots=1), ESHAPE)]


@pytest.mark.parametrize("kw,status", SCAN)
def test_scan_refusals(kw, status):
    assert _status(sc.sparseconv_selective_scan, _scan(**kw)) == status


def test_scan_workspace_is_asked_for():
    """A long axis with few channels is cut: the call needs the workspace it says, aligned and apart."""
    far = dict(L=8192, x_batch=8 * 8192, x_channel=8192, dt_batch=8 * 8192, dt_channel=8192, z=0, out=64 * A0, out_batch=8 * 8192,
               out_channel=8192, b_batch=4 * 8192, b_group=4 * 8192, b_state=8192, c_batch=4 * 8192, c_group=4 * 8192, c_state=8192)
    need = sc.sparseconv_selective_scan_workspace(_scan(**far))
    assert need > 0 and need % 4 == 0
    places = dict(x=16 * A0, dt=24 * A0, b=32 * A0, c=40 * A0)
    for kw in (dict(), dict(workspace=128 * A0, workspace_bytes=need - 1), dict(workspace=128 * A0 + 8, workspace_bytes=need),
               dict(workspace=64 * A0, workspace_bytes=need), dict(workspace=16 * A0, workspace_bytes=need),
               dict(workspace=11 * A0, workspace_bytes=need)):
        assert _status(sc.sparseconv_selective_scan, _scan(**far, **places, **kw)) == EINVAL
    assert sc.sparseconv_selective_scan_workspace(_scan(L=1)) == 0
    assert sc.sparseconv_selective_scan_workspace(_scan(L=64)) == 0
    assert sc.sparseconv_selective_scan_workspace(_scan(B=0)) == 0


ADAPTER = [(dict(dtype=3), EINVAL), (dict(reserved=5), EINVAL), (dict(B=-1), ESHAPE), (dict(C=0), ESHAPE), (dict(M=0), ESHAPE),
           (dict(R=0), ESHAPE), (dict(adapters=0), ESHAPE), (dict(L=-1), ESHAPE), (dict(R=129), EUNSUPPORTED),
           (dict(L=1 << 30), EUNSUPPORTED), (dict(C=1 << 30), EUNSUPPORTED), (dict(M=1 << 30), EUNSUPPORTED)] + \
          [({k: 0}, EINVAL) for k in ("x", "out", "down", "up", "index", "workspace")] + \
          [({k: A0 * i + 2}, EINVAL) for k, i in (("x", 1), ("base", 2), ("out", 3), ("scale", 6), ("index", 7))] + \
          [({k: A0 * i + 8}, EINVAL) for k, i in (("down", 4), ("up", 5), ("workspace", 8))] + \
          [(dict(workspace_bytes=16), EINVAL), (dict(out_channel=15), EINVAL), (dict(x_channel=-1), ESHAPE), (dict(out=A0), EINVAL),
           (dict(out=2 * A0 + 64), EINVAL), (dict(out=2 * A0, out_batch=128), EINVAL), (dict(out=4 * A0), EINVAL),
           (dict(out=8 * A0), EINVAL), (dict(workspace=A0), EINVAL)]


@pytest.mark.parametrize("kw,status", ADAPTER)
def test_adapter_refusals(kw, status):
    assert _status(sc.sparseconv_adapter_apply, _adapter(**kw)) == status


def test_null_arguments():
    for f in (sc._lib.sparseconv_causal_conv, sc._lib.sparseconv_selective_scan, sc._lib.sparseconv_adapter_apply):
        assert f(None, None) == EINVAL
    n = ctypes.c_int64()
    for f in (sc._lib.sparseconv_selective_scan_workspace, sc._lib.sparseconv_adapter_workspace):
        assert f(None, ctypes.byref(n)) == EINVAL
    assert sc._lib.sparseconv_selective_scan_workspace(_scan(), None) == EINVAL


def test_empty_calls_do_nothing():
    sc.sparseconv_causal_conv(_conv(B=0, x=0, out=0), 0)
    sc.sparseconv_selective_scan(_scan(B=0, x=0), 0)
    sc.sparseconv_adapter_apply(_adapter(B=0, x=0), 0)
    sc.sparseconv_adapter_apply(_adapter(L=0, x=0), 0)


def test_one_tensor_holds_input_and_output():
    """Two channel ranges of one tensor are apart; ranges that meet are not.  (Accepted calls end at the
    device: SC_EDEVICE where there is none.)"""
    half = dict(x_batch=256, out_batch=256)
    assert _status(sc.sparseconv_causal_conv, _conv(out=A0 + 4 * 127, **half)) == EINVAL
    assert _status(sc.sparseconv_causal_conv, _conv(out=A0 + 4 * 112, **half)) == EINVAL
    import torch
    if not torch.cuda.is_available():
        assert _status(sc.sparseconv_causal_conv, _conv(out=A0 + 4 * 128, **half)) == sc.SC_EDEVICE


def test_argument_structures_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "sparseconv.h"\nint main(void) {\n'
                   '  printf("%zu %zu %zu\\n", sizeof(sc_causal_conv), sizeof(sc_selective_scan), sizeof(sc_adapter));\n'
                   '  printf("%zu %zu %zu\\n", offsetof(sc_causal_conv, dtype), offsetof(sc_selective_scan, dtype), '
                   'offsetof(sc_adapter, dtype));\n  return 0;\n}\n')
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-std=c11", "-I" + os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in out[:3]] == [sq.sc_causal_conv.size, sq.sc_selective_scan.size, sq.sc_adapter.size]
    heads = (_conv(dtype=2), _scan(dtype=2), _adapter(dtype=2))
    for at, b in zip(out[3:], heads):
        assert int.from_bytes(b[int(at):int(at) + 4], "little") == 2


def test_the_binding_refuses_host_tensors():
    import torch
    x, w = torch.zeros(2, 8, 16), torch.zeros(8, 4)
    for f in (lambda: sc.causal_conv(x, w), lambda: sc.causal_conv_step(x[..., 0], torch.zeros(2, 8, 3), w),
              lambda: sc.selective_scan(x, x, w, x, x), lambda: sc.adapter_apply(x, x, x, x), lambda: sc.causal_conv([1.0], w)):
        with pytest.raises(ValueError):
            f()


def test_conv_limit_is_the_documented_one():
    """B * D * ceil(L / 8) < 2^31, to the last row.  (Accepted calls end at the device: SC_EDEVICE where there is none.)"""
    import torch
    far = dict(x=1 << 44, out=1 << 45, weight=1 << 42, bias=0, initial=0, final=0, lengths=0, num_slots=1 << 30)

    def status(B, D, L):
        return _status(sc.sparseconv_causal_conv, _conv(B=B, D=D, L=L, x_channel=L, out_channel=L, x_batch=D * L, out_batch=D * L,
                                                        **far))
    assert status(8, 1, (1 << 31) - 1) == EUNSUPPORTED and status(1 << 14, 1 << 14, 64) == EUNSUPPORTED
    assert status(1 << 15, 1 << 16, 1) == EUNSUPPORTED
    if not torch.cuda.is_available():
        for B, D, L in ((7, 1, (1 << 31) - 1), (1, 7, (1 << 31) - 7), ((1 << 14) - 1, 1 << 14, 64), ((1 << 15) - 1, 1 << 16, 1)):
            assert status(B, D, L) == sc.SC_EDEVICE


def _far_scan(B, D, L, N, G):
    """A scan of dense tensors that lie apart; the workspace is what it asks for."""
    kw = dict(B=B, D=D, L=L, N=N, G=G, z=0, skip=0, dt_bias=0, lengths=0, slots=0, initial=0, final=0, num_slots=B,
              x=1 << 44, dt=2 << 44, b=3 << 44, c=4 << 44, out=5 << 44, A=6 << 44, workspace=7 << 44, workspace_bytes=1 << 40)
    for k in ("x", "dt", "z", "out"):
        kw |= {k + "_channel": L, k + "_batch": D * L}
    for k in ("b", "c"):
        kw |= {k + "_state": L, k + "_group": N * L, k + "_batch": G * N * L}
    return _scan(**kw)


def test_scan_launches_fit_the_grid():
    """2^24 workgroups are more threads than a launch holds: refused before it, and by the workspace query.  What
    single positions take fewer workgroups for stays accepted.  (SC_EDEVICE: a call that got past the checks.)"""
    import torch
    for B, D, L, N, G in ((1 << 12, 1 << 12, 5, 4, 1 << 12), (1 << 16, 1 << 12, 2, 4, 1), (1 << 24, 3, 7, 16, 1),
                          (1 << 12, 1 << 12, 1, 4, 1 << 12), (1 << 24, 64, 1, 64, 1), (1 << 17, 1 << 13, 1, 40, 1), (1, (1 << 31) - 1, 1, 1, 1)):
        args = _far_scan(B, D, L, N, G)
        assert _status(sc.sparseconv_selective_scan, args) == EUNSUPPORTED, (B, D, L, N, G)
        with pytest.raises(sc.SparseConvError, match="SC_EUNSUPPORTED"):
            sc.sparseconv_selective_scan_workspace(args)
    if torch.cuda.is_available():
        return
    for B, D, L, N, G in (((1 << 12) - 1, 1 << 12, 5, 4, 1 << 12), (1 << 16, (1 << 12) - 16, 2, 4, 1), ((1 << 24) - 1, 3, 7, 16, 1),
                          (1 << 16, 1 << 12, 1, 4, 1), (1 << 17, 1 << 13, 1, 30, 1), (1, (1 << 31) - 257, 1, 1, 1)):
        assert _status(sc.sparseconv_selective_scan, _far_scan(B, D, L, N, G)) == sc.SC_EDEVICE, (B, D, L, N, G)


def test_adapter_launches_fit_the_grid():
    """As for the scan: the documented limits, on both sides."""
    import torch

    def args(dtype, B, C, M, L, R=1):
        return _adapter(dtype=dtype, B=B, C=C, M=M, L=L, R=R, adapters=1, x=1 << 44, base=0, out=2 << 44, down=3 << 44, up=4 << 44,
                        scale=0, index=5 << 44, workspace=6 << 44, workspace_bytes=1 << 43, x_channel=L, x_batch=C * L, out_channel=L,
                        out_batch=M * L)
    for case in ((0, 1 << 23, 1, 1, 64), (0, 1 << 22, 1, 2, 65), (1, 1 << 23, 1, 1, 128), (2, 1 << 13, 1, 1, 1 << 17), (0, 1 << 23, 1, 1, 1),
                 (1, 1 << 21, 1, 1000, 4), (1, 1 << 20, 1, 1025, 4), (0, 1, (1 << 31) - 1023, 1, 1), (1, 1, 1, (1 << 31) - 1023, 9),
                 (0, (1 << 23), 1, 1, 40, 128)):
        assert _status(sc.sparseconv_adapter_apply, args(*case)) == EUNSUPPORTED, case
        with pytest.raises(sc.SparseConvError, match="SC_EUNSUPPORTED"):
            sc.sparseconv_adapter_workspace(args(*case))
    if torch.cuda.is_available():
        return
    for case in ((0, (1 << 23) - 1, 1, 1, 64), (0, (1 << 22) - 1, 1, 2, 65), (1, (1 << 23) - 1, 1, 1, 128), (2, (1 << 13) - 1, 1, 1, 1 << 17),
                 (0, (1 << 23) - 1, 1, 1, 1), (1, (1 << 21) - 1, 1, 1000, 4), (0, 1, (1 << 31) - 1024, 1, 1), (1, 1, 1, (1 << 31) - 1024, 9),
                 (0, (1 << 23) - 1, 1, 1, 40, 128), (1, 1, 1, 1000, (1 << 30) - 128)):
        assert _status(sc.sparseconv_adapter_apply, args(*case)) == sc.SC_EDEVICE, case
