"""The attention operators' entry points on the host (CPU only): argument structures, workspaces, launch plans and every refusal,
none of which touches the device.  Addresses are made up; a call that should be refused is refused before anything
reads them."""
import os
import shutil
import subprocess

import pytest

import sparse_weight_direct_amd as sc
from sparse_weight_direct_amd import attention as at
from test_sequence_sanitizers import CSRC, ROOT, SAN

A0 = 1 << 24  # addresses far apart
NAN, INF = float("nan"), float("inf")
EINVAL, ESHAPE, EUNSUPPORTED = sc.SC_EINVAL, sc.SC_ESHAPE, sc.SC_EUNSUPPORTED


def _attend(**kw):
    v = dict(q=A0, out=2 * A0, k_pages=3 * A0, v_pages=4 * A0, table=5 * A0, past=6 * A0, lengths=7 * A0, prefix=8 * A0, slopes=9 * A0,
             workspace=10 * A0, workspace_bytes=1 << 23, q_batch=64 * 20, q_channel=20, out_batch=64 * 20, out_channel=20, k_page=2 * 16 * 16,
             v_page=2 * 16 * 16, table_batch=3, scale=0.25, cap=0.0, dtype=0, B=2, H=4, G=2, D=16, L=20, P=16, width=3, pages=8, window=0,
             flags=0, reserved=0)
    assert set(kw) <= set(v)
    return at.sc_paged_attention.pack(*{**v, **kw}.values())


def _append(**kw):
    v = dict(q=A0, q_out=2 * A0, k=3 * A0, v=4 * A0, k_pages=5 * A0, v_pages=6 * A0, freqs=7 * A0, axes=8 * A0, positions=9 * A0,
             table=10 * A0, past=11 * A0, lengths=12 * A0, q_batch=64 * 20, q_channel=20, q_out_batch=64 * 20, q_out_channel=20,
             k_batch=32 * 20, k_channel=20, v_batch=32 * 20, v_channel=20, k_page=2 * 16 * 16, v_page=2 * 16 * 16, table_batch=3,
             positions_batch=60, positions_axis=20, dtype=0, cache_dtype=0, B=2, H=4, G=2, D=16, L=20, P=16, width=3, pages=8, pairs=8,
             num_axes=3, flags=0, reserved=0)
    assert set(kw) <= set(v)
    return at.sc_cache_append.pack(*{**v, **kw}.values())


def _copy(**kw):
    v = dict(pool=A0, source=2 * A0, target=3 * A0, outer_stride=8 * 64, page_stride=64, page_bytes=64, outer=4, pages=8, count=3, reserved=0)
    assert set(kw) <= set(v)
    return at.sc_cache_copy.pack(*{**v, **kw}.values())


def _norm(**kw):
    v = dict(x=A0, y=2 * A0, gate=3 * A0, sum=4 * A0, out=5 * A0, weight=6 * A0, bias=7 * A0, post_weight=8 * A0, post_bias=9 * A0,
             x_batch=160, x_channel=20, y_batch=160, y_channel=20, sum_batch=160, sum_channel=20, out_batch=160, out_channel=20,
             gate_batch=160, gate_channel=20, gate_position=1, scale=1.0, eps=1e-6, dtype=0, B=2, C=8, L=20, flags=0, reserved=0)
    assert set(kw) <= set(v)
    return at.sc_residual_norm.pack(*{**v, **kw}.values())


def _status(call, args):
    with pytest.raises(sc.SparseConvError) as e:
        call(args, 0)
    assert str(e.value).split(": ", 2)[2], "a message"
    return e.value.status


CACHE = [(dict(G=0), ESHAPE), (dict(G=3), ESHAPE), (dict(D=0), ESHAPE), (dict(pages=0), ESHAPE), (dict(width=-1), ESHAPE),
         (dict(D=12), EUNSUPPORTED), (dict(D=264), EUNSUPPORTED), (dict(P=8), EUNSUPPORTED), (dict(P=48), EUNSUPPORTED),
         (dict(P=512), EUNSUPPORTED), (dict(width=(1 << 26) + 1), EUNSUPPORTED), (dict(G=1 << 17, H=1 << 17), EUNSUPPORTED),
         (dict(k_pages=0), EINVAL), (dict(v_pages=0), EINVAL), (dict(table=0), EINVAL), (dict(past=0), EINVAL),
         (dict(k_page=511), ESHAPE), (dict(v_page=0), ESHAPE), (dict(k_page=1 << 41), ESHAPE), (dict(k_page=513), EINVAL),
         (dict(table_batch=-1), ESHAPE), (dict(B=-1), ESHAPE), (dict(L=-1), ESHAPE), (dict(L=1 << 30), EUNSUPPORTED),
         (dict(dtype=3), EINVAL), (dict(flags=2), EINVAL), (dict(reserved=1), EINVAL)]


@pytest.mark.parametrize("kw,status", [c for c in CACHE if "H" not in c[0]] + [
    (dict(G=1 << 17, H=1 << 17), EUNSUPPORTED), (dict(H=0), ESHAPE), (dict(H=5), ESHAPE), (dict(window=-1), ESHAPE),
    (dict(H=1 << 17), EUNSUPPORTED), (dict(B=1 << 20, L=1000), EUNSUPPORTED),
    (dict(q=0), EINVAL), (dict(out=0), EINVAL), (dict(scale=NAN), EINVAL), (dict(scale=INF), EINVAL), (dict(cap=-1.0), EINVAL),
    (dict(cap=NAN), EINVAL), (dict(q=A0 + 2), EINVAL), (dict(out=2 * A0 + 2), EINVAL), (dict(k_pages=3 * A0 + 8), EINVAL),
    (dict(v_pages=4 * A0 + 4), EINVAL), (dict(table=5 * A0 + 2), EINVAL), (dict(past=6 * A0 + 1), EINVAL),
    (dict(lengths=7 * A0 + 2), EINVAL), (dict(prefix=8 * A0 + 3), EINVAL), (dict(slopes=9 * A0 + 1), EINVAL),
    (dict(q_channel=-1), ESHAPE), (dict(out_batch=1 << 41), ESHAPE), (dict(out_channel=19), EINVAL), (dict(out_batch=0), EINVAL),
    (dict(out=A0), EINVAL), (dict(out=3 * A0), EINVAL), (dict(out=4 * A0 + 16), EINVAL), (dict(out=5 * A0 - 4), EINVAL),
    (dict(out=6 * A0), EINVAL), (dict(out=7 * A0), EINVAL), (dict(out=8 * A0), EINVAL), (dict(out=9 * A0), EINVAL),
    (dict(dtype=1, flags=1, out=2 * A0 + 2), EINVAL)])
def test_attention_refusals(kw, status):
    assert _status(sc.sparseconv_paged_attention, _attend(**kw)) == status


@pytest.mark.parametrize("kw", [dict(scale=3e38), dict(scale=-3e38), dict(cap=3e38), dict(scale=1.0, cap=1e-39), dict(scale=1e30, cap=1e-10)])
def test_scales_that_leave_the_range_are_refused(kw):
    assert _status(sc.sparseconv_paged_attention, _attend(**kw)) == EINVAL


def test_attention_workspace_is_asked_for():
    far = dict(L=1, B=1, width=1000, table_batch=1000, q_channel=1, q_batch=64, out_channel=1, out_batch=64)
    need = sc.sparseconv_paged_attention_workspace(_attend(**far))
    assert need > 0
    for kw in (dict(workspace=0), dict(workspace_bytes=need - 1), dict(workspace=10 * A0 + 8), dict(workspace=A0), dict(workspace=2 * A0),
               dict(workspace=3 * A0 - 16), dict(workspace=5 * A0)):
        assert _status(sc.sparseconv_paged_attention, _attend(**far, **kw)) == EINVAL
    assert sc.sparseconv_paged_attention_workspace(_attend()) == 0  # a short context
    assert sc.sparseconv_paged_attention_workspace(_attend(**{**far, "B": 0})) == 0
    assert sc.sparseconv_paged_attention_workspace(_attend(**{**far, "L": 0})) == 0
    with pytest.raises(sc.SparseConvError):
        sc.sparseconv_paged_attention_workspace(_attend(P=20))


@pytest.mark.parametrize("kw,status", [c for c in CACHE if "H" not in c[0] and c[0] != dict(G=3)] + [
    (dict(cache_dtype=5), EINVAL), (dict(dtype=1, cache_dtype=0), EINVAL), (dict(dtype=1, cache_dtype=2), EINVAL), (dict(H=0), ESHAPE),
    (dict(H=1 << 17), EUNSUPPORTED), (dict(pairs=9), ESHAPE), (dict(pairs=-1), ESHAPE), (dict(num_axes=0), ESHAPE),
    (dict(B=1 << 23, L=100), EUNSUPPORTED), (dict(B=1 << 30, L=1), EUNSUPPORTED), (dict(q_out=0), EINVAL), (dict(k=0), EINVAL),
    (dict(v=0), EINVAL), (dict(freqs=0), EINVAL), (dict(q=A0 + 2), EINVAL), (dict(q_out=2 * A0 + 2), EINVAL), (dict(k=3 * A0 + 1), EINVAL),
    (dict(v=4 * A0 + 2), EINVAL), (dict(k_pages=5 * A0 + 8), EINVAL), (dict(freqs=7 * A0 + 4), EINVAL), (dict(axes=8 * A0 + 2), EINVAL),
    (dict(positions=9 * A0 + 1), EINVAL), (dict(table=10 * A0 + 2), EINVAL), (dict(past=11 * A0 + 2), EINVAL),
    (dict(lengths=12 * A0 + 2), EINVAL), (dict(k_channel=-1), ESHAPE), (dict(positions_axis=-1), ESHAPE), (dict(q_out_channel=19), EINVAL),
    (dict(q_out=A0 + 16), EINVAL), (dict(q_out=A0, q_out_batch=64 * 40), EINVAL), (dict(q_out=3 * A0), EINVAL), (dict(q_out=5 * A0), EINVAL),
    (dict(k_pages=A0), EINVAL), (dict(v_pages=5 * A0), EINVAL), (dict(v_pages=5 * A0 + 16), EINVAL), (dict(k_pages=3 * A0), EINVAL),
    (dict(v_pages=4 * A0), EINVAL), (dict(k_pages=7 * A0), EINVAL), (dict(v_pages=10 * A0), EINVAL), (dict(k_pages=11 * A0), EINVAL),
    (dict(v_pages=9 * A0), EINVAL), (dict(v_pages=12 * A0), EINVAL), (dict(v_pages=8 * A0), EINVAL)])
def test_append_refusals(kw, status):
    assert _status(sc.sparseconv_cache_append, _append(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(reserved=1), EINVAL), (dict(outer=-1), ESHAPE), (dict(pages=-1), ESHAPE), (dict(count=-1), ESHAPE), (dict(page_bytes=-1), ESHAPE),
    (dict(page_bytes=1 << 41), EUNSUPPORTED), (dict(outer=1 << 12, count=1 << 12), EUNSUPPORTED),
    (dict(outer=1 << 30, count=1 << 30, page_bytes=1 << 40), EUNSUPPORTED), (dict(pool=0), EINVAL), (dict(source=0), EINVAL),
    (dict(target=0), EINVAL), (dict(source=2 * A0 + 2), EINVAL), (dict(target=3 * A0 + 1), EINVAL), (dict(page_stride=-64), ESHAPE),
    (dict(outer_stride=1 << 41), ESHAPE), (dict(page_stride=63), EINVAL), (dict(outer_stride=64), EINVAL), (dict(source=A0 + 64), EINVAL),
    (dict(target=A0 - 8), EINVAL)])
def test_copy_refusals(kw, status):
    assert _status(sc.sparseconv_cache_copy, _copy(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=-1), EINVAL), (dict(flags=2), EINVAL), (dict(reserved=1), EINVAL), (dict(B=-1), ESHAPE), (dict(L=-1), ESHAPE),
    (dict(C=0), ESHAPE), (dict(C=1 << 20), EUNSUPPORTED), (dict(L=1 << 30), EUNSUPPORTED), (dict(B=1 << 20, L=40), EUNSUPPORTED),
    (dict(x=0), EINVAL), (dict(sum=0, out=0), EINVAL), (dict(y=0), EINVAL), (dict(y=0, gate=0), EINVAL), (dict(post_weight=0), EINVAL),
    (dict(out=0), EINVAL), (dict(scale=INF), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=NAN), EINVAL), (dict(x=A0 + 2), EINVAL),
    (dict(y=2 * A0 + 1), EINVAL), (dict(gate=3 * A0 + 2), EINVAL), (dict(sum=4 * A0 + 2), EINVAL), (dict(out=5 * A0 + 2), EINVAL),
    (dict(weight=6 * A0 + 2), EINVAL), (dict(bias=7 * A0 + 2), EINVAL), (dict(post_weight=8 * A0 + 1), EINVAL),
    (dict(post_bias=9 * A0 + 2), EINVAL), (dict(gate_position=2), ESHAPE), (dict(gate_position=-1), ESHAPE), (dict(x_channel=-1), ESHAPE),
    (dict(gate_channel=-1), ESHAPE), (dict(sum_channel=19), EINVAL), (dict(out_batch=0), EINVAL), (dict(sum=A0 + 16), EINVAL),
    (dict(sum=A0, sum_batch=320), EINVAL), (dict(out=A0), EINVAL), (dict(sum=2 * A0), EINVAL), (dict(out=2 * A0 + 80), EINVAL),
    (dict(out=4 * A0), EINVAL), (dict(sum=3 * A0), EINVAL), (dict(out=3 * A0 - 4), EINVAL), (dict(sum=6 * A0), EINVAL),
    (dict(out=7 * A0), EINVAL), (dict(out=8 * A0 - 4), EINVAL), (dict(sum=9 * A0), EINVAL)])
def test_norm_refusals(kw, status):
    assert _status(sc.sparseconv_residual_norm, _norm(**kw)) == status


def test_empty_calls_do_nothing():
    sc.sparseconv_paged_attention(_attend(B=0), 0)
    sc.sparseconv_paged_attention(_attend(L=0), 0)
    sc.sparseconv_cache_append(_append(B=0), 0)
    sc.sparseconv_cache_append(_append(L=0), 0)
    for kw in (dict(outer=0), dict(pages=0), dict(count=0), dict(page_bytes=0)):
        sc.sparseconv_cache_copy(_copy(**kw), 0)
    sc.sparseconv_residual_norm(_norm(B=0), 0)
    sc.sparseconv_residual_norm(_norm(L=0), 0)


def test_structures_have_the_headers_sizes(tmp_path):
    src = tmp_path / "sizes.cpp"
    src.write_text('#include "sparseconv.h"\n#include <cstdio>\nint main() { std::printf("%zu %zu %zu %zu", sizeof(sc_paged_attention), '
                   'sizeof(sc_cache_append), sizeof(sc_cache_copy), sizeof(sc_residual_norm)); }\n')
    exe = str(tmp_path / "sizes")
    subprocess.run(["g++", "-I" + os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(n) for n in got] == [s.size for s in (at.sc_paged_attention, at.sc_cache_append, at.sc_cache_copy, at.sc_residual_norm)]


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_argument_checks_under_sanitizers(tmp_path):
    """attention.cpp under AddressSanitizer and UndefinedBehaviorSanitizer with seeded random argument structures; a call that it
    accepts has to fit the launch, and to write where nothing else is."""
    exe = str(tmp_path / "fuzz_attention")
    cmd = ["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + CSRC, "-I" + os.path.join(ROOT, "include"),
           os.path.join(CSRC, "attention.cpp"), os.path.join(ROOT, "tests", "sanitize", "fuzz_attention.cpp"), "-o", exe] + SAN + \
          ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe, "20000"], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "failed checks 0" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
