"""The C ABI of the operators around the mixer without a GPU: the host code
under the sanitizers (tests/sanitize/block_checks.cpp), the built library's
refusals with stand-in pointers, and the checks of the Python binding."""
import os
import shutil
import subprocess

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "kalman_delta_rule_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


def test_host_code_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(os.path.join(ROCM, "include", "hip")):
        pytest.skip("needs g++ and the HIP headers")
    exe = str(tmp_path / "block_checks")
    sources = [os.path.join(CSRC, n) for n in ("kdn_api.cpp", "kdn_plan.cpp", "kdn_block_api.cpp")]
    sources += [os.path.join(HERE, "sanitize", n)
                for n in ("launch_stubs.cpp", "block_stubs.cpp", "block_checks.cpp")]
    flags = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
             "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
             "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
             "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    res = subprocess.run([gxx] + flags + sources + ["-o", exe], capture_output=True, text=True)
    if res.returncode != 0 and "asan" in res.stderr.lower():
        pytest.skip("sanitizer runtime not available: " + res.stderr[-300:])
    assert res.returncode == 0, res.stderr[-3000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                         env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0"))
    assert run.returncode == 0, run.stdout[-3000:] + run.stderr[-3000:]
    assert "all checks passed" in run.stdout


@pytest.fixture(scope="module")
def L():
    from kalman_delta_rule_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from kalman_delta_rule_amd import build
        build.build_library()
    return _lib.lib()


def test_workspace_sizes(L):
    # a short row needs none; the others are pure functions of the shape
    assert L.kdn_rec_fwd_workspace_size(2, 64, 100) == 0
    assert L.kdn_layer_norm_bwd_workspace_size(0, 64) == 0
    assert L.kdn_conv_bwd_workspace_size(2, 0, 64, 4) == 0
    for f, good, bad in ((L.kdn_rec_fwd_workspace_size, (1, 65536, 2048), (0, 64, 64)),
                         (L.kdn_rec_bwd_workspace_size, (1, 65536, 2048), (1, -1, 64)),
                         (L.kdn_layer_norm_bwd_workspace_size, (32768, 2048), (4, 0)),
                         (L.kdn_conv_bwd_workspace_size, (8, 4096, 2048, 4), (8, 4096, 2048, 1))):
        assert f(*good) == f(*good) >= 0
        assert f(*bad) == 0


@pytest.mark.skipif(torch.cuda.is_available(),
                    reason="stand-in pointers are only used where no GPU is visible")
def test_library_refuses(L):
    P, G = 1 << 20, 1 << 32
    msg = lambda: L.kdn_last_error_message().decode()
    assert L.kdn_layer_norm_fwd(4, 0, 1, 1e-5, P, 0, None, None, P + G, None, None, None) == -1
    assert "D >= 1" in msg()
    assert L.kdn_layer_norm_fwd(4, 64, 1, 1e-5, P, 64, None, None, P, None, None, None) == -1
    assert "y must not overlap x" in msg()
    assert L.kdn_conv_fwd(1, 8, 64, 7, 1, 0, P, 64, P + G, None, None, None, 0, P + 2 * G, None, None) == -2
    assert "taps" in msg()
    assert L.kdn_conv_step(4, 64, 4, 1, 0, P, 64, P + G, None, None, P + 2 * G, None) == -1
    assert "state must not be NULL" in msg()
    assert L.kdn_rec_fwd(2, 8, 64, 1, 1, 0, P, 64, P + G, 64, None, P + 2 * G, 3, P + 3 * G, None,
                         None, None, 0, None) == -1
    assert "B = 1" in msg()
    assert L.kdn_rec_step(4, 64, 1, 3, 0, P, 64, P + G, 64, P + 2 * G, P + 3 * G, None) == -1
    assert "gate" in msg()


def test_binding_refuses(L):
    import kalman_delta_rule_amd as kda
    x = torch.zeros(2, 8, 16)
    with pytest.raises(ValueError, match="HIP device"):
        kda.kdn_layer_norm_fwd(x)
    with pytest.raises(ValueError, match="3 axes"):
        kda.kdn_rec_fwd(x[0], x[0])
    with pytest.raises(TypeError, match="torch.Tensor"):
        kda.kdn_conv_fwd([1.0], x)


def test_row_strides():
    from kalman_delta_rule_amd.api import _row_stride
    wide = torch.zeros(2, 5, 3, 40)
    assert _row_stride(wide, "x") == 40
    assert _row_stride(wide[..., 7:20], "x") == 40
    assert _row_stride(wide[:, :, :1], "x") == 120
    assert _row_stride(wide[:, :, 1, :9], "x") == 120
    assert _row_stride(wide[:1, 2:4, 0], "x") == 120
    assert _row_stride(wide[0, 0, 0], "x") == 40
    assert _row_stride(wide[..., 3:4], "x") == 40       # one channel, 40 apart
    assert _row_stride(torch.zeros(0, 4), "x") == 4
    for bad in (wide[:, 1:3, :2], wide.transpose(-1, -2), wide[..., ::2],
                torch.zeros(1, 4).expand(6, 4)):
        with pytest.raises(ValueError):
            _row_stride(bad, "x")
