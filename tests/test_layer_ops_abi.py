"""The C ABI of linear attention, group norm and dropout without a GPU: the host
code under the sanitizers (tests/sanitize/layer_ops_checks.cpp), workspace sizes,
and the checks of the Python binding."""
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
    exe = str(tmp_path / "layer_ops_checks")
    sources = [os.path.join(CSRC, n) for n in ("kdn_api.cpp", "kdn_plan.cpp", "kdn_linattn_api.cpp",
                                               "kdn_layer_ops_api.cpp")]
    sources += [os.path.join(HERE, "sanitize", n)
                for n in ("launch_stubs.cpp", "layer_ops_stubs.cpp", "layer_ops_checks.cpp")]
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
    # pure functions of the shape; none where the heads fill the chip, or for short rows
    assert L.kdn_linattn_fwd_workspace_size(8, 4096, 16, 128, 128) == 0
    assert L.kdn_linattn_fwd_workspace_size(1, 100, 1, 64, 64) == 0
    n = L.kdn_linattn_fwd_workspace_size(1, 65536, 16, 128, 128)
    assert n >= 2 * 16 * 128 * 128 * 4 and n == L.kdn_linattn_fwd_workspace_size(1, 65536, 16, 128, 128)
    # shared keys: fp32 gradients of every head
    assert L.kdn_linattn_bwd_workspace_size(64, 100, 4, 2, 64, 64) >= 2 * 64 * 100 * 4 * 64 * 4
    assert L.kdn_linattn_bwd_workspace_size(64, 100, 4, 4, 64, 64) == 0
    assert L.kdn_group_norm_fwd_workspace_size(32768, 1, 2048, 16) == 0
    assert L.kdn_group_norm_fwd_workspace_size(1, 65536, 64, 2) > 0
    for f, bad in ((L.kdn_group_norm_fwd_workspace_size, (4, 4, 64, 3)),
                   (L.kdn_group_norm_bwd_workspace_size, (-1, 4, 64, 4)),
                   (L.kdn_linattn_fwd_workspace_size, (1, 4096, 1, 257, 64)),
                   (L.kdn_linattn_bwd_workspace_size, (1, 4096, 3, 2, 64, 64))):
        assert f(*bad) == 0


def test_binding_refuses(L):
    import kalman_delta_rule_amd as kda
    q = torch.zeros(2, 8, 4, 16)
    g = torch.ones(4)
    with pytest.raises(ValueError, match="HIP device"):
        kda.kdn_linattn_fwd(q, q, q, g)
    with pytest.raises(ValueError, match="4 axes"):
        kda.kdn_linattn_fwd(q[0], q[0], q[0], g)
    with pytest.raises(ValueError, match="3 axes"):
        kda.kdn_linattn_step(q, q, q, g, q)
    with pytest.raises(TypeError, match="torch.Tensor"):
        kda.kdn_group_norm_fwd([1.0], 2)
    with pytest.raises(ValueError, match="mean"):
        kda.kdn_group_norm_bwd(q, q, None, None)
    with pytest.raises(ValueError, match="HIP device"):
        kda.kdn_dropout_fwd(q, 0.1, 0)


def test_heads_and_their_strides():
    from kalman_delta_rule_amd.api import _heads
    f32 = torch.float32
    wide = torch.zeros(2, 5, 3, 40)
    strides = lambda t: _heads(t, "q", t.shape, f32, t.device)[1:]
    assert strides(wide) == (120, 40)
    assert strides(wide[..., 7:20]) == (120, 40)
    assert strides(wide[:, :, 1:]) == (120, 40)
    assert strides(wide[:, :, :1])[0] == 120
    assert strides(torch.zeros(2, 5, 3 * 16 + 7)[..., 3:51].unflatten(-1, (3, 16))) == (55, 16)
    assert strides(wide[0, :, :, :8]) == (120, 40)  # one token of several sequences: [B, H, D]
    assert strides(torch.zeros(0, 5, 3, 40)) == (120, 40)
    for bad in (wide[:, 1:3], wide.transpose(1, 2), wide[..., ::2], torch.zeros(2, 5, 1, 40).expand(2, 5, 3, 40),
                torch.zeros(1, 1, 3, 40).expand(2, 5, 3, 40)):
        with pytest.raises(ValueError):
            strides(bad)


def test_seeds():
    from kalman_delta_rule_amd.api import _seed
    cpu = torch.device("cpu")
    assert _seed(5, (1 << 64) - 1, cpu) == (5, (1 << 64) - 1, None)
    t = torch.tensor([1, 2])
    assert _seed(t, 0, cpu) == (0, 0, t.data_ptr())
    for seed, offset in ((-1, 0), (1 << 64, 0), (1.5, 0), (0, -1), (True, 0), (t, 1)):
        with pytest.raises(ValueError):
            _seed(seed, offset, cpu)
    with pytest.raises(TypeError):
        _seed(t.float(), 0, cpu)
