"""The package without the sequence operators' extension: the convolutions'
planner works, and a sequence operator says what is missing (no GPU)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "convolution_nhwc_conv2d_amd"

CHECK = f"""
import {PKG} as cn
assert cn.plan2d((1, 8, 8, 32), (32, 3, 3, 32), padding=1).out_h == 8
for name in ("layer_norm", "causal_conv1d_step", "selective_scan_backward", "ScanGrads", "sequence"):
    try:
        getattr(cn, name)
    except ImportError as e:
        assert "_seq" in str(e), e
    else:
        raise AssertionError(name)
try:
    from {PKG} import selective_scan
except ImportError as e:
    assert "_seq" in str(e), e
try:
    import {PKG}.sequence
except ImportError as e:
    assert "_seq" in str(e), e
else:
    raise AssertionError("sequence")
assert not hasattr(cn, "no_such_name")
print("fine")
"""


def test_convolutions_import_without_the_extension(tmp_path):
    pkg = tmp_path / PKG
    pkg.mkdir()
    for name in os.listdir(os.path.join(ROOT, PKG)):
        if name.endswith(".py") or name == "libcnhwc.so":
            os.symlink(os.path.join(ROOT, PKG, name), pkg / name)
    r = subprocess.run([sys.executable, "-c", CHECK], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]
