"""What needs no CUDA build of torch: importing the package, its layout helpers
and the refusals of its C ABI."""
import subprocess
import sys

import pytest

from conftest import ROOT

IMPORT = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
taken = {n: getattr(torch._C, n) for n in ("_cuda_getDevice", "_cuda_getCurrentRawStream") if hasattr(torch._C, n)}
for name in taken:
    delattr(torch._C, name)
import quantize_block_scaled_rht_b200 as mx
assert mx.mma_scales_bytes(129, 2880) == 2 * 23 * 512
assert mx.lib().mxfp4_dropout(None, 0, None, 0, 1, 1, 0, 0.5, 1, 0, None, 0, None) == mx.MXFP4_ERR_INVALID_ARG
try:
    mx.mxfp4_int8_quantize(torch.zeros((4, 32), dtype=torch.bfloat16))
except ValueError as e:
    assert "CUDA tensors" in str(e)
else:
    raise SystemExit("a CPU tensor was taken")
"""

CALL = IMPORT + """
torch._C._cuda_getDevice = taken["_cuda_getDevice"]       # torch's own functions need it on a GPU
x = torch.randn((40, 64), device="cuda").to(torch.bfloat16)
q = mx.mxfp4_int8_quantize(x)
s = torch.cuda.Stream()
s.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(s):
    r = mx.mxfp4_int8_quantize(x)
torch.cuda.synchronize()
assert torch.equal(q.codes, r.codes) and int(q.codes.abs().max()) == 127
"""


def _python(code, *args):
    r = subprocess.run([sys.executable, "-c", code, ROOT, *args], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]


def test_import_without_the_cuda_names_of_torch():
    _python(IMPORT)


OLD_LIBRARY = """
import sys
sys.path.insert(0, sys.argv[1])
import quantize_block_scaled_rht_b200 as mx
mx.LIB_PATH = sys.argv[2]
try:
    mx.mma_scales_bytes(128, 128)
except ImportError as e:
    assert "older sources" in str(e) and "mxfp4_dropout" in str(e) and "mxfp4_version" not in str(e), e
else:
    raise SystemExit("taken")
"""


def test_a_library_without_the_newer_symbols_is_named(tmp_path):
    """A library of the same version number that lacks entry points is refused when
    it is loaded, with their names."""
    src, so = tmp_path / "old.c", tmp_path / "libold.so"
    src.write_text("int mxfp4_version(void) { return 105; }\n")
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    _python(OLD_LIBRARY, str(so))


@pytest.mark.gpu
def test_calls_without_the_private_names_of_torch():
    _python(CALL)
