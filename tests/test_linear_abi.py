"""Host-side checks of the linear-layer and routing entry points: no GPU is needed."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__
    __graft_entry__.build()
    import programming_tiled_gemm_gb300 as p
    return p


def test_null_handle_and_arguments_are_rejected(pkg):
    lib, p = pkg.library(), 256
    bad = pkg.GEMM_ERR_INVALID_ARG
    assert lib.gemm_linear(None, pkg.LinearArgs(), None) == bad
    assert lib.gemm_linear_backward(None, pkg.LinearGradArgs(), None) == bad
    assert lib.moe_route(None, 1, 8, 2, p, 8, 0, 1, p, p, p, p, p, None) == bad
    assert lib.moe_route_backward(None, 1, 8, 2, p, p, 8, 0, p, 1, p, 8, None) == bad
    assert lib.moe_dispatch(None, 1, 8, 2, p, 8, 0, p, p, 8, None) == bad
    assert lib.moe_combine(None, 1, 8, 2, p, 8, 2, 0, p, p, None, 0, p, 8, None) == bad
    assert lib.moe_combine_backward(None, 1, 8, 2, p, 8, p, 8, 0, p, p, p, p, 8, p, None) == bad


@pytest.mark.parametrize("name,cls", [("gemm_linear_args", "LinearArgs"), ("gemm_linear_grad_args", "LinearGradArgs")])
def test_argument_structs_match_the_header(pkg, name, cls, tmp_path):
    """The binding's structures have the header's fields at the header's offsets."""
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("no gcc")
    struct = getattr(pkg, cls)
    fields = [f for f, _ in struct._fields_]
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gemm.h"\nint main(void) {\n' +
                   "".join('    printf("%%zu\\n", offsetof(%s, %s));\n' % (name, f) for f in fields) +
                   '    printf("%%zu\\n", sizeof(%s));\n    return 0;\n}\n' % name)
    exe = tmp_path / "s"
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(struct, f).offset for f in fields] + [ctypes.sizeof(struct)]
    text = open(os.path.join(ROOT, "include", "gemm.h")).read()
    body = re.search(r"typedef struct %s \{(.*?)\}" % name, text, flags=re.S).group(1)
    assert len(re.findall(r"[\w*]\s*(?:,|;)", body)) == len(fields)


def test_activation_codes_match_the_header(pkg):
    text = open(os.path.join(ROOT, "include", "gemm.h")).read()
    codes = {n.lower(): int(v) for n, v in re.findall(r"GEMM_ACT_(\w+) = (\d)", text)}
    assert codes == pkg.ACTIVATIONS
