"""Host-side checks of the entry points of a served step: no GPU is needed."""
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
    assert lib.gemm_linear_adapted(None, pkg.LinearArgs(), pkg.AdapterArgs(), None) == bad
    assert lib.gemm_linear_adapted(None, None, None, None) == bad
    assert lib.moe_layer(None, pkg.MoeLayerArgs(), None) == bad
    assert lib.token_logprobs(None, 1, 8, p, 8, 0, p, 1.0, p, None, p, 0, None, None, None) == bad
    assert lib.token_logprobs_backward(None, 1, 8, p, 8, 0, p, 1.0, p, None, p, None, p, 8, None) == bad


@pytest.mark.parametrize("name,cls", [("gemm_adapter_args", "AdapterArgs"), ("moe_layer_args", "MoeLayerArgs")])
def test_argument_structs_match_the_header(pkg, name, cls, tmp_path):
    """The binding's structures, and the formats it packs them with, have the header's fields at the header's offsets."""
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
    packed = {"AdapterArgs": pkg._ADAPTERS, "MoeLayerArgs": pkg._LAYER}[cls]
    codes = {ctypes.c_int64: "q", ctypes.c_void_p: "P", ctypes.c_int: "i"}
    assert packed.format == "@" + "".join(codes[t] for _, t in struct._fields_)


def test_wrong_shapes_are_refused_before_the_library_is_called(pkg):
    """The binding's own checks, on a handle that is none: none of these may reach it."""
    import torch
    lib = pkg.Gemm.__new__(pkg.Gemm)
    lib.device, lib.handle, lib._dev = 0, None, None
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lib.adapted_linear(x[0], x, x, x, x)
    with pytest.raises(ValueError):
        lib.moe_layer(x, x, x, x, 1)
    with pytest.raises(ValueError):
        lib.token_logprobs(x[0], x)
    with pytest.raises(ValueError):
        lib.token_logprobs_backward(None, x[0], x, None)
    with pytest.raises(ValueError):  # not on the handle's device
        lib.token_logprobs(x.float(), torch.zeros(4, dtype=torch.int64))
    lib.handle = None
