"""The staged attention for trees loads from memory straight to LDS in inline assembly, which sets a
register that cannot be named as overwritten: nothing else in the kernels may use it."""
import os
import re
import subprocess

import pytest

from test_serving_host import build_module


@pytest.mark.parametrize("name", ["kernels_tree_f16", "kernels_tree_bf16", "kernels_tree_f32"])
def test_the_address_register_is_the_loads_own(name):
    B = build_module()
    src, path = "serving/%s.hip" % name, os.path.join(B.BUILD, name + ".s")
    folder = os.path.join(B.CSRC, "serving")
    newest = max(os.path.getmtime(os.path.join(folder, f)) for f in os.listdir(folder))
    if not os.path.exists(path) or os.path.getmtime(path) < newest:
        os.makedirs(B.BUILD, exist_ok=True)
        subprocess.run([B.HIPCC, *B.FLAGS, *B.FILE_FLAGS.get(src, []), "-x", "hip", "--offload-device-only", "-S",
                        os.path.join(B.CSRC, src), "-o", path], check=True, capture_output=True)
    text = open(path).read()
    whole = re.findall(r"^\t;;#ASMSTART\n\ts_mov_b32 m0, s\d+\n\ts_nop 1\n\tglobal_load_lds_dwordx4 v\[\d+:\d+\], off\n\t;;#ASMEND$", text, re.M)
    code = [line for line in text.splitlines() if not line.lstrip().startswith(";")]
    assert len(whole) == sum(1 for line in code if re.search(r"\bm0\b", line))
    assert len(whole) == sum(1 for line in code if "global_load_lds" in line)
    assert (len(whole) > 50) == (name != "kernels_tree_f32")
