"""ft.LIB_PATH names the one copy of the library that every call goes to, the marshalled ones among them."""
import os
import shutil
import subprocess
import sys

from block_quantized_matvec_amd import ft

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import sys
from block_quantized_matvec_amd import ft
ft.LIB_PATH = sys.argv[1]
ft._bind()
print(*sorted({l.split()[-1] for l in open("/proc/self/maps") if "libft" in l}))
"""


def test_one_copy_is_loaded(tmp_path):
    copy = str(tmp_path / "libft_copy.so")
    shutil.copy(ft.LIB_PATH, copy)
    r = subprocess.run([sys.executable, "-c", PROGRAM, copy], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == [copy]
