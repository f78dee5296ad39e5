"""The matrix products' device code (built here from source, no GPU needed):
it compiles without a warning of its own, and nothing but the asynchronous
loads, which write it right in front of themselves, uses the register that
holds their LDS address."""
import os
import re
import subprocess

from signal_pad_sync_amd import build as B


def test_products_compile_clean_and_keep_m0_to_the_loads(tmp_path):
    out = tmp_path / "linear.s"
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC")]
    r = subprocess.run([B.HIPCC, *flags, "--cuda-device-only", "-S", os.path.join(B.CSRC, "arx_linear.hip"), "-o",
                        str(out)], check=True, capture_output=True, text=True, timeout=600)
    assert "[-Winline-asm]" not in r.stderr and "arx_linear.hip:" not in r.stderr, r.stderr[:2000]
    code = [ln.split(";")[0].strip() for ln in out.read_text().splitlines()]
    code = [ln for ln in code if ln and not ln.startswith(".")]
    loads = 0
    for i, ln in enumerate(code):
        if re.search(r"\bm0\b", ln):
            assert re.match(r"s_mov_b32 m0, s\d+$", ln), ln
            assert code[i + 1] == "s_nop 0" and code[i + 2].startswith("global_load_lds_dwordx4"), code[i:i + 3]
        loads += ln.startswith("global_load_lds_dwordx4")
    assert loads > 100
