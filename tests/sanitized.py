"""libq8ta with its host code under AddressSanitizer and UndefinedBehaviorSanitizer and no device code, for
runs on a runtime that launches nothing (recorder.py)."""
import contextlib
import glob
import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

from int8_quantized_amd import build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _flags():
    out = [f for f in b.CFLAGS if f != "-O3"] + ["-O1", "--offload-host-only"]
    for f in ("-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer",
              "-g"):
        out += ["-Xarch_host", f]
    return out


@contextlib.contextmanager
def sanitized():
    with tempfile.TemporaryDirectory() as tmp:
        def compile_one(src):
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            subprocess.run([b.hipcc()] + _flags() + ["-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj], check=True,
                           capture_output=True)
            return obj
        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
            objs = list(ex.map(compile_one, sorted(glob.glob(os.path.join(b.CSRC, "*.hip")))))
        # the device code's place, which is empty
        names = subprocess.run(["nm", "-u"] + objs, check=True, capture_output=True, text=True).stdout.split()
        with open(os.path.join(tmp, "fatbin.c"), "w") as f:
            f.writelines(f"const char {n}[16] = {{0}};\n" for n in sorted(set(names)) if n.startswith("__hip_fatbin_"))
        lib = os.path.join(tmp, "libq8ta_san.so")
        subprocess.run(["gcc", "-shared", "-fPIC", "-Wl,-rpath,/opt/rocm/lib", "-L/opt/rocm/lib", "-o", lib] + objs +
                       [f.name, "-lamdhip64", "-lstdc++"], check=True, capture_output=True)
        yield lib
