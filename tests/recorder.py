"""Runs a piece of Python with libq8ta on a HIP runtime that writes calls down instead of running them
(hip_recorder.c): what a call would launch, allocate and wait for, on a CPU."""
import json
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

_PRELUDE = """
import ctypes, json, sys
sys.path[:0] = [{root!r}, {here!r}]
import int8_quantized_amd as q8
rec = ctypes.CDLL({so!r})
rec.recorder_text.restype = ctypes.c_char_p
l, F = q8.lib(), ctypes.c_void_p(1 << 20)   # F: 16-byte aligned, never dereferenced

def calls():
    lines = [x.split() for x in rec.recorder_text().decode().splitlines()]
    rec.recorder_clear()
    return lines
"""


def recorded(code, lib=None, preload=(), env=None):
    """What `code` leaves in the name `result` (plain values)."""
    with tempfile.TemporaryDirectory() as tmp:
        so = os.path.join(tmp, "recorder.so")
        subprocess.run(["gcc", "-O1", "-std=c11", "-Wall", "-Werror", "-shared", "-fPIC", "-o", so,
                        os.path.join(HERE, "hip_recorder.c")], check=True)
        text = _PRELUDE.format(root=ROOT, here=HERE, so=so)
        if lib:
            text = text.replace("l, F =", f"q8.LIB_PATH = {lib!r}\nl, F =")
        e = dict(os.environ, LD_PRELOAD=" ".join(list(preload) + [so]), **(env or {}))
        r = subprocess.run([sys.executable, "-c", text + code + "\nprint('RESULT', json.dumps(result))"],
                           cwd=ROOT, env=e, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
        return json.loads(r.stdout.rsplit("RESULT ", 1)[1])


def have_recorder():
    """Whether libq8ta is built and a compiler is there."""
    import shutil
    return shutil.which("gcc") is not None
