"""Host code of the decode-step operators over their ranges, on the CPU: index arithmetic and the planning
of launches and workspaces, as built and under AddressSanitizer and UndefinedBehaviorSanitizer.

The runtime is one that writes calls down (hip_recorder.c), so that every call gets through planning,
workspace bookkeeping and its launches; a launch out of range is an error there.
"""
import glob
import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest

from int8_quantized_amd import build as b
from recorder import recorded
from test_host_sanitizers import SAN_ENV, _clang_asan_runtime

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def _sizes(n):
    """n seeded calls of each operator, small and large sizes mixed, within the stated ranges."""
    g = np.random.Generator(np.random.PCG64(77))

    def one(lo, hi):
        return int(np.clip(round(float(np.exp(g.uniform(np.log(lo), np.log(hi))))), lo, hi))
    rope, attn, samp, lora = [], [], [], []
    for _ in range(n):
        d, hk = int(g.choice([1, 7, 64, 80, 128, 256, 512, 1000])), int(g.choice([1, 2, 8]))
        rope.append((one(1, 2 ** 31 - 1) if g.random() < 0.3 else one(1, 20000), hk * int(g.choice([1, 4, 7])), hk, d,
                     d // 2 * 2 if g.random() < 0.7 else 0, int(g.integers(0, 3)), int(g.integers(0, 2)),
                     0 if d % 8 == 0 and g.random() < 0.7 else 1))
        page = int(g.choice([16, 48, 64, 256, 1 << 20]))
        attn.append((one(1, 65535), one(1, 64), hk * int(g.choice([1, 4, 7, 16])), hk, int(g.choice([16, 64, 80, 128, 256])),
                     page, max(1, min(one(1, (1 << 31) // page), (2 ** 31 - 1024) // page)), int(g.integers(1, 3))))
        samp.append((one(1, 70000), one(1, 1 << 24), int(g.integers(0, 3))))
        K = one(1, 1 << 16)
        N = min(one(1, 1 << 30), (1 << 40) // K)
        M = min(one(1, 1 << 21), (1 << 40) // K, (1 << 37) // N)
        r = one(1, 512)
        lora.append((M, K, N, r, min(one(1, 1 << 24), max(1, (1 << 40) // (r * max(K, N)))), int(g.integers(1, 3)),
                     int(g.integers(0, 3)), 0 if g.random() < 0.8 else 1))
    attn += [(65535, 1, 1, 1, 64, 16, (2 ** 31 - 1024) // 16, 1), (1, 64, 65535 // 4, 1, 64, 16, 1, 2),
             (65535, 1, 8192, 8192, 16, 16, 1, 1), (1024, 1, 4, 1, 64, 1 << 20, 2047, 2), (1, 1, 1, 1, 256, 16, 1, 1)]
    lora += [(1, 64, 1 << 30, 1, 1, 1, 0, 0), (64, 1, 1 << 30, 512, 1, 2, 1, 1), (1 << 21, 64, 64, 512, 1 << 15, 1, 2, 0)]
    samp += [(1, 1, 0), (1024, 1 << 20, 0), (3000, 262144, 2), (70000, 1, 1)]
    return rope, attn, samp, lora


SWEEP = """
def at(odd):
    return ctypes.c_void_p((1 << 20) + odd)
bad = []
def note(what, rc, lines, kernels):
    grids = [[int(v) for v in x[2:8]] for x in lines if x[0] == "launch"]
    names = [x[1] for x in lines if x[0] == "launch"]
    if rc != 0 or not all(any(k in n for n in names) for k in kernels):
        bad.append((what, rc, q8.q8ta_last_error(), names, grids))
    got, back = sum(x[0] == "malloc" for x in lines), sum(x[0] == "free" for x in lines)
    count[what[0]] = count.get(what[0], 0) + 1
    return names, grids
count = {}
rope, attn, samp, lora = SIZES
for T, hq, hk, d, rot, dt, il, odd in rope:
    w = (hq + 2 * hk) * d
    rc = l.q8ta_rope_append(at(2 * odd), w + odd, d, F, w + odd, d, F, w + odd, d, dt, T, hq, hk, d, F, F, F, rot, 1.0,
                            il, F, F, F, 4, 16, None)
    if T * hq * d > 1 << 40:
        assert rc == q8.Q8TA_ERR_SHAPE
        continue
    names, grids = note(("rope", T, hq, hk, d, rot, dt, il, odd), rc, calls(), ["k_rope_append"])
    if sum(g[0] for g in grids) != T:
        bad.append(("rope tokens", T, grids))
for B, T, hq, hk, d, page, tp, dt in attn:
    rc = l.q8ta_tree_attention(F, T * hq * d, hq * d, d, dt, B, T, hq, hk, d, F, F, 9, page, F, tp, F, None, None, 0.1, F,
                               None, None)
    r = hk * (-(-T * (hq // hk) // 16))
    if r > 65535 or B * r > 1 << 29:
        assert rc == q8.Q8TA_ERR_SHAPE
        continue
    names, grids = note(("attn", B, T, hq, hk, d, page, tp, dt), rc, calls(), ["k_attn"])
for R, V, dt in samp:
    for k, p, mp in ((F, F, F), (None, None, None)):
        rc = l.q8ta_sample(F, V + 1, dt, R, V, F, k, p, mp, F, F, None, None)
        names, grids = note(("sample", R, V, dt), rc, calls(), [])
        if sum(g[0] for n, g in zip(names, grids) if "pick" in n or "long" in n) != R:
            bad.append(("sample rows", R, V, grids))
for M, K, N, r, na, ad, out, odd in lora:
    rc = l.q8ta_linear_lora(at(odd), M, K, 0.02, 3, F, N, F, None, F, F, ad, na, r, None, None, F, b"relu", F, out, None)
    names, grids = note(("lora", M, K, N, r, na, ad, out, odd), rc, calls(), ["k_lora_down"])
    down = [g for n, g in zip(names, grids) if "down" in n]
    if len(down) != 1 or down[0][0] * 16 < M or down[0][2] * 32 < r:
        bad.append(("lora down", M, r, down))
result = [bad[:5], count]
"""


def _sweep(**kw):
    bad, count = recorded(SWEEP.replace("SIZES", repr(_sizes(150))), **kw)
    assert not bad, bad
    assert set(count) == {"rope", "attn", "sample", "lora"} and min(count.values()) > 50, count


def _arithmetic(extra, env=None):
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "arithmetic")
        subprocess.run([b.hipcc(), "-x", "hip", f"--offload-arch={b.ARCH}", "--offload-host-only", "-O1", "-std=c++17"] +
                       extra + [os.path.join(HERE, "decode_arithmetic.cpp"), "-o", exe], check=True, capture_output=True)
        r = subprocess.run([exe], capture_output=True, text=True, timeout=120, env=dict(os.environ, **(env or {})))
        assert r.stdout.strip() == "ok" and r.returncode == 0, r.stdout + r.stderr[-3000:]


def _host_flags():
    out = []
    for f in ("-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer",
              "-g"):
        out += ["-Xarch_host", f]
    return out


def test_index_arithmetic():
    _arithmetic([])


def test_planning_sweep():
    _sweep()


def test_index_arithmetic_and_planning_under_asan_ubsan():
    asan = _clang_asan_runtime()
    if asan is None:
        pytest.skip("clang's AddressSanitizer runtime is not installed")
    _arithmetic(_host_flags(), SAN_ENV)
    flags = [f for f in b.CFLAGS if f != "-O3"] + ["-O1", "--offload-host-only"] + _host_flags()
    with tempfile.TemporaryDirectory() as tmp:
        def compile_one(src):
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            subprocess.run([b.hipcc()] + flags + ["-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj], check=True,
                           capture_output=True)
            return obj
        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
            objs = list(ex.map(compile_one, sorted(glob.glob(os.path.join(b.CSRC, "*.hip")))))
        # the device code's place, which is empty
        names = subprocess.run(["nm", "-u"] + objs, check=True, capture_output=True, text=True).stdout.split()
        with open(os.path.join(tmp, "fatbin.c"), "w") as f:
            f.writelines(f"const char {n}[16] = {{0}};\n" for n in sorted(set(names)) if n.startswith("__hip_fatbin_"))
        objs.append(f.name)
        lib = os.path.join(tmp, "libq8ta_san.so")
        subprocess.run(["gcc", "-shared", "-fPIC", "-Wl,-rpath,/opt/rocm/lib", "-L/opt/rocm/lib", "-o", lib] + objs +
                       ["-lamdhip64", "-lstdc++"], check=True, capture_output=True)
        _sweep(lib=lib, preload=[asan], env=SAN_ENV)
