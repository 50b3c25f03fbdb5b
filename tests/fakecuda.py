"""libdspark.so's C entries over a stand-in for the CUDA runtime (fake_cudart.cpp), in a process of its own: which
kernels a call launches, with what grid and shared memory, and on which device.  Nothing runs on a GPU, so pointers
are any numbers that pass the checks.

    python fakecuda.py <libdspark.so> <binding.py> < calls (json)
"""
import ctypes
import json
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
P = 1 << 20  # a pointer
WS = 1 << 40


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + \
        [(n, ctypes.c_int) for n in ("dtype", "layers", "n_pages", "page_size", "heads", "head_dim")] + \
        [(n, ctypes.c_longlong) for n in ("layer_stride", "page_stride", "token_stride", "head_stride")]


class Rotary(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("n_positions", ctypes.c_int),
                ("dim", ctypes.c_int), ("interleaved", ctypes.c_int)]


def cache(dtype, D, heads=8, page=64):
    if dtype == "fp4":
        c = Cache(P, P, 2, 1, 1000, page, heads, D, 0, page * heads * 9 * D // 16, 9 * D, page * 9 * D // 16)
    else:
        c = Cache(P, P, int(dtype == "bf16"), 1, 1000, page, heads, D, 0, page * heads * D, heads * D, D)
    return ctypes.byref(c)


def call(L, op, **a):
    """Status of one call."""
    D, heads, R, T, G = a.get("D", 128), a.get("heads", 8), a.get("R", 4), a.get("T", 4), a.get("G", 4)
    kind, bf = a.get("cache", "fp4"), int(a.get("dtype", "bf16") == "bf16")
    c, Hq = cache(kind, D, heads), heads * G
    if op == "attention" and kind == "fp4":
        return L.dspark_paged_attention_fp4(P, Hq * D, D, Hq, bf, c, 0, 1.0, 1.0, P, P, P, R, T, 100, 0.1, P, P, P, WS, None)
    if op == "attention":
        return L.dspark_paged_attention(P, Hq * D, D, Hq, c, 0, P, P, P, R, T, 100, 0.1, P, P, P, WS, None)
    if op == "append":
        rot = Rotary(P, None, 1000, a.get("rot", D), a.get("interleaved", 0))
        return L.dspark_cache_append_rotary(c, 0, 1.0, 1.0, ctypes.byref(rot), bf, P, P, heads * D, D, P, Hq * D, D, Hq, P,
                                            Hq * D, D, P, P, P, R, T, 100, P, WS, None)
    if op == "read":
        return L.dspark_cache_read(c, 0, 1.0, 1.0, bf, P, P, P, R, T, 100, P, P, P, WS, None)
    if op == "resize":
        return L.dspark_pages_resize(c, P, P, P, P, R, 100, P, P, P, P, P, WS, None)
    if op == "compact":
        return L.dspark_pages_compact(c, P, P, P, R, 100, P, P, P, P, P, WS, None)
    if op == "copy":
        return L.dspark_pages_copy(c, P, P, 3, P, WS, None)
    if op == "logprobs":
        return L.dspark_logprobs(P, bf, 4096, P, R, 4096, 1.0, 5, P, P, P, P, P, P, WS, None)
    if op == "draft":
        return L.dspark_draft_sample(P, P, P, P, bf, R, 4, 4096, 256, 1.0, 0, P, P, P, P, P, WS, None)
    if op == "schedule":
        return L.dspark_schedule(P, P, R * 5 + 1, R, 4, P, P, P, WS, None)
    if op == "verify":
        return L.dspark_verify(P, P, P, P, P, bf, P, R, 4, 151936, 1.0, 0, P, P, P, P, P, P, WS, None)
    raise KeyError(op)


def run(calls, where):
    """calls: dicts of `op`, `device` and sizes.  Returns of each its status and its launches, dicts of device, grid,
    smem and kernel (its name and template arguments as the compiler mangles them)."""
    from speculative_decoding_draft_05_gb300 import binding, build

    lib = build.build()
    fake = os.path.join(str(where), "fake_cudart.so")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-O1", "-I" + include, "-o", fake,
                    os.path.join(HERE, "fake_cudart.cpp")], check=True)
    r = subprocess.run([sys.executable, os.path.abspath(__file__), lib, binding.__file__], input=json.dumps(calls),
                       capture_output=True, text=True, env=dict(os.environ, LD_PRELOAD=fake))
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout)


def main():
    import importlib.util
    import types

    sys.modules["torch"] = types.ModuleType("torch")  # (the binding's tensors are not used)
    spec = importlib.util.spec_from_file_location("binding", sys.argv[2])
    binding = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(binding)
    binding.LIB_PATH = sys.argv[1]
    fake = ctypes.CDLL(os.environ["LD_PRELOAD"])
    fake.fake_launches.restype = ctypes.c_char_p
    L, out = binding.load(), []
    for a in json.load(sys.stdin):
        fake.fake_set_device(a.pop("device", 0))
        fake.fake_clear()
        st = call(L, **a)
        found = []
        for line in fake.fake_launches().decode().splitlines():
            dev, grid, smem, name = line.split(" ", 3)
            found.append(dict(device=int(dev), grid=int(grid), smem=int(smem), kernel=re.sub("EEv.*", "", name)))
        out.append(dict(status=st, launches=found))
    json.dump(out, sys.stdout)


if __name__ == "__main__":
    main()
