"""Calls of the C library in a process whose C++ allocations fail: a status comes back, nothing is thrown (no GPU needed).

A small library preloaded into a child process replaces operator new; while its flag is set, every allocation fails.
An exception that left a C entry point would end the child.
"""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

NEW = r"""
#include <cstdlib>
#include <new>
extern "C" { int refuse_new = 0; }
static void* take(std::size_t n) { return refuse_new ? nullptr : std::malloc(n ? n : 1); }
void* operator new(std::size_t n) { if (void* p = take(n)) return p; throw std::bad_alloc(); }
void* operator new[](std::size_t n) { if (void* p = take(n)) return p; throw std::bad_alloc(); }
void* operator new(std::size_t n, const std::nothrow_t&) noexcept { return take(n); }
void* operator new[](std::size_t n, const std::nothrow_t&) noexcept { return take(n); }
void operator delete(void* p) noexcept { std::free(p); }
void operator delete[](void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
void operator delete[](void* p, std::size_t) noexcept { std::free(p); }
"""

CHILD = r"""
import ctypes, json, os, struct, sys, tempfile
sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]
import block_scaled_fp8_linear_amd as B
from test_fused_host import FAKE, _experts, _member
L = B.lib()
flag = ctypes.c_int.in_dll(ctypes.CDLL(NEW), "refuse_new")
ok, experts = _experts([_member()])
assert ok == "OK"
parts = [{k: dict(d, shape=d["shape"][1:]) for k, d in _member(E=1).items()}]
arr, keep = B._members_array(parts)
weight = ctypes.c_void_p()
decl = B._decl()
assert L.bsf8_weight_create(ctypes.byref(decl), arr, 1, ctypes.byref(weight)) == 0
earr, ekeep = B._members_array([_member()])
file = os.path.join(tempfile.mkdtemp(), "m.safetensors")
head = json.dumps({"a.b.c.proj.weight": dict(dtype="F8_E4M3", shape=[128, 128], data_offsets=[0, 128 * 128])}).encode()
with open(file, "wb") as f:
    f.write(struct.pack("<Q", len(head)) + head + bytes(128 * 128))
config = json.dumps({"quantization_config": {"quant_method": "fp8", "weight_block_size": [128, 128]}}).encode()
out, h, n = B.Decl(), ctypes.c_void_p(), ctypes.c_int32()
calls = {
    "parse": lambda: L.bsf8_parse_quant_config(config, ctypes.byref(out)),
    "inspect": lambda: L.bsf8_inspect_safetensors(file.encode(), ctypes.byref(decl), None, 0, ctypes.byref(n)),
    "validate": lambda: L.bsf8_validate(ctypes.byref(B._decl("fp8", (64, 64))), arr, 1),
    "weight": lambda: L.bsf8_weight_create(ctypes.byref(decl), arr, 1, ctypes.byref(h)),
    "experts": lambda: L.bsf8_experts_create(ctypes.byref(decl), earr, 1, ctypes.byref(h)),
    "norm": lambda: L.bsf8_quant_norm(ctypes.byref(B.NormArgs(4, 256, 7)), None),
    "plan": lambda: L.bsf8_expert_plan(None, 3, 1, 1, 1, None, None, None, None),
    "epilogue": lambda: L.bsf8_linear_w8a8_epilogue(weight, None, 0, None, 0, 0, 4, ctypes.byref(B.Epilogue()), None, 5, 0, None, 0, None),
    "product": lambda: L.bsf8_linear_w8a8_experts(experts, FAKE, 256, FAKE, 2, 1, 4, FAKE, FAKE, 8, FAKE, B.DT_BF16, 1, None),
    "describe": lambda: L.bsf8_describe(weight, B.ARM_W8A8_EPILOGUE, 200),
    "describe_experts": lambda: L.bsf8_experts_describe(experts, 200),
}
for name in ("describe", "describe_experts"):
    calls[name]()          # (the first asks for the device's properties)
got = {}
for name, call in calls.items():
    print(name, flush=True)
    flag.value = 1
    st = call()
    flag.value = 0
    got[name] = st.decode() if isinstance(st, bytes) else B.status_name(st) + " | " + L.bsf8_last_error().decode()
assert not h.value
print("GOT " + json.dumps(got), flush=True)
"""


def test_no_exception_leaves_a_c_entry(tmp_path):
    import json
    import shutil
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    src, so = tmp_path / "new.cpp", tmp_path / "libnew.so"
    src.write_text(NEW)
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    child = f"ROOT, NEW = {ROOT!r}, {str(so)!r}\n" + CHILD
    r = subprocess.run([sys.executable, "-c", child], env=dict(os.environ, LD_PRELOAD=str(so)), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout[-500:], r.stderr[-2000:])
    got = json.loads(r.stdout.split("GOT ")[1])
    for name in ("parse", "inspect", "weight", "experts"):
        assert got[name].startswith("UNSUPPORTED | ") and got[name].endswith("out of host memory"), (name, got[name])
    for name, status in (("validate", "DECL"), ("norm", "INVALID_ARG"), ("plan", "INVALID_ARG"), ("epilogue", "INVALID_ARG"),
                         ("product", "INVALID_ARG")):
        assert got[name].startswith(f"{status} | {status}: "), (name, got[name])
    for name in ("describe", "describe_experts"):
        assert got[name].startswith("out of host memory | "), (name, got[name])
