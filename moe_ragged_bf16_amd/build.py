"""Ahead-of-time build of the gfx950 HIP library ``libmoe_ragged_bf16.so``.

One ``hipcc`` invocation compiles the kernels and the C ABI for gfx950 only and
links them into the package directory; a C++ one compiles ``_binding.so``, the Python
calls of the operators around the products.  Run ``python -m moe_ragged_bf16_amd.build``.
"""
from __future__ import annotations

import os
import re
import shutil
import tempfile
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libmoe_ragged_bf16.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
SOURCES = ["grouped_gemm_kernels.hip", "moe_kernels.hip", "fp8_kernels.hip",
           "capi.cpp", "capi_moe.cpp", "capi_fp8.cpp"]

HIP_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # the accumulate epilogue and the split reduction are plain IEEE adds
    "-ffp-contract=off",
    # never emit packed fp32 arithmetic (v_pk_add/mul/fma_f32).  The feature
    # belongs to the gfx950 device pass; the host pass prints that it does not
    # know it and ignores it.  check_no_packed_fp32() verifies the result.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # export only the entry points the public header marks MDG_API
    "-fvisibility=hidden",
]

BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(PKG_DIR, "_binding.so")

LLVM_BIN = "/opt/rocm/llvm/bin"
DEVICE_TARGET = "hipv4-amdgcn-amd-amdhsa--gfx950"
PACKED_FP32 = re.compile(r"\bv_pk_(add|mul|fma)_f32\b")


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build the HIP library)")


def build(verbose: bool = False) -> str:
    """Compile the library (always) and return its path."""
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    cmd = [hipcc(), *HIP_FLAGS, "-I", INCLUDE, "-I", CSRC]
    for s in SOURCES:
        cmd += ["-x", "hip", os.path.join(CSRC, s)]
    cmd += ["-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("hipcc failed building %s" % LIB_NAME)
    try:
        check_no_packed_fp32(tmp)
        check_mfma_sources(tmp)
    except Exception:
        os.unlink(tmp)
        raise
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def device_assembly(lib_path: str = LIB_PATH) -> str:
    """AMD assembly of the gfx950 code objects built into `lib_path` (its
    .hip_fatbin section holds one bundle for each source file; each is unbundled
    and disassembled with ROCm's LLVM tools)."""
    magic = b"__CLANG_OFFLOAD_BUNDLE__"

    def run(what, *cmd):
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("%s failed: %s" % (what, res.stderr))
        return res.stdout

    with tempfile.TemporaryDirectory() as d:
        fat = os.path.join(d, "fatbin.bin")
        run("extracting the device code", os.path.join(LLVM_BIN, "llvm-objcopy"), "--dump-section",
            ".hip_fatbin=" + fat, lib_path)
        with open(fat, "rb") as f:
            bundles = f.read().split(magic)[1:]
        out = []
        for i, bundle in enumerate(bundles):
            one, co = os.path.join(d, "%d.bundle" % i), os.path.join(d, "%d.co" % i)
            with open(one, "wb") as f:
                f.write(magic + bundle)
            run("extracting the gfx950 code object", os.path.join(LLVM_BIN, "clang-offload-bundler"), "--unbundle",
                "--type=o", "--input=" + one, "--targets=" + DEVICE_TARGET, "--output=" + co)
            out.append(run("llvm-objdump", os.path.join(LLVM_BIN, "llvm-objdump"), "-d", co))
        return "".join(out)


def check_no_packed_fp32(lib_path: str = LIB_PATH) -> int:
    """Raises if the built device code holds a packed fp32 add, multiply or
    fma; returns the number of MFMA instructions seen (a sanity count)."""
    asm = device_assembly(lib_path)
    bad = [ln.strip() for ln in asm.splitlines() if PACKED_FP32.search(ln)]
    if bad:
        raise RuntimeError("packed fp32 arithmetic in the gfx950 code: %d instructions, e.g. %s" % (len(bad), bad[0]))
    return sum(1 for ln in asm.splitlines() if "v_mfma" in ln)


_REGS = re.compile(r"\b([va])(?:(\d+)\b|\[(\d+):(\d+)\])")


def _registers(operand: str) -> set:
    """The vector registers an operand names ({"v12", ...})."""
    out = set()
    for kind, one, first, last in _REGS.findall(operand):
        out |= {kind + str(i) for i in range(int(one or first), int(one or last) + 1)}
    return out


def mfma_source_hazards(asm: str) -> list:
    """Scaled matrix instructions of a disassembly with a source register that one
    of the two instructions before wrote as a vector instruction (the hardware
    needs two wait states there; the compiler adds them for its own instructions,
    not around the asm statements of the 8-bit kernels)."""
    bad, before = [], []           # before: (wait states, registers written, text) of the latest instructions
    for line in asm.splitlines():
        text = line.split("//")[0].strip()
        m = re.match(r"([a-z]\w+)\s*(.*)", text)
        if not m or text.endswith(":"):
            before = []            # a label: another path may lead here, whose last instructions are its own
            continue
        name, args = m.group(1), m.group(2)
        operands = re.split(r",\s*(?![^\[]*\])", args)
        if name.startswith("v_mfma_scale"):
            sources, states = set().union(*(_registers(o) for o in operands[1:])), 0
            for waits, written, what in reversed(before):
                if states >= 2:
                    break
                if written & sources:
                    bad.append("%s; %s" % (what, text))
                states += waits
        valu = name.startswith("v_") and not name.startswith("v_mfma") and not name.startswith("v_cmp")
        waits = 1 + (int(args, 0) if name == "s_nop" else 0)
        before = before[-3:] + [(waits, _registers(operands[0]) if valu else set(), text)]
    return bad


def check_mfma_sources(lib_path: str = LIB_PATH) -> None:
    bad = mfma_source_hazards(device_assembly(lib_path))
    if bad:
        raise RuntimeError("a matrix instruction too close behind a write of its source: %d, e.g. %s" % (len(bad), bad[0]))


C_SMOKE_SRC = os.path.join(ROOT, "tests", "c_abi_smoke.cpp")
C_SMOKE_BIN = os.path.join(ROOT, "tests", "c_abi_smoke")


def build_c_smoke(verbose: bool = False) -> str:
    """Compile the C++ caller of the C ABI used by the tests (host code only,
    linked against the library with a relative rpath)."""
    cmd = [hipcc(), "-O2", "-std=c++17", "-I", INCLUDE, C_SMOKE_SRC, "-L", PKG_DIR, "-lmoe_ragged_bf16",
           "-Wl,-rpath,$ORIGIN/../moe_ragged_bf16_amd", "-o", C_SMOKE_BIN]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("hipcc failed building %s" % C_SMOKE_BIN)
    return C_SMOKE_BIN


def build_binding(verbose: bool = False) -> str:
    """Compile binding.cpp (host code only) against torch and return its path."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    tmp = BINDING_PATH + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, "-I", INCLUDE]
    for path in include_paths() + [sysconfig.get_paths()["include"]]:
        cmd += ["-I", path]
    cmd += [BINDING_SRC, "-o", tmp, "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python",
            "-ltorch", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("the C++ compiler failed building %s" % BINDING_PATH)
    os.replace(tmp, BINDING_PATH)
    return BINDING_PATH


if __name__ == "__main__":
    print(build(verbose=True))
    print(build_binding(verbose=True))
    print(build_c_smoke(verbose=True))
