"""Ahead-of-time build of the gfx950 HIP library ``libmoe_ragged_bf16.so``.

``hipcc`` compiles the kernels and the C ABI for gfx950 only, one file each, and
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
from concurrent.futures import ThreadPoolExecutor
from functools import lru_cache

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libmoe_ragged_bf16.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
SOURCES = ["grouped_gemm_kernels.hip", "moe_kernels.hip", "fp8_kernels.hip", "gated_kernels.hip", "gated_few_kernels.hip",
           "norm_kernels.hip", "clip_kernels.hip", "capi.cpp", "capi_moe.cpp", "capi_fp8.cpp", "capi_gated.cpp",
           "capi_norm.cpp", "capi_clip.cpp"]

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

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            sys.stderr.write(res.stdout + res.stderr)
            raise RuntimeError("hipcc failed building %s" % LIB_NAME)

    with tempfile.TemporaryDirectory() as d:
        objects = [os.path.join(d, s + ".o") for s in SOURCES]
        flags = [f for f in HIP_FLAGS if f != "-shared"]
        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(run, [[hipcc(), *flags, "-I", INCLUDE, "-I", CSRC, "-x", "hip", "-c", os.path.join(CSRC, s),
                                 "-o", o] for s, o in zip(SOURCES, objects)]))
        run([hipcc(), "--offload-arch=gfx950", "-shared", *objects, "-o", tmp])
    try:
        asm = device_assembly(tmp)
        check_no_packed_fp32(tmp, asm)
        check_mfma_sources(tmp, asm)
        check_mfma_results(tmp, asm)
    except Exception:
        os.unlink(tmp)
        raise
    finally:
        _functions.cache_clear()
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


def check_no_packed_fp32(lib_path: str = LIB_PATH, asm: str = "") -> int:
    """Raises if the built device code holds a packed fp32 add, multiply or
    fma; returns the number of MFMA instructions seen (a sanity count).  `asm`:
    the library's disassembly, where the caller has it."""
    asm = asm or device_assembly(lib_path)
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


class _Instruction:
    """A line of a disassembly: what it is, the registers it names and which
    instructions may run next or may have run before (indexes in its function)."""
    __slots__ = ("name", "text", "operands", "states", "next", "before")

    def __init__(self, text: str):
        name, _, args = text.partition(" ")
        self.name, self.text, self.next, self.before = name, text, [], []
        self.operands = [_registers(o) for o in re.split(r",\s*(?![^\[]*\])", args)] if args else []
        self.states = 1 + (int(args, 0) if name == "s_nop" else 0)  # wait states it lets pass

    @property
    def mfma(self) -> bool:
        return self.name.startswith(("v_mfma", "v_smfma"))


@lru_cache(maxsize=1)
def _functions(asm: str) -> list:
    """The instructions of each function of a disassembly, with the branches
    between them (a branch names its target as <function+offset>)."""
    out, here, at, name, base = [], [], {}, None, 0

    def finish():
        for i, (ins, target) in enumerate(here):
            falls = ins.name not in ("s_branch", "s_endpgm", "s_setpc_b64")
            to = ([i + 1] if falls and i + 1 < len(here) else []) + ([at[target]] if target in at else [])
            ins.next = to
            for j in to:
                here[j][0].before.append(i)
        if here:
            out.append([ins for ins, _ in here])

    for line in asm.splitlines():
        m = re.match(r"([0-9a-f]+) <(.*)>:$", line)
        if m:
            finish()
            here, at, base, name = [], {}, int(m.group(1), 16), m.group(2)
            continue
        text, _, comment = line.partition("//")
        text = re.sub(r"\s+", " ", text).strip()
        if not re.match(r"[a-z]\w+( |$)", text):
            continue
        m = re.match(r"\s*([0-9A-F]+):", comment)
        if m:
            at[int(m.group(1), 16)] = len(here)
        target = None
        if text.startswith(("s_branch", "s_cbranch")):
            m = re.search(r"<%s(?:\+0x([0-9a-f]+))?>" % re.escape(name or ""), comment)
            target = base + int(m.group(1) or "0", 16) if m else None
        here.append((_Instruction(text), target))
    finish()
    return out


def _within(function: list, i: int, states: int, edges: str):
    """The instructions that instruction i reaches along `edges` (\"next\", \"before\")
    with fewer than `states` wait states between them."""
    todo, best = [(j, 0) for j in getattr(function[i], edges)], {}
    while todo:
        j, passed = todo.pop()
        if passed >= states or best.get(j, states) <= passed:
            continue
        best[j] = passed
        yield function[j]
        todo += [(k, passed + function[j].states) for k in getattr(function[j], edges)]


def mfma_source_hazards(asm: str) -> list:
    """Scaled matrix instructions of a disassembly with a source register that a
    vector instruction wrote within two wait states before (the hardware
    needs two there; the compiler adds them for its own instructions,
    not around the asm statements of the 8-bit kernels)."""
    bad = []
    for f in _functions(asm):
        for i, ins in enumerate(f):
            if not ins.name.startswith("v_mfma_scale"):
                continue
            sources = set().union(*ins.operands[1:])
            for w in _within(f, i, 2, "before"):
                if w.name.startswith("v_") and not w.mfma and not w.name.startswith("v_cmp") and w.operands \
                        and w.operands[0] & sources:
                    bad.append("%s; %s" % (w.text, ins.text))
    return bad


# Wait states between a matrix instruction of 8 passes (the longest here: 16x16x128 in
# 8 bits) and another instruction's access of its result: passes + 4 on gfx950.
MFMA_RESULT_STATES = 12
# and where it has 4 (what the compiler keeps for its own).
MFMA_RESULT_STATES_OF = {"v_mfma_f32_16x16x32_bf16": 8}


def mfma_result_hazards(asm: str) -> list:
    """Accesses of a matrix instruction's result that come before it is there: by
    another instruction than a matrix instruction that accumulates onto all of it
    (which the hardware waits for), within that many wait states."""
    bad = []
    for f in _functions(asm):
        for i, ins in enumerate(f):
            if not ins.mfma:
                continue
            result = ins.operands[0]
            for r in _within(f, i, MFMA_RESULT_STATES_OF.get(ins.name, MFMA_RESULT_STATES), "next"):
                if r.mfma and r.operands[3] == result and not result & set().union(*r.operands[1:3]) and \
                        (r.operands[0] == result or not r.operands[0] & result):
                    continue
                if result & set().union(*r.operands):
                    bad.append("%s; %s" % (ins.text, r.text))
    return bad


def check_mfma_sources(lib_path: str = LIB_PATH, asm: str = "") -> None:
    bad = mfma_source_hazards(asm or device_assembly(lib_path))
    if bad:
        raise RuntimeError("a matrix instruction too close behind a write of its source: %d, e.g. %s" % (len(bad), bad[0]))


def check_mfma_results(lib_path: str = LIB_PATH, asm: str = "") -> None:
    bad = mfma_result_hazards(asm or device_assembly(lib_path))
    if bad:
        raise RuntimeError("an access of a matrix instruction's result before it is there: %d, e.g. %s" % (len(bad), bad[0]))


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
