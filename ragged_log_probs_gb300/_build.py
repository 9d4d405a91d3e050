"""Build the C-ABI shared library in-tree with nvcc for sm_103a (GB300), and the compiled
Python binding of the head operators beside it."""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor
from importlib import metadata

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_NAME = "liblp_ragged.so"
SOURCES = ["lp_ragged.cu", "lp_norm.cu", "lp_process.cu", "lp_project.cu", "lp_adapters.cu"]
HEADERS = ["lp_device.cuh", "lp_kernels.cuh", "lp_head_common.h", "lp_adapters.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


BINDING = "lp_head_binding.cpp"  # Python binding of the head operators (torch's headers, g++)


def lib_path() -> str:
    return os.path.join(LIB_DIR, LIB_NAME)


def binding_path() -> str:
    """Where the binding is: named after the interpreter and the torch whose C++ ABI it has, so that
    after an upgrade of either none is found, instead of one that does not fit."""
    return os.path.join(LIB_DIR, f"lp_head_binding.torch-{metadata.version('torch')}.{sysconfig.get_config_var('SOABI')}.so")


def _binding_commands(work: str):
    """The binding's compiler and linker calls."""
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    obj, torch_lib = os.path.join(work, "binding.o"), os.path.join(torch_dir, "lib")
    includes = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
                os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    compile_ = [os.environ.get("CXX", "g++"), "-O2", "-std=c++20", "-fPIC", "-c", os.path.join(CSRC, BINDING), "-o", obj]
    for d in includes:
        compile_ += ["-isystem" if d != INCLUDE else "-I", d]
    tmp = binding_path() + f".tmp{os.getpid()}"
    link = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", LIB_DIR, f"-l:{LIB_NAME}", "-L", torch_lib,
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}"]
    return compile_, link, tmp


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS + [BINDING]]
    files += [os.path.join(INCLUDE, f) for f in ("lp_ragged.h", "lp_head.h")]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(lib_path()) or not os.path.exists(binding_path()):
        return False
    t = min(os.path.getmtime(lib_path()), os.path.getmtime(binding_path()))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _run(commands, verbose: bool) -> str:
    """Run the commands at once; return what they print, raise if one fails."""
    if verbose:
        print("\n".join(" ".join(c) for c in commands), file=sys.stderr)
    with ThreadPoolExecutor(len(commands)) as pool:
        results = list(pool.map(lambda c: subprocess.run(c, capture_output=True, text=True), commands))
    for cmd, res in zip(commands, results):
        if res.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    return "".join(res.stdout + res.stderr for res in results)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False, out: str | None = None,
          defines=()) -> str:
    """Compile the library if a source changed; return its path. ``defines`` (e.g.
    ``["LP_UNROLL=8"]``) override the kernel's tuning knobs; use with ``out``."""
    out = out or lib_path()
    if not force and not defines and out == lib_path() and up_to_date():
        return out
    os.makedirs(os.path.dirname(os.path.abspath(out)), exist_ok=True)
    tmp = out + f".tmp{os.getpid()}"
    flags = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC]
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]
    flags += [f"-D{d}" for d in defines]
    with tempfile.TemporaryDirectory(prefix="lp_build_") as work:
        objects = [os.path.join(work, f + ".o") for f in SOURCES]
        commands = [[_nvcc(), *flags, "-c", os.path.join(CSRC, f), "-o", o] for f, o in zip(SOURCES, objects)]
        binding = out == lib_path()
        if binding:
            binding_compile, binding_link, binding_tmp = _binding_commands(work)
            commands.append(binding_compile)
        # one compiler per source, all at once; then the links (the binding's against the library)
        report = _run(commands, verbose) + _run([[_nvcc(), *ARCH, "-shared", "-o", tmp, *objects]], verbose)
        os.replace(tmp, out)
        if binding:
            report += _run([binding_link], verbose)
            os.replace(binding_tmp, binding_path())
    if verbose or ptxas_verbose:
        sys.stderr.write(report)
    return out


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv)
