"""Builds libpsgd.so in-tree with nvcc for sm_103a (GB300).

Each translation unit is compiled in its own nvcc process, in parallel, then
linked into one shared library.  Used by ``__graft_entry__.build()``.

Whether to rebuild is decided by content, not by file times: a SHA-256 over
every source file, the public header, this script, the compiler flags and
``nvcc --version`` is compiled into the library (``psgd_build_id()``), and an
existing ``libpsgd.so`` is reused only when it carries that exact hash and was
built for this machine's architecture.  The training operators' Python binding
``_bind.so`` (host code only, against torch's and Python's headers) is built
beside it and carries the same hash with torch's and Python's versions.  The
library needs nvcc alone: where torch, its CUDA headers, Python's headers or g++
are missing the binding is left out with a note, and where the binding does not
compile the library is in place before that is raised.  ``-Xptxas -v`` register,
spill and shared-memory lines of every kernel are written to ``_build/ptxas.log``.
"""

from __future__ import annotations

import concurrent.futures
import hashlib
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpsgd.so")
BIND = os.path.join(HERE, "_bind.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
PTXAS_LOG = os.path.join(BUILD, "ptxas.log")

SOURCES = ["psgd_api.cu", "psgd_misc.cu", "psgd_static.cu", "psgd_group.cu",
           "psgd_embedding.cu", "psgd_layernorm.cu", "psgd_distill.cu"] + \
          [f"kern_rp{r}.cu" for r in (1, 2, 4, 8, 16, 32)]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v", "-I", INCLUDE]
BIND_SOURCE = "psgd_bind.cpp"
BIND_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wno-attributes"]
HASH_MARKER = b"psgd-source-hash:"
BIND_MARKER = b"psgd-bind-hash:"

# ELF e_machine of the machines this builds on
_ELF_MACHINE = {"x86_64": 62, "aarch64": 183, "arm64": 183}


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libpsgd.so")
    return cand


def source_hash() -> str:
    """SHA-256 (hex, 32 chars) of everything the library is built from."""
    h = hashlib.sha256()
    for f in sorted(os.listdir(CSRC)):
        path = os.path.join(CSRC, f)
        if os.path.isfile(path):
            h.update(f.encode() + b"\0")
            with open(path, "rb") as fh:
                h.update(fh.read())
    for path in (os.path.join(INCLUDE, "psgd.h"), os.path.abspath(__file__)):
        with open(path, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(ARCH + FLAGS + SOURCES + [BIND_SOURCE] + BIND_FLAGS).encode())
    try:
        h.update(subprocess.run([_nvcc(), "--version"], capture_output=True, text=True).stdout.encode())
    except Exception:
        h.update(b"nvcc-unknown")
    return h.hexdigest()[:32]


def bind_hash() -> str:
    """What the binding depends on: the sources, and the torch and Python it is
    compiled against."""
    import torch

    h = hashlib.sha256(source_hash().encode())
    h.update(f"{torch.__version__} {sys.version}".encode())
    return h.hexdigest()[:32]


def library_hash(path: str = LIB, marker: bytes = HASH_MARKER):
    """The source hash compiled into an existing library file, or None when it
    is missing, has none, or was built for another architecture."""
    try:
        with open(path, "rb") as fh:
            data = fh.read()
    except OSError:
        return None
    if len(data) < 20 or data[:4] != b"\x7fELF":
        return None
    want = _ELF_MACHINE.get(platform.machine())
    got = int.from_bytes(data[18:20], "little")
    if want is not None and got != want:
        return None
    i = data.find(marker)
    if i < 0:
        return None
    j = i + len(marker)
    return data[j:j + 32].decode("ascii", "replace")


def _bind_command(obj):
    """The compiler's command line for the binding's one object file."""
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    return ["g++", *BIND_FLAGS, f'-DPSGD_BIND_HASH="{bind_hash()}"', f'-DPSGD_SOURCE_HASH="{source_hash()}"',
            f'-DPSGD_BIND_TORCH="{torch.__version__}"',
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", inc, "-isystem",
            os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda, "-isystem",
            sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, BIND_SOURCE), "-o", obj]


def _binding_obstacle():
    """Why this machine cannot build the binding, or None."""
    try:
        import torch
    except Exception as e:  # ImportError, or a library that torch itself misses
        return f"torch cannot be imported ({e})"
    for header in (os.path.join(os.path.dirname(torch.__file__), "include", "c10", "cuda", "CUDAStream.h"),
                   os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(header):
            return f"{header} is missing"
    return None if shutil.which("g++") else "g++ is missing"


def build(force: bool = False, verbose: bool = False) -> str:
    obstacle = _binding_obstacle()
    want, want_bind = source_hash(), None if obstacle else bind_hash()
    lib_ok = not force and library_hash() == want
    bind_ok = bool(obstacle) or (not force and library_hash(BIND, BIND_MARKER) == want_bind)
    if obstacle:
        print(f"the training operators' Python binding is not built: {obstacle}", file=sys.stderr)
    if lib_ok and bind_ok:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        if src == BIND_SOURCE:
            cmd = _bind_command(obj)
        else:
            extra = [f'-DPSGD_SOURCE_HASH="{want}"'] if src == "psgd_api.cu" else []
            cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed on {src}:\n{r.stderr}")
        return src, r.stderr

    sources = ([] if bind_ok else [BIND_SOURCE]) + ([] if lib_ok else SOURCES)
    workers = min(len(sources), max(1, os.cpu_count() or 1))
    with concurrent.futures.ThreadPoolExecutor(max_workers=workers) as ex:
        jobs = {src: ex.submit(compile_one, src) for src in sources}
    if not lib_ok:
        results = [jobs[src].result() for src in SOURCES]
        with open(PTXAS_LOG, "w") as log:
            log.write(f"source hash {want}\n")
            for src, err in results:
                log.write(f"==== {src}\n{err}")
        if verbose:
            for src, err in results:
                spills = [ln for ln in err.splitlines() if "spill" in ln and not ln.strip().startswith("0 bytes")]
                bad = [ln for ln in spills if " 0 bytes spill stores, 0 bytes spill loads" not in ln]
                if bad:
                    print(f"{src}: " + "\n".join(bad), file=sys.stderr)
        objs = [os.path.join(BUILD, s.replace(".cu", ".o")) for s in SOURCES]
        _link([nvcc, *ARCH, "-shared"], objs, LIB)
        if library_hash() != want:
            raise RuntimeError("the built library does not carry its source hash")
    if not bind_ok:
        import torch

        jobs[BIND_SOURCE].result()
        torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
        _link(["g++", "-shared"], [os.path.join(BUILD, "psgd_bind.o"), "-L", HERE, "-l:libpsgd.so", "-Wl,-rpath,$ORIGIN",
                                  "-L", torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], BIND)
        if library_hash(BIND, BIND_MARKER) != want_bind:
            raise RuntimeError("the built binding does not carry its hash")
    return LIB


def _link(command, objects, target):
    tmp = target + ".tmp"
    r = subprocess.run([*command, "-o", tmp, *objects], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {os.path.basename(target)} failed:\n{r.stderr}")
    os.replace(tmp, target)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
