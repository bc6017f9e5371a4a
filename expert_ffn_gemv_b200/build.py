"""Build the sm_100a shared library libmoe_b200.so in-tree (nvcc, no JIT cache), and, where PyTorch is
installed, the host-side binding of the block operators for its tensors, _block_ext.so (g++).

    python -m expert_ffn_gemv_b200.build        # or: import expert_ffn_gemv_b200.build as b; b.build()
"""
from __future__ import annotations

import importlib.util
import os
import re
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
OUT_DIR = PKG / "_lib"
LIB = OUT_DIR / "libmoe_b200.so"
SOURCES = ["api.cu", "decode.cu", "repack.cu", "prefill.cu", "noalloc.cu", "norms.cu", "adapters.cu", "ffn.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", str(ROOT / "include"), "-I", str(CSRC)]


# CPython binding of the block operators for torch tensors (host code, built against the installed torch)
EXT = OUT_DIR / "_block_ext.so"
EXT_SOURCES = [CSRC / "bind.cpp", ROOT / "include" / "moe.h"]


def ext_target() -> str:
    """What a binding has to be built against to be loaded here."""
    import torch

    return f"torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"


def ext_built_for(path: Path) -> str | None:
    """What a binding was built against (bind.cpp keeps it as text), None where it does not say."""
    m = re.search(rb"moe-block-ext-for:([^\0]*)\0", path.read_bytes())
    return m.group(1).decode() if m else None


def build_ext(force: bool = False) -> Path:
    target = ext_target()
    if not force and EXT.exists() and all(p.stat().st_mtime <= EXT.stat().st_mtime for p in EXT_SOURCES) \
            and ext_built_for(EXT) == target:
        return EXT
    import sysconfig

    from torch.utils import cpp_extension as ce

    OUT_DIR.mkdir(exist_ok=True)
    cuda = str(Path(nvcc()).resolve().parent.parent / "include")
    inc = [*ce.include_paths(), cuda, sysconfig.get_paths()["include"], str(ROOT / "include")]
    import torch

    libs = Path(torch.__file__).parent / "lib"
    tmp = EXT.with_suffix(f".{os.getpid()}.tmp")
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++20", "-shared", "-fPIC", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f'-DMOE_EXT_TARGET="{target}"',
           *[f"-I{i}" for i in inc], str(CSRC / "bind.cpp"), "-o", str(tmp),
           f"-L{libs}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on bind.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)
    return EXT


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def _stale() -> bool:
    if not LIB.exists():
        return True
    t = LIB.stat().st_mtime
    deps = [p for p in CSRC.glob("*") if p.suffix != ".cpp"] + [ROOT / "include" / "moe.h", Path(__file__)]
    return any(p.stat().st_mtime > t for p in deps)


def build(force: bool = False, verbose: bool = False, defines=(), out: Path | None = None) -> Path:
    """Compile every .cu into one shared library; `defines` (e.g. ["MOE_DECODE_STAGES=2"]) and
    `out` build a variant elsewhere."""
    lib = LIB if out is None else Path(out)
    if not force and not defines and out is None and not _stale():
        return _with_ext(lib, force)
    OUT_DIR.mkdir(exist_ok=True)
    tag = "" if out is None else "_" + lib.stem
    objs = []

    def compile_one(src: str) -> Path:
        obj = OUT_DIR / (Path(src).stem + tag + ".o")
        cmd = [nvcc(), *ARCH, *FLAGS, *[f"-D{d}" for d in defines], "-c", str(CSRC / src), "-o", str(obj)]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = lib.with_suffix(f".{os.getpid()}.tmp")
    cmd = [nvcc(), *ARCH, "-shared", "-o", str(tmp), *map(str, objs)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    for o in objs:
        o.unlink(missing_ok=True)
    return lib if out is not None else _with_ext(lib, force)


def _with_ext(lib: Path, force: bool) -> Path:
    """The library needs nvcc alone: without PyTorch there is nothing to bind to."""
    if importlib.util.find_spec("torch") is not None:
        build_ext(force)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
