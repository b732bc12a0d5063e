"""Build ``libfmha_gb300.so`` (and its checked twin) in-tree for sm_103a.

Each ``csrc/*.cu`` translation unit is compiled by nvcc in parallel
(``-gencode arch=compute_103a,code=sm_103a -lineinfo -O3``) and linked into one
shared library next to this file.  The checked build compiles the same sources
with ``-DFMHA_CHECKED`` (every computed index of the kernels is tested before
its access, see ``include/fmha.h``) into ``libfmha_gb300_checked.so``.  The Python
binding's argument packer, ``csrc/tensor_args.cpp``, is built by g++ against the installed
torch into the extension module ``_tensor_args.so``; the libraries need neither, and are
built where it cannot be.  Usage:
``python -m head_attention_forward_fmha_gb300.build [--force] [--verbose]
[--checked | --all]``.
"""
import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libfmha_gb300.so")
CHECKED_LIB_PATH = os.path.join(PKG, "libfmha_gb300_checked.so")
ARGS_SRC = os.path.join(CSRC, "tensor_args.cpp")
ARGS_PATH = os.path.join(PKG, "_tensor_args.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _variant(checked):
    """(library path, object directory, extra nvcc flags) of one build variant."""
    if checked:
        return CHECKED_LIB_PATH, BUILD_DIR + "_checked", ["-DFMHA_CHECKED"]
    return LIB_PATH, BUILD_DIR, []


def up_to_date(checked=False):
    lib = _variant(checked)[0]
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def build_args(force=False):
    """The argument packer; against another torch or Python than it was built with (a stamp says which) it is built again."""
    import torch

    stamp, built_for = os.path.join(BUILD_DIR, "tensor_args.torch"), "%s %s" % (torch.__version__, sys.version)
    if not force and os.path.exists(ARGS_PATH) and os.path.exists(stamp) and open(stamp).read() == built_for and \
            os.path.getmtime(ARGS_PATH) >= max(os.path.getmtime(ARGS_SRC), os.path.getmtime(os.path.abspath(__file__))):
        return ARGS_PATH
    gxx = os.environ.get("CXX") or shutil.which("g++")
    if not gxx:
        raise RuntimeError("g++ not found (set CXX)")
    os.makedirs(BUILD_DIR, exist_ok=True)
    home = os.path.dirname(os.path.abspath(torch.__file__))
    inc, lib = os.path.join(home, "include"), os.path.join(home, "lib")
    tmp = "%s.%d.tmp" % (ARGS_PATH, os.getpid())
    cmd = [gxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           "-I", sysconfig.get_paths()["include"], "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-I", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include"), ARGS_SRC,
           "-o", tmp, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on tensor_args.cpp:\n%s" % r.stdout)
    os.replace(tmp, ARGS_PATH)
    with open(stamp, "w") as f:
        f.write(built_for)
    return ARGS_PATH


def _build_variants(variants, force, verbose, extra_flags):
    _build_libraries(variants, force, verbose, extra_flags)
    try:
        build_args(force)
    except (ImportError, RuntimeError) as e:
        warnings.warn("the serving operators' argument packer was not built: %s" % e)


def _build_libraries(variants, force, verbose, extra_flags):
    todo = [c for c in variants if force or not up_to_date(c)]
    if not todo:
        return
    nvcc = _nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                     "--expt-relaxed-constexpr"] + list(extra_flags)
    if verbose:
        common += ["-Xptxas", "-v"]
    jobs = []
    for checked in todo:
        _, obj_dir, flags = _variant(checked)
        os.makedirs(obj_dir, exist_ok=True)
        for src in _sources():
            obj = os.path.join(obj_dir, os.path.splitext(os.path.basename(src))[0] + ".o")
            jobs.append((checked, src, obj, [nvcc] + common + flags + ["-c", src, "-o", obj]))

    def compile_one(job):
        r = subprocess.run(job[3], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        return job, r.returncode, r.stdout

    objs = {c: [] for c in todo}
    with cf.ThreadPoolExecutor(max_workers=max(1, min(16, os.cpu_count() or 1))) as ex:
        for (checked, src, obj, _), rc, out in ex.map(compile_one, jobs):
            if rc != 0:
                raise RuntimeError("nvcc failed on %s%s:\n%s" % (src, " (checked)" if checked else "", out))
            if verbose and out.strip():
                sys.stdout.write(out)
            objs[checked].append(obj)
    for checked in todo:
        lib = _variant(checked)[0]
        tmp = lib + ".tmp"
        cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs[checked] + ["-lcudart_static", "-ldl", "-lpthread", "-lrt"]
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s" % r.stdout)
        os.replace(tmp, lib)


def build(force=False, verbose=False, extra_flags=(), checked=False):
    """Build one variant (the normal library, or the checked one); returns its path."""
    _build_variants([checked], force, verbose, extra_flags)
    return _variant(checked)[0]


def build_all(force=False, verbose=False):
    """Build the normal and the checked library (all translation units in one pool)."""
    _build_variants([False, True], force, verbose, ())
    return LIB_PATH, CHECKED_LIB_PATH


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    g = ap.add_mutually_exclusive_group()
    g.add_argument("--checked", action="store_true", help="build only the checked library")
    g.add_argument("--all", action="store_true", help="build the normal and the checked library")
    args = ap.parse_args()
    if args.all:
        print("\n".join(build_all(force=args.force, verbose=args.verbose)))
    else:
        print(build(force=args.force, verbose=args.verbose, checked=args.checked))
