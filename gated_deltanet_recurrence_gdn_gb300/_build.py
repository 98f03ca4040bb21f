"""Builds libgdn.so in-tree with nvcc for sm_103a (no cmake, no torch), and beside it, where that can
be done, _bind.so, the binding's native part, with the host compiler against Python's and PyTorch's
headers."""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdn.so")
BIND, BIND_SRC = os.path.join(PKG, "_bind.so"), os.path.join(CSRC, "gdn_bind.cpp")
BIND_MADE_OF = os.path.join(BUILD, "bind.txt")     # what _bind.so was built by and against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC = os.environ.get("NVCC", "nvcc")


def _flags():
    return ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                   "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(out, deps):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch():
    """PyTorch's folder (it is not imported for this), None where there is none."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _bind_job(at, out):
    """The command that builds _bind.so as `out` against PyTorch in folder `at`."""
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    system = [sysconfig.get_paths()["include"], os.path.join(at, "include"),
              os.path.join(at, "include", "torch", "csrc", "api", "include"),
              os.path.join(cuda, "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           "-I", os.path.join(ROOT, "include")]
    for path in system:
        cmd += ["-isystem", path]
    return cmd + [BIND_SRC, "-o", out, "-L" + os.path.join(at, "lib"), "-ltorch_python",
                  "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _bind_made_of(at):
    """What a _bind.so is good for: the command, Python's ABI, and the PyTorch, whatever its date."""
    with open(os.path.join(at, "version.py")) as f:
        version = f.read()
    return "\n".join(_bind_job(at, "") + [str(sysconfig.get_config_var("SOABI")), version])


def _build_bind(force, headers, run):
    """Builds _bind.so where it is not up to date.  Answers why that cannot be done (None: it is
    done): calls then go by Python, and one that is out of date is taken away."""
    at = _torch()
    if at is None:
        return "there is no PyTorch"
    tmp = BIND + ".tmp%d" % os.getpid()
    try:
        made_of = _bind_made_of(at)
        if not force and not _stale(BIND, [BIND_SRC] + headers) and os.path.exists(BIND_MADE_OF):
            with open(BIND_MADE_OF) as f:
                if f.read() == made_of:
                    return None
        run(_bind_job(at, tmp))
        os.replace(tmp, BIND)
        with open(BIND_MADE_OF, "w") as f:
            f.write(made_of)
        return None
    except (OSError, RuntimeError) as e:
        for path in (tmp, BIND):
            if os.path.exists(path):
                os.remove(path)
        return str(e)


# Build variants: name -> extra nvcc flags.  "check" is the debug
# bounds-check build (csrc/gdn_check.cuh); its objects and library sit beside
# the normal ones under their own names.
VARIANTS = {"check": ["-DGDN_BOUNDS_CHECK"]}


def build_variant(name: str, force: bool = False, verbose: bool = False) -> str:
    return build(force=force, verbose=verbose, extra=VARIANTS[name], variant=name)


def build(force: bool = False, verbose: bool = False, extra=(), variant=None) -> str:
    build_dir = BUILD if variant is None else os.path.join(PKG, "_build_" + variant)
    lib_path = LIB if variant is None else os.path.join(PKG, "libgdn_%s.so" % variant)
    os.makedirs(build_dir, exist_ok=True)
    headers = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    objs = []
    jobs = []
    for src in sources():
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            jobs.append([NVCC] + _flags() + list(extra) + ["-c", src, "-o", obj])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("compiler failed:\n%s\n%s" % (" ".join(cmd), r.stdout + r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)

    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        bind = ex.submit(_build_bind, force, headers, run) if variant is None else None
        list(ex.map(run, jobs))
    error = bind.result() if bind else None
    if error:
        warnings.warn("the binding's native part is not built: %s" % error, RuntimeWarning)
    if force or jobs or _stale(lib_path, objs):
        tmp = lib_path + ".tmp%d" % os.getpid()
        run([NVCC] + ARCH + ["-shared", "-o", tmp] + objs)
        os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
