"""Build the KDA CUDA library in-tree for sm_103a.

    python -m kda_chunked_prefill_02_gb300.build [--force] [--no-binding]

Compiles csrc/*.cu (one nvcc per translation unit, in parallel) and links
  libkda.so          the product library (C ABI of include/kda.h and include/kda_ops.h)
  libkda_selftest.so test-only checks of the tcgen05 / TMA building blocks
  _kda_ops.so        the Python binding of include/kda_ops.h (csrc/ops_binding.cpp)
next to this file.  Objects go to _build/ (git-ignored).  The first two need nvcc
alone; the binding, which only Python callers use, needs torch with its headers
and g++, and is left out with --no-binding or where there is no torch.
"""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
ROOT = os.path.dirname(HERE)
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "-I" + os.path.join(ROOT, "include"), "-diag-suppress", "1160"]

LIB_SOURCES = ["kda_api.cu", "kda_prep.cu", "kda_state.cu", "kda_state_head.cu", "kda_verify.cu",
               "kda_verify_wy.cu", "kda_noalloc.cu", "kda_host.cu", "kda_ops_api.cu", "kda_conv.cu",
               "kda_rope.cu", "kda_tree.cu", "kda_tree_mma.cu", "kda_chunk.cu",
               "kda_chunk_mma.cu", "kda_residual.cu", "kda_pool.cu"]
SELFTEST_SOURCES = ["selftest.cu"]
BINDING_SOURCE = "ops_binding.cpp"
HEADERS = ["sm103.cuh", "kda_internal.h", "ops_internal.h", "warp_mma.cuh", "attn_mma.cuh", "tmap.h"]

LIB = os.path.join(HERE, "libkda.so")
SELFTEST_LIB = os.path.join(HERE, "libkda_selftest.so")
BINDING = os.path.join(HERE, "_kda_ops.so")


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest_input(srcs):
    files = [os.path.join(CSRC, s) for s in srcs + HEADERS] + [
        os.path.join(ROOT, "include", "kda.h"), os.path.join(ROOT, "include", "kda_ops.h"),
        os.path.abspath(__file__)]
    return max(os.path.getmtime(f) for f in files)


def _compile(src):
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [_nvcc()] + ARCH + FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    return obj


def _link(objs, out):
    tmp = out + ".tmp.%d" % os.getpid()
    cmd = [_nvcc()] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed for %s:\n%s\n%s" % (out, r.stdout, r.stderr))
    os.replace(tmp, out)


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s\n%s" % (what, r.stdout, r.stderr))


def _compile_binding():
    """The Python binding against this interpreter's torch."""
    import torch
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    inc = [root, os.path.join(root, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
           os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    obj = os.path.join(BUILD, "ops_binding.o")
    _run(["g++", "-O2", "-fPIC", "-std=c++17", "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
          "-c", os.path.join(CSRC, BINDING_SOURCE), "-o", obj] + ["-I" + i for i in inc], "g++ for " + BINDING_SOURCE)
    return obj


def _link_binding(obj):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp.%d" % os.getpid()
    _run(["g++", "-shared", obj, "-o", tmp, "-L" + HERE, "-l:libkda.so", "-Wl,-rpath,$ORIGIN", "-L" + lib, "-lc10",
          "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath," + lib], "link of " + BINDING)
    os.replace(tmp, BINDING)


def _torch_is_there() -> bool:
    try:
        import torch  # noqa: F401
    except ImportError:
        print("no torch: %s is left out (the C library is complete)" % os.path.basename(BINDING), file=sys.stderr)
        return False
    return True


def build(force: bool = False, binding: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    todo = []
    for out, srcs in ((LIB, LIB_SOURCES), (SELFTEST_LIB, SELFTEST_SOURCES)):
        if force or not os.path.exists(out) or os.path.getmtime(out) < _newest_input(srcs):
            todo.append((out, srcs))
    if binding:
        stale = force or not os.path.exists(BINDING) or os.path.getmtime(BINDING) < _newest_input([BINDING_SOURCE])
        binding = stale and _torch_is_there()
    if not todo and not binding:
        return LIB
    all_srcs = sorted({s for _, srcs in todo for s in srcs})
    with cf.ThreadPoolExecutor(max_workers=min(8, len(all_srcs) + 1)) as ex:
        bound = ex.submit(_compile_binding) if binding else None
        objs = dict(zip(all_srcs, ex.map(_compile, all_srcs)))
    for out, srcs in todo:
        _link([objs[s] for s in srcs], out)
    if bound:
        _link_binding(bound.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, binding="--no-binding" not in sys.argv))
