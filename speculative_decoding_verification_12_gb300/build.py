"""Builds the CUDA library in-tree for sm_103a (GB300) with nvcc, and the compiled binding with g++.

The shared objects land next to this file as libspecverify.so and _binding.so.  The library links
the CUDA runtime dynamically, so a process that already loaded PyTorch's libcudart.so.13 shares
it; the binding links PyTorch's libraries, which its user has loaded.
"""
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libspecverify.so")
BINDING = os.path.join(HERE, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def deps():
    out = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    include = os.path.join(os.path.dirname(HERE), "include")
    out.extend(os.path.join(include, f) for f in sorted(os.listdir(include)))
    return out


def start_binding(tmp: str):
    """The g++ process that compiles the binding to `tmp`; None without PyTorch, for whose users it is."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    torch = list(spec.submodule_search_locations)[0]
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("g++ not found")
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", f"-I{torch}/include",
           f"-I{sysconfig.get_paths()['include']}", "-o", tmp, os.path.join(CSRC, "binding.cpp"), f"-L{torch}/lib",
           "-ltorch_python", "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{torch}/lib"]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libspecverify.so and _binding.so unless they are newer than every source.  Each
    translation unit (one per logits dtype and scheme, the entry points, the cache-side kernels)
    compiles in its own process, in parallel; one link makes the library.  The library comes first:
    it is there also where the binding is not (no PyTorch) or fails to compile (which raises)."""
    made = [LIB] + ([BINDING] if importlib.util.find_spec("torch") else [])
    if not force and all(os.path.exists(p) for p in made):
        t = min(os.path.getmtime(p) for p in made)
        if all(os.path.getmtime(p) <= t for p in deps()):
            return LIB
    tag = f"{os.getpid()}"
    objs, procs = [], []
    for src in sources():
        obj = os.path.join(CSRC, os.path.basename(src)[:-3] + f".{tag}.o")
        cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-c", "-o", obj, src]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        objs.append(obj)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    binding_tmp = BINDING + f".tmp{tag}"
    binding = start_binding(binding_tmp)
    failed = False
    for src, pr in procs:
        out, _ = pr.communicate()
        if pr.returncode != 0 or verbose:
            sys.stderr.write(out)
        failed = failed or pr.returncode != 0
    binding_out = binding.communicate()[0] if binding else ""
    try:
        if failed:
            raise RuntimeError("nvcc failed building libspecverify.so")
        tmp = LIB + f".tmp{tag}"
        res = subprocess.run([nvcc(), *ARCH, "-shared", "-cudart", "shared", "-Xlinker",
                              "-rpath,/usr/local/cuda/lib64", "-o", tmp, *objs], capture_output=True, text=True)
        if res.returncode != 0:
            sys.stderr.write(res.stdout + res.stderr)
            raise RuntimeError("linking libspecverify.so failed")
        os.replace(tmp, LIB)
        if binding is not None:
            if binding.returncode != 0 or verbose:
                sys.stderr.write(binding_out)
            if binding.returncode != 0:
                raise RuntimeError("compiling _binding.so failed")
            os.replace(binding_tmp, BINDING)
    finally:
        for o in [*objs, binding_tmp]:
            if os.path.exists(o):
                os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
