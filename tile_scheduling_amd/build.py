"""Build libtsgemm.so (HIP kernels + C ABI) for gfx950, and the Python module _binding.so over it, in-tree.

    python tile_scheduling_amd/build.py      # once built, also: python -m tile_scheduling_amd.build

Each .hip file under csrc/ is compiled to an object in parallel with hipcc, then
linked into tile_scheduling_amd/libtsgemm.so.  Packed fp32 instructions are
disabled for every HIP compilation (-packed-fp32-ops).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libtsgemm.so")
BINDING = os.path.join(HERE, "_binding.so")
ARCH = "gfx950"

HIPFLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


# the compiler's per-kernel resource report (registers, spills, LDS, occupancy)
REMARKS = ["-Rpass-analysis=kernel-resource-usage"]
_FIELDS = {"TotalSGPRs": "sgprs", "VGPRs": "vgprs", "AGPRs": "agprs", "ScratchSize [bytes/lane]": "scratch",
           "Occupancy [waves/SIMD]": "occupancy", "SGPRs Spill": "sgpr_spill", "VGPRs Spill": "vgpr_spill",
           "LDS Size [bytes/block]": "lds"}
_RE_NAME = re.compile(r"remark: Function Name: (\S+)")
_RE_FIELD = re.compile(r"remark:\s+([A-Za-z][A-Za-z /\[\]]*?): (\d+)")


def parse_resource_remarks(text: str) -> dict:
    """{mangled kernel name: {field: value}} from -Rpass-analysis=kernel-resource-usage output."""
    table, cur = {}, None
    for line in text.splitlines():
        m = _RE_NAME.search(line)
        if m:
            cur = table.setdefault(m.group(1), {})
            continue
        m = _RE_FIELD.search(line)
        if m and cur is not None and m.group(1) in _FIELDS:
            cur[_FIELDS[m.group(1)]] = int(m.group(2))
    return table


def _compile(src: str, extra, verbose: bool):
    obj = os.path.join(BUILD, os.path.basename(src)[:-4] + ".o")
    cmd = [_hipcc()] + HIPFLAGS + REMARKS + list(extra) + ["-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, parse_resource_remarks(r.stderr)


def write_resource_table(table: dict, path: str) -> None:
    """A C++ source holding the compiler's resource report of every kernel, sorted by
    mangled name, for ts_query (looked up through the kernel handle's symbol name)."""
    keys = ("vgprs", "agprs", "sgprs", "scratch", "vgpr_spill", "sgpr_spill", "occupancy", "lds")
    lines = ["// Generated by tile_scheduling_amd/build.py from the compiler's kernel resource report.",
             '#include "resource_table.hpp"', "namespace ts {", "const KernelResources kKernelResources[] = {"]
    for name in sorted(table):
        v = table[name]
        lines.append('    {"%s", %s},' % (name, ", ".join(str(v.get(k, -1)) for k in keys)))
    lines += ["};", f"const int kNumKernelResources = {len(table)};", "}  // namespace ts", ""]
    with open(path, "w") as f:
        f.write("\n".join(lines))


def _local_includes(path: str, seen=None) -> set:
    """`path` and every csrc/ header it includes with #include "...", transitively."""
    seen = set() if seen is None else seen
    if path in seen or not os.path.exists(path):
        return seen
    seen.add(path)
    with open(path) as f:
        for line in f:
            m = re.match(r'\s*#\s*include\s+"([^"]+)"', line)
            if m:
                _local_includes(os.path.normpath(os.path.join(os.path.dirname(path), m.group(1))), seen)
    return seen


def _up_to_date(src: str) -> bool:
    """The object of `src` and its recorded resource report are newer than `src`
    and every header it includes (for --incremental rebuilds)."""
    obj = os.path.join(BUILD, os.path.basename(src)[:-4] + ".o")
    rep = obj + ".res"
    if not (os.path.exists(obj) and os.path.exists(rep)):
        return False
    newest = max(os.path.getmtime(f) for f in _local_includes(src))
    return min(os.path.getmtime(obj), os.path.getmtime(rep)) > newest


def _compile_cached(src: str, extra, verbose: bool, incremental: bool):
    import json

    obj = os.path.join(BUILD, os.path.basename(src)[:-4] + ".o")
    if incremental and _up_to_date(src):
        with open(obj + ".res") as f:
            return obj, json.load(f)
    obj, table = _compile(src, extra, verbose)
    with open(obj + ".res", "w") as f:
        json.dump(table, f)
    return obj, table


def build(verbose: bool = False, extra=(), jobs: int = 0, incremental: bool = False) -> str:
    """Compile every csrc/*.hip (all of them, unless `incremental`) and link the library."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    jobs = jobs or min(len(srcs), max(1, min(16, os.cpu_count() or 1)))
    with cf.ThreadPoolExecutor(jobs) as ex:
        results = list(ex.map(lambda s: _compile_cached(s, extra, verbose, incremental), srcs))
    objs = [o for o, _ in results]
    table = {}
    for _, t in results:
        table.update(t)
    gen = os.path.join(BUILD, "resource_table.cpp")
    write_resource_table(table, gen)
    gen_obj = gen[:-4] + ".o"
    subprocess.run([_hipcc(), "-O2", "-std=c++17", "-fPIC", "-I", CSRC, "-c", gen, "-o", gen_obj], check=True)
    objs.append(gen_obj)
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs + ["-ldl"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    build_binding(verbose)
    return LIB


def build_binding(verbose: bool = False) -> str:
    """The Python module of the operators' calls (csrc/binding.cpp), against the torch that is installed."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    lib_dir = os.path.join(os.path.dirname(torch.__file__), "lib")
    # it takes the tensors of one torch and the calls of one Python: __init__.py compares
    target = f"torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wno-unknown-pragmas", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DTS_BUILT_FOR="{target}"']
    cmd += [f"-I{d}" for d in cpp_extension.include_paths() + [sysconfig.get_paths()["include"],
            os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_hipcc()))), "include")]]
    cmd += [os.path.join(CSRC, "binding.cpp"), "-o", tmp, f"-L{lib_dir}", "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python",
            f"-L{HERE}", "-l:libtsgemm.so", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    return BINDING


if __name__ == "__main__":
    print(build(verbose="-q" not in sys.argv, incremental="--incremental" in sys.argv))
