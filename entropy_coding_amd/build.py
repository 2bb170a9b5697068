"""Builds libkvc.so in-tree with hipcc for gfx950.

Flags that matter for bit-exactness of the shared CDF: no floating-point
contraction (-ffp-contract=off), float32 denormals kept
(-fno-gpu-flush-denormals-to-zero), and no packed-fp32 instructions.
"""
import concurrent.futures
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkvc.so")
ARCH = os.environ.get("KVC_OFFLOAD_ARCH", "gfx950")

KERNELS = ["kvc_kernels.hip", "kvc_paged.hip", "kvc_attention.hip", "kvc_attention_wide.hip"]
HOST = ["kvc_api.cpp", "kvc_paged_api.cpp"]

COMMON = [
    "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off",
    "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
]
DEVICE = [
    "-x", "hip", f"--offload-arch={ARCH}", "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]
RESOURCES = "-Rpass-analysis=kernel-resource-usage"     # (what a kernel takes, as remarks)


def hipcc() -> str:
    for c in (os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc"), shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found")


def resource_file(src: str) -> str:
    return os.path.join(HERE, "_build", os.path.splitext(src)[0] + ".resources")


def resources(src: str) -> dict:
    """What the kernels of a source take, as its last build() reported it:
    {kernel's mangled name: {"VGPRs": ..., "ScratchSize [bytes/lane]": ..., ...}}."""
    kernels, at = {}, None
    with open(resource_file(src)) as f:
        for line in f:
            key, value = re.search(r"remark:\s*([^:]+): (\S+) \[", line).groups()
            if key == "Function Name":
                at = kernels.setdefault(value, {})
            else:
                at[key] = int(value) if value.isdigit() else value
    return kernels


def build(verbose: bool = False) -> str:
    cc = hipcc()
    obj_dir = os.path.join(HERE, "_build")
    os.makedirs(obj_dir, exist_ok=True)
    rocm = os.path.dirname(os.path.dirname(cc))
    host_cxx = shutil.which("g++") or "g++"
    host = ["-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(rocm, "include"), "-Wall", "-Wextra"]
    steps = [(cc, src, [*DEVICE, RESOURCES]) for src in KERNELS]
    # the C ABI layer is host code only: plain g++ against the HIP runtime API
    steps += [(host_cxx, src, host) for src in HOST]

    def compile_one(step):
        comp, src, extra = step
        obj = os.path.join(obj_dir, os.path.splitext(src)[0] + ".o")
        cmd = [comp, *COMMON, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        done = subprocess.run(cmd, stderr=subprocess.PIPE, text=True)
        remarks = [x for x in done.stderr.splitlines() if RESOURCES in x]
        if done.returncode or verbose or not remarks:
            print(done.stderr, end="", file=sys.stderr)
        done.check_returncode()
        if remarks:
            with open(resource_file(src), "w") as f:
                f.write("\n".join(remarks) + "\n")
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=4) as pool:
        objs = list(pool.map(compile_one, steps))
    tmp = LIB + ".tmp"
    cmd = [cc, "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


CHECKED_DIR = os.path.join(HERE, "_build", "checked")
CHECKED_LIB = os.path.join(CHECKED_DIR, "libkvc_checked.so")


def build_checked(verbose: bool = False) -> str:
    """A second build for the CPU tests only: the C ABI layer (HOST) compiled with
    AddressSanitizer and UndefinedBehaviorSanitizer (g++; any finding aborts
    the process), linked with the same device code into
    _build/checked/libkvc_checked.so.  The host tests load it in a child
    process that preloads the sanitizer runtime (the Python interpreter is
    not built with it).  It is never loaded on a GPU."""
    cc = hipcc()
    os.makedirs(CHECKED_DIR, exist_ok=True)
    rocm = os.path.dirname(os.path.dirname(cc))
    obj = lambda where, src: os.path.join(where, os.path.splitext(src)[0] + ".o")
    kern = {src: obj(os.path.join(HERE, "_build"), src) for src in KERNELS}     # the device code of build()
    api = {src: obj(CHECKED_DIR, src) for src in HOST}
    host_cxx = shutil.which("g++") or "g++"
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g"]
    cmds = [[cc, *COMMON, *DEVICE, "-c", os.path.join(CSRC, src), "-o", o]
            for src, o in kern.items() if not os.path.exists(o)]
    cmds += [[host_cxx, *[f for f in COMMON if f != "-O3"], "-O1", *san, "-D__HIP_PLATFORM_AMD__",
              "-I" + os.path.join(rocm, "include"), "-Wall", "-Wextra", "-c", os.path.join(CSRC, src), "-o", o]
             for src, o in api.items()]
    cmds += [
        [host_cxx, "-shared", *san, *kern.values(), *api.values(), "-o", CHECKED_LIB + ".tmp", "-L" + os.path.join(rocm, "lib"),
         "-Wl,-rpath," + os.path.join(rocm, "lib"), "-lamdhip64"],
    ]
    for cmd in cmds:
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
    os.replace(CHECKED_LIB + ".tmp", CHECKED_LIB)
    return CHECKED_LIB


if __name__ == "__main__":
    print(build(verbose=True))
    if "--checked" in sys.argv:
        print(build_checked(verbose=True))
