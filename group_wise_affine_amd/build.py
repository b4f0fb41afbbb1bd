"""Build libqmm.so (HIP, gfx950) in-tree with hipcc.

Sources are compiled to objects in parallel under _build/ and linked into
group_wise_affine_amd/libqmm.so. Flags:
  --offload-arch=gfx950                  CDNA4 only
  -fhip-fp32-correctly-rounded-divide-sqrt  IEEE division (the quantizer's
                                         codes depend on it)
  -Xclang -target-feature -Xclang -packed-fp32-ops
                                         no packed fp32 VALU instructions
The compiler's resource report says of every kernel in NO_SCRATCH that it spills
no vector registers; a build in which one does fails.
"""
import concurrent.futures as cf
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libqmm.so")
CEILING_LIB = os.path.join(HERE, "libqmm_ceiling.so")
BINDING = os.path.join(HERE, "_serving.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = ["api.cpp", "quantize.hip", "qmv.hip", "qmn.hip", "qmn_tile.hip", "fpq.hip", "apk.hip", "qmv_mfma_f16.hip", "qmv_mfma_bf16.hip", "qmm.hip",
           "tile_gemm_f16.hip", "tile_gemm_bf16.hip", "tile_conv_f16.hip", "tile_conv_bf16.hip",
           "tile_fp.hip", "tile_apk.hip", "api_serving.cpp", "i8.hip", "kv8.hip", "kv8_attn.hip",
           "kv8_pages.hip"]
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++20", "-fPIC",
    "-fhip-fp32-correctly-rounded-divide-sqrt", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unknown-warning-option",
    "-I" + os.path.join(ROOT, "include"),
]

# Sources whose kernels may not use scratch memory: the compiler has put the
# stores of spilled registers between a branch that some lanes take and its end,
# so that the other lanes read back what they never stored.
NO_SCRATCH = {"i8.hip", "kv8.hip", "kv8_attn.hip", "kv8_pages.hip"}
REPORT = "-Rpass-analysis=kernel-resource-usage"


def check_no_scratch(src, report):
    """Raises unless the compiler's resource report names kernels of src and no
    scratch memory or spilled vector register in any of them."""
    kernel, seen, bad = None, set(), []
    for line in report.splitlines():
        m = re.search(r"remark: .*?(Function Name|ScratchSize \[bytes/lane\]|VGPRs Spill): (\S+)", line)
        if not m:
            continue
        if m[1] == "Function Name":
            kernel = m[2]
            continue
        seen.add((kernel, m[1]))
        if m[2] != "0":
            bad.append(f"{kernel}: {m[1]} {m[2]}")
    kernels = {k for k, _ in seen}
    if not kernels or len(seen) != 2 * len(kernels):
        raise RuntimeError(f"{src}: the compiler reported no kernel's registers ({REPORT})")
    if bad:
        raise RuntimeError(f"{src}: kernels that may not use scratch memory do:\n" + "\n".join(bad))


def _compile(src):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    checked = src in NO_SCRATCH
    cmd = [HIPCC, *FLAGS, *([REPORT, "-fno-caret-diagnostics"] if checked else []), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stderr}")
    if checked:
        check_no_scratch(src, r.stderr)
    # the host pass warns about the device-only target feature; drop that noise
    msgs = [l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l
            and "not a recognized feature" not in l and REPORT not in l]
    return obj, "\n".join(msgs)


def build(verbose=False, jobs=None):
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(len(SOURCES), os.cpu_count() or 4, 16)
    with cf.ThreadPoolExecutor(jobs) as ex:
        results = list(ex.map(_compile, SOURCES))
    objs = []
    for obj, msg in results:
        objs.append(obj)
        if verbose and msg.strip():
            print(msg)
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-Wl,-soname,libqmm.so", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stderr}")
    os.replace(tmp, LIB)
    build_ceiling()
    build_binding()
    return LIB


def build_ceiling():
    """libqmm_ceiling.so: the benchmark's single-launch floor kernels
    (csrc/ceiling.hip, include/qmm_ceiling.h), separate from libqmm."""
    tmp = CEILING_LIB + ".tmp"
    cmd = [HIPCC, *FLAGS, "-shared", os.path.join(CSRC, "ceiling.hip"), "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for ceiling.hip:\n{' '.join(cmd)}\n{r.stderr}")
    os.replace(tmp, CEILING_LIB)
    return CEILING_LIB


def build_binding():
    """_serving.so: the native part of the Python binding (csrc/binding.cpp),
    host code against PyTorch's headers, linked to libqmm.so beside it."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall",
           "-D__HIP_PLATFORM_AMD__", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", "/opt/rocm/include",
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, LIB,
           "-L" + os.path.join(root, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python",
           "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,$ORIGIN", "-Wl,--no-as-needed"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for binding.cpp:\n{r.stderr}")
    os.replace(tmp, BINDING)
    return BINDING


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
