"""Build libqmm.so (HIP, gfx950) in-tree with hipcc.

Sources are compiled to objects in parallel under _build/ and linked into
group_wise_affine_amd/libqmm.so. Flags:
  --offload-arch=gfx950                  CDNA4 only
  -fhip-fp32-correctly-rounded-divide-sqrt  IEEE division (the quantizer's
                                         codes depend on it)
  -Xclang -target-feature -Xclang -packed-fp32-ops
                                         no packed fp32 VALU instructions
The compiler's resource report says of every kernel in NO_SCRATCH that it spills
no vector registers, and the assembly of the sources in ASM_PRODUCTS that it
leaves the sums of matrix products written in assembly alone between them; a
build in which this is not so fails.
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
           "kv8_attn_window.hip", "kv8_attn_tree.hip", "kv8_pages.hip", "rope.hip", "logprobs.hip"]
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
NO_SCRATCH = {"i8.hip", "kv8.hip", "kv8_attn.hip", "kv8_attn_window.hip", "kv8_attn_tree.hip", "kv8_pages.hip",
              "rope.hip", "logprobs.hip"}
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


# Sources with matrix products in inline assembly, of whose results the compiler
# knows nothing: read or moved less than 12 instructions after the product, they
# are not there yet. The products' blocks stand in loops; the last block of an
# iteration ends with the wait where the loop ends.
ASM_PRODUCTS = {"i8.hip"}
_SUMS = re.compile(r"\ba(\d|\[\d)|accvgpr")


def check_products(src, asm):
    """Raises if, in this assembly, a sum (they are in the accumulation registers)
    is touched between one block of products and the next, on the way back of a
    loop too, or if the last block of a loop does not end with a wait."""
    found = 0
    for name, body in re.findall(r"^(_Z\w+):[^\n]*\n(.*?)^\.Lfunc_end", asm, re.S | re.M):
        lines = body.split("\n")
        code = [re.sub(r";.*", "", l).strip() if "#ASM" not in l else l.strip() for l in lines]
        blocks, start = [], None
        for i, l in enumerate(code):
            if l.endswith("#ASMSTART"):
                start = i
            elif l.endswith("#ASMEND") and any("v_mfma" in x for x in code[start:i]):
                blocks.append((start, i))
        found += len(blocks)

        def bad(what, i):
            raise RuntimeError(f"{src}: {name}: {what}: {lines[i].strip()}")

        for (a, end), nxt in zip(blocks, [*blocks[1:], None]):
            # as far as the code runs straight on to the next block
            stop = nxt[0] if nxt else len(code)
            branch = next((i for i in range(end, stop) if re.match(r"s_c?branch", code[i])), None)
            for i in range(end + 1, stop if branch is None else branch):
                if _SUMS.search(code[i]):
                    bad("a sum is touched between products", i)
            if branch is None and nxt:
                continue
            if not any(x.startswith("s_nop 15") for x in code[a:end]):
                bad("no wait after the last products", end)
            label = code[branch].split()[1] + ":" if branch is not None else None
            if label in code:   # the loop's way back, to its first block
                back = code.index(label)
                for i in range(back, next((s for s, _ in blocks if s > back), back)):
                    if back < end and _SUMS.search(code[i]):
                        bad("a sum is touched between products", i)
    if not found:
        raise RuntimeError(f"{src}: no matrix products in its assembly")


def _compile(src):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    checked = src in NO_SCRATCH
    cmd = [HIPCC, *FLAGS, *([REPORT, "-fno-caret-diagnostics"] if checked else []), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stderr}")
    if checked:
        check_no_scratch(src, r.stderr)
    if src in ASM_PRODUCTS:
        check_products(src, _assembly(src))
    # the host pass warns about the device-only target feature; drop that noise
    msgs = [l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l
            and "not a recognized feature" not in l and REPORT not in l
            and not l.startswith("In file included from")]
    return obj, "\n".join(msgs)


def _assembly(src):
    cmd = [HIPCC, *[f for f in FLAGS if f != "-fPIC"], "--cuda-device-only", "-S", os.path.join(CSRC, src), "-o", "-"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stderr}")
    return r.stdout


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
