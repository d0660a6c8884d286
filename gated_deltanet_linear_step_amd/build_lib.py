"""Build libgdn.so (all HIP kernels + the C ABI) for gfx950, in-tree.

    python -m gated_deltanet_linear_step_amd.build_lib

hipcc cross-compiles for gfx950 without a GPU. Packed-FP32 instructions are
disabled for the device code (``-packed-fp32-ops``).
"""
from concurrent.futures import ThreadPoolExecutor
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libgdn.so")
SOURCES = ["gdn_api.cpp", "gdn_conv.hip", "gdn_decode.hip", "gdn_prefill.hip",
           "gdn_prefill_generic.hip", "gdn_linattn.hip",
           "gdn_linattn_bf16.hip", "gdn_linattn_f16.hip", "gdn_linattn_f32.hip", "gdn_norm.hip",
           "gdn_matmul.hip", "gdn_attn_api.cpp", "gdn_rope.hip", "gdn_pages.hip", "gdn_attn.hip",
           "gdn_attn_bf16.hip", "gdn_attn_f16.hip"]
ARCH = os.environ.get("GDN_OFFLOAD_ARCH", "gfx950")


def build(verbose: bool = False, out: str = LIB, defines=()) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    flags = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             # keep MFMA accumulators in ordinary VGPRs: the prefill carry scales
             # and converts its accumulators with VALU work every chunk
             "-mllvm", "-amdgpu-mfma-vgpr-form",
             "-Wall", "-Wno-unused-command-line-argument",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC] + [f"-D{d}" for d in defines]

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        # the host pass does not know the gfx950 packed-fp32 feature; drop that notice
        for line in (res.stdout + res.stderr).splitlines():
            if "packed-fp32-ops" not in line and "unused during compilation" not in line:
                print(line, file=sys.stderr)
        if res.returncode != 0:
            raise subprocess.CalledProcessError(res.returncode, cmd)

    # one compilation per source, side by side; the objects live in a folder of their own
    with tempfile.TemporaryDirectory() as tmp:
        objs = [os.path.join(tmp, os.path.splitext(s)[0] + ".o") for s in SOURCES]
        jobs = [[hipcc] + flags + ["-x", "hip", "-c", os.path.join(CSRC, s), "-o", o]
                for s, o in zip(SOURCES, objs)]
        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(run, jobs))
        run([hipcc, "-shared", "-fPIC", f"--offload-arch={ARCH}"] + objs + ["-o", out + ".tmp"])
    os.replace(out + ".tmp", out)
    return out


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
    print(LIB)
