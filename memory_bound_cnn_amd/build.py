"""Build libwtconv.so (HIP kernels + C ABI) for gfx950, in place.

    python -m memory_bound_cnn_amd.build

Every HIP source is compiled with packed-FP32 instructions disabled; the
objects are linked into memory_bound_cnn_amd/libwtconv.so.  The PyTorch module
of the token operators, host code alone, is linked to it as _tokens.so; it is
left out where there is no PyTorch for ROCm, which the library does not need.
"""
import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libwtconv.so")
TORCH_OUT = os.path.join(HERE, "_tokens.so")
OBJDIR = os.path.join(HERE, "_build")
ARCH = os.environ.get("WTC_OFFLOAD_ARCH", "gfx950")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX") or ("g++" if shutil.which("g++") else os.path.join(os.path.dirname(HIPCC), "amdclang++"))

COMMON = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-variable", "-Wno-unused-function", "-Wno-uninitialized",
    "-Wno-unknown-warning-option", "-Wno-sometimes-uninitialized",
]

SOURCES = ["wtconv_fused.hip", "wtconv_fused_k1.hip", "wtconv_fused_k3.hip", "wtconv_fused_k5.hip",
           "wtconv_fused_k7.hip", "wtconv_fused_s_p64.hip", "wtconv_fused_s_p32.hip",
           "wtconv_fused_s_p128a.hip", "wtconv_fused_s_p128b.hip", "wtconv_fused_s_small.hip", "wtconv_fused_s_p112.hip",
           "wtconv_fused_s_dw.hip",
           "wtconv_tiny.hip", "wtconv_lane.hip", "wtconv_unfused.hip", "wtconv_top.hip", "wtconv_layout.hip", "wtconv_noalloc.hip", "wtconv_corr.hip", "wtconv_api.cpp", "wtconv_plan.cpp",
           "wtconv_tok_rms.hip", "wtconv_tok_rotary.hip", "wtconv_tok_dropout.hip", "wtconv_tok_attn.hip",
           "wtconv_tok_attn_bf16.hip", "wtconv_tok_attn_fp32.hip", "wtconv_tok_layer.hip", "wtconv_tok_scan.hip",
           "wtconv_tok_expert.hip", "wtconv_tok_product.hip", "wtconv_tok_product_bf16.hip", "wtconv_tok_product_fp32.hip",
           "wtconv_tok_api.cpp"]


def _compile(src):
    obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
    cmd = [HIPCC] + COMMON + ["-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _compile_torch():
    """The object file of the PyTorch module and what it is linked with; None
    without a PyTorch for ROCm."""
    try:
        import torch
    except ImportError:
        return None
    if torch.version.hip is None:
        return None
    base = os.path.dirname(torch.__file__)
    obj = os.path.join(OBJDIR, "wtconv_tok_torch.cpp.o")
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "include")]
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           "-DTORCH_EXTENSION_NAME=_tokens", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += ["-I" + d for d in inc] + ["-c", os.path.join(CSRC, "wtconv_tok_torch.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed for wtconv_tok_torch.cpp:\n{r.stdout}\n{r.stderr}")
    return obj, ["-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip"]


def _link(cmd, out):
    r = subprocess.run(cmd + ["-o", out + ".tmp"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(out + ".tmp", out)


def build(verbose=False):
    os.makedirs(OBJDIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        torch_part = ex.submit(_compile_torch)
        results = list(ex.map(_compile, SOURCES))
    objs = [o for o, _ in results]
    if verbose:
        for _, err in results:
            if err.strip():
                print(err, file=sys.stderr)
    _link([HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}"] + objs, OUT)
    if torch_part.result() is None:
        print("no PyTorch for ROCm here: _tokens.so (the token operators' PyTorch module) is not built", file=sys.stderr)
        return OUT
    obj, libs = torch_part.result()
    _link([CXX, "-shared", "-fPIC", obj, "-L" + HERE, "-l:" + os.path.basename(OUT), "-Wl,-rpath,$ORIGIN"] + libs,
          TORCH_OUT)
    return OUT


if __name__ == "__main__":
    print(build(verbose=True))
