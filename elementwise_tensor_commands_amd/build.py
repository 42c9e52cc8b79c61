"""Build libecmd.so (the C ABI and its gfx950 kernels) and, where torch is
installed, _binding.*.so (the compiled part of the Python binding, for the
interpreter that runs this) in-tree.

    python elementwise_tensor_commands_amd/build.py [-v]

(run it as a script: importing the package would load the library first).

Every source is compiled for gfx950 only, non-relocatable device code (each
kernel's device code lives in its own translation unit, as clang's HIP support
document describes for the default -fno-gpu-rdc mode), with:
  -ffp-contract=off     every binary32 operation rounds on its own;
  -Xclang -target-feature -Xclang -packed-fp32-ops
                        no packed binary32 instructions;
  -mllvm -simplifycfg-sink-common=false
                        keeps the interpreter's register-slot switches from
                        being merged into one runtime-indexed (scratch) access.
Denormals are left at the default (kept; no -fgpu-flush-denormals-to-zero).

The device headers the run-time compiler uses (JIT_HEADERS) are embedded into
the library as text, with the same device flags (JIT_OPTIONS), by a generated
translation unit (_build/ecmd_jit_sources.cpp); libhiprtc is linked.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libecmd.so")
# with the interpreter's tag: another one, whose objects may differ, does not load it
BINDING = os.path.join(PKG, "_binding" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

SOURCES = ["ecmd_host.cpp", "ecmd_serial.cpp", "ecmd_jit.cpp", "kernels_linear.hip", "kernels_interp.hip",
           "kernels_tiled.hip", "kernels_rows.hip", "kernels_gather.hip", "serving/ecmd_serving.cpp",
           "serving/kernels_rope.hip", "serving/kernels_attention_f16.hip", "serving/kernels_attention_bf16.hip",
           "serving/kernels_attention_f32.hip", "serving/kernels_pages.hip", "serving/ecmd_serving_cache.cpp",
           "serving/kernels_tree_f16.hip", "serving/kernels_tree_bf16.hip", "serving/kernels_tree_f32.hip",
           "serving/kernels_tree_join.hip", "serving/kernels_accept.hip", "serving/kernels_select.hip",
           "serving/kernels_mass_f16.hip", "serving/kernels_mass_bf16.hip", "serving/kernels_mass_f32.hip"]
# Device headers the run-time compiler needs: embedded into the library as text.
JIT_HEADERS = ["ecmd_tape.h", "ecmd_eval.h", "ecmd_kern_linear.h", "ecmd_kern_rows.h", "ecmd_kern_tiled.h",
               "ecmd_kern_gather.h"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = [
    "--offload-arch=" + ARCH, "-O3", "-std=c++20", "-fPIC", "-ffp-contract=off", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-mllvm", "-simplifycfg-sink-common=false",
    "-Wall", "-Wno-unused-function", "-I", os.path.join(ROOT, "include"),
]

# Further flags of single sources.  Attention: matrix results in the general
# registers; with the accumulation registers, which the compiler otherwise gives
# half of the file, the loop moved 32 values there and back in every turn.
FILE_FLAGS = {"serving/kernels_%s_%s.hip" % (k, t): ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]
              for k in ("attention", "tree", "mass") for t in ("f16", "bf16", "f32")}

# Options for run-time compilation: the device side of FLAGS.
JIT_OPTIONS = ["--offload-arch=" + ARCH, "-O3", "-std=c++20", "-ffp-contract=off", "-fno-fast-math",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-mllvm", "-simplifycfg-sink-common=false"]


def _c_string(text: str) -> str:
    return "R\"ECMDSRC(" + text + ")ECMDSRC\""


def write_jit_sources(path: str) -> str:
    """Generate the translation unit that embeds the device headers and the
    run-time compile options; their hash keys the compiled-kernel cache."""
    import hashlib
    h = hashlib.sha256()
    texts = []
    for name in JIT_HEADERS:
        with open(os.path.join(CSRC, name)) as f:
            t = f.read()
        assert ")ECMDSRC" not in t
        texts.append(t)
        h.update(name.encode() + b"\0" + t.encode() + b"\0")
    for o in JIT_OPTIONS:
        h.update(o.encode() + b"\0")
    lines = ["// Generated by build.py from the device headers; do not edit.",
             "namespace ecmd {",
             "extern const int kJitHeaderCount = %d;" % len(JIT_HEADERS),
             "extern const char *const kJitHeaderNames[] = {%s};" % ", ".join('"%s"' % n for n in JIT_HEADERS),
             "extern const char *const kJitHeaderTexts[] = {"]
    lines += ["    %s," % _c_string(t) for t in texts]
    lines += ["};",
              "extern const int kJitOptionCount = %d;" % len(JIT_OPTIONS),
              "extern const char *const kJitOptions[] = {%s};" % ", ".join('"%s"' % o for o in JIT_OPTIONS),
              'extern const char *const kJitSourcesHash = "%s";' % h.hexdigest()[:16],
              "}  // namespace ecmd", ""]
    text = "\n".join(lines)
    if not os.path.exists(path) or open(path).read() != text:
        with open(path, "w") as f:
            f.write(text)
    return path


def _run_all(cmds):
    procs = [(c, subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)) for c in cmds]
    errors = []
    for c, p in procs:
        out = p.communicate()[0].decode(errors="replace")
        # hipcc's host pass does not know the packed-fp32 target feature; that warning is noise.
        lines = [l for l in out.splitlines()
                 if l.strip() and "packed-fp32-ops" not in l and "'--hip-link'" not in l]
        if p.returncode != 0:
            errors.append("$ %s\n%s" % (" ".join(c), "\n".join(lines)))
        elif lines:
            sys.stderr.write("\n".join(lines) + "\n")
    if errors:
        raise RuntimeError("hipcc failed:\n" + "\n\n".join(errors))


def binding_command(out: str):
    """The command that builds the Python extension module _binding: host code
    against torch's and Python's headers, with the host compiler.  None where there
    is no torch: the C library does without."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    torch = os.path.dirname(spec.origin)
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(HIPCC)))
    inc = [sysconfig.get_paths()["include"], os.path.join(torch, "include"),
           os.path.join(torch, "include", "torch", "csrc", "api", "include"), os.path.join(rocm, "include")]
    lib = os.path.join(torch, "lib")
    return [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
            "-DUSE_ROCM=1", *[x for i in inc for x in ("-isystem", i)], os.path.join(CSRC, "ecmd_binding.cpp"), "-o", out,
            "-L" + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip", "-Wl,-rpath," + lib]


def build(asm: bool = True, verbose: bool = False) -> str:
    """Compile every source and link libecmd.so next to this file.  With asm,
    also write each kernel file's gfx950 assembly to _build/<name>.s (used by the
    tests that inspect the generated code)."""
    os.makedirs(BUILD, exist_ok=True)
    objs, cmds = [], []
    gen = write_jit_sources(os.path.join(BUILD, "ecmd_jit_sources.cpp"))
    for src in SOURCES + [gen]:
        path = src if os.path.isabs(src) else os.path.join(CSRC, src)
        obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
        objs.append(obj)
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        extra = FILE_FLAGS.get(src, [])
        cmds.append([HIPCC, *FLAGS, *extra, *lang, "-c", path, "-o", obj])
        if asm and src.endswith(".hip"):
            cmds.append([HIPCC, *FLAGS, *extra, "-x", "hip", "--offload-device-only", "-S",
                         os.path.join(CSRC, src), "-o", os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".s")])
    tmp_binding = BINDING + ".tmp%d" % os.getpid()
    binding = binding_command(tmp_binding)
    if binding:
        cmds.append(binding)
    else:
        sys.stderr.write("no torch: the library is built without the Python binding of the serving operators\n")
    if verbose:
        for c in cmds:
            print(" ".join(c))
    _run_all(cmds)
    tmp = LIB + ".tmp%d" % os.getpid()
    rocm_lib = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(HIPCC))), "lib")
    _run_all([[HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp, *objs,
               "-L" + rocm_lib, "-lhiprtc", "-Wl,-rpath," + rocm_lib]])
    os.replace(tmp, LIB)
    if binding:
        os.replace(tmp_binding, BINDING)
        untagged = os.path.join(PKG, "_binding.so")   # of earlier builds: any interpreter would load it
        if untagged != BINDING and os.path.exists(untagged):
            os.remove(untagged)
    return LIB


if __name__ == "__main__":
    print(build(asm=True, verbose="-v" in sys.argv))
