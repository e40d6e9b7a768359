"""Build step for libbole.so: compiles the HIP sources in csrc/ for gfx950 with hipcc
and links them into a shared library next to this file (in-tree, so it ships with the
repository snapshot). Also builds libbole_probe.so, the benchmark's memory-only reference
kernels (not part of the library)."""
import concurrent.futures
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build", "bole")
LIB = os.path.join(HERE, "libbole.so")
PROBE_LIB = os.path.join(HERE, "libbole_probe.so")
PROBE_SOURCES = ["pattern_probe.hip"]
SOURCES = ["bole_api.hip", "topology.hip", "validate.hip", "verify_generic.hip", "verify_mfma.hip", "verify_vec.hip",
           "verify_naive.hip", "commit.hip", "tree_build.hip",
           "tree_accept.hip", "delta_api.hip", "delta_walk.hip", "delta_verify.hip",
           "delta_prefill.hip", "window_api.hip", "window_attention.hip",
           "window_mfma.hip", "window_mfma_f32.hip", "linear_api.hip", "linear_walk.hip",
           "linear_prefill.hip", "rotary.hip", "append.hip", "prefix_attention.hip", "prefix_mfma.hip"]
ARCH = "gfx950"

# Packed-fp32 instructions stay off: the compiler would otherwise form them from
# ordinary float code.
CFLAGS = ["-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC", "-Wall", "-fvisibility=hidden",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def hipcc() -> str:
    exe = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    return exe


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *CFLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    msgs = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                     if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{msgs}")
    if verbose and msgs.strip():
        print(msgs, flush=True)
    return obj


def _link(objs, lib: str, verbose: bool) -> None:
    tmp = lib + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp,
           "-Wl,-rpath,/opt/rocm/lib"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True, capture_output=not verbose)
    os.replace(tmp, lib)


def build(verbose: bool = False) -> str:
    """Compile every HIP source and link libbole.so and libbole_probe.so; returns the
    path of libbole.so."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = SOURCES + PROBE_SOURCES
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = dict(zip(srcs, ex.map(lambda s: _compile(s, verbose), srcs)))
    _link([objs[s] for s in SOURCES], LIB, verbose)
    _link([objs[s] for s in PROBE_SOURCES], PROBE_LIB, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
