"""Build the HIP library libgc.so (gfx950 only) next to this file, and the same library at
other tile geometries (libgc_<name>.so, see VARIANTS) for the tests that check that no result
depends on the geometry.

Flags that the results depend on:
  -ffp-contract=off                  no fused multiply-add: u = fl(fl(m*u) + g)
  -fno-gpu-flush-denormals-to-zero   fp32 denormals are kept
  -fhip-fp32-correctly-rounded-divide-sqrt   |v| / scale is correctly rounded
  -target-feature -packed-fp32-ops   no packed fp32 instructions
"""
from __future__ import annotations

import os
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libgc.so")
# The compressors, whose kernels follow the tile geometry, and the activation operators and those over
# many tensors, whose kernels do not (every library holds all).
TILED = [os.path.join(HERE, "csrc", f) for f in ("gc_pass.hip", "gc_topk.hip", "gc_codecs.hip",
                                                     "gc_scatter.hip", "gc_api.hip")]
ACTIVATION = [os.path.join(HERE, "csrc", f) for f in ("gc_act.hip", "gc_norm.hip", "gc_wgrad.hip",
                                                          "gc_gated.hip", "gc_act_api.hip",
                                                          "gc_grads.hip", "gc_grads_api.hip")]
SOURCES = TILED + ACTIVATION
ARCH = "gfx950"

# Tile geometries besides the default (1024 threads x 2 slots, 8192-element tiles).  A tile is
# threads * 4 * slots elements; a different geometry moves every tile, chunk and run boundary,
# the cold-start sample and the order of the per-tile partial sums.
VARIANTS = {
    "t512s4": ("GC_TILE_THREADS=512", "GC_TILE_SLOTS=4"),    # 8192 elements, 8 waves
    "t1024s1": ("GC_TILE_THREADS=1024", "GC_TILE_SLOTS=1"),  # 4096 elements, 16 waves
    "t256s2": ("GC_TILE_THREADS=256", "GC_TILE_SLOTS=2"),    # 2048 elements, 4 waves
}


def variant_path(name: str) -> str:
    if name not in VARIANTS:
        raise KeyError(f"unknown tile geometry {name!r}; built ones: {sorted(VARIANTS)}")
    return os.path.join(HERE, f"libgc_{name}.so")


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def flags() -> list[str]:
    return [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
            "-ffp-contract=off", "-fno-gpu-flush-denormals-to-zero",
            "-fhip-fp32-correctly-rounded-divide-sqrt",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wall", "-Wno-unused-result", "-I", os.path.join(ROOT, "include"),
            "-I", os.path.join(HERE, "csrc")]


def _run(cmd, verbose: bool):
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in (res.stdout + res.stderr).splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    if verbose and err.strip():
        print(err)


def _build(jobs, verbose: bool) -> list[str]:
    """Compile each library's sources side by side, then link it; ``jobs`` lists (output,
    defines).  The activation sources are compiled once for all of them."""
    compile_flags = [f for f in flags() if f != "-shared"]
    with tempfile.TemporaryDirectory() as tmp, \
            ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 1)) as ex:
        def compiled(src, tag, defines):
            obj = os.path.join(tmp, f"{os.path.basename(src)}.{tag}.o")
            cmd = [hipcc(), *compile_flags, *[f"-D{d}" for d in defines], "-c", src, "-o", obj]
            return obj, ex.submit(_run, cmd, verbose)

        tiled = [[compiled(src, i, defines) for src in TILED]
                 for i, (_, defines) in enumerate(jobs)]
        shared = [compiled(src, "act", ()) for src in ACTIVATION]

        def link(out, objs):
            for _, fut in objs:
                fut.result()
            new = out + f".tmp{os.getpid()}"
            _run([hipcc(), *flags(), *[o for o, _ in objs], "-o", new], verbose)
            os.replace(new, out)
            return out

        return [link(out, objs + shared) for (out, _), objs in zip(jobs, tiled)]


def build(verbose: bool = False, out: str = LIB, defines=()) -> str:
    """Compile libgc.so; ``defines`` (e.g. "GC_TILE_SLOTS=4") override the compile-time
    configuration of the streaming pass."""
    return _build([(out, defines)], verbose)[0]


def build_all(verbose: bool = False) -> list[str]:
    """libgc.so and every VARIANTS geometry."""
    return _build([(LIB, ())] + [(variant_path(n), d) for n, d in VARIANTS.items()], verbose)


if __name__ == "__main__":
    print("\n".join(build_all(verbose=True)))
