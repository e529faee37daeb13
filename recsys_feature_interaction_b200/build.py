"""Builds libwukong.so (the C ABI of include/wukong.h) for sm_100a, in-tree.

nvcc -gencode arch=compute_100a,code=sm_100a -O3 -lineinfo, static CUDA runtime,
so the library loads (and exports its symbols) on a machine without a GPU and
uses the caller's CUDA context when there is one.
"""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "_lib", "libwukong.so")
COMMON = ["common.cuh", "host.cuh"]
# each source and the headers it is compiled from
SOURCES = {
    "wk_api.cu": COMMON + ["gemm_tc.cuh", "gemm_tc2.cuh", "lcb_tc.cuh", "fm_tc.cuh", "front_tc.cuh", "res_ln.cuh",
                           "res_ln_ring.cuh", "simt.cuh", "convert.cuh", "moe.cuh", "head.cuh", "whale.cuh",
                           "backward.cuh", "bw_tc.cuh"],
    "wk_seq.cu": COMMON + ["seq_index.h", "seq_args.cuh", "seq_back.cuh", "seq_cache.cuh", "seq_rows.cuh", "seq_tile.cuh",
                           "whale.cuh"],
}


def _object(source):
    return os.path.join(HERE, "_lib", source.replace(".cu", ".o"))


def _older(target, source):
    """Whether `target` is missing, older than the source, its headers or the public header, or made with other
    flags than today's."""
    if not os.path.exists(target) or _flags_changed(source):
        return True
    t = os.path.getmtime(target)
    deps = [os.path.join(CSRC, f) for f in [source] + SOURCES[source]] + [os.path.join(INCLUDE, "wukong.h")]
    return any(os.path.getmtime(p) > t for p in deps)


def _flag_line():
    """The flags as a line; without the include paths, which go by where the tree lies."""
    return "flags: " + " ".join(f for f in nvcc_flags() if not f.startswith("-I"))


def _flags_changed(source):
    """Whether the log of the source's object, which begins with its flags, names others."""
    try:
        with open(_object(source) + ".log") as log:
            return log.readline().rstrip("\n") != _flag_line()
    except FileNotFoundError:
        return False


def _stale():
    return any(_older(LIB, s) for s in SOURCES)


def nvcc_flags():
    return ["-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
            "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "-cudart", "static",
            "-I" + INCLUDE, "-I" + CSRC, "--expt-relaxed-constexpr", "-Xptxas", "-v"]


def build(force=False, verbose=False):
    """Compiles the sources that changed side by side, one object each, and links them."""
    if not force and not _stale():
        return LIB
    libdir = os.path.dirname(LIB)
    os.makedirs(libdir, exist_ok=True)
    running = []
    for s in SOURCES:
        if force or _older(_object(s), s):
            with open(_object(s) + ".log", "w") as log:
                log.write(_flag_line() + "\n")
                log.flush()
                cmd = ["nvcc", "-c"] + nvcc_flags() + ["-o", _object(s), os.path.join(CSRC, s)]
                running.append((s, subprocess.Popen(cmd, stdout=log, stderr=subprocess.STDOUT)))
    failed = [s for s, p in running if p.wait() != 0]
    logs = "".join(open(_object(s) + ".log").read() for s in (failed or SOURCES) if os.path.exists(_object(s) + ".log"))
    if failed:
        for s in failed:
            if os.path.exists(_object(s)):
                os.remove(_object(s))
        raise RuntimeError("nvcc failed:\n" + logs)
    r = subprocess.run(["nvcc", "-shared"] + nvcc_flags() + ["-o", LIB] + [_object(s) for s in SOURCES],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + r.stdout + r.stderr)
    with open(os.path.join(libdir, "ptxas.log"), "w") as f:
        f.write(logs)
    if verbose:
        print(logs)
    return LIB


def main():
    """python -m recsys_feature_interaction_b200.build: compiles everything anew."""
    print(build(force=True))


if __name__ == "__main__":
    main()
