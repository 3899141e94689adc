"""Compiles a small host program against the library's plain C++ headers and runs it
(no test functions here)."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_263_gb300", "csrc")


def run_host(tmp_path, source, *args, given=""):
    src, exe = tmp_path / "host.cpp", tmp_path / "host"
    src.write_text(source)
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe), *map(str, args)], input=given, capture_output=True, text=True, check=True).stdout
