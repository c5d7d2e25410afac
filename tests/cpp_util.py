"""Compile and run a small C++ program against the library's plain C++ headers."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tma_pipelined_tensor_fp16_gb300", "csrc")


def run_cpp(tmp_path, source):
    """The output of `source`, compiled with g++ as C++17."""
    src, exe = tmp_path / "program.cpp", tmp_path / "program"
    src.write_text(source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-pthread", "-I", CSRC, str(src), "-o",
                    str(exe)], check=True, capture_output=True, text=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
