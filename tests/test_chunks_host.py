"""CPU test of the chunks that long vocabulary rows are streamed in."""
import os
import re
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "response_replay_gb300", "csrc")


def test_chunks_fit_and_cover_the_row(tmp_path):
    exe = tmp_path / "chunk_check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC,
                    os.path.join(HERE, "chunk_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "chunks ok" in r.stdout


def test_the_kernel_streams_these_chunks():
    with open(os.path.join(CSRC, "token_logp.cu")) as f:
        src = f.read()
    loads = re.findall(r"bulk_load\(ring0[^;]*;", src)
    assert len(loads) == 1 and re.search(r"\bbytes\b", loads[0])
    assert "bytes = ls_chunk_bytes<kGroupBytes, kThreads>(" in src
