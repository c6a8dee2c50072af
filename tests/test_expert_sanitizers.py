"""The argument checks of the experts' operators under AddressSanitizer and UndefinedBehaviorSanitizer (host code only),
on boundary values (tests/native/experts_validate.cpp)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_checks_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "experts_validate")
    subprocess.run(["g++", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1",
                    "-std=c++17", "-Wall", "-Werror", os.path.join(ROOT, "tests", "native", "experts_validate.cpp"), "-o", exe],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    print(r.stdout[-2000:], r.stderr[-4000:])
    assert r.returncode == 0
