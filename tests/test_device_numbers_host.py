"""What a launch asks the runtime once for each device: a question that failed is asked again."""

import os
import subprocess

import padding_free_packed_gb300.build as build

PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include "pe_common.cuh"

int main() {
  static pe::DeviceNumber known;
  int asked = 0, answer = 0;
  auto ask = [&] { ++asked; return answer; };
  auto expect = [&](int device, int number, int times) {
    const int got = known.of(device, ask);
    if (got != number || asked != times) {
      std::printf("device %d: %d after %d questions, not %d after %d\\n", device, got, asked,
                  number, times);
      std::exit(1);
    }
  };
  expect(0, 0, 1);        // failed
  expect(0, 0, 2);        // and again
  answer = 3;
  expect(0, 3, 3);
  answer = 5;
  expect(0, 3, 3);        // known
  expect(1, 5, 4);        // of each device by itself
  answer = 0;
  expect(1, 5, 4);
  expect(63, 0, 5);
  answer = 7;
  expect(64, 7, 6);       // past those that are remembered: asked every time
  expect(64, 7, 7);
  expect(-1, 7, 8);
  return 0;
}
"""


def test_only_answers_are_remembered(tmp_path):
    source, program = tmp_path / "numbers.cu", tmp_path / "numbers"
    source.write_text(PROGRAM)
    subprocess.run([build._nvcc(), "-std=c++17", "-I", build.CSRC, "-I", build.INCLUDE, str(source),
                    "-o", str(program)], check=True)
    done = subprocess.run([str(program)], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout


def test_no_launch_keeps_its_first_answer_for_good():
    for name in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, name)) as fh:
            for number, line in enumerate(fh, 1):
                assert not line.lstrip().startswith("static const int "), f"{name}:{number}"
