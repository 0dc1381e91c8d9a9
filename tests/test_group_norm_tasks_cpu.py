"""The order of the tasks in group norm's stream, compiled for the host: every task once, and behind all that it waits for
(blocks take tasks in their order, so that order is what keeps a resident grid from waiting for itself)."""
import os
import subprocess

import pytest

from conv_batchnorm_relu_gb300 import build

MAIN = """
#include <cstdio>
#include <cstdlib>
#include "group_norm_tasks.h"
using namespace cbr::gn;
int main(int argc, char** argv) {
  for (int k = 1; k + 2 < argc; k += 3) {
    const uint32_t images = atoi(argv[k]), runs = atoi(argv[k + 1]), lag = atoi(argv[k + 2]), n = Task::total(images, runs);
    const Order order{images, runs, (lag + 1) / 2, lag};
    for (uint32_t i = 0; i < n; ++i) {
      const Task t = Task::of(order, i);
      printf("%d %u %u ", (int)t.kind, t.image, t.run);
    }
    printf("\\n");
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    folder = tmp_path_factory.mktemp("tasks")
    (folder / "main.cpp").write_text(MAIN)
    exe = str(folder / "tasks")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", build.CSRC, str(folder / "main.cpp"), "-o", exe], check=True)
    return exe


def test_the_kernel_takes_its_tasks_from_there():
    text = open(os.path.join(build.CSRC, "group_norm.cu")).read()
    assert '#include "group_norm_tasks.h"' in text and "Task::of(f.order, i)" in text and "struct Task" not in text


@pytest.mark.parametrize("images", [1, 2, 3, 5, 17, 40, 128])
def test_every_task_once_and_behind_what_it_waits_for(program, images):
    """(128 images in 17 runs with a lag of 10 are what a forward over 112x112x128 maps of 16 bits has.)"""
    orders = [(images, runs, lag) for runs in (1, 2, 3, 17, 33) for lag in sorted({1, 2, 3, 4, 9, 10, images - 1, images}) if 1 <= lag <= images]
    lines = subprocess.run([program, *(str(v) for o in orders for v in o)], check=True, capture_output=True, text=True).stdout.splitlines()
    assert len(lines) == len(orders)
    for (_, runs, lag), line in zip(orders, lines):
        v = list(map(int, line.split()))
        tasks = list(zip(v[::3], v[1::3], v[2::3]))
        place = {t: i for i, t in enumerate(tasks)}
        assert len(tasks) == len(place) == images * (2 * runs + 1)
        for image in range(images):
            merge = place[(1, image, 0)]
            assert all(place[(0, image, r)] < merge < place[(2, image, r)] for r in range(runs)), (runs, lag, image)
