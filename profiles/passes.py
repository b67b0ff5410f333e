"""Passes of one case of perf/operators.py through the library, for a profiler: passes.py CASE[,CASE] COUNT.
Inputs are made once and the case is run COUNT times; run from anywhere."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "perf")]

import torch  # noqa: E402

import operators  # noqa: E402


def main():
    names, count = sys.argv[1].split(","), int(sys.argv[2])
    operators.own = True
    for case in operators.listed():
        if case["name"] in names:
            state = operators.prepare(case, 3)
            torch.cuda.synchronize()
            for _ in range(count):
                operators.run(state)
            torch.cuda.synchronize()
            print(case["name"], flush=True)


if __name__ == "__main__":
    main()
