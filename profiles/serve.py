"""Runs cases of perf/operators.py by the library, for a profiler to watch:
`python3 profiles/serve.py NAME ...` from the repository's root takes each named
case 40 times, on three sets of inputs in turn.  Without names, all cases."""

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "perf")]
import torch  # noqa: E402

import operators  # noqa: E402

operators.own = True
names = sys.argv[1:]
for case in operators.listed():
    if not names or case["name"] in names:
        states = [operators.prepare(case, seed) for seed in range(3)]
        for i in range(40):
            operators.run(states[i % 3])
        torch.cuda.synchronize()
        print("ran", case["name"], flush=True)
