"""Runs cases of the latent-attention operators (the cache, the absorbed and the expanded
form, the gradients), for a profiler:

    python3 deepseekmoe_routing_fp8_amd/bench/latent_cases.py NAME[,NAME...] [CALLS]

NAME is a case of perf/operators.py; the inputs are seeded."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.dirname(os.path.abspath(__file__)))))

import torch  # noqa: E402

from perf import operators  # noqa: E402


def main():
    operators.own = True
    cases = {c["name"]: c for c in operators.listed()}
    for name in sys.argv[1].split(","):
        state = operators.prepare(cases[name], 1)
        for _ in range(int(sys.argv[2]) if len(sys.argv) > 2 else 6):
            operators.run(state)
        torch.cuda.synchronize()
        print(name, flush=True)


if __name__ == "__main__":
    main()
