"""Which kernels a grouped product's call launches: the library's own rule
(``csrc/grouped_plan.h``), compiled for the host."""
import os
import subprocess

from mixture_experts_layer_exclusive_amd import build as B

PROGRAM = r"""
#include "grouped_plan.h"
#include <cstdio>
#include <cstring>
using namespace moe;
// a line per problem: op type rows E N K -> every launch as mode:variant:parts:tiles
int main() {
    char op[16], type[8];
    long rows;
    int E, N, K;
    while (scanf("%15s %7s %ld %d %d %d", op, type, &rows, &E, &N, &K) == 6) {
        const moe_grouped_t g{rows, E, N, K, strcmp(type, "f32") ? MOE_DTYPE_BF16 : MOE_DTYPE_F32};
        auto show = [&](const char* mode, const Plan& p) {
            printf("%s:%d:%d:%ld ", mode, static_cast<int>(p.v), p.parts, static_cast<long>(p.tiles));
        };
        if (!strcmp(op, "backward")) {
            const Plan pa = plan_for(g, kNN, false), pw = plan_for(g, kTN, false);
            if (pairs(g, pa, pw)) printf("joint ");
            show("NN", pa);
            show("TN", pw);
        } else {
            show("NT", plan_for(g, kNT, !strcmp(op, "int8")));
        }
        printf("\n");
    }
}
"""
NAMES = ["split32", "split64", "tile64", "tile64x128", "tile128", "tile256"]


def build(folder):
    """The program's path; host code only, nothing is compiled for a device."""
    src, exe = os.path.join(folder, "choice.hip"), os.path.join(folder, "choice")
    with open(src, "w") as f:
        f.write(PROGRAM)
    r = subprocess.run([B.hipcc(), "--cuda-host-only", "-O1", "-std=c++17", f"-I{B.INCLUDE}", f"-I{B.CSRC}", src, "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return exe


def kernels(exe, problems):
    """For every (op, type, rows, E, N, K) the list of its launches, each a
    tuple (mode, variant, parts, tiles); the gradients of a joint launch come
    as one tuple ("joint", variant of da, variant of dw, parts, tiles of da)."""
    text = "".join("%s %s %d %d %d %d\n" % p for p in problems)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=120).stdout
    res = []
    for line in out.splitlines():
        words = line.split()
        joint = words[0] == "joint"
        runs = [w.split(":") for w in words[joint:]]
        runs = [(m, NAMES[int(v)], int(p), int(t)) for m, v, p, t in runs]
        if joint:
            (_, va, _, ta), (_, vw, parts, _) = runs
            res.append([("joint", va, vw, parts, ta)])
        else:
            res.append(runs)
    assert len(res) == len(problems)
    return res
