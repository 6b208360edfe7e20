"""Which kernels a call launches, by the profiler's record of them: a test that is
meant for one kernel says so, and fails when a call's sizes come to choose another."""
import re

import torch

_ARGS = {"DF16b": "bf16", "f": "f32", "float": "f32", "true": "1", "false": "0"}


def _plain(name):
    """A name as the source has it: from the mangled form, or, where the profiler
    knows all its types, the C++ one."""
    m = re.match(r"_ZN3spc12_GLOBAL__N_1(\d+)(\w+)", name)
    if m:
        name, rest = m[2][:int(m[1])], m[2][int(m[1]):]
        m = re.match(r"I((?:DF16b|f|L[a-z]\d+E)+)E", rest)
        args = re.findall(r"DF16b|L[a-z]\d+E|f", m[1]) if m else []
        args = [a[2:-1] if a[0] == "L" else a for a in args]
    else:
        m = re.match(r"(?:void )?spc::\(anonymous namespace\)::(\w+)(?:<([^>]*)>)?", name)
        if not m:
            return None
        name, args = m[1], m[2].split(", ") if m[2] else []
    return name + ("<" + ", ".join(_ARGS.get(a, a) for a in args) + ">" if args else "")


def launched(call):
    """Names of this library's kernels that call() launches, such as "k_attn<bf16, 64>";
    template arguments that are truth values are 0 and 1."""
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        call()
        torch.cuda.synchronize()
    return {_plain(e.name) for e in prof.events()} - {None}


def assert_launches(call, *want):
    """call() launches each of the named kernels (once under the profiler's eyes)."""
    names = launched(call)
    for w in want:
        assert w in names, f"meant for {w}, launched {sorted(names)}"
